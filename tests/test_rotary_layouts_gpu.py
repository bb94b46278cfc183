"""Rotary positions on two-map tensors [B, S, H, 2, D] whose head and map axes are
not one run of heads: projections that keep the maps apart, and the gradients that
a consumer's own layout hands back."""
import pytest
import torch

from exact_io_aware_96_b200 import fa
from exact_io_aware_96_b200.autograd import diff_attn_func, rotary_func

pytestmark = pytest.mark.gpu
SECTIONS = (3, 2, 3)


def setup(B=2, S=37, H=4, Hk=2, D=24, dtype=torch.bfloat16):
    g = torch.Generator("cuda").manual_seed(5)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(dtype)  # noqa: E731
    pos = torch.randint(0, 500, (3, B, S), generator=g, device="cuda", dtype=torch.int32)
    return rnd(B, S, 2, H, D), rnd(B, S, 2, Hk, D), pos, fa.rotary_inv_freq(SECTIONS)


def dense(t):
    return t.clone(memory_format=torch.contiguous_format)


@pytest.mark.parametrize("inter", [False, True])
def test_map_major_views(fa_lib, inter):
    """A projection viewed as [B, S, 2, H, D], its maps last but one by transpose; also as the output, in place."""
    xq, xk, pos, f = setup()
    q, k = xq.transpose(2, 3), xk.transpose(2, 3)
    wq, wk = fa.rotary(dense(q), dense(k), pos, f, SECTIONS, interleaved=inter)
    gq, gk = fa.rotary(q, k, pos, f, SECTIONS, interleaved=inter)
    assert torch.equal(gq, wq) and torch.equal(gk, wk)
    # only one of the two is map-major; q alone
    gq, gk = fa.rotary(dense(q), k, pos, f, SECTIONS, interleaved=inter)
    assert torch.equal(gq, wq) and torch.equal(gk, wk)
    gq, gk = fa.rotary(q, dense(k), pos, f, SECTIONS, interleaved=inter)
    assert torch.equal(gq, wq) and torch.equal(gk, wk)
    gq, none = fa.rotary(q, None, pos, f, SECTIONS, interleaved=inter)
    assert torch.equal(gq, wq) and none is None
    # dense inputs into map-major outputs, then in place
    oq, ok = torch.full_like(xq, float("nan")), torch.full_like(xk, float("nan"))
    fa.rotary(dense(q), dense(k), pos, f, SECTIONS, interleaved=inter, out_q=oq.transpose(2, 3), out_k=ok.transpose(2, 3))
    assert torch.equal(oq.transpose(2, 3), wq) and torch.equal(ok.transpose(2, 3), wk)
    fa.rotary(q, k, pos, f, SECTIONS, interleaved=inter, out_q=q, out_k=k)
    assert torch.equal(q, wq) and torch.equal(k, wk)
    assert fa.fa_last_device_status()[0] == 0


def test_gradient_of_a_map_major_projection(fa_lib):
    xq, xk, pos, f = setup()
    xq.requires_grad_()
    xk.requires_grad_()
    oq, ok = rotary_func(xq.transpose(2, 3), xk.transpose(2, 3), pos, f, SECTIONS)
    gq, gk = torch.randn_like(oq), torch.randn_like(ok)
    dq, dk = torch.autograd.grad((oq, ok), (xq, xk), (gq, gk))
    wq, wk = fa.rotary(gq, gk, pos, f, SECTIONS, inverse=True)
    assert torch.equal(dq, wq.transpose(2, 3)) and torch.equal(dk, wk.transpose(2, 3))


@pytest.mark.parametrize("order", [(0, 1, 3, 2, 4), (0, 3, 2, 1, 4)], ids=["map-head", "map-head-row"])
def test_consumers_that_reorder_the_output(fa_lib, order):
    """The output's gradient comes back in the layout of what the consumer made of it."""
    xq, xk, pos, f = setup()
    q, k = dense(xq.transpose(2, 3)).requires_grad_(), dense(xk.transpose(2, 3)).requires_grad_()
    oq, ok = rotary_func(q, k, pos, f, SECTIONS)
    cq, ck = oq.permute(order).contiguous(), ok.permute(order).contiguous()
    gq, gk = torch.randn_like(cq), torch.randn_like(ck)
    dq, dk = torch.autograd.grad((cq, ck), (q, k), (gq, gk))
    back = [order.index(i) for i in range(5)]
    wq, wk = fa.rotary(dense(gq.permute(back)), dense(gk.permute(back)), pos, f, SECTIONS, inverse=True)
    assert torch.equal(dq, wq) and torch.equal(dk, wk)


def test_map_major_projection_through_the_attention(fa_lib):
    """Projection -> rotary -> differential attention -> gradients: the same as from dense tensors."""
    xq, xk, pos, f = setup()
    v = torch.randn((2, 37, 2, 48), device="cuda").to(xq.dtype).requires_grad_()
    lam = torch.full((4,), 0.3, device="cuda", requires_grad=True)
    grads = []
    for layout in (lambda t: t.transpose(2, 3), lambda t: dense(t.transpose(2, 3))):
        a, b = xq.detach().requires_grad_(), xk.detach().requires_grad_()
        q, k = rotary_func(layout(a), layout(b), pos, f, SECTIONS)
        o = diff_attn_func(q, k, v, lam, causal=True, deterministic=True)
        grads.append(torch.autograd.grad(o, (a, b, v, lam), torch.ones_like(o)))
    assert all(torch.equal(x, y) for x, y in zip(*grads))


def test_a_refused_call_writes_nothing(fa_lib):
    """Maps 4 elements off the 8-element grid, in q or in k, in place."""
    _, _, pos, f = setup()
    room = torch.randn((2, 37, 2, 4 * 24 + 4), device="cuda").half()
    odd = room[..., :4 * 24].unflatten(-1, (4, 24)).transpose(2, 3)
    good = torch.randn((2, 37, 2, 4, 24), device="cuda").half().transpose(2, 3)
    kept = room.clone(), good.clone()
    for q, k in ((odd, good), (good, odd), (odd, None)):
        with pytest.raises((ValueError, fa.FaError)):
            fa.rotary(q, k, pos, f, SECTIONS, out_q=q, out_k=k)
    torch.cuda.synchronize()
    assert torch.equal(room, kept[0]) and torch.equal(good, kept[1])
    with pytest.raises((ValueError, fa.FaError)):  # k's rows off the grid: q's maps are not turned either
        bad = torch.randn((2, 37, 4 * 24 + 4), device="cuda").half()[..., :4 * 24].unflatten(-1, (4, 24))
        fa.rotary(good, bad, pos, f, SECTIONS, out_q=good)
    torch.cuda.synchronize()
    assert torch.equal(good, kept[1])
