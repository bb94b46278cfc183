"""Differential attention and rotary positions as programs use them: the run of
both with gradients, graphs, streams, guard bands, far strides, the check build."""
import os

import numpy as np
import pytest
import torch

from exact_io_aware_96_b200 import build, fa
from exact_io_aware_96_b200.autograd import diff_attn_func, rotary_func
from oracle.differential import differential
from tests.test_differential_gpu import CASES, IDS, ROUND, case, check_lse, full_check, np64, status_clear, within

pytestmark = pytest.mark.gpu
SECTIONS = (8, 12, 12)


def grid_positions(B, S):
    at = torch.arange(S, device="cuda")
    return torch.stack((at // 36, at // 6 % 6, at % 6))[:, None].expand(3, B, S).to(torch.int32)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_rotary_then_attention_with_gradients(fa_lib, dtype):
    """Project -> turn q and k -> differential attention -> gradients of everything."""
    B, S, H, Hk, D, Dv = 2, 150, 4, 2, 64, 128
    q, k, v, lam, do = (x.cuda() for x in case(B, S, S, H, Hk, D, Dv, dtype, 3, "head", torch.float32))
    pos, f = grid_positions(B, S), fa.rotary_inv_freq(SECTIONS)
    leaves = [x.requires_grad_() for x in (q, k, v, lam)]
    rq, rk = rotary_func(q, k, pos, f, SECTIONS)
    assert rq.shape == q.shape and rk.shape == k.shape
    o = diff_attn_func(rq, rk, v, lam, causal=True, deterministic=True)
    got = torch.autograd.grad(o, leaves, do)
    # attention on what rotary returned, against the oracle
    u, t = ROUND[dtype]
    want = differential(np64(rq), np64(rk), np64(v), np64(lam), D ** -0.5, True, np64(do), u=u, t=t)
    within("o", o, want["o"], want["o_bound"])
    within("dv", got[2], want["dv"], want["dv_bound"])
    # the chain: the attention's gradients turned back
    with torch.no_grad():
        a, lse, a2 = fa.diff_forward(rq, rk, v, lam, causal=True, need_o2=True)
        dq, dk, dv, dlam = fa.diff_backward(rq, rk, v, lam, a, a2, lse, do, causal=True, deterministic=True)
        bq, bk = fa.rotary(dq, dk, pos, f, SECTIONS, inverse=True)
    status_clear()
    assert torch.equal(o, a)
    for x, y in zip(got, (bq, bk, dv, dlam)):
        assert torch.equal(x, y)


@pytest.mark.parametrize("Sq", [1, 3, 200])
def test_graph_of_the_forward(fa_lib, Sq):
    """Captured and replayed on new inputs; another graph between the replays; equal to the eager call."""
    B, Sk, H, Hk, D, Dv = 2, 1500, 4, 2, 64, 128
    sets = [[x.cuda() for x in case(B, Sq, Sk, H, Hk, D, Dv, torch.bfloat16, 60 + i, "head", torch.float32)]
            for i in range(3)]
    lens = torch.tensor([Sk, 700], dtype=torch.int32, device="cuda")
    call = lambda q, k, v, lam, _: fa.diff_forward(q, k, v, lam, causal=True, k_lens=lens, need_o2=True)  # noqa: E731
    want = [[y.clone() for y in call(*x)] for x in sets]
    graphs, outs, ins = [], [], []
    for i in range(2):
        ins.append([x.clone() for x in sets[i]])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call(*ins[i]))
        graphs.append(g)
    for order in ((0, 0), (1, 1), (0, 2), (1, 0), (0, 1)):
        g, s = order
        for dst, src in zip(ins[g], sets[s]):
            dst.copy_(src)
        graphs[g].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs[g], want[s])), order
    status_clear()


@pytest.mark.parametrize("c", [(1, 1000, 1000, 8, 1, 64, 128, torch.bfloat16, True),
                               (1, 900, 130, 6, 2, 40, 64, torch.float16, False),
                               (2, 700, 1100, 4, 1, 64, 72, torch.float16, True)], ids=["8-1", "6-2", "4-1"])
def test_backward_in_parts(fa_lib, c):
    """Many query heads on few key heads: the key blocks' lists are cut into parts and joined."""
    B, Sq, Sk, H, Hk, D, Dv, dtype, causal = c
    whole = 4 * (B * H * -(-Sq // 128) * 128 * (2 * 64 + 5) + B * H * Sq) + 256 + 4096  # the workspace of one part
    assert fa.fa_diff_bwd_workspace_size(B, H, Hk, Sq, Sk, D, Dv, int(causal), 0) > whole
    x = case(B, Sq, Sk, H, Hk, D, Dv, dtype, 43, "head", torch.float32)
    full_check(x, causal)
    one, two = (full_check(x, causal, deterministic=True) for _ in range(2))
    assert all(torch.equal(a, b) for a, b in zip(one, two))


def test_graph_of_a_training_pass(fa_lib):
    B, Sq, Sk, H, Hk, D, Dv = 1, 200, 260, 4, 2, 64, 128
    sets = [[x.cuda() for x in case(B, Sq, Sk, H, Hk, D, Dv, torch.float16, 70 + i, "token")] for i in range(2)]

    def call(q, k, v, lam, do):
        o, lse, o2 = fa.diff_forward(q, k, v, lam, causal=True, need_o2=True)
        return (o, *fa.diff_backward(q, k, v, lam, o, o2, lse, do, causal=True, deterministic=True))

    want = [call(*x) for x in sets]
    ins = [x.clone() for x in sets[0]]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = call(*ins)
    for s in (1, 0, 1):
        for dst, src in zip(ins, sets[s]):
            dst.copy_(src)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want[s]))
    status_clear()


@pytest.mark.parametrize("raw", [False, True])
def test_given_stream(fa_lib, raw):
    """Everything on a side stream: helper allocations belong to it, nothing waits on the current stream."""
    c = [x.cuda() for x in case(1, 300, 300, 2, 2, 64, 128, torch.bfloat16, 81)]
    q, k, v, lam, do = c
    pos, f = grid_positions(1, 300), fa.rotary_inv_freq(SECTIONS)
    want_r = fa.rotary(q, k, pos, f, SECTIONS)
    o, lse, o2 = fa.diff_forward(q, k, v, lam, need_o2=True)
    want = fa.diff_backward(q, k, v, lam, o, o2, lse, do, deterministic=True)
    one, _, _ = fa.diff_forward(q[:, :1], k, v, lam[:, :1])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    s = side.cuda_stream if raw else side
    torch.cuda._sleep(20_000_000)  # the current stream is busy for about 10 ms
    for _ in range(20):
        r = fa.rotary(q, k, pos, f, SECTIONS, stream=s)
        p, l2, p2 = fa.diff_forward(q, k, v, lam, need_o2=True, stream=s)
        got = fa.diff_backward(q, k, v, lam, p, p2, l2, do, deterministic=True, stream=s)
        single, _, _ = fa.diff_forward(q[:, :1], k, v, lam[:, :1], stream=s)
    side.synchronize()
    assert torch.equal(p, o) and torch.equal(single, one)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all(torch.equal(a, b) for a, b in zip(r, want_r))
    status_clear()


def test_two_streams_at_once(fa_lib):
    sets = [[x.cuda() for x in case(2, 1, 3000, 8, 2, 64, 128, torch.bfloat16, 90 + i, "head")] for i in range(2)]
    want = [fa.diff_forward(*x[:4])[0] for x in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(50):
        got = []
        for s, x in zip(streams, sets):
            with torch.cuda.stream(s):
                got.append(fa.diff_forward(*x[:4])[0])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    status_clear()


def banded(t, fill):
    """A copy of `t`'s shape inside a larger buffer of `fill`: rows and columns of margin on every side."""
    shape = list(t.shape)
    big = torch.full([n + 2 for n in shape[:-1]] + [shape[-1] + 16], fill, dtype=t.dtype, device=t.device)
    view = big[tuple(slice(1, -1) for _ in shape[:-1]) + (slice(8, -8),)]
    return big, view


@pytest.mark.parametrize("c", [CASES[3], CASES[6], CASES[7], (2, 2, 700, 4, 2, 40, 72, torch.bfloat16, True, "head")],
                         ids=[IDS[3], IDS[6], IDS[7], "rows"])
def test_guard_bands(fa_lib, c):
    """Nothing outside the outputs and the exact workspace is written."""
    B, Sq, Sk, H, Hk, D, Dv, dtype, causal, lam = c
    q, k, v, w, do = (x.cuda() for x in case(B, Sq, Sk, H, Hk, D, Dv, dtype, 7, lam))
    fill = 123.0
    bands = {}

    def out(name, like):
        big, view = banded(like, fill)
        bands[name] = (big, view)
        return view

    def flat(n, dt):
        big = torch.full((n + 512,), 77, dtype=dt, device="cuda")
        return big, big[256:256 + n]

    o_like = torch.empty(B, Sq, H, Dv, dtype=dtype, device="cuda")
    lse_big, lse = flat(2 * B * H * Sq, torch.float32)
    n = fa.fa_diff_fwd_workspace_size(B, H, Hk, Sq, Sk, D, Dv, int(causal))
    fws_big, fws = flat(n, torch.uint8)
    o, lse, o2 = fa.diff_forward(q, k, v, w, causal=causal, out=out("o", o_like), out2=out("o2", o_like),
                                 lse=lse.view(2, B, H, Sq), workspace=fws if n else None)
    n = fa.fa_diff_bwd_workspace_size(B, H, Hk, Sq, Sk, D, Dv, int(causal), 0)
    ws_big, ws = flat(n, torch.uint8)
    dl_big, dl = flat(max(1, w.numel()), w.dtype)
    fa.diff_backward(q, k, v, w, o.contiguous(), o2.contiguous(), lse, do, causal=causal, dq=out("dq", q),
                     dk=out("dk", k), dv=out("dv", v), dlam=dl[:w.numel()].view(w.shape), workspace=ws)
    status_clear()
    for name, (big, view) in bands.items():
        assert torch.isfinite(view.float()).all(), name
        view.fill_(fill)
        assert (big == fill).all(), name
    for big in (lse_big, fws_big, ws_big, dl_big):
        assert (big[:256] == 77).all() and (big[-256:] == 77).all()


def test_strides_past_32_bits(fa_lib):
    """Batch entries more than 2^31 elements apart, in q, k, v, o and the gradients."""
    B, Sq, Sk, H, Hk, D, Dv, dtype = 2, 130, 140, 2, 1, 64, 128, torch.bfloat16
    c = case(B, Sq, Sk, H, Hk, D, Dv, dtype, 13)
    far = 2 ** 31 + 1024
    room = torch.empty(far + 8 * 1024 * 1024, dtype=dtype, device="cuda")
    at = 0

    def place(t):
        nonlocal at
        n = t[0].numel()
        view = room.as_strided(t.shape, (far,) + torch.empty(t.shape[1:]).stride(), at)
        at += (n + 63) // 64 * 64
        return view

    q, k, v, lam, do = (x.cuda() for x in c)
    views = [place(x) for x in (q, k, v, do)]
    for dst, src in zip(views, (q, k, v, do)):
        dst.copy_(src)
    fq, fk, fv, fdo = views
    o, lse, o2 = fa.diff_forward(q, k, v, lam, causal=True, need_o2=True)
    want = fa.diff_backward(q, k, v, lam, o, o2, lse, do, causal=True, deterministic=True)
    p, l2, p2 = fa.diff_forward(fq, fk, fv, lam, causal=True, out=place(o), out2=place(o))
    got = fa.diff_backward(fq, fk, fv, lam, p, p2, l2, fdo, causal=True, deterministic=True, dq=place(q), dk=place(k),
                           dv=place(v))
    assert torch.equal(p, o) and torch.equal(l2, lse) and all(torch.equal(a, b) for a, b in zip(got, want))
    assert torch.equal(fa.diff_forward(fq[:, :1], fk, fv, lam[:, :1], causal=True)[0],
                       fa.diff_forward(q[:, :1], k, v, lam[:, :1], causal=True)[0])
    pos, f = torch.arange(Sk, device="cuda").expand(1, B, Sk), fa.rotary_inv_freq((32,))
    r, _ = fa.rotary(fk, None, pos, f)
    assert torch.equal(r, fa.rotary(k, None, pos, f)[0])
    status_clear()


def test_weights_of_rows_without_a_key_do_not_count(fa_lib):
    """A row that sees nothing is 0 and has no gradient, whatever its weight holds."""
    B, Sq, Sk, H, D, Dv = 1, 40, 16, 2, 64, 128
    q, k, v, lam, do = (x.cuda() for x in case(B, Sq, Sk, H, H, D, Dv, torch.float16, 17))
    lam[:, :Sq - Sk] = float("nan")
    o, lse, o2 = fa.diff_forward(q, k, v, lam, causal=True, need_o2=True)
    dq, dk, dv, dlam = fa.diff_backward(q, k, v, lam, o, o2, lse, do, causal=True)
    status_clear()
    assert (o[:, :Sq - Sk] == 0).all() and (lse[..., :Sq - Sk] == -float("inf")).all()
    assert (dq[:, :Sq - Sk] == 0).all() and (dlam[:, :Sq - Sk] == 0).all()
    for x in (o, dq, dk, dv, dlam):
        assert torch.isfinite(x.float()).all()


def test_autograd_takes_what_programs_hand_it(fa_lib):
    """Transposed and misaligned inputs, an expanded output gradient, gradients of some inputs only."""
    B, S, H, D, Dv = 2, 64, 2, 64, 128
    q, k, v, lam, _ = (x.cuda() for x in case(B, S, S, H, H, D, Dv, torch.bfloat16, 19, "one", torch.float32))
    ref = [x.clone().requires_grad_() for x in (q, k, v, lam)]
    diff_attn_func(*ref, deterministic=True).float().sum().backward()
    qt = q.permute(0, 2, 3, 4, 1).contiguous().permute(0, 4, 1, 2, 3).requires_grad_()     # last axis strided
    off = torch.empty(v.numel() + 1, dtype=v.dtype, device="cuda")[1:].view(v.shape)       # 2-byte aligned
    off.copy_(v)
    off.requires_grad_()
    o = diff_attn_func(qt, k, off, lam, deterministic=True)
    dq, dv = torch.autograd.grad(o, (qt, off), torch.ones((), dtype=o.dtype, device="cuda").expand(o.shape))
    status_clear()
    assert torch.equal(dq, ref[0].grad) and torch.equal(dv, ref[2].grad)
    with torch.no_grad():
        assert torch.equal(diff_attn_func(q, k, v, lam), o)


def test_strides_of_axes_of_length_one(fa_lib):
    """torch calls a tensor contiguous whatever the stride of an axis of length 1."""
    q, k, v, lam, do = (x.cuda() for x in case(1, 1, 200, 1, 1, 64, 128, torch.bfloat16, 47))
    odd = lambda t: t.as_strided(t.shape, [1 if n == 1 else s for n, s in zip(t.shape, t.stride())])  # noqa: E731
    o, lse, o2 = fa.diff_forward(q, k, v, lam, need_o2=True)
    want = fa.diff_backward(q, k, v, lam, o, o2, lse, do, deterministic=True)
    p, l2, p2 = fa.diff_forward(odd(q), odd(k), odd(v), lam, out=odd(torch.empty_like(o)), need_o2=True)
    got = fa.diff_backward(odd(q), odd(k), odd(v), lam, odd(p), odd(p2), l2, odd(do), deterministic=True)
    pos, f = torch.arange(200, device="cuda")[None], fa.rotary_inv_freq((32,))
    r, s = fa.rotary(odd(k), None, pos, f)[0], fa.rotary(k, None, pos, f)[0]
    status_clear()
    assert torch.equal(o, p) and torch.equal(r, s) and all(torch.equal(a, b) for a, b in zip(got, want))


def test_rotary_of_q_alone_with_gradient(fa_lib):
    q = torch.randn((1, 30, 2, 64), device="cuda").half().requires_grad_()
    pos, f = torch.arange(30, device="cuda")[None], fa.rotary_inv_freq((32,))
    out, none = rotary_func(q, None, pos, f)
    (g,) = torch.autograd.grad(out, q, torch.ones_like(out))
    assert none is None
    assert torch.equal(g, fa.rotary(torch.ones_like(q), None, pos, f, inverse=True)[0])


FIRST_CALL = """
import torch
from exact_io_aware_96_b200 import fa
q, k, v = (torch.randn(s, device="cuda").half() for s in ((1, {Sq}, 2, 2, 64), (1, 600, 2, 2, 64), (1, 600, 2, 128)))
lam = torch.rand(2, device="cuda")
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    o, lse, o2 = fa.diff_forward(q, k, v, lam, need_o2=True)
    grads = fa.diff_backward(q, k, v, lam, o, o2, lse, o, deterministic=True)
g.replay()
torch.cuda.synchronize()
p, l2, p2 = fa.diff_forward(q, k, v, lam, need_o2=True)
assert torch.equal(o, p)
assert all(torch.equal(a, b) for a, b in zip(grads, fa.diff_backward(q, k, v, lam, p, p2, l2, p, deterministic=True)))
assert fa.fa_last_device_status()[0] == 0
print("captured first")
"""


@pytest.mark.parametrize("Sq", [1, 200])
def test_first_call_inside_a_capture(fa_lib, Sq):
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    out = subprocess.run([sys.executable, "-c", FIRST_CALL.format(Sq=Sq)], cwd=root, capture_output=True, text=True,
                         timeout=200)
    assert "captured first" in out.stdout, out.stderr[-1500:]


def test_refusals_on_the_device(fa_lib):
    q, k, v, lam, _ = (x.cuda() for x in case(1, 8, 12, 4, 2, 64, 128, torch.float16, 53))
    pos, f = torch.zeros((3, 1, 8), dtype=torch.int32, device="cuda"), fa.rotary_inv_freq(SECTIONS)
    x = q.flatten(2, 3)
    for call, error in (
            (lambda: fa.diff_forward(q, k, v, lam[:, :3]), ValueError),
            (lambda: fa.diff_forward(q, k, v, lam.bfloat16()), TypeError),
            (lambda: fa.diff_forward(q, k, v, lam.cpu()), ValueError),
            (lambda: fa.diff_forward(q, k, v.cpu(), lam), ValueError),
            (lambda: fa.diff_forward(q, k, v, lam, k_lens=torch.ones(1, device="cuda")), TypeError),
            (lambda: fa.diff_forward(q, k, v, lam, k_lens=torch.ones(2, dtype=torch.int32, device="cuda")), ValueError),
            (lambda: fa.diff_forward(q, k, v, lam, out=v), ValueError),
            (lambda: fa.diff_forward(q, k, v, lam, scale=-1.0), fa.FaError),
            (lambda: fa.diff_forward(q[:, :1].expand(1, 8, 4, 2, 64), k, v, lam), fa.FaError),
            (lambda: fa.diff_forward(q[:0], k[:0], v[:0], lam[:0]), fa.FaError),
            (lambda: fa.diff_forward(q[:, :1], k, v, lam[:, :1], workspace=torch.empty(0, dtype=torch.uint8)), ValueError),
            (lambda: fa.diff_forward(q[..., :4], k[..., :4], v, lam), fa.FaError),
            (lambda: fa.rotary(x, None, pos, f, (8, 12)), ValueError),
            (lambda: fa.rotary(x, None, pos, f, (8, 12, 11)), ValueError),
            (lambda: fa.rotary(x, None, pos, f, (40, -20, 12)), ValueError),
            (lambda: fa.rotary(x, None, pos.float(), f, SECTIONS), TypeError),
            (lambda: fa.rotary(x, None, pos[:, :, :7], f, SECTIONS), ValueError),
            (lambda: fa.rotary(x[..., :32], None, pos, f, SECTIONS), ValueError),
            (lambda: fa.rotary(x, None, pos, f.half(), SECTIONS), TypeError),
            (lambda: fa.rotary(x, None, pos, f.cpu(), SECTIONS), ValueError),
            (lambda: fa.rotary(x, None, pos, f, SECTIONS, out_k=x), ValueError)):
        with pytest.raises(error):
            call()
    status_clear()


def test_no_second_derivative(fa_lib):
    q, k, v, lam, _ = (x.cuda() for x in case(1, 8, 8, 1, 1, 64, 64, torch.float16, 23))
    q.requires_grad_()
    (dq,) = torch.autograd.grad(diff_attn_func(q, k, v, lam).float().sum(), q, create_graph=True)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(dq.float().sum(), q)


@pytest.fixture
def check_lib():
    if not os.path.exists(fa.LIB_CHECK_PATH):
        build.build(check=True)
    normal = fa.LIB_PATH
    fa.use_library(fa.LIB_CHECK_PATH)
    try:
        yield fa.lib()
    finally:
        fa.use_library(normal)


@pytest.mark.parametrize("c", CASES[3:9], ids=IDS[3:9])
def test_check_build(check_lib, c):
    """The bounds-checking build: same results, no check fails."""
    B, Sq, Sk, H, Hk, D, Dv, dtype, causal, lam = c
    x = case(B, Sq, Sk, H, Hk, D, Dv, dtype, 29, lam)
    full_check(x, causal)
    full_check(x, causal, deterministic=True)


def test_check_build_few_rows(check_lib):
    u, t = ROUND[torch.bfloat16]
    for B, Sq, Sk, H, Hk in ((2, 3, 2111, 8, 2), (1, 16, 300, 4, 1)):
        q, k, v, lam, _ = case(B, Sq, Sk, H, Hk, 64, 128, torch.bfloat16, 31)
        want = differential(np64(q), np64(k), np64(v), np64(lam), 0.125, True, u=u, t=t)
        o, lse, _ = fa.diff_forward(q.cuda(), k.cuda(), v.cuda(), lam.cuda(), causal=True)
        status_clear()
        check_lse(lse, want["lse"])
        within("o", o, want["o"], want["o_bound"])


def test_dlambda_of_few_and_many_terms(fa_lib):
    """Sums of 1, a few, thousands and hundreds of thousands of row terms."""
    B, S, H, Dv = 3, 1500, 8, 64
    q, k, v, _, do = (x.cuda() for x in case(B, S, 40, H, 2, 64, Dv, torch.bfloat16, 37, "one"))
    full = None
    for shape in ((B, S, H), (1, S, H), (B, S, 1), (B, 1, H), (H,), (S, 1), (B, 1, 1), ()):
        lam = torch.full(shape, 0.5, device="cuda")
        o, lse, o2 = fa.diff_forward(q, k, v, lam, need_o2=True)
        dlam = fa.diff_backward(q, k, v, lam, o, o2, lse, do)[3]
        if full is None:
            full = dlam.double()
        want = full
        for a, e in enumerate((1,) * (3 - len(shape)) + shape):
            if e == 1:
                want = want.sum(a, keepdim=True)
        mass = full.abs().sum() / want.numel()
        # fp32 sums of up to 36000 terms in chains of a few hundred: 2^-24 x 300 of the terms' mass
        assert torch.all((dlam.double() - want.reshape(shape)).abs() <= 2e-5 * mass)
    status_clear()
