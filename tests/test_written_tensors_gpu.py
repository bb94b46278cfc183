"""Tensors that the helpers write into: autograd learns of it, or the call is
refused; and what a call cannot give a gradient to is refused."""
import pytest
import torch

from exact_io_aware_96_b200 import fa
from exact_io_aware_96_b200.autograd import rotary_func

pytestmark = pytest.mark.gpu


def half(*s):
    return torch.randn(s, device="cuda").half()


def positions(S):
    return torch.arange(S, device="cuda")[None], fa.rotary_inv_freq((32,))


def recorded(t):
    """(saved, loss): a tensor whose values a later backward needs."""
    x = t.clone().requires_grad_()
    y = x * 2
    return y, (y * y).float().sum()


def test_in_place_rotary_is_seen_by_autograd(fa_lib):
    pos, f = positions(10)
    y, loss = recorded(half(1, 10, 2, 64))
    with torch.no_grad():
        fa.rotary(y, None, pos, f, out_q=y)
    with pytest.raises(RuntimeError, match="inplace"):
        loss.backward()
    y, loss = recorded(half(1, 10, 2, 64))
    with torch.no_grad():
        fa.rotary(half(1, 10, 2, 64), y, pos, f, out_k=y)
    with pytest.raises(RuntimeError, match="inplace"):
        loss.backward()


def test_given_outputs_are_seen_by_autograd(fa_lib):
    q, k, v, lam = half(1, 9, 2, 2, 64), half(1, 9, 2, 2, 64), half(1, 9, 2, 128), torch.full((2,), 0.5, device="cuda")
    o, lse, o2 = fa.diff_forward(q, k, v, lam, need_o2=True)
    do = half(1, 9, 2, 128)
    kept = dict(dq=q, dk=k, dv=v, dlam=lam)
    for name in ("out", "out2", "lse"):
        y, loss = recorded(lse if name == "lse" else o)
        with torch.no_grad():
            fa.diff_forward(q, k, v, lam, **{name: y})
        with pytest.raises(RuntimeError, match="inplace"):
            loss.backward()
    for name, like in kept.items():
        y, loss = recorded(like)
        with torch.no_grad():
            fa.diff_backward(q, k, v, lam, o, o2, lse, do, **{name: y})
        with pytest.raises(RuntimeError, match="inplace"):
            loss.backward()


def test_outputs_that_require_a_gradient_are_refused(fa_lib):
    pos, f = positions(9)
    x = half(1, 9, 2, 64).requires_grad_()
    y = x * 1
    for t in (x, y):
        before = t.detach().clone()
        for kw in (dict(out_q=t), dict(out_k=t)):
            with pytest.raises(ValueError, match="gradient"):
                fa.rotary(before, before, pos, f, **kw)
        torch.cuda.synchronize()
        assert torch.equal(t.detach(), before)
    q, k, v, lam = half(1, 9, 2, 2, 64), half(1, 9, 2, 2, 64), half(1, 9, 2, 128), torch.full((2,), 0.5, device="cuda")
    o, lse, o2 = fa.diff_forward(q, k, v, lam, need_o2=True)
    for kw in (dict(out=o), dict(out2=o2), dict(lse=lse)):
        name, t = next(iter(kw.items()))
        with pytest.raises(ValueError, match="gradient"):
            fa.diff_forward(q, k, v, lam, **{name: t.clone().requires_grad_()})
    for name, t in dict(dq=q, dk=k, dv=v, dlam=lam).items():
        with pytest.raises(ValueError, match="gradient"):
            fa.diff_backward(q, k, v, lam, o, o2, lse, o, **{name: t.clone().requires_grad_()})
    with torch.no_grad():  # nothing is recorded: written like any tensor
        leaf = half(1, 9, 2, 64).requires_grad_()
        want = fa.rotary(leaf, None, pos, f)[0]
        fa.rotary(leaf, None, pos, f, out_q=leaf)
    assert torch.equal(leaf.detach(), want)


def test_outputs_of_inference_mode(fa_lib):
    pos, f = positions(9)
    with torch.inference_mode():
        x = half(1, 9, 2, 64)
        want = fa.rotary(x, None, pos, f)[0]
        fa.rotary(x, None, pos, f, out_q=x)
        assert torch.equal(x, want)
    fa.rotary(half(1, 9, 2, 64), None, pos, f, out_q=x)  # outside of it too: no version to raise
    assert fa.fa_last_device_status()[0] == 0


def test_frequencies_get_no_gradient(fa_lib):
    pos, f = positions(9)
    x = half(1, 9, 2, 64).requires_grad_()
    with pytest.raises(ValueError, match="inv_freq"):
        rotary_func(x, None, pos, f.requires_grad_())
    with torch.no_grad():
        assert torch.equal(rotary_func(x, None, pos, f)[0], fa.rotary(x.detach(), None, pos, f.detach())[0])
