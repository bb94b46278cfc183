"""Refusals of outputs and inputs that autograd would lose track of, found before any CUDA call."""
import pytest
import torch

from exact_io_aware_96_b200 import fa
from exact_io_aware_96_b200.autograd import rotary_func


def half(*s):
    return torch.zeros(s).half()


def test_outputs_that_require_a_gradient(fa_lib):
    x, pos, f = half(1, 4, 2, 64), torch.zeros(1, 1, 4, dtype=torch.int32), torch.ones(32, dtype=torch.float64)
    for name in ("out_q", "out_k"):
        with pytest.raises(ValueError, match="gradient"):
            fa.rotary(x, x, pos, f, **{name: half(1, 4, 2, 64).requires_grad_()})
    q, v, lam = half(1, 4, 2, 2, 64), half(1, 4, 2, 128), torch.ones(2)
    for name, t in dict(out=v, out2=v, lse=torch.zeros(2, 1, 2, 4)).items():
        with pytest.raises(ValueError, match="gradient"):
            fa.diff_forward(q, q, v, lam, **{name: t.clone().requires_grad_()})
    for name, t in dict(dq=q, dk=q, dv=v, dlam=lam).items():
        with pytest.raises(ValueError, match="gradient"):
            fa.diff_backward(q, q, v, lam, v, v, torch.zeros(2, 1, 2, 4), v, **{name: t.clone().requires_grad_()})


def test_frequencies_get_no_gradient(fa_lib):
    x, pos, f = half(1, 4, 2, 64), torch.zeros(1, 1, 4, dtype=torch.int32), torch.ones(32, dtype=torch.float64)
    with pytest.raises(ValueError, match="inv_freq"):
        rotary_func(x, None, pos, f.requires_grad_())
