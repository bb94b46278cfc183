"""Differential attention and rotary positions without a GPU: workspace sizes, refusals (all on the host, before any CUDA call), the oracle."""
import ctypes

import numpy as np
import pytest
import torch

from exact_io_aware_96_b200 import fa
from oracle.differential import differential, rotary

A = 0x10000  # an aligned fake address: validation fails before any use


def tens(S=128, H=2, D=64, at=A):
    return fa.FaTensor(at, S * H * D, H * D, D)


def lam(**kw):
    d = dict(ptr=A, stride_b=0, stride_s=0, stride_h=1, extent_b=1, extent_s=1, extent_h=2, dtype=fa.FA_LAMBDA_FP32)
    d.update(kw)
    return fa.DiffLambda(**d)


def fwd(**kw):
    q, k = (fa.FaTensor * 2)(tens(), tens()), (fa.FaTensor * 2)(tens(), tens())
    p = fa.DiffFwdParams(q=q, k=k, v=tens(D=128), lam=lam(), o=tens(D=128), o2=tens(D=128), lse=A, B=1, H=2, Hk=2,
                         Sq=128, Sk=128, D=64, Dv=128, scale=0.125, causal=0, dtype=fa.FA_FP16)
    for n, v in kw.items():
        if n in ("q", "k"):
            getattr(p, n)[1] = v
        else:
            setattr(p, n, v)
    return fa.fa_diff_fwd(p)


def bwd(**kw):
    two = lambda: (fa.FaTensor * 2)(tens(), tens())  # noqa: E731
    wide = tens(D=128)
    p = fa.DiffBwdParams(q=two(), k=two(), v=wide, o=wide, o2=wide, dO=wide, lse=A, lam=lam(), dq=two(), dk=two(),
                         dv=wide, dlam=A, B=1, H=2, Hk=2, Sq=128, Sk=128, D=64, Dv=128, scale=0.125, causal=0,
                         dtype=fa.FA_FP16, workspace=A, workspace_bytes=1 << 30, deterministic=0)
    for n, v in kw.items():
        if n in ("q", "k", "dq", "dk"):
            getattr(p, n)[1] = v
        else:
            setattr(p, n, v)
    return fa.fa_diff_bwd(p)


SHARED = [
    (dict(q=tens(at=None)), -1), (dict(v=tens(at=None)), -1), (dict(lse=None), -1), (dict(lam=lam(ptr=None)), -1),
    (dict(B=0), -1), (dict(Hk=0), -1), (dict(H=3, lam=lam(extent_h=3)), -1), (dict(Sk=0), -1),
    (dict(scale=0.0), -1), (dict(scale=float("nan")), -1), (dict(scale=3e38), -1), (dict(causal=2), -1),
    (dict(D=72), -2), (dict(D=4), -2), (dict(Dv=136), -2), (dict(Dv=12), -2), (dict(dtype=2), -2),
    (dict(lam=lam(dtype=fa.FA_BF16)), -2), (dict(lam=lam(extent_h=3)), -1), (dict(lam=lam(stride_h=-1)), -1),
    (dict(lam=lam(ptr=A + 2)), -3), (dict(k=tens(at=A + 8)), -3), (dict(q=fa.FaTensor(A, 128 * 128, 130, 64)), -3),
    (dict(k=fa.FaTensor(A, 128 * 128, 0, 64)), -1), (dict(q=fa.FaTensor(A, 128 * 128, 128, 0)), -1),
    (dict(B=1 << 12, H=1 << 10, Hk=1, Sq=1 << 8, lam=lam(extent_h=1)), -1), (dict(lse=A + 2), -3),
]


@pytest.mark.parametrize("kw,code", SHARED + [(dict(o=tens(D=128, at=A + 8)), -3), (dict(k_lens=A + 1), -3),
                                              (dict(o2=tens(D=128, at=A + 4)), -3), (dict(workspace=A + 16), -3)])
def test_forward_refuses(fa_lib, kw, code):
    assert fwd(**kw) == code


@pytest.mark.parametrize("kw,code", SHARED + [
    (dict(dlam=None), -1), (dict(dlam=A + 2), -3), (dict(o2=tens(D=128, at=None)), -1), (dict(dk=tens(at=None)), -1),
    (dict(dq=fa.FaTensor(A, 128 * 128, 0, 64)), -1), (dict(deterministic=2), -1), (dict(workspace=None), -7),
    (dict(workspace_bytes=100), -7), (dict(workspace=A + 128), -3)])
def test_backward_refuses(fa_lib, kw, code):
    assert bwd(**kw) == code


def test_null_params(fa_lib):
    assert fa_lib.fa_diff_fwd(None, None) == fa_lib.fa_diff_bwd(None, None) == fa_lib.fa_rotary(None, None) == -1


def rot(**kw):
    x = tens()
    d = dict(q=x, k=x, q_out=x, k_out=x, positions=A, pos_stride_axis=128, pos_stride_b=128, pos_stride_s=1, pos_int64=0,
             inv_freq=A, inv_freq_fp64=1, axes=3, sections=(ctypes.c_int * 8)(8, 12, 12), B=1, S=128, H=2, Hk=2, D=64,
             interleaved=0, inverse=0, dtype=fa.FA_FP16)
    d.update(kw)
    return fa.fa_rotary(fa.RotaryParams(**d))


@pytest.mark.parametrize("kw,code", [
    (dict(q=tens(at=None)), -1), (dict(k_out=tens(at=None)), -1), (dict(positions=None), -1), (dict(inv_freq=None), -1),
    (dict(axes=0), -1), (dict(axes=9), -1), (dict(sections=(ctypes.c_int * 8)(8, -1, 12)), -1),
    (dict(sections=(ctypes.c_int * 8)(0, 0, 0)), -1), (dict(sections=(ctypes.c_int * 8)(20, 12, 12)), -1),
    (dict(S=0), -1), (dict(H=0), -1), (dict(Hk=-1), -1), (dict(interleaved=2), -1), (dict(inverse=-1), -1),
    (dict(D=12), -2), (dict(D=264), -2), (dict(dtype=2), -2), (dict(q=tens(at=A + 8)), -3),
    (dict(positions=A + 2), -3), (dict(positions=A + 4, pos_int64=1), -3), (dict(inv_freq=A + 4), -3),
    (dict(q_out=fa.FaTensor(A, 0, 0, 64)), -1),
])
def test_rotary_refuses(fa_lib, kw, code):
    assert rot(**kw) == code


def test_workspace_sizes(fa_lib):
    # both maps' accumulators [2, B*H*Sq_pad, 64], five row terms, one per row (rounded up), 4 KB (one part:
    # three query blocks a head are too few to cut)
    rows = 2 * 3 * 256
    want = (rows * (128 + 5) * 4 + 2 * 3 * 200 * 4 + 255) // 256 * 256 + 4096
    assert fa.fa_diff_bwd_workspace_size(2, 3, 3, 200, 300, 64, 128, 0, 0) == want
    det = (2 * 3 * 2 * 3 * 2 * 128 * 64 * 4 + rows * 5 * 4 + 2 * 3 * 200 * 4 + 255) // 256 * 256 + 4096
    assert fa.fa_diff_bwd_workspace_size(2, 3, 3, 200, 300, 64, 128, 0, 1) == det
    assert fa.fa_diff_bwd_workspace_size(2, 3, 3, 200, 300, 64, 128, 0, 2) == 0
    assert fa.fa_diff_bwd_workspace_size(2, 3, 3, 0, 300, 64, 128, 0, 0) == 0
    assert fa.fa_diff_fwd_workspace_size(1, 8, 8, 4096, 4096, 64, 128, 1) == 0
    assert fa.fa_diff_fwd_workspace_size(1, 8, 3, 1, 4096, 64, 128, 1) == 0  # refused: 3 does not divide 8


def test_cpu_tensors_are_refused(fa_lib):
    q, k, v = torch.zeros(1, 4, 2, 2, 64).half(), torch.zeros(1, 4, 2, 2, 64).half(), torch.zeros(1, 4, 2, 128).half()
    with pytest.raises(ValueError, match="CUDA"):
        fa.diff_forward(q, k, v, torch.ones(2))
    with pytest.raises(ValueError, match="CUDA"):
        fa.rotary(v, None, torch.zeros(1, 1, 4, dtype=torch.int32), torch.ones(64))
    with pytest.raises(TypeError):
        fa.diff_forward(q.float(), k.float(), v.float(), torch.ones(2))
    with pytest.raises(ValueError, match="expected q"):
        fa.diff_forward(v, k, v, torch.ones(2))


def test_helpers_check_their_tensors(fa_lib):
    """Shapes and dtypes, found before any CUDA call."""
    half = lambda *s: torch.zeros(s).half()  # noqa: E731
    q, k, v, lam = half(1, 4, 2, 2, 64), half(1, 6, 2, 2, 64), half(1, 6, 2, 128), torch.ones(2)
    for bad, error in (((q, half(1, 6, 2, 2, 32), v, lam), ValueError), ((q, k, half(1, 5, 2, 128), lam), ValueError),
                       ((q, k.bfloat16(), v, lam), TypeError), ((q, half(1, 6, 3, 2, 64), half(1, 6, 3, 128), lam), ValueError),
                       ((q, k, v, 0.5), TypeError)):
        with pytest.raises(error):
            fa.diff_forward(*bad)
    x, pos, f = half(1, 4, 2, 64), torch.zeros(3, 1, 4, dtype=torch.int32), torch.ones(32, dtype=torch.float64)
    with pytest.raises(ValueError, match="CUDA"):
        fa.rotary(x, None, pos, f, (8, 12, 12))
    with pytest.raises(TypeError, match="fp16/bf16"):
        fa.rotary(x.float(), None, pos, f, (8, 12, 12))


def test_oracle_gradients_are_its_differences():
    rng = np.random.default_rng(0)
    q, k, v = rng.standard_normal((1, 5, 4, 2, 8)), rng.standard_normal((1, 7, 2, 2, 8)), rng.standard_normal((1, 7, 2, 8))
    lam, do = rng.random((1, 5, 4)), rng.standard_normal((1, 5, 4, 8))
    for causal in (False, True):
        z = differential(q, k, v, lam, 0.4, causal, do)
        for name, x in (("dq", q), ("dk", k), ("dv", v), ("dlam", lam)):
            d = rng.standard_normal(x.shape)
            f = [float((differential(*(y + s * 1e-6 * d if y is x else y for y in (q, k, v, lam)), 0.4, causal)["o"]
                        * do).sum()) for s in (1, -1)]
            assert abs((f[0] - f[1]) / 2e-6 - float((z[name] * d).sum())) < 1e-6, name
        # lam = 0 is plain attention on the first maps
        plain = differential(q, k, v, 0 * lam, 0.4, causal)
        import oracle
        o, lse = oracle.attention_forward(q[:, :, :, 0], np.repeat(k[:, :, :, 0], 2, 2), np.repeat(v, 2, 2), 0.4, causal)
        assert np.allclose(plain["o"], o, atol=1e-12) and np.allclose(plain["lse"][0], lse, atol=1e-12)


def test_oracle_rotary_is_a_rotation():
    rng = np.random.default_rng(1)
    x, pos = rng.standard_normal((2, 3, 2, 16)), rng.integers(-50, 50, (2, 2, 3))
    f = 10.0 ** -rng.random(6)
    for inter in (False, True):
        y = rotary(x, pos, f, (2, 4), inter)
        assert np.allclose(rotary(y, pos, f, (2, 4), inter, inverse=True), x)
        assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1)) and not np.allclose(y, x)
        assert np.array_equal(y[..., 12:], x[..., 12:])
    # relative positions: the product of two turned vectors depends on the difference only
    a, b = x[:, :, :1], x[:, :, 1:]
    d1 = (rotary(a, pos + 7, f, (2, 4)) * rotary(b, pos, f, (2, 4))).sum()
    d2 = (rotary(a, pos + 14, f, (2, 4)) * rotary(b, pos + 7, f, (2, 4))).sum()
    assert abs(d1 - d2) < 1e-9
