"""Rotary positions with several axes on the GPU against the fp64 oracle. Each
result is one fp32 rotation (error below 1e-6 of the pair's norm) rounded once."""
import numpy as np
import pytest
import torch

from exact_io_aware_96_b200 import fa
from exact_io_aware_96_b200.autograd import rotary_func
from oracle.differential import rotary

pytestmark = pytest.mark.gpu
ROUND = {torch.bfloat16: (2.0 ** -8, 0.0), torch.float16: (2.0 ** -11, 2.0 ** -25)}


def np64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def check(got, x, positions, inv_freq, sections, interleaved, inverse):
    want = rotary(np64(x), positions.cpu().numpy(), inv_freq.cpu().double().numpy(), sections, interleaved, inverse)
    u, t = ROUND[x.dtype]
    err = np.abs(np64(got) - want)
    size = np.abs(np64(x)).max()
    assert np.all(err <= u * np.abs(want) + t + 2e-6 * size), err.max()
    R = len(inv_freq)
    assert torch.equal(got[..., 2 * R:].cpu(), x[..., 2 * R:].cpu())  # the rest is copied


def inputs(B, S, H, D, axes, dtype, seed, far=1000, pos_dtype=torch.int32):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((B, S, H, D), generator=g).to(dtype).cuda()
    pos = torch.randint(-far // 10, far, (axes, B, S), generator=g).to(pos_dtype).cuda()
    return x, pos


CASES = [  # B, S, H, Hk, D, sections, interleaved, dtype
    (1, 1, 1, 1, 8, (4,), False, torch.float16),
    (2, 77, 4, 2, 64, (8, 12, 12), False, torch.bfloat16),
    (2, 77, 4, 2, 64, (8, 12, 12), True, torch.float16),
    (1, 130, 3, 1, 80, (5, 3, 9), False, torch.bfloat16),   # odd pair count, columns left over
    (1, 130, 3, 1, 80, (5, 3, 9), True, torch.bfloat16),
    (3, 33, 2, 5, 128, (6, 0, 20), False, torch.float16),   # an axis without pairs; 26 pairs
    (1, 1000, 8, 8, 24, (4, 4, 4), False, torch.bfloat16),
    (1, 19, 1, 1, 256, (128,), True, torch.float16),
]


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("c", CASES, ids=lambda c: f"S{c[1]}D{c[4]}s{'-'.join(map(str, c[5]))}i{int(c[6])}")
def test_rotary(fa_lib, c, inverse):
    B, S, H, Hk, D, sections, inter, dtype = c
    q, pos = inputs(B, S, H, D, len(sections), dtype, S + D)
    k, _ = inputs(B, S, Hk, D, 1, dtype, S + D + 1)
    f = fa.rotary_inv_freq(sections)
    oq, ok = fa.rotary(q, k, pos, f, sections, interleaved=inter, inverse=inverse)
    torch.cuda.synchronize()
    check(oq, q, pos, f, sections, inter, inverse)
    check(ok, k, pos, f, sections, inter, inverse)


@pytest.mark.parametrize("pos_dtype,far", [(torch.int32, 2 ** 30), (torch.int64, 2 ** 40)])
@pytest.mark.parametrize("freq_dtype", [torch.float32, torch.float64])
def test_far_positions_keep_their_angle(fa_lib, pos_dtype, far, freq_dtype):
    """fp64 reduction: at 2^40 positions the turns hold 2^-52 x 2^40 / 2 pi, about 4e-5; sin and cos follow."""
    q, pos = inputs(1, 50, 2, 64, 3, torch.float16, 5, far, pos_dtype)
    f = fa.rotary_inv_freq((8, 12, 12), per_axis=True).to(freq_dtype)
    oq, none = fa.rotary(q, None, pos, f, (8, 12, 12))
    assert none is None
    want = rotary(np64(q), pos.cpu().numpy(), f.cpu().double().numpy(), (8, 12, 12))
    # angle errors of both sides: |theta| 2^-52 each (and one rounding of freq / 2 pi): 4 |theta| 2^-53
    slack = 2e-6 + far * 4 * 2.0 ** -53
    bound = 2.0 ** -11 * np.abs(want) + 2.0 ** -25 + slack * np.abs(np64(q)).max() * 2
    assert np.all(np.abs(np64(oq) - want) <= bound)


def test_in_place_views_and_shared_positions(fa_lib):
    """q and k as views of a packed projection, turned in place; v untouched; one position row for all."""
    x, _ = inputs(2, 65, 8, 64, 1, torch.bfloat16, 8)
    ref = x.clone()
    pos = torch.arange(65, device="cuda", dtype=torch.int64)[None, None].expand(3, 2, 65)
    f = fa.rotary_inv_freq((8, 12, 12))
    q, k = x[:, :, :4], x[:, :, 4:6]
    fa.rotary(q, k, pos, f, (8, 12, 12), out_q=q, out_k=k)
    check(q, ref[:, :, :4], pos, f, (8, 12, 12), False, False)
    check(k, ref[:, :, 4:6], pos, f, (8, 12, 12), False, False)
    assert torch.equal(x[:, :, 6:], ref[:, :, 6:])


def test_gradient(fa_lib):
    q, pos = inputs(2, 40, 3, 48, 2, torch.float16, 11)
    k, _ = inputs(2, 40, 1, 48, 1, torch.float16, 12)
    gq, _ = inputs(2, 40, 3, 48, 1, torch.float16, 13)
    gk, _ = inputs(2, 40, 1, 48, 1, torch.float16, 14)
    f = fa.rotary_inv_freq((10, 9))
    q.requires_grad_()
    k.requires_grad_()
    oq, ok = rotary_func(q, k, pos, f, (10, 9))
    dq, dk = torch.autograd.grad((oq, ok), (q, k), (gq, gk))
    check(dq, gq, pos, f, (10, 9), False, True)
    check(dk, gk, pos, f, (10, 9), False, True)
