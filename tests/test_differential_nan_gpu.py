"""NaN and infinite scores among the keys that count: whichever key holds one, and
whichever kernel runs, every row that sees it says so, and no other row does."""
import numpy as np
import pytest
import torch

from exact_io_aware_96_b200 import fa
from oracle.differential import differential
from tests.test_differential_gpu import ROUND, case, check_lse, np64, status_clear, within

pytestmark = pytest.mark.gpu
BLOCK = 256  # first key of the third block of 128


def planted(Sq, Sk, value, dtype, Dv=16):
    """One key of the third block of every (batch, head) scores `value` in one map: each
    of the block's 128 columns in some head, map 1 in even batch entries, map 2 in odd
    ones. q is a unit vector, so a score is k's first column. Returns the inputs and
    [B, H] key indices."""
    B, H, D = 8, 32, 8
    q, k, v, lam, do = case(B, Sq, Sk, H, H, D, Dv, dtype, 91)
    q.zero_()
    q[..., 0] = 1
    k.clamp_(-1, 1)
    at = np.zeros((B, H), dtype=np.int64)
    for b in range(B):
        for h in range(H):
            at[b, h] = BLOCK + (b // 2) * H + h
            k[b, at[b, h], h, b % 2, 0] = value
    return q, k, v, lam, do, at


def oracle_without(q, k, v, lam, do, causal, dtype):
    u, t = ROUND[dtype]
    kz = torch.where(torch.isfinite(k), k, torch.zeros_like(k))
    return differential(np64(q), np64(kz), np64(v), np64(lam), 1.0, causal, np64(do), u=u, t=t)


@pytest.mark.parametrize("value", [float("nan"), float("inf")], ids=["nan", "inf"])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("Sq,causal", [(32, False), (512, True), (1, True), (3, False)])
def test_forward(fa_lib, Sq, causal, dtype, value):
    Sk = 512
    q, k, v, lam, do, at = planted(Sq, Sk, value, dtype)
    want = oracle_without(q, k, v, lam, do, causal, dtype)
    o, lse, o2 = fa.diff_forward(*(x.cuda() for x in (q, k, v, lam)), causal=causal, scale=1.0, need_o2=True)
    status_clear()
    o, o2, lse = np64(o), np64(o2), np64(lse)
    B, H = at.shape
    sees = np.arange(Sq)[None, None] + (Sk - Sq if causal else Sk) >= at[:, :, None]  # [B, H, Sq]
    rows = sees.transpose(0, 2, 1)
    assert np.isnan(o[rows]).all()
    for c, got in ((0, lse[0]), (1, lse[1])):
        hit = sees & (np.arange(B) % 2 == c)[:, None, None]
        assert np.isnan(got[hit]).all(), f"LSE of map {c + 1}"
        assert np.isfinite(got[~hit]).all()
    odd = rows & (np.arange(B) % 2 == 1)[:, None, None]
    assert np.isnan(o2[odd]).all() and np.isfinite(o2[~odd]).all()
    for name, got in (("o", o), ("o2", o2)):
        ok = ~rows
        within(name, torch.from_numpy(got[ok]), want[name][ok], want[name + "_bound"][ok])


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_a_score_of_minus_infinity_is_a_masked_key(fa_lib, dtype):
    for Sq in (32, 1):
        q, k, v, lam, do, at = planted(Sq, 512, float("-inf"), dtype)
        u, t = ROUND[dtype]
        low = torch.where(torch.isfinite(k), k, torch.full_like(k, -30000.0))  # its exponential is 0 in fp64 too
        want = differential(np64(q), np64(low), np64(v), np64(lam), 1.0, False, None, u=u, t=t)
        o, lse, o2 = fa.diff_forward(*(x.cuda() for x in (q, k, v, lam)), scale=1.0, need_o2=True)
        status_clear()
        check_lse(lse, want["lse"])
        within("o", o, want["o"], want["o_bound"])
        within("o2", o2, want["o2"], want["o2_bound"])


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("Sq,causal", [(160, False), (512, True)])
def test_backward(fa_lib, Sq, causal, dtype):
    """The NaN reaches dv and the NaN map's dk at every key that such a row sees, its dq
    in every such row, dlambda where it is in map 2. Rows that do not see it keep their
    dlambda, and their dq where no block of theirs holds the key (0 x NaN is NaN)."""
    Sk = 512
    q, k, v, lam, do, at = planted(Sq, Sk, float("nan"), dtype)
    want = oracle_without(q, k, v, lam, do, causal, dtype)
    cu = [x.cuda() for x in (q, k, v, lam, do)]
    o, lse, o2 = fa.diff_forward(*cu[:4], causal=causal, scale=1.0, need_o2=True)
    dq, dk, dv, dlam = (np64(x) for x in fa.diff_backward(*cu[:4], o, o2, lse, cu[4], causal=causal, scale=1.0))
    status_clear()
    B, H = at.shape
    rows = (np.arange(Sq)[None, :, None] + (Sk - Sq if causal else Sk)) >= at[:, None, :]  # [B, Sq, H]
    # Every key is seen by a NaN row: the last row sees them all.
    assert rows[:, -1].all() and np.isnan(dv).all()
    for c in (0, 1):
        mine = np.arange(B) % 2 == c
        assert np.isnan(dk[mine][:, :, :, c, 0]).all()  # dS is NaN; q's first column is 1
        hit = rows & mine[:, None, None]
        assert np.isnan(dq[:, :, :, c][hit]).all()
    assert np.isnan(dlam[rows & (np.arange(B) % 2 == 1)[:, None, None]]).all()
    for name, got, ok in (("dq", dq, ~rows & (np.arange(Sq) < BLOCK)[None, :, None]), ("dlam", dlam, ~rows)):
        w, bd = want[name][ok], want[name + "_bound"][ok]
        u, t = ROUND[dtype]
        within(name, torch.from_numpy(got[ok]), w, bd + u * np.abs(w) + t)
