"""Differential attention on the GPU against the fp64 oracle, elementwise within
the bounds that its 16-bit roundings allow (oracle/differential.py)."""
import numpy as np
import pytest
import torch

from exact_io_aware_96_b200 import fa
from exact_io_aware_96_b200.autograd import diff_attn_func
from oracle.differential import differential

pytestmark = pytest.mark.gpu

# Largest relative rounding error, and half the smallest subnormal step.
ROUND = {torch.bfloat16: (2.0 ** -8, 0.0), torch.float16: (2.0 ** -11, 2.0 ** -25)}
# Both logsumexps: relative error of l (polynomial exp2 7.5e-5, sums) plus fp32
# scores, absolute; then fp32's own rounding.
LSE_ABS, LSE_REL = 3e-4, 1e-6


def case(B, Sq, Sk, H, Hk, D, Dv, dtype, seed, lam="token", lam_dtype=None, std=1.0):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    q, k = (rnd(B, Sq, H, 2, D) * std).to(dtype), (rnd(B, Sk, Hk, 2, D) * std).to(dtype)
    v, do = rnd(B, Sk, Hk, Dv).to(dtype), rnd(B, Sq, H, Dv).to(dtype)
    shape = {"token": (B, Sq, H), "head": (H,), "one": (), "row": (Sq, 1), "batch": (B, 1, 1)}[lam]
    w = (torch.rand(shape, generator=g) * 0.9 + 0.05).to(lam_dtype or dtype)
    return q, k, v, w, do


def np64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def status_clear():
    st, detail = fa.fa_last_device_status()
    assert st == 0, (st, detail)


def within(name, got, want, bound):
    err = np.abs(np64(got) - want)
    bad = ~(err <= bound + 1e-30)
    assert not bad.any(), (f"{name}: {bad.sum()} of {bad.size} outside, worst {np.max(err[bad] / bound[bad]):.3g} x "
                           f"its bound at {np.argwhere(bad)[0]}")


def check_lse(got, want):
    got = np64(got)
    assert np.array_equal(np.isneginf(got), np.isneginf(want))
    fin = np.isfinite(want)
    assert np.all(np.abs(got[fin] - want[fin]) <= LSE_ABS + LSE_REL * np.abs(want[fin]))


def close_in_norm(name, got, want, tol):
    n = np.linalg.norm(want)
    rel = np.linalg.norm(np64(got) - want) / n if n else 0.0
    assert rel <= tol, f"{name}: relative L2 {rel:.3e} > {tol:.3e}"


def fold_lam(x, lam):
    """The oracle's [B, Sq, H] summed to lam's shape."""
    ext = (1,) * (3 - lam.dim()) + tuple(lam.shape)
    for a, e in enumerate(ext):
        if e == 1:
            x = x.sum(axis=a, keepdims=True)
    return x.reshape(tuple(lam.shape))


def full_check(c, causal, scale=None, deterministic=False, n_keys=None):
    q, k, v, lam, do = c
    D = q.shape[-1]
    scale = D ** -0.5 if scale is None else scale
    u, t = ROUND[q.dtype]
    want = differential(np64(q), np64(k), np64(v), np64(lam), scale, causal, np64(do), u=u, t=t)
    cu = [x.cuda() for x in c]
    o, lse, o2 = fa.diff_forward(*cu[:4], causal=causal, scale=scale, need_o2=True)
    dq, dk, dv, dlam = fa.diff_backward(*cu[:4], o, o2, lse, cu[4], causal=causal, scale=scale,
                                        deterministic=deterministic)
    status_clear()
    check_lse(lse, want["lse"])
    for name, got in (("o", o), ("o2", o2), ("dq", dq), ("dk", dk), ("dv", dv)):
        within(name, got, want[name], want[name + "_bound"])
    ul = {torch.float32: 2.0 ** -24}.get(lam.dtype, u)
    dl = fold_lam(want["dlam"], lam)
    within("dlam", dlam, dl, fold_lam(want["dlam_bound"], lam) + ul * np.abs(dl) + t)
    # Roundings are independent: root mean square well below the worst case.
    for name, got in (("o", o), ("dq", dq), ("dk", dk), ("dv", dv)):
        close_in_norm(name, got, want[name], 4 * u)
    return o, lse, o2, dq, dk, dv, dlam


CASES = [  # B, Sq, Sk, H, Hk, D, Dv, dtype, causal, lam
    (1, 1, 1, 1, 1, 64, 128, torch.bfloat16, False, "token"),
    (1, 1, 1, 2, 1, 8, 8, torch.float16, True, "head"),
    (1, 128, 128, 2, 2, 64, 128, torch.float16, False, "token"),
    (1, 129, 127, 1, 1, 64, 128, torch.bfloat16, False, "one"),
    (2, 64, 300, 3, 3, 64, 64, torch.bfloat16, True, "token"),
    (1, 300, 64, 2, 2, 64, 128, torch.float16, True, "head"),     # rows without a key
    (2, 257, 257, 4, 2, 40, 80, torch.bfloat16, True, "row"),     # shared key heads
    (1, 200, 385, 6, 2, 24, 72, torch.float16, False, "batch"),
    (2, 193, 320, 4, 1, 64, 96, torch.float16, True, "token"),
    (1, 700, 700, 2, 2, 56, 128, torch.bfloat16, True, "token"),
    (1, 513, 1, 2, 1, 64, 128, torch.bfloat16, False, "token"),
    (3, 65, 640, 1, 1, 16, 120, torch.float16, False, "one"),
]
IDS = [f"B{c[0]}q{c[1]}k{c[2]}h{c[3]}-{c[4]}d{c[5]}-{c[6]}c{int(c[8])}" for c in CASES]


@pytest.mark.parametrize("c", CASES, ids=IDS)
def test_forward_and_backward(fa_lib, c):
    B, Sq, Sk, H, Hk, D, Dv, dtype, causal, lam = c
    full_check(case(B, Sq, Sk, H, Hk, D, Dv, dtype, 1 + Sq + Sk + D, lam), causal)


@pytest.mark.parametrize("lam", ["token", "head", "one", "row", "batch"])
def test_fp32_lambda_of_every_shape(fa_lib, lam):
    full_check(case(2, 150, 170, 4, 2, 64, 128, torch.bfloat16, 77, lam, torch.float32), True)


@pytest.mark.parametrize("c", [CASES[3], CASES[5], CASES[8]], ids=[IDS[3], IDS[5], IDS[8]])
def test_deterministic_backward_repeats(fa_lib, c):
    B, Sq, Sk, H, Hk, D, Dv, dtype, causal, lam = c
    x = case(B, Sq, Sk, H, Hk, D, Dv, dtype, 5 + Sq, lam)
    one = full_check(x, causal, deterministic=True)
    two = full_check(x, causal, deterministic=True)
    assert all(torch.equal(a, b) for a, b in zip(one, two))


def test_wide_scores(fa_lib):
    """Scores spread over hundreds: the running maximum is raised in most blocks."""
    full_check(case(1, 260, 640, 2, 2, 64, 128, torch.bfloat16, 9, std=4.0), False)
    full_check(case(1, 640, 640, 2, 2, 64, 128, torch.float16, 10, std=3.0), True)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("jump", [4.5, 5.5, 7.0, 90.0, 200.0, 2000.0])
@pytest.mark.parametrize("whole", [False, True])
def test_a_late_key_raises_the_maximum(fa_lib, jump, whole, dtype):
    """One key of the third block (every column of it, one to a head), or all of
    them, scores `jump` above the rest: past the point where the old maximum will
    do, past 2^128 where an exponential on the FMA pipe is anything, or just
    below. q is a unit vector, so scores are k's first column, without rounding."""
    B, H, Sq, Sk, D, Dv = 4, 32, 32, 512, 8, 16
    q, k, v, lam, _ = case(B, Sq, Sk, H, H, D, Dv, dtype, 31)
    q.zero_()
    q[..., 0] = 1
    k.clamp_(-1, 1)
    for b in range(B):
        for h in range(H):
            col = b * H + h
            for c in range(2):
                at = slice(256, 384) if whole else 256 + (col if c == 0 else 127 - col)
                k[b, at, h, c, 0] = jump
    u, t = ROUND[dtype]
    want = differential(np64(q), np64(k), np64(v), np64(lam), 1.0, False, None, u=u, t=t)
    o, lse, o2 = fa.diff_forward(*(x.cuda() for x in (q, k, v, lam)), scale=1.0, need_o2=True)
    status_clear()
    check_lse(lse, want["lse"])
    within("o", o, want["o"], want["o_bound"])
    within("o2", o2, want["o2"], want["o2_bound"])


def test_strided_views_and_given_outputs(fa_lib):
    """q, k, v as slices of one projection, gradients into slices of another."""
    B, S, H, D, Dv = 2, 140, 2, 64, 128
    u, t = ROUND[torch.bfloat16]
    x = torch.randn((B, S, H, 4 * D + Dv), generator=torch.Generator().manual_seed(3)).to(torch.bfloat16)
    lam = torch.full((H,), 0.4)
    cut = lambda y: (y[..., :2 * D].unflatten(-1, (2, D)), y[..., 2 * D:4 * D].unflatten(-1, (2, D)),  # noqa: E731
                     y[..., 4 * D:])
    do = torch.randn((B, S, H, Dv), generator=torch.Generator().manual_seed(4)).to(torch.bfloat16)
    q, k, v = cut(x)
    want = differential(np64(q), np64(k), np64(v), np64(lam), D ** -0.5, True, np64(do), u=u, t=t)
    xc, gx = x.cuda(), torch.full_like(x, float("nan"), device="cuda")
    q, k, v = cut(xc)
    dq, dk, dv = cut(gx)
    o, lse, o2 = fa.diff_forward(q, k, v, lam.cuda(), causal=True, need_o2=True)
    fa.diff_backward(q, k, v, lam.cuda(), o, o2, lse, do.cuda(), causal=True, dq=dq, dk=dk, dv=dv)
    status_clear()
    for name, got in (("o", o), ("dq", dq), ("dk", dk), ("dv", dv)):
        within(name, got, want[name], want[name + "_bound"])
    assert torch.isfinite(gx).all()


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("Sq,Sk", [(1, 700), (5, 300), (130, 257)])
def test_key_lengths(fa_lib, Sq, Sk, causal):
    """Each batch entry has a length of its own, 0 and Sk among them; what lies behind it may be NaN or inf."""
    lens = [0, 1, 5, 128, 129, Sk - 1, Sk, Sk + 50]
    used = [min(n, Sk) for n in lens]
    B, H, Hk, D, Dv = len(lens), 4, 2, 64, 128
    dtype = torch.bfloat16
    u, t = ROUND[dtype]
    q, k, v, lam, _ = case(B, Sq, Sk, H, Hk, D, Dv, dtype, 21 + Sq, "head", torch.float32)
    want = differential(np64(q), np64(k), np64(v), np64(lam), D ** -0.5, causal, n_keys=used, u=u, t=t)
    for b, n in enumerate(used):
        k[b, n:], v[b, n:] = float("nan"), float("inf")
    o, lse, o2 = fa.diff_forward(q.cuda(), k.cuda(), v.cuda(), lam.cuda(), causal=causal, need_o2=True,
                                 k_lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    status_clear()
    check_lse(lse, want["lse"])
    within("o", o, want["o"], want["o_bound"])
    within("o2", o2, want["o2"], want["o2_bound"])


@pytest.mark.parametrize("Dv", [64, 128])
@pytest.mark.parametrize("Sq,H,Hk", [(1, 8, 8), (3, 4, 2), (16, 4, 1)])
@pytest.mark.parametrize("Sk", [128, 300, 640, 1000])
def test_entries_shared_by_a_cluster(fa_lib, Sk, Sq, H, Hk, Dv):
    """Caches whose keys 1, 2, 4 or 8 CTAs take together: lengths that leave some of
    them, or all, without a key, and lengths that end inside a unit of 64. The
    same call in a graph, replayed, gives the same bits."""
    lens = [0, 1, 63, 64, 65, Sk - 1, Sk]
    B, D, dtype = len(lens), 64, torch.float16
    u, t = ROUND[dtype]
    q, k, v, lam, _ = case(B, Sq, Sk, H, Hk, D, Dv, dtype, 41 + Sk, "head", torch.float32)
    want = differential(np64(q), np64(k), np64(v), np64(lam), D ** -0.5, True, n_keys=lens, u=u, t=t)
    for b, n in enumerate(lens):
        k[b, n:], v[b, n:] = float("nan"), float("inf")
    x = [y.cuda() for y in (q, k, v, lam)]
    kw = dict(causal=True, need_o2=True, k_lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    o, lse, o2 = fa.diff_forward(*x, **kw)
    status_clear()
    check_lse(lse, want["lse"])
    within("o", o, want["o"], want["o_bound"])
    within("o2", o2, want["o2"], want["o2_bound"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = fa.diff_forward(*x, **kw)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    status_clear()
    assert all(torch.equal(g, w) for g, w in zip(again, (o, lse, o2)))


ROWS = [  # B, Sq, Sk, H, Hk, D, Dv, dtype, causal: few rows over many keys
    (1, 1, 16, 1, 1, 64, 128, torch.bfloat16, False),
    (1, 1, 129, 8, 8, 64, 128, torch.float16, True),
    (2, 3, 5000, 8, 2, 64, 128, torch.bfloat16, True),     # 12 rows a key head, many runs
    (1, 16, 1111, 4, 1, 64, 64, torch.float16, True),      # 64 rows: four row tiles
    (3, 7, 333, 6, 2, 40, 80, torch.bfloat16, False),      # 21 rows: a ragged second tile
    (1, 16, 8, 3, 3, 16, 8, torch.float16, True),          # fewer keys than rows
    (1, 17, 700, 4, 1, 64, 128, torch.bfloat16, True),     # one row more than the few-row form takes
    (40, 2, 200, 4, 4, 8, 128, torch.bfloat16, True),
]


@pytest.mark.parametrize("c", ROWS, ids=lambda c: f"B{c[0]}q{c[1]}k{c[2]}h{c[3]}-{c[4]}d{c[5]}-{c[6]}c{int(c[8])}")
def test_few_rows(fa_lib, c):
    B, Sq, Sk, H, Hk, D, Dv, dtype, causal = c
    u, t = ROUND[dtype]
    q, k, v, lam, _ = case(B, Sq, Sk, H, Hk, D, Dv, dtype, 40 + Sk, "token")
    want = differential(np64(q), np64(k), np64(v), np64(lam), D ** -0.5, causal, u=u, t=t)
    o, lse, o2 = fa.diff_forward(q.cuda(), k.cuda(), v.cuda(), lam.cuda(), causal=causal, need_o2=True)
    status_clear()
    check_lse(lse, want["lse"])
    within("o", o, want["o"], want["o_bound"])
    within("o2", o2, want["o2"], want["o2_bound"])
    close_in_norm("o", o, want["o"], 4 * u)


def test_many_ragged_lengths(fa_lib):
    """Stretches of the line that cross batch entries, entries of length 0 among them, in a row and at the ends."""
    g = torch.Generator().manual_seed(5)
    for B, Sq, Sk, H, Hk, low in ((70, 1, 900, 4, 2, 0), (33, 2, 400, 3, 1, 300), (5, 1, 2600, 16, 16, 0)):
        lens = torch.randint(low, Sk + 1, (B,), generator=g, dtype=torch.int32)
        lens[torch.randint(0, B, (B // 4,), generator=g)] = 0
        lens[0] = lens[-1] = 0
        u, t = ROUND[torch.float16]
        q, k, v, lam, _ = case(B, Sq, Sk, H, Hk, 64, 64, torch.float16, B, "head", torch.float32)
        want = differential(np64(q), np64(k), np64(v), np64(lam), 0.125, True, n_keys=lens.tolist(), u=u, t=t)
        o, lse, _ = fa.diff_forward(q.cuda(), k.cuda(), v.cuda(), lam.cuda(), causal=True, k_lens=lens.cuda())
        status_clear()
        check_lse(lse, want["lse"])
        within("o", o, want["o"], want["o_bound"])
    # no keys at all
    o, lse, _ = fa.diff_forward(q.cuda(), k.cuda(), v.cuda(), lam.cuda(), k_lens=torch.zeros_like(lens).cuda())
    status_clear()
    assert (o == 0).all() and torch.isneginf(lse).all()


def test_autograd_against_differences(fa_lib):
    """The gradients against central differences of the oracle along random directions."""
    c = case(1, 70, 90, 2, 1, 64, 128, torch.float16, 31, "head", torch.float32)
    q, k, v, lam, do = c
    leaves = [x.cuda().requires_grad_() for x in (q, k, v, lam)]
    o = diff_attn_func(*leaves, causal=True)
    grads = torch.autograd.grad(o, leaves, do.cuda())
    status_clear()
    rng = np.random.default_rng(1)
    base = [np64(x) for x in (q, k, v, lam)]
    loss = lambda xs: float((differential(*xs, 64 ** -0.5, True)["o"] * np64(do)).sum())  # noqa: E731
    for i, g in enumerate(grads):
        d = rng.standard_normal(base[i].shape)
        h = 1e-5
        plus, minus = list(base), list(base)
        plus[i], minus[i] = base[i] + h * d, base[i] - h * d
        slope = (loss(plus) - loss(minus)) / (2 * h)
        # The gradient's roundings (within 4 u in norm), random against d.
        tol = 4 * 2.0 ** -11 * np.linalg.norm(np64(g)) * 6 + 1e-3
        assert abs(slope - float((np64(g) * d).sum())) <= tol, i
