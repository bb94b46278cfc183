"""Calls on a stream of their own while the current one is busy, and outputs that
start as NaN inside guard bands: every element is written, and no other."""
import pytest
import torch

from exact_io_aware_96_b200 import fa
from tests.test_differential_gpu import CASES, IDS, case, status_clear

pytestmark = pytest.mark.gpu
SECTIONS = (8, 12, 12)


@pytest.mark.parametrize("raw", [False, True])
def test_a_given_stream_does_not_wait_for_the_current_one(fa_lib, raw):
    """The current stream sleeps all along: were a call launched there, or behind an
    event of it, its results would not be there before the sleep ends."""
    q, k, v, lam, do = (x.cuda() for x in case(1, 300, 300, 2, 2, 64, 128, torch.bfloat16, 81))
    pos = torch.arange(300, device="cuda", dtype=torch.int32)[None, None].expand(3, 1, 300)
    f = fa.rotary_inv_freq(SECTIONS)

    def calls(**kw):
        r = fa.rotary(q, k, pos, f, SECTIONS, **kw)
        o, lse, o2 = fa.diff_forward(q, k, v, lam, need_o2=True, **kw)
        g = fa.diff_backward(q, k, v, lam, o, o2, lse, do, deterministic=True, **kw)
        one, l1, _ = fa.diff_forward(q[:, :1], k, v, lam[:, :1], **kw)
        return (*r, o, lse, o2, *g, one, l1)

    want = [x.cpu() for x in calls()]
    side = torch.cuda.Stream()
    calls(stream=side)  # the side stream's memory pool and kernels are set up
    torch.cuda.synchronize()
    asleep = torch.cuda.Event()
    torch.cuda._sleep(2_000_000_000)  # about a second
    asleep.record()
    got = calls(stream=side.cuda_stream if raw else side)
    side.synchronize()
    with torch.cuda.stream(side):  # copied while the current stream still sleeps
        got = [x.cpu() for x in got]
    assert not asleep.query(), "the sleep ended before the copies: nothing is shown"
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    torch.cuda.synchronize()
    status_clear()


def banded(t):
    """A NaN view of t's shape inside a buffer of 123: rows and columns of margin on every side."""
    shape = list(t.shape)
    big = torch.full([n + 2 for n in shape[:-1]] + [shape[-1] + 16], 123.0, dtype=t.dtype, device=t.device)
    view = big[tuple(slice(1, -1) for _ in shape[:-1]) + (slice(8, -8),)]
    view.fill_(float("nan"))
    return big, view


@pytest.mark.parametrize("c", [CASES[3], CASES[6], CASES[7], (2, 2, 700, 4, 2, 40, 72, torch.bfloat16, True, "head"),
                               (2, 1, 500, 4, 4, 64, 128, torch.float16, True, "head")],
                         ids=[IDS[3], IDS[6], IDS[7], "rows", "cluster"])
def test_every_element_of_the_outputs_is_written(fa_lib, c):
    B, Sq, Sk, H, Hk, D, Dv, dtype, causal, lam = c
    q, k, v, w, do = (x.cuda() for x in case(B, Sq, Sk, H, Hk, D, Dv, dtype, 7, lam))
    bands = {}

    def out(name, like):
        bands[name] = banded(like)
        return bands[name][1]

    want = dict(zip(("o", "lse", "o2"), fa.diff_forward(q, k, v, w, causal=causal, need_o2=True)))
    want.update(zip(("dq", "dk", "dv", "dlam"), fa.diff_backward(q, k, v, w, want["o"], want["o2"], want["lse"], do,
                                                                 causal=causal, deterministic=True)))
    lse = torch.full_like(want["lse"], float("nan"))
    dlam = torch.full_like(want["dlam"], float("nan"))
    fa.diff_forward(q, k, v, w, causal=causal, out=out("o", want["o"]), out2=out("o2", want["o2"]), lse=lse)
    fa.diff_backward(q, k, v, w, want["o"], want["o2"], want["lse"], do, causal=causal, dq=out("dq", q), dk=out("dk", k),
                     dv=out("dv", v), dlam=dlam, deterministic=True)
    status_clear()
    assert torch.equal(lse, want["lse"]) and torch.equal(dlam, want["dlam"])
    for name, (big, view) in bands.items():
        assert torch.equal(view, want[name]), name
        view.fill_(123.0)
        assert (big == 123.0).all(), name


@pytest.mark.parametrize("D,sections,inter", [(64, SECTIONS, False), (80, (5, 3, 9), False), (80, (5, 3, 9), True)])
def test_every_element_of_the_turned_tensors_is_written(fa_lib, D, sections, inter):
    q, k = (torch.randn((2, 77, h, D), device="cuda").half() for h in (3, 2))
    pos = torch.arange(77, device="cuda")[None, None].expand(3, 2, 77)
    f = fa.rotary_inv_freq(sections)
    want = fa.rotary(q, k, pos, f, sections, interleaved=inter)
    bands = [banded(q), banded(k)]
    fa.rotary(q, k, pos, f, sections, interleaved=inter, out_q=bands[0][1], out_k=bands[1][1])
    status_clear()
    for (big, view), w in zip(bands, want):
        assert torch.equal(view, w)
        view.fill_(123.0)
        assert (big == 123.0).all()
