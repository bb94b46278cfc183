"""Calls from a host thread that has made no CUDA call before: the library binds
the device's context itself (buffers, workspace and kernel attributes are all
set up by another thread, so no other call does)."""
import threading

import pytest
import torch

from exact_io_aware_96_b200 import fa

pytestmark = pytest.mark.gpu


def in_new_thread(call):
    got = []
    t = threading.Thread(target=lambda: got.append(call()))
    t.start()
    t.join()
    return got[0]


def test_plain_forward_from_a_fresh_thread(fa_lib):
    B, S, H, D = 1, 200, 2, 64
    q = torch.randn((B, S, H, D), device="cuda").to(torch.float16)
    o, lse = fa.forward(q, q, q, split_ranks=-1)
    o2, lse2 = torch.empty_like(o), torch.empty_like(lse)
    stream = torch.cuda.current_stream().cuda_stream
    torch.cuda.synchronize()
    args = (q.data_ptr(),) * 3 + (o2.data_ptr(), lse2.data_ptr(), B, H, S, S, D, D ** -0.5, 0, fa.FA_FP16, stream)
    assert in_new_thread(lambda: fa.fa_fwd(*args)) == 0
    torch.cuda.synchronize()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_differential_forward_from_a_fresh_thread(fa_lib):
    for Sq in (1, 200):
        q = torch.randn((1, Sq, 2, 2, 64), device="cuda").to(torch.float16)
        k, v = torch.randn((1, 200, 2, 2, 64), device="cuda").half(), torch.randn((1, 200, 2, 128), device="cuda").half()
        lam = torch.full((2,), 0.5, device="cuda")
        o, lse, _ = fa.diff_forward(q, k, v, lam)
        o2, lse2 = torch.empty_like(o), torch.empty_like(lse)
        ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
        dev = (fa.FaTensor * 2)
        view = lambda t: fa.FaTensor(t.data_ptr(), t.stride(0), t.stride(1), t.stride(2))  # noqa: E731
        p = fa.DiffFwdParams(dev(view(q[:, :, :, 0]), view(q[:, :, :, 1])), dev(view(k[:, :, :, 0]), view(k[:, :, :, 1])),
                             view(v), fa.DiffLambda(lam.data_ptr(), 0, 0, 1, 1, 1, 2, fa.FA_LAMBDA_FP32), None, view(o2),
                             fa.FaTensor(), lse2.data_ptr(), 1, 2, 2, Sq, 200, 64, 128, 0.125, 0, fa.FA_FP16,
                             ws.data_ptr(), ws.numel())
        stream = torch.cuda.current_stream().cuda_stream
        torch.cuda.synchronize()
        assert in_new_thread(lambda: fa.fa_diff_fwd(p, stream)) == 0
        torch.cuda.synchronize()
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
