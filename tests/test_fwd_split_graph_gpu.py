"""The key-range split under graph replay: every replay of a captured launch carries
the same epoch, so a ticket that kept it would pair a CTA with its partner's partial
result of the replay before."""
import pytest
import torch

from exact_io_aware_96_b200 import fa

pytestmark = pytest.mark.gpu


def inputs(seed, B=2, S=1000, H=4, D=128):
    g = torch.Generator("cuda").manual_seed(seed)
    return [torch.randn((B, S, H, D), generator=g, device="cuda").to(torch.bfloat16) for _ in range(3)]


@pytest.mark.parametrize("causal", [False, True])
def test_tickets_are_clear_after_a_launch(fa_lib, causal):
    q, k, v = inputs(1)
    n, ns = fa.fwd_workspace_size(2, 4, 1000, 1000, 128, causal, 64)
    assert ns > 0
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        fa.forward(q, k, v, causal=causal, split_ranks=64, workspace=ws)
        torch.cuda.synchronize()
        assert (ws[:2 * 4 * ns * 8] == 0).all()  # a ticket of 8 bytes per split (b, h, rank)


@pytest.mark.parametrize("causal", [False, True])
def test_replays_on_new_inputs(fa_lib, causal):
    sets = [inputs(i) for i in range(3)]
    n, ns = fa.fwd_workspace_size(2, 4, 1000, 1000, 128, causal, 64)
    want = [fa.forward(*x, causal=causal, split_ranks=64) for x in sets]
    live, ws = [x.clone() for x in sets[0]], torch.empty(n, dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = fa.forward(*live, causal=causal, split_ranks=64, workspace=ws)
    off = 2 * 4 * ns * 8
    for i in (0, 1, 2, 0, 2, 1) * 5:
        for dst, src in zip(live, sets[i]):
            dst.copy_(src)
        ws[off:].fill_(255)  # the partial results of the replay before are NaN
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want[i]))
    assert fa.fa_last_device_status()[0] == 0
