"""The 8-bit layer state at the limits of E and k, and small batches captured in a graph."""
import pytest
import torch

from helpers import require_gpu
from test_gpu_ckpt import backward, case, check_backward, check_forward, forward, opts, status_ok

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,H,I,E,k", [(1, 64, 32, 256, 16), (5, 72, 40, 256, 16), (300, 64, 72, 256, 16),
                                       (2100, 64, 32, 256, 1), (40, 64, 32, 16, 16)])
def test_most_experts_and_choices(T, H, I, E, k):
    require_gpu()
    d = case(T, H, I, E, k, sigmoid=k == 1)
    out, st = forward(d)
    status_ok()
    check_forward(d, out, st)
    g = backward(d, st)
    status_ok()
    check_backward(d, st, g)


# the router moves the rows itself; so it does not at T = 9; the MLP in one launch
@pytest.mark.parametrize("T,H,I,E,k", [(1, 128, 64, 8, 2), (8, 128, 64, 8, 2), (9, 128, 64, 8, 2), (64, 128, 256, 40, 2)])
def test_small_batches_captured(T, H, I, E, k):
    require_gpu()
    import routing_grouped_gemm_score_b200 as m
    d, other = case(T, H, I, E, k), case(T, H, I, E, k, seed=1)
    c = d["cuda"]
    w = (c["w_gate_up"], c["w_down"])

    def step(logits, x, dout):
        out, st = m.moe_layer_forward_ckpt(logits, x, *w, k, opts(d))
        return [out, *st.values(), *m.moe_grouped_mlp_backward_ckpt(dout, st, *w).values()]

    ins = [[b[n] for n in ("logits", "x", "dout")] for b in (c, other["cuda"])]
    want = [[t.clone() for t in step(*i)] for i in ins]
    held = [t.clone() for t in ins[0]]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*held)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(*held)
    for i in (0, 1, 0):
        for h, t in zip(held, ins[i]):
            h.copy_(t)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(got, want[i]))
    status_ok()
