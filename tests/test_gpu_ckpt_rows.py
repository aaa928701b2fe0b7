"""moe_grouped_mlp_backward_ckpt with wrong rows: an assignment whose row is out of range
has no part in any gradient, whatever the workspace held before."""
import pytest
import torch

import reference64 as ref
from helpers import force_kernels, require_gpu
from test_gpu_ckpt import backward, case, forward, status_ok

pytestmark = pytest.mark.gpu


def check_without(d, st, g, dropped):
    """g against the 64-bit gradients of the assignments that are not dropped: each as a
    token of its own, with the dropped ones' dout zero."""
    x = ref.decode(st["x_q"].cpu(), st["x_scale"].cpu())
    gu = ref.decode(st["gu_q"].cpu(), st["gu_scale"].cpu().t(), 2)
    T, k = st["row_of"].shape
    dout = d["dout"].double().repeat_interleave(k, dim=0)
    for t, j in dropped:
        dout[t * k + j] = 0.0
    r = ref.layer_backward(dout, x.repeat_interleave(k, dim=0), gu, st["topk_prob"].cpu().double().reshape(-1, 1),
                           d["w_gate_up"].double(), d["w_down"].double(), st["row_of"].cpu().reshape(-1, 1),
                           st["offsets"].cpu())
    for n in ("dw_down", "dw_gate_up"):
        ref.assert_within(g[n], r[n], r[n + "_tol"], n)
    ref.assert_within(g["dprob"], r["dprob"].reshape(T, k), r["dprob_tol"].reshape(T, k), "dprob")
    dx, tol = (r[n].reshape(T, k, -1).sum(dim=1) for n in ("dx", "dx_tol"))   # a token's sum is rounded once more
    ref.assert_within(g["dx"], dx, tol + ref.BF16 * (dx.abs() + tol), "dx")
    for t, j in dropped:
        assert float(g["dprob"][t, j]) == 0.0


# single-CTA and pair tiles; blocks of several tiles; rows of no whole number of anything
@pytest.mark.parametrize("tiles", ["single", "pair"])
@pytest.mark.parametrize("T,H,I,E,k", [(61, 128, 64, 4, 2), (300, 264, 328, 3, 2), (40, 200, 40, 16, 4), (700, 96, 64, 2, 1)])
@pytest.mark.parametrize("before", ["NaN", "another call", "the call without the fault"])
def test_rows_out_of_range_are_left_out(T, H, I, E, k, tiles, before):
    require_gpu()
    import routing_grouped_gemm_score_b200 as m
    d = case(T, H, I, E, k)
    force_kernels(gemm_tiles=tiles)
    _, st = forward(d)
    ws = m.LayerWorkspace(T, H, I, E, k, backward=True, ckpt=True)
    dropped = [(3, k - 1), (4, 0), (T - 1, 0)]
    bad = dict(st, row_of=st["row_of"].clone())
    for (t, j), row in zip(dropped, (-1, T * k, 2 ** 31 - 1)):
        bad["row_of"][t, j] = row
    if before == "NaN":
        ws.bwd8.fill_(255)
    elif before == "another call":
        other = case(T, H, I, E, k, seed=1)
        backward(other, forward(other)[1], workspace=ws)
    else:
        backward(d, st, workspace=ws)
    status_ok()
    g = backward(d, bad, workspace=ws)
    assert m.moe_get_device_status() == m.MOE_ERR_DEVICE_CHECK
    check_without(d, st, g, dropped)
    full = backward(d, st, workspace=ws)
    status_ok()
    check_without(d, st, full, [])


def test_a_row_given_twice_is_reported():
    require_gpu()
    import routing_grouped_gemm_score_b200 as m
    T, H, I, E, k = 61, 128, 64, 4, 2
    d = case(T, H, I, E, k)
    _, st = forward(d)
    ws = m.LayerWorkspace(T, H, I, E, k, backward=True, ckpt=True)
    want = backward(d, st, workspace=ws)
    bad = dict(st, row_of=st["row_of"].clone())
    bad["row_of"][7, 0] = bad["row_of"][9, 1]
    got = backward(d, bad, workspace=ws)
    assert m.moe_get_device_status() == m.MOE_ERR_DEVICE_CHECK
    rest = [t for t in range(T) if t not in (7, 9)]   # the other tokens' rows are their own
    assert torch.equal(got["dx"][rest], want["dx"][rest]) and torch.equal(got["dprob"][rest], want["dprob"][rest])
    backward(d, st, workspace=ws)
    status_ok()
