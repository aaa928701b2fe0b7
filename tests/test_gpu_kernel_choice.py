"""Which kernels a call launches, as the profiler names them: the calls that keep no
8-bit state neither carry its store nor take other tiles because of it."""
import pytest
import torch

from helpers import require_gpu
from test_gpu_ckpt import backward, case, forward, opts

pytestmark = pytest.mark.gpu


def launched(call):
    """Names of the library's kernels that call() launches, in order."""
    from torch.profiler import ProfilerActivity, profile
    call()   # modules loaded, limits set
    torch.cuda.synchronize()
    with profile(activities=[ProfilerActivity.CUDA]) as p:
        call()
        torch.cuda.synchronize()
    kernels = [e for e in p.events() if "CUDA" in str(e.device_type) and "moe::" in e.name]
    if not kernels:
        pytest.skip("the profiler sees no kernels here")
    return [e.name for e in sorted(kernels, key=lambda e: e.time_range.start)]


# swap-AB tiles in two launches; in one launch; 16 rows a tile; single-CTA tiles; CTA pairs
@pytest.mark.parametrize("T,H,I,E,k", [(64, 128, 256, 8, 2), (64, 128, 256, 40, 2), (8, 128, 256, 40, 2),
                                       (700, 264, 200, 3, 2), (1500, 96, 64, 2, 2)])
def test_the_plain_forward_has_kernels_of_its_own(T, H, I, E, k):
    require_gpu()
    import routing_grouped_gemm_score_b200 as m
    d = case(T, H, I, E, k)
    c = d["cuda"]
    plain = launched(lambda: m.moe_layer_forward(c["logits"], c["x"], c["w_gate_up"], c["w_down"], k, opts(d)))
    ckpt = launched(lambda: forward(d))
    gemms = [n for n in plain if "gemm" in n]
    assert len(gemms) in (1, 2)   # one launch for the MLP, or gate_up and down
    assert len([n for n in gemms if n in ckpt]) == len(gemms) - 1   # the down GEMM alone is the same


# rows an expert: the gate_up dgrad takes CTA pairs where the other group-M products do,
# in every backward (from 1024 rows an expert on)
@pytest.mark.parametrize("T,E,k,pairs", [(512, 4, 2, 0), (1024, 4, 2, 0), (1500, 2, 2, 2)])
def test_tiles_of_the_dgrads(T, E, k, pairs):
    require_gpu()
    import routing_grouped_gemm_score_b200 as m
    H, I = 128, 64
    d = case(T, H, I, E, k)
    c = d["cuda"]
    w = (c["w_gate_up"], c["w_down"])
    _, st = m.moe_layer_forward(c["logits"], c["x"], *w, k, opts(d), save_for_backward=True)
    p = m.moe_permute(c["x"], st["topk_idx"], st["offsets"])
    scale = torch.empty(T * k, device="cuda")
    scale[p["row_of"].reshape(-1).long()] = st["topk_prob"].reshape(-1)
    h = m.moe_grouped_mlp_scaled(p["x_perm"], st["offsets"], *w, scale, save=True)
    _, st8 = forward(d)
    for call in (lambda: m.moe_grouped_mlp_backward(c["dout"], st, *w),
                 lambda: m.moe_grouped_mlp_scaled_backward(c["dout"], p["row_of"], p["sorted_token"], scale,
                                                           st["offsets"], p["x_perm"], h["gu"], h["h"], *w),
                 lambda: backward(d, st8)):
        assert sum("gemm_pair_kernel" in n for n in launched(call)) == pairs
