"""The 8-bit layer state at sizes far from one, with scales that the reference gives, and
the exact workspace of its backward."""
import pytest
import torch

import reference64 as ref
from helpers import require_gpu
from test_gpu_ckpt import backward, case, check_backward, check_forward, forward, status_ok

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("std", [1e-20, 1e-15, 300.0, 1e12])
@pytest.mark.parametrize("T,H,I,E,k", [(61, 128, 64, 4, 2), (700, 264, 200, 3, 2)])
def test_scales_follow_the_sizes(T, H, I, E, k, std):
    """Scale bytes within the reference's, on swap-AB and on token-major tiles; and the
    backward where its products are neither denormal nor saturate the sigmoid's bound."""
    require_gpu()
    d = case(T, H, I, E, k, std=std)
    out, st = forward(d)
    status_ok()
    check_forward(d, out, st)
    if 1e-15 <= std <= 300:
        g = backward(d, st)
        status_ok()
        check_backward(d, st, g)


def test_a_scale_that_is_too_large_is_not_accepted():
    """What check_forward holds the bytes to: 20 steps too far is outside, all zeros or not."""
    x = torch.randn(4, 64, dtype=torch.float64) * 1e-20
    _, bytes_ = ref.quantize(x)
    mag = ref.split_blocks(x.abs(), 1)[0].amax(dim=2)
    hi = ref.exponents(mag * (1 + 2.0 ** -10)) + 127
    assert bool((bytes_ <= hi).all()) and bool((bytes_.int() + 20 > hi).all())


@pytest.mark.parametrize("T,H,I,E,k", [(1, 8, 8, 1, 1), (61, 128, 256, 8, 2), (300, 264, 104, 16, 3)])
def test_the_workspace_is_as_large_as_asked_for(T, H, I, E, k):
    """Exactly the size asked for is enough, and nothing past it is written; one byte less is refused."""
    require_gpu()
    import routing_grouped_gemm_score_b200 as m
    d = case(T, H, I, E, k)
    _, st = forward(d)
    want = backward(d, st)
    n = m.lib().moe_grouped_mlp_backward_ckpt_workspace_size(T, H, I, E, k)
    # at least the padded rows in bf16 (x, [dg | du], h), a weight and a sum a row, and the two row maps
    rows = T * k + 15 * min(E, T * k)
    assert n >= rows * (2 * (H + 3 * I) + 4 + 4 * -(-I // 64) + 4) + 4 * (E + 1) + 4 * T * k
    memory = torch.full((n + 4096,), 171, dtype=torch.uint8, device="cuda")
    ws = m.LayerWorkspace(T, H, I, E, k, backward=True, ckpt=True)
    ws.bwd8 = memory[:n]
    got = backward(d, st, workspace=ws)
    status_ok()
    for name in want:
        assert torch.equal(got[name], want[name]), name
    assert bool((memory[n:] == 171).all())
    ws.bwd8 = memory[:n - 1]
    with pytest.raises(m.MoEError, match="WORKSPACE"):
        backward(d, st, workspace=ws)


def test_no_tokens_need_no_workspace():
    require_gpu()
    import routing_grouped_gemm_score_b200 as m
    gu, down = (torch.ones(2, 64, n, dtype=torch.bfloat16, device="cuda") for n in (32, 16))
    down = down.reshape(2, 16, 64)
    s = m.lib().moe_grouped_mlp_backward_ckpt(None, 0, 64, 16, 2, 1, *[None] * 9, None, gu.data_ptr(), down.data_ptr(),
                                              None, None, 0, torch.cuda.current_stream().cuda_stream)
    assert s == 0 and not gu.any() and not down.any()
