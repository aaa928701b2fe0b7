"""moe_quantize_rows and moe_dequantize_rows against the 64-bit format, bit for bit."""
import pytest
import torch

import reference64 as ref
from helpers import require_gpu

pytestmark = pytest.mark.gpu


def rows(R, width, seed, wide=False):
    g = torch.Generator().manual_seed(seed)
    v = torch.randn(R, width, generator=g)
    if wide:   # every size that bf16 has, denormals among them
        v = v * torch.exp2(torch.randint(-130, 125, (R, width), generator=g).float())
    return v.to(torch.bfloat16)


def check(x, parts, block_major):
    import routing_grouped_gemm_score_b200 as m
    want, bytes_ = ref.quantize(x.double(), parts)
    q, scale = m.moe_quantize_rows(x.cuda(), parts, block_major)
    back = m.moe_dequantize_rows(q, scale, parts, block_major)
    s = scale.cpu().t() if block_major else scale.cpu()
    assert torch.equal(s, bytes_)
    ref.assert_within(ref.decode(q.cpu(), s, parts), want, torch.zeros_like(want), "stored values")
    ref.assert_within(back, want, torch.zeros_like(want), "values read back")
    fin = torch.isfinite(x.double())
    tol = ref.BF16 * 16 * x.double().abs() + 2.0 ** -10 * ref.per_column(
        torch.exp2(bytes_.double() - 127), x.shape[1] // parts, parts)
    ref.assert_within(back.cpu()[fin], x.double()[fin], tol[fin], "the format's error")


@pytest.mark.parametrize("R,cols,parts,block_major", [
    (1, 8, 1, 0), (1, 32, 1, 1), (3, 40, 2, 1), (5, 1000, 1, 0), (37, 768, 2, 1), (64, 2048, 1, 0),
    (7, 4104, 2, 0), (300, 24, 2, 1), (2, 5120, 1, 1)])
@pytest.mark.parametrize("wide", [False, True])
def test_rows(R, cols, parts, block_major, wide):
    require_gpu()
    check(rows(R, parts * cols, R + cols, wide), parts, bool(block_major))


def test_borders_and_special_values():
    """A block's largest magnitude at and next to 448 * 2^e, ties between two E4M3
    values, zeros of both signs, infinities and NaN."""
    require_gpu()
    x = torch.zeros(12, 64)
    x[0, 0], x[1, 0], x[2, 0] = 448.0, 450.0, 446.0                    # 1.75 * 2^8 and its bf16 neighbours
    x[3, :16] = torch.arange(16) / 16 + 1                              # ties of 3 fraction bits
    x[3, 31] = 448.0
    x[4, 5], x[4, 6] = float("inf"), 3.0
    x[5, 5], x[5, 40] = float("nan"), -7.0
    x[6] = -0.0
    x[7, 0], x[7, 33] = 3.3895e38, -3.3895e38                          # the largest bf16
    x[8, 0], x[8, 33] = 2.0 ** -133, -(2.0 ** -126)                    # the smallest bf16
    x[9] = float("inf")
    x[10, ::2] = float("-inf")
    x[11, 0], x[11, 1] = 448.0 * 2.0 ** -124, 2.0 ** -133              # the smallest exponent
    check(x.to(torch.bfloat16), 1, False)
    check(x.to(torch.bfloat16), 2, True)


def test_no_rows_and_large_offsets():
    require_gpu()
    import routing_grouped_gemm_score_b200 as m
    q, s = m.moe_quantize_rows(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"))
    assert q.shape == (0, 64) and s.shape == (0, 2)
    assert m.moe_dequantize_rows(q, s).shape == (0, 64)
    R, cols = (1 << 18) + 3, 8192                                      # more than 2^31 elements
    x = torch.zeros(R, cols, dtype=torch.bfloat16, device="cuda")
    last = rows(2, cols, 9)
    x[-2:] = last.cuda()
    for block_major in (False, True):
        q, s = m.moe_quantize_rows(x, 1, block_major)
        want, bytes_ = ref.quantize(last.double())
        assert torch.equal((s[:, -2:].t() if block_major else s[-2:]).cpu(), bytes_)
        back = m.moe_dequantize_rows(q, s, 1, block_major)
        ref.assert_within(back[-2:], want, torch.zeros_like(want), "last rows")
        assert not back[:-2].any()
        del q, s, back
