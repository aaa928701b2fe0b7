"""moe_rmsnorm row by row: a row's bits are its own, whatever batch it stands in."""
import pytest
import torch

import reference64 as ref
from helpers import require_gpu
from test_gpu_rmsnorm import EPS, RSTD

pytestmark = pytest.mark.gpu


def batch(T, H, seed):
    g = torch.Generator().manual_seed(seed + H)
    size = torch.exp(torch.randn(T, 1, generator=g))
    return ((size * torch.randn(T, H, generator=g)).to(torch.bfloat16).cuda(),
            torch.randn(T, H, generator=g).to(torch.bfloat16).cuda(),
            (1 + 0.3 * torch.randn(H, generator=g)).to(torch.bfloat16).cuda())


# each number of columns a thread takes, for few rows and for many; groups of 32 chunks that end anywhere
@pytest.mark.parametrize("H", [8, 264, 1000, 1032, 2048, 2056, 4096, 4104, 5120, 8192, 8200, 12296, 16384])
def test_a_row_alone_and_in_a_batch(H):
    require_gpu()
    import routing_grouped_gemm_score_b200 as m
    T = 400                                       # more rows than the GPU has SMs
    x, r, w = batch(T, H, 1)
    many = m.moe_rmsnorm(x, w, EPS, residual=r, quantize=True)
    rows = range(0, T, 3)
    alone = [m.moe_rmsnorm(x[i:i + 1], w, EPS, residual=r[i:i + 1], quantize=True) for i in rows]
    for n in many:
        assert torch.equal(torch.cat([a[n] for a in alone]), many[n][::3]), n
    s = many["sum"].double().cpu()
    _, rstd = ref.rmsnorm(s, w.cpu().double(), EPS)
    ref.assert_within(many["rstd"], rstd, RSTD * rstd, "rstd")
    # and its gradient, which depends on the row alone as well
    some = m.moe_rmsnorm_backward(r, many["sum"], w, many["rstd"])
    one = [m.moe_rmsnorm_backward(r[i:i + 1], a["sum"], w, a["rstd"]) for i, a in zip(rows, alone)]
    assert torch.equal(torch.cat([o["dx"] for o in one]), some["dx"][::3])
