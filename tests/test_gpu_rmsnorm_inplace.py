"""moe_rmsnorm on its own inputs' memory: what is kept and what is refused."""
import pytest
import torch

from helpers import require_gpu
from test_gpu_rmsnorm import EPS, inputs

pytestmark = pytest.mark.gpu


def test_y_may_not_replace_the_sum():
    require_gpu()
    import routing_grouped_gemm_score_b200 as m
    d = {n: t.cuda() for n, t in inputs(37, 264, 3).items()}
    x, res = d["x"].clone(), d["r"].clone()
    for both in (x, res, torch.empty_like(x)):
        with pytest.raises(m.MoEError, match="INVALID_ARG"):
            m.moe_rmsnorm(x, d["w"], EPS, residual=res, out={"sum": both, "y": both})
    assert torch.equal(x, d["x"]) and torch.equal(res, d["r"])   # nothing was launched
    # next to each other in one allocation they do not overlap
    both = torch.empty(2, *x.shape, dtype=x.dtype, device="cuda")
    want = m.moe_rmsnorm(x, d["w"], EPS, residual=res)
    got = m.moe_rmsnorm(x, d["w"], EPS, residual=res, out={"sum": both[0], "y": both[1]})
    assert torch.equal(got["sum"], want["sum"]) and torch.equal(got["y"], want["y"])


def test_y_over_x_leaves_no_sum():
    """Without a residual the sum is x itself; where y replaced it, there is none."""
    require_gpu()
    import routing_grouped_gemm_score_b200 as m
    d = {n: t.cuda() for n, t in inputs(37, 264, 4).items()}
    want = m.moe_rmsnorm(d["x"], d["w"], EPS)
    assert want["sum"] is d["x"]
    x = d["x"].clone()
    got = m.moe_rmsnorm(x, d["w"], EPS, out={"y": x})
    assert got["sum"] is None and got["y"] is x
    assert torch.equal(x, want["y"]) and torch.equal(got["rstd"], want["rstd"])
    other = torch.empty_like(x)
    assert m.moe_rmsnorm(d["x"], d["w"], EPS, out={"y": other})["sum"] is d["x"]
    none = torch.empty(0, 264, dtype=x.dtype, device="cuda")
    assert m.moe_rmsnorm(none, d["w"], EPS, out={"y": none})["sum"] is none
