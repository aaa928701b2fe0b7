"""What moe_rmsnorm refuses beside sizes and missing pointers (addresses that are never
dereferenced, each output with its own)."""
import pytest

INVALID = 1


@pytest.fixture(scope="session")
def m():
    from routing_grouped_gemm_score_b200 import build
    build.build()
    import routing_grouped_gemm_score_b200 as m
    return m


T, H = 4, 64
SIZE = 2 * T * H
X, RESIDUAL, WEIGHT, SUM, Y, Y_Q, Y_SCALE, RSTD = ((i + 1) << 20 for i in range(8))


# the same memory; a part of it, from either side; the two ways to the same memory that are allowed alone
@pytest.mark.parametrize("s,y", [(SUM, SUM), (SUM, SUM + SIZE - 16), (SUM, SUM - SIZE + 16), (SUM, SUM + 16), (X, X),
                                 (RESIDUAL, RESIDUAL)])
def test_sum_and_y_in_the_same_memory(m, s, y):
    assert m.lib().moe_rmsnorm(X, RESIDUAL, WEIGHT, T, H, 1e-6, s, y, Y_Q, Y_SCALE, RSTD, None) == INVALID


GOOD = dict(x=X, residual=RESIDUAL, weight=WEIGHT, T=T, H=H, eps=1e-6, sum=SUM, y=Y, y_q=Y_Q, y_scale=Y_SCALE, rstd=RSTD)


# one thing wrong at a time, with every output in memory of its own
@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(T=1 << 31), dict(H=0), dict(H=-8), dict(eps=-1e-6), dict(eps=float("nan")), dict(eps=float("inf")),
    dict(x=None), dict(weight=None), dict(y=None, y_q=None, y_scale=None), dict(y_q=None), dict(y_scale=None),
    dict(residual=None), dict(x=X + 2), dict(residual=RESIDUAL + 8), dict(weight=WEIGHT + 2), dict(sum=SUM + 2),
    dict(y=Y + 8), dict(y_q=Y_Q + 8), dict(y_scale=Y_SCALE + 1), dict(rstd=RSTD + 4)])
def test_one_thing_wrong(m, bad):
    a = {**GOOD, **bad}
    assert m.lib().moe_rmsnorm(a["x"], a["residual"], a["weight"], a["T"], a["H"], a["eps"], a["sum"], a["y"], a["y_q"],
                               a["y_scale"], a["rstd"], None) == INVALID
