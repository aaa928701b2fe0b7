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
