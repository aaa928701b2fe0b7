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


SIZES = [-133, -130, -126, -110, -80, -75, -70, -63, -52, -50, -48, -20, 0, 30, 58, 63, 64, 90, 120, 126]


# eps: none, the smallest fp32, one that counts for some of the small rows, usual ones
@pytest.mark.parametrize("eps", [0.0, 2.0 ** -149, 2.0 ** -105, 1e-12, 1e-6])
@pytest.mark.parametrize("H,copies", [(64, 1), (2048, 1), (2048, 20), (5120, 1), (5120, 20), (16384, 1)])
def test_rows_of_every_size(H, copies, eps):
    """Rows of sizes 2^-133 .. 2^126, whose squares leave fp32's range on either side."""
    require_gpu()
    import routing_grouped_gemm_score_b200 as m
    x, dy, w = batch(len(SIZES), H, 2)
    row = (x.float() / x.float().abs().amax(dim=1, keepdim=True)).double()   # magnitude 1
    x = torch.stack([r * 2.0 ** e for r, e in zip(row, SIZES)]).to(torch.bfloat16).repeat(copies, 1)
    dy = dy.repeat(copies, 1)
    r = m.moe_rmsnorm(x, w, eps, quantize=True)
    s, wd = x.double().cpu(), w.cpu().double()
    y, rstd = ref.rmsnorm(s, wd, eps)
    stored = rstd.float().double()   # as fp32 holds it: 2^-150 off where it is denormal, inf from 2^128 on
    ref.assert_within(r["rstd"], stored, RSTD * stored + 2.0 ** -149, "rstd")
    ref.assert_within(r["y"], y, (ref.BF16 + RSTD + 2 * ref.F32) * y.abs() + 2.0 ** -134, "y")
    back = ref.decode(r["y_q"].cpu(), r["y_scale"].cpu())
    unit = ref.per_column(torch.exp2(r["y_scale"].cpu().double() - 127), H)
    d = RSTD + 2 * ref.F32
    mag = ref.split_blocks(y.abs(), 1)[0].amax(dim=2)
    lo, hi = ref.exponents(mag * (1 - d)) + 127, ref.exponents(mag * (1 + d)) + 127
    assert bool(((r["y_scale"].cpu() >= lo) & (r["y_scale"].cpu() <= hi)).all())
    ref.assert_within(back, y, (2.0 ** -4 * (1 + d) + d) * y.abs() + 2.0 ** -10 * unit, "y in 8 bits")
    # the backward, which has rstd from the forward, where it is a number
    ok = torch.isfinite(r["rstd"]).cpu()
    g = m.moe_rmsnorm_backward(dy[ok.cuda()], x[ok.cuda()], w, r["rstd"][ok.cuda()])
    s, dyd, rs = s[ok], dy.cpu().double()[ok], r["rstd"].cpu().double()[ok]
    dx, dw = ref.rmsnorm_backward(dyd, s, wd, rs)
    xhat = (s * rs[:, None]).abs()
    c_abs = (wd * dyd * xhat).abs().sum(dim=1, keepdim=True) / H
    terms = rs[:, None] * ((wd * dyd).abs() + xhat * c_abs)
    tol = ref.BF16 * dx.abs() + 64 * ref.F32 * terms + 2.0 ** -134
    got = g["dx"].cpu().double()
    # rstd is up to 2^128, so some gradients pass bf16's largest value, 2^128 - 2^119, which is stored as an infinity
    past = dx.abs() + tol >= torch.finfo(torch.bfloat16).max
    ref.assert_within(got[~past], dx[~past], tol[~past], "dx")
    assert bool(((got - dx).abs() <= tol)[past].logical_or(got[past] == dx[past].sign() * float("inf")).all())
    n = int(ok.sum())
    ref.assert_within(g["dweight"], dw, (n + 64 + 2) * ref.F32 * (dyd * xhat).abs().sum(dim=0) + 2.0 ** -130, "dweight")


def test_zeros_infinities_and_one_large_value():
    require_gpu()
    import routing_grouped_gemm_score_b200 as m
    H = 264
    x, _, w = batch(8, H, 3)
    x[0] = 0.0
    x[1] = 0.0
    x[1, 7] = 2.0 ** -133                                  # one value, the smallest
    x[2] = 2.0 ** -120
    x[2, 5] = 2.0 ** 126                                   # one that dwarfs the row
    x[3, 5], x[4, 5] = float("inf"), float("nan")
    x[5] = 3.3895e38
    for eps in (0.0, EPS):
        r = m.moe_rmsnorm(x, w, eps, quantize=True)
        y, rstd = ref.rmsnorm(x.cpu().double(), w.cpu().double(), eps)
        y[3], rstd[3] = 0.0, 0.0                           # finite values over an infinite length
        y[3, 5] = float("nan")                             # inf / inf
        stored = rstd.float().double()
        ref.assert_within(r["rstd"], stored, RSTD * stored + 2.0 ** -149, "rstd")
        ref.assert_within(r["y"], y, (ref.BF16 + RSTD + 2 * ref.F32) * y.abs() + 2.0 ** -134, "y")
        if eps == 0.0:
            assert torch.isnan(r["y"][0]).all()            # 0 / 0
            assert float(r["y"][1, 7]) == float((w[7].float() * H ** 0.5).to(torch.bfloat16))


@pytest.mark.parametrize("e", [-80, 70])
@pytest.mark.parametrize("H", [264, 5120])
def test_such_rows_with_a_residual_and_in_place(H, e):
    """The path of these rows reads them again: from the sum, or from x and residual."""
    require_gpu()
    import routing_grouped_gemm_score_b200 as m
    x, r, w = (t if t.dim() == 1 else (t.float() * 2.0 ** e).to(t.dtype) for t in batch(200, H, 4))
    want = m.moe_rmsnorm(x, w, 0.0, residual=r, quantize=True)
    s = (x.double() + r.double()).to(torch.bfloat16).double().cpu()
    assert torch.equal(want["sum"].cpu().double(), s)
    y, rstd = ref.rmsnorm(s, w.cpu().double(), 0.0)
    ref.assert_within(want["rstd"], rstd, RSTD * rstd, "rstd")
    ref.assert_within(want["y"], y, (ref.BF16 + RSTD + 2 * ref.F32) * y.abs(), "y")
    for where in ({"sum": None}, {"sum": "x"}, {"sum": "r"}, {"y": "x"}, {"y": "x", "sum": None}, {"y": "x", "sum": "r"}):
        c = {"x": x.clone(), "r": r.clone()}
        got = m.moe_rmsnorm(c["x"], w, 0.0, residual=c["r"], quantize=True,
                            out={n: c.get(t) for n, t in where.items()})
        for n in want:
            assert got[n] is None if where.get(n, n) is None else torch.equal(got[n], want[n]), (where, n)
    c = want["sum"].clone()
    got = m.moe_rmsnorm(c, w, 0.0, quantize=True, out={"y": c})
    assert torch.equal(c, want["y"]) and torch.equal(got["y_q"], want["y_q"]) and torch.equal(got["rstd"], want["rstd"])
    alone = m.moe_rmsnorm(x[8:9], w, 0.0, residual=r[8:9], quantize=True)
    for n in want:
        assert torch.equal(alone[n], want[n][8:9]), n


@pytest.mark.parametrize("H", [72, 512, 4096])
def test_gradient_against_differences_of_the_kernel_itself(H):
    """<dx, v> of the backward kernel against (L(s + h v) - L(s - h v)) / 2h with
    L(s) = <dy, w s rstd>, rstd from the forward kernel (fp32; y in bf16 is too coarse),
    the rest in 64 bits. s has multiples of h = 2^-6 below 2, and v signs, so that the
    three rows are bf16 numbers. v takes the signs of the formula's gradient, so <dx, v> is
    the sum of its magnitudes: far above the tolerance, which a dx of zeros would miss."""
    require_gpu()
    import routing_grouped_gemm_score_b200 as m
    T, h = 5, 2.0 ** -6
    g = torch.Generator().manual_seed(H)
    s = torch.randint(-126, 127, (T, H), generator=g).double() * h
    dy = torch.randn(T, H, generator=g).to(torch.bfloat16)
    w = (1 + 0.3 * torch.randn(H, generator=g)).to(torch.bfloat16)
    dyw, wd = dy.double() * w.double(), w.double()
    v = ref.rmsnorm_backward(dy.double(), s, wd, ref.rmsnorm(s, wd, EPS)[1])[0].sign()
    rows = [(s + k * h * v).to(torch.bfloat16) for k in (0, 1, -1)]
    assert all(torch.equal(r.double(), s + k * h * v) for r, k in zip(rows, (0, 1, -1)))
    rstd = [m.moe_rmsnorm(r.cuda(), w.cuda(), EPS)["rstd"] for r in rows]
    loss = lambda r, rs: (dyw * r.double()).sum(dim=1) * rs.double().cpu()  # noqa: E731
    up, down = loss(rows[1], rstd[1]), loss(rows[2], rstd[2])
    got = m.moe_rmsnorm_backward(dy.cuda(), rows[0].cuda(), w.cuda(), rstd[0])["dx"].double().cpu()
    along = (got * v).sum(dim=1)
    # the difference's own error, h^2 L''' / 6 and more: the formula's difference less its derivative, in 64 bits
    exact = lambda k: loss(s + k * h * v, ref.rmsnorm(s + k * h * v, wd, EPS)[1])  # noqa: E731
    dx = ref.rmsnorm_backward(dy.double(), s, wd, ref.rmsnorm(s, wd, EPS)[1])[0]
    cut = ((exact(1) - exact(-1)) / (2 * h) - (dx * v).sum(dim=1)).abs()
    xhat = s * rstd[0].double().cpu()[:, None]
    terms = rstd[0].double().cpu()[:, None] * (dyw.abs() + xhat.abs() * (dyw * xhat).abs().sum(dim=1, keepdim=True) / H)
    # rstd of the two rows; dx to bf16 and its fp32 terms, as in test_backward; rstd of s enters dx twice
    tol = cut + RSTD * (up.abs() + down.abs()) / (2 * h) + ref.BF16 * dx.abs().sum(dim=1) + (
        64 * ref.F32 + 3 * RSTD) * terms.sum(dim=1)
    assert bool((along > 20 * tol).all())
    assert bool(((up - down) / (2 * h) - along).abs().le(tol).all())
