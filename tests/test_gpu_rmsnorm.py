"""moe_rmsnorm and moe_rmsnorm_backward against the 64-bit formulas."""
import pytest
import torch

import reference64 as ref
from helpers import require_gpu

pytestmark = pytest.mark.gpu

EPS = 1e-6
SHAPES = [(1, 8), (1, 2048), (2, 40), (61, 128), (33, 1000), (130, 2048), (7, 4096), (5, 5120), (3, 8200), (2, 16384),
          (700, 264)]


def inputs(T, H, seed=0):
    g = torch.Generator().manual_seed(seed + 131 * T + H)
    bf = lambda t: t.to(torch.bfloat16)  # noqa: E731
    channel = torch.exp(torch.randn(H, generator=g))
    return {"x": bf(torch.randn(T, H, generator=g)), "r": bf(3 * torch.randn(T, H, generator=g) * channel),
            "w": bf(1 + 0.3 * torch.randn(H, generator=g)), "dy": bf(torch.randn(T, H, generator=g)),
            "ds": bf(torch.randn(T, H, generator=g))}


# The sum of H squares: each thread adds at most 32 of its row, then 5 shuffles
# and 16 warps: 53 additions, one rounding each, and the square itself. All terms
# are positive, so the sum is off by at most 54 roundings and its root by half of
# them; the division, eps, root and reciprocal add 4.
RSTD = (27 + 4) * ref.F32


def check_y8(q, scale, y, cols, what):
    """The 8-bit rows of fp32 values that are within `d` of the float64 y."""
    d = RSTD + 2 * ref.F32
    s = scale.cpu()
    mag = ref.split_blocks(y.abs(), 1)[0].amax(dim=2)
    lo, hi = ref.exponents(mag * (1 - d)) + 127, ref.exponents(mag * (1 + d)) + 127
    assert bool(((s >= lo) & (s <= hi)).all()), f"{what}: scale bytes"
    got = ref.decode(q.cpu(), s)
    unit = ref.per_column(torch.exp2(s.double() - 127), cols)
    ref.assert_within(got, y, (2.0 ** -4 * (1 + d) + d) * y.abs() + 2.0 ** -10 * unit, what)


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("residual", [False, True])
def test_forward(T, H, residual):
    require_gpu()
    import routing_grouped_gemm_score_b200 as m
    d = inputs(T, H)
    r = m.moe_rmsnorm(d["x"].cuda(), d["w"].cuda(), EPS, residual=d["r"].cuda() if residual else None, quantize=True)
    s = d["x"].double()
    if residual:
        s = (s + d["r"].double()).to(torch.bfloat16).double()
        assert torch.equal(r["sum"].cpu().double(), s)
    y, rstd = ref.rmsnorm(s, d["w"].double(), EPS)
    ref.assert_within(r["rstd"], rstd, RSTD * rstd, "rstd")
    ref.assert_within(r["y"], y, (ref.BF16 + RSTD + 2 * ref.F32) * y.abs() + 2.0 ** -134, "y")
    check_y8(r["y_q"], r["y_scale"], y, H, "y in 8 bits")


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("with_dsum", [False, True])
def test_backward(T, H, with_dsum):
    require_gpu()
    import routing_grouped_gemm_score_b200 as m
    d = inputs(T, H, 5)
    s, w, dy = d["r"].double(), d["w"].double(), d["dy"].double()
    rstd = ref.rmsnorm(s, w, EPS)[1].float()
    ds = d["ds"] if with_dsum else None
    r = m.moe_rmsnorm_backward(d["dy"].cuda(), d["r"].cuda(), d["w"].cuda(), rstd.cuda(),
                               dsum=None if ds is None else ds.cuda())
    rs = rstd.double()
    dx, dw = ref.rmsnorm_backward(dy, s, w, rs, None if ds is None else ds.double())
    xhat = (s * rs[:, None]).abs()
    c_abs = (w * dy * xhat).abs().sum(dim=1, keepdim=True) / H
    # c: 3 products and 53 additions (as above); then 6 more roundings on either term
    terms = rs[:, None] * ((w * dy).abs() + xhat * c_abs) + (0 if ds is None else ds.double().abs())
    ref.assert_within(r["dx"], dx, ref.BF16 * dx.abs() + 64 * ref.F32 * terms + 2.0 ** -134, "dx")
    # dweight: 2 products; a block (one to eight an SM) adds its rows, then the blocks are added 32 apart, then 32
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    adds = -(-T // sms) + -(-8 * sms // 32) + 32
    ref.assert_within(r["dweight"], dw, (adds + 2) * ref.F32 * (dy * xhat).abs().sum(dim=0) + 2.0 ** -140, "dweight")


def test_reference_gradient_against_differences():
    """The formula that the kernels are held to is the derivative of the forward's."""
    g = torch.Generator().manual_seed(3)
    s, w, dy, ds = (torch.randn(*n, generator=g, dtype=torch.float64) for n in ((4, 24), (24,), (4, 24), (4, 24)))
    f = lambda s, w: (dy * ref.rmsnorm(s, w, EPS)[0]).sum() + (ds * s).sum()  # noqa: E731
    dx, dw = ref.rmsnorm_backward(dy, s, w, ref.rmsnorm(s, w, EPS)[1], ds)
    h = 1e-6
    for v, grad, at in ((s, dx, 0), (w, dw, 1)):
        for i in range(v.numel()):
            step = torch.zeros(v.numel(), dtype=torch.float64)
            step[i] = h
            step = step.reshape(v.shape)
            up, down = (f(s + k * step, w) if at == 0 else f(s, w + k * step) for k in (1, -1))
            assert abs((up - down) / (2 * h) - grad.reshape(-1)[i]) < 1e-7   # h^2 and 2^-52 / h


def test_backward_against_differences_of_the_forward():
    """The kernels' own gradient along a direction against the kernels' forward
    (rstd, which is fp32): d rstd / d step = -rstd^3 <s, v> / H."""
    require_gpu()
    import routing_grouped_gemm_score_b200 as m
    T, H = 5, 512
    d = inputs(T, H, 8)
    one = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    s = d["x"].cuda()
    r = m.moe_rmsnorm(s, one, 0.0)
    # dy = s: <s, y> = H^(1/2) |s|, whose gradient is y itself
    b = m.moe_rmsnorm_backward(s, s, one, r["rstd"])
    scaled = m.moe_rmsnorm((s.float() * 2).to(torch.bfloat16), one, 0.0)
    assert torch.equal(scaled["y"], r["y"])                       # the norm does not see the length
    # so the gradient along s vanishes, up to the roundings of its terms (|dy| |s| rstd each)
    along = (b["dx"].double() * s.double()).sum(dim=1).cpu()
    size = (s.double().square() * r["rstd"].double()[:, None]).sum(dim=1).cpu()
    assert bool((along.abs() <= 80 * ref.F32 * size + ref.BF16 * (b["dx"].double() * s.double()).abs().sum(dim=1).cpu()).all())


def test_without_outputs_in_place_and_empty():
    require_gpu()
    import routing_grouped_gemm_score_b200 as m
    T, H = 37, 1000
    d = {n: t.cuda() for n, t in inputs(T, H, 2).items()}
    full = m.moe_rmsnorm(d["x"], d["w"], EPS, residual=d["r"], quantize=True)
    # on the stored sum, without a residual: the same bits
    again = m.moe_rmsnorm(full["sum"], d["w"], EPS, quantize=True)
    for n in ("y", "rstd", "y_q", "y_scale"):
        assert torch.equal(full[n], again[n]), n
    # only the 8-bit output
    some = m.moe_rmsnorm(d["x"], d["w"], EPS, residual=d["r"], quantize=True, out={"y": None, "sum": None, "rstd": None})
    assert some["y"] is None and torch.equal(some["y_q"], full["y_q"]) and torch.equal(some["y_scale"], full["y_scale"])
    # the residual stream updated in place; the rows overwritten by the result
    res, x = d["r"].clone(), d["x"].clone()
    inplace = m.moe_rmsnorm(x, d["w"], EPS, residual=res, out={"sum": res, "y": x})
    assert inplace["sum"] is res and torch.equal(res, full["sum"]) and torch.equal(x, full["y"])
    b = m.moe_rmsnorm_backward(d["dy"], full["sum"], d["w"], full["rstd"], dsum=d["ds"])
    for target in ("dy", "ds"):
        c = {n: t.clone() for n, t in d.items()}
        got = m.moe_rmsnorm_backward(c["dy"], full["sum"], c["w"], full["rstd"], dsum=c["ds"], dx=c[target])
        assert got["dx"] is c[target] and torch.equal(got["dx"], b["dx"]) and torch.equal(got["dweight"], b["dweight"])
    got = m.moe_rmsnorm_backward(d["dy"], full["sum"], d["w"], full["rstd"], dsum=d["ds"], want_dweight=False)
    assert got["dweight"] is None and torch.equal(got["dx"], b["dx"])
    none = torch.empty(0, H, dtype=torch.bfloat16, device="cuda")
    e = m.moe_rmsnorm(none, d["w"], EPS, residual=none, quantize=True)
    assert e["y"].shape == (0, H) and e["y_scale"].shape == (0, 32)
    g = m.moe_rmsnorm_backward(none, none, d["w"], e["rstd"])
    assert g["dx"].shape == (0, H) and not g["dweight"].any()


def test_rows_that_are_not_numbers():
    """A row with a NaN or an infinity spoils itself only; zeros with eps stay zeros."""
    require_gpu()
    import routing_grouped_gemm_score_b200 as m
    T, H = 6, 72
    d = inputs(T, H, 4)
    x = d["x"].clone()
    x[1, 3], x[2, 70], x[3] = float("nan"), float("inf"), 0.0
    r = m.moe_rmsnorm(x.cuda(), d["w"].cuda(), EPS, quantize=True)
    clean = m.moe_rmsnorm(d["x"].cuda(), d["w"].cuda(), EPS, quantize=True)
    for i in (0, 4, 5):
        for n in ("y", "rstd", "y_q", "y_scale"):
            assert torch.equal(r[n][i], clean[n][i])
    assert torch.isnan(r["y"][1]).all() and torch.isnan(r["y"][2, 70]) and not r["y"][2, :70].any()
    assert not r["y"][3].any()
    back = m.moe_dequantize_rows(r["y_q"], r["y_scale"])
    assert torch.isnan(back[1]).all() and torch.isnan(back[2, 70]) and not back[2, :64].any() and not back[3].any()
    b = m.moe_rmsnorm_backward(d["dy"].cuda(), x.cuda(), d["w"].cuda(), r["rstd"])
    cb = m.moe_rmsnorm_backward(d["dy"].cuda(), d["x"].cuda(), d["w"].cuda(), clean["rstd"])
    for i in (0, 4, 5):
        assert torch.equal(b["dx"][i], cb["dx"][i])


def test_many_rows_and_repeatable():
    require_gpu()
    import routing_grouped_gemm_score_b200 as m
    T, H = (1 << 18) + 5, 8192                                     # more than 2^31 elements
    d = inputs(3, H, 6)
    x = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    x[-3:] = d["x"].cuda()
    few = m.moe_rmsnorm(d["x"].cuda(), d["w"].cuda(), EPS, quantize=True)
    r = m.moe_rmsnorm(x, d["w"].cuda(), EPS, quantize=True)
    for n in ("y", "rstd", "y_q", "y_scale"):
        assert torch.equal(r[n][-3:], few[n]), n
    del r["y_q"]
    dy = r["y"]
    b = m.moe_rmsnorm_backward(dy, x, d["w"].cuda(), r["rstd"])
    fb = m.moe_rmsnorm_backward(few["y"], d["x"].cuda(), d["w"].cuda(), few["rstd"])
    assert torch.equal(b["dx"][-3:], fb["dx"]) and not b["dx"][:-3].any()
    again = m.moe_rmsnorm_backward(dy, x, d["w"].cuda(), r["rstd"])
    assert torch.equal(again["dweight"], b["dweight"])
