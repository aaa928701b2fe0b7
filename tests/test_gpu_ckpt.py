"""The layer with its training state in 8 bits: moe_layer_forward_ckpt and
moe_grouped_mlp_backward_ckpt against the layer, the format and the 64-bit formulas."""
import pytest
import torch

import reference64 as ref
from helpers import force_kernels, require_gpu

pytestmark = pytest.mark.gpu


def case(T, H, I, E, k, seed=0, dead=0, sigmoid=False, std=1.0):
    g = torch.Generator().manual_seed(seed + 7 * T + 11 * H + 13 * I + E)
    bias = torch.zeros(E)
    if dead:
        bias[torch.randperm(E, generator=g)[:dead]] = -1e4
    bf = lambda t: t.to(torch.bfloat16)  # noqa: E731
    d = {"logits": torch.randn(T, E, generator=g) + bias, "x": bf(std * torch.randn(T, H, generator=g)),
         "w_gate_up": bf(torch.randn(E, H, 2 * I, generator=g) / H ** 0.5),
         "w_down": bf(torch.randn(E, I, H, generator=g) / I ** 0.5), "dout": bf(torch.randn(T, H, generator=g))}
    d["cuda"] = {n: t.cuda() for n, t in d.items()}
    d["k"], d["sigmoid"] = k, sigmoid
    return d


def opts(d):
    import routing_grouped_gemm_score_b200 as m
    return m.RouterOpts(m.SCORE_SIGMOID, renormalize=False) if d["sigmoid"] else m.RouterOpts()


def forward(d, **kw):
    import routing_grouped_gemm_score_b200 as m
    c = d["cuda"]
    return m.moe_layer_forward_ckpt(c["logits"], c["x"], c["w_gate_up"], c["w_down"], d["k"], opts(d), **kw)


def status_ok():
    import routing_grouped_gemm_score_b200 as m
    assert m.moe_get_device_status() == 0


def check_forward(d, out, st):
    """out and routing as the layer's; x8 exactly; gu8 within the format of the 64-bit products."""
    import routing_grouped_gemm_score_b200 as m
    c = d["cuda"]
    plain, pst = m.moe_layer_forward(c["logits"], c["x"], c["w_gate_up"], c["w_down"], d["k"], opts(d),
                                     save_for_backward=True)
    assert torch.equal(out, plain)
    for n in ("topk_idx", "topk_prob", "counts", "offsets", "row_of"):
        assert torch.equal(st[n], pst[n]), n
    x = d["x"].double()
    want, bytes_ = ref.quantize(x)
    assert torch.equal(st["x_scale"].cpu(), bytes_)
    ref.assert_within(ref.decode(st["x_q"].cpu(), bytes_), want, torch.zeros_like(want), "x8")
    offs, row_of = st["offsets"].cpu(), st["row_of"].cpu()
    xr = x[ref.token_of_row(row_of)]
    gu, _ = ref.mlp_rows(xr, d["w_gate_up"].double(), d["w_down"].double(), offs)
    mag, _ = ref.mlp_rows(xr.abs(), d["w_gate_up"].double().abs(), d["w_down"].double(), offs)
    acc = x.shape[1] * ref.TC * mag                                # the accumulator's error
    I = d["w_down"].shape[1]
    s = st["gu_scale"].cpu().t()
    big = lambda v: ref.split_blocks(v.clamp(min=0), 2)[0].amax(dim=2)  # noqa: E731
    lo, hi = ref.exponents(big(gu.abs() - acc)) + 127, ref.exponents(big(gu.abs() + acc)) + 127
    assert bool(((s >= lo) & (s <= hi)).all()), "gu scale bytes"
    got = ref.decode(st["gu_q"].cpu(), s, 2)
    unit = ref.per_column(torch.exp2(s.double() - 127), I, 2)
    ref.assert_within(got, gu, 2.0 ** -4 * (gu.abs() + acc) + acc + 2.0 ** -10 * unit, "gu8")
    back = m.moe_dequantize_rows(st["gu_q"], st["gu_scale"], parts=2, block_major=True)
    assert torch.equal(back.cpu().double(), got)


def check_backward(d, st, g):
    x = ref.decode(st["x_q"].cpu(), st["x_scale"].cpu())
    gu = ref.decode(st["gu_q"].cpu(), st["gu_scale"].cpu().t(), 2)
    r = ref.layer_backward(d["dout"].double(), x, gu, st["topk_prob"].cpu().double(), d["w_gate_up"].double(),
                           d["w_down"].double(), st["row_of"].cpu(), st["offsets"].cpu())
    for n in ("dprob", "dw_down", "dw_gate_up", "dx"):
        ref.assert_within(g[n], r[n], r[n + "_tol"], n)


def backward(d, st, **kw):
    import routing_grouped_gemm_score_b200 as m
    c = d["cuda"]
    return m.moe_grouped_mlp_backward_ckpt(c["dout"], st, c["w_gate_up"], c["w_down"], **kw)


# T, H, I, E, k: one token; one expert; widths that end inside a block of 32 and
# inside a tile; experts without rows; each kernel family by its own rule
SHAPES = [(1, 8, 8, 1, 1), (1, 64, 72, 5, 3), (61, 128, 256, 8, 2), (40, 200, 40, 16, 4), (64, 264, 104, 4, 4),
          (300, 128, 328, 3, 2), (1500, 96, 64, 2, 1), (257, 512, 24, 1, 1), (130, 64, 520, 12, 12),
          (700, 264, 200, 3, 2)]


@pytest.mark.parametrize("T,H,I,E,k", SHAPES)
@pytest.mark.parametrize("tiles", ["auto", "single", "pair", "swap", "swap_unfused"])
def test_forward_and_backward(T, H, I, E, k, tiles):
    require_gpu()
    if tiles == "swap" and T > 64:
        tiles = "swap_unfused"   # the one-launch kernel holds at most 64 rows an expert
    force_kernels(gemm_tiles=tiles)
    d = case(T, H, I, E, k, dead=(E - k) // 2, sigmoid=k == 1)
    out, st = forward(d)
    status_ok()
    check_forward(d, out, st)
    g = backward(d, st)
    status_ok()
    check_backward(d, st, g)


@pytest.mark.parametrize("T,H,E,k", [(5000, 1032, 3, 2), (2400, 2056, 8, 7), (1400, 1032, 16, 16)])
def test_more_units_than_warps(T, H, E, k):
    """Rows of several units each, more of them than the steps by token have warps."""
    require_gpu()
    d = case(T, H, 8, E, k)
    _, st = forward(d)
    g = backward(d, st)
    status_ok()
    check_backward(d, st, g)


@pytest.mark.parametrize("T,H,k", [(9, 40, 2), (300, 264, 3), (70, 4096, 4), (33, 4104, 2), (5, 8192, 1), (400, 5120, 16)])
@pytest.mark.parametrize("permute", ["auto", "warp"])
def test_x8_from_every_permute(T, H, k, permute):
    """x8 comes from whichever kernel moves the rows (or its own), bit for bit."""
    require_gpu()
    force_kernels(permute=permute)
    d = case(T, H, 8, 16, k)
    d["x"][T // 2, H - 3], d["x"][0, 1] = float("inf"), -3.3895e38
    d["cuda"]["x"] = d["x"].cuda()
    _, st = forward(d)
    status_ok()
    want, bytes_ = ref.quantize(d["x"].double())
    assert torch.equal(st["x_scale"].cpu(), bytes_)
    ref.assert_within(ref.decode(st["x_q"].cpu(), bytes_), want, torch.zeros_like(want), "x8")


def test_folded_permute():
    require_gpu()
    d = case(300, 128, 328, 3, 2)
    out, st = forward(d)
    force_kernels(gemm_tiles="single", fold_permute=True)
    out2, st2 = forward(d)
    status_ok()
    check_forward(d, out2, st2)
    assert torch.equal(st2["row_of"], st["row_of"])


@pytest.mark.parametrize("std", [1e-20, 1e12])
def test_sizes_far_from_one(std):
    """x8 and gu8 near neither end of the E4M3 range: the scales take them there."""
    require_gpu()
    d = case(61, 128, 64, 4, 2, std=std)
    out, st = forward(d)
    x = d["x"].double()
    want, bytes_ = ref.quantize(x)
    assert torch.equal(st["x_scale"].cpu(), bytes_)
    offs, row_of = st["offsets"].cpu(), st["row_of"].cpu()
    xr = x[ref.token_of_row(row_of)]
    gu, _ = ref.mlp_rows(xr, d["w_gate_up"].double(), d["w_down"].double(), offs)
    mag, _ = ref.mlp_rows(xr.abs(), d["w_gate_up"].double().abs(), d["w_down"].double(), offs)
    s = st["gu_scale"].cpu().t()
    unit = ref.per_column(torch.exp2(s.double() - 127), 64, 2)
    acc = 128 * ref.TC * mag
    ref.assert_within(ref.decode(st["gu_q"].cpu(), s, 2), gu, 2.0 ** -4 * (gu.abs() + acc) + acc + 2.0 ** -10 * unit,
                      "gu8")


def test_infinite_and_missing_values_stay_in_their_rows():
    require_gpu()
    import routing_grouped_gemm_score_b200 as m
    d = case(61, 128, 64, 4, 2)
    out, st = forward(d)
    d["cuda"]["x"] = d["cuda"]["x"].clone()
    d["cuda"]["x"][7, 5], d["cuda"]["x"][9, 127] = float("nan"), float("inf")
    out2, st2 = forward(d)
    hit = [7, 9]
    rest = [t for t in range(61) if t not in hit]
    rows = st["row_of"][rest].reshape(-1).long()
    for n in ("x_q", "x_scale"):
        assert torch.equal(st2[n][rest], st[n][rest])
    assert torch.equal(st2["gu_q"][rows], st["gu_q"][rows]) and torch.equal(st2["gu_scale"][:, rows], st["gu_scale"][:, rows])
    gu = m.moe_dequantize_rows(st2["gu_q"], st2["gu_scale"], parts=2, block_major=True)
    assert torch.isnan(gu[st["row_of"][7].long()]).all() and torch.isnan(gu[st["row_of"][9].long()]).all()
    assert torch.equal(out2[rest], out[rest])


def test_norm_layer_and_both_backwards_together():
    """As a block uses them: norm with the residual (its 8-bit rows are the layer's
    x8), layer, layer's backward, norm's backward with the residual's gradient."""
    require_gpu()
    import routing_grouped_gemm_score_b200 as m
    T, H, I, E, k = 130, 264, 104, 8, 2
    d = case(T, H, I, E, k, seed=3)
    c = d["cuda"]
    g = torch.Generator().manual_seed(11)
    res = torch.randn(T, H, generator=g).to(torch.bfloat16).cuda()
    w = (1 + 0.2 * torch.randn(H, generator=g)).to(torch.bfloat16).cuda()
    n = m.moe_rmsnorm(c["x"], w, 1e-6, residual=res, quantize=True)
    d["x"], c["x"] = n["y"].cpu(), n["y"]
    kept = n["y_q"].clone(), n["y_scale"].clone()
    out, st = forward(d, x8=(n["y_q"], n["y_scale"]))
    assert st["x_q"] is n["y_q"] and torch.equal(st["x_q"], kept[0]) and torch.equal(st["x_scale"], kept[1])
    assert torch.equal(out, m.moe_layer_forward(c["logits"], c["x"], c["w_gate_up"], c["w_down"], k))
    gr = backward(d, st)
    status_ok()
    check_backward(d, st, gr)
    b = m.moe_rmsnorm_backward(gr["dx"], n["sum"], w, n["rstd"], dsum=c["dout"])
    s, rs = n["sum"].cpu().double(), n["rstd"].cpu().double()
    dx, _ = ref.rmsnorm_backward(gr["dx"].cpu().double(), s, w.cpu().double(), rs, d["dout"].double())
    dy, xhat = gr["dx"].cpu().double(), (s * rs[:, None]).abs()
    wd = (w.cpu().double() * dy).abs()
    terms = rs[:, None] * (wd + xhat * (wd * xhat).sum(dim=1, keepdim=True) / H) + d["dout"].double().abs()
    ref.assert_within(b["dx"], dx, ref.BF16 * dx.abs() + 64 * ref.F32 * terms, "dx of the block")
    # the whole run again: the same bits
    out2, st2 = forward(d, x8=(n["y_q"], n["y_scale"]))
    gr2 = backward(d, st2)
    for name in gr:
        assert torch.equal(gr[name], gr2[name]), name


def test_reference_gradient_against_differences():
    """The formulas that the kernels are held to are the layer's derivatives."""
    g = torch.Generator().manual_seed(5)
    T, H, I, E, k = 3, 6, 4, 2, 2
    r = lambda *n: torch.randn(*n, generator=g, dtype=torch.float64)  # noqa: E731
    v = {"x": r(T, H), "p": r(T, k).abs(), "w_gate_up": r(E, H, 2 * I), "w_down": r(E, I, H)}
    dout = r(T, H)
    row_of = torch.tensor([[0, 3], [1, 4], [2, 5]])                # token t: expert 0 then 1
    offsets, tok = torch.tensor([0, 3, 6]), torch.tensor([0, 1, 2, 0, 1, 2])

    def loss(v):
        _, y = ref.mlp_rows(v["x"][tok], v["w_gate_up"], v["w_down"], offsets)
        return (dout * (v["p"][:, :, None] * y[row_of]).sum(dim=1)).sum()

    gu, _ = ref.mlp_rows(v["x"][tok], v["w_gate_up"], v["w_down"], offsets)
    got = ref.layer_backward(dout, v["x"], gu, v["p"], v["w_gate_up"], v["w_down"], row_of, offsets)
    h = 1e-6
    for name, grad in (("x", "dx"), ("p", "dprob"), ("w_gate_up", "dw_gate_up"), ("w_down", "dw_down")):
        for i in range(v[name].numel()):
            step = torch.zeros(v[name].numel(), dtype=torch.float64)
            step[i] = h
            up, down = (loss({**v, name: v[name] + s * step.reshape(v[name].shape)}) for s in (1, -1))
            assert abs((up - down) / (2 * h) - got[grad].reshape(-1)[i]) < 1e-6   # h^2 and 2^-52 |loss| / h


def test_near_the_bf16_state():
    """Both backward passes of one batch: what 8 bits cost. Each saved value is off by
    at most 2^-4, so the gradients' 2-norms differ by a few hundredths, never more
    than 2^-3 (g, u and x enter every product once, silu' at most twice)."""
    require_gpu()
    import routing_grouped_gemm_score_b200 as m
    d = case(300, 256, 256, 4, 2)
    c = d["cuda"]
    _, pst = m.moe_layer_forward(c["logits"], c["x"], c["w_gate_up"], c["w_down"], 2, save_for_backward=True)
    want = m.moe_grouped_mlp_backward(c["dout"], pst, c["w_gate_up"], c["w_down"])
    _, st = forward(d)
    got = backward(d, st)
    for n in want:
        off = (got[n].double() - want[n].double()).norm() / want[n].double().norm()
        assert float(off) < 2.0 ** -3, (n, float(off))
    saved = lambda s, names: sum(s[n].numel() * s[n].element_size() for n in names)  # noqa: E731
    T, H, I, A = 300, 256, 256, 600   # 33/32 bytes a value of x by token and of [g | u]; against 4H + 6I a row
    ours = saved(st, ("x_q", "x_scale", "gu_q", "gu_scale"))
    assert ours == T * H * 33 // 32 + A * 2 * I * 33 // 32
    assert saved(pst, ("x_perm", "gu", "h", "y_perm")) == A * (4 * H + 6 * I)


def test_no_tokens():
    require_gpu()
    import routing_grouped_gemm_score_b200 as m
    d = case(0, 64, 32, 4, 2)
    out, st = forward(d)
    assert out.shape == (0, 64) and not st["counts"].any() and not st["offsets"].any()
    grads = {"dw_gate_up": torch.ones_like(d["cuda"]["w_gate_up"]), "dw_down": torch.ones_like(d["cuda"]["w_down"])}
    g = backward(d, st, grads=grads)
    status_ok()
    assert g["dx"].shape == (0, 64) and not g["dw_gate_up"].any() and not g["dw_down"].any()
    assert m.lib().moe_grouped_mlp_backward_ckpt_workspace_size(0, 64, 32, 4, 2) >= 0


def test_experts_without_rows_get_zero_gradients():
    require_gpu()
    d = case(61, 128, 64, 8, 2, dead=5)
    _, st = forward(d)
    grads = {"dw_gate_up": torch.full_like(d["cuda"]["w_gate_up"], 7), "dw_down": torch.full_like(d["cuda"]["w_down"], 7)}
    g = backward(d, st, grads=grads)
    empty = (st["counts"] == 0).cpu()
    assert int(empty.sum()) >= 5
    assert not g["dw_gate_up"][empty.cuda()].any() and not g["dw_down"][empty.cuda()].any()


def test_shared_expert_bias_workspace_and_reused_state():
    require_gpu()
    import routing_grouped_gemm_score_b200 as m
    T, H, I, E, k = 200, 128, 64, 8, 2
    d = case(T, H, I, E, k, seed=2)
    c = d["cuda"]
    g = torch.Generator().manual_seed(1)
    sgu = (torch.randn(H, 2 * I, generator=g) / H ** 0.5).to(torch.bfloat16).cuda()
    sd = (torch.randn(I, H, generator=g) / I ** 0.5).to(torch.bfloat16).cuda()
    o = m.RouterOpts(m.SCORE_SIGMOID, True, 2.5, torch.randn(E, generator=g).cuda())
    ws = m.LayerWorkspace(T, H, I, E, k, True, backward=True, ckpt=True)
    args = (c["logits"], c["x"], c["w_gate_up"], c["w_down"], k, o, sgu, sd)
    out, st = m.moe_layer_forward_ckpt(*args, workspace=ws)
    want, pst = m.moe_layer_forward(*args, save_for_backward=True)
    assert torch.equal(out, want) and torch.equal(st["topk_prob"], pst["topk_prob"])
    first = backward(d, st, workspace=ws)
    check_backward(d, st, first)
    keep = {n: t.clone() for n, t in st.items()}
    first = {n: t.clone() for n, t in first.items()}
    # another batch into the same state and gradients, then the first one again
    d2 = case(T, H, I, E, k, seed=9)
    m.moe_layer_forward_ckpt(d2["cuda"]["logits"], d2["cuda"]["x"], *args[2:], workspace=ws, state=st)
    assert not torch.equal(st["gu_q"], keep["gu_q"])
    out2, st2 = m.moe_layer_forward_ckpt(*args, workspace=ws, state=st, out=out)
    assert out2 is out and torch.equal(out, want)
    for n in keep:
        assert st2[n] is st[n] and torch.equal(st2[n], keep[n]), n
    again = backward(d, st2, workspace=ws, grads={n: torch.empty_like(t) for n, t in first.items()})
    for n in first:
        assert torch.equal(first[n], again[n]), n


@pytest.mark.parametrize("T,H,I,E,k", [(61, 128, 256, 8, 2), (1500, 96, 64, 2, 1)])
def test_captured_and_on_two_streams(T, H, I, E, k):
    require_gpu()
    import routing_grouped_gemm_score_b200 as m
    d = case(T, H, I, E, k)
    c = d["cuda"]
    w = torch.ones(H, dtype=torch.bfloat16, device="cuda")

    def step(x, dout):
        n = m.moe_rmsnorm(x, w, 1e-6, quantize=True)
        out, st = m.moe_layer_forward_ckpt(c["logits"], n["y"], c["w_gate_up"], c["w_down"], k, opts(d),
                                           x8=(n["y_q"], n["y_scale"]))
        g = m.moe_grouped_mlp_backward_ckpt(dout, st, c["w_gate_up"], c["w_down"])
        b = m.moe_rmsnorm_backward(g["dx"], n["sum"], w, n["rstd"], dsum=dout)
        return [out, g["dw_gate_up"], g["dw_down"], g["dprob"], b["dx"], b["dweight"]]

    want = [t.clone() for t in step(c["x"], c["dout"])]
    other = [t.clone() for t in step(c["dout"], c["x"])]
    x, dout = c["x"].clone(), c["dout"].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(x, dout)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(x, dout)
    for a, b, expect in ((c["x"], c["dout"], want), (c["dout"], c["x"], other), (c["x"], c["dout"], want)):
        x.copy_(a)
        dout.copy_(b)
        graph.replay()
        for g, e in zip(got, expect):
            assert torch.equal(g, e)
    # two steps on two streams at once, each with its own memory
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    results = []
    for s, (a, b) in zip(streams, ((c["x"], c["dout"]), (c["dout"], c["x"]))):
        with torch.cuda.stream(s):
            results.append(step(a, b))
    torch.cuda.synchronize()
    for r, expect in zip(results, (want, other)):
        for g, e in zip(r, expect):
            assert torch.equal(g, e)
    status_ok()


def test_rows_past_32_bit_offsets():
    """[g | u] of more than 2^31 values: the last tokens' state and gradients."""
    require_gpu()
    T, H, I, E, k = 32768, 64, 33000, 1, 1
    d = case(4, H, I, E, k, seed=1)
    c = d["cuda"]
    few_out, few = forward(d)
    few_g = backward(d, few)
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
    dout = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    x[-4:], dout[-4:] = c["x"], c["dout"]
    big = dict(d, cuda=dict(c, x=x, dout=dout, logits=torch.zeros(T, 1, device="cuda")))
    out, st = forward(big)
    assert st["gu_q"].numel() > 2 ** 31
    # the same rows, on other tiles: the accumulators may differ in their last bits
    assert float((out[-4:].float() - few_out.float()).norm() / few_out.float().norm()) < 2 * ref.BF16
    a, b = st["gu_q"][-4:].view(torch.float8_e4m3fn).float(), few["gu_q"].view(torch.float8_e4m3fn).float()
    assert float((a != b).float().mean()) < 1e-3 and float((st["gu_scale"][:, -4:] != few["gu_scale"]).float().mean()) < 1e-3
    for n in ("gu_q", "gu_scale"):   # from here on the same state, so the same gradients up to roundings
        (st[n][-4:] if n == "gu_q" else st[n][:, -4:]).copy_(few[n])
    gr = backward(big, st)
    status_ok()
    r = ref.layer_backward(d["dout"].double(), ref.decode(few["x_q"].cpu(), few["x_scale"].cpu()),
                           ref.decode(few["gu_q"].cpu(), few["gu_scale"].cpu().t(), 2),
                           few["topk_prob"].cpu().double(), d["w_gate_up"].double(), d["w_down"].double(),
                           few["row_of"].cpu(), few["offsets"].cpu())
    for n in ("dx", "dprob"):
        ref.assert_within(gr[n][-4:], r[n], r[n + "_tol"], n)
        ref.assert_within(few_g[n], r[n], r[n + "_tol"], n)
    assert not gr["dx"][:-4].any() and not gr["dprob"][:-4].any()
    for n in ("dw_gate_up", "dw_down"):   # the other rows add zeros
        ref.assert_within(gr[n], r[n], r[n + "_tol"], n)


def test_row_outside_its_range_is_reported():
    require_gpu()
    import routing_grouped_gemm_score_b200 as m
    d = case(61, 128, 64, 4, 2)
    _, st = forward(d)
    bad = dict(st, row_of=st["row_of"].clone())
    bad["row_of"][3, 1], bad["row_of"][4, 0] = -1, 61 * 2
    backward(d, bad)
    assert m.moe_get_device_status() == m.MOE_ERR_DEVICE_CHECK
    check_backward(d, st, backward(d, st))
    status_ok()
