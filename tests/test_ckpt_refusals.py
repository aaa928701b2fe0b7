"""What the norm, the 8-bit rows and the 8-bit layer state refuse, before any device is
touched (the C entry points get addresses that are never dereferenced)."""
import ctypes

import pytest
import torch

FAKE = 1 << 20
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 4


@pytest.fixture(scope="session")
def m():
    from routing_grouped_gemm_score_b200 import build
    build.build()
    import routing_grouped_gemm_score_b200 as m
    return m


def test_rows(m):
    l = m.lib()
    good = dict(rows=4, cols=64, parts=1, major=0)
    for bad in (dict(rows=-1), dict(rows=1 << 31), dict(cols=0), dict(cols=12), dict(cols=-8), dict(parts=0),
                dict(parts=3), dict(major=2), dict(cols=(1 << 24) + 8)):
        a = {**good, **bad}
        assert l.moe_quantize_rows(FAKE, a["rows"], a["cols"], a["parts"], a["major"], FAKE, FAKE, None) == INVALID, bad
        assert l.moe_dequantize_rows(FAKE, FAKE, a["rows"], a["cols"], a["parts"], a["major"], FAKE, None) == INVALID, bad
    for i in range(3):
        for wrong in (None, FAKE + 8):
            p = [FAKE] * 3
            p[i] = wrong
            assert l.moe_quantize_rows(p[0], 4, 64, 1, 0, p[1], p[2], None) == INVALID
            assert l.moe_dequantize_rows(p[0], p[1], 4, 64, 1, 0, p[2], None) == INVALID
    assert l.moe_quantize_rows(None, 0, 64, 1, 0, None, None, None) == 0
    assert l.moe_dequantize_rows(None, None, 0, 64, 2, 1, None, None) == 0


def norm(l, T=4, H=64, eps=1e-6, x=FAKE, residual=FAKE, weight=FAKE, s=FAKE, y=FAKE, q=FAKE, scale=FAKE, rstd=FAKE):
    return l.moe_rmsnorm(x, residual, weight, T, H, eps, s, y, q, scale, rstd, None)


def test_rmsnorm(m):
    l = m.lib()
    for bad in (dict(T=-1), dict(T=1 << 31), dict(H=0), dict(H=-8), dict(eps=-1e-6), dict(eps=float("nan")),
                dict(eps=float("inf")), dict(x=None), dict(weight=None), dict(y=None, q=None, scale=None), dict(q=None),
                dict(scale=None), dict(residual=None), dict(x=FAKE + 2), dict(y=FAKE + 8), dict(q=FAKE + 8),
                dict(rstd=FAKE + 4), dict(s=FAKE + 2), dict(weight=FAKE + 2), dict(scale=FAKE + 1)):
        assert norm(l, **bad) == INVALID, bad
    assert norm(l, H=12) == UNSUPPORTED and norm(l, H=16392) == UNSUPPORTED
    assert norm(l, T=0, x=None, weight=None, y=None, residual=None, s=None) == 0


def test_rmsnorm_backward(m):
    l = m.lib()

    def call(T=4, H=64, dy=FAKE, s=FAKE, w=FAKE, rstd=FAKE, dsum=FAKE, dx=FAKE, dw=FAKE, ws=FAKE, n=1 << 20):
        return l.moe_rmsnorm_backward(dy, s, w, rstd, dsum, T, H, dx, dw, ws, n, None)

    for bad in (dict(T=-1), dict(T=1 << 31), dict(H=0), dict(dy=None), dict(s=None), dict(w=None), dict(rstd=None),
                dict(dx=None), dict(dy=FAKE + 2), dict(dsum=FAKE + 2), dict(dw=FAKE + 4), dict(dx=FAKE + 8)):
        assert call(**bad) == INVALID, bad
    assert call(H=20) == UNSUPPORTED and call(H=16392) == UNSUPPORTED
    for bad in (dict(ws=None), dict(n=0), dict(ws=FAKE + 8)):
        assert call(**bad) == WORKSPACE, bad
    assert l.moe_rmsnorm_backward_workspace_size(4, 64) > 0
    for T, H in ((-1, 64), (4, 12), (4, 16392), (4, 0), (1 << 31, 64)):
        assert l.moe_rmsnorm_backward_workspace_size(T, H) == 0


def test_layer_forward(m):
    l = m.lib()
    o = m.RouterOpts().c()
    names = ["logits", "x", "w_gate_up", "w_down", "out", "topk_idx", "topk_prob", "counts", "offsets", "row_of", "x_q",
             "x_scale", "gu_q", "gu_scale"]

    def call(T=4, H=64, I=32, E=4, k=2, given=0, shared=(None, None), ws=FAKE, n=1 << 40, **p):
        a = {name: FAKE for name in names}
        a.update(p)
        return l.moe_layer_forward_ckpt(a["logits"], a["x"], T, H, I, E, k, ctypes.byref(o), a["w_gate_up"], a["w_down"],
                                        *shared, a["out"], a["topk_idx"], a["topk_prob"], a["counts"], a["offsets"],
                                        a["row_of"], a["x_q"], a["x_scale"], given, a["gu_q"], a["gu_scale"], ws, n, None)

    for name in names:
        assert call(**{name: FAKE + 2}) == INVALID, name
        if name != "counts":
            assert call(**{name: None}) == INVALID, name
    for bad in (dict(T=-1), dict(E=0), dict(k=5), dict(k=0), dict(E=300), dict(given=2), dict(shared=(FAKE, None)),
                dict(H=0), dict(I=0)):
        assert call(**bad) == INVALID, bad
    assert call(H=12) == UNSUPPORTED and call(I=12) == UNSUPPORTED
    assert call(ws=None) == WORKSPACE and call(n=16) == WORKSPACE
    assert call(given=1, x_q=None, x_scale=None, n=16) == WORKSPACE   # x_q is not asked for


def test_layer_backward(m):
    l = m.lib()
    names = ["dout", "w_gate_up", "w_down", "row_of", "topk_prob", "offsets", "x_q", "x_scale", "gu_q", "gu_scale", "dx",
             "dw_gate_up", "dw_down", "dprob"]

    def call(T=4, H=64, I=32, E=4, k=2, ws=FAKE, n=1 << 40, **p):
        a = {name: FAKE for name in names}
        a.update(p)
        return l.moe_grouped_mlp_backward_ckpt(a["dout"], T, H, I, E, k, *[a[name] for name in names[1:]], ws, n, None)

    for name in names:
        assert call(**{name: None}) == INVALID, name
        assert call(**{name: FAKE + 8}) == INVALID, name
    for bad in (dict(T=-1), dict(E=0), dict(k=5), dict(E=300), dict(H=0), dict(I=-8)):
        assert call(**bad) == INVALID, bad
    assert call(H=12) == UNSUPPORTED and call(I=12) == UNSUPPORTED
    for bad in (dict(ws=None), dict(n=16), dict(ws=FAKE + 8)):
        assert call(**bad) == WORKSPACE, bad
    assert l.moe_grouped_mlp_backward_ckpt_workspace_size(4, 64, 32, 4, 2) > 0
    for T, H, I, E, k in ((-1, 64, 32, 4, 2), (4, 12, 32, 4, 2), (4, 64, 12, 4, 2), (4, 64, 32, 4, 5)):
        assert l.moe_grouped_mlp_backward_ckpt_workspace_size(T, H, I, E, k) == 0


def test_the_binding_refuses_host_tensors_and_wrong_types(m):
    bf = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.zeros(64, dtype=torch.bfloat16)
    u8 = torch.zeros(4, 64, dtype=torch.uint8)
    for call in (lambda: m.moe_quantize_rows(bf), lambda: m.moe_dequantize_rows(u8, u8),
                 lambda: m.moe_rmsnorm(bf, w, 1e-6), lambda: m.moe_rmsnorm_backward(bf, bf, w, torch.zeros(4))):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    for call in (lambda: m.moe_quantize_rows(bf.float()), lambda: m.moe_dequantize_rows(bf, u8),
                 lambda: m.moe_rmsnorm(bf.half(), w, 1e-6)):
        with pytest.raises(TypeError):
            call()


@pytest.mark.gpu
def test_the_binding_refuses_wrong_shapes(m):
    bf = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(64, dtype=torch.bfloat16, device="cuda")
    rstd = torch.zeros(4, device="cuda")
    q, s = m.moe_quantize_rows(bf)
    wgu = torch.zeros(2, 64, 16, dtype=torch.bfloat16, device="cuda")
    wd = torch.zeros(2, 8, 64, dtype=torch.bfloat16, device="cuda")
    lg = torch.zeros(4, 2, device="cuda")
    out, st = m.moe_layer_forward_ckpt(lg, bf, wgu, wd, 1)
    for call in (lambda: m.moe_quantize_rows(bf, parts=3), lambda: m.moe_quantize_rows(bf[0]),
                 lambda: m.moe_quantize_rows(bf.t()), lambda: m.moe_dequantize_rows(q, s[:, :1].contiguous()),
                 lambda: m.moe_dequantize_rows(q, s, out=bf[:2]), lambda: m.moe_rmsnorm(bf, w[:32], 1e-6),
                 lambda: m.moe_rmsnorm(bf, w, 1e-6, residual=bf[:2]), lambda: m.moe_rmsnorm(bf, w, 1e-6, out={"sum": bf}),
                 lambda: m.moe_rmsnorm(bf, w, 1e-6, out={"y": bf[:2]}),
                 lambda: m.moe_rmsnorm_backward(bf, bf[:2], w, rstd), lambda: m.moe_rmsnorm_backward(bf, bf, w, rstd[:2]),
                 lambda: m.moe_layer_forward_ckpt(lg, bf, wgu, wd, 3), lambda: m.moe_layer_forward_ckpt(lg, bf, wgu, wd, 0),
                 lambda: m.moe_layer_forward_ckpt(lg[:2], bf, wgu, wd, 1),
                 lambda: m.moe_layer_forward_ckpt(lg, bf, wgu[:, :32].contiguous(), wd, 1),
                 lambda: m.moe_layer_forward_ckpt(lg, bf, wgu, wd, 1, shared_gate_up=wgu[0]),
                 lambda: m.moe_layer_forward_ckpt(lg, bf, wgu, wd, 1, x8=(q, s[:2])),
                 lambda: m.moe_layer_forward_ckpt(lg, bf, wgu, wd, 1, state={"gu_q": q}),
                 lambda: m.moe_grouped_mlp_backward_ckpt(bf[:2], st, wgu, wd),
                 lambda: m.moe_grouped_mlp_backward_ckpt(bf, {**st, "gu_scale": st["gu_scale"][:1]}, wgu, wd),
                 lambda: m.moe_grouped_mlp_backward_ckpt(bf, st, wgu, wd, grads={"dx": bf[:2]})):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(m.MoEError, match="UNSUPPORTED"):
        m.moe_rmsnorm(torch.zeros(2, 20, dtype=torch.bfloat16, device="cuda"), w[:20].contiguous(), 1e-6)
    with pytest.raises(m.MoEError, match="WORKSPACE"):
        m.moe_rmsnorm_backward(bf, bf, w, rstd, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
