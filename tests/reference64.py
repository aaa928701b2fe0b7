"""Plain 64-bit implementations (torch, CPU) of the 8-bit row format, the RMSNorm
and the layer with its 8-bit training state, for the tests of those operators.

Rounding constants: a rounding to bf16 is off by at most 2^-8 of the value, to
fp32 by 2^-24, to E4M3 by 2^-4 (or by 2^-10 times the block's scale below the
normal range). Sums on the tensor cores are taken to be off by at most 2^-23 of
the sum of magnitudes per term: fp32 accumulation that may truncate.
"""
import torch

BF16, F32, TC = 2.0 ** -8, 2.0 ** -24, 2.0 ** -23
BLOCK = 32


def blocks(cols):
    return -(-cols // BLOCK)


def round_e4m3(v):
    """float64 -> nearest E4M3 value (ties to even), |v| <= 448 taken for granted."""
    m, ex = torch.frexp(v)                                  # |v| = m 2^ex, m in [0.5, 1)
    step = torch.exp2((torch.clamp(ex - 1, min=-6) - 3).double())
    return torch.round(v / step) * step


def exponents(a):
    """The exponent of blocks whose largest magnitudes are a (float64)."""
    m, ex = torch.frexp(a)                                  # 448 = 0.875 * 2^9
    e = torch.where(m <= 0.875, ex - 9, ex - 8)
    return torch.where(a == 0, torch.full_like(e, -124), e).clamp(-124, 120)


def split_blocks(v, parts):
    """Rows [R, parts * cols] as [R, parts * S, 32], zero-padded, and a function back."""
    R, width = v.shape
    cols = width // parts
    S = blocks(cols)
    p = torch.zeros(R, parts, S * BLOCK, dtype=v.dtype)
    p[:, :, :cols] = v.reshape(R, parts, cols)
    return (p.reshape(R, parts * S, BLOCK),
            lambda b: b.reshape(R, parts, S * BLOCK)[:, :, :cols].reshape(R, width))


def quantize(v, parts=1):
    """(values that the rows stand for, scale bytes [R, blocks]) of float64 rows."""
    b, back = split_blocks(v, parts)
    fin = torch.isfinite(b)
    mag = torch.where(fin, b.abs(), torch.zeros_like(b))
    e = exponents(mag.amax(dim=2))
    scale = torch.exp2(e.double())[:, :, None]
    q = round_e4m3(torch.where(fin, b, torch.zeros_like(b)) / scale)
    q = torch.where((e == 120)[:, :, None], q.clamp(-240, 240), q) * scale   # 256 * 2^120 is past bf16
    q = torch.where(fin, q, torch.full_like(q, float("nan")))
    return back(q), (e + 127).to(torch.uint8)


def decode(q, scale, parts=1):
    """float64 values of E4M3 bytes [R, parts * cols] with scale bytes [R, blocks]."""
    b = q.to(torch.int64)
    ex, fr = (b >> 3) & 15, (b & 7).double()
    v = torch.where(ex > 0, (1 + fr / 8) * torch.exp2((ex - 7).double()), fr * 2.0 ** -9)
    v = torch.where(b >= 128, -v, v)
    v = torch.where((b & 127) == 127, torch.full_like(v, float("nan")), v)
    vb, back = split_blocks(v, parts)
    return back(vb * torch.exp2(scale.double() - 127)[:, :, None])


def per_column(per_block, cols, parts=1):
    """Values [R, parts * S] spread over their blocks' columns [R, parts * cols]."""
    R = per_block.shape[0]
    return per_block.reshape(R, parts, -1, 1).expand(-1, -1, -1, BLOCK).reshape(R, parts, -1)[:, :, :cols].reshape(
        R, parts * cols)


# ------------------------------------------------------------------ RMSNorm
def rmsnorm(s, w, eps):
    """y, rstd of float64 rows s."""
    rstd = 1.0 / torch.sqrt((s * s).sum(dim=1) / s.shape[1] + eps)
    return s * rstd[:, None] * w, rstd


def rmsnorm_backward(dy, s, w, rstd, dsum=None):
    xhat = s * rstd[:, None]
    c = (w * dy * xhat).sum(dim=1, keepdim=True) / s.shape[1]
    dx = rstd[:, None] * (w * dy - xhat * c)
    return dx if dsum is None else dx + dsum, (dy * xhat).sum(dim=0)


# -------------------------------------------------------------------- layer
def silu_parts(g):
    s = 1.0 / (1.0 + torch.exp(-g))
    return s, g * s


def mlp_rows(x_rows, w_gate_up, w_down, offsets):
    """g, u, y by row for expert-contiguous rows."""
    I = w_down.shape[1]
    gu = torch.zeros(x_rows.shape[0], 2 * I, dtype=torch.float64)
    y = torch.zeros(x_rows.shape[0], w_down.shape[2], dtype=torch.float64)
    for e in range(w_down.shape[0]):
        a, b = int(offsets[e]), int(offsets[e + 1])
        gu[a:b] = x_rows[a:b] @ w_gate_up[e]
        y[a:b] = (silu_parts(gu[a:b, :I])[1] * gu[a:b, I:]) @ w_down[e]
    return gu, y


def token_of_row(row_of):
    T, k = row_of.shape
    tok = torch.empty(T * k, dtype=torch.int64)
    tok[row_of.reshape(-1).long()] = torch.arange(T)[:, None].expand(T, k).reshape(-1)
    return tok


def layer_backward(dout, x, gu, p, w_gate_up, w_down, row_of, offsets):
    """Gradients {dx, dw_gate_up, dw_down, dprob} and, by the same keys with
    "_tol", how far the kernels' results may be from them: every rounding that
    they make, carried through the products in magnitude."""
    T, H = dout.shape
    E, I, _ = w_down.shape
    tok = token_of_row(row_of)
    A = tok.numel()
    pr = torch.empty(A, dtype=torch.float64)
    pr[row_of.reshape(-1).long()] = p.reshape(-1)
    r = {"dw_gate_up": torch.zeros(E, H, 2 * I, dtype=torch.float64), "dw_down": torch.zeros(E, I, H, dtype=torch.float64)}
    tol = {n: torch.zeros_like(v) for n, v in r.items()}
    dot, dot_tol = torch.zeros(A, dtype=torch.float64), torch.zeros(A, dtype=torch.float64)
    dxr, dxr_tol = torch.zeros(A, H, dtype=torch.float64), torch.zeros(A, H, dtype=torch.float64)
    for e in range(E):
        a, b = int(offsets[e]), int(offsets[e + 1])
        n = b - a
        if n == 0:
            continue
        dy, xe = dout[tok[a:b]], x[tok[a:b]]
        g, u, pe = gu[a:b, :I], gu[a:b, I:], pr[a:b, None]
        s, silu = silu_parts(g)
        act = silu * u
        dh = dy @ w_down[e].T
        # fp32 products of H terms; the sigmoid s: __expf is off by 2 + 1.173 |g| ulp (2 F32 each), which moves
        # s by (1 - s) times that, __fdividef by 2 ulp; and the few products after it: 8 fp32 roundings
        dh_tol = H * TC * (dy.abs() @ w_down[e].abs().T)
        few = (8 + 2 * 2 + 2 * (2 + 1.173 * g.abs())) * F32
        dot[a:b] = (dh * act).sum(dim=1)
        dot_tol[a:b] = (dh_tol * act.abs() + (few + (64 + I // 64 + 2) * F32) * (dh * act).abs()).sum(dim=1)
        slope = s + silu * (1 - s)
        # s + silu (1 - s): relative to its terms; and the rounding of s (5 F32) passes through 1 - s
        slope_tol = few * (s + silu.abs() * (1 - s)) + 5 * F32 * silu.abs() * s
        dgu = torch.cat([pe * dh * u * slope, pe * dh * silu], dim=1)
        from_dh = torch.cat([pe * u.abs() * slope.abs(), pe * silu.abs()], dim=1).abs() * dh_tol.repeat(1, 2)
        from_s = torch.cat([pe * u.abs() * slope_tol, few * pe * silu.abs()], dim=1).abs() * (dh.abs() + dh_tol).repeat(1, 2)
        dgu_tol = BF16 * dgu.abs() + (from_dh + from_s) * (1 + BF16)
        h, h_tol = pe * act, (BF16 + few) * (pe * act).abs()
        r["dw_down"][e] = h.T @ dy
        tol["dw_down"][e] = h_tol.T @ dy.abs() + n * TC * (h.abs().T @ dy.abs())
        r["dw_gate_up"][e] = xe.T @ dgu
        tol["dw_gate_up"][e] = xe.abs().T @ dgu_tol + n * TC * (xe.abs().T @ dgu.abs())
        dxr[a:b] = dgu @ w_gate_up[e].T
        dxr_tol[a:b] = dgu_tol @ w_gate_up[e].abs().T + 2 * I * TC * (dgu.abs() @ w_gate_up[e].abs().T)
    dxr_tol += BF16 * (dxr.abs() + dxr_tol)          # each row's dx is stored in bf16
    rows = row_of.long()
    r["dx"], tol["dx"] = dxr[rows].sum(dim=1), dxr_tol[rows].sum(dim=1) + row_of.shape[1] * F32 * dxr[rows].abs().sum(dim=1)
    r["dprob"], tol["dprob"] = dot[rows], dot_tol[rows]
    for n in ("dx", "dw_gate_up", "dw_down"):         # the stored result
        tol[n] = tol[n] + BF16 * (r[n].abs() + tol[n]) + 2.0 ** -133
    r.update({n + "_tol": v for n, v in tol.items()})
    return r


def assert_within(got, ref, tol, what):
    got, ref, tol = got.double().cpu(), ref.double(), tol.double()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), f"{what}: NaN in other places"
    err = torch.where(torch.isnan(ref) | (got == ref), torch.zeros_like(ref), (got - ref).abs())
    bad = ~(err <= tol) & ~torch.isnan(ref)
    if bad.any():
        at = tuple(int(i) for i in bad.nonzero()[0])
        worst = (err / tol.clamp(min=1e-300))[bad].max()
        raise AssertionError(f"{what}: {int(bad.sum())} of {ref.numel()} off; first at {at}: {got[at]} for {ref[at]} "
                             f"(tolerance {tol[at]}); worst {float(worst)} tolerances")
