"""The gated linear recurrence and sliding-window attention in 64 bits, each
with a bound on the error a call of the library may make against it.

The bounds follow the roundings of the arithmetic, term by term: U = 2^-24 is
half a step of fp32, the fast exponential errs by 2 + 1.2 |x| steps, the fast
division by 2; every output is rounded once more, by at most half a step of
its type (finfo.eps / 2)."""
import torch

U = 2.0 ** -24
STEP = 2.0 ** -23


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def pieces(x, ga, gx, lam):
    """(r, i, la, a, m, b) of the recurrence and relative bounds (ur, ui, ula, ua, um2, ub)."""
    x, ga, gx, lam = (t.double() for t in (x, ga, gx, lam))
    r, i = torch.sigmoid(ga), torch.sigmoid(gx)
    sp = torch.logaddexp(lam, torch.zeros_like(lam))
    la = -8 * sp * r
    a = torch.exp(la)
    m2 = -torch.expm1(2 * la)
    m = m2.sqrt()
    b = m * i * x

    def usig(v):
        # e^-v enters 1 + e^-v at most in full
        return (6 + 1.2 * v.abs().clamp(max=88)) * STEP

    ur, ui = usig(ga), usig(gx)
    ula = ur + 6 * STEP
    ua = la.abs().clamp(max=120) * ula + (2 + 1.2 * la.abs().clamp(max=120)) * STEP
    # series below |2 la| = 1/4 (8 roundings and the term left out), 1 - a^2 above it
    um2 = torch.where(2 * la.abs() < 0.24, ula + 10 * STEP, 2 * a * a * ua / m2.clamp(min=0.2) + 2 * STEP + ula)
    ub = um2 / 2 + ui + 5 * STEP
    return (r, i, la, a, m, b, sp), (ur, ui, ula, ua, um2, ub)


def lru(x, ga, gx, lam, h0=None):
    """y, h_T and the bounds on their errors before the rounding to y's type."""
    (r, i, la, a, m, b, sp), (ur, ui, ula, ua, um2, ub) = pieces(x, ga, gx, lam)
    B, T, D = b.shape
    h = torch.zeros(B, D, dtype=torch.float64, device=b.device) if h0 is None else h0.double()
    e = torch.zeros_like(h)
    hs, es = torch.empty_like(b), torch.empty_like(b)
    for t in range(T):
        # parts of a run are composed, so a product of a's is rounded at most twice per token
        e = a[:, t] * e + (a[:, t] * h).abs() * (ua[:, t] + 4 * U) + b[:, t].abs() * (ub[:, t] + 4 * U)
        h = a[:, t] * h + b[:, t]
        e = e + 2 * U * h.abs() + 1e-37
        hs[:, t], es[:, t] = h, e
    return hs, h, es, e


def lru_grads(x, ga, gx, lam, h0, dy, dhT):
    """(dx, dga, dgx, dlam, dh0) and bounds on their errors before the final rounding."""
    (r, i, la, a, m, b, sp), (ur, ui, ula, ua, um2, ub) = pieces(x, ga, gx, lam)
    B, T, D = b.shape
    zero = torch.zeros(B, D, dtype=torch.float64, device=b.device)
    h0 = zero if h0 is None else h0.double()
    hs, _, es, _ = lru(x, ga, gx, lam, h0)
    hp, ep = torch.cat([h0[:, None], hs[:, :-1]], 1), torch.cat([zero[:, None], es[:, :-1]], 1)
    ep = ep + 4 * U * hp.abs()
    c = zero if dhT is None else dhT.double()
    e = zero
    g, eg = torch.empty_like(hs), torch.empty_like(hs)
    dy = dy.double()
    for t in range(T - 1, -1, -1):
        c = c + dy[:, t]
        e = e + 2 * U * c.abs()
        g[:, t], eg[:, t] = c, e
        e = a[:, t] * e + (a[:, t] * c).abs() * (ua[:, t] + 4 * U) + 1e-37
        c = a[:, t] * c
    ratio = torch.where(la < 0, la / (m * m).clamp(min=1e-300), torch.full_like(la, -0.5))
    first, second = a * hp * la, b * a * a * ratio
    s = g * (first - second)
    es_ = eg * (first - second).abs() + g.abs() * (
        (a * la).abs() * ep + first.abs() * (ua + ula + 6 * STEP) + second.abs() * (2 * ua + ub + ula + um2 + 8 * STEP))
    xd = x.double()
    dx = g * m * i
    edx = eg * m * i + dx.abs() * (um2 / 2 + ui + 6 * STEP)
    dgx = g * m * i * xd * (1 - i)
    # 1 - i loses what i carries: an absolute error ui * i
    edgx = eg * (b * (1 - i)).abs() + (g * b).abs() * ((1 - i) * (ub + 6 * STEP) + i * ui + STEP)
    dga = s * (1 - r)
    edga = es_ * (1 - r) + s.abs() * (r * ur + STEP + (1 - r) * 2 * STEP)
    factor = torch.sigmoid(lam.double()) / sp.clamp(min=1e-300)
    factor = torch.where(sp > 0, factor, torch.ones_like(factor))
    dlam = s.sum((0, 1)) * factor
    adds = 8 + T / 64 + 8 + 8 * B + 16
    edlam = factor * (es_.sum((0, 1)) + s.abs().sum((0, 1)) * adds * U) + dlam.abs() * 10 * STEP
    return (dx, dga, dgx, dlam, c), (edx, edga, edgx, edlam, e)


def check(got, ref, bound, what):
    """|got - ref| <= bound + half a step of got's type, everywhere."""
    hs = half_step(got.dtype)
    lim = bound + hs * (ref.abs() + bound) + (1e-40 if got.dtype == torch.float32 else 1e-38)
    bad = ~((got.double() - ref).abs() <= lim)
    if bad.any():
        w = ((got.double() - ref).abs() / lim).nan_to_num(float("inf"))
        k = int(w.argmax())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float(w.max()):.3g} times the "
                             f"bound at {k} (got {float(got.flatten()[k])}, want {float(ref.flatten()[k])})")


def hidden(T, S, window, sinks, device):
    p = torch.arange(S - T, S, device=device)[:, None]
    j = torch.arange(S, device=device)[None]
    return ~((j <= p) & ((p - j < window) | (j < sinks)))


def swa(q, k, v, window, sinks, scale=None, matrix=False, dout=None):
    """{name: (value, bound)} of out and lse, and of dq, dk, dv where dout is
    given. `matrix`: weights and dS are rounded to bf16 before their products.
    The gradients' bound takes `out` as rounded to q's type."""
    B, Hq, T, d = q.shape
    G = Hq // k.shape[1]
    S = k.shape[2]
    scale = d ** -0.5 if scale is None else scale
    qd, kd, vd = q.double(), k.double().repeat_interleave(G, 1), v.double().repeat_interleave(G, 1)
    hid = hidden(T, S, window, sinks, q.device)
    s = (qd @ kd.transpose(-1, -2) * scale).masked_fill(hid, float("-inf"))
    # a score errs by d + 4 roundings of its terms
    es = (qd.abs() @ kd.abs().transpose(-1, -2) * scale).masked_fill(hid, 0.0) * (d + 4) * U
    es = es.amax(-1, keepdim=True) + s.masked_fill(hid, 0.0).abs().amax(-1, keepdim=True) * 4 * U
    lse = torch.logsumexp(s, -1)
    w = torch.exp(s - lse[..., None])
    out = w @ vd
    # exponent within 2 es of the truth, the exponential's own error, n + 8 additions
    spread = (s.amax(-1, keepdim=True) - s.masked_fill(hid, 0.0).amin(-1, keepdim=True)).clamp(min=0)
    uw = 2 * es + (12 + 3 * spread) * STEP + (S / 16 + 64) * U
    up = uw + (half_step(torch.bfloat16) if matrix else 0.0)
    res = {"lse": (lse, (es + (S / 16 + 64) * U + (4 + 2 * spread) * STEP)[..., 0] + 4 * U * lse.abs())}
    eout = (w * (up + uw)) @ vd.abs() + (S + 8) * U * (w @ vd.abs())
    res["out"] = (out, eout)
    if dout is None:
        return res
    do = dout.double()
    dw = do @ vd.transpose(-1, -2)
    edw = (do.abs() @ vd.abs().transpose(-1, -2)) * (d + 2) * U
    delta = (do * out).sum(-1, keepdim=True)
    eout_r = eout + half_step(q.dtype) * (out.abs() + eout)
    edelta = (do.abs() * eout_r).sum(-1, keepdim=True) + (do * out).abs().sum(-1, keepdim=True) * (d + 2) * U
    ds = w * (dw - delta) * scale
    rds = half_step(torch.bfloat16) if matrix else 0.0
    eds = w * scale * ((dw - delta).abs() * (uw + 4 * STEP) + edw + edelta) * (1 + rds) + ds.abs() * rds

    def shared(t):                       # sum over the query heads of a shared head
        return t.view(B, k.shape[1], G, S, d).sum(2)
    res["dq"] = (ds @ kd, eds @ kd.abs() + (S + 8) * U * (ds.abs() @ kd.abs()))
    n = (T * G + 16) * U
    res["dk"] = (shared(ds.transpose(-1, -2) @ qd),
                 shared(eds.transpose(-1, -2) @ qd.abs() + n * (ds.abs().transpose(-1, -2) @ qd.abs())))
    wt = w.transpose(-1, -2)
    res["dv"] = (shared(wt @ do), shared((w * up).transpose(-1, -2) @ do.abs() + n * (wt @ do.abs())))
    return res


def matrix_path(dtype, d):
    return dtype == torch.bfloat16 and d in (64, 128)
