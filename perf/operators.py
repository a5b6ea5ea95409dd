"""The layers a hybrid stack puts beside the Mesa layer, as measured work.

Two operators, each with its training and its decode form:

  lru   a gated linear recurrence over time (real-gated linear recurrent unit):
            r = sigmoid(gate_a), i = sigmoid(gate_x), log a = -8 softplus(lam) r
            h_t = a_t h_{t-1} + sqrt(1 - a_t^2) (i_t x_t),   y = h
  swa   causal attention over a sliding window whose first `sinks` tokens stay
        visible: query position p sees key j if j <= p and (j > p - window or
        j < sinks); heads of queries may share heads of keys and values.

``run`` computes a case in plain torch (own = False) or through the package's
public calls (own = True). ``exact`` restates each operator in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

LRU_C = 8.0


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def listed():
    return [
        # one layer of the benchmark's shape: batch 8, 8192 tokens, 16 heads of 128 channels
        dict(name="lru_forward_bf16", op="lru_forward", dtype="bf16", B=8, T=8192, D=2048),
        # one long document: nothing but the time axis to split
        dict(name="lru_forward_long", op="lru_forward", dtype="bf16", B=1, T=65536, D=1024),
        # training step of a layer, activations in bf16
        dict(name="lru_train_bf16", op="lru_train", dtype="bf16", B=8, T=2048, D=2048),
        # training in float32 with a ragged length and an odd width
        dict(name="lru_train_f32_ragged", op="lru_train", dtype="f32", B=3, T=2037, D=1003),
        # one decoded token for a batch of sequences: a call's latency
        dict(name="lru_step", op="lru_step", dtype="bf16", B=64, D=2048),
        # prefill at the benchmark's heads and length, the customary window of 1024
        dict(name="swa_forward_bf16", op="swa_forward", dtype="bf16", B=4, Hq=16, Hkv=16, T=8192, S=8192, d=128,
             window=1024, sinks=4),
        # a later piece of a prompt against its history: shared heads, ragged sizes, narrow heads
        dict(name="swa_forward_ragged", op="swa_forward", dtype="bf16", B=2, Hq=12, Hkv=4, T=1337, S=2741, d=64,
             window=515, sinks=7),
        # training step of an attention layer, shared key-value heads
        dict(name="swa_train_bf16", op="swa_train", dtype="bf16", B=2, Hq=16, Hkv=4, T=8192, S=8192, d=128,
             window=1024, sinks=4),
        # the float32 mode, small and ragged
        dict(name="swa_train_f32", op="swa_train", dtype="f32", B=1, Hq=4, Hkv=2, T=777, S=777, d=64, window=128,
             sinks=4),
        # serving: one token for a batch of sequences over full rolling caches
        dict(name="swa_step_batch", op="swa_step", dtype="bf16", B=64, Hq=16, Hkv=4, d=128, window=4096, sinks=4),
        # serving: a single sequence with a long window, the cache's length is all there is to split
        dict(name="swa_step_single", op="swa_step", dtype="bf16", B=1, Hq=16, Hkv=2, d=128, window=16384, sinks=4),
        # the smallest call: a short window, few heads
        dict(name="swa_step_small", op="swa_step", dtype="bf16", B=3, Hq=8, Hkv=8, d=64, window=256, sinks=1),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["lru_forward", "lru_train", "lru_step", "swa_forward", "swa_train", "swa_step"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "lru_step":
        return dict(op=op, dtype=dtype, B=_log_int(rng, 1, 512), D=_log_int(rng, 1, 8192))
    if op in ("lru_forward", "lru_train"):
        limit = 1 << (26 if op == "lru_forward" else 24)
        B = _log_int(rng, 1, 16)
        D = _log_int(rng, 16, 4096)
        T = _log_int(rng, 1, max(1, min(65536, limit // (B * D))))
        return dict(op=op, dtype=dtype, B=B, T=T, D=D)
    Hkv = rng.choice([1, 2, 3, 4, 8])
    group = rng.choice([1, 1, 2, 3, 4, 8])
    d = rng.choice([16, 32, 64, 64, 128, 128, 128])
    sinks = rng.choice([0, 1, 4, rng.randint(0, 128)])
    if op == "swa_step":
        window = _log_int(rng, 1, 16384)
        B = _log_int(rng, 1, max(1, min(64, (1 << 20) // (Hkv * (window + sinks)))))
        return dict(op=op, dtype=dtype, B=B, Hq=Hkv * group, Hkv=Hkv, d=d, window=window, sinks=sinks)
    big = 8192 if dtype == "bf16" else 2048
    T = _log_int(rng, 1, big)
    S = T if rng.random() < 0.6 else min(big, T + _log_int(rng, 1, big))
    window = _log_int(rng, 1, 2048)
    budget = (1 << 37) if dtype == "bf16" else (1 << 32)
    B = rng.randint(1, 4)
    case = dict(op=op, dtype=dtype, B=B, Hq=Hkv * group, Hkv=Hkv, T=T, S=max(S, T), d=d, window=window, sinks=sinks)
    while work(case)["flops"] > budget and case["T"] > 1:
        cut = case["T"] - case["T"] // 2
        case["T"] -= cut
        case["S"] -= cut
    return case


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt = _dtype(case)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev)

    st = dict(case=dict(case))
    op = case["op"]
    if op.startswith("lru"):
        B, D = case["B"], case["D"]
        # decays at full gate uniform in [0.9, 0.999]: log a = -8 softplus(lam)
        a = 0.9 + 0.099 * torch.rand(D, generator=g, device=dev, dtype=torch.float64)
        st["lam"] = torch.log(torch.expm1(-torch.log(a) / LRU_C)).float()
        shape = (B, D) if op == "lru_step" else (B, case["T"], D)
        st["x"] = normal(*shape).to(dt)
        st["gate_a"] = normal(*shape).to(dt)
        st["gate_x"] = normal(*shape).to(dt)
        st["h"] = normal(B, D)                         # state carried in from before the call
        if op == "lru_train":
            st["dy"] = normal(*shape).to(dt)
            st["dh"] = normal(B, D)                    # gradient of the state handed on
        if op == "lru_step":
            st["h_next"] = torch.empty_like(st["h"])
        return st
    B, Hq, Hkv, d = case["B"], case["Hq"], case["Hkv"], case["d"]
    # queries share a direction that the first keys answer to, as trained sinks do
    u = normal(d)
    u = u / u.norm() * d ** 0.5
    if op == "swa_step":
        W, n0 = case["window"], case["sinks"]
        st["q"] = (normal(B, Hq, d) + 0.5 * u).to(dt)
        st["k"] = normal(B, Hkv, d).to(dt)
        st["v"] = normal(B, Hkv, d).to(dt)
        kc = normal(B, Hkv, n0 + W, d)
        kc[:, :, :n0] += 0.3 * u
        st["k_cache"] = kc.to(dt)
        st["v_cache"] = normal(B, Hkv, n0 + W, d).to(dt)
        # most sequences are past the window, every fourth is still filling it
        pos = n0 + W + torch.randint(0, 4 * (n0 + W), (B,), generator=g, device=dev)
        young = torch.randint(0, n0 + W, (B,), generator=g, device=dev)
        late = torch.arange(B, device=dev) % 4 == 3
        st["pos"] = torch.where(late, young, pos).to(torch.int32)
        return st
    T, S = case["T"], case["S"]
    st["q"] = (normal(B, Hq, T, d) + 0.5 * u).to(dt)
    k = normal(B, Hkv, S, d)
    k[:, :, :case["sinks"]] += 0.3 * u
    st["k"] = k.to(dt)
    st["v"] = normal(B, Hkv, S, d).to(dt)
    if op == "swa_train":
        st["dout"] = normal(B, Hq, T, d).to(dt)
    return st


# --------------------------------------------------------------------------
# plain forms
# --------------------------------------------------------------------------

def _lru_gates(x, gate_a, gate_x, lam):
    x, ga, gx = x.float(), gate_a.float(), gate_x.float()
    r = torch.sigmoid(ga)
    i = torch.sigmoid(gx)
    la = -LRU_C * torch.log1p(torch.exp(-lam.abs())).add(lam.clamp(min=0)) * r
    a = torch.exp(la)
    m = torch.sqrt(-torch.expm1(2 * la))
    return x, r, i, la, a, m


def _scan(a, b, h0):
    """h_t = a_t h_{t-1} + b_t along dim 1: blocks side by side, then their carries."""
    B, T, D = a.shape
    L = max(1, int(math.isqrt(T)))
    n = -(-T // L)
    if n * L != T:
        pad = n * L - T
        a = torch.cat([a, a.new_ones(B, pad, D)], 1)
        b = torch.cat([b, b.new_zeros(B, pad, D)], 1)
    a = a.view(B, n, L, D)
    b = b.view(B, n, L, D)
    h = torch.empty_like(b)
    p = torch.empty_like(a)
    h[:, :, 0] = b[:, :, 0]
    p[:, :, 0] = a[:, :, 0]
    for t in range(1, L):
        h[:, :, t] = a[:, :, t] * h[:, :, t - 1] + b[:, :, t]
        p[:, :, t] = a[:, :, t] * p[:, :, t - 1]
    carry = torch.empty(B, n, D, device=a.device, dtype=a.dtype)
    c = h0
    for j in range(n):
        carry[:, j] = c
        c = p[:, j, -1] * c + h[:, j, -1]
    h += p * carry[:, :, None]
    return h.view(B, n * L, D)[:, :T]


def _plain_lru_forward(x, gate_a, gate_x, lam, h0):
    xf, r, i, la, a, m = _lru_gates(x, gate_a, gate_x, lam)
    h = _scan(a, m * i * xf, h0)
    return h


def _plain_lru_train(x, gate_a, gate_x, lam, h0, dy, dh):
    xf, r, i, la, a, m = _lru_gates(x, gate_a, gate_x, lam)
    h = _scan(a, m * i * xf, h0)
    prev = torch.cat([h0[:, None], h[:, :-1]], 1)
    # g_t = dy_t + a_{t+1} g_{t+1}, run from the end
    a_next = torch.cat([a[:, 1:], torch.ones_like(a[:, :1])], 1)
    g = _scan(a_next.flip(1), dy.float().flip(1), dh).flip(1)
    dx = g * m * i
    dgx = g * m * xf * i * (1 - i)
    # a dm/da through log a: dm = -a^2/m dlog a, kept as (-la/m) so that a -> 1 stays finite
    ratio = torch.where(m > 0, -la / m.clamp(min=1e-38), torch.zeros_like(m))
    s = g * (a * prev * la + i * xf * a * a * ratio)              # dL/dlog a times log a
    dga = s * (1 - r)
    sp = torch.log1p(torch.exp(-lam.abs())).add(lam.clamp(min=0))
    dlam = s.double().sum((0, 1)).float() * torch.sigmoid(lam) / sp
    dh0 = a[:, 0] * g[:, 0]
    return h, dx, dga, dgx, dlam, dh0


def _plain_swa(q, k, v, window, sinks, dout=None, block=512):
    B, Hq, T, d = q.shape
    Hkv, S = k.shape[1], k.shape[2]
    G = Hq // Hkv
    off = S - T
    scale = d ** -0.5
    qf = q.float().view(B, Hkv, G, T, d)
    kf, vf = k.float(), v.float()
    out = torch.empty_like(qf)
    lse = torch.empty(B, Hkv, G, T, device=q.device)
    if dout is not None:
        dof = dout.float().view(B, Hkv, G, T, d)
        dq, dk, dv = torch.empty_like(qf), torch.zeros_like(kf), torch.zeros_like(vf)
    for t0 in range(0, T, block):
        t1 = min(T, t0 + block)
        lo = max(0, off + t0 - window + 1)
        first = min(sinks, lo)
        idx = torch.cat([torch.arange(0, first, device=q.device), torch.arange(lo, off + t1, device=q.device)])
        p = torch.arange(off + t0, off + t1, device=q.device)[:, None]
        seen = (idx <= p) & ((idx > p - window) | (idx < sinks))
        kb, vb = kf[:, :, idx], vf[:, :, idx]
        n = t1 - t0
        qb = qf[:, :, :, t0:t1].reshape(B, Hkv, G * n, d)
        s = (qb @ kb.transpose(-1, -2) * scale).view(B, Hkv, G, n, -1)
        s = s.masked_fill(~seen, float("-inf"))
        mx = s.amax(-1, keepdim=True)
        e = torch.exp(s - mx)
        z = e.sum(-1, keepdim=True)
        w = (e / z).view(B, Hkv, G * n, -1)
        o = w @ vb
        out[:, :, :, t0:t1] = o.view(B, Hkv, G, n, d)
        lse[:, :, :, t0:t1] = (mx + torch.log(z))[..., 0]
        if dout is not None:
            dob = dof[:, :, :, t0:t1].reshape(B, Hkv, G * n, d)
            dw = dob @ vb.transpose(-1, -2)
            ds = w * (dw - (dob * o).sum(-1, keepdim=True)) * scale
            dq[:, :, :, t0:t1] = (ds @ kb).view(B, Hkv, G, n, d)
            dkb = ds.transpose(-1, -2) @ qb
            dvb = w.transpose(-1, -2) @ dob
            dk[:, :, :first] += dkb[:, :, :first]
            dv[:, :, :first] += dvb[:, :, :first]
            dk[:, :, lo:off + t1] += dkb[:, :, first:]
            dv[:, :, lo:off + t1] += dvb[:, :, first:]
    out = out.view(B, Hq, T, d)
    lse = lse.view(B, Hq, T)
    if dout is None:
        return out, lse
    return out, lse, dq.view(B, Hq, T, d), dk, dv


def _plain_swa_step(q, k, v, k_cache, v_cache, pos, window, sinks):
    B, Hq, d = q.shape
    Hkv = k.shape[1]
    pos = pos.long()
    slot = torch.where(pos < sinks, pos, sinks + (pos - sinks).clamp(min=0) % window)
    rows = torch.arange(B, device=q.device)
    k_cache[rows, :, slot] = k
    v_cache[rows, :, slot] = v
    n = (pos + 1).clamp(max=sinks + window)                        # slots in use, the first n
    s = (q.float().view(B, Hkv, Hq // Hkv, d) @ k_cache.float().transpose(-1, -2)) * d ** -0.5
    used = torch.arange(sinks + window, device=q.device)[None] < n[:, None]
    s = s.masked_fill(~used[:, None, None], float("-inf"))
    e = torch.exp(s - s.amax(-1, keepdim=True))
    o = (e / e.sum(-1, keepdim=True)) @ v_cache.float()
    return o.view(B, Hq, d)


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------

def run(st):
    if own:
        return _run_own(st)
    c = st["case"]
    op, dt = c["op"], _dtype(c)
    if op == "lru_forward":
        h = _plain_lru_forward(st["x"], st["gate_a"], st["gate_x"], st["lam"], st["h"])
        return h.to(dt), h[:, -1].clone()
    if op == "lru_train":
        h, dx, dga, dgx, dlam, dh0 = _plain_lru_train(st["x"], st["gate_a"], st["gate_x"], st["lam"], st["h"],
                                                      st["dy"], st["dh"])
        return h.to(dt), h[:, -1].clone(), dx.to(dt), dga.to(dt), dgx.to(dt), dlam, dh0
    if op == "lru_step":
        xf, r, i, la, a, m = _lru_gates(st["x"], st["gate_a"], st["gate_x"], st["lam"])
        st["h_next"].copy_(a * st["h"] + m * i * xf)
        return st["h_next"].to(dt), st["h_next"]
    if op == "swa_forward":
        out, lse = _plain_swa(st["q"], st["k"], st["v"], c["window"], c["sinks"])
        return out.to(dt), lse
    if op == "swa_train":
        out, lse, dq, dk, dv = _plain_swa(st["q"], st["k"], st["v"], c["window"], c["sinks"], st["dout"])
        return out.to(dt), lse, dq.to(dt), dk.to(dt), dv.to(dt)
    out = _plain_swa_step(st["q"], st["k"], st["v"], st["k_cache"], st["v_cache"], st["pos"], c["window"], c["sinks"])
    return out.to(dt), st["k_cache"], st["v_cache"]


def _run_own(st):
    from test_sequence_layer_b200 import mesa
    c = st["case"]
    op = c["op"]
    if op == "lru_forward":
        return mesa.lru_forward(st["x"], st["gate_a"], st["gate_x"], st["lam"], h0=st["h"], return_state=True)
    if op == "lru_train":
        y, hT, saved = mesa.lru_forward(st["x"], st["gate_a"], st["gate_x"], st["lam"], h0=st["h"],
                                        return_state=True, return_saved=True)
        grads = mesa.lru_backward(st["x"], st["gate_a"], st["gate_x"], st["lam"], st["dy"], saved=saved, dh_T=st["dh"])
        return (y, hT) + tuple(grads)                  # dx, dgate_a, dgate_x, dlam, dh0
    if op == "lru_step":
        y = mesa.lru_step(st["x"], st["gate_a"], st["gate_x"], st["lam"], st["h"], h_out=st["h_next"])
        return y, st["h_next"]
    if op == "swa_forward":
        return mesa.swa_forward(st["q"], st["k"], st["v"], window=c["window"], sinks=c["sinks"], return_lse=True)
    if op == "swa_train":
        out, lse = mesa.swa_forward(st["q"], st["k"], st["v"], window=c["window"], sinks=c["sinks"], return_lse=True)
        grads = mesa.swa_backward(st["q"], st["k"], st["v"], out, lse, st["dout"], window=c["window"],
                                  sinks=c["sinks"])
        return (out, lse) + tuple(grads)               # dq, dk, dv
    out = mesa.swa_step(st["q"], st["k"], st["v"], st["k_cache"], st["v_cache"], st["pos"], window=c["window"],
                        sinks=c["sinks"])
    return out, st["k_cache"], st["v_cache"]


# --------------------------------------------------------------------------
# definitions in 64 bits
# --------------------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op.startswith("lru"):
        return _exact_lru(st, op)
    if op == "swa_step":
        return _exact_swa_step(st, case)
    return _exact_swa(st, case)


def _exact_lru(st, op):
    x, ga, gx = (st[n].double() for n in ("x", "gate_a", "gate_x"))
    lam, h = st["lam"].double(), st["h"].double()
    r, i = 1 / (1 + torch.exp(-ga)), 1 / (1 + torch.exp(-gx))
    sp = torch.logaddexp(lam, torch.zeros_like(lam))
    la = -LRU_C * sp * r
    a = torch.exp(la)
    m = torch.sqrt(-torch.expm1(2 * la))
    b = m * i * x
    if op == "lru_step":
        h = a * h + b
        return h, h
    T = x.shape[1]
    hs = torch.empty_like(b)
    h0 = h
    for t in range(T):
        h = torch.addcmul(b[:, t], a[:, t], h)
        hs[:, t] = h
    if op == "lru_forward":
        return hs, h
    del b
    g = torch.empty_like(hs)
    c = st["dh"].double()
    dy = st["dy"].double()
    for t in range(T - 1, -1, -1):
        c = dy[:, t] + c
        g[:, t] = c
        c = a[:, t] * c
    prev = torch.cat([h0[:, None], hs[:, :-1]], 1)
    dla = g * (a * prev - i * x * a * a / m)
    dlam = (dla * r).sum((0, 1)) * (-LRU_C) / (1 + torch.exp(-lam))
    dga = dla * (-LRU_C * sp) * r * (1 - r)
    return hs, hs[:, -1], g * m * i, dga, g * m * x * i * (1 - i), dlam, c


def _exact_swa(st, case):
    B, Hq, Hkv, T, S, d = (case[n] for n in ("B", "Hq", "Hkv", "T", "S", "d"))
    dev = st["q"].device
    p = torch.arange(S - T, S, device=dev)[:, None]
    j = torch.arange(S, device=dev)[None]
    hidden = ~((j <= p) & ((p - j < case["window"]) | (j < case["sinks"])))
    train = case["op"] == "swa_train"
    out = torch.empty(B, Hq, T, d, dtype=torch.float64, device=dev)
    lse = torch.empty(B, Hq, T, dtype=torch.float64, device=dev)
    if train:
        dq = torch.empty_like(out)
        dk = torch.zeros(B, Hkv, S, d, dtype=torch.float64, device=dev)
        dv = torch.zeros_like(dk)
    for b in range(B):
        for h in range(Hq):
            q, k, v = st["q"][b, h].double(), st["k"][b, h // (Hq // Hkv)].double(), \
                st["v"][b, h // (Hq // Hkv)].double()
            s = torch.mm(q, k.t()).div_(math.sqrt(d)).masked_fill_(hidden, float("-inf"))
            z = torch.logsumexp(s, -1)
            w = s.sub_(z[:, None]).exp_()
            lse[b, h] = z
            out[b, h] = w @ v
            if train:
                do = st["dout"][b, h].double()
                dw = do @ v.t()
                dv[b, h // (Hq // Hkv)] += w.t() @ do
                ds = w.mul_(dw - (w * dw).sum(-1, keepdim=True)).div_(math.sqrt(d))
                dq[b, h] = ds @ k
                dk[b, h // (Hq // Hkv)] += ds.t() @ q
    return (out, lse, dq, dk, dv) if train else (out, lse)


def _exact_swa_step(st, case):
    B, Hq, Hkv, d, W, n0 = (case[n] for n in ("B", "Hq", "Hkv", "d", "window", "sinks"))
    q = st["q"].double()
    kc, vc = st["k_cache"].double(), st["v_cache"].double()
    out = torch.empty(B, Hq, d, dtype=torch.float64, device=q.device)
    for b in range(B):
        p = int(st["pos"][b])
        own_slot = p if p < n0 else n0 + (p - n0) % W
        kc[b, :, own_slot] = st["k"][b].double()
        vc[b, :, own_slot] = st["v"][b].double()
        # where each visible position lies in the rolling cache
        seen = list(range(min(n0, p + 1))) + list(range(max(n0, p - W + 1), p + 1))
        at = torch.tensor([x if x < n0 else n0 + (x - n0) % W for x in seen], device=q.device)
        for h in range(Hq):
            kv = h // (Hq // Hkv)
            w = torch.softmax(kc[b, kv, at] @ q[b, h] / math.sqrt(d), 0)
            out[b, h] = w @ vc[b, kv, at]
    return out, kc, vc


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------

def _pairs(T, S, window, sinks):
    """Visible (query, key) pairs of one head."""
    def tri(n):                                        # sum of 1..n
        return n * (n + 1) // 2

    def visible(n):                                    # sum over the first n positions of the keys each one sees
        cap = window + sinks                           # most keys a position sees
        full = max(0, n - cap)
        return tri(n - full) + full * cap
    return visible(S) - visible(S - T)


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    B = case["B"]
    if op.startswith("lru"):
        D = case["D"]
        n = B * case.get("T", 1) * D
        if op == "lru_step":
            return dict(bytes=n * (4 * e + 8) + 4 * D, flops=25 * n)
        if op == "lru_forward":
            return dict(bytes=n * 4 * e + 8 * B * D + 4 * D, flops=25 * n)
        # forward: three tensors in, one out; backward: four in, three out
        return dict(bytes=n * 11 * e + 16 * B * D + 12 * D, flops=80 * n)
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    if op == "swa_step":
        # the cache's used part is at most the whole of it; every fourth sequence fills half on average
        n = case["window"] + case["sinks"]
        late = B // 4
        used = (B - late) * n + late * (n + 1) // 2
        return dict(bytes=2 * used * Hkv * d * e + B * (2 * Hq + 4 * Hkv) * d * e + 4 * B, flops=4 * used * Hq * d)
    T, S = case["T"], case["S"]
    pairs = B * Hq * _pairs(T, S, case["window"], case["sinks"])
    qb, kb = B * Hq * T * d * e, B * Hkv * S * d * e
    lse = 4 * B * Hq * T
    if op == "swa_forward":
        return dict(bytes=2 * qb + 2 * kb + lse, flops=4 * pairs * d)
    # forward, then q, k, v, out, lse, dout in and dq, dk, dv out
    return dict(bytes=2 * qb + 2 * kb + lse + 4 * qb + 4 * kb + lse, flops=14 * pairs * d)
