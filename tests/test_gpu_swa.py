"""Sliding-window attention with sinks on the GPU against its definition in 64 bits."""
import pytest
import torch

import mixers_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mesa():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from test_sequence_layer_b200 import build, mesa
    build.build()
    return mesa


DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def inputs(B, Hq, Hkv, T, S, d, dtype, seed=0, gain=1.0):
    g = torch.Generator().manual_seed(seed)

    def one(*shape):
        return torch.randn(shape, generator=g).cuda()
    q, k, v, do = one(B, Hq, T, d), one(B, Hkv, S, d), one(B, Hkv, S, d), one(B, Hq, T, d)
    return (q * gain).to(DT[dtype]), k.to(DT[dtype]), v.to(DT[dtype]), do.to(DT[dtype])


# (B, Hq, Hkv, T, S, window, sinks)
CASES = [
    (1, 1, 1, 1, 1, 1, 0), (1, 2, 1, 1, 5, 3, 1), (2, 2, 2, 2, 2, 7, 1), (1, 1, 1, 5, 5, 1, 0), (1, 1, 1, 5, 5, 1, 2),
    (1, 3, 1, 63, 63, 20, 4), (1, 2, 2, 64, 64, 64, 0), (1, 4, 2, 65, 65, 64, 1), (2, 2, 1, 127, 127, 33, 3),
    (1, 2, 1, 128, 128, 128, 4), (1, 2, 1, 129, 129, 127, 4), (1, 4, 4, 200, 200, 500, 0), (1, 2, 1, 257, 257, 1, 4),
    (1, 2, 1, 300, 300, 100, 64), (1, 2, 1, 300, 300, 50, 65), (1, 2, 1, 400, 400, 90, 128), (1, 1, 1, 260, 260, 2, 128),
    (1, 2, 1, 1, 400, 100, 4), (2, 4, 2, 77, 333, 100, 5), (1, 2, 1, 130, 700, 129, 4), (1, 8, 1, 513, 513, 256, 4),
    (1, 2, 2, 129, 1000, 300, 0), (1, 16, 2, 200, 330, 140, 33), (1, 2, 1, 1000, 1000, 250, 17),
]


@pytest.mark.parametrize("d", [16, 32, 64, 128])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_forward_and_backward(mesa, case, dtype, d):
    B, Hq, Hkv, T, S, window, sinks = case
    q, k, v, do = inputs(B, Hq, Hkv, T, S, d, dtype, seed=T + S)
    kw = dict(window=window, sinks=sinks)
    out, lse = mesa.swa_forward(q, k, v, return_lse=True, **kw)
    want = ref.swa(q, k, v, window, sinks, matrix=ref.matrix_path(q.dtype, d), dout=do)
    ref.check(out, *want["out"], "out")
    ref.check(lse, *want["lse"], "lse")
    grads = mesa.swa_backward(q, k, v, out, lse, do, **kw)
    for n, g in zip(("dq", "dk", "dv"), grads):
        ref.check(g, *want[n], n)
    assert torch.equal(out, mesa.swa_forward(q, k, v, **kw))
    for a, b in zip(grads, mesa.swa_backward(q, k, v, out, lse, do, **kw)):
        assert torch.equal(a, b)                                      # no order of atomics in it


@pytest.mark.parametrize("dtype,d", [("f32", 32), ("bf16", 64), ("bf16", 128)])
def test_scale_and_large_scores(mesa, dtype, d):
    """A scale of the caller's, and scores far apart: the running maximum moves from tile to tile."""
    q, k, v, do = inputs(1, 2, 1, 300, 420, d, dtype, seed=2, gain=6.0)
    k *= torch.linspace(0.1, 3.0, 420, device="cuda").to(k)[:, None]
    for scale in (0.05, 0.3):
        out, lse = mesa.swa_forward(q, k, v, window=200, sinks=9, scale=scale, return_lse=True)
        want = ref.swa(q, k, v, 200, 9, scale=scale, matrix=ref.matrix_path(q.dtype, d), dout=do)
        ref.check(out, *want["out"], "out")
        ref.check(lse, *want["lse"], "lse")
        for n, g in zip(("dq", "dk", "dv"), mesa.swa_backward(q, k, v, out, lse, do, window=200, sinks=9, scale=scale)):
            ref.check(g, *want[n], n)


@pytest.mark.parametrize("dtype,d", [("f32", 16), ("bf16", 128)])
def test_gradients_against_differences(mesa, dtype, d):
    q, k, v, do = inputs(1, 4, 2, 90, 150, d, dtype, seed=3)
    out, lse = mesa.swa_forward(q, k, v, window=40, sinks=3, return_lse=True)
    grads = mesa.swa_backward(q, k, v, out, lse, do, window=40, sinks=3)
    want = ref.swa(q, k, v, 40, 3, matrix=ref.matrix_path(q.dtype, d), dout=do)
    args = [t.double() for t in (q, k, v)]
    gen = torch.Generator().manual_seed(1)
    for i, n in enumerate(("dq", "dk", "dv")):
        dr = torch.randn(args[i].shape, generator=gen, dtype=torch.float64).cuda()
        up, dn = list(args), list(args)
        up[i], dn[i] = args[i] + 1e-5 * dr, args[i] - 1e-5 * dr
        diff = sum(s * (ref.swa(*a, 40, 3)["out"][0] * do.double()).sum() for s, a in ((1, up), (-1, dn))) / 2e-5
        val, bound = want[n]
        slack = ((bound + ref.half_step(q.dtype) * (val.abs() + bound)) * dr.abs()).sum()
        assert abs(float(diff - (grads[i].double() * dr).sum())) <= float(slack) + 1e-5 * float((val * dr).abs().sum())


def test_no_queries(mesa):
    q, k, v, do = inputs(1, 2, 1, 0, 50, 64, "bf16")
    out, lse = mesa.swa_forward(q, k, v, window=10, return_lse=True)
    assert out.shape == q.shape and lse.shape == (1, 2, 0)
    dq, dk, dv = mesa.swa_backward(q, k, v, out, lse, do, window=10)
    assert torch.count_nonzero(dk) == 0 and torch.count_nonzero(dv) == 0


@pytest.mark.parametrize("dtype,d", [("f32", 64), ("bf16", 64), ("bf16", 128)])
def test_rows_behind_a_sequence_do_not_matter(mesa, dtype, d):
    """A right-padded batch: what the padding holds changes nothing before it, and
    zero gradients there leave it out of the sums."""
    T, n = 300, 211
    q, k, v, do = inputs(2, 2, 1, T, T, d, dtype, seed=4)
    do[1, :, n:] = 0
    kw = dict(window=64, sinks=4)
    out, lse = mesa.swa_forward(q, k, v, return_lse=True, **kw)
    g = mesa.swa_backward(q, k, v, out, lse, do, **kw)
    q2, k2, v2 = q.clone(), k.clone(), v.clone()
    q2[1, :, n:], k2[1, :, n:], v2[1, :, n:] = 100.0, -50.0, 1000.0
    out2, lse2 = mesa.swa_forward(q2, k2, v2, return_lse=True, **kw)
    g2 = mesa.swa_backward(q2, k2, v2, out2, lse2, do, **kw)
    assert torch.equal(out[1, :, :n], out2[1, :, :n]) and torch.equal(out[0], out2[0])
    for a, b in zip(g, g2):
        assert torch.equal(a[1, :, :n], b[1, :, :n]) and torch.count_nonzero(b[1, :, n:]) == 0


def test_stream_and_graph(mesa):
    a = inputs(1, 4, 2, 200, 260, 128, "bf16", seed=5)
    b = inputs(1, 4, 2, 200, 260, 128, "bf16", seed=6)
    q, k, v, do = (t.clone() for t in a)
    kw = dict(window=100, sinks=4)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = mesa.swa_forward(q, k, v, stream=s, **kw)
    s.synchronize()
    assert torch.equal(out, mesa.swa_forward(q, k, v, **kw))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        oc, lc = mesa.swa_forward(q, k, v, return_lse=True, **kw)
        gc = mesa.swa_backward(q, k, v, oc, lc, do, **kw)
    for t, n in zip((q, k, v, do), b):
        t.copy_(n)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    o, l = mesa.swa_forward(b[0], b[1], b[2], return_lse=True, **kw)
    assert torch.equal(oc, o) and torch.equal(lc, l)
    for x, y in zip(gc, mesa.swa_backward(b[0], b[1], b[2], o, l, b[3], **kw)):
        assert torch.equal(x, y)


def test_two_streams_at_once(mesa):
    """Calls that overlap, each with its own workspace."""
    sets = [inputs(2, 4, 2, 700, 700, 128, "bf16", seed=i) for i in (10, 11)]
    kw = dict(window=200, sinks=4)
    want = []
    for q, k, v, do in sets:
        o, l = mesa.swa_forward(q, k, v, return_lse=True, **kw)
        want.append((o, l) + mesa.swa_backward(q, k, v, o, l, do, **kw))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [None, None]
    for _ in range(3):
        for i, (s, (q, k, v, do)) in enumerate(zip(streams, sets)):
            o, l = mesa.swa_forward(q, k, v, return_lse=True, stream=s, **kw)
            got[i] = (o, l) + mesa.swa_backward(q, k, v, o, l, do, stream=s, **kw)
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        for a, b in zip(g, w):
            assert torch.equal(a, b)


def test_refusals(mesa):
    q, k, v, do = inputs(1, 4, 2, 20, 30, 64, "bf16")
    kw = dict(window=8, sinks=2)
    out, lse = mesa.swa_forward(q, k, v, return_lse=True, **kw)
    with pytest.raises(TypeError):
        mesa.swa_forward(q.half(), k, v, **kw)
    with pytest.raises(TypeError):
        mesa.swa_forward(q, k.float(), v, **kw)
    with pytest.raises(ValueError):
        mesa.swa_forward(q, k, v[:, :, :5], **kw)
    with pytest.raises(ValueError):
        mesa.swa_forward(q.transpose(1, 2), k, v, **kw)
    with pytest.raises(ValueError):
        mesa.swa_forward(q, k, v, window=2 ** 32 + 1)
    for bad, status in ((dict(window=0), 1), (dict(window=4, sinks=-1), 1), (dict(window=4, sinks=129), 2),
                        (dict(window=4, scale=float("nan")), 1), (dict(window=4, scale=0.0), 1)):
        with pytest.raises(mesa.MesaError) as e:
            mesa.swa_forward(q, k, v, **bad)
        assert e.value.status == status
    with pytest.raises(mesa.MesaError) as e:
        mesa.swa_forward(q[:, :3].contiguous(), k, v, **kw)           # 3 heads over 2
    assert e.value.status == 1
    with pytest.raises(mesa.MesaError) as e:
        mesa.swa_forward(k, q[:, :2].contiguous(), q[:, :2].contiguous(), **kw)      # more queries than keys
    assert e.value.status == 1
    with pytest.raises(mesa.MesaError) as e:
        mesa.swa_forward(q, k, v, out=q, **kw)
    assert e.value.status == 1
    with pytest.raises(mesa.MesaError) as e:
        mesa.swa_backward(q, k, v, out, lse, do, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"), **kw)
    assert e.value.status == 3


# ---- decode ----

def step_ref(q, kc, vc, pos, window, sinks, matrix):
    """Rows of (out, bound) from caches that already hold the new token."""
    B, Hq, d = q.shape
    Hkv = kc.shape[1]
    outs, bounds = [], []
    for b in range(B):
        p = int(pos[b])
        seen = [j for j in range(min(sinks, p + 1))] + list(range(max(sinks, p - window + 1), p + 1))
        at = [j if j < sinks else sinks + (j - sinks) % window for j in seen]
        r = ref.swa(q[b:b + 1, :, None], kc[b:b + 1, :, at], vc[b:b + 1, :, at], len(at), 0, matrix=matrix)["out"]
        outs.append(r[0][:, :, 0])
        bounds.append(r[1][:, :, 0])
    return torch.cat(outs), torch.cat(bounds)


STEPS = [  # (B, Hq, Hkv, window, sinks)
    (1, 1, 1, 1, 0), (2, 2, 1, 1, 3), (3, 4, 2, 7, 2), (2, 8, 8, 33, 1), (4, 8, 1, 64, 4), (2, 16, 1, 100, 0),
    (2, 24, 1, 130, 5), (5, 12, 4, 257, 4), (1, 16, 2, 1500, 128), (1, 9, 1, 4000, 4),
]


@pytest.mark.parametrize("d", [16, 32, 64, 128])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", STEPS, ids=lambda c: "-".join(map(str, c)))
def test_step(mesa, case, dtype, d):
    B, Hq, Hkv, window, sinks = case
    cap = window + sinks
    g = torch.Generator().manual_seed(cap + d)
    kc, vc = (torch.randn(B, Hkv, cap, d, generator=g).cuda().to(DT[dtype]) for _ in range(2))
    for trial in range(4):
        pos = [[0, cap - 1, cap, 3 * cap + 1, 2 ** 31 - 1], [1, sinks, cap - 2, 5 * cap, cap // 2],
               [-1, cap // 3, 2 * cap, 0, 1], [sinks + 1, cap, -1, -7, cap + 3]][trial]
        pos = torch.tensor([max(p, -9) for p in pos][:B], dtype=torch.int32)
        q = torch.randn(B, Hq, d, generator=g).cuda().to(DT[dtype])
        k, v = (torch.randn(B, Hkv, d, generator=g).cuda().to(DT[dtype]) for _ in range(2))
        wk, wv = kc.clone(), vc.clone()
        # slots the sequence has not reached yet are never read
        ik, iv = kc.clone(), vc.clone()
        for b in range(B):
            p = int(pos[b])
            if p >= 0:
                slot = p if p < sinks else sinks + (p - sinks) % window
                wk[b, :, slot], wv[b, :, slot] = k[b], v[b]
                ik[b, :, p + 1:], iv[b, :, p + 1:] = float("nan"), float("nan")
                ik[b, :, slot], iv[b, :, slot] = float("nan"), float("nan")
        out = mesa.swa_step(q, k, v, ik, iv, pos.cuda(), window=window, sinks=sinks)
        for b in range(B):
            p = int(pos[b])
            if p < 0:
                assert torch.count_nonzero(out[b]) == 0
                assert torch.equal(ik[b], kc[b]) and torch.equal(iv[b], vc[b])
                continue
            n = min(p + 1, cap)
            assert torch.equal(ik[b, :, :n], wk[b, :, :n]) and torch.equal(iv[b, :, :n], wv[b, :, :n])
            assert torch.isnan(ik[b, :, n:]).all()
            one = slice(b, b + 1)
            want, bound = step_ref(q[one], wk[one], wv[one], pos[one], window, sinks, ref.matrix_path(q.dtype, d))
            ref.check(out[one], want, bound, f"row {b}")
        kc, vc = wk, wv


@pytest.mark.parametrize("dtype,d", [("f32", 64), ("bf16", 64), ("bf16", 128), ("bf16", 32)])
def test_prompt_then_steps_follow_the_whole_sequence(mesa, dtype, d):
    """forward on a prompt, cache_fill, then steps: the rows of one forward over everything."""
    B, Hq, Hkv, P, N, window, sinks = 2, 6, 2, 75, 60, 40, 3
    T = P + N
    q, k, v, _ = inputs(B, Hq, Hkv, T, T, d, dtype, seed=12)
    want = ref.swa(q, k, v, window, sinks, matrix=ref.matrix_path(q.dtype, d))["out"]
    lens = torch.tensor([P, P - 30], dtype=torch.int32, device="cuda")       # a padded batch of prompts
    kc = torch.full((B, Hkv, sinks + window, d), float("nan"), device="cuda", dtype=q.dtype)
    vc = kc.clone()
    mesa.swa_cache_fill(k[:, :, :P].contiguous(), v[:, :, :P].contiguous(), kc, vc, window=window, sinks=sinks, lens=lens)
    for i in range(N):
        at = lens.long() + i
        rows = torch.arange(B, device="cuda")
        out = mesa.swa_step(q[rows, :, at].contiguous(), k[rows, :, at].contiguous(), v[rows, :, at].contiguous(), kc, vc,
                            at.int(), window=window, sinks=sinks)
        ref.check(out, want[0][rows, :, at], want[1][rows, :, at], f"token {i}")


@pytest.mark.parametrize("start,S", [(0, 1), (0, 9), (0, 10), (0, 47), (5, 3), (7, 30), (46, 4), (100, 1)])
def test_cache_fill_is_the_steps(mesa, start, S):
    window, sinks, d = 16, 5, 32
    q, k, v, _ = inputs(3, 2, 2, S, S, d, "bf16", seed=S)
    kc = torch.randn(3, 2, window + sinks, d, device="cuda").to(q.dtype)
    vc = kc + 1
    wk, wv = kc.clone(), vc.clone()
    lens = torch.tensor([S, max(S - 3, 0), -2], dtype=torch.int32, device="cuda")
    for i in range(S):
        pos = torch.where(lens > i, start + i, -1).int()
        mesa.swa_step(q[:, :, i].contiguous(), k[:, :, i].contiguous(), v[:, :, i].contiguous(), wk, wv, pos,
                      window=window, sinks=sinks)
    mesa.swa_cache_fill(k, v, kc, vc, window=window, sinks=sinks, start=start, lens=lens)
    assert torch.equal(kc, wk) and torch.equal(vc, wv)


def test_step_graph_follows_pos(mesa):
    """One captured step replayed for a run of tokens: pos advances on the device."""
    B, Hq, Hkv, d, window, sinks = 2, 4, 2, 128, 20, 2
    T = 50
    q, k, v, _ = inputs(B, Hq, Hkv, T, T, d, "bf16", seed=14)
    want = ref.swa(q, k, v, window, sinks, matrix=True)["out"]
    kc, vc = (torch.zeros(B, Hkv, window + sinks, d, device="cuda", dtype=q.dtype) for _ in range(2))
    qi, ki, vi = q[:, :, 0].clone(), k[:, :, 0].clone(), v[:, :, 0].clone()
    pos = torch.zeros(B, dtype=torch.int32, device="cuda")
    mesa.swa_step(qi, ki, vi, kc, vc, pos, window=window, sinks=sinks)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = mesa.swa_step(qi, ki, vi, kc, vc, pos, window=window, sinks=sinks)
        pos.add_(1)
    for t in range(T):
        for dst, src in ((qi, q), (ki, k), (vi, v)):
            dst.copy_(src[:, :, t])
        graph.replay()
        ref.check(out, want[0][:, :, t], want[1][:, :, t], f"token {t}")


def test_cache_past_32_bit_offsets(mesa):
    """The last head of caches of more than 2^31 elements."""
    B, Hkv, d, window, sinks = 2, 2, 128, (1 << 22) + 3, 4
    cap = window + sinks
    assert B * Hkv * cap * d > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(15)
    kc, vc = (torch.empty(B, Hkv, cap, d, device="cuda", dtype=torch.bfloat16).normal_(generator=g) for _ in range(2))
    q = torch.randn(B, Hkv, d, generator=g, device="cuda").bfloat16()
    k, v = (torch.randn(B, Hkv, d, generator=g, device="cuda").bfloat16() for _ in range(2))
    pos = torch.tensor([cap - 1, 2 * cap - sinks - 1], dtype=torch.int32, device="cuda")
    out = mesa.swa_step(q, k, v, kc, vc, pos, window=window, sinks=sinks)
    assert torch.equal(kc[0, :, cap - 1], k[0])
    one = slice(1, 2)
    want, bound = ref.swa(q[one, 1:, None], kc[one, 1:], vc[one, 1:], cap, 0, matrix=True)["out"]
    ref.check(out[one, 1:], want[:, :, 0], bound[:, :, 0], "out")


def test_step_refusals(mesa):
    q, k, v, _ = inputs(2, 4, 2, 1, 1, 64, "bf16")
    q, k, v = q[:, :, 0].contiguous(), k[:, :, 0].contiguous(), v[:, :, 0].contiguous()
    kc, vc = (torch.zeros(2, 2, 12, 64, device="cuda", dtype=q.dtype) for _ in range(2))
    pos = torch.zeros(2, dtype=torch.int32, device="cuda")
    mesa.swa_step(q, k, v, kc, vc, pos, window=10, sinks=2)
    with pytest.raises(ValueError):
        mesa.swa_step(q, k, v, kc, vc, pos, window=10, sinks=3)
    with pytest.raises(TypeError):
        mesa.swa_step(q, k, v, kc, vc, pos.long(), window=10, sinks=2)
    with pytest.raises(ValueError):
        mesa.swa_step(q, k, v, kc, vc, pos.cpu(), window=10, sinks=2)
    with pytest.raises(ValueError):
        mesa.swa_step(q, k, v, kc[:, :, ::2], vc, pos, window=10, sinks=2)
    with pytest.raises(mesa.MesaError) as e:
        mesa.swa_step(q, k, v, kc, kc, pos, window=10, sinks=2)
    assert e.value.status == 1


@pytest.mark.parametrize("T,S,window,sinks", [(400, 460, 1, 1), (400, 460, 2, 0), (400, 460, 3, 0), (400, 460, 2, 2),
                                              (400, 460, 7, 1), (400, 460, 9, 0), (3, 3, 50, 100), (6, 8, 8, 128)])
@pytest.mark.parametrize("d", [16, 32, 64, 128])
def test_few_keys_keep_their_gradients(mesa, d, T, S, window, sinks):
    """With two or three keys dP - delta cancels: the gradients' error as a whole
    stays within the roundings of P, dS and the result to bf16, 3 x 2^-9 in the
    root mean square (a half step is 2^-9 on average over a binade at most)."""
    q, k, v, do = inputs(1, 4, 2, T, S, d, "bf16", seed=31)
    out, lse = mesa.swa_forward(q, k, v, window=window, sinks=sinks, return_lse=True)
    want = ref.swa(q, k, v, window, sinks, matrix=True, dout=do)
    for n, g in zip(("dq", "dk", "dv"), mesa.swa_backward(q, k, v, out, lse, do, window=window, sinks=sinks)):
        err = (g.double() - want[n][0]).norm() / want[n][0].norm()
        assert float(err) <= 3 * 2.0 ** -9, (n, float(err))


@pytest.mark.parametrize("dtype,d", [("f32", 32), ("bf16", 16), ("bf16", 64), ("bf16", 128)])
def test_one_visible_key_has_no_score_gradient(mesa, dtype, d):
    for T, S, window, sinks in ((130, 200, 1, 0), (1, 1, 9, 4)):
        q, k, v, do = inputs(2, 4, 2, T, S, d, dtype, seed=32)
        out, lse = mesa.swa_forward(q, k, v, window=window, sinks=sinks, return_lse=True)
        dq, dk, dv = mesa.swa_backward(q, k, v, out, lse, do, window=window, sinks=sinks)
        assert torch.count_nonzero(dq) == 0 and torch.count_nonzero(dk) == 0
        want = ref.swa(q, k, v, window, sinks, matrix=ref.matrix_path(q.dtype, d), dout=do)
        ref.check(dv, *want["dv"], "dv")


# (B, Hq, Hkv, T, window, sinks): every SM's CTA walks several pairs of query tiles. Heads that
# share no keys in pairs with an odd number of 128-row tiles: the pair's second tile is empty.
WALKS = [
    (32, 16, 16, 100, 40, 3),        # one tile a head, 512 pairs, all second tiles empty
    (30, 10, 10, 300, 70, 2),        # three tiles, two pairs a head: every second one half empty
    (6, 16, 16, 800, 150, 4),        # seven tiles
    (34, 9, 3, 129, 64, 0),          # groups of three, both tiles live
    (16, 40, 20, 200, 90, 1),        # pairs of heads
    (150, 3, 1, 1, 5, 0),            # one query a head
]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("case", WALKS, ids=lambda c: "-".join(map(str, c)))
def test_forward_walks_several_pairs(mesa, case, d):
    B, Hq, Hkv, T, window, sinks = case
    S = T + 30 if T < 200 else T
    pairs = B * Hq // 2 * -(-T // 128) if (Hq // Hkv) % 2 == 0 else B * Hq * -(-T // 256)
    assert pairs > 2 * 148
    q, k, v, _ = inputs(B, Hq, Hkv, T, S, d, "bf16", seed=41)
    assert mesa.get_error() == 0
    out, lse = mesa.swa_forward(q, k, v, window=window, sinks=sinks, return_lse=True)
    assert mesa.get_error() == 0                                      # no wait gave up
    for b in range(0, B, 2):
        at = slice(b, b + 2)
        want = ref.swa(q[at], k[at], v[at], window, sinks, matrix=True)
        ref.check(out[at], *want["out"], f"out of sequences {b}, {b + 1}")
        ref.check(lse[at], *want["lse"], f"lse of sequences {b}, {b + 1}")
    assert torch.equal(out, mesa.swa_forward(q, k, v, window=window, sinks=sinks))


def test_cache_of_the_most_slots(mesa):
    """sinks + window = 2^31 - 1: slot numbers pass 31 bits within a step of the last CTA."""
    d, sinks = 16, 4
    cap = 2 ** 31 - 1
    window = cap - sinks
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 2 * cap * d * 2 + (2 << 30):
        pytest.skip("needs 140 GB of device memory")
    kc, vc = (torch.zeros(1, 1, cap, d, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    # scores of 0 but for a few slots of score 32, those in the last steps among them
    at = torch.tensor([0, 7, 2 ** 30 + 1, cap - 2049, cap - 2047, cap - 129, cap - 128, cap - 2, cap - 1], device="cuda")
    g = torch.Generator().manual_seed(43)
    kc[0, 0, at] = 8.0
    vc[0, 0, at] = torch.randn(len(at), d, generator=g).cuda().bfloat16()
    q, k = torch.ones(1, 1, d, device="cuda").bfloat16(), torch.zeros(1, 1, d, device="cuda").bfloat16()
    v = k.clone()
    pos = torch.tensor([cap], dtype=torch.int32, device="cuda")            # slot 4; every slot is in use
    out = mesa.swa_step(q, k, v, kc, vc, pos, window=window, sinks=sinks)
    want = vc[0, 0, at].double().sum(0) / (len(at) + (cap - len(at)) * 2.718281828459045 ** -32)
    # exponents of 46 in log2 units err by 46 U; the 2^31 weights of e^-32, lost or not in a sum of nine, are 2.7e-5 < 2^-15
    bound = 2.0 ** -14 * vc[0, 0, at].double().abs().sum(0)
    ref.check(out[0, 0], want, bound, "out")
    assert mesa.get_error() == 0
    del kc, vc
    torch.cuda.empty_cache()


# ---- decode over caches of 8 MB and more: equal shares of all runs of 64 slots, parts joined by a second launch ----

SHARES = [  # (B, Hq, Hkv, window, sinks); all of 8 MB and more at d = 64
    (48, 8, 4, 600, 4),          # several parts a head, joined by small blocks
    (40, 9, 1, 1000, 0),         # a group above eight
    (4, 24, 1, 9000, 5),         # two blocks of heads in a group, many parts a head, joined by large blocks
    (1, 2, 1, 40000, 4),         # one head over all SMs
    (300, 4, 2, 64, 0),          # one run a head, two heads a share: no parts at all
    (30, 10, 10, 130, 128),      # many heads of few runs
    (90, 16, 1, 272, 128),       # sinks over two runs
]


def share_positions(trial, B, cap, g):
    """Positions of a batch: full and young rows mixed, edges of a run, idle rows, one row alone, none."""
    edges = [0, cap - 1, 63, -1, 64, 4 * cap + 7, 127, 1, -5, 2 ** 31 - 1, cap, cap // 2]
    if trial == 0:
        return [edges[b % len(edges)] for b in range(B)]
    if trial == 1:                                       # a short one between long ones, idle first and last
        pos = [2 * cap + 3 if b % 3 else b % 5 for b in range(B)]
        if B > 2:
            pos[0] = pos[-1] = -1
        return pos
    if trial == 2:
        return torch.randint(0, 2 * cap, (B,), generator=g).tolist()
    if trial == 3:                                       # the last row alone
        return [-1] * (B - 1) + [cap + 1]
    return [-1 - b for b in range(B)]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("case", SHARES, ids=lambda c: "-".join(map(str, c)))
def test_step_in_equal_shares(mesa, case, d):
    B, Hq, Hkv, window, sinks = case
    cap = window + sinks
    assert B * Hkv * cap * d * 4 >= 8 << 20
    kw = dict(window=window, sinks=sinks)
    g = torch.Generator().manual_seed(cap + d)
    kc, vc = (torch.randn(B, Hkv, cap, d, generator=g).cuda().bfloat16() for _ in range(2))
    assert mesa._load().mesa_swa_step_workspace_size(B, Hq, Hkv, d, window, sinks, 1) > 0
    for trial in range(5):
        pos = share_positions(trial, B, cap, g)
        q = torch.randn(B, Hq, d, generator=g).cuda().bfloat16()
        k, v = (torch.randn(B, Hkv, d, generator=g).cuda().bfloat16() for _ in range(2))
        wk, wv, ik, iv = kc.clone(), vc.clone(), kc.clone(), vc.clone()
        for b, p in enumerate(pos):                      # NaN where nothing may be read
            if p >= 0:
                slot = p if p < sinks else sinks + (p - sinks) % window
                wk[b, :, slot], wv[b, :, slot] = k[b], v[b]
                for t in (ik, iv):
                    t[b, :, p + 1:] = float("nan")
                    t[b, :, slot] = float("nan")
            else:
                ik[b], iv[b] = float("nan"), float("nan")
        gk, gv = ik.clone(), iv.clone()
        pd = torch.tensor(pos, dtype=torch.int32, device="cuda")
        out = torch.full_like(q, float("nan"))
        mesa.swa_step(q, k, v, gk, gv, pd, out=out, **kw)
        for b, p in enumerate(pos):
            one = slice(b, b + 1)
            if p < 0:
                assert torch.count_nonzero(out[b]) == 0 and torch.isnan(gk[b]).all() and torch.isnan(gv[b]).all()
                continue
            n = min(p + 1, cap)
            assert torch.equal(gk[b, :, :n], wk[b, :, :n]) and torch.equal(gv[b, :, :n], wv[b, :, :n])
            assert torch.isnan(gk[b, :, n:]).all() and torch.isnan(gv[b, :, n:]).all()
            want, bound = step_ref(q[one], wk[one], wv[one], pd[one], window, sinks, True)
            ref.check(out[one], want, bound, f"trial {trial} row {b}")
        assert torch.equal(out, mesa.swa_step(q, k, v, ik, iv, pd, **kw))          # no order in it
        kc, vc = wk, wv


@pytest.mark.parametrize("B,Hq,Hkv,d,window", [(24, 8, 4, 128, 300), (2, 12, 1, 64, 20000)])
def test_captured_shares_follow_pos(mesa, B, Hq, Hkv, d, window):
    """Both launches of a step in a graph, replayed while the positions advance."""
    sinks, T = 3, 60
    cap = window + sinks
    assert B * Hkv * cap * d * 4 >= 8 << 20
    g = torch.Generator().manual_seed(51)
    q = torch.randn(T, B, Hq, d, generator=g).cuda().bfloat16()
    k, v = (torch.randn(T, B, Hkv, d, generator=g).cuda().bfloat16() for _ in range(2))
    first = torch.randint(0, 2 * cap, (B,), generator=g).int().cuda()
    first[0] = -3                                        # idle for three steps, then a first token
    caches = [torch.randn(B, Hkv, cap, d, generator=g).cuda().bfloat16() for _ in range(2)]
    want, eager, pos = [], [c.clone() for c in caches], first.clone()
    for t in range(T):
        want.append(mesa.swa_step(q[t], k[t], v[t], *eager, pos, window=window, sinks=sinks))
        pos += 1
    qi, ki, vi, pos = q[0].clone(), k[0].clone(), v[0].clone(), first.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = mesa.swa_step(qi, ki, vi, *caches, pos, window=window, sinks=sinks)
        pos.add_(1)
    for t in range(T):
        for dst, src in ((qi, q), (ki, k), (vi, v)):
            dst.copy_(src[t])
        graph.replay()
        assert torch.equal(out, want[t]), t
    for a, b in zip(caches, eager):
        assert torch.equal(a, b)


def test_shares_on_two_streams(mesa):
    """Steps that overlap, each with its own caches and workspace."""
    B, Hq, Hkv, d, window, sinks = 20, 8, 2, 128, 1000, 4
    g = torch.Generator().manual_seed(52)
    sets = []
    for _ in range(2):
        q = torch.randn(B, Hq, d, generator=g).cuda().bfloat16()
        k, v = (torch.randn(B, Hkv, d, generator=g).cuda().bfloat16() for _ in range(2))
        kc, vc = (torch.randn(B, Hkv, window + sinks, d, generator=g).cuda().bfloat16() for _ in range(2))
        sets.append((q, k, v, kc, vc, torch.randint(0, 3000, (B,), generator=g).int().cuda()))
    want = [mesa.swa_step(*s, window=window, sinks=sinks) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[], []]
    for _ in range(10):
        for i, (st, s) in enumerate(zip(streams, sets)):
            got[i].append(mesa.swa_step(*s, window=window, sinks=sinks, stream=st))
    torch.cuda.synchronize()
    for w, outs in zip(want, got):
        assert all(torch.equal(w, o) for o in outs)


@pytest.mark.parametrize("d", [64])
def test_one_query_over_two_hundred_million_keys(mesa, d):
    """A pair of tiles whose second is empty, over more key tiles than one bounded wait lasts."""
    S = 200_000_000
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 2 * S * d * 2 + (2 << 30):
        pytest.skip("needs 54 GB of device memory")
    k, v = (torch.zeros(1, 1, S, d, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    at = torch.tensor([0, 5, 127, 128, 31_234_567, 50_000_000, S - 129, S - 1], device="cuda")
    g = torch.Generator().manual_seed(61)
    k[0, 0, at] = 4.0                                    # scores of 32, all others 0
    v[0, 0, at] = torch.randn(len(at), d, generator=g).cuda().bfloat16()
    q = torch.ones(1, 1, 1, d, device="cuda", dtype=torch.bfloat16)
    out, lse = mesa.swa_forward(q, k, v, window=S, return_lse=True)
    assert mesa.get_error() == 0
    vd = v[0, 0, at].double()
    rest = (S - len(at)) * 2.718281828459045 ** -32      # weights of e^-32, 2.6e-6 together, lost or not
    want = vd.sum(0) / (len(at) + rest)
    # P rounds to bf16 (1 = e^0 exactly, on a reference that a row with larger weights moves to its maximum); fp32 sums
    ref.check(out[0, 0, 0], want, 2.0 ** -17 * vd.abs().sum(0), "out")
    assert abs(float(lse[0, 0, 0]) - 32 - torch.log(torch.tensor(len(at) + rest, dtype=torch.float64)).item()) < 40 * 2.0 ** -22
    del k, v
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_sequences_past_32_bit_offsets(mesa, dtype):
    """The last rows of the last head of tensors of more than 2^31 elements, and a key head summed over all query heads."""
    Hq, T, d, window, rows = 66, 256 * 1024 + 5, 128, 16, 200
    assert Hq * T * d > 2 ** 31
    torch.cuda.empty_cache()
    g = torch.Generator(device="cuda").manual_seed(62)
    q, do = (torch.empty(1, Hq, T, d, device="cuda", dtype=DT[dtype]).normal_(generator=g) for _ in range(2))
    k, v = (torch.empty(1, Hq, T, d, device="cuda", dtype=DT[dtype]).normal_(generator=g) for _ in range(2))
    out, lse = mesa.swa_forward(q, k, v, window=window, return_lse=True)
    dq, dk, dv = mesa.swa_backward(q, k, v, out, lse, do, window=window)
    assert mesa.get_error() == 0
    head, last = slice(Hq - 1, Hq), slice(T - rows, T)
    seen = slice(T - rows - window + 1, T)               # the keys that these rows see
    want = ref.swa(q[:, head, last], k[:, head, seen], v[:, head, seen], window, 0, matrix=dtype == "bf16",
                   dout=do[:, head, last])
    ref.check(out[:, head, last], *want["out"], "out")
    ref.check(lse[:, head, last], *want["lse"], "lse")
    ref.check(dq[:, head, last], *want["dq"], "dq")
    for n, t in (("dk", dk), ("dv", dv)):                # keys whose queries are all among the rows
        w, b = want[n]
        ref.check(t[:, head, last], w[:, :, window - 1:], b[:, :, window - 1:], n)
    del q, k, v, do, out, dq, dk, dv
    torch.cuda.empty_cache()


@pytest.mark.parametrize("call", ["forward", "backward", "step", "lru_forward", "lru_backward"])
def test_first_call_of_a_host_thread(mesa, call):
    """A thread that has made no CUDA call before, once the library has been used by another."""
    import threading
    lib = mesa._load()
    q, k, v, do = inputs(1, 2, 1, 200, 200, 64, "bf16", seed=71)
    out, lse = mesa.swa_forward(q, k, v, window=50, return_lse=True)
    grads = mesa.swa_backward(q, k, v, out, lse, do, window=50)
    x, ga, gx, dy = (t.view(1, 400, 64) for t in (q, do, out, out))
    lam = torch.full((64,), -4.0, device="cuda")
    y, saved = mesa.lru_forward(x, ga, gx, lam, return_saved=True)
    lgrads = mesa.lru_backward(x, ga, gx, lam, dy, saved=saved)
    kc, vc = (torch.zeros(1, 1, 200, 64, device="cuda", dtype=q.dtype) for _ in range(2))
    pos = torch.zeros(1, dtype=torch.int32, device="cuda")
    o1 = mesa.swa_step(q[:, :, 0].contiguous(), k[:, :, 0].contiguous(), v[:, :, 0].contiguous(), kc, vc, pos, window=200)
    ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    p = [t.data_ptr() for t in (q, k, v, out, lse, do)]
    new = {"forward": (out, lse), "backward": grads, "step": (o1,), "lru_forward": (y,), "lru_backward": lgrads}[call]
    got = [torch.full_like(t, float("nan")) for t in new]
    g = [t.data_ptr() for t in got]
    first = [t[:, :, 0].contiguous() for t in (q, k, v)]
    lp = [t.data_ptr() for t in (x, ga, gx, lam)] + [1, 400, 64, 1, None]
    torch.cuda.synchronize()
    scale = 64 ** -0.5
    run = {
        "forward": lambda: lib.mesa_swa_forward(*p[:3], 1, 2, 1, 200, 200, 64, 50, 0, scale, 1, *g, None),
        "backward": lambda: lib.mesa_swa_backward(*p, 1, 2, 1, 200, 200, 64, 50, 0, scale, 1, *g, ws.data_ptr(), ws.numel(), None),
        "step": lambda: lib.mesa_swa_step(*[t.data_ptr() for t in first], kc.data_ptr(), vc.data_ptr(), pos.data_ptr(), 1, 2, 1,
                                          64, 200, 0, scale, 1, *g, ws.data_ptr(), ws.numel(), None),
        "lru_forward": lambda: lib.mesa_lru_forward(*lp, *g, None, None, None),
        "lru_backward": lambda: lib.mesa_lru_backward(*lp, saved.data_ptr(), dy.data_ptr(), None, *g, ws.data_ptr(), ws.numel(),
                                                      None),
    }[call]
    status = []
    t = threading.Thread(target=lambda: status.append(run()))
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert status == [0]
    for a, b in zip(got, new):
        assert torch.equal(a, b)


@pytest.mark.parametrize("call", ["lru_forward", "lru_backward", "lru_step", "forward", "backward", "step", "cache_fill"])
def test_inputs_dropped_while_a_call_is_to_run(mesa, call):
    """Tensors of one stream, a call on another that is still busy, and their memory given up at once."""
    g = torch.Generator().manual_seed(81)
    bf = torch.bfloat16

    def make(*shape, dtype=bf):
        return torch.randn(shape, generator=g).cuda().to(dtype)
    x = [make(2, 300, 64) for _ in range(4)]
    lam, h0 = make(64, dtype=torch.float32) - 4, make(2, 64, dtype=torch.float32)
    y, saved = mesa.lru_forward(*x[:3], lam, h0=h0, return_saved=True)
    q, k, v, do = make(2, 4, 300, 64), make(2, 2, 300, 64), make(2, 2, 300, 64), make(2, 4, 300, 64)
    out, lse = mesa.swa_forward(q, k, v, window=60, return_lse=True)
    kc, vc, pos = make(2, 2, 60, 64), make(2, 2, 60, 64), torch.tensor([7, 99], dtype=torch.int32, device="cuda")
    first = [t[:, :, 0].contiguous() for t in (q, k, v)]
    args, run = {
        "lru_forward": (x[:3] + [lam, h0], lambda a, s: mesa.lru_forward(*a[:4], h0=a[4], return_state=True, stream=s)),
        "lru_backward": (x[:3] + [lam, x[3], saved, h0], lambda a, s: mesa.lru_backward(*a[:5], saved=a[5], dh_T=a[6], stream=s)),
        "lru_step": ([t[:, 0].contiguous() for t in x[:3]] + [lam, h0], lambda a, s: (mesa.lru_step(*a, stream=s),)),
        "forward": ([q, k, v], lambda a, s: (mesa.swa_forward(*a, window=60, stream=s),)),
        "backward": ([q, k, v, out, lse, do], lambda a, s: mesa.swa_backward(*a, window=60, stream=s)),
        "step": (first + [kc, vc, pos], lambda a, s: (mesa.swa_step(*a, window=60, stream=s),)),
        "cache_fill": ([k, v], lambda a, s: mesa.swa_cache_fill(*a, kd, vd, window=60, stream=s)),
    }[call]
    kd, vd = torch.zeros_like(kc), torch.zeros_like(vc)
    want = run([t.clone() for t in args], None) or (kd.clone(), vd.clone())
    kd.zero_(), vd.zero_()
    side = torch.cuda.Stream()
    copies = [t.clone() for t in args]
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)                    # about 50 ms
    got = run(copies, side) or (kd, vd)
    shapes = [(t.shape, t.dtype) for t in copies]
    del copies
    junk = [torch.full(s, 77 if d == torch.int32 else float("nan"), dtype=d, device="cuda") for s, d in shapes for _ in range(2)]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    del junk


def test_named_stream_while_capturing(mesa):
    """The capturing stream given by name, an input dropped during the capture."""
    q, k, v, _ = inputs(1, 4, 2, 200, 260, 128, "bf16", seed=91)
    want = mesa.swa_forward(q, k, v, window=100, sinks=4)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        doubled = q * 2
        half = doubled / 2
        del doubled
        out = mesa.swa_forward(half, k, v, window=100, sinks=4, stream=torch.cuda.current_stream())
        del half
        after = out + 0
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(after, want)
