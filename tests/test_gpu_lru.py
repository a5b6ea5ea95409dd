"""The gated linear recurrence on the GPU against its definition in 64 bits."""
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


def inputs(B, T, D, dtype, seed=0, shift=0):
    """Gates, inputs and decays as a trained layer has them; `shift` elements
    move the first tensors off the allocation's alignment."""
    g = torch.Generator().manual_seed(seed)

    def one(*shape):
        n = 1
        for s in shape:
            n *= s
        t = torch.empty(n + shift, dtype=DT[dtype], device="cuda")[shift:].view(shape)
        return t.copy_(torch.randn(shape, generator=g))
    a = 0.9 + 0.099 * torch.rand(D, generator=g, dtype=torch.float64)
    lam = torch.log(torch.expm1(-torch.log(a) / 8)).float().cuda()
    x, ga, gx, dy = (one(B, T, D) for _ in range(4))
    h0, dh = (torch.randn(B, D, generator=g).cuda() for _ in range(2))
    return x, ga, gx, lam, dy, h0, dh


SHAPES = [(1, 1, 1), (2, 5, 3), (1, 15, 64), (2, 16, 66), (1, 17, 33), (1, 63, 32), (1, 64, 64), (2, 65, 66),
          (1, 127, 130), (1, 128, 64), (1, 129, 128), (3, 300, 70), (1, 2049, 34), (2, 1025, 200), (16, 70, 1024)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,D", SHAPES)
def test_forward(mesa, B, T, D, dtype):
    x, ga, gx, lam, _, h0, _ = inputs(B, T, D, dtype, seed=T)
    for start in (None, h0):
        y, hT, saved = mesa.lru_forward(x, ga, gx, lam, h0=start, return_state=True, return_saved=True)
        want, wT, ey, eT = ref.lru(x, ga, gx, lam, start)
        ref.check(y, want, ey, "y")
        ref.check(hT, wT, eT, "h_T")
        first = torch.zeros_like(h0) if start is None else start
        at = torch.cat([first.double()[:, None], want[:, 63::64]], 1)[:, :saved.shape[1]]
        eat = torch.cat([torch.zeros_like(first).double()[:, None], ey[:, 63::64]], 1)[:, :saved.shape[1]]
        ref.check(saved, at, eat, "saved")
    assert torch.equal(y, mesa.lru_forward(x, ga, gx, lam, h0=h0))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,D", SHAPES)
def test_backward(mesa, B, T, D, dtype):
    x, ga, gx, lam, dy, h0, dh = inputs(B, T, D, dtype, seed=T + 1)
    names = ("dx", "dgate_a", "dgate_x", "dlam", "dh0")
    for start, end in ((None, None), (h0, dh)):
        _, saved = mesa.lru_forward(x, ga, gx, lam, h0=start, return_saved=True)
        got = mesa.lru_backward(x, ga, gx, lam, dy, saved=saved, dh_T=end)
        want, bound = ref.lru_grads(x, ga, gx, lam, start, dy, end)
        for n, o, w, b in zip(names, got, want, bound):
            ref.check(o, w, b, n)
        again = mesa.lru_backward(x, ga, gx, lam, dy, h0=start, dh_T=end)        # states recomputed
        for n, o, o2 in zip(names, got, again):
            assert torch.equal(o, o2), n


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_fast_decays(mesa, dtype):
    """Channels from slow to total decay side by side (not one CTA of slow ones alone)."""
    x, ga, gx, lam, dy, h0, dh = inputs(2, 210, 150, dtype, seed=21)
    lam += torch.linspace(0.0, 12.0, 150, device="cuda")
    y, hT, saved = mesa.lru_forward(x, ga, gx, lam, h0=h0, return_state=True, return_saved=True)
    want, wT, ey, eT = ref.lru(x, ga, gx, lam, h0)
    ref.check(y, want, ey, "y")
    ref.check(hT, wT, eT, "h_T")
    got = mesa.lru_backward(x, ga, gx, lam, dy, saved=saved, dh_T=dh)
    want, bound = ref.lru_grads(x, ga, gx, lam, h0, dy, dh)
    for n, o, w, b in zip(("dx", "dgate_a", "dgate_x", "dlam", "dh0"), got, want, bound):
        ref.check(o, w, b, n)


@pytest.mark.parametrize("D,shift", [(66, 1), (65, 0), (64, 1), (64, 2)])
def test_alignment(mesa, D, shift):
    """Odd widths and bases that allow only single-element accesses."""
    x, ga, gx, lam, dy, h0, dh = inputs(2, 77, D, "bf16", seed=9, shift=shift)
    y, saved = mesa.lru_forward(x, ga, gx, lam, h0=h0, return_saved=True)
    want, _, ey, _ = ref.lru(x, ga, gx, lam, h0)
    ref.check(y, want, ey, "y")
    got = mesa.lru_backward(x, ga, gx, lam, dy, saved=saved, dh_T=dh)
    want, bound = ref.lru_grads(x, ga, gx, lam, h0, dy, dh)
    for o, w, b in zip(got, want, bound):
        ref.check(o, w, b, "gradient")
    hn = torch.empty_like(h0)
    y1 = mesa.lru_step(x[:, 0].contiguous(), ga[:, 0].contiguous(), gx[:, 0].contiguous(), lam, h0, h_out=hn)
    want, _, ey, _ = ref.lru(x[:, :1], ga[:, :1], gx[:, :1], lam, h0)
    ref.check(y1, want[:, 0], ey[:, 0], "step")


@pytest.mark.parametrize("lams", [(-120.0, -95.0, -60.0, -25.0, -15.0, -3.0, 0.0, 5.0, 60.0),
                                  (-120.0, -95.0, -60.0, -25.0, -15.0, -8.0, -6.0, -5.0, -4.0)],
                         ids=["any decay", "slow decays"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_extreme_gates(mesa, dtype, lams):
    """Closed, open and saturated gates; decays from none to total, or slow ones alone."""
    B, T = 1, 200
    vals = torch.tensor([-float("inf"), -90.0, -60.0, -30.0, -10.0, 0.0, 10.0, 40.0, 100.0, float("inf")])
    lams = torch.tensor(lams)
    D = len(vals) * len(lams)
    x, ga, gx, lam, dy, h0, dh = inputs(B, T, D, dtype, seed=3)
    ga[:] = vals.repeat(len(lams)).to(ga)
    gx[:] = vals.flip(0).repeat(len(lams)).to(gx)
    gx[:, ::2] = torch.randn(100, D).to(gx)
    lam[:] = lams.repeat_interleave(len(vals)).to(lam)
    y, hT, saved = mesa.lru_forward(x, ga, gx, lam, h0=h0, return_state=True, return_saved=True)
    assert torch.isfinite(y).all() and torch.isfinite(hT).all()
    closed = torch.isinf(ga[0, 0].float()) & (ga[0, 0] < 0)
    assert torch.equal(hT[:, closed], h0[:, closed])                  # a closed gate holds the state exactly
    gf = ga.float().clamp(-104, 104)                                  # beyond: the sigmoid is 0 or 1 in fp32
    want, wT, ey, eT = ref.lru(x, gf, gx.float().clamp(-104, 104), lam, h0)
    # a gate below the smallest fp32 sigmoid counts as closed: sqrt(2 * 8 softplus * e^-87) per token
    eps = T * 64 * 1e-18
    ref.check(y, want, ey + eps, "y")
    for g in mesa.lru_backward(x, ga, gx, lam, dy, saved=saved, dh_T=dh):
        assert torch.isfinite(g).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gradients_against_differences(mesa, dtype):
    """Directional differences of the 64-bit layer along every input."""
    B, T, D = 2, 70, 5
    x, ga, gx, lam, dy, h0, dh = inputs(B, T, D, dtype, seed=4)
    got = mesa.lru_backward(x, ga, gx, lam, dy, h0=h0, dh_T=dh)
    args = [t.double() for t in (x, ga, gx, lam, h0)]

    def loss(a):
        y, hT, _, _ = ref.lru(*a[:4], h0=a[4])
        return (y * dy.double()).sum() + (hT * dh.double()).sum()
    want, bound = ref.lru_grads(x, ga, gx, lam, h0, dy, dh)
    order = (0, 1, 2, 4, 3)                                           # lam and h0 in the call's order of gradients
    gen = torch.Generator().manual_seed(1)
    for n, (i, o) in enumerate(zip((0, 1, 2, 3, 4), got)):
        d = torch.randn(args[i].shape, generator=gen, dtype=torch.float64).cuda()
        step = 1e-5
        up, dn = list(args), list(args)
        up[i], dn[i] = args[i] + step * d, args[i] - step * d
        diff = (loss(up) - loss(dn)) / (2 * step)
        slack = ((bound[n] + ref.half_step(o.dtype) * (want[n].abs() + bound[n])) * d.abs()).sum()
        # a central difference errs by step^2 / 6 of the third derivative: far below 1e-5 of the gradient's size
        assert abs(float(diff - (o.double() * d).sum())) <= float(slack) + 1e-5 * float((want[n].abs() * d.abs()).sum())
    del order


def test_empty_sequence(mesa):
    x, ga, gx, lam, dy, h0, dh = inputs(2, 0, 6, "bf16")
    y, hT, saved = mesa.lru_forward(x, ga, gx, lam, h0=h0, return_state=True, return_saved=True)
    assert y.shape == (2, 0, 6) and saved.shape == (2, 0, 6) and torch.equal(hT, h0)
    _, hT = mesa.lru_forward(x, ga, gx, lam, return_state=True)
    assert torch.count_nonzero(hT) == 0
    dx, _, _, dlam, dh0 = mesa.lru_backward(x, ga, gx, lam, dy, h0=h0, dh_T=dh)
    assert dx.shape == (2, 0, 6) and torch.count_nonzero(dlam) == 0 and torch.equal(dh0, dh)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_steps_and_pieces_agree_with_the_whole(mesa, dtype):
    B, T, D = 3, 150, 40
    x, ga, gx, lam, _, h0, _ = inputs(B, T, D, dtype, seed=5)
    want, wT, ey, eT = ref.lru(x, ga, gx, lam, h0)
    h = h0.clone()
    for t in range(T):
        y = mesa.lru_step(x[:, t].contiguous(), ga[:, t].contiguous(), gx[:, t].contiguous(), lam, h)
        ref.check(y, want[:, t], ey[:, t], f"step {t}")
    ref.check(h, wT, eT, "state")
    cut = 83
    _, mid = mesa.lru_forward(*(t[:, :cut].contiguous() for t in (x, ga, gx)), lam, h0=h0, return_state=True)
    y2, end = mesa.lru_forward(*(t[:, cut:].contiguous() for t in (x, ga, gx)), lam, h0=mid, return_state=True)
    ref.check(y2, want[:, cut:], ey[:, cut:], "second piece")
    ref.check(end, wT, eT, "end state")


def test_stream_and_graph(mesa):
    """On a stream of its own, captured and replayed on new inputs."""
    B, T, D = 2, 200, 64
    a = inputs(B, T, D, "bf16", seed=6)
    b = inputs(B, T, D, "bf16", seed=7)
    bufs = [t.clone() for t in a]
    x, ga, gx, lam, dy, h0, dh = bufs
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = mesa.lru_forward(x, ga, gx, lam, h0=h0, stream=s)
    s.synchronize()
    assert torch.equal(y, mesa.lru_forward(x, ga, gx, lam, h0=h0))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        yc, sc = mesa.lru_forward(x, ga, gx, lam, h0=h0, return_saved=True)
        gc = mesa.lru_backward(x, ga, gx, lam, dy, saved=sc, dh_T=dh)
    for t, n in zip(bufs, b):
        t.copy_(n)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    want = mesa.lru_forward(b[0], b[1], b[2], b[3], h0=b[5])
    assert torch.equal(yc, want)
    for o, w in zip(gc, mesa.lru_backward(b[0], b[1], b[2], b[3], b[4], h0=b[5], dh_T=b[6])):
        assert torch.equal(o, w)


def test_past_32_bit_offsets(mesa):
    """The last sequence of a batch of more than 2^31 elements."""
    B, T, D = 2, 1100, 1 << 20
    assert B * T * D > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(8)
    x, ga, gx = (torch.empty(B, T, D, dtype=torch.bfloat16, device="cuda").normal_(generator=g) for _ in range(3))
    lam = torch.randn(D, generator=g, device="cuda") - 4
    y = mesa.lru_forward(x, ga, gx, lam)
    cols = slice(D - 64, D)
    xs, gas, gxs = (t[1:, :, cols].contiguous() for t in (x, ga, gx))
    want, _, ey, _ = ref.lru(xs, gas, gxs, lam[cols])
    ref.check(y[1:, :, cols], want, ey, "y")


def test_refusals(mesa):
    x, ga, gx, lam, dy, h0, dh = inputs(2, 10, 8, "bf16")
    with pytest.raises(TypeError):
        mesa.lru_forward(x.half(), ga, gx, lam)
    with pytest.raises(TypeError):
        mesa.lru_forward(x, ga.float(), gx, lam)
    with pytest.raises(ValueError):
        mesa.lru_forward(x, ga[:, :5], gx, lam)
    with pytest.raises(ValueError):
        mesa.lru_forward(x.transpose(0, 1), ga, gx, lam)
    with pytest.raises(ValueError):
        mesa.lru_forward(x, ga.cpu(), gx, lam)
    with pytest.raises(TypeError):
        mesa.lru_forward(x, ga, gx, lam.bfloat16())
    with pytest.raises(ValueError):
        mesa.lru_backward(x, ga, gx, lam, dy, saved=torch.empty(2, 3, 8, device="cuda"))
    with pytest.raises(mesa.MesaError) as e:
        mesa.lru_backward(x, ga, gx, lam, dy, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 3
    with pytest.raises(mesa.MesaError) as e:
        mesa.lru_forward(x, ga, gx, lam, y=x)
    assert e.value.status == 1


# (B, T, D, shift): rows that only single-element loads can take, and numbers of 64-token tiles
# that leave a cluster's last round with tiles that do not exist
PLAIN = [(1, 130, 17, 0), (1, 300, 33, 0), (1, 1900, 33, 0), (1, 1900, 1003, 0), (1, 6000, 31, 0), (2, 130, 34, 1),
         (3, 321, 64, 1), (1, 2000, 130, 1)]


@pytest.mark.parametrize("B,T,D,shift", PLAIN)
def test_rows_of_single_elements(mesa, B, T, D, shift):
    x, ga, gx, lam, dy, h0, dh = inputs(B, T, D, "bf16", seed=T + D, shift=shift)
    y, hT, saved = mesa.lru_forward(x, ga, gx, lam, h0=h0, return_state=True, return_saved=True)
    want, wT, ey, eT = ref.lru(x, ga, gx, lam, h0)
    ref.check(y, want, ey, "y")
    ref.check(hT, wT, eT, "h_T")
    got = mesa.lru_backward(x, ga, gx, lam, dy, saved=saved, dh_T=dh)
    want, bound = ref.lru_grads(x, ga, gx, lam, h0, dy, dh)
    for n, o, w, b in zip(("dx", "dgate_a", "dgate_x", "dlam", "dh0"), got, want, bound):
        ref.check(o, w, b, n)
    assert mesa.get_error() == 0


@pytest.mark.parametrize("B,T,D", [(1, 1, 32), (1, 130, 64), (1, 256, 32), (2, 300, 130), (1, 2049, 64), (1, 5000, 33),
                                   (40, 257, 256)])
def test_state_in_place(mesa, B, T, D):
    """h_T may be h0 itself, also where several CTAs share a sequence and all read h0."""
    x, ga, gx, lam, _, h0, _ = inputs(B, T, D, "bf16", seed=T)
    want, wT = mesa.lru_forward(x, ga, gx, lam, h0=h0, return_state=True)
    lib, y, h = mesa._load(), torch.empty_like(x), torch.empty_like(h0)
    stream = torch.cuda.current_stream().cuda_stream
    for _ in range(20):
        h.copy_(h0)
        assert lib.mesa_lru_forward(x.data_ptr(), ga.data_ptr(), gx.data_ptr(), lam.data_ptr(), B, T, D, 1, h.data_ptr(),
                                    y.data_ptr(), h.data_ptr(), None, stream) == 0
        assert torch.equal(h, wT) and torch.equal(y, want)


# Walks of five tiles and more a CTA: clusters of 16, 8, 4, 2 and none, by tensor copies and by 4-byte copies
LONG = [("bf16", 1, 10277, 64), ("bf16", 3, 4173, 512), ("bf16", 3, 2200, 1024), ("bf16", 5, 1100, 1024),
        ("bf16", 10, 1100, 1024), ("bf16", 1, 10277, 66), ("f32", 1, 10277, 32), ("f32", 2, 4173, 512),
        ("f32", 5, 1100, 520), ("f32", 1, 10277, 33), ("f32", 5, 1100, 1003)]


@pytest.mark.parametrize("dtype,B,T,D", LONG)
def test_long_walks(mesa, dtype, B, T, D):
    x, ga, gx, lam, dy, h0, dh = inputs(B, T, D, dtype, seed=T + D)
    y, hT, saved = mesa.lru_forward(x, ga, gx, lam, h0=h0, return_state=True, return_saved=True)
    want, wT, ey, eT = ref.lru(x, ga, gx, lam, h0)
    ref.check(y, want, ey, "y")
    ref.check(hT, wT, eT, "h_T")
    at, eat = want[:, 63:-1:64], ey[:, 63:-1:64]
    ref.check(saved[:, 1:], at, eat, "saved")
    del want, ey
    got = mesa.lru_backward(x, ga, gx, lam, dy, saved=saved, dh_T=dh)
    want, bound = ref.lru_grads(x, ga, gx, lam, h0, dy, dh)
    for n, o, w, b in zip(("dx", "dgate_a", "dgate_x", "dlam", "dh0"), got, want, bound):
        ref.check(o, w, b, n)
    for o, o2 in zip(got, mesa.lru_backward(x, ga, gx, lam, dy, saved=saved, dh_T=dh)):
        assert torch.equal(o, o2)
    assert mesa.get_error() == 0


@pytest.mark.parametrize("lams", [(-120.0, -95.0, -60.0, -25.0, -15.0, -3.0, 0.0, 5.0, 60.0),
                                  (-120.0, -95.0, -60.0, -25.0, -15.0, -8.0, -6.0, -5.0, -4.0)],
                         ids=["any decay", "slow decays"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gradients_at_extreme_gates(mesa, dtype, lams):
    """The gradients' values where gates are closed, open and saturated."""
    B, T = 1, 200
    vals = torch.tensor([-float("inf"), -90.0, -60.0, -30.0, -10.0, 0.0, 10.0, 40.0, 100.0, float("inf")])
    lams = torch.tensor(lams)
    D = len(vals) * len(lams)
    x, ga, gx, lam, dy, h0, dh = inputs(B, T, D, dtype, seed=3)
    ga[:] = vals.repeat(len(lams)).to(ga)
    gx[:] = vals.flip(0).repeat(len(lams)).to(gx)
    gx[:, ::2] = torch.randn(100, D, generator=torch.Generator().manual_seed(5)).to(gx)
    lam[:] = lams.repeat_interleave(len(vals)).to(lam)
    _, saved = mesa.lru_forward(x, ga, gx, lam, h0=h0, return_saved=True)
    got = mesa.lru_backward(x, ga, gx, lam, dy, saved=saved, dh_T=dh)
    want, bound = ref.lru_grads(x, ga.float().clamp(-104, 104), gx.float().clamp(-104, 104), lam, h0, dy, dh)
    # A sigmoid below 2^-126 counts as 0, and 1 - a^2 is held to 1e-36: m = sqrt(2 * 8 softplus(60) * 2^-126) < 4e-18
    # may be lost, and an i below 2^-63. Times x, h (below 8 and 100) and g, sums of up to T + 1 terms below 6 (1206):
    # 4e-18 * 100 * 1206 < 5e-13 of an element, T of them in dlam.
    eps = 5e-13
    for n, o, w, b in zip(("dx", "dgate_a", "dgate_x", "dlam", "dh0"), got, want, bound):
        ref.check(o, w, b + (T * eps if n == "dlam" else eps), n)


def test_two_host_threads(mesa):
    """Calls from two host threads whose clusters, and so whose shared memory, differ in size."""
    import threading
    sets = [inputs(1, T, 64, "bf16", seed=T) for T in (300, 3000)]        # clusters of 2 (forward) or 4, and of 16

    def once(s):
        x, ga, gx, lam, dy, h0, dh = s
        y, saved = mesa.lru_forward(x, ga, gx, lam, h0=h0, return_saved=True)
        return (y,) + mesa.lru_backward(x, ga, gx, lam, dy, saved=saved, dh_T=dh)
    want = [once(s) for s in sets]
    torch.cuda.synchronize()
    wrong = []

    def loop(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                torch.cuda.current_stream().wait_stream(torch.cuda.default_stream())
                for _ in range(2000):
                    got = once(sets[i])
                torch.cuda.current_stream().synchronize()
            if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                wrong.append((i, "values"))
        except Exception as e:                                            # a refused launch
            wrong.append((i, str(e)))
    threads = [threading.Thread(target=loop, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong
    assert mesa.get_error() == 0


def test_two_host_threads_launch(mesa):
    """The same at the rate of the C ABI: no launch of a larger cluster is refused because a smaller one was prepared meanwhile."""
    import threading
    lib, refused, keep, args = mesa._load(), [0, 0], [], []
    for T in (300, 3000):
        x, ga, gx, lam, _, _, _ = inputs(1, T, 64, "bf16", seed=T)
        y, stream = torch.empty_like(x), torch.cuda.Stream()
        keep.append((x, ga, gx, lam, y, stream))
        args.append((x.data_ptr(), ga.data_ptr(), gx.data_ptr(), lam.data_ptr(), 1, T, 64, 1, None, y.data_ptr(), None, None,
                     stream.cuda_stream))
    torch.cuda.synchronize()

    def loop(i):
        for _ in range(60000):
            refused[i] += lib.mesa_lru_forward(*args[i]) != 0
    threads = [threading.Thread(target=loop, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert refused == [0, 0]
    for x, ga, gx, lam, y, _ in keep:
        assert torch.equal(y, mesa.lru_forward(x, ga, gx, lam))
