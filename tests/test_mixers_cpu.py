"""The entry points of mesa_mixers.h refuse bad arguments on the host, before
any launch; and the 64-bit references the GPU tests compare with agree with
autograd and with one another. No GPU needed."""
import ctypes
import math

import pytest
import torch

import mixers_ref as ref

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
A = [(i + 1) << 32 for i in range(16)]        # far apart, aligned, never dereferenced


@pytest.fixture(scope="module")
def lib():
    from test_sequence_layer_b200 import build, mesa
    build.build()
    return mesa._load()


def lru_fwd(lib, **kw):
    a = dict(x=A[0], ga=A[1], gx=A[2], lam=A[3], B=2, T=70, D=8, dt=1, h0=None, y=A[4], hT=None, saved=None)
    a.update(kw)
    return lib.mesa_lru_forward(*a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(B=0), INVALID), (dict(T=-1), INVALID), (dict(D=0), INVALID), (dict(dt=2), INVALID), (dict(x=None), INVALID),
    (dict(gx=None), INVALID), (dict(lam=None), INVALID), (dict(y=None), INVALID), (dict(x=A[0] + 1), INVALID),
    (dict(dt=0, y=A[4] + 2), INVALID), (dict(lam=A[3] + 2), INVALID), (dict(h0=A[5] + 2), INVALID),
    (dict(saved=A[5] + 1), INVALID), (dict(y=A[0]), INVALID), (dict(y=A[0] + 2 * 70 * 8 * 2 - 2), INVALID),
    (dict(hT=A[4]), INVALID), (dict(h0=A[4], hT=A[4]), INVALID), (dict(saved=A[3]), INVALID),
    (dict(T=(1 << 30) + 1), UNSUPPORTED), (dict(B=1 << 26, D=1 << 10), UNSUPPORTED)])
def test_lru_forward_refusals(lib, kw, want):
    assert lru_fwd(lib, **kw) == want


def lru_bwd(lib, **kw):
    a = dict(x=A[0], ga=A[1], gx=A[2], lam=A[3], B=2, T=70, D=8, dt=1, h0=None, saved=A[4], dy=A[5], dhT=None, dx=A[6],
             dga=A[7], dgx=A[8], dlam=A[9], dh0=A[10], ws=A[11], n=1 << 20)
    a.update(kw)
    return lib.mesa_lru_backward(*a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(dy=None), INVALID), (dict(dlam=None), INVALID), (dict(dx=None), INVALID), (dict(dx=A[0]), INVALID),
    (dict(dga=A[6]), INVALID), (dict(dh0=A[9]), INVALID), (dict(ws=None), WORKSPACE), (dict(n=16), WORKSPACE),
    (dict(ws=A[11] + 16), INVALID), (dict(ws=A[0]), INVALID), (dict(saved=A[4] + 2), INVALID), (dict(B=0), INVALID)])
def test_lru_backward_refusals(lib, kw, want):
    assert lru_bwd(lib, **kw) == want


def test_lru_sizes(lib):
    assert lib.mesa_lru_saved_size(2, 65, 10) == 2 * 2 * 10 * 4
    assert lib.mesa_lru_saved_size(0, 65, 10) == 0
    with_saved = lib.mesa_lru_backward_workspace_size(2, 65, 10, 1, 1)
    assert 0 < with_saved < lib.mesa_lru_backward_workspace_size(2, 65, 10, 1, 0)
    a = [A[0], A[1], A[2], A[3], 2, 8, 1, A[4], A[4], A[5], None]
    for i, bad in ((0, None), (7, None), (9, A[4]), (4, 0), (9, A[5] + 1)):
        b = list(a)
        b[i] = bad
        assert lib.mesa_lru_step(*b) == INVALID, i


def swa_fwd(lib, **kw):
    a = dict(q=A[0], k=A[1], v=A[2], B=2, Hq=4, Hkv=2, T=10, S=20, d=64, window=8, sinks=2,
             scale=ctypes.c_float(0.1), dt=1, out=A[3], lse=A[4])
    a.update(kw)
    return lib.mesa_swa_forward(*a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(B=0), INVALID), (dict(Hq=3), INVALID), (dict(Hkv=0), INVALID), (dict(T=21), INVALID), (dict(T=-1), INVALID),
    (dict(window=0), INVALID), (dict(sinks=-1), INVALID), (dict(dt=5), INVALID), (dict(q=None), INVALID),
    (dict(out=None), INVALID), (dict(k=A[1] + 8), INVALID), (dict(lse=A[4] + 2), INVALID), (dict(out=A[0]), INVALID),
    (dict(lse=A[3]), INVALID), (dict(scale=ctypes.c_float(math.nan)), INVALID), (dict(scale=ctypes.c_float(-1)), INVALID),
    (dict(scale=ctypes.c_float(math.inf)), INVALID), (dict(d=48), UNSUPPORTED), (dict(d=256), UNSUPPORTED),
    (dict(sinks=129), UNSUPPORTED), (dict(B=40000), UNSUPPORTED), (dict(S=(1 << 30) + 1), UNSUPPORTED),
    (dict(T=0, q=None), OK)])
def test_swa_forward_refusals(lib, kw, want):
    assert swa_fwd(lib, **kw) == want


def swa_bwd(lib, **kw):
    a = dict(q=A[0], k=A[1], v=A[2], out=A[3], lse=A[4], dout=A[5], B=2, Hq=4, Hkv=2, T=10, S=20, d=64, window=8,
             sinks=2, scale=ctypes.c_float(0.1), dt=1, dq=A[6], dk=A[7], dv=A[8], ws=A[9], n=1 << 24)
    a.update(kw)
    return lib.mesa_swa_backward(*a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(lse=None), INVALID), (dict(dout=None), INVALID), (dict(dk=None), INVALID), (dict(dq=A[0]), INVALID),
    (dict(dv=A[7]), INVALID), (dict(ws=None), WORKSPACE), (dict(n=8), WORKSPACE), (dict(ws=A[9] + 64), INVALID),
    (dict(ws=A[1]), INVALID), (dict(d=80), UNSUPPORTED), (dict(S=0, T=0), OK)])
def test_swa_backward_refusals(lib, kw, want):
    assert swa_bwd(lib, **kw) == want
    if kw == dict(S=0, T=0):
        assert lib.mesa_swa_backward_workspace_size(2, 4, 2, 10, 20, 64, 129, 1) == 0


def swa_step(lib, **kw):
    a = dict(q=A[0], k=A[1], v=A[2], kc=A[3], vc=A[4], pos=A[5], B=2, Hq=4, Hkv=2, d=64, window=8, sinks=2,
             scale=ctypes.c_float(0.1), dt=1, out=A[6], ws=A[7], n=1 << 24)
    a.update(kw)
    return lib.mesa_swa_step(*a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(pos=None), INVALID), (dict(pos=A[5] + 2), INVALID), (dict(kc=None), INVALID), (dict(vc=A[3]), INVALID),
    (dict(out=A[0]), INVALID), (dict(out=A[3] + 16), INVALID), (dict(Hq=5), INVALID), (dict(window=0), INVALID),
    (dict(window=2 ** 31 - 1), UNSUPPORTED), (dict(sinks=200), UNSUPPORTED), (dict(d=24), UNSUPPORTED),
    (dict(window=1 << 20, ws=None), WORKSPACE), (dict(window=1 << 20, n=100), WORKSPACE),
    (dict(window=1 << 20, ws=A[7] + 16), INVALID), (dict(window=1 << 20, ws=A[6]), INVALID)])
def test_swa_step_refusals(lib, kw, want):
    assert swa_step(lib, **kw) == want


def test_swa_cache_fill_refusals(lib):
    a = dict(k=A[0], v=A[1], kc=A[2], vc=A[3], lens=None, B=2, Hkv=2, S=20, d=64, window=8, sinks=2, start=0, dt=1)

    def call(**kw):
        return lib.mesa_swa_cache_fill(*{**a, **kw}.values(), None)
    assert call(S=-1) == INVALID and call(start=-1) == INVALID and call(k=None) == INVALID
    assert call(vc=A[2]) == INVALID and call(lens=A[4] + 1) == INVALID and call(kc=A[0]) == INVALID
    assert call(start=2 ** 31 - 10) == UNSUPPORTED and call(S=0) == OK


def test_binding_refuses_host_tensors():
    from test_sequence_layer_b200 import mesa
    x = torch.zeros(1, 4, 8)
    with pytest.raises(ValueError, match="CUDA"):
        mesa.lru_forward(x, x, x, torch.zeros(8))
    with pytest.raises(ValueError, match="CUDA"):
        mesa.swa_forward(x[None, :, :, :], x[None], x[None], window=4)
    with pytest.raises(TypeError):
        mesa.lru_forward(x.double(), x, x, torch.zeros(8))


def test_reference_gradients_agree_with_autograd():
    torch.manual_seed(0)
    x, ga, gx = (torch.randn(2, 9, 3, dtype=torch.float64, requires_grad=True) for _ in range(3))
    lam = torch.randn(3, dtype=torch.float64, requires_grad=True)
    h0 = torch.randn(2, 3, dtype=torch.float64, requires_grad=True)
    dy, dh = torch.randn(2, 9, 3, dtype=torch.float64), torch.randn(2, 3, dtype=torch.float64)
    a = torch.exp(-8 * torch.nn.functional.softplus(lam) * torch.sigmoid(ga))
    h, loss = h0, 0
    for t in range(9):
        h = a[:, t] * h + torch.sqrt(1 - a[:, t] ** 2) * torch.sigmoid(gx[:, t]) * x[:, t]
        loss = loss + (h * dy[:, t]).sum()
    want = torch.autograd.grad(loss + (h * dh).sum(), (x, ga, gx, lam, h0))
    got, _ = ref.lru_grads(*(t.detach() for t in (x, ga, gx, lam, h0)), dy, dh)
    for w, g in zip(want, got):
        assert torch.allclose(w, g, rtol=1e-10, atol=1e-12)


def test_reference_attention_agrees_with_autograd_and_loops():
    torch.manual_seed(1)
    q = torch.randn(1, 4, 9, 16, dtype=torch.float64, requires_grad=True)
    k, v = (torch.randn(1, 2, 13, 16, dtype=torch.float64, requires_grad=True) for _ in range(2))
    do = torch.randn(1, 4, 9, 16, dtype=torch.float64)
    rows = []
    for h in range(4):
        for t in range(9):
            p = 13 - 9 + t
            seen = [j for j in range(p + 1) if p - j < 4 or j < 2]
            w = torch.softmax(k[0, h // 2, seen] @ q[0, h, t] / 4, 0)
            rows.append(w @ v[0, h // 2, seen])
    out = torch.stack(rows).view(1, 4, 9, 16)
    want = torch.autograd.grad((out * do).sum(), (q, k, v))
    r = ref.swa(q.detach(), k.detach(), v.detach(), 4, 2, dout=do)
    assert torch.allclose(r["out"][0], out, rtol=1e-10, atol=1e-12)
    for n, w in zip(("dq", "dk", "dv"), want):
        assert torch.allclose(r[n][0], w, rtol=1e-10, atol=1e-12), n


def test_no_kernel_that_no_call_reaches(lib):
    """bf16 of 64 and 128 columns runs on matrix instructions alone: the library holds no fp32-arithmetic kernel for it."""
    import shutil
    import subprocess
    from test_sequence_layer_b200 import mesa
    if not shutil.which("nm"):
        pytest.skip("needs nm")
    names = subprocess.run(["nm", "-C", mesa.library_path()], check=True, capture_output=True, text=True).stdout
    for kernel in ("swa_fwd_kernel", "swa_dq_kernel", "swa_dkv_kernel", "swa_dkv_sum_kernel", "swa_step_simt_kernel"):
        for d in (16, 32):
            assert f"{kernel}<__nv_bfloat16, {d}>" in names, (kernel, d)
        for d in (64, 128):
            assert f"{kernel}<float, {d}>" in names and f"{kernel}<__nv_bfloat16, {d}>" not in names, (kernel, d)


def test_fault_injection_is_in_the_debug_library_alone(lib):
    from test_sequence_layer_b200 import build
    assert not hasattr(lib, "mesa_debug_lose_signal")
    dlib = ctypes.CDLL(build.build(debug=True))
    assert dlib.mesa_debug_lose_signal(-1) == INVALID
