// mixers_api.cu -- the extern "C" entry points of mesa_mixers.h: argument
// checks, workspace carving and dispatch.
#include <math.h>

#include <initializer_list>

#include "mesa_common.cuh"
#include "mesa_internal.h"
#include "mixers_internal.h"

using namespace mesa;

namespace {

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
size_t elem_size(mesa_dtype d) { return d == MESA_BF16 ? 2 : 4; }
bool dtype_ok(mesa_dtype d) { return d == MESA_F32 || d == MESA_BF16; }

struct Range {
    const void* p;
    size_t n;
};
bool overlap(const Range& a, const Range& b) {
    const char* x = static_cast<const char*>(a.p);
    const char* y = static_cast<const char*>(b.p);
    return x && y && a.n && b.n && x < y + b.n && y < x + a.n;
}
// true if an output overlaps an input or another output
bool clash(std::initializer_list<Range> outs, std::initializer_list<Range> ins) {
    for (const Range* o = outs.begin(); o != outs.end(); ++o) {
        for (const Range& i : ins)
            if (overlap(*o, i)) return true;
        for (const Range* q = o + 1; q != outs.end(); ++q)
            if (overlap(*o, *q)) return true;
    }
    return false;
}
bool given(std::initializer_list<const void*> ps, size_t align) {
    for (const void* p : ps)
        if (!p || !aligned(p, align)) return false;
    return true;
}

mesa_status status(cudaError_t e) { return e == cudaSuccess ? MESA_OK : MESA_ERR_CUDA; }

// ---- recurrence ----
// Grids are one-dimensional: one CTA for each 32 channels or more of a sequence,
// up to kLruMaxCluster where that leaves SMs idle.
mesa_status lru_shape(int B, int T, int D, mesa_dtype dtype) {
    if (B < 1 || T < 0 || D < 1 || !dtype_ok(dtype)) return MESA_ERR_INVALID_ARG;
    if (T > (1 << 30) || (long long)B * ((D + 31LL) / 32) > (1LL << 27)) return MESA_ERR_UNSUPPORTED;
    return MESA_OK;
}

// ---- attention ----
mesa_status swa_shape(int B, int Hq, int Hkv, int d, int window, int sinks, float scale, mesa_dtype dtype) {
    if (B < 1 || Hq < 1 || Hkv < 1 || window < 1 || sinks < 0 || !dtype_ok(dtype)) return MESA_ERR_INVALID_ARG;
    if (Hq % Hkv != 0) return MESA_ERR_INVALID_ARG;
    if (!isfinite(scale) || !(scale > 0.f)) return MESA_ERR_INVALID_ARG;
    if (d != 16 && d != 32 && d != 64 && d != 128) return MESA_ERR_UNSUPPORTED;
    if (sinks > 128) return MESA_ERR_UNSUPPORTED;
    if ((long long)B * Hq > 65535) return MESA_ERR_UNSUPPORTED;          // grid.y limit
    return MESA_OK;
}
mesa_status swa_lengths(int T, int S) {
    if (T < 0 || S < T) return MESA_ERR_INVALID_ARG;
    if (S > (1 << 30)) return MESA_ERR_UNSUPPORTED;
    return MESA_OK;
}

mesa_status step_shape(int B, int Hq, int Hkv, int d, int window, int sinks, float scale, mesa_dtype dtype) {
    const mesa_status s = swa_shape(B, Hq, Hkv, d, window, sinks, scale, dtype);
    if (s != MESA_OK) return s;
    return (long long)sinks + window > 0x7fffffffLL ? MESA_ERR_UNSUPPORTED : MESA_OK;
}

#ifdef MESA_DEBUG
int g_lose_signals = 0;
#endif

}  // namespace

#ifdef MESA_DEBUG
int mesa::debug_lose_signal() { return g_lose_signals > 0 ? g_lose_signals--, 1 : 0; }
#endif

extern "C" {

size_t mesa_lru_saved_size(int B, int T, int D) {
    if (lru_shape(B, T, D, MESA_F32) != MESA_OK) return 0;
    return (size_t)B * ((T + kLruSave - 1) / kLruSave) * D * sizeof(float);
}

mesa_status mesa_lru_forward(const void* x, const void* gate_a, const void* gate_x, const float* lambda,
                             int B, int T, int D, mesa_dtype dtype, const float* h0, void* y, float* h_T,
                             float* saved, void* stream) {
    mesa_status s = lru_shape(B, T, D, dtype);
    if (s != MESA_OK) return s;
    const size_t es = elem_size(dtype), n = (size_t)B * T * D * es, nh = (size_t)B * D * 4;
    if (!given({lambda}, 4)) return MESA_ERR_INVALID_ARG;
    if (T > 0 && (!given({x, gate_a, gate_x, y}, es))) return MESA_ERR_INVALID_ARG;
    for (const void* p : {(const void*)h0, (const void*)h_T, (const void*)saved})
        if (!aligned(p, 4)) return MESA_ERR_INVALID_ARG;
    const Range hr{h_T == h0 ? nullptr : h0, nh};                     // the state may be updated in place
    if (clash({{y, n}, {h_T, nh}, {saved, mesa_lru_saved_size(B, T, D)}},
              {{x, n}, {gate_a, n}, {gate_x, n}, {lambda, (size_t)D * 4}, hr}))
        return MESA_ERR_INVALID_ARG;
    if (h_T && h_T == h0 && (overlap({h0, nh}, {y, n}) || overlap({h0, nh}, {saved, mesa_lru_saved_size(B, T, D)})))
        return MESA_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (T == 0) {
        if (!h_T || h_T == h0) return MESA_OK;
        return status(h0 ? cudaMemcpyAsync(h_T, h0, nh, cudaMemcpyDeviceToDevice, st) : cudaMemsetAsync(h_T, 0, nh, st));
    }
    return status(lru_forward({x, gate_a, gate_x, lambda, B, T, D, dtype, h0, y, h_T, saved}, st));
}

size_t mesa_lru_backward_workspace_size(int B, int T, int D, mesa_dtype dtype, int have_saved) {
    if (lru_shape(B, T, D, dtype) != MESA_OK) return 0;
    return round_up(lru_backward_rows(B, T) * D * sizeof(float), 256) +
           (have_saved ? 0 : round_up(mesa_lru_saved_size(B, T, D), 256));
}

mesa_status mesa_lru_backward(const void* x, const void* gate_a, const void* gate_x, const float* lambda,
                              int B, int T, int D, mesa_dtype dtype, const float* h0, const float* saved,
                              const void* dy, const float* dh_T, void* dx, void* dgate_a, void* dgate_x,
                              float* dlambda, float* dh0, void* workspace, size_t ws_bytes, void* stream) {
    mesa_status s = lru_shape(B, T, D, dtype);
    if (s != MESA_OK) return s;
    const size_t es = elem_size(dtype), n = (size_t)B * T * D * es, nh = (size_t)B * D * 4, nd = (size_t)D * 4;
    if (!given({lambda, dlambda}, 4)) return MESA_ERR_INVALID_ARG;
    if (T > 0 && !given({x, gate_a, gate_x, dy, dx, dgate_a, dgate_x}, es)) return MESA_ERR_INVALID_ARG;
    for (const void* p : {(const void*)h0, (const void*)saved, (const void*)dh_T, (const void*)dh0})
        if (!aligned(p, 4)) return MESA_ERR_INVALID_ARG;
    const size_t ns = mesa_lru_saved_size(B, T, D), need = mesa_lru_backward_workspace_size(B, T, D, dtype, saved != nullptr);
    if (clash({{dx, n}, {dgate_a, n}, {dgate_x, n}, {dlambda, nd}, {dh0, nh}, {T > 0 ? workspace : nullptr, need}},
              {{x, n}, {gate_a, n}, {gate_x, n}, {lambda, nd}, {h0, nh}, {saved, ns}, {dy, n}, {dh_T, nh}}))
        return MESA_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (T == 0) {
        cudaError_t e = cudaMemsetAsync(dlambda, 0, nd, st);
        if (e == cudaSuccess && dh0)
            e = dh_T ? cudaMemcpyAsync(dh0, dh_T, nh, cudaMemcpyDeviceToDevice, st) : cudaMemsetAsync(dh0, 0, nh, st);
        return status(e);
    }
    if (!workspace || ws_bytes < need) return MESA_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return MESA_ERR_INVALID_ARG;
    char* w = static_cast<char*>(workspace);
    float* partial = reinterpret_cast<float*>(w);
    LruArgs f{x, gate_a, gate_x, lambda, B, T, D, dtype, h0, nullptr, nullptr, const_cast<float*>(saved)};
    if (!saved) {
        f.saved = reinterpret_cast<float*>(w + round_up(lru_backward_rows(B, T) * D * sizeof(float), 256));
        cudaError_t e = lru_forward(f, st);
        if (e != cudaSuccess) return MESA_ERR_CUDA;
    }
    return status(lru_backward({f, dy, dh_T, dx, dgate_a, dgate_x, dlambda, dh0, partial}, st));
}

mesa_status mesa_lru_step(const void* x, const void* gate_a, const void* gate_x, const float* lambda,
                          int B, int D, mesa_dtype dtype, const float* h_in, float* h_out, void* y, void* stream) {
    mesa_status s = lru_shape(B, 1, D, dtype);
    if (s != MESA_OK) return s;
    const size_t es = elem_size(dtype), n = (size_t)B * D * es, nh = (size_t)B * D * 4;
    if (!given({lambda, h_in, h_out}, 4) || !given({x, gate_a, gate_x, y}, es)) return MESA_ERR_INVALID_ARG;
    if (clash({{y, n}, {h_out, nh}},
              {{x, n}, {gate_a, n}, {gate_x, n}, {lambda, (size_t)D * 4}, {h_in == h_out ? nullptr : h_in, nh}}))
        return MESA_ERR_INVALID_ARG;
    return status(lru_step(x, gate_a, gate_x, lambda, B, D, dtype, h_in, h_out, y, static_cast<cudaStream_t>(stream)));
}

mesa_status mesa_swa_forward(const void* q, const void* k, const void* v, int B, int Hq, int Hkv, int T, int S,
                             int d, int window, int sinks, float scale, mesa_dtype dtype, void* out, float* lse,
                             void* stream) {
    mesa_status s = swa_shape(B, Hq, Hkv, d, window, sinks, scale, dtype);
    if (s == MESA_OK) s = swa_lengths(T, S);
    if (s != MESA_OK) return s;
    if (T == 0) return MESA_OK;
    if (!given({q, k, v, out}, 16) || !aligned(lse, 4)) return MESA_ERR_INVALID_ARG;
    const size_t es = elem_size(dtype), nq = (size_t)B * Hq * T * d * es, nk = (size_t)B * Hkv * S * d * es;
    if (clash({{out, nq}, {lse, (size_t)B * Hq * T * 4}}, {{q, nq}, {k, nk}, {v, nk}})) return MESA_ERR_INVALID_ARG;
    SwaArgs a{q, k, v, B, Hq, Hkv, T, S, d, window < S ? window : S, sinks, scale, dtype, out, lse};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return status(swa_tc_supported(d, dtype) ? swa_forward_tc(a, st) : swa_forward_simt(a, st));
}

size_t mesa_swa_backward_workspace_size(int B, int Hq, int Hkv, int T, int S, int d, int sinks, mesa_dtype dtype) {
    if (swa_shape(B, Hq, Hkv, d, 1, sinks, 1.f, dtype) != MESA_OK || swa_lengths(T, S) != MESA_OK) return 0;
    return swa_tc_supported(d, dtype) ? swa_tc_workspace_bytes(B, Hq, Hkv, T, d, sinks)
                                      : round_up(swa_simt_workspace_bytes(B, Hq, Hkv, T, S, d, sinks), 256);
}

mesa_status mesa_swa_backward(const void* q, const void* k, const void* v, const void* out, const float* lse,
                              const void* dout, int B, int Hq, int Hkv, int T, int S, int d, int window, int sinks,
                              float scale, mesa_dtype dtype, void* dq, void* dk, void* dv, void* workspace,
                              size_t ws_bytes, void* stream) {
    mesa_status s = swa_shape(B, Hq, Hkv, d, window, sinks, scale, dtype);
    if (s == MESA_OK) s = swa_lengths(T, S);
    if (s != MESA_OK) return s;
    if (S == 0) return MESA_OK;
    const size_t es = elem_size(dtype), nq = (size_t)B * Hq * T * d * es, nk = (size_t)B * Hkv * S * d * es;
    if (!given({dk, dv}, 16)) return MESA_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (T == 0) {
        if (clash({{dk, nk}, {dv, nk}}, {{k, nk}, {v, nk}})) return MESA_ERR_INVALID_ARG;
        cudaError_t e = cudaMemsetAsync(dk, 0, nk, st);
        return status(e == cudaSuccess ? cudaMemsetAsync(dv, 0, nk, st) : e);
    }
    if (!given({q, k, v, out, dout, dq}, 16) || !given({lse}, 4)) return MESA_ERR_INVALID_ARG;
    const size_t need = mesa_swa_backward_workspace_size(B, Hq, Hkv, T, S, d, sinks, dtype);
    if (clash({{dq, nq}, {dk, nk}, {dv, nk}, {workspace, need}},
              {{q, nq}, {k, nk}, {v, nk}, {out, nq}, {lse, (size_t)B * Hq * T * 4}, {dout, nq}}))
        return MESA_ERR_INVALID_ARG;
    if (!workspace || ws_bytes < need) return MESA_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return MESA_ERR_INVALID_ARG;
    SwaArgs f{q, k, v, B, Hq, Hkv, T, S, d, window < S ? window : S, sinks, scale, dtype,
              const_cast<void*>(out), const_cast<float*>(lse)};
    SwaBackwardArgs a{f, dout, dq, dk, dv, workspace};
    cudaError_t e = swa_tc_supported(d, dtype) ? swa_backward_tc(a, st) : swa_backward_simt(a, st);
    if (e == cudaSuccess && (S == 1 || (window == 1 && sinks == 0))) {
        // every query sees one key, at weight 1 whatever the score: the
        // gradients are zero, not the rounding of dP - delta
        e = cudaMemsetAsync(dq, 0, nq, st);
        if (e == cudaSuccess) e = cudaMemsetAsync(dk, 0, nk, st);
    }
    return status(e);
}

size_t mesa_swa_step_workspace_size(int B, int Hq, int Hkv, int d, int window, int sinks, mesa_dtype dtype) {
    if (step_shape(B, Hq, Hkv, d, window, sinks, 1.f, dtype) != MESA_OK) return 0;
    SwaStepArgs a{};
    a.B = B, a.Hq = Hq, a.Hkv = Hkv, a.d = d, a.window = window, a.sinks = sinks, a.dtype = dtype;
    return round_up(swa_step_workspace_bytes(a), 256);
}

mesa_status mesa_swa_step(const void* q, const void* k, const void* v, void* k_cache, void* v_cache,
                          const int32_t* pos, int B, int Hq, int Hkv, int d, int window, int sinks, float scale,
                          mesa_dtype dtype, void* out, void* workspace, size_t ws_bytes, void* stream) {
    mesa_status s = step_shape(B, Hq, Hkv, d, window, sinks, scale, dtype);
    if (s != MESA_OK) return s;
    if (!given({q, k, v, k_cache, v_cache, out}, 16) || !given({pos}, 4)) return MESA_ERR_INVALID_ARG;
    const size_t es = elem_size(dtype), nq = (size_t)B * Hq * d * es, nk = (size_t)B * Hkv * d * es;
    const size_t nc = nk * ((size_t)sinks + window);
    const size_t need = mesa_swa_step_workspace_size(B, Hq, Hkv, d, window, sinks, dtype);
    if (need && (!workspace || ws_bytes < need)) return MESA_ERR_WORKSPACE;
    if (need && !aligned(workspace, 256)) return MESA_ERR_INVALID_ARG;
    if (clash({{out, nq}, {k_cache, nc}, {v_cache, nc}, {workspace, need}},
              {{q, nq}, {k, nk}, {v, nk}, {pos, (size_t)B * 4}}))
        return MESA_ERR_INVALID_ARG;
    return status(swa_step({q, k, v, k_cache, v_cache, pos, B, Hq, Hkv, d, window, sinks, scale, dtype, out, workspace},
                           static_cast<cudaStream_t>(stream)));
}

mesa_status mesa_swa_cache_fill(const void* k, const void* v, void* k_cache, void* v_cache, const int32_t* lens,
                                int B, int Hkv, int S, int d, int window, int sinks, int start, mesa_dtype dtype,
                                void* stream) {
    mesa_status s = swa_shape(B, Hkv, Hkv, d, window, sinks, 1.f, dtype);
    if (s != MESA_OK) return s;
    if (S < 0 || start < 0) return MESA_ERR_INVALID_ARG;
    if ((long long)sinks + window > 0x7fffffffLL || (long long)start + S > 0x7fffffffLL) return MESA_ERR_UNSUPPORTED;
    if (S == 0) return MESA_OK;
    if (!given({k, v, k_cache, v_cache}, 16) || !aligned(lens, 4)) return MESA_ERR_INVALID_ARG;
    const size_t row = (size_t)B * Hkv * d * elem_size(dtype), nk = row * S, nc = row * ((size_t)sinks + window);
    if (clash({{k_cache, nc}, {v_cache, nc}}, {{k, nk}, {v, nk}, {lens, (size_t)B * 4}})) return MESA_ERR_INVALID_ARG;
    return status(swa_cache_fill(k, v, k_cache, v_cache, lens, B, Hkv, S, d, window, sinks, start, dtype,
                                 static_cast<cudaStream_t>(stream)));
}

#ifdef MESA_DEBUG
mesa_status mesa_debug_lose_signal(int launches) {
    if (launches < 0) return MESA_ERR_INVALID_ARG;
    g_lose_signals = launches;
    return MESA_OK;
}
#endif

}  // extern "C"
