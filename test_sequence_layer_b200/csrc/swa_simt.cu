// swa_simt.cu -- sliding-window attention with sinks in fp32 on the CUDA cores:
// every type and width the tensor-core kernels do not take.
//
// 64 x 64 tiles of scores; a thread holds a 4 x 4 block of them (rows 4 ty + i,
// columns tx + 16 j). Rows of shared tiles are padded by four floats, so the
// 16-byte row reads of eight neighbouring lanes touch all banks once. The
// forward keeps a running maximum and sum per row; the backward is two kernels,
// one per query tile (dq) and one per key tile (dk, dv), each summing in
// registers, so no gradient depends on the order of atomics.
#include <math.h>

#include "mesa_common.cuh"
#include "mesa_internal.h"
#include "mixers_internal.h"
#include "swa_common.cuh"

namespace mesa {
namespace {

constexpr int kT = 64;                          // tile edge
constexpr int kPS = kT + 4;                     // padded row of a score tile
constexpr int kThreads = 256;

__device__ __forceinline__ void st_out(float* p, float v) { *p = v; }
__device__ __forceinline__ void st_out(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// rows [r0, r0 + 64) of a [rows][D] tensor into a padded fp32 tile; rows past
// the end become zeros
template <typename T, int D>
__device__ __forceinline__ void load_tile(float* s, const T* g, int r0, int rows) {
    for (int i = threadIdx.x; i < kT * D; i += kThreads) {
        const int r = i / D, c = i % D;
        s[r * (D + 4) + c] = r0 + r < rows ? ld_in(g, (size_t)(r0 + r) * D + c) : 0.f;
    }
}

// acc[i][j] += rows (4 ty + i) of A . rows (tx + 16 j) of B
template <int D>
__device__ __forceinline__ void dot_tile(const float* A, const float* B, int ty, int tx, float (&acc)[4][4]) {
#pragma unroll 4
    for (int c = 0; c < D; c += 4) {
        float4 a[4], b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const float4*>(A + (4 * ty + i) * (D + 4) + c);
#pragma unroll
        for (int j = 0; j < 4; ++j) b[j] = *reinterpret_cast<const float4*>(B + (tx + 16 * j) * (D + 4) + c);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                acc[i][j] = fmaf(a[i].x, b[j].x, acc[i][j]);
                acc[i][j] = fmaf(a[i].y, b[j].y, acc[i][j]);
                acc[i][j] = fmaf(a[i].z, b[j].z, acc[i][j]);
                acc[i][j] = fmaf(a[i].w, b[j].w, acc[i][j]);
            }
    }
}

// acc[i][c] += sum_k W[4 ty + i][k] B[k][tx + 16 c], or with W transposed
// (W[k][4 ty + i]); W is a padded score tile
template <int D, bool TRANS>
__device__ __forceinline__ void weighted_rows(const float* W, const float* B, int ty, int tx, float (&acc)[4][D / 16]) {
#pragma unroll 4
    for (int k = 0; k < kT; ++k) {
        float w[4];
        if (TRANS) {
            const float4 v = *reinterpret_cast<const float4*>(W + k * kPS + 4 * ty);
            w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = W[(4 * ty + i) * kPS + k];
        }
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
            const float b = B[k * (D + 4) + tx + 16 * c];
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[i][c] = fmaf(w[i], b, acc[i][c]);
        }
    }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) swa_fwd_kernel(SwaArgs p) {
    extern __shared__ float4 smem4[];
    float* sQ = reinterpret_cast<float*>(smem4);
    float* sK = sQ + kT * (D + 4);
    float* sV = sK + kT * (D + 4);
    float* sP = sV + kT * (D + 4);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int bh = blockIdx.y, b = bh / p.Hq, h = bh % p.Hq, hk = h / (p.Hq / p.Hkv);
    const int t0 = blockIdx.x * kT, off = p.S - p.T;
    const T* q = static_cast<const T*>(p.q) + (size_t)bh * p.T * D;
    const T* k = static_cast<const T*>(p.k) + ((size_t)b * p.Hkv + hk) * p.S * D;
    const T* v = static_cast<const T*>(p.v) + ((size_t)b * p.Hkv + hk) * p.S * D;
    load_tile<T, D>(sQ, q, t0, p.T);
    const int p0 = off + t0, p1 = off + min(t0 + kT, p.T) - 1;
    const swa::KeyTiles kt(p0, p1, p.window, p.sinks, kT);
    float m[4], l[4], o[4][D / 16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m[i] = -INFINITY, l[i] = 0.f;
#pragma unroll
        for (int c = 0; c < D / 16; ++c) o[i][c] = 0.f;
    }
    for (int n = 0; n < kt.n; ++n) {
        const int j0 = kt.tile(n) * kT;
        __syncthreads();
        load_tile<T, D>(sK, k, j0, p.S);
        load_tile<T, D>(sV, v, j0, p.S);
        __syncthreads();
        float s[4][4] = {};
        dot_tile<D>(sQ, sK, ty, tx, s);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float mx = m[i];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[i][j] = swa::visible(p0 + 4 * ty + i, j0 + tx + 16 * j, p.window, p.sinks) ? s[i][j] * p.scale : -INFINITY;
                mx = fmaxf(mx, s[i][j]);
            }
#pragma unroll
            for (int x = 8; x; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, x));
            const float ref = mx == -INFINITY ? 0.f : mx;        // nothing visible yet in this row
            const float keep = expf(m[i] - ref);
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float e = expf(s[i][j] - ref);
                sum += e;
                sP[(4 * ty + i) * kPS + tx + 16 * j] = e;
            }
#pragma unroll
            for (int x = 8; x; x >>= 1) sum += __shfl_xor_sync(~0u, sum, x);
            m[i] = mx;
            l[i] = l[i] * keep + sum;
#pragma unroll
            for (int c = 0; c < D / 16; ++c) o[i][c] *= keep;
        }
        __syncwarp();                            // a score row lives in one half warp
        weighted_rows<D, false>(sP, sV, ty, tx, o);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int t = t0 + 4 * ty + i;
        if (t >= p.T) continue;
        const float inv = 1.f / l[i];
        T* out = static_cast<T*>(p.out) + ((size_t)bh * p.T + t) * D;
#pragma unroll
        for (int c = 0; c < D / 16; ++c) st_out(out + tx + 16 * c, o[i][c] * inv);
        if (p.lse && tx == 0) p.lse[(size_t)bh * p.T + t] = m[i] + logf(l[i]);
    }
}

// delta = rowsum(dout * out): one warp per row
template <typename T>
__global__ void swa_delta_kernel(const T* __restrict__ out, const T* __restrict__ dout, size_t rows, int d, float* delta) {
    const size_t r = (size_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (r >= rows) return;
    float s = 0.f;
    for (int c = threadIdx.x & 31; c < d; c += 32) s = fmaf(ld_in(out, r * d + c), ld_in(dout, r * d + c), s);
#pragma unroll
    for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(~0u, s, x);
    if ((threadIdx.x & 31) == 0) delta[r] = s;
}

// P and dS of one 64 x 64 tile pair into shared memory (rows: queries)
template <int D>
__device__ __forceinline__ void grad_scores(const SwaArgs& p, const float* sQ, const float* sK, const float* sDo,
                                            const float* sV, const float* sL, const float* sDl, int p0, int tleft,
                                            int j0, int ty, int tx, float* sP, float* sDs) {
    float s[4][4] = {}, dp[4][4] = {};
    dot_tile<D>(sQ, sK, ty, tx, s);
    dot_tile<D>(sDo, sV, ty, tx, dp);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 4 * ty + i;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int c = tx + 16 * j;
            const bool vis = r < tleft && swa::visible(p0 + r, j0 + c, p.window, p.sinks);
            const float w = vis ? expf(s[i][j] * p.scale - sL[r]) : 0.f;
            if (sP) sP[r * kPS + c] = w;
            sDs[r * kPS + c] = vis ? w * (dp[i][j] - sDl[r]) * p.scale : 0.f;
        }
    }
}

__device__ __forceinline__ void load_stats(float* sL, float* sDl, const float* lse, const float* delta, int t0, int T) {
    if (threadIdx.x < kT) {
        const bool in = t0 + (int)threadIdx.x < T;
        sL[threadIdx.x] = in ? lse[t0 + threadIdx.x] : 0.f;
        sDl[threadIdx.x] = in ? delta[t0 + threadIdx.x] : 0.f;
    }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) swa_dq_kernel(SwaBackwardArgs a, const float* delta) {
    const SwaArgs& p = a.f;
    extern __shared__ float4 smem4[];
    float* sQ = reinterpret_cast<float*>(smem4);
    float* sDo = sQ + kT * (D + 4);
    float* sK = sDo + kT * (D + 4);
    float* sV = sK + kT * (D + 4);
    float* sDs = sV + kT * (D + 4);
    float* sL = sDs + kT * kPS;
    float* sDl = sL + kT;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int bh = blockIdx.y, b = bh / p.Hq, hk = (bh % p.Hq) / (p.Hq / p.Hkv);
    const int t0 = blockIdx.x * kT, off = p.S - p.T;
    const T* k = static_cast<const T*>(p.k) + ((size_t)b * p.Hkv + hk) * p.S * D;
    const T* v = static_cast<const T*>(p.v) + ((size_t)b * p.Hkv + hk) * p.S * D;
    load_tile<T, D>(sQ, static_cast<const T*>(p.q) + (size_t)bh * p.T * D, t0, p.T);
    load_tile<T, D>(sDo, static_cast<const T*>(a.dout) + (size_t)bh * p.T * D, t0, p.T);
    load_stats(sL, sDl, p.lse + (size_t)bh * p.T, delta + (size_t)bh * p.T, t0, p.T);
    const int p0 = off + t0, p1 = off + min(t0 + kT, p.T) - 1;
    const swa::KeyTiles kt(p0, p1, p.window, p.sinks, kT);
    float dq[4][D / 16] = {};
    for (int n = 0; n < kt.n; ++n) {
        const int j0 = kt.tile(n) * kT;
        __syncthreads();
        load_tile<T, D>(sK, k, j0, p.S);
        load_tile<T, D>(sV, v, j0, p.S);
        __syncthreads();
        grad_scores<D>(p, sQ, sK, sDo, sV, sL, sDl, p0, p.T - t0, j0, ty, tx, nullptr, sDs);
        __syncwarp();
        weighted_rows<D, false>(sDs, sK, ty, tx, dq);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int t = t0 + 4 * ty + i;
        if (t >= p.T) continue;
        T* o = static_cast<T*>(a.dq) + ((size_t)bh * p.T + t) * D;
#pragma unroll
        for (int c = 0; c < D / 16; ++c) st_out(o + tx + 16 * c, dq[i][c]);
    }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) swa_dkv_kernel(SwaBackwardArgs a, const float* delta) {
    const SwaArgs& p = a.f;
    extern __shared__ float4 smem4[];
    float* sK = reinterpret_cast<float*>(smem4);
    float* sV = sK + kT * (D + 4);
    float* sQ = sV + kT * (D + 4);
    float* sDo = sQ + kT * (D + 4);
    float* sP = sDo + kT * (D + 4);
    float* sDs = sP + kT * kPS;
    float* sL = sDs + kT * kPS;
    float* sDl = sL + kT;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int G = p.Hq / p.Hkv, b = blockIdx.y / p.Hkv, hk = blockIdx.y % p.Hkv;
    const int j0 = blockIdx.x * kT, off = p.S - p.T;
    const size_t kv = ((size_t)b * p.Hkv + hk) * p.S * D;
    load_tile<T, D>(sK, static_cast<const T*>(p.k) + kv, j0, p.S);
    load_tile<T, D>(sV, static_cast<const T*>(p.v) + kv, j0, p.S);
    int ta, tb;
    swa::query_range(j0, min(j0 + kT, p.S) - 1, p.T, p.S, p.window, p.sinks, ta, tb);
    float dk[4][D / 16] = {}, dv[4][D / 16] = {};
    for (int g = 0; g < G; ++g) {
        const size_t row = ((size_t)b * p.Hq + hk * G + g) * p.T;
        for (int t0 = ta / kT * kT; t0 < tb; t0 += kT) {
            __syncthreads();
            load_tile<T, D>(sQ, static_cast<const T*>(p.q) + row * D, t0, p.T);
            load_tile<T, D>(sDo, static_cast<const T*>(a.dout) + row * D, t0, p.T);
            load_stats(sL, sDl, p.lse + row, delta + row, t0, p.T);
            __syncthreads();
            grad_scores<D>(p, sQ, sK, sDo, sV, sL, sDl, off + t0, p.T - t0, j0, ty, tx, sP, sDs);
            __syncthreads();
            weighted_rows<D, true>(sP, sDo, ty, tx, dv);
            weighted_rows<D, true>(sDs, sQ, ty, tx, dk);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int j = j0 + 4 * ty + i;
        if (j >= p.S) continue;
        T* ok = static_cast<T*>(a.dk) + kv + (size_t)j * D;
        T* ov = static_cast<T*>(a.dv) + kv + (size_t)j * D;
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
            st_out(ok + tx + 16 * c, dk[i][c]);
            st_out(ov + tx + 16 * c, dv[i][c]);
        }
    }
}

template <typename K>
cudaError_t allow_smem(K* kernel, int bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

template <typename T, int D>
cudaError_t fwd(const SwaArgs& a, cudaStream_t st) {
    const int smem = (3 * kT * (D + 4) + kT * kPS) * 4;
    cudaError_t e = allow_smem(swa_fwd_kernel<T, D>, smem);
    if (e != cudaSuccess) return e;
    swa_fwd_kernel<T, D><<<dim3((a.T + kT - 1) / kT, a.B * a.Hq), kThreads, smem, st>>>(a);
    return cudaGetLastError();
}

template <typename T, int D>
cudaError_t bwd(const SwaBackwardArgs& a, const float* delta, cudaStream_t st) {
    const int sq = (4 * kT * (D + 4) + kT * kPS + 2 * kT) * 4, sk = sq + kT * kPS * 4;
    cudaError_t e = allow_smem(swa_dq_kernel<T, D>, sq);
    if (e == cudaSuccess) e = allow_smem(swa_dkv_kernel<T, D>, sk);
    if (e != cudaSuccess) return e;
    swa_dq_kernel<T, D><<<dim3((a.f.T + kT - 1) / kT, a.f.B * a.f.Hq), kThreads, sq, st>>>(a, delta);
    swa_dkv_kernel<T, D><<<dim3((a.f.S + kT - 1) / kT, a.f.B * a.f.Hkv), kThreads, sk, st>>>(a, delta);
    return cudaGetLastError();
}

template <typename T>
cudaError_t fwd_d(const SwaArgs& a, cudaStream_t st) {
    switch (a.d) {
        case 16: return fwd<T, 16>(a, st);
        case 32: return fwd<T, 32>(a, st);
        case 64: return fwd<T, 64>(a, st);
        default: return fwd<T, 128>(a, st);
    }
}

template <typename T>
cudaError_t bwd_d(const SwaBackwardArgs& a, const float* delta, cudaStream_t st) {
    switch (a.f.d) {
        case 16: return bwd<T, 16>(a, delta, st);
        case 32: return bwd<T, 32>(a, delta, st);
        case 64: return bwd<T, 64>(a, delta, st);
        default: return bwd<T, 128>(a, delta, st);
    }
}

}  // namespace

cudaError_t swa_delta(const SwaArgs& a, const void* dout, float* delta, cudaStream_t st) {
    const size_t rows = (size_t)a.B * a.Hq * a.T;
    const unsigned grid = (unsigned)((rows + 7) / 8);
    if (a.dtype == MESA_F32)
        swa_delta_kernel<float><<<grid, 256, 0, st>>>((const float*)a.out, (const float*)dout, rows, a.d, delta);
    else
        swa_delta_kernel<__nv_bfloat16><<<grid, 256, 0, st>>>((const __nv_bfloat16*)a.out, (const __nv_bfloat16*)dout,
                                                              rows, a.d, delta);
    return cudaGetLastError();
}

cudaError_t swa_forward_simt(const SwaArgs& a, cudaStream_t st) {
    LaunchTimer lt(kKindSwa, st);
    return a.dtype == MESA_F32 ? fwd_d<float>(a, st) : fwd_d<__nv_bfloat16>(a, st);
}

cudaError_t swa_backward_simt(const SwaBackwardArgs& a, cudaStream_t st) {
    LaunchTimer lt(kKindSwaBwd, st);
    float* delta = static_cast<float*>(a.workspace);
    cudaError_t e = swa_delta(a.f, a.dout, delta, st);
    if (e != cudaSuccess) return e;
    return a.f.dtype == MESA_F32 ? bwd_d<float>(a, delta, st) : bwd_d<__nv_bfloat16>(a, delta, st);
}

}  // namespace mesa
