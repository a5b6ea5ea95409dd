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
    constexpr int kPer = 16 / (int)sizeof(T);             // elements of a 16-byte piece
#pragma unroll 4
    for (int i = threadIdx.x; i < kT * D / kPer; i += kThreads) {
        const int r = i / (D / kPer), c = i % (D / kPer) * kPer;
        float* d = s + r * (D + 4) + c;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (r0 + r < rows) v = *reinterpret_cast<const uint4*>(g + (size_t)(r0 + r) * D + c);
        if (sizeof(T) == 4) {
            *reinterpret_cast<uint4*>(d) = v;
        } else {
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 8; e += 4)
                *reinterpret_cast<float4*>(d + e) =
                    make_float4(__uint_as_float(w[e / 2] << 16), __uint_as_float(w[e / 2] & 0xffff0000u),
                                __uint_as_float(w[e / 2 + 1] << 16), __uint_as_float(w[e / 2 + 1] & 0xffff0000u));
        }
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
    if (TRANS) {
#pragma unroll 4
        for (int k = 0; k < kT; ++k) {
            const float4 v = *reinterpret_cast<const float4*>(W + k * kPS + 4 * ty);
            const float w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
                const float b = B[k * (D + 4) + tx + 16 * c];
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[i][c] = fmaf(w[i], b, acc[i][c]);
            }
        }
    } else {
#pragma unroll 2
        for (int k = 0; k < kT; k += 4) {
            float w[4][4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                *reinterpret_cast<float4*>(w[i]) = *reinterpret_cast<const float4*>(W + (4 * ty + i) * kPS + k);
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int c = 0; c < D / 16; ++c) {
                    const float b = B[(k + u) * (D + 4) + tx + 16 * c];
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[i][c] = fmaf(w[i][u], b, acc[i][c]);
                }
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

// the same from the weights, for rows of few keys
__global__ void swa_delta_few_kernel(SwaArgs a, const __nv_bfloat16* __restrict__ dout, size_t rows, float* delta) {
    using bf = __nv_bfloat16;
    const size_t r = (size_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (r >= rows) return;
    const size_t head = r / a.T;
    const size_t kv = head / (a.Hq / a.Hkv) * a.S * a.d;
    const swa::FewKeys keys(a.S - a.T + (int)(r % a.T), a.window, a.sinks);
    const float lse = a.lse[r];
    float s = 0.f;
    for (int i = 0; i < keys.n; ++i) {
        const size_t j = kv + (size_t)keys.key(i) * a.d;
        float qk = 0.f, dv = 0.f;
        for (int c = threadIdx.x & 31; c < a.d; c += 32) {
            qk = fmaf(ld_in(static_cast<const bf*>(a.q), r * a.d + c), ld_in(static_cast<const bf*>(a.k), j + c), qk);
            dv = fmaf(ld_in(dout, r * a.d + c), ld_in(static_cast<const bf*>(a.v), j + c), dv);
        }
#pragma unroll
        for (int x = 16; x; x >>= 1) {
            qk += __shfl_xor_sync(~0u, qk, x);
            dv += __shfl_xor_sync(~0u, dv, x);
        }
        s = fmaf(expf(qk * a.scale - lse), dv, s);
    }
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

// How the queries of a key tile are shared out: the tiles that hold a sink, seen
// by every later query, in chunks of about a window; where key tiles alone do
// not fill the GPU, each query head of a group apart. A tile of one part writes
// its gradients; the others leave fp32 parts, added in order afterwards.
struct DkvPlan {
    int sink_tiles, chunks, chunk_len, heads;             // heads: parts of a group (1 or G)
    __host__ __device__ int parts_of(int tile) const { return (tile < sink_tiles ? chunks : 1) * heads; }
    __host__ __device__ int items(int tiles) const { return (sink_tiles * chunks + tiles - sink_tiles) * heads; }
};

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) swa_dkv_kernel(SwaBackwardArgs a, const float* delta, DkvPlan pl, float* parts) {
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
    const int item = blockIdx.x / pl.heads, hpart = blockIdx.x % pl.heads;
    const int sink_items = pl.sink_tiles * pl.chunks;
    const int tile = item < sink_items ? item / pl.chunks : item - sink_items + pl.sink_tiles;
    const int chunk = item < sink_items ? item % pl.chunks : 0;
    const int j0 = tile * kT, off = p.S - p.T;
    const size_t kv = ((size_t)b * p.Hkv + hk) * p.S * D;
    load_tile<T, D>(sK, static_cast<const T*>(p.k) + kv, j0, p.S);
    load_tile<T, D>(sV, static_cast<const T*>(p.v) + kv, j0, p.S);
    int ta, tb;
    swa::query_range(j0, min(j0 + kT, p.S) - 1, p.T, p.S, p.window, p.sinks, ta, tb);
    ta = ta / kT * kT;
    if (tile < pl.sink_tiles) {
        ta = max(ta, chunk * pl.chunk_len);
        tb = min(tb, (chunk + 1) * pl.chunk_len);
    }
    const int g0 = pl.heads > 1 ? hpart : 0, g1 = pl.heads > 1 ? hpart + 1 : G;
    float dk[4][D / 16] = {}, dv[4][D / 16] = {};
    for (int g = g0; g < g1; ++g) {
        const size_t row = ((size_t)b * p.Hq + hk * G + g) * p.T;
        for (int t0 = ta; t0 < tb; t0 += kT) {
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
    const bool whole = pl.parts_of(tile) == 1;
    // this part's place: [2][64][D]
    float* part = parts + ((size_t)blockIdx.y * gridDim.x + blockIdx.x) * 2 * kT * D;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int j = j0 + 4 * ty + i;
        if (j >= p.S) continue;
        T* ok = static_cast<T*>(a.dk) + kv + (size_t)j * D;
        T* ov = static_cast<T*>(a.dv) + kv + (size_t)j * D;
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
            const int d = tx + 16 * c;
            if (whole) {
                st_out(ok + d, dk[i][c]);
                st_out(ov + d, dv[i][c]);
            } else {
                part[(4 * ty + i) * D + d] = dk[i][c];
                part[(kT + 4 * ty + i) * D + d] = dv[i][c];
            }
        }
    }
}

// one tile's parts, added in order: blocks (tile, sequence and head)
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) swa_dkv_sum_kernel(SwaBackwardArgs a, DkvPlan pl, const float* parts, int items) {
    const int tile = blockIdx.x, n = pl.parts_of(tile);
    if (n == 1) return;
    const int first = (tile < pl.sink_tiles ? tile * pl.chunks : pl.sink_tiles * pl.chunks + tile - pl.sink_tiles) * pl.heads;
    const float* p = parts + ((size_t)blockIdx.y * items + first) * 2 * kT * D;
    for (int i = threadIdx.x; i < 2 * kT * D; i += kThreads) {
        const int which = i / (kT * D), r = i % (kT * D), j = tile * kT + r / D;
        if (j >= a.f.S) continue;
        float s = 0.f;
#pragma unroll 4
        for (int k = 0; k < n; ++k) s += p[(size_t)k * 2 * kT * D + i];
        st_out(static_cast<T*>(which ? a.dv : a.dk) + ((size_t)blockIdx.y * a.f.S + j) * D + r % D, s);
    }
}

// `window` decides the chunks; with 1 the plan has the most parts
DkvPlan dkv_plan(int B, int Hq, int Hkv, int T, int S, int window, int sinks) {
    DkvPlan pl{0, 1, T > 0 ? T : 1, 1};
    const int tiles = (S + kT - 1) / kT;
    if ((long long)tiles * B * Hkv < 2 * 148) pl.heads = Hq / Hkv;
    const int sink_tiles = (sinks + kT - 1) / kT < tiles ? (sinks + kT - 1) / kT : tiles;
    if (sink_tiles == 0) return pl;
    constexpr int kMaxChunks = 32;
    long long len = ((long long)window + kT + kT - 1) / kT * kT;
    const long long least = (((long long)T + kMaxChunks - 1) / kMaxChunks + kT - 1) / kT * kT;
    if (len < least) len = least;
    if (len >= T) return pl;
    pl.sink_tiles = sink_tiles;
    pl.chunk_len = (int)len;
    pl.chunks = (int)((T + len - 1) / len);
    return pl;
}

size_t dkv_parts_bytes(const DkvPlan& pl, int B, int Hkv, int S, int d) {
    if (pl.heads == 1 && pl.sink_tiles == 0) return 0;
    return (size_t)B * Hkv * pl.items((S + kT - 1) / kT) * 2 * kT * d * 4;
}
size_t up256(size_t x) { return (x + 255) / 256 * 256; }

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
    const SwaArgs& f = a.f;
    const DkvPlan pl = dkv_plan(f.B, f.Hq, f.Hkv, f.T, f.S, f.window, f.sinks);
    const int tiles = (f.S + kT - 1) / kT, items = pl.items(tiles);
    float* parts = reinterpret_cast<float*>(static_cast<char*>(a.workspace) + up256((size_t)f.B * f.Hq * f.T * 4));
    swa_dkv_kernel<T, D><<<dim3(items, f.B * f.Hkv), kThreads, sk, st>>>(a, delta, pl, parts);
    if (dkv_parts_bytes(pl, f.B, f.Hkv, f.S, D))
        swa_dkv_sum_kernel<T, D><<<dim3(pl.heads > 1 ? tiles : pl.sink_tiles, f.B * f.Hkv), kThreads, 0, st>>>(a, pl, parts,
                                                                                                          items);
    swa_dq_kernel<T, D><<<dim3((f.T + kT - 1) / kT, f.B * f.Hq), kThreads, sq, st>>>(a, delta);
    return cudaGetLastError();
}

// bf16 of 64 and 128 columns never comes here: the tensor cores take it
cudaError_t fwd_any(const SwaArgs& a, cudaStream_t st) {
    using bf = __nv_bfloat16;
    if (a.dtype == MESA_BF16) return a.d == 16 ? fwd<bf, 16>(a, st) : fwd<bf, 32>(a, st);
    switch (a.d) {
        case 16: return fwd<float, 16>(a, st);
        case 32: return fwd<float, 32>(a, st);
        case 64: return fwd<float, 64>(a, st);
        default: return fwd<float, 128>(a, st);
    }
}

cudaError_t bwd_any(const SwaBackwardArgs& a, const float* delta, cudaStream_t st) {
    using bf = __nv_bfloat16;
    if (a.f.dtype == MESA_BF16) return a.f.d == 16 ? bwd<bf, 16>(a, delta, st) : bwd<bf, 32>(a, delta, st);
    switch (a.f.d) {
        case 16: return bwd<float, 16>(a, delta, st);
        case 32: return bwd<float, 32>(a, delta, st);
        case 64: return bwd<float, 64>(a, delta, st);
        default: return bwd<float, 128>(a, delta, st);
    }
}

}  // namespace

size_t swa_simt_workspace_bytes(int B, int Hq, int Hkv, int T, int S, int d, int sinks) {
    return up256((size_t)B * Hq * T * 4) + dkv_parts_bytes(dkv_plan(B, Hq, Hkv, T, S, 1, sinks), B, Hkv, S, d);
}

cudaError_t swa_delta(const SwaArgs& a, const void* dout, float* delta, cudaStream_t st) {
    const size_t rows = (size_t)a.B * a.Hq * a.T;
    const unsigned grid = (unsigned)((rows + 7) / 8);
    if (a.dtype == MESA_F32)
        swa_delta_kernel<float><<<grid, 256, 0, st>>>((const float*)a.out, (const float*)dout, rows, a.d, delta);
    else if (swa::few_keys(a.window, a.sinks, a.S))
        swa_delta_few_kernel<<<grid, 256, 0, st>>>(a, (const __nv_bfloat16*)dout, rows, delta);
    else
        swa_delta_kernel<__nv_bfloat16><<<grid, 256, 0, st>>>((const __nv_bfloat16*)a.out, (const __nv_bfloat16*)dout,
                                                              rows, a.d, delta);
    return cudaGetLastError();
}

cudaError_t swa_forward_simt(const SwaArgs& a, cudaStream_t st) {
    LaunchTimer lt(kKindSwa, st);
    return fwd_any(a, st);
}

cudaError_t swa_backward_simt(const SwaBackwardArgs& a, cudaStream_t st) {
    LaunchTimer lt(kKindSwaBwd, st);
    float* delta = static_cast<float*>(a.workspace);
    cudaError_t e = swa_delta(a.f, a.dout, delta, st);
    if (e != cudaSuccess) return e;
    return bwd_any(a, delta, st);
}

}  // namespace mesa
