// lru.cu -- gated linear recurrence (mesa_lru_*): forward, backward, decode step.
//
//   r = sigmoid(ga), i = sigmoid(gx), la = -8 softplus(lambda) r, a = e^la,
//   h_t = a_t h_{t-1} + sqrt(1 - a_t^2) i_t x_t
//
// A CTA owns 32 VEC channels of one sequence (a lane holds VEC of them, so a
// warp reads whole 64- or 128-byte rows) and walks time in tiles. Inside a
// tile each warp takes a run of tokens: it forms a and b of its run once, in
// registers, reduces them to the run's map h -> A h + Hl, and after one
// barrier every thread composes the maps of the runs before its own and
// rescans its registers. Nothing is read or computed twice. The next tile's
// rows are loaded into registers before the barrier, which keeps 48 (forward)
// or 32 (backward) 128-byte rows per warp in flight.
// Where channels alone do not fill the GPU, a cluster of 2 to 8 CTAs shares a
// sequence: CTA r takes tiles r, r + n, ..., and per round the CTAs exchange
// their tiles' maps through distributed shared memory.
#include <cooperative_groups.h>

#include "mesa_common.cuh"
#include "mesa_internal.h"
#include "mixers_internal.h"

namespace cg = cooperative_groups;

namespace mesa {
namespace {

constexpr float kC = 8.f;
constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;

__device__ __forceinline__ float softplus(float v) { return log1pf(expf(-fabsf(v))) + fmaxf(v, 0.f); }

// ---- element access: VEC channels of a row as one load ----
template <typename T, int VEC> struct Row;
template <> struct Row<float, 1> {
    using Raw = float;
    static __device__ __forceinline__ Raw load(const void* p, size_t i) { return static_cast<const float*>(p)[i]; }
    static __device__ __forceinline__ Raw zero() { return 0.f; }
    static __device__ __forceinline__ void unpack(Raw r, float (&f)[1]) { f[0] = r; }
    static __device__ __forceinline__ void store(void* p, size_t i, const float (&f)[1]) { static_cast<float*>(p)[i] = f[0]; }
};
template <> struct Row<__nv_bfloat16, 1> {
    using Raw = uint32_t;
    static __device__ __forceinline__ Raw load(const void* p, size_t i) { return static_cast<const unsigned short*>(p)[i]; }
    static __device__ __forceinline__ Raw zero() { return 0u; }
    static __device__ __forceinline__ void unpack(Raw r, float (&f)[1]) { f[0] = __uint_as_float(r << 16); }
    static __device__ __forceinline__ void store(void* p, size_t i, const float (&f)[1]) {
        static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(f[0]);
    }
};
template <> struct Row<__nv_bfloat16, 2> {
    using Raw = uint32_t;
    static __device__ __forceinline__ Raw load(const void* p, size_t i) {
        return *reinterpret_cast<const uint32_t*>(static_cast<const unsigned short*>(p) + i);
    }
    static __device__ __forceinline__ Raw zero() { return 0u; }
    static __device__ __forceinline__ void unpack(Raw r, float (&f)[2]) {
        f[0] = __uint_as_float(r << 16);
        f[1] = __uint_as_float(r & 0xffff0000u);
    }
    static __device__ __forceinline__ void store(void* p, size_t i, const float (&f)[2]) {
        *reinterpret_cast<__nv_bfloat162*>(static_cast<__nv_bfloat16*>(p) + i) = __floats2bfloat162_rn(f[0], f[1]);
    }
};

__device__ __forceinline__ float sqrt_fast(float v) {
    float y;
    asm("sqrt.approx.f32 %0, %1;" : "=f"(y) : "f"(v));
    return y;
}

__device__ __forceinline__ float sigmoid(float v) { return __fdividef(1.f, 1.f + __expf(-v)); }

// 1 - e^(2 la), la <= 0: below t = -2 la = 1/4 by the series of 1 - e^-t
// (first term left out: t^6 / 5040 relative, 5e-8), above it without
// cancellation from a.
__device__ __forceinline__ float one_minus_a2(float la, float a) {
    const float t = -2.f * la;
    float p = -1.f / 720.f;
    p = fmaf(p, t, 1.f / 120.f);
    p = fmaf(p, t, -1.f / 24.f);
    p = fmaf(p, t, 1.f / 6.f);
    p = fmaf(p, t, -0.5f);
    p = fmaf(p, t, 1.f) * t;
    return t < 0.25f ? p : fmaf(-a, a, 1.f);
}

// ---- forward ----
constexpr int kFwdSeg = 16;                     // tokens per warp and tile
constexpr int kFwdTile = kWarps * kFwdSeg;      // 128
static_assert(kFwdTile == 2 * kLruSave, "a forward tile saves two states");

template <typename T, int VEC>
__global__ void __launch_bounds__(kThreads, 2) lru_forward_kernel(LruArgs p, int groups, int ncta) {
    using R = Row<T, VEC>;
    __shared__ float2 seg[2][kWarps][32 * VEC];
    __shared__ float2 peer[2][kLruMaxCluster][32 * VEC];
    const int rank = ncta > 1 ? blockIdx.x % ncta : 0;
    const unsigned work = blockIdx.x / ncta;
    const int b = work / groups;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c0 = (work % groups) * (32 * VEC) + lane * VEC;
    const bool live = c0 < p.D;                 // VEC divides D
    const size_t base = (size_t)b * p.T * p.D + c0;
    const int tiles = (p.T + kFwdTile - 1) / kFwdTile;
    const int rounds = (tiles + ncta - 1) / ncta;

    float k8[VEC], carry[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        k8[e] = live ? -kC * softplus(p.lambda[c0 + e]) : 0.f;
        carry[e] = live && p.h0 ? p.h0[(size_t)b * p.D + c0 + e] : 0.f;
    }
    typename R::Raw rx[kFwdSeg], ra[kFwdSeg], rg[kFwdSeg];
    auto fetch = [&](int tile) {
        const long long t0 = (long long)tile * kFwdTile + warp * kFwdSeg;
#pragma unroll
        for (int s = 0; s < kFwdSeg; ++s) {
            const bool in = live && t0 + s < p.T;
            const size_t o = base + (size_t)(t0 + s) * p.D;
            rx[s] = in ? R::load(p.x, o) : R::zero();
            ra[s] = in ? R::load(p.ga, o) : R::zero();
            rg[s] = in ? R::load(p.gx, o) : R::zero();
        }
    };
    fetch(rank);
    for (int j = 0; j < rounds; ++j) {
        const int tile = j * ncta + rank, par = j & 1;
        const long long t0 = (long long)tile * kFwdTile + warp * kFwdSeg;
        float a[kFwdSeg][VEC], h[kFwdSeg][VEC], A[VEC], Hl[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) A[e] = 1.f, Hl[e] = 0.f;
#pragma unroll
        for (int s = 0; s < kFwdSeg; ++s) {
            float x[VEC], ga[VEC], gx[VEC];
            R::unpack(rx[s], x);
            R::unpack(ra[s], ga);
            R::unpack(rg[s], gx);
            const bool in = t0 + s < p.T;
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float la = k8[e] * sigmoid(ga[e]);
                const float av = __expf(la);
                const float bv = sqrt_fast(one_minus_a2(la, av)) * (sigmoid(gx[e]) * x[e]);
                a[s][e] = in ? av : 1.f;        // tokens past the end change nothing
                h[s][e] = in ? bv : 0.f;
                Hl[e] = fmaf(a[s][e], Hl[e], h[s][e]);
                A[e] *= a[s][e];
            }
        }
        if (j + 1 < rounds) fetch(tile + ncta);
#pragma unroll
        for (int e = 0; e < VEC; ++e) seg[par][warp][lane * VEC + e] = make_float2(A[e], Hl[e]);
        __syncthreads();
        if (ncta > 1) {
            cg::cluster_group cl = cg::this_cluster();
            // warp w hands this tile's map to CTA w of the cluster
            if (warp < ncta) {
                float2* dst = cl.map_shared_rank(&peer[par][rank][0], warp);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    float TA = 1.f, TH = 0.f;
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) {
                        const float2 m = seg[par][w][lane * VEC + e];
                        TH = fmaf(m.x, TH, m.y);
                        TA *= m.x;
                    }
                    dst[lane * VEC + e] = make_float2(TA, TH);
                }
            }
            cl.sync();
        }
        float hv[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            if (ncta > 1) {
                float c = carry[e];
                hv[e] = c;
                for (int r = 0; r < ncta; ++r) {
                    if (r == rank) hv[e] = c;
                    const float2 m = peer[par][r][lane * VEC + e];
                    c = fmaf(m.x, c, m.y);
                }
                carry[e] = c;
                for (int w = 0; w < warp; ++w) {
                    const float2 m = seg[par][w][lane * VEC + e];
                    hv[e] = fmaf(m.x, hv[e], m.y);
                }
            } else {
                float c = carry[e];
                hv[e] = c;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    if (w == warp) hv[e] = c;
                    const float2 m = seg[par][w][lane * VEC + e];
                    c = fmaf(m.x, c, m.y);
                }
                carry[e] = c;
            }
        }
        if (p.saved && live && (warp * kFwdSeg) % kLruSave == 0 && t0 < p.T) {
            const size_t row = (size_t)b * ((p.T + kLruSave - 1) / kLruSave) + t0 / kLruSave;
#pragma unroll
            for (int e = 0; e < VEC; ++e) p.saved[row * p.D + c0 + e] = hv[e];
        }
        if (p.y && live) {
#pragma unroll
            for (int s = 0; s < kFwdSeg; ++s) {
#pragma unroll
                for (int e = 0; e < VEC; ++e) hv[e] = fmaf(a[s][e], hv[e], h[s][e]);
                if (t0 + s < p.T) R::store(p.y, base + (size_t)(t0 + s) * p.D, hv);
            }
        }
    }
    if (p.hT && live && rank == 0 && warp == 0) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) p.hT[(size_t)b * p.D + c0 + e] = carry[e];
    }
}

// ---- backward ----
// g_t = dy_t + c_t with c_{t-1} = a_t g_t: the same map per run, composed from
// the end. The states h_{t-1} are rescanned inside the tile from the saved
// state before it, so the tiles only pass c on. s = dL/dlog a * log a feeds
// both dgate_a = s (1 - r) and dlambda.
constexpr int kBwdSeg = 8;
constexpr int kBwdTile = kWarps * kBwdSeg;
static_assert(kBwdTile == kLruSave, "a backward tile starts at a saved state");

template <typename T, int VEC>
__global__ void __launch_bounds__(kThreads, 2) lru_backward_kernel(LruBackwardArgs q, int groups, int ncta) {
    using R = Row<T, VEC>;
    const LruArgs& p = q.f;
    __shared__ float4 seg[2][kWarps][32 * VEC];               // A, Hl, Cl of a run
    __shared__ float2 peer[2][kLruMaxCluster][32 * VEC];
    __shared__ float red[kWarps][32 * VEC];
    const int rank = ncta > 1 ? blockIdx.x % ncta : 0;
    const unsigned work = blockIdx.x / ncta;
    const int b = work / groups;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c0 = (work % groups) * (32 * VEC) + lane * VEC;
    const bool live = c0 < p.D;
    const size_t base = (size_t)b * p.T * p.D + c0;
    const int tiles = (p.T + kBwdTile - 1) / kBwdTile;
    const int rounds = (tiles + ncta - 1) / ncta;

    float k8[VEC], carry[VEC], acc[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        k8[e] = live ? -kC * softplus(p.lambda[c0 + e]) : 0.f;
        carry[e] = live && q.dhT ? q.dhT[(size_t)b * p.D + c0 + e] : 0.f;
        acc[e] = 0.f;
    }
    typename R::Raw rx[kBwdSeg], ra[kBwdSeg], rg[kBwdSeg], rd[kBwdSeg];
    float hs[VEC];
    // tile numbers run down from the last; tiles below 0 (a cluster's last
    // round) are empty
    auto fetch = [&](int tile) {
        const long long t0 = (long long)tile * kBwdTile + warp * kBwdSeg;
#pragma unroll
        for (int s = 0; s < kBwdSeg; ++s) {
            const bool in = live && tile >= 0 && t0 + s < p.T;
            const size_t o = base + (size_t)(t0 + s) * p.D;
            rx[s] = in ? R::load(p.x, o) : R::zero();
            ra[s] = in ? R::load(p.ga, o) : R::zero();
            rg[s] = in ? R::load(p.gx, o) : R::zero();
            rd[s] = in ? R::load(q.dy, o) : R::zero();
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            hs[e] = live && tile >= 0 ? p.saved[((size_t)b * tiles + tile) * p.D + c0 + e] : 0.f;
    };
    fetch(tiles - 1 - rank);
    for (int j = 0; j < rounds; ++j) {
        const int tile = tiles - 1 - (j * ncta + rank), par = j & 1;
        const long long t0 = (long long)tile * kBwdTile + warp * kBwdSeg;
        float a[kBwdSeg][VEC], bb[kBwdSeg][VEC], r[kBwdSeg][VEC], iv[kBwdSeg][VEC], dy[kBwdSeg][VEC];
        float A[VEC], Hl[VEC], Cl[VEC], hv[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) A[e] = 1.f, Hl[e] = 0.f, Cl[e] = 0.f, hv[e] = hs[e];
#pragma unroll
        for (int s = 0; s < kBwdSeg; ++s) {
            float x[VEC], ga[VEC], gx[VEC];
            R::unpack(rx[s], x);
            R::unpack(ra[s], ga);
            R::unpack(rg[s], gx);
            R::unpack(rd[s], dy[s]);
            const bool in = tile >= 0 && t0 + s < p.T;
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                r[s][e] = sigmoid(ga[e]);
                iv[s][e] = sigmoid(gx[e]);
                const float la = k8[e] * r[s][e];
                const float av = __expf(la);
                const float bv = sqrt_fast(one_minus_a2(la, av)) * (iv[s][e] * x[e]);
                a[s][e] = in ? av : 1.f;
                bb[s][e] = in ? bv : 0.f;
                Hl[e] = fmaf(a[s][e], Hl[e], bb[s][e]);
                A[e] *= a[s][e];
            }
        }
#pragma unroll
        for (int s = kBwdSeg - 1; s >= 0; --s)
#pragma unroll
            for (int e = 0; e < VEC; ++e) Cl[e] = a[s][e] * (dy[s][e] + Cl[e]);
        if (j + 1 < rounds) fetch(tile - ncta);
#pragma unroll
        for (int e = 0; e < VEC; ++e) seg[par][warp][lane * VEC + e] = make_float4(A[e], Hl[e], Cl[e], 0.f);
        __syncthreads();
        if (ncta > 1) {
            cg::cluster_group cl = cg::this_cluster();
            if (warp < ncta) {
                float2* dst = cl.map_shared_rank(&peer[par][rank][0], warp);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    float TA = 1.f, TC = 0.f;
#pragma unroll
                    for (int w = kWarps - 1; w >= 0; --w) {
                        const float4 m = seg[par][w][lane * VEC + e];
                        TC = fmaf(m.x, TC, m.z);
                        TA *= m.x;
                    }
                    dst[lane * VEC + e] = make_float2(TA, TC);
                }
            }
            cl.sync();
        }
        float g[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            float c = carry[e];
            g[e] = c;
            if (ncta > 1) {
                for (int t = 0; t < ncta; ++t) {
                    if (t == rank) g[e] = c;
                    const float2 m = peer[par][t][lane * VEC + e];
                    c = fmaf(m.x, c, m.y);
                }
                carry[e] = c;
                c = g[e];
            }
#pragma unroll
            for (int w = kWarps - 1; w >= 0; --w) {
                if (w == warp) g[e] = c;
                const float4 m = seg[par][w][lane * VEC + e];
                c = fmaf(m.x, c, m.z);
            }
            if (ncta == 1) carry[e] = c;
            for (int w = 0; w < warp; ++w) {
                const float4 m = seg[par][w][lane * VEC + e];
                hv[e] = fmaf(m.x, hv[e], m.y);
            }
        }
        float hp[kBwdSeg][VEC], part[VEC];
#pragma unroll
        for (int s = 0; s < kBwdSeg; ++s)
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                hp[s][e] = hv[e];
                hv[e] = fmaf(a[s][e], hv[e], bb[s][e]);
            }
#pragma unroll
        for (int e = 0; e < VEC; ++e) part[e] = 0.f;
#pragma unroll
        for (int s = kBwdSeg - 1; s >= 0; --s) {
            float dx[VEC], dga[VEC], dgx[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float gv = dy[s][e] + g[e];
                const float la = k8[e] * r[s][e];
                const float m2 = one_minus_a2(la, a[s][e]);
                const float m = sqrt_fast(m2);
                // log a / m^2 tends to -1/2 as log a -> 0
                const float lm = m2 > 1e-30f ? __fdividef(la, m2) : -0.5f;
                const float sv = gv * (a[s][e] * (hp[s][e] * la - bb[s][e] * a[s][e] * lm));
                dx[e] = gv * m * iv[s][e];
                dgx[e] = gv * bb[s][e] * (1.f - iv[s][e]);
                dga[e] = sv * (1.f - r[s][e]);
                part[e] += (tile >= 0 && t0 + s < p.T) ? sv : 0.f;
                g[e] = a[s][e] * gv;
            }
            if (live && tile >= 0 && t0 + s < p.T) {
                const size_t o = base + (size_t)(t0 + s) * p.D;
                R::store(q.dx, o, dx);
                R::store(q.dga, o, dga);
                R::store(q.dgx, o, dgx);
            }
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e) acc[e] += part[e];
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) red[warp][lane * VEC + e] = acc[e];
    __syncthreads();
    if (warp == 0 && live) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) s += red[w][lane * VEC + e];
            q.partial[((size_t)b * ncta + rank) * p.D + c0 + e] = s;
            if (q.dh0 && rank == 0) q.dh0[(size_t)b * p.D + c0 + e] = carry[e];
        }
    }
}

// dlambda = sigmoid(lambda) / softplus(lambda) * sum over rows of partial
__global__ void lru_dlambda_kernel(const float* __restrict__ partial, size_t rows, int D, const float* lambda,
                                   float* dlambda) {
    __shared__ float red[8][32];
    const int c = blockIdx.x * 32 + threadIdx.x;
    float s = 0.f;
    if (c < D)
        for (size_t r = threadIdx.y; r < rows; r += 8) s += partial[r * D + c];
    red[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0 && c < D) {
#pragma unroll
        for (int w = 1; w < 8; ++w) s += red[w][threadIdx.x];
        const float l = lambda[c];              // sigmoid / softplus tends to 1 (within e^l / 2) as l falls
        dlambda[c] = l > -20.f ? s / (softplus(l) * (1.f + expf(-l))) : s;
    }
}

// ---- decode ----
template <typename T, int VEC>
__global__ void lru_step_kernel(const void* x, const void* ga, const void* gx, const float* __restrict__ lambda,
                                size_t n, int D, const float* h_in, float* h_out, void* y) {
    using R = Row<T, VEC>;
    const size_t i = ((size_t)blockIdx.x * blockDim.x + threadIdx.x) * VEC;
    if (i >= n) return;
    const int c = (int)(i % D);
    float xv[VEC], av[VEC], gv[VEC], h[VEC];
    R::unpack(R::load(x, i), xv);
    R::unpack(R::load(ga, i), av);
    R::unpack(R::load(gx, i), gv);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        const float la = -kC * softplus(lambda[c + e]) * sigmoid(av[e]);
        const float a = __expf(la);
        h[e] = fmaf(a, h_in[i + e], sqrt_fast(one_minus_a2(la, a)) * (sigmoid(gv[e]) * xv[e]));
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) h_out[i + e] = h[e];
    R::store(y, i, h);
}

bool pair_ok(int D, std::initializer_list<const void*> ps) {
    if (D % 2) return false;
    for (const void* q : ps)
        if (reinterpret_cast<uintptr_t>(q) % 4) return false;
    return true;
}

// CTAs per sequence and channel group: doubled while the grid is below two
// CTAs per SM and every CTA still gets a tile.
int cluster_size(long long blocks, int tiles) {
    int n = 1;
    while (n < kLruMaxCluster && blocks * n < 2 * 148 && tiles >= 2 * n) n *= 2;
    return n;
}

template <typename F, typename... A>
cudaError_t launch_cluster(F* kernel, unsigned grid, int ncta, cudaStream_t st, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = ncta;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = ncta > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

struct Plan {
    int groups, ncta;
    unsigned grid;
};
Plan plan(int B, int T, int D, int vec, int tile) {
    Plan pl;
    pl.groups = (D + 32 * vec - 1) / (32 * vec);
    const long long blocks = (long long)B * pl.groups;
    pl.ncta = cluster_size(blocks, (T + tile - 1) / tile);
    pl.grid = (unsigned)(blocks * pl.ncta);
    return pl;
}

}  // namespace

size_t lru_backward_rows(int B, int T) {
    const int t = (T + kBwdTile - 1) / kBwdTile;          // a CTA of a cluster has a tile
    return (size_t)B * (t < 1 ? 1 : t < kLruMaxCluster ? t : kLruMaxCluster);
}

cudaError_t lru_forward(const LruArgs& a, cudaStream_t st) {
    LaunchTimer lt(kKindLru, st);
    const bool pair = a.dtype == MESA_BF16 && pair_ok(a.D, {a.x, a.ga, a.gx, a.y});
    const Plan pl = plan(a.B, a.T, a.D, pair ? 2 : 1, kFwdTile);
    if (a.dtype == MESA_F32) return launch_cluster(lru_forward_kernel<float, 1>, pl.grid, pl.ncta, st, a, pl.groups, pl.ncta);
    if (pair) return launch_cluster(lru_forward_kernel<__nv_bfloat16, 2>, pl.grid, pl.ncta, st, a, pl.groups, pl.ncta);
    return launch_cluster(lru_forward_kernel<__nv_bfloat16, 1>, pl.grid, pl.ncta, st, a, pl.groups, pl.ncta);
}

cudaError_t lru_backward(const LruBackwardArgs& q, cudaStream_t st) {
    const LruArgs& a = q.f;
    const bool pair = a.dtype == MESA_BF16 && pair_ok(a.D, {a.x, a.ga, a.gx, q.dy, q.dx, q.dga, q.dgx});
    const Plan pl = plan(a.B, a.T, a.D, pair ? 2 : 1, kBwdTile);
    cudaError_t e;
    {
        LaunchTimer lt(kKindLruBwd, st);
        if (a.dtype == MESA_F32)
            e = launch_cluster(lru_backward_kernel<float, 1>, pl.grid, pl.ncta, st, q, pl.groups, pl.ncta);
        else if (pair)
            e = launch_cluster(lru_backward_kernel<__nv_bfloat16, 2>, pl.grid, pl.ncta, st, q, pl.groups, pl.ncta);
        else
            e = launch_cluster(lru_backward_kernel<__nv_bfloat16, 1>, pl.grid, pl.ncta, st, q, pl.groups, pl.ncta);
    }
    if (e != cudaSuccess) return e;
    LaunchTimer lt(kKindLruBwd, st);
    lru_dlambda_kernel<<<(a.D + 31) / 32, dim3(32, 8), 0, st>>>(q.partial, (size_t)a.B * pl.ncta, a.D, a.lambda,
                                                               q.dlambda);
    return cudaGetLastError();
}

cudaError_t lru_step(const void* x, const void* ga, const void* gx, const float* lambda, int B, int D,
                     mesa_dtype dtype, const float* h_in, float* h_out, void* y, cudaStream_t st) {
    LaunchTimer lt(kKindLru, st);
    const size_t n = (size_t)B * D;
    const bool pair = dtype == MESA_BF16 && pair_ok(D, {x, ga, gx, y});
    const size_t threads = pair ? n / 2 : n;
    const unsigned grid = (unsigned)((threads + 127) / 128);
    if (dtype == MESA_F32)
        lru_step_kernel<float, 1><<<grid, 128, 0, st>>>(x, ga, gx, lambda, n, D, h_in, h_out, y);
    else if (pair)
        lru_step_kernel<__nv_bfloat16, 2><<<grid, 128, 0, st>>>(x, ga, gx, lambda, n, D, h_in, h_out, y);
    else
        lru_step_kernel<__nv_bfloat16, 1><<<grid, 128, 0, st>>>(x, ga, gx, lambda, n, D, h_in, h_out, y);
    return cudaGetLastError();
}

}  // namespace mesa
