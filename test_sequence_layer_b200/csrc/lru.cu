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

// ---- element access: VEC channels of a row as one load; closed(): -inf ----
template <typename T, int VEC> struct Row;
template <> struct Row<float, 1> {
    using Raw = float;
    static __device__ __forceinline__ Raw load(const void* p, size_t i) { return static_cast<const float*>(p)[i]; }
    static __device__ __forceinline__ Raw zero() { return 0.f; }
    static __device__ __forceinline__ Raw closed() { return __int_as_float(0xff800000); }
    static __device__ __forceinline__ void unpack(Raw r, float (&f)[1]) { f[0] = r; }
    static __device__ __forceinline__ void store(void* p, size_t i, const float (&f)[1]) { static_cast<float*>(p)[i] = f[0]; }
};
template <> struct Row<__nv_bfloat16, 1> {
    using Raw = uint32_t;
    static __device__ __forceinline__ Raw load(const void* p, size_t i) { return static_cast<const unsigned short*>(p)[i]; }
    static __device__ __forceinline__ Raw zero() { return 0u; }
    static __device__ __forceinline__ Raw closed() { return 0xff80u; }
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
    static __device__ __forceinline__ Raw closed() { return 0xff80ff80u; }
    static __device__ __forceinline__ void unpack(Raw r, float (&f)[2]) {
        f[0] = __uint_as_float(r << 16);
        f[1] = __uint_as_float(r & 0xffff0000u);
    }
    static __device__ __forceinline__ void store(void* p, size_t i, const float (&f)[2]) {
        *reinterpret_cast<__nv_bfloat162*>(static_cast<__nv_bfloat16*>(p) + i) = __floats2bfloat162_rn(f[0], f[1]);
    }
};

// ---- arithmetic on VEC channels: packed fp32 pairs where there are two ----
__device__ __forceinline__ float ex2(float v) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(v));
    return y;
}
__device__ __forceinline__ float rcp(float v) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(v));
    return y;
}
__device__ __forceinline__ float rsq(float v) {
    float y;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(v));
    return y;
}
__device__ __forceinline__ float min_nan(float a, float b) {             // NaN if either is
    float y;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

template <int VEC> struct V;
template <> struct V<1> {
    float v[1];
    __device__ __forceinline__ static V all(float x) { return {{x}}; }
    __device__ __forceinline__ static V fma(V a, V b, V c) { return {{fmaf(a.v[0], b.v[0], c.v[0])}}; }
    __device__ __forceinline__ static V mul(V a, V b) { return {{a.v[0] * b.v[0]}}; }
    __device__ __forceinline__ static V add(V a, V b) { return {{a.v[0] + b.v[0]}}; }
};
template <> struct V<2> {
    float v[2];
    __device__ __forceinline__ static V all(float x) { return {{x, x}}; }
    using U = unsigned long long;
    static __device__ __forceinline__ U pack(V a) {
        U u;
        asm("mov.b64 %0, {%1, %2};" : "=l"(u) : "f"(a.v[0]), "f"(a.v[1]));
        return u;
    }
    static __device__ __forceinline__ V unpack(U u) {
        V a;
        asm("mov.b64 {%0, %1}, %2;" : "=f"(a.v[0]), "=f"(a.v[1]) : "l"(u));
        return a;
    }
    __device__ __forceinline__ static V fma(V a, V b, V c) {
        U d;
        asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(pack(a)), "l"(pack(b)), "l"(pack(c)));
        return unpack(d);
    }
    __device__ __forceinline__ static V mul(V a, V b) {
        U d;
        asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(pack(a)), "l"(pack(b)));
        return unpack(d);
    }
    __device__ __forceinline__ static V add(V a, V b) {
        U d;
        asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(pack(a)), "l"(pack(b)));
        return unpack(d);
    }
};
template <int VEC, float (*F)(float)> __device__ __forceinline__ V<VEC> each(V<VEC> a) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) a.v[e] = F(a.v[e]);
    return a;
}

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kTiny = 1e-36f;      // a normal number: keeps rsqrt finite where 1 - a^2 = 0

// 1 - e^(2 la) from la2 = la log2 e <= 0 and a: below t = -2 la = 1/4 by the
// series of 1 - e^-t (first term left out: t^6 / 5040 relative, 5e-8), above
// it without cancellation from a.
template <int VEC> __device__ __forceinline__ V<VEC> one_minus_a2(V<VEC> la2, V<VEC> a) {
    using W = V<VEC>;
    const W t = W::mul(la2, W::all(-2.f * kLn2));
    W p = W::fma(t, W::all(-1.f / 720.f), W::all(1.f / 120.f));
    p = W::fma(p, t, W::all(-1.f / 24.f));
    p = W::fma(p, t, W::all(1.f / 6.f));
    p = W::fma(p, t, W::all(-0.5f));
    p = W::fma(p, t, W::all(1.f));
    p = W::mul(p, t);
    const W q = W::fma(W::mul(a, W::all(-1.f)), a, W::all(1.f));
#pragma unroll
    for (int e = 0; e < VEC; ++e) p.v[e] = t.v[e] < 0.25f ? p.v[e] : q.v[e];
    return p;
}

// 1 + e^-v
template <int VEC> __device__ __forceinline__ V<VEC> one_plus_exp(V<VEC> v) {
    return V<VEC>::add(each<VEC, ex2>(V<VEC>::mul(v, V<VEC>::all(-kLog2e))), V<VEC>::all(1.f));
}

// a and b = sqrt(1 - a^2) i x of a token, with five special-function
// operations: i m = m^2 / sqrt(m^2 (1 + e^-gx)^2) needs one where a division
// and a root need two. i below 2^-63 counts as 2^-63, so the square stays
// finite.
template <int VEC>
__device__ __forceinline__ void gates(V<VEC> x, V<VEC> ga, V<VEC> gx, V<VEC> k2, V<VEC>& a, V<VEC>& b) {
    using W = V<VEC>;
    const W la2 = W::mul(k2, each<VEC, rcp>(one_plus_exp<VEC>(ga)));
    a = each<VEC, ex2>(la2);
    const W m2 = one_minus_a2<VEC>(la2, a);
    W z = W::mul(gx, W::all(-kLog2e));
#pragma unroll
    for (int e = 0; e < VEC; ++e) z.v[e] = min_nan(z.v[e], 63.f);
    const W w = W::add(each<VEC, ex2>(z), W::all(1.f));
    const W s = W::fma(W::mul(m2, w), w, W::all(kTiny));
    b = W::mul(W::mul(x, m2), each<VEC, rsq>(s));
}

// ---- forward ----
constexpr int kFwdSeg = 16;                     // tokens per warp and tile
constexpr int kFwdTile = kWarps * kFwdSeg;      // 128
static_assert(kFwdTile == 2 * kLruSave, "a forward tile saves two states");

template <typename T, int VEC>
__global__ void __launch_bounds__(kThreads, 2) lru_forward_kernel(LruArgs p, int groups, int ncta) {
    using R = Row<T, VEC>;
    using W = V<VEC>;
    __shared__ float2 seg[2][kWarps][VEC][32];
    __shared__ float2 peer[2][kLruMaxCluster][VEC][32];
    const int rank = ncta > 1 ? blockIdx.x % ncta : 0;
    const unsigned work = blockIdx.x / ncta;
    const int b = work / groups;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c0 = (work % groups) * (32 * VEC) + lane * VEC;
    const bool live = c0 < p.D;                 // VEC divides D
    const size_t base = (size_t)b * p.T * p.D + c0;
    const int tiles = (p.T + kFwdTile - 1) / kFwdTile;
    const int rounds = (tiles + ncta - 1) / ncta;

    W k2, carry;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        k2.v[e] = live ? -kC * kLog2e * softplus(p.lambda[c0 + e]) : 0.f;
        carry.v[e] = live && p.h0 ? p.h0[(size_t)b * p.D + c0 + e] : 0.f;
    }
    typename R::Raw rx[kFwdSeg], ra[kFwdSeg], rg[kFwdSeg];
    // tokens past the end get a closed gate: a = 1 and b = 0 exactly
    auto fetch = [&](int tile) {
        const long long t0 = (long long)tile * kFwdTile + warp * kFwdSeg;
        const size_t o = base + (size_t)t0 * p.D;
        const T* x = static_cast<const T*>(p.x) + o;
        const T* ga = static_cast<const T*>(p.ga) + o;
        const T* gx = static_cast<const T*>(p.gx) + o;
        if (live && t0 + kFwdSeg <= p.T) {
#pragma unroll
            for (int s = 0; s < kFwdSeg; ++s) {
                rx[s] = R::load(x, (size_t)s * p.D);
                ra[s] = R::load(ga, (size_t)s * p.D);
                rg[s] = R::load(gx, (size_t)s * p.D);
            }
        } else {
#pragma unroll
            for (int s = 0; s < kFwdSeg; ++s) {
                const bool in = live && t0 + s < p.T;
                rx[s] = in ? R::load(x, (size_t)s * p.D) : R::zero();
                ra[s] = in ? R::load(ga, (size_t)s * p.D) : R::closed();
                rg[s] = in ? R::load(gx, (size_t)s * p.D) : R::zero();
            }
        }
    };
    fetch(rank);
    for (int j = 0; j < rounds; ++j) {
        const int tile = j * ncta + rank, par = j & 1;
        const long long t0 = (long long)tile * kFwdTile + warp * kFwdSeg;
        W a[kFwdSeg], h[kFwdSeg], A = W::all(1.f), Hl = W::all(0.f);
#pragma unroll
        for (int s = 0; s < kFwdSeg; ++s) {
            W x, ga, gx;
            R::unpack(rx[s], x.v);
            R::unpack(ra[s], ga.v);
            R::unpack(rg[s], gx.v);
            gates<VEC>(x, ga, gx, k2, a[s], h[s]);
            Hl = W::fma(a[s], Hl, h[s]);
            A = W::mul(A, a[s]);
        }
        if (j + 1 < rounds) fetch(tile + ncta);
#pragma unroll
        for (int e = 0; e < VEC; ++e) seg[par][warp][e][lane] = make_float2(A.v[e], Hl.v[e]);
        __syncthreads();
        if (ncta > 1) {
            cg::cluster_group cl = cg::this_cluster();
            // this tile's map goes to every CTA of the cluster, one warp each
            if (warp < ncta) {
                float2 m[VEC];
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    m[e] = make_float2(1.f, 0.f);
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) {
                        const float2 g = seg[par][w][e][lane];
                        m[e].y = fmaf(g.x, m[e].y, g.y);
                        m[e].x *= g.x;
                    }
                }
                for (int r = warp; r < ncta; r += kWarps) {
                    float2* dst = cl.map_shared_rank(&peer[par][rank][0][0], r);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) dst[e * 32 + lane] = m[e];
                }
            }
            cl.sync();
        }
        W hv;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            float c = carry.v[e];
            hv.v[e] = c;
            if (ncta > 1) {
                for (int r = 0; r < ncta; ++r) {
                    if (r == rank) hv.v[e] = c;
                    const float2 m = peer[par][r][e][lane];
                    c = fmaf(m.x, c, m.y);
                }
                carry.v[e] = c;
                for (int w = 0; w < warp; ++w) {
                    const float2 m = seg[par][w][e][lane];
                    hv.v[e] = fmaf(m.x, hv.v[e], m.y);
                }
            } else {
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    if (w == warp) hv.v[e] = c;
                    const float2 m = seg[par][w][e][lane];
                    c = fmaf(m.x, c, m.y);
                }
                carry.v[e] = c;
            }
        }
        if (p.saved && live && (warp * kFwdSeg) % kLruSave == 0 && t0 < p.T) {
            const size_t row = (size_t)b * ((p.T + kLruSave - 1) / kLruSave) + t0 / kLruSave;
#pragma unroll
            for (int e = 0; e < VEC; ++e) p.saved[row * p.D + c0 + e] = hv.v[e];
        }
        if (p.y && live) {
            T* y = static_cast<T*>(p.y) + base + (size_t)t0 * p.D;
            if (t0 + kFwdSeg <= p.T) {
#pragma unroll
                for (int s = 0; s < kFwdSeg; ++s) {
                    hv = W::fma(a[s], hv, h[s]);
                    R::store(y, (size_t)s * p.D, hv.v);
                }
            } else {
#pragma unroll
                for (int s = 0; s < kFwdSeg; ++s) {
                    hv = W::fma(a[s], hv, h[s]);
                    if (t0 + s < p.T) R::store(y, (size_t)s * p.D, hv.v);
                }
            }
        }
    }
    if (p.hT && live && rank == 0 && warp == 0) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) p.hT[(size_t)b * p.D + c0 + e] = carry.v[e];
    }
}

// ---- backward ----
// g_t = dy_t + c_t with c_{t-1} = a_t g_t: the same map per run, composed from
// the end. The states h_{t-1} are rescanned inside the tile from the saved
// state before it, so the tiles only pass c on. s = dL/dlog a * log a feeds
// both dgate_a = s (1 - r) and dlambda. Registers bound the tile: a, r, i and
// g of a run are kept, b and sqrt(1 - a^2) are formed again in the last pass.
constexpr int kBwdSeg = 8;
constexpr int kBwdTile = kWarps * kBwdSeg;
static_assert(kBwdTile == kLruSave, "a backward tile starts at a saved state");

template <typename T, int VEC>
__global__ void __launch_bounds__(kThreads, 2) lru_backward_kernel(LruBackwardArgs q, int groups, int ncta) {
    using R = Row<T, VEC>;
    using W = V<VEC>;
    const LruArgs& p = q.f;
    __shared__ float2 segh[2][kWarps][VEC][32];               // A, Hl of a run
    __shared__ float segc[2][kWarps][VEC][32];                // Cl of a run
    __shared__ float2 peer[2][kLruMaxCluster][VEC][32];
    __shared__ float red[kWarps][VEC][32];
    const int rank = ncta > 1 ? blockIdx.x % ncta : 0;
    const unsigned work = blockIdx.x / ncta;
    const int b = work / groups;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c0 = (work % groups) * (32 * VEC) + lane * VEC;
    const bool live = c0 < p.D;
    const size_t base = (size_t)b * p.T * p.D + c0;
    const int tiles = (p.T + kBwdTile - 1) / kBwdTile;
    const int rounds = (tiles + ncta - 1) / ncta;

    W k2, carry, acc = W::all(0.f);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        k2.v[e] = live ? -kC * kLog2e * softplus(p.lambda[c0 + e]) : 0.f;
        carry.v[e] = live && q.dhT ? q.dhT[(size_t)b * p.D + c0 + e] : 0.f;
    }
    typename R::Raw rx[kBwdSeg], ra[kBwdSeg], rg[kBwdSeg], rd[kBwdSeg];
    W hs;
    // tile numbers run down from the last; tiles below 0 (a cluster's last
    // round) are empty: closed gates and no gradient
    auto fetch = [&](int tile) {
        const long long t0 = (long long)tile * kBwdTile + warp * kBwdSeg;
#pragma unroll
        for (int s = 0; s < kBwdSeg; ++s) {
            const bool in = live && tile >= 0 && t0 + s < p.T;
            const size_t o = base + (size_t)(t0 + s) * p.D;
            rx[s] = in ? R::load(p.x, o) : R::zero();
            ra[s] = in ? R::load(p.ga, o) : R::closed();
            rg[s] = in ? R::load(p.gx, o) : R::zero();
            rd[s] = in ? R::load(q.dy, o) : R::zero();
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            hs.v[e] = live && tile >= 0 ? p.saved[((size_t)b * tiles + tile) * p.D + c0 + e] : 0.f;
    };
    fetch(tiles - 1 - rank);
    for (int j = 0; j < rounds; ++j) {
        const int tile = tiles - 1 - (j * ncta + rank), par = j & 1;
        const long long t0 = (long long)tile * kBwdTile + warp * kBwdSeg;
        W a[kBwdSeg], r[kBwdSeg], iv[kBwdSeg], g[kBwdSeg];
        typename R::Raw xk[kBwdSeg];
        W A = W::all(1.f), Hl = W::all(0.f), Cl = W::all(0.f), hv = hs;
#pragma unroll
        for (int s = 0; s < kBwdSeg; ++s) {
            W x, ga, gx;
            xk[s] = rx[s];
            R::unpack(rx[s], x.v);
            R::unpack(ra[s], ga.v);
            R::unpack(rg[s], gx.v);
            R::unpack(rd[s], g[s].v);
            r[s] = each<VEC, rcp>(one_plus_exp<VEC>(ga));
            iv[s] = each<VEC, rcp>(one_plus_exp<VEC>(gx));
            const W la2 = W::mul(k2, r[s]);
            a[s] = each<VEC, ex2>(la2);
            const W m2 = one_minus_a2<VEC>(la2, a[s]);
            const W m = W::mul(m2, each<VEC, rsq>(W::add(m2, W::all(kTiny))));
            Hl = W::fma(a[s], Hl, W::mul(W::mul(m, iv[s]), x));
            A = W::mul(A, a[s]);
        }
#pragma unroll
        for (int s = kBwdSeg - 1; s >= 0; --s) Cl = W::mul(a[s], W::add(g[s], Cl));
        if (j + 1 < rounds) fetch(tile - ncta);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            segh[par][warp][e][lane] = make_float2(A.v[e], Hl.v[e]);
            segc[par][warp][e][lane] = Cl.v[e];
        }
        __syncthreads();
        if (ncta > 1) {
            cg::cluster_group cl = cg::this_cluster();
            if (warp < ncta) {
                float2 m[VEC];
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    m[e] = make_float2(1.f, 0.f);
#pragma unroll
                    for (int w = kWarps - 1; w >= 0; --w) {
                        const float A1 = segh[par][w][e][lane].x;
                        m[e].y = fmaf(A1, m[e].y, segc[par][w][e][lane]);
                        m[e].x *= A1;
                    }
                }
                for (int t = warp; t < ncta; t += kWarps) {
                    float2* dst = cl.map_shared_rank(&peer[par][rank][0][0], t);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) dst[e * 32 + lane] = m[e];
                }
            }
            cl.sync();
        }
        W gc;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            float c = carry.v[e];
            if (ncta > 1) {
                float mine = c;
                for (int t = 0; t < ncta; ++t) {
                    if (t == rank) mine = c;
                    const float2 m = peer[par][t][e][lane];
                    c = fmaf(m.x, c, m.y);
                }
                carry.v[e] = c;
                c = mine;
                for (int w = kWarps - 1; w > warp; --w) c = fmaf(segh[par][w][e][lane].x, c, segc[par][w][e][lane]);
                gc.v[e] = c;
            } else {
                gc.v[e] = c;
#pragma unroll
                for (int w = kWarps - 1; w >= 0; --w) {
                    if (w == warp) gc.v[e] = c;
                    c = fmaf(segh[par][w][e][lane].x, c, segc[par][w][e][lane]);
                }
                carry.v[e] = c;
            }
            for (int w = 0; w < warp; ++w) {
                const float2 m = segh[par][w][e][lane];
                hv.v[e] = fmaf(m.x, hv.v[e], m.y);
            }
        }
#pragma unroll
        for (int s = kBwdSeg - 1; s >= 0; --s) {
            g[s] = W::add(g[s], gc);
            gc = W::mul(a[s], g[s]);
        }
        W part = W::all(0.f);
        const bool tail = !live || tile < 0 || t0 + kBwdSeg > p.T;
#pragma unroll
        for (int s = 0; s < kBwdSeg; ++s) {
            W x;
            R::unpack(xk[s], x.v);
            const W la2 = W::mul(k2, r[s]), la = W::mul(la2, W::all(kLn2));
            const W m2 = one_minus_a2<VEC>(la2, a[s]);
            const W im = each<VEC, rsq>(W::add(m2, W::all(kTiny)));           // 1 / m
            const W mi = W::mul(W::mul(m2, im), iv[s]);
            const W bb = W::mul(mi, x), dx = W::mul(g[s], mi);
            // log a (a h_{t-1} - b a^2 / m^2); log a / m^2 tends to -1/2 as log a -> 0
            const W ala = W::mul(a[s], la), ba = W::mul(bb, a[s]);
            const W second = W::mul(W::mul(W::mul(ba, im), im), ala);
            const W sv = W::mul(g[s], W::fma(ala, hv, W::mul(second, W::all(-1.f))));
            const W dga = W::fma(W::mul(sv, W::all(-1.f)), r[s], sv);
            const W gb = W::mul(g[s], bb);
            const W dgx = W::fma(W::mul(gb, W::all(-1.f)), iv[s], gb);
            part = W::add(part, sv);
            hv = W::fma(a[s], hv, bb);
            if (!tail || (live && tile >= 0 && t0 + s < p.T)) {
                const size_t o = base + (size_t)(t0 + s) * p.D;
                R::store(q.dx, o, dx.v);
                R::store(q.dga, o, dga.v);
                R::store(q.dgx, o, dgx.v);
            }
        }
        acc = W::add(acc, part);
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) red[warp][e][lane] = acc.v[e];
    __syncthreads();
    if (warp == 0 && live) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) s += red[w][e][lane];
            q.partial[((size_t)b * ncta + rank) * p.D + c0 + e] = s;
            if (q.dh0 && rank == 0) q.dh0[(size_t)b * p.D + c0 + e] = carry.v[e];
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
    V<VEC> xv, av, gv, k2, a, h;
    R::unpack(R::load(x, i), xv.v);
    R::unpack(R::load(ga, i), av.v);
    R::unpack(R::load(gx, i), gv.v);
#pragma unroll
    for (int e = 0; e < VEC; ++e) k2.v[e] = -kC * kLog2e * softplus(lambda[c + e]);
    gates<VEC>(xv, av, gv, k2, a, h);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        h.v[e] = fmaf(a.v[e], h_in[i + e], h.v[e]);
        h_out[i + e] = h.v[e];
    }
    R::store(y, i, h.v);
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
