// lru.cu -- gated linear recurrence (mesa_lru_*): forward, backward, decode step.
//
//   r = sigmoid(ga), i = sigmoid(gx), la = -8 softplus(lambda) r, a = e^la,
//   h_t = a_t h_{t-1} + sqrt(1 - a_t^2) i_t x_t
//
// A CTA owns 32 VEC channels of one sequence (a lane holds VEC of them) and
// walks time in tiles of 64 tokens. Inside a tile each of eight warps takes a
// run of eight tokens: it forms a and b of its run, reduces them to the run's
// map h -> A h + Hl, and after one barrier every thread composes the maps of
// the runs before its own and rescans its registers. Each row is read once.
// Tiles arrive in shared memory two ahead (one thread issues tensor copies;
// widths a tensor copy cannot take use 4-byte asynchronous copies, odd bf16
// widths plain loads), so registers are left for the run.
// A cluster of up to 16 CTAs shares a sequence: CTA r takes tiles r, r + n,
// ..., and per round every CTA sends its tile's map to the others with
// asynchronous remote stores that count on the receiver's mbarrier, so no CTA
// waits for more than the maps themselves.
#include "swa_tc.cuh"

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
using swa::ex2;
using swa::kLog2e;
constexpr float kLn2 = 0.6931471805599453f;
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

// ---- tiles and the maps between them ----
constexpr int kSeg = 8;                         // tokens per warp and tile
constexpr int kTile = kWarps * kSeg;
static_assert(kTile == kLruSave, "a tile starts at a saved state");

enum Load { kTensor, kAsync4, kPlain };

// NT input tensors of a CTA's channels, two tiles ahead in shared memory.
// Words of 4 bytes, [stage][tensor][token][lane]: a lane's VEC channels.
template <typename T, int VEC, int NT, int LOAD> struct Stager {
    using R = Row<T, VEC>;
    static constexpr int kStageBytes = NT * kTile * 32 * 4;
    static constexpr int kBytes = LOAD == kPlain ? 0 : 2 * kStageBytes;
    const CUtensorMap* maps[NT];
    const T* src[NT];                           // the CTA's sequence, at this lane's channels
    uint32_t* buf;
    uint64_t* full;                             // [2]
    int T_, D, c_cta, b;
    bool live;

    // rounds up to 2 ahead; call by all threads, tile < 0 or past the end: nothing to load
    __device__ __forceinline__ void issue(int round, int tile, int tiles) {
        if (tile < 0 || tile >= tiles) return;
        const int st = round & 1, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        if (LOAD == kTensor) {
            if (threadIdx.x == 0) {
                tc::mbar_arrive_expect_tx(&full[st], kStageBytes);
#pragma unroll
                for (int i = 0; i < NT; ++i)
                    swa::tma_load(buf + (st * NT + i) * kTile * 32, maps[i], c_cta, tile * kTile, b, &full[st]);
            }
        } else if (LOAD == kAsync4) {
            const int t0 = tile * kTile + warp * kSeg;
#pragma unroll
            for (int s = 0; s < kSeg; ++s)
                if (live && t0 + s < T_) {
#pragma unroll
                    for (int i = 0; i < NT; ++i)
                        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(tc::smem_addr(
                                         buf + ((st * NT + i) * kTile + warp * kSeg + s) * 32 + lane)),
                                     "l"(src[i] + (size_t)(t0 + s) * D)
                                     : "memory");
                }
        }
        if (LOAD == kAsync4) asm volatile("cp.async.commit_group;" ::: "memory");
    }
    // the tile of this round has landed; `ahead`: one more tile is on its way
    __device__ __forceinline__ bool wait(int round, bool ahead) {
        if (LOAD == kTensor) return tc::mbar_wait(&full[round & 1], (round >> 1) & 1);
        if (LOAD == kAsync4) {
            if (ahead) asm volatile("cp.async.wait_group 1;" ::: "memory");
            else asm volatile("cp.async.wait_group 0;" ::: "memory");
        }
        return true;
    }
    __device__ __forceinline__ typename R::Raw get(int round, int i, int tile, int s) const {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        if (LOAD == kPlain) {
            const int t = tile * kTile + warp * kSeg + s;
            return live && t < T_ ? R::load(src[i], (size_t)t * D) : R::zero();
        }
        const uint32_t w = buf[(((round & 1) * NT + i) * kTile + warp * kSeg + s) * 32 + lane];
        return *reinterpret_cast<const typename R::Raw*>(&w);
    }
};

// maps x -> v.x * x + v.y per channel, exchanged between the CTAs of a cluster
template <int VEC> struct Exchange {
    float2* peer;                               // [2][ncta][VEC][32]
    uint64_t* bar;                              // [2]
    int ncta, rank;
    // by one warp: this CTA's map to every CTA of the cluster, itself included
    __device__ __forceinline__ void send(int round, const float2 (&m)[VEC]) {
        const int par = round & 1, lane = threadIdx.x & 31;
        if (lane == 0) tc::mbar_arrive_expect_tx(&bar[par], ncta * VEC * 32 * 8);
        __syncwarp();
        const uint32_t b0 = tc::smem_addr(&bar[par]);
        for (int r = 0; r < ncta; ++r) {
            uint32_t rb;
            asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(rb) : "r"(b0), "r"(r));
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                uint32_t ra;
                asm("mapa.shared::cluster.u32 %0, %1, %2;"
                    : "=r"(ra)
                    : "r"(tc::smem_addr(&peer[((par * ncta + rank) * VEC + e) * 32 + lane])), "r"(r));
                asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(ra),
                             "f"(m[e].x), "f"(m[e].y), "r"(rb)
                             : "memory");
            }
        }
    }
    __device__ __forceinline__ bool wait(int round) { return tc::mbar_wait(&bar[round & 1], (round >> 1) & 1); }
    __device__ __forceinline__ float2 get(int round, int r, int e) const {
        return peer[(((round & 1) * ncta + r) * VEC + e) * 32 + (threadIdx.x & 31)];
    }
};

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

struct Where {
    int rank, b, c0, c_cta, tiles, rounds;
    bool live;
    size_t base;
    template <int VEC> __device__ __forceinline__ static Where make(const LruArgs& p, int groups, int ncta) {
        Where w;
        w.rank = ncta > 1 ? blockIdx.x % ncta : 0;
        const unsigned work = blockIdx.x / ncta;
        w.b = work / groups;
        w.c_cta = (work % groups) * (32 * VEC);
        w.c0 = w.c_cta + (threadIdx.x & 31) * VEC;
        w.live = w.c0 < p.D;                    // VEC divides D
        w.base = (size_t)w.b * p.T * p.D + w.c0;
        w.tiles = (p.T + kTile - 1) / kTile;
        w.rounds = (w.tiles + ncta - 1) / ncta;
        return w;
    }
};

template <int VEC> __host__ __device__ constexpr int peer_bytes(int ncta) { return ncta > 1 ? 2 * ncta * VEC * 32 * 8 : 0; }

// ---- forward ----
template <typename T, int VEC, int LOAD>
__global__ void __launch_bounds__(kThreads, 3)
lru_forward_kernel(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap ma,
                   const __grid_constant__ CUtensorMap mg, LruArgs p, int groups, int ncta, unsigned* err) {
    using R = Row<T, VEC>;
    using W = V<VEC>;
    using St = Stager<T, VEC, 3, LOAD>;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float2 seg[2][kWarps][VEC][32];
    __shared__ uint64_t bars[4];
    const Where w = Where::make<VEC>(p, groups, ncta);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    St in{{&mx, &ma, &mg},
          {static_cast<const T*>(p.x) + w.base, static_cast<const T*>(p.ga) + w.base, static_cast<const T*>(p.gx) + w.base},
          reinterpret_cast<uint32_t*>(smem), bars, p.T, p.D, w.c_cta, w.b, w.live};
    Exchange<VEC> ex{reinterpret_cast<float2*>(smem + St::kBytes), bars + 2, ncta, w.rank};
    if (threadIdx.x == 0) {
        for (int i = 0; i < 4; ++i) tc::mbar_init(&bars[i], 1);
        tc::fence_mbar_init();
    }
    if (ncta > 1) cluster_sync(); else __syncthreads();
    bool ok = true;

    W k2, carry;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        k2.v[e] = w.live ? -kC * kLog2e * softplus(p.lambda[w.c0 + e]) : 0.f;
        carry.v[e] = w.live && p.h0 ? p.h0[(size_t)w.b * p.D + w.c0 + e] : 0.f;
    }
    in.issue(0, w.rank, w.tiles);
    in.issue(1, w.rank + ncta, w.tiles);
    for (int j = 0; j < w.rounds; ++j) {
        const int tile = j * ncta + w.rank, par = j & 1;
        const int t0 = tile * kTile + warp * kSeg;
        const bool any = tile < w.tiles;
        W a[kSeg], h[kSeg], A = W::all(1.f), Hl = W::all(0.f);
        if (any && ok) ok = in.wait(j, tile + ncta < w.tiles);
#pragma unroll
        for (int s = 0; s < kSeg; ++s) {
            W x, ga, gx;
            R::unpack(in.get(j, 0, tile, s), x.v);
            R::unpack(in.get(j, 1, tile, s), ga.v);
            R::unpack(in.get(j, 2, tile, s), gx.v);
            gates<VEC>(x, ga, gx, k2, a[s], h[s]);
        }
        if (t0 + kSeg > p.T) {                   // tokens past the end change nothing
#pragma unroll
            for (int s = 0; s < kSeg; ++s)
                if (t0 + s >= p.T) a[s] = W::all(1.f), h[s] = W::all(0.f);
        }
#pragma unroll
        for (int s = 0; s < kSeg; ++s) {
            Hl = W::fma(a[s], Hl, h[s]);
            A = W::mul(A, a[s]);
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e) seg[par][warp][e][lane] = make_float2(A.v[e], Hl.v[e]);
        __syncthreads();
        in.issue(j, tile + 2 * ncta, w.tiles);   // every thread has read the stage
        W hv;
        if (ncta > 1) {
            if (warp == 0) {
                float2 m[VEC];
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    m[e] = make_float2(1.f, 0.f);
#pragma unroll
                    for (int u = 0; u < kWarps; ++u) {
                        const float2 g = seg[par][u][e][lane];
                        m[e].y = fmaf(g.x, m[e].y, g.y);
                        m[e].x *= g.x;
                    }
                }
                ex.send(j, m);
            }
            if (ok) ok = ex.wait(j);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                float c = carry.v[e];
                for (int r = 0; r < ncta; ++r) {
                    if (r == w.rank) hv.v[e] = c;
                    const float2 m = ex.get(j, r, e);
                    c = fmaf(m.x, c, m.y);
                }
                carry.v[e] = c;
                for (int u = 0; u < warp; ++u) {
                    const float2 m = seg[par][u][e][lane];
                    hv.v[e] = fmaf(m.x, hv.v[e], m.y);
                }
            }
        } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                float c = carry.v[e];
#pragma unroll
                for (int u = 0; u < kWarps; ++u) {
                    if (u == warp) hv.v[e] = c;
                    const float2 m = seg[par][u][e][lane];
                    c = fmaf(m.x, c, m.y);
                }
                carry.v[e] = c;
            }
        }
        if (p.saved && w.live && warp == 0 && any) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) p.saved[((size_t)w.b * w.tiles + tile) * p.D + w.c0 + e] = hv.v[e];
        }
        if (p.y && w.live) {
            T* y = static_cast<T*>(p.y) + w.base + (size_t)t0 * p.D;
            if (t0 + kSeg <= p.T) {
#pragma unroll
                for (int s = 0; s < kSeg; ++s) {
                    hv = W::fma(a[s], hv, h[s]);
                    R::store(y, (size_t)s * p.D, hv.v);
                }
            } else {
#pragma unroll
                for (int s = 0; s < kSeg; ++s) {
                    hv = W::fma(a[s], hv, h[s]);
                    if (t0 + s < p.T) R::store(y, (size_t)s * p.D, hv.v);
                }
            }
        }
    }
    if (p.hT && w.live && w.rank == 0 && warp == 0) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) p.hT[(size_t)w.b * p.D + w.c0 + e] = carry.v[e];
    }
    if (!ok) record_error(err, kErrTimeout);
}

// ---- backward ----
// g_t = dy_t + c_t with c_{t-1} = a_t g_t: the same map per run, composed from
// the end. The states h_{t-1} are rescanned inside the tile from the saved
// state before it, so the tiles only pass c on. s = dL/dlog a * log a feeds
// both dgate_a = s (1 - r) and dlambda. Registers bound the tile: a, r, i and
// g of a run are kept, b and sqrt(1 - a^2) are formed again in the last pass.
template <typename T, int VEC, int LOAD>
__global__ void __launch_bounds__(kThreads, 2)
lru_backward_kernel(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap ma,
                    const __grid_constant__ CUtensorMap mg, const __grid_constant__ CUtensorMap md, LruBackwardArgs q,
                    int groups, int ncta, unsigned* err) {
    using R = Row<T, VEC>;
    using W = V<VEC>;
    using St = Stager<T, VEC, 4, LOAD>;
    const LruArgs& p = q.f;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float2 segh[2][kWarps][VEC][32];               // A, Hl of a run
    __shared__ float segc[2][kWarps][VEC][32];                // Cl of a run
    __shared__ float red[kWarps][VEC][32];
    __shared__ uint64_t bars[4];
    const Where w = Where::make<VEC>(p, groups, ncta);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    St in{{&mx, &ma, &mg, &md},
          {static_cast<const T*>(p.x) + w.base, static_cast<const T*>(p.ga) + w.base, static_cast<const T*>(p.gx) + w.base,
           static_cast<const T*>(q.dy) + w.base},
          reinterpret_cast<uint32_t*>(smem), bars, p.T, p.D, w.c_cta, w.b, w.live};
    Exchange<VEC> ex{reinterpret_cast<float2*>(smem + St::kBytes), bars + 2, ncta, w.rank};
    if (threadIdx.x == 0) {
        for (int i = 0; i < 4; ++i) tc::mbar_init(&bars[i], 1);
        tc::fence_mbar_init();
    }
    if (ncta > 1) cluster_sync(); else __syncthreads();
    bool ok = true;

    W k2, carry, acc = W::all(0.f);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        k2.v[e] = w.live ? -kC * kLog2e * softplus(p.lambda[w.c0 + e]) : 0.f;
        carry.v[e] = w.live && q.dhT ? q.dhT[(size_t)w.b * p.D + w.c0 + e] : 0.f;
    }
    // tile numbers run down from the last; tiles below 0 (a cluster's last
    // round) are empty: closed gates and no gradient
    const int top = w.tiles - 1 - w.rank;
    auto state = [&](int tile) {
        W s;
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            s.v[e] = w.live && tile >= 0 ? p.saved[((size_t)w.b * w.tiles + tile) * p.D + w.c0 + e] : 0.f;
        return s;
    };
    in.issue(0, top, w.tiles);
    in.issue(1, top - ncta, w.tiles);
    W hs = state(top);
    for (int j = 0; j < w.rounds; ++j) {
        const int tile = top - j * ncta, par = j & 1;
        const int t0 = tile * kTile + warp * kSeg;
        const bool any = tile >= 0;
        W a[kSeg], r[kSeg], iv[kSeg], g[kSeg];
        typename R::Raw xk[kSeg];
        W A = W::all(1.f), Hl = W::all(0.f), Cl = W::all(0.f), hv = hs;
        hs = state(tile - ncta);
        if (any && ok) ok = in.wait(j, tile - ncta >= 0);
        const bool tail = !any || t0 + kSeg > p.T;
#pragma unroll
        for (int s = 0; s < kSeg; ++s) {
            W x, ga, gx;
            xk[s] = in.get(j, 0, tile, s);
            typename R::Raw ra = in.get(j, 1, tile, s), rg = in.get(j, 2, tile, s), rd = in.get(j, 3, tile, s);
            if (tail && (!any || t0 + s >= p.T)) {
                xk[s] = rg = rd = R::zero();
                ra = R::closed();
            }
            R::unpack(xk[s], x.v);
            R::unpack(ra, ga.v);
            R::unpack(rg, gx.v);
            R::unpack(rd, g[s].v);
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
        for (int s = kSeg - 1; s >= 0; --s) Cl = W::mul(a[s], W::add(g[s], Cl));
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            segh[par][warp][e][lane] = make_float2(A.v[e], Hl.v[e]);
            segc[par][warp][e][lane] = Cl.v[e];
        }
        __syncthreads();
        in.issue(j, tile - 2 * ncta, w.tiles);
        W gc;
        if (ncta > 1) {
            if (warp == 0) {
                float2 m[VEC];
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    m[e] = make_float2(1.f, 0.f);
#pragma unroll
                    for (int u = kWarps - 1; u >= 0; --u) {
                        const float A1 = segh[par][u][e][lane].x;
                        m[e].y = fmaf(A1, m[e].y, segc[par][u][e][lane]);
                        m[e].x *= A1;
                    }
                }
                ex.send(j, m);
            }
            if (ok) ok = ex.wait(j);
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            float c = carry.v[e];
            if (ncta > 1) {
                float mine = c;
                for (int t = 0; t < ncta; ++t) {
                    if (t == w.rank) mine = c;
                    const float2 m = ex.get(j, t, e);
                    c = fmaf(m.x, c, m.y);
                }
                carry.v[e] = c;
                c = mine;
                for (int u = kWarps - 1; u > warp; --u) c = fmaf(segh[par][u][e][lane].x, c, segc[par][u][e][lane]);
                gc.v[e] = c;
            } else {
#pragma unroll
                for (int u = kWarps - 1; u >= 0; --u) {
                    if (u == warp) gc.v[e] = c;
                    c = fmaf(segh[par][u][e][lane].x, c, segc[par][u][e][lane]);
                }
                carry.v[e] = c;
            }
            for (int u = 0; u < warp; ++u) {
                const float2 m = segh[par][u][e][lane];
                hv.v[e] = fmaf(m.x, hv.v[e], m.y);
            }
        }
#pragma unroll
        for (int s = kSeg - 1; s >= 0; --s) {
            g[s] = W::add(g[s], gc);
            gc = W::mul(a[s], g[s]);
        }
        W part = W::all(0.f);
        const size_t o0 = w.base + (size_t)t0 * p.D;
        T* pdx = static_cast<T*>(q.dx) + o0;
        T* pda = static_cast<T*>(q.dga) + o0;
        T* pdg = static_cast<T*>(q.dgx) + o0;
#pragma unroll
        for (int s = 0; s < kSeg; ++s) {
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
            if (w.live && (!tail || (any && t0 + s < p.T))) {
                R::store(pdx, (size_t)s * p.D, dx.v);
                R::store(pda, (size_t)s * p.D, dga.v);
                R::store(pdg, (size_t)s * p.D, dgx.v);
            }
        }
        acc = W::add(acc, part);
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) red[warp][e][lane] = acc.v[e];
    __syncthreads();
    if (warp == 0 && w.live) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            float s = 0.f;
#pragma unroll
            for (int u = 0; u < kWarps; ++u) s += red[u][e][lane];
            q.partial[((size_t)w.b * ncta + w.rank) * p.D + w.c0 + e] = s;
            if (q.dh0 && w.rank == 0) q.dh0[(size_t)w.b * p.D + w.c0 + e] = carry.v[e];
        }
    }
    if (!ok) record_error(err, kErrTimeout);
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

bool all_aligned(std::initializer_list<const void*> ps, uintptr_t n) {
    for (const void* q : ps)
        if (reinterpret_cast<uintptr_t>(q) % n) return false;
    return true;
}
bool pair_ok(int D, std::initializer_list<const void*> ps) { return D % 2 == 0 && all_aligned(ps, 4); }

// [B][T][D] as a 3-D map of tiles of 64 tokens by 128 bytes of channels
bool channel_map(CUtensorMap* m, const LruArgs& a, const void* base) {
    const bool f32 = a.dtype == MESA_F32;
    return swa::encode_map(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, f32 ? 4 : 2, base,
                           a.D, a.T, a.B, f32 ? 32 : 64, kTile, CU_TENSOR_MAP_SWIZZLE_NONE);
}

// CTAs per sequence and channel group. Eight where every CTA still walks four
// tiles: many short CTAs leave the SMs evenly loaded. Sixteen if the grid
// would otherwise not give every SM two.
int cluster_size(long long blocks, int tiles) {
    int n = 1;
    while (n < 8 && tiles >= 8 * n && blocks * n < 16 * 148) n *= 2;
    while (n < kLruMaxCluster && tiles >= 2 * n && blocks * n < 2 * 148) n *= 2;
    return n;
}

template <typename F, typename... A>
cudaError_t launch_cluster(F* kernel, unsigned grid, int ncta, int smem, cudaStream_t st, A... args) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess && ncta > 8) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
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
Plan plan(int B, int T, int D, int vec) {
    Plan pl;
    pl.groups = (D + 32 * vec - 1) / (32 * vec);
    const long long blocks = (long long)B * pl.groups;
    pl.ncta = cluster_size(blocks, (T + kTile - 1) / kTile);
    pl.grid = (unsigned)(blocks * pl.ncta);
    return pl;
}

template <typename T, int VEC, int LOAD>
cudaError_t forward(const LruArgs& a, const CUtensorMap (&m)[4], unsigned* err, cudaStream_t st) {
    const Plan pl = plan(a.B, a.T, a.D, VEC);
    return launch_cluster(lru_forward_kernel<T, VEC, LOAD>, pl.grid, pl.ncta,
                          Stager<T, VEC, 3, LOAD>::kBytes + peer_bytes<VEC>(pl.ncta), st, m[0], m[1], m[2], a, pl.groups,
                          pl.ncta, err);
}

template <typename T, int VEC, int LOAD>
cudaError_t backward(const LruBackwardArgs& q, const CUtensorMap (&m)[4], unsigned* err, cudaStream_t st) {
    const LruArgs& a = q.f;
    const Plan pl = plan(a.B, a.T, a.D, VEC);
    cudaError_t e = launch_cluster(lru_backward_kernel<T, VEC, LOAD>, pl.grid, pl.ncta,
                                   Stager<T, VEC, 4, LOAD>::kBytes + peer_bytes<VEC>(pl.ncta), st, m[0], m[1], m[2], m[3],
                                   q, pl.groups, pl.ncta, err);
    if (e != cudaSuccess) return e;
    lru_dlambda_kernel<<<(a.D + 31) / 32, dim3(32, 8), 0, st>>>(q.partial, (size_t)a.B * pl.ncta, a.D, a.lambda,
                                                               q.dlambda);
    return cudaGetLastError();
}

// whether tensor copies can take these rows: 16-byte bases and row lengths
bool tensor_ok(const LruArgs& a, std::initializer_list<const void*> ps) {
    return (size_t)a.D * (a.dtype == MESA_F32 ? 4 : 2) % 16 == 0 && all_aligned(ps, 16);
}

}  // namespace

size_t lru_backward_rows(int B, int T) {
    const int t = (T + kTile - 1) / kTile;                // a CTA of a cluster has a tile
    return (size_t)B * (t < 1 ? 1 : t < kLruMaxCluster ? t : kLruMaxCluster);
}

cudaError_t lru_forward(const LruArgs& a, cudaStream_t st) {
    LaunchTimer lt(kKindLru, st);
    unsigned* err = error_word_ptr();
    if (!err) return cudaErrorUnknown;
    CUtensorMap m[4] = {};
    using bf = __nv_bfloat16;
    if (tensor_ok(a, {a.x, a.ga, a.gx}) && all_aligned({a.y}, 4)) {
        if (!channel_map(&m[0], a, a.x) || !channel_map(&m[1], a, a.ga) || !channel_map(&m[2], a, a.gx))
            return cudaErrorInvalidValue;
        return a.dtype == MESA_F32 ? forward<float, 1, kTensor>(a, m, err, st) : forward<bf, 2, kTensor>(a, m, err, st);
    }
    if (a.dtype == MESA_F32) return forward<float, 1, kAsync4>(a, m, err, st);
    return pair_ok(a.D, {a.x, a.ga, a.gx, a.y}) ? forward<bf, 2, kAsync4>(a, m, err, st)
                                                : forward<bf, 1, kPlain>(a, m, err, st);
}

cudaError_t lru_backward(const LruBackwardArgs& q, cudaStream_t st) {
    LaunchTimer lt(kKindLruBwd, st);
    const LruArgs& a = q.f;
    unsigned* err = error_word_ptr();
    if (!err) return cudaErrorUnknown;
    CUtensorMap m[4] = {};
    using bf = __nv_bfloat16;
    if (tensor_ok(a, {a.x, a.ga, a.gx, q.dy}) && all_aligned({q.dx, q.dga, q.dgx}, 4)) {
        if (!channel_map(&m[0], a, a.x) || !channel_map(&m[1], a, a.ga) || !channel_map(&m[2], a, a.gx) ||
            !channel_map(&m[3], a, q.dy))
            return cudaErrorInvalidValue;
        return a.dtype == MESA_F32 ? backward<float, 1, kTensor>(q, m, err, st) : backward<bf, 2, kTensor>(q, m, err, st);
    }
    if (a.dtype == MESA_F32) return backward<float, 1, kAsync4>(q, m, err, st);
    return pair_ok(a.D, {a.x, a.ga, a.gx, q.dy, q.dx, q.dga, q.dgx}) ? backward<bf, 2, kAsync4>(q, m, err, st)
                                                                     : backward<bf, 1, kPlain>(q, m, err, st);
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
