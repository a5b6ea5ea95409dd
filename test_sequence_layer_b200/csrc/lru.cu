// lru.cu -- gated linear recurrence (mesa_lru_*): forward, backward, decode step.
//
//   r = sigmoid(ga), i = sigmoid(gx), la = -8 softplus(lambda) r, a = e^la,
//   h_t = a_t h_{t-1} + sqrt(1 - a_t^2) i_t x_t
//
// A CTA owns 32 VEC channels of one sequence (a lane holds VEC of them) and
// walks time in tiles. Inside a tile each warp takes a run of tokens: it forms
// a and b of its run in registers, reduces them to the run's map h -> A h + Hl,
// one warp composes the maps into the state before each run, and every warp
// rescans its registers from there. Each row is read once. (Every thread
// composing for itself cost as many instructions as the gates did.)
// Tiles arrive in shared memory ahead of their use (one thread issues tensor
// copies; widths a tensor copy cannot take use 4-byte asynchronous copies, odd
// bf16 widths plain loads), so registers are left for the run.
// Where channels do not fill the GPU a cluster of up to 16 CTAs shares a
// sequence: CTA r takes tiles r, r + n, ..., and per round every CTA sends its
// tile's map to the others with asynchronous remote stores that count on the
// receiver's mbarrier.
//
// What bounds it: special-function operations (four a token and channel in
// the forward) and memory come close to one another in bf16, the rest is the
// wait for a tile's slowest warp. Batch 8, 8192 tokens, width 2048, bf16:
// 238 us forward, 4.5 TB/s (no cluster; 267 us with clusters of two). The backward
// of 8 x 2048 x 2048 takes 142 us: 128 registers a thread, 16 warps per SM, and
// about 280 bytes a thread spilled in bf16.
#include "swa_tc.cuh"

namespace mesa {
namespace {

constexpr float kC = 8.f;

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
template <> struct alignas(4) V<1> {
    float v[1];
    __device__ __forceinline__ static V all(float x) { return {{x}}; }
    __device__ __forceinline__ static V fma(V a, V b, V c) { return {{fmaf(a.v[0], b.v[0], c.v[0])}}; }
    __device__ __forceinline__ static V mul(V a, V b) { return {{a.v[0] * b.v[0]}}; }
    __device__ __forceinline__ static V add(V a, V b) { return {{a.v[0] + b.v[0]}}; }
};
template <> struct alignas(8) V<2> {
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

// A channel's constants and the gate arithmetic. log a = k r with k = -8
// softplus(lambda) lies in [k, 0], so a CTA whose channels all have |k| <= 1/4
// (every decay above 0.78; trained layers start above 0.9) takes polynomials
// on that interval instead of the general forms:
//     a = 1 + la P(la),  sqrt(1 - a^2) = sqrt(2 |k| r) F(la),
//     1 / F^2 = G(la),   F = sqrt((1 - e^(2 la)) / (-2 la)),
// least-maximum-error fits of degree 4, within 5e-9 relative. That leaves four
// special-function operations a token (five in the general form) and no
// selection between two forms. One faster channel sends its CTA's 32 or 64 to the
// general forms: 238 us against 270 for the forward of 8 x 8192 x 2048, 206 against
// 221 for one sequence of 65536 x 1024, 142 against 151 for the backward of
// 8 x 2048 x 2048 (bf16; decays from 0.9 up against from 0.2 up). sqrt(r) i = 1 / sqrt((1 + e^-ga) (1 + e^-gx)^2)
// takes one operation in place of a root and a division; where the product
// overflows, i sqrt(r) is below 1e-19 and counts as 0.
template <int VEC, bool SMALL> struct Channel {
    using W = V<VEC>;
    W k, c;                                     // SMALL: k and sqrt(2 |k|); else k log2 e
    __device__ __forceinline__ Channel(W kn) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            k.v[e] = SMALL ? kn.v[e] : kn.v[e] * kLog2e;
            c.v[e] = SMALL ? sqrtf(-2.f * kn.v[e]) : 0.f;
        }
    }
    __device__ __forceinline__ static W poly(W x, float c4, float c3, float c2, float c1, float c0) {
        W p = W::fma(x, W::all(c4), W::all(c3));
        p = W::fma(p, x, W::all(c2));
        p = W::fma(p, x, W::all(c1));
        return W::fma(p, x, W::all(c0));
    }
    __device__ __forceinline__ static W polyF(W la) {
        return poly(la, 0.012341252528f, 0.062206134200f, 0.208307415247f, 0.499999195337f, 1.f);
    }
    // a from r = 1 / (1 + e^-ga)
    __device__ __forceinline__ W decay(W r) const {
        const W la = W::mul(k, r);
        if (!SMALL) return each<VEC, ex2>(la);
        return W::fma(la, poly(la, 0.007514995988f, 0.041491348296f, 0.166651189327f, 0.499999523163f, 1.f), W::all(1.f));
    }
    // a and b = sqrt(1 - a^2) i x
    __device__ __forceinline__ void forward(W x, W ga, W gx, W& a, W& b) const {
        const W u = one_plus_exp<VEC>(ga), r = each<VEC, rcp>(u);
        a = decay(r);
        if (SMALL) {
            const W w = one_plus_exp<VEC>(gx);
            const W q = each<VEC, rsq>(W::mul(W::mul(u, w), w));
            b = W::mul(W::mul(x, c), W::mul(q, polyF(W::mul(k, r))));
        } else {
            const W m2 = one_minus_a2<VEC>(W::mul(k, r), a);
            W z = W::mul(gx, W::all(-kLog2e));
#pragma unroll
            for (int e = 0; e < VEC; ++e) z.v[e] = min_nan(z.v[e], 63.f);     // the square stays finite
            const W w = W::add(each<VEC, ex2>(z), W::all(1.f));
            const W s = W::fma(W::mul(m2, w), w, W::all(kTiny));
            b = W::mul(W::mul(x, m2), each<VEC, rsq>(s));
        }
    }
    // r, i, a and m i = sqrt(1 - a^2) i
    __device__ __forceinline__ void backward(W ga, W gx, W& r, W& i, W& a, W& mi) const {
        const W u = one_plus_exp<VEC>(ga), w = one_plus_exp<VEC>(gx);
        r = each<VEC, rcp>(u);
        i = each<VEC, rcp>(w);
        a = decay(r);
        if (SMALL) {
            const W q = each<VEC, rsq>(W::mul(W::mul(u, w), w));
            mi = W::mul(W::mul(q, c), polyF(W::mul(k, r)));
        } else {
            const W m2 = one_minus_a2<VEC>(W::mul(k, r), a);
            mi = W::mul(W::mul(m2, each<VEC, rsq>(W::add(m2, W::all(kTiny)))), i);
        }
    }
    // log a and -log a / (1 - a^2), which tends to 1/2 as log a -> 0
    __device__ __forceinline__ void logs(W r, W a, W& la, W& lm) const {
        const W x = W::mul(k, r);
        if (SMALL) {
            la = x;
            lm = poly(x, -0.010837296955f, 0.000080529244f, 0.166674852371f, -0.499999731779f, 0.5f);
        } else {
            la = W::mul(x, W::all(kLn2));
            const W m2 = one_minus_a2<VEC>(x, a);
            const W im = each<VEC, rsq>(W::add(m2, W::all(kTiny)));
            lm = W::mul(W::mul(W::mul(la, W::all(-1.f)), im), im);
        }
    }
};

// ---- tiles and the maps between them ----
// NW warps with runs of SEG tokens, NS tiles in flight
template <int NW_, int SEG_, int NS_> struct Shape {
    static constexpr int NW = NW_, SEG = SEG_, NS = NS_, kTokens = NW * SEG;
    static_assert(kTokens % kLruSave == 0, "a tile starts at a saved state");
};

enum Load { kTensor, kAsync4, kPlain };

// A cluster's last round has tiles past the end (forward) or below 0
// (backward): their tokens are not in memory.
__host__ __device__ constexpr bool token_exists(int t, int T) { return t >= 0 && t < T; }
static_assert(!token_exists(-1, 5) && !token_exists(-64, 5) && token_exists(0, 5) && token_exists(4, 5) && !token_exists(5, 5),
              "reads outside a sequence");

// NT input tensors of a CTA's channels, NS tiles ahead in shared memory.
// Words of 4 bytes, [stage][tensor][token][lane]: a lane's VEC channels.
template <typename T, int VEC, int NT, int LOAD, typename S> struct Stager {
    using R = Row<T, VEC>;
    static constexpr int kTile = S::kTokens, kSeg = S::SEG, NS = S::NS;
    static constexpr int kStageBytes = NT * kTile * 32 * 4;
    static constexpr int kBytes = LOAD == kPlain ? 0 : NS * kStageBytes;
    const CUtensorMap* maps[NT];
    const T* src[NT];                           // the CTA's sequence, at this lane's channels
    uint32_t* buf;
    uint64_t* full;                             // [NS]
    int T_, D, c_cta, b;
    bool live;
#ifdef MESA_DEBUG
    bool lose = false;
#endif

    // A round up to NS ahead; call by all threads, tile < 0 or past the end: nothing to load.
    // After a wait that was given up thread 0 issues no more: the barrier's phase is open.
    __device__ __forceinline__ void issue(int round, int tile, int tiles, bool ok) {
        if (tile < 0 || tile >= tiles) return;
        const int st = round % NS, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        if (LOAD == kTensor) {
            if (threadIdx.x == 0 && ok) {
                tc::mbar_arrive_expect_tx(&full[st], kStageBytes);
#pragma unroll
                for (int i = 0; i < NT; ++i) {
#ifdef MESA_DEBUG
                    if (lose && round == 0 && i == 0) continue;       // fault injection: this copy never lands
#endif
                    swa::tma_load(buf + (st * NT + i) * kTile * 32, maps[i], c_cta, tile * kTile, b, &full[st]);
                }
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
        if (LOAD == kTensor) return tc::mbar_wait(&full[round % NS], (round / NS) & 1);
        if (LOAD == kAsync4) {
            if (NS > 1 && ahead) asm volatile("cp.async.wait_group 1;" ::: "memory");
            else asm volatile("cp.async.wait_group 0;" ::: "memory");
        }
        return true;
    }
    __device__ __forceinline__ typename R::Raw get(int round, int i, int tile, int s) const {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        if (LOAD == kPlain) {
            const int t = tile * kTile + warp * kSeg + s;
            return live && token_exists(t, T_) ? R::load(src[i], (size_t)t * D) : R::zero();
        }
        const uint32_t w = buf[(((round % NS) * NT + i) * kTile + warp * kSeg + s) * 32 + lane];
        return *reinterpret_cast<const typename R::Raw*>(&w);
    }
};

// a map x -> a x + b per channel
template <int VEC> struct alignas(8 * VEC) W2 {
    V<VEC> a, b;
};

// maps exchanged between the CTAs of a cluster, by one warp of each
template <int VEC> struct Exchange {
    W2<VEC>* peer;                              // [2][ncta][32]
    uint64_t* bar;                              // [2]
    int ncta, rank;
    // This CTA's map to every CTA of the cluster, itself included. Lanes that
    // gave up a wait send no more, so that the others give up as well.
    __device__ __forceinline__ void send(int round, const W2<VEC>& m) {
        const int par = round & 1, lane = threadIdx.x & 31;
        if (lane == 0) tc::mbar_arrive_expect_tx(&bar[par], ncta * 32 * (int)sizeof(W2<VEC>));
        const uint32_t b0 = tc::smem_addr(&bar[par]), a0 = tc::smem_addr(&peer[(par * ncta + rank) * 32 + lane]);
        for (int r = 0; r < ncta; ++r) {
            uint32_t rb, ra;
            asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(rb) : "r"(b0), "r"(r));
            asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(ra) : "r"(a0), "r"(r));
            if (VEC == 2)
                asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::
                                 "r"(ra), "f"(m.a.v[0]), "f"(m.a.v[VEC - 1]), "f"(m.b.v[0]), "f"(m.b.v[VEC - 1]), "r"(rb)
                             : "memory");
            else
                asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(ra),
                             "f"(m.a.v[0]), "f"(m.b.v[0]), "r"(rb)
                             : "memory");
        }
    }
    __device__ __forceinline__ bool wait(int round) { return tc::mbar_wait(&bar[round & 1], (round >> 1) & 1); }
    __device__ __forceinline__ W2<VEC> get(int round, int r) const {
        return peer[((round & 1) * ncta + r) * 32 + (threadIdx.x & 31)];
    }
};

__device__ __forceinline__ void cluster_arrive() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_sync() {
    cluster_arrive();
    cluster_wait();
}

// End of a kernel. A CTA that gave up a wait says so, and leaves when nothing
// can write to its shared memory any more. Its copies have had that wait's second
// to land, since the last was issued before it began; the other CTAs, which may
// still send it their maps, are done (threads that have returned count as
// arrived). A CTA that met all its waits has received everything.
__device__ __forceinline__ void leave(bool ok, int ncta, unsigned* err) {
    if (!ok) {
        record_error(err, kErrTimeout);
        asm volatile("cp.async.wait_all;" ::: "memory");
    }
    if (ncta > 1 && __syncthreads_or(!ok)) cluster_sync();
}

struct Where {
    int rank, b, c0, c_cta, tiles, rounds;
    bool live;
    size_t base;
    template <int VEC, int TILE> __device__ __forceinline__ static Where make(const LruArgs& p, int groups, int ncta) {
        Where w;
        w.rank = ncta > 1 ? blockIdx.x % ncta : 0;
        const unsigned work = blockIdx.x / ncta;
        w.b = work / groups;
        w.c_cta = (work % groups) * (32 * VEC);
        w.c0 = w.c_cta + (threadIdx.x & 31) * VEC;
        w.live = w.c0 < p.D;                    // VEC divides D
        w.base = (size_t)w.b * p.T * p.D + w.c0;
        w.tiles = (p.T + TILE - 1) / TILE;
        w.rounds = (w.tiles + ncta - 1) / ncta;
        return w;
    }
};

template <int VEC> __host__ __device__ constexpr int peer_bytes(int ncta) { return ncta > 1 ? 2 * ncta * VEC * 32 * 8 : 0; }

// -8 softplus(lambda) of a lane's channels; whether all of the CTA's lie in [-1/4, 0]
template <int VEC> __device__ __forceinline__ V<VEC> channel_k(const LruArgs& p, const Where& w, bool& small) {
    V<VEC> k;
    bool s = true;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        k.v[e] = w.live ? -kC * softplus(p.lambda[w.c0 + e]) : 0.f;
        s = s && k.v[e] >= -0.25f;
    }
    small = __syncthreads_and(s);
    return k;
}

// ---- forward ----
template <int VEC, int NW> struct FwdShared {
    W2<VEC> run[NW][32];                        // the map of each run
    V<VEC> before[NW][32];                      // the state before it
    uint64_t bars[4];
};

template <typename T, int VEC, int LOAD, typename S, bool SMALL>
__device__ __forceinline__ bool forward_walk(const LruArgs& p, const Where& w, int ncta, V<VEC> k,
                                             Stager<T, VEC, 3, LOAD, S>& in, Exchange<VEC>& ex, FwdShared<VEC, S::NW>& sh) {
    constexpr int kSeg = S::SEG, NW = S::NW;
    using R = Row<T, VEC>;
    using W = V<VEC>;
    const Channel<VEC, SMALL> ch(k);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    bool ok = true;
    W carry;
#pragma unroll
    for (int e = 0; e < VEC; ++e) carry.v[e] = w.live && p.h0 ? p.h0[(size_t)w.b * p.D + w.c0 + e] : 0.f;
    // h_T in the place of h0 is written only when every CTA has read h0
    const bool in_place = ncta > 1 && p.h0 && p.h0 == p.hT;
    if (in_place) cluster_arrive();
    for (int j = 0; j < w.rounds; ++j) {
        const int tile = j * ncta + w.rank;
        const int t0 = tile * S::kTokens + warp * kSeg;
        const bool any = tile < w.tiles;
        W a[kSeg], h[kSeg], A = W::all(1.f), Hl = W::all(0.f);
        if (any && ok) ok = in.wait(j, tile + ncta < w.tiles);
#pragma unroll
        for (int s = 0; s < kSeg; ++s) {
            W x, ga, gx;
            R::unpack(in.get(j, 0, tile, s), x.v);
            R::unpack(in.get(j, 1, tile, s), ga.v);
            R::unpack(in.get(j, 2, tile, s), gx.v);
            ch.forward(x, ga, gx, a[s], h[s]);
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
        sh.run[warp][lane] = {A, Hl};
        __syncthreads();
        in.issue(j, tile + S::NS * ncta, w.tiles, ok);   // every thread has read the stage
        if (warp == 0) {
            W c = carry;
            if (ncta > 1) {
                W2<VEC> m = sh.run[0][lane];
#pragma unroll
                for (int u = 1; u < NW; ++u) {
                    const W2<VEC> g = sh.run[u][lane];
                    m = {W::mul(g.a, m.a), W::fma(g.a, m.b, g.b)};
                }
                if (ok) {
                    ex.send(j, m);
                    ok = ex.wait(j);
                }
                W mine = c;
                for (int r = 0; r < ncta; ++r) {
                    if (r == w.rank) mine = c;
                    const W2<VEC> o = ex.get(j, r);
                    c = W::fma(o.a, c, o.b);
                }
                carry = c;
                c = mine;
            }
#pragma unroll
            for (int u = 0; u < NW; ++u) {
                const W2<VEC> g = sh.run[u][lane];
                sh.before[u][lane] = c;
                c = W::fma(g.a, c, g.b);
            }
            if (ncta == 1) carry = c;
        }
        __syncthreads();
        W hv = sh.before[warp][lane];
        if (p.saved && w.live && (warp * kSeg) % kLruSave == 0 && t0 < p.T) {
            const size_t row = (size_t)w.b * ((p.T + kLruSave - 1) / kLruSave) + t0 / kLruSave;
#pragma unroll
            for (int e = 0; e < VEC; ++e) p.saved[row * p.D + w.c0 + e] = hv.v[e];
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
    if (in_place) cluster_wait();
    if (p.hT && w.live && w.rank == 0 && warp == 0) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) p.hT[(size_t)w.b * p.D + w.c0 + e] = carry.v[e];
    }
    return ok;
}

template <typename T, int VEC, int LOAD, typename S>
__global__ void __launch_bounds__(S::NW * 32, 2)
lru_forward_kernel(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap ma,
                   const __grid_constant__ CUtensorMap mg, LruArgs p, int groups, int ncta, unsigned* err) {
    using St = Stager<T, VEC, 3, LOAD, S>;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ FwdShared<VEC, S::NW> sh;
    const Where w = Where::make<VEC, S::kTokens>(p, groups, ncta);
    St in{{&mx, &ma, &mg},
          {static_cast<const T*>(p.x) + w.base, static_cast<const T*>(p.ga) + w.base, static_cast<const T*>(p.gx) + w.base},
          reinterpret_cast<uint32_t*>(smem), sh.bars, p.T, p.D, w.c_cta, w.b, w.live};
#ifdef MESA_DEBUG
    in.lose = p.lose && w.rank == 0;
#endif
    Exchange<VEC> ex{reinterpret_cast<W2<VEC>*>(smem + St::kBytes), sh.bars + 2, ncta, w.rank};
    if (threadIdx.x == 0) {
        for (int i = 0; i < 4; ++i) tc::mbar_init(&sh.bars[i], 1);
        tc::fence_mbar_init();
    }
    if (ncta > 1) cluster_sync(); else __syncthreads();
    for (int i = 0; i < S::NS; ++i) in.issue(i, w.rank + i * ncta, w.tiles, true);
    bool small;
    const V<VEC> k = channel_k<VEC>(p, w, small);
    const bool ok = small ? forward_walk<T, VEC, LOAD, S, true>(p, w, ncta, k, in, ex, sh)
                          : forward_walk<T, VEC, LOAD, S, false>(p, w, ncta, k, in, ex, sh);
    leave(ok, ncta, err);
}

// ---- backward ----
// g_t = dy_t + c_t with c_{t-1} = a_t g_t: the same map per run, composed from
// the end. The states h_{t-1} are rescanned inside the tile from the saved
// state before it, so the tiles only pass c on. s = dL/dlog a * log a feeds
// both dgate_a = s (1 - r) and dlambda.
template <int VEC, int NW> struct BwdShared {
    W2<VEC> run[NW][32];                        // A, Hl of a run
    V<VEC> runc[NW][32];                        // Cl of a run
    W2<VEC> before[NW][32];                     // (c, h) entering it
    uint64_t bars[4];
};

template <typename T, int VEC, int LOAD, typename S, bool SMALL>
__device__ __forceinline__ bool backward_walk(const LruBackwardArgs& q, const Where& w, int ncta, V<VEC> k,
                                              Stager<T, VEC, 4, LOAD, S>& in, Exchange<VEC>& ex,
                                              BwdShared<VEC, S::NW>& sh) {
    constexpr int kSeg = S::SEG, NW = S::NW;
    using R = Row<T, VEC>;
    using W = V<VEC>;
    const LruArgs& p = q.f;
    const Channel<VEC, SMALL> ch(k);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    bool ok = true;
    W carry, acc = W::all(0.f);
#pragma unroll
    for (int e = 0; e < VEC; ++e) carry.v[e] = w.live && q.dhT ? q.dhT[(size_t)w.b * p.D + w.c0 + e] : 0.f;
    // tile numbers run down from the last; tiles below 0 (a cluster's last
    // round) are empty: closed gates and no gradient
    const int top = w.tiles - 1 - w.rank;
    const size_t save0 = (size_t)w.b * ((p.T + kLruSave - 1) / kLruSave);
    auto state = [&](int tile) {                 // warp 1 composes the states
        W s;
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            s.v[e] = warp == 1 && w.live && tile >= 0
                         ? p.saved[(save0 + (size_t)tile * (S::kTokens / kLruSave)) * p.D + w.c0 + e] : 0.f;
        return s;
    };
    W hs = state(top);
    for (int j = 0; j < w.rounds; ++j) {
        const int tile = top - j * ncta;
        const int t0 = tile * S::kTokens + warp * kSeg;
        const bool any = tile >= 0;
        W a[kSeg], r[kSeg], iv[kSeg], mi[kSeg], g[kSeg];
        typename R::Raw xk[kSeg];
        W A = W::all(1.f), Hl = W::all(0.f), Cl = W::all(0.f);
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
            ch.backward(ga, gx, r[s], iv[s], a[s], mi[s]);
            Hl = W::fma(a[s], Hl, W::mul(mi[s], x));
            A = W::mul(A, a[s]);
        }
#pragma unroll
        for (int s = kSeg - 1; s >= 0; --s) Cl = W::mul(a[s], W::add(g[s], Cl));
        sh.run[warp][lane] = {A, Hl};
        sh.runc[warp][lane] = Cl;
        __syncthreads();
        in.issue(j, tile - S::NS * ncta, w.tiles, ok);
        if (warp == 0) {
            W c = carry;
            if (ncta > 1) {
                W2<VEC> m = {sh.run[NW - 1][lane].a, sh.runc[NW - 1][lane]};
#pragma unroll
                for (int u = NW - 2; u >= 0; --u) {
                    const W ra = sh.run[u][lane].a;
                    m = {W::mul(ra, m.a), W::fma(ra, m.b, sh.runc[u][lane])};
                }
                if (ok) {
                    ex.send(j, m);
                    ok = ex.wait(j);
                }
                W mine = c;
                for (int t = 0; t < ncta; ++t) {
                    if (t == w.rank) mine = c;
                    const W2<VEC> o = ex.get(j, t);
                    c = W::fma(o.a, c, o.b);
                }
                carry = c;
                c = mine;
            }
#pragma unroll
            for (int u = NW - 1; u >= 0; --u) {
                sh.before[u][lane].a = c;
                c = W::fma(sh.run[u][lane].a, c, sh.runc[u][lane]);
            }
            if (ncta == 1) carry = c;
        } else if (warp == 1) {
            W hv = hs;
            hs = state(tile - ncta);
#pragma unroll
            for (int u = 0; u < NW; ++u) {
                const W2<VEC> o = sh.run[u][lane];
                sh.before[u][lane].b = hv;
                hv = W::fma(o.a, hv, o.b);
            }
        }
        __syncthreads();
        W gc = sh.before[warp][lane].a, hv = sh.before[warp][lane].b, part = W::all(0.f);
#pragma unroll
        for (int s = kSeg - 1; s >= 0; --s) {
            g[s] = W::add(g[s], gc);
            gc = W::mul(a[s], g[s]);
        }
        const size_t o0 = w.base + (size_t)t0 * p.D;
        T* pdx = static_cast<T*>(q.dx) + o0;
        T* pda = static_cast<T*>(q.dga) + o0;
        T* pdg = static_cast<T*>(q.dgx) + o0;
#pragma unroll
        for (int s = 0; s < kSeg; ++s) {
            W x, la, lm;
            R::unpack(xk[s], x.v);
            ch.logs(r[s], a[s], la, lm);
            const W b = W::mul(mi[s], x), dx = W::mul(g[s], mi[s]);
            // g log a (a h_{t-1} - b a^2 / m^2), with -log a / m^2 = lm
            const W inner = W::fma(la, hv, W::mul(W::mul(b, a[s]), lm));
            const W sv = W::mul(W::mul(g[s], a[s]), inner);
            const W dga = W::fma(W::mul(sv, W::all(-1.f)), r[s], sv);
            const W gb = W::mul(g[s], b);
            const W dgx = W::fma(W::mul(gb, W::all(-1.f)), iv[s], gb);
            part = W::add(part, sv);
            hv = W::fma(a[s], hv, b);
            if (w.live && (!tail || (any && t0 + s < p.T))) {
                R::store(pdx, (size_t)s * p.D, dx.v);
                R::store(pda, (size_t)s * p.D, dga.v);
                R::store(pdg, (size_t)s * p.D, dgx.v);
            }
        }
        acc = W::add(acc, part);
    }
    sh.runc[warp][lane] = acc;                   // last read before the loop's last barrier
    __syncthreads();
    if (warp == 0 && w.live) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            float s = 0.f;
#pragma unroll
            for (int u = 0; u < NW; ++u) s += sh.runc[u][lane].v[e];
            q.partial[((size_t)w.b * ncta + w.rank) * p.D + w.c0 + e] = s;
            if (q.dh0 && w.rank == 0) q.dh0[(size_t)w.b * p.D + w.c0 + e] = carry.v[e];
        }
    }
    return ok;
}

template <typename T, int VEC, int LOAD, typename S>
__global__ void __launch_bounds__(S::NW * 32, 2)
lru_backward_kernel(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap ma,
                    const __grid_constant__ CUtensorMap mg, const __grid_constant__ CUtensorMap md, LruBackwardArgs q,
                    int groups, int ncta, unsigned* err) {
    using St = Stager<T, VEC, 4, LOAD, S>;
    const LruArgs& p = q.f;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ BwdShared<VEC, S::NW> sh;
    const Where w = Where::make<VEC, S::kTokens>(p, groups, ncta);
    St in{{&mx, &ma, &mg, &md},
          {static_cast<const T*>(p.x) + w.base, static_cast<const T*>(p.ga) + w.base, static_cast<const T*>(p.gx) + w.base,
           static_cast<const T*>(q.dy) + w.base},
          reinterpret_cast<uint32_t*>(smem), sh.bars, p.T, p.D, w.c_cta, w.b, w.live};
#ifdef MESA_DEBUG
    in.lose = p.lose && w.rank == 0;
#endif
    Exchange<VEC> ex{reinterpret_cast<W2<VEC>*>(smem + St::kBytes), sh.bars + 2, ncta, w.rank};
    if (threadIdx.x == 0) {
        for (int i = 0; i < 4; ++i) tc::mbar_init(&sh.bars[i], 1);
        tc::fence_mbar_init();
    }
    if (ncta > 1) cluster_sync(); else __syncthreads();
    for (int i = 0; i < S::NS; ++i) in.issue(i, w.tiles - 1 - w.rank - i * ncta, w.tiles, true);
    bool small;
    const V<VEC> k = channel_k<VEC>(p, w, small);
    const bool ok = small ? backward_walk<T, VEC, LOAD, S, true>(q, w, ncta, k, in, ex, sh)
                          : backward_walk<T, VEC, LOAD, S, false>(q, w, ncta, k, in, ex, sh);
    leave(ok, ncta, err);
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
    V<VEC> xv, av, gv, k, a, h;
    R::unpack(R::load(x, i), xv.v);
    R::unpack(R::load(ga, i), av.v);
    R::unpack(R::load(gx, i), gv.v);
#pragma unroll
    for (int e = 0; e < VEC; ++e) k.v[e] = -kC * softplus(lambda[c + e]);
    Channel<VEC, false>(k).forward(xv, av, gv, a, h);
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

// [B][T][D] as a 3-D map of tiles of 128 bytes of channels
bool channel_map(CUtensorMap* m, const LruArgs& a, const void* base, int tile) {
    const bool f32 = a.dtype == MESA_F32;
    return swa::encode_map(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, f32 ? 4 : 2, base,
                           a.D, a.T, a.B, f32 ? 32 : 64, tile, CU_TENSOR_MAP_SWIZZLE_NONE);
}

// CTAs per sequence and channel group: doubled while the grid leaves SMs idle
// and every CTA still gets a tile. An exchange between CTAs costs about as much
// as a tile's arithmetic, so a grid that fills the SMs takes none.
int cluster_size(long long blocks, int tiles) {
    int n = 1;
    while (n < kLruMaxCluster && tiles >= 2 * n && blocks * n < 148) n *= 2;
    return n;
}

// Shared memory of a launch: the stager's, and the maps of ncta CTAs. The
// kernel's limit is set to what any launch may ask for, always: another host
// thread may be about to launch it for a larger cluster.
template <int VEC, typename F, typename... A>
cudaError_t launch_cluster(F* kernel, unsigned grid, int threads, int ncta, int stager_bytes, cudaStream_t st, A... args) {
    const int smem = stager_bytes + peer_bytes<VEC>(ncta);
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         stager_bytes + peer_bytes<VEC>(kLruMaxCluster));
    if (e == cudaSuccess && ncta > 8) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
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
// Few sequences and channels: long runs, so that a cluster exchanges maps
// seldom. Many: more warps.
using FwdWide = Shape<16, 8, 2>;
using FwdLong = Shape<8, 16, 1>;
using Bwd = Shape<8, 8, 2>;

Plan plan(int B, int T, int D, int vec, int tile) {
    Plan pl;
    pl.groups = (D + 32 * vec - 1) / (32 * vec);
    const long long blocks = (long long)B * pl.groups;
    pl.ncta = cluster_size(blocks, (T + tile - 1) / tile);
    pl.grid = (unsigned)(blocks * pl.ncta);
    return pl;
}

template <typename T, int VEC, int LOAD, typename S>
cudaError_t forward(const LruArgs& a, const Plan& pl, unsigned* err, cudaStream_t st) {
    CUtensorMap m[3] = {};
    if (LOAD == kTensor && (!channel_map(&m[0], a, a.x, S::kTokens) || !channel_map(&m[1], a, a.ga, S::kTokens) ||
                            !channel_map(&m[2], a, a.gx, S::kTokens)))
        return cudaErrorInvalidValue;
    return launch_cluster<VEC>(lru_forward_kernel<T, VEC, LOAD, S>, pl.grid, S::NW * 32, pl.ncta,
                               Stager<T, VEC, 3, LOAD, S>::kBytes, st, m[0], m[1], m[2], a, pl.groups, pl.ncta, err);
}

template <typename T, int VEC, int LOAD>
cudaError_t forward(const LruArgs& a, unsigned* err, cudaStream_t st) {
    const Plan pl = plan(a.B, a.T, a.D, VEC, FwdWide::kTokens);
    return pl.ncta > 1 ? forward<T, VEC, LOAD, FwdLong>(a, pl, err, st) : forward<T, VEC, LOAD, FwdWide>(a, pl, err, st);
}

template <typename T, int VEC, int LOAD>
cudaError_t backward(const LruBackwardArgs& q, unsigned* err, cudaStream_t st) {
    using S = Bwd;
    const LruArgs& a = q.f;
    CUtensorMap m[4] = {};
    if (LOAD == kTensor && (!channel_map(&m[0], a, a.x, S::kTokens) || !channel_map(&m[1], a, a.ga, S::kTokens) ||
                            !channel_map(&m[2], a, a.gx, S::kTokens) || !channel_map(&m[3], a, q.dy, S::kTokens)))
        return cudaErrorInvalidValue;
    const Plan pl = plan(a.B, a.T, a.D, VEC, S::kTokens);
    cudaError_t e = launch_cluster<VEC>(lru_backward_kernel<T, VEC, LOAD, S>, pl.grid, S::NW * 32, pl.ncta,
                                        Stager<T, VEC, 4, LOAD, S>::kBytes, st, m[0], m[1], m[2], m[3], q, pl.groups,
                                        pl.ncta, err);
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
    const int t = (T + Bwd::kTokens - 1) / Bwd::kTokens;  // every CTA of a cluster has a tile
    return (size_t)B * (t < 1 ? 1 : t < kLruMaxCluster ? t : kLruMaxCluster);
}

cudaError_t lru_forward(const LruArgs& args, cudaStream_t st) {
    LaunchTimer lt(kKindLru, st);
    LruArgs a = args;
#ifdef MESA_DEBUG
    a.lose = debug_lose_signal();
#endif
    unsigned* err = error_word_ptr();
    if (!err) return cudaErrorUnknown;
    using bf = __nv_bfloat16;
    if (tensor_ok(a, {a.x, a.ga, a.gx}) && all_aligned({a.y}, 4))
        return a.dtype == MESA_F32 ? forward<float, 1, kTensor>(a, err, st) : forward<bf, 2, kTensor>(a, err, st);
    if (a.dtype == MESA_F32) return forward<float, 1, kAsync4>(a, err, st);
    return pair_ok(a.D, {a.x, a.ga, a.gx, a.y}) ? forward<bf, 2, kAsync4>(a, err, st) : forward<bf, 1, kPlain>(a, err, st);
}

cudaError_t lru_backward(const LruBackwardArgs& args, cudaStream_t st) {
    LaunchTimer lt(kKindLruBwd, st);
    LruBackwardArgs q = args;
    const LruArgs& a = q.f;
#ifdef MESA_DEBUG
    q.f.lose = debug_lose_signal();
#endif
    unsigned* err = error_word_ptr();
    if (!err) return cudaErrorUnknown;
    using bf = __nv_bfloat16;
    if (tensor_ok(a, {a.x, a.ga, a.gx, q.dy}) && all_aligned({q.dx, q.dga, q.dgx}, 4))
        return a.dtype == MESA_F32 ? backward<float, 1, kTensor>(q, err, st) : backward<bf, 2, kTensor>(q, err, st);
    if (a.dtype == MESA_F32) return backward<float, 1, kAsync4>(q, err, st);
    return pair_ok(a.D, {a.x, a.ga, a.gx, q.dy, q.dx, q.dga, q.dgx}) ? backward<bf, 2, kAsync4>(q, err, st)
                                                                     : backward<bf, 1, kPlain>(q, err, st);
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
