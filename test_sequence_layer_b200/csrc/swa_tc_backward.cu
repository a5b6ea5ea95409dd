// swa_tc_backward.cu -- sliding-window attention backward on the tensor cores
// (bf16, d = 64 or 128).
//
//   P = exp(scale q k^T - lse),  dS = P (dout v^T - delta),
//   dq = scale dS k,  dk = scale dS^T q,  dv = P^T dout
//
// Two kernels, each recomputing the scores: one per 128-query tile (dq), one
// per 128-key tile (dk, dv). A single kernel would save two of seven products
// but would have to add up dq across CTAs with atomics, whose order changes
// the result. Sums stay in fp32 in tensor memory; P and dS are rounded to bf16
// as the left operands of their products, which read them from tensor memory.
// swa_stats_kernel first forms (lse log2 e, delta) for every query, padded to whole
// tiles with lse = +inf, so that rows past the end weigh nothing.
//
// The tile that holds the sinks is seen by every query: its query range is cut
// into chunks of about a window, one CTA each, whose fp32 parts are added in a
// fixed order afterwards.
//
// What bounds it: the issue of products, about 80 cycles each whether 64 or 128
// columns wide, in chains the arithmetic warps interrupt; tensor pipe 46 % busy
// in both kernels. Batch 2, 16 over 4 heads, 8192 tokens, d = 128, window 1024:
// 638 us in all. Steps of 64 queries let dk, dv run two stages; with 128 their
// scores and sums leave tensor memory no room for a second at d = 128, and both
// widths use the same columns.
#include "swa_tc.cuh"

namespace mesa {

using namespace tc;

namespace {

constexpr int kTile = 128;                           // queries or keys a CTA owns; keys per step of dq
constexpr int kSub = 64;                             // queries per step of dk, dv
constexpr int kThreads = 320;                        // 8 warps of arithmetic, one of copies, one of products
constexpr int kMaxChunks = 32;

struct BwdParams {
    SwaArgs a;
    const float2* stats;                             // [B Hq][tpad]
    int tpad;
    void* dq;
    void* dk;
    void* dv;
    float* parts;                                    // [B Hkv][chunks][2][128][D]
    int chunks, chunk_len;                           // of the sink tile's queries
    unsigned* err;
#ifdef MESA_DEBUG
    int lose;
#endif
};

// ---- (lse log2 e, delta) per query ----
__device__ __forceinline__ float dot8(const uint4& x, const uint4& y) {
    const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        s = fmaf(__uint_as_float(xs[i] << 16), __uint_as_float(ys[i] << 16), s);
        s = fmaf(__uint_as_float(xs[i] & 0xffff0000u), __uint_as_float(ys[i] & 0xffff0000u), s);
    }
    return s;
}

template <int D, bool FEW>
__global__ void swa_stats_kernel(SwaArgs a, const __nv_bfloat16* __restrict__ dout, int tpad, float2* __restrict__ stats) {
    using bf = __nv_bfloat16;
    constexpr int kLanes = D / 8;                    // 16-byte pieces of a row
    const int row = (blockIdx.x * blockDim.x + threadIdx.x) / kLanes, piece = threadIdx.x % kLanes;
    if (row >= tpad) return;                         // whole groups of kLanes lanes
    const bool in = row < a.T;
    const size_t src = (size_t)blockIdx.y * a.T + (in ? row : 0);
    auto sum = [&](float v) {
#pragma unroll
        for (int i = kLanes / 2; i; i >>= 1) v += __shfl_xor_sync(~0u, v, i);
        return v;
    };
    const float lse2 = a.lse[src] * swa::kLog2e;
    const uint4 g = reinterpret_cast<const uint4*>(dout + src * D)[piece];
    float delta;
    if (FEW) {
        const size_t kv = (size_t)(blockIdx.y / (a.Hq / a.Hkv)) * a.S * D;
        const uint4 q = reinterpret_cast<const uint4*>(static_cast<const bf*>(a.q) + src * D)[piece];
        const swa::FewKeys keys(a.S - a.T + (in ? row : 0), a.window, a.sinks);
        delta = 0.f;
#pragma unroll
        for (int i = 0; i < swa::kFewKeys; ++i) {      // every lane of a warp runs all steps
            const int j = keys.key(i);
            const uint4 k = reinterpret_cast<const uint4*>(static_cast<const bf*>(a.k) + kv + (size_t)j * D)[piece];
            const uint4 v = reinterpret_cast<const uint4*>(static_cast<const bf*>(a.v) + kv + (size_t)j * D)[piece];
            const float w = swa::ex2(fmaf(sum(dot8(q, k)), a.scale * swa::kLog2e, -lse2)), dp = sum(dot8(g, v));
            if (i < keys.n) delta = fmaf(w, dp, delta);
        }
    } else {
        delta = sum(dot8(reinterpret_cast<const uint4*>(static_cast<const bf*>(a.out) + src * D)[piece], g));
    }
    if (piece == 0) stats[(size_t)blockIdx.y * tpad + row] = make_float2(in ? lse2 : INFINITY, in ? delta : 0.f);
}

__device__ __forceinline__ uint8_t* align_smem(uint8_t* p) {
    return reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(p) + 1023) & ~uintptr_t(1023));
}

// 32 columns of scores and of dP -> 32 columns of P and dS, packed to bf16.
// st(e): the column's (lse log2 e, delta). Bit e of `vis`: it is visible.
template <bool kWantP, typename Stat>
__device__ __forceinline__ void weights32(const float (&s)[32], const float (&dp)[32], float sc, uint32_t vis,
                                          bool whole, Stat st, float (&pk)[16], float (&dk)[16]) {
    const float2 sc2 = make_float2(sc, sc);
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
        const float2 a = st(e), b = st(e + 1);
        float2 w = swa::fma2(make_float2(s[e], s[e + 1]), sc2, make_float2(-a.x, -b.x));
        w.x = swa::ex2(w.x);
        w.y = swa::ex2(w.y);
        if (!whole) {
            if (!(vis & (1u << e))) w.x = 0.f;
            if (!(vis & (2u << e))) w.y = 0.f;
        }
        const float2 g = swa::mul2(w, swa::add2(make_float2(dp[e], dp[e + 1]), make_float2(-a.y, -b.y)));
        if (kWantP) pk[e / 2] = __uint_as_float(swa::pack_bf16(w.x, w.y));
        dk[e / 2] = __uint_as_float(swa::pack_bf16(g.x, g.y));
    }
}

template <int D>
__device__ __forceinline__ void store_row(__nv_bfloat16* dst, uint32_t taddr, int c0, int n, float f, bool in) {
#pragma unroll
    for (int c = 0; c < D; c += 32) {
        if (c >= n) break;
        float o[32];
        tmem_ld32_x32(taddr + c0 + c, o);
        tmem_wait_ld();
        if (!in) continue;
        uint4* d4 = reinterpret_cast<uint4*>(dst + c0 + c);
#pragma unroll
        for (int e = 0; e < 32; e += 8)
            d4[e / 8] = make_uint4(swa::pack_bf16(o[e] * f, o[e + 1] * f), swa::pack_bf16(o[e + 2] * f, o[e + 3] * f),
                                   swa::pack_bf16(o[e + 4] * f, o[e + 5] * f), swa::pack_bf16(o[e + 6] * f, o[e + 7] * f));
    }
}

// ---- dq ----
// Tensor memory: two score buffers (columns 0, 128), dP (256), dq (384). Each
// half of dS(n) replaces the front of its half of S(n). The arithmetic warps take S and dP into
// registers first and release dP, so dP(n + 1) and S(n + 2) are computed under
// the exponentials of step n.
template <int D> struct DqSmem {
    static constexpr int kBytes = 128 * D * 2;
    static constexpr int kKStages = 3, kVStages = 2;
    static constexpr int oQ = 0, oDo = kBytes, oK = 2 * kBytes, oV = oK + kKStages * kBytes;
    static constexpr int oBar = oV + kVStages * kBytes;
    static constexpr int bytes = oBar + 16 * 8 + 16 + 1024;
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
swa_tc_dq_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mdo,
                 const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv, const BwdParams f) {
    using L = DqSmem<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = align_smem(smem_raw);
    uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + L::oBar);      // [3]
    uint64_t* k_empty = k_full + 3;                                      // [3]
    uint64_t* v_full = k_empty + 3;                                      // [2]
    uint64_t* v_empty = v_full + 2;                                      // [2]
    uint64_t* bar_q = v_empty + 2;
    uint64_t* s_full = bar_q + 1;                                        // S(n) and dP(n) are in tensor memory
    uint64_t* dp_free = s_full + 1;                                      // dP(n) has been read
    uint64_t* ds_ready = dp_free + 1;                                    // dS(n) has been written
    uint64_t* done = ds_ready + 1;
    uint32_t* slot = reinterpret_cast<uint32_t*>(done + 1);
    const SwaArgs& a = f.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int head = blockIdx.y, hkv = head / (a.Hq / a.Hkv), t0 = blockIdx.x * kTile;
    const int p0 = a.S - a.T + t0, p1 = a.S - a.T + min(t0 + kTile, a.T) - 1;
    const swa::KeyTiles kt(p0, p1, a.window, a.sinks, kTile);
    if (tid == 0) {
        for (int i = 0; i < 3; ++i) mbar_init(&k_full[i], 1), mbar_init(&k_empty[i], 1);
        for (int i = 0; i < 2; ++i) mbar_init(&v_full[i], 1), mbar_init(&v_empty[i], 1);
        mbar_init(bar_q, 1);
        mbar_init(s_full, 1);
        mbar_init(dp_free, 8);
        mbar_init(ds_ready, 8);
        mbar_init(done, 1);
        fence_mbar_init();
    }
    if (warp == 8) tmem_alloc(slot, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = *slot, tDp = tm + 256, tDq = tm + 384;
    bool ok = true;

    if (warp == 8) {
        if (lane == 0) {
            mbar_arrive_expect_tx(bar_q, 2 * L::kBytes);
            for (int c = 0; c < D / 64; ++c) {
                swa::tma_load(smem + L::oQ + c * 16384, &mq, c * 64, t0, head, bar_q);
                swa::tma_load(smem + L::oDo + c * 16384, &mdo, c * 64, t0, head, bar_q);
            }
            int nk = 0, nv = 0;                              // tiles whose copies were issued
            for (int n = 0; n < kt.n && ok; ++n) {
                const int sk = n % 3, sv = n & 1, j0 = kt.tile(n) * kTile;
                ok = swa::wait_bar(&k_empty[sk], ((n / 3) & 1) ^ 1);
                if (!ok) break;
                nk = n + 1;
                mbar_arrive_expect_tx(&k_full[sk], L::kBytes);
                for (int c = 0; c < D / 64; ++c)
                    swa::tma_load(smem + L::oK + sk * L::kBytes + c * 16384, &mk, c * 64, j0, hkv, &k_full[sk]);
                ok = swa::wait_bar(&v_empty[sv], ((n >> 1) & 1) ^ 1);
                if (!ok) break;
                nv = n + 1;
                mbar_arrive_expect_tx(&v_full[sv], L::kBytes);
                for (int c = 0; c < D / 64; ++c)
                    swa::tma_load(smem + L::oV + sv * L::kBytes + c * 16384, &mv, c * 64, j0, hkv, &v_full[sv]);
            }
            // leave only when every copy has landed
            bool landed = mbar_wait(bar_q, 0);
            for (int n = max(0, nk - 3); n < nk && landed; ++n) landed = mbar_wait(&k_full[n % 3], (n / 3) & 1);
            for (int n = max(0, nv - 2); n < nv && landed; ++n) landed = mbar_wait(&v_full[n & 1], (n >> 1) & 1);
        }
    } else if (warp == 9) {
        if (lane == 0) {
            constexpr uint32_t idS = swa::idesc_bf16(128, 128, false, false);
            constexpr uint32_t idQ = swa::idesc_bf16(128, D, false, true);
            const uint32_t sq = smem_addr(smem + L::oQ), sdo = smem_addr(smem + L::oDo);
            const uint32_t sk = smem_addr(smem + L::oK), sv = smem_addr(smem + L::oV);
            auto product = [&](uint32_t d, uint32_t x, uint32_t y) {      // d = x y^T over D
#pragma unroll
                for (int s = 0; s < D / 16; ++s) {
                    const uint32_t o = (s / 4) * 16384 + (s % 4) * 32;
                    mma_f16(d, sdesc(x + o, 0, 1024), sdesc(y + o, 0, 1024), idS, s > 0);
                }
            };
            auto scores = [&](int n) {
                if (!swa::wait_bar(&k_full[n % 3], (n / 3) & 1)) return false;
                product(tm + 128 * (n & 1), sq, sk + (n % 3) * L::kBytes);
                return true;
            };
            auto dprobs = [&](int n) {
                if (!swa::wait_bar(&v_full[n & 1], (n >> 1) & 1)) return false;
                product(tDp, sdo, sv + (n & 1) * L::kBytes);
#ifdef MESA_DEBUG
                if (!(f.lose && n == 0))               // fault injection: nothing signals the first
#endif
                mma_commit(s_full);
                mma_commit(&v_empty[n & 1]);
                return true;
            };
            ok = swa::wait_bar(bar_q, 0) && scores(0) && dprobs(0);
            if (ok && kt.n > 1) ok = scores(1);
            for (int n = 0; n < kt.n && ok; ++n) {
                if (n + 1 < kt.n) {
                    ok = swa::wait_bar(dp_free, n & 1);
                    tc_fence_after();
                    ok = ok && dprobs(n + 1);
                    if (!ok) break;
                }
                ok = swa::wait_bar(ds_ready, n & 1);
                if (!ok) break;
                tc_fence_after();
                const uint32_t k = sk + (n % 3) * L::kBytes;
#pragma unroll
                for (int s = 0; s < kTile / 16; ++s)
                    swa::mma_ts(tDq, tm + 128 * (n & 1) + 64 * (s / 4) + 8 * (s % 4), sdesc(k + s * 2048, 16384, 1024), idQ, n > 0 || s > 0);
                mma_commit(&k_empty[n % 3]);
                if (n + 2 < kt.n) ok = scores(n + 2);
            }
            mma_commit(done);
            swa::wait_bar(done, 0);                      // nothing in flight when tensor memory is freed
        }
    } else {
        // warps 0-3 take columns 0-63 of a row, warps 4-7 columns 64-127
        const int half = warp >> 2, row = (warp & 3) * 32 + lane, pos = p0 + row;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const float2 stat = f.stats[(size_t)head * f.tpad + t0 + row];
        const float sc = a.scale * swa::kLog2e;
        for (int n = 0; n < kt.n; ++n) {
            const int j0 = kt.tile(n) * kTile;
            ok = __all_sync(~0u, swa::wait_bar(s_full, n & 1));      // a warp leaves as one
            if (!ok) break;
            tc_fence_after();
            const uint32_t tS = tm + 128 * (n & 1) + lanes;
            float s[2][32], dp[2][32];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                tmem_ld32_x32(tS + 64 * half + 32 * c, s[c]);
                tmem_ld32_x32(tDp + lanes + 64 * half + 32 * c, dp[c]);
            }
            tmem_wait_ld();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) swa::mbar_arrive(dp_free);
            const bool whole = j0 + kTile - 1 <= p0 && p0 + kTile - 1 - j0 < a.window;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int base = j0 + 64 * half + 32 * c;
                float pk[16], ds[16];
                // the visible keys of a row are [0, sinks) and (pos - window, pos]
                const uint32_t vis = swa::below(pos + 1 - base) &
                                     (~swa::below(pos - a.window + 1 - base) | swa::below(a.sinks - base));
                weights32<false>(s[c], dp[c], sc, vis, whole, [&](int) { return stat; }, pk, ds);
                tmem_st32_x16(tS + 64 * half + 16 * c, ds);         // over columns this thread has read
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) swa::mbar_arrive(ds_ready);
        }
        if (ok) ok = swa::wait_bar(done, 0);
        tc_fence_after();
        const int t = t0 + row;
        store_row<D>(static_cast<__nv_bfloat16*>(f.dq) + ((size_t)head * a.T + t) * D, tDq + lanes, half * (D / 2), D / 2,
                     a.scale, ok && t < a.T);
        tc_fence_before();
    }
    if (!ok) record_error(f.err, kErrTimeout);
    __syncthreads();
    if (warp == 8) tmem_dealloc(tm, 512);
}

// ---- dk, dv ----
// Steps of 64 queries over the query heads that share the keys. Tensor memory:
// two stages of (S^T, dP^T), 64 columns each, dv at 256, dk at 384. P^T and
// dS^T replace the front halves of their scores. Each group of four warps
// serves every second step; while it works, the tensor pipe runs the other
// stage's products.
template <int D> struct DkvSmem {
    static constexpr int kBytes = 128 * D * 2;       // K or V tile
    static constexpr int kPiece = kSub * D * 2;      // Q or dout rows of a step
    static constexpr int kStages = 4;
    static constexpr int oK = 0, oV = kBytes, oRing = 2 * kBytes;
    static constexpr int oStat = oRing + kStages * 2 * kPiece;
    static constexpr int oBar = oStat + kStages * kSub * 8;
    static constexpr int bytes = oBar + (2 * kStages + 6) * 8 + 16 + 1024;
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
swa_tc_dkv_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mdo,
                  const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv, const BwdParams f) {
    using L = DkvSmem<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = align_smem(smem_raw);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::oBar);
    uint64_t* empty = full + L::kStages;
    uint64_t* bar_k = empty + L::kStages;
    uint64_t* s_full = bar_k + 1;                    // [2]
    uint64_t* p_ready = s_full + 2;                  // [2]
    uint64_t* done = p_ready + 2;
    uint32_t* slot = reinterpret_cast<uint32_t*>(done + 1);
    const SwaArgs& a = f.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = a.Hq / a.Hkv, hkv = blockIdx.y, off = a.S - a.T;
    const int chunk = (int)blockIdx.x < f.chunks ? (int)blockIdx.x : 0;
    const int j0 = ((int)blockIdx.x < f.chunks ? 0 : (int)blockIdx.x - f.chunks + 1) * kTile;
    int ta, tb;
    swa::query_range(j0, min(j0 + kTile, a.S) - 1, a.T, a.S, a.window, a.sinks, ta, tb);
    ta = ta / kSub * kSub;
    if (j0 == 0) {
        ta += chunk * f.chunk_len;
        if (chunk + 1 < f.chunks) tb = min(tb, ta + f.chunk_len);
    }
    const int per = tb > ta ? (tb - ta + kSub - 1) / kSub : 0, steps = per * G;
    if (tid == 0) {
        for (int i = 0; i < L::kStages; ++i) mbar_init(&full[i], 1), mbar_init(&empty[i], 1);
        mbar_init(bar_k, 1);
        for (int i = 0; i < 2; ++i) mbar_init(&s_full[i], 1), mbar_init(&p_ready[i], 4);
        mbar_init(done, 1);
        fence_mbar_init();
    }
    if (warp == 8) tmem_alloc(slot, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = *slot, tDv = tm + 256, tDk = tm + 384;
    bool ok = true;

    if (warp == 8) {
        if (lane == 0 && steps > 0) {
            mbar_arrive_expect_tx(bar_k, 2 * L::kBytes);
            for (int c = 0; c < D / 64; ++c) {
                swa::tma_load(smem + L::oK + c * 16384, &mk, c * 64, j0, hkv, bar_k);
                swa::tma_load(smem + L::oV + c * 16384, &mv, c * 64, j0, hkv, bar_k);
            }
            int issued = 0;
            for (int n = 0; n < steps && ok; ++n) {
                const int st = n % L::kStages, head = hkv * G + n / per, t = ta + (n % per) * kSub;
                ok = swa::wait_bar(&empty[st], ((n / L::kStages) & 1) ^ 1);
                if (!ok) break;
                issued = n + 1;
                mbar_arrive_expect_tx(&full[st], 2 * L::kPiece + kSub * 8);
                uint8_t* dst = smem + L::oRing + st * 2 * L::kPiece;
                for (int c = 0; c < D / 64; ++c) {
                    swa::tma_load(dst + c * 8192, &mq, c * 64, t, head, &full[st]);
                    swa::tma_load(dst + L::kPiece + c * 8192, &mdo, c * 64, t, head, &full[st]);
                }
                bulk_g2s(smem + L::oStat + st * kSub * 8, f.stats + (size_t)head * f.tpad + t, kSub * 8, &full[st]);
            }
            // leave only when every copy has landed
            bool landed = mbar_wait(bar_k, 0);
            for (int n = max(0, issued - L::kStages); n < issued && landed; ++n)
                landed = mbar_wait(&full[n % L::kStages], (n / L::kStages) & 1);
        }
    } else if (warp == 9) {
        if (lane == 0 && steps > 0) {
            constexpr uint32_t idS = swa::idesc_bf16(128, kSub, false, false);
            constexpr uint32_t idO = swa::idesc_bf16(128, D, false, true);
            const uint32_t sk = smem_addr(smem + L::oK), sv = smem_addr(smem + L::oV), sr = smem_addr(smem + L::oRing);
            auto scores = [&](int n) {
                if (!swa::wait_bar(&full[n % L::kStages], (n / L::kStages) & 1)) return false;
                const uint32_t q = sr + (n % L::kStages) * 2 * L::kPiece, o = q + L::kPiece, t = tm + 128 * (n & 1);
#pragma unroll
                for (int s = 0; s < D / 16; ++s) {
                    const uint32_t x = (s / 4) * 16384 + (s % 4) * 32, y = (s / 4) * 8192 + (s % 4) * 32;
                    mma_f16(t, sdesc(sk + x, 0, 1024), sdesc(q + y, 0, 1024), idS, s > 0);
                }
#pragma unroll
                for (int s = 0; s < D / 16; ++s) {
                    const uint32_t x = (s / 4) * 16384 + (s % 4) * 32, y = (s / 4) * 8192 + (s % 4) * 32;
                    mma_f16(t + 64, sdesc(sv + x, 0, 1024), sdesc(o + y, 0, 1024), idS, s > 0);
                }
#ifdef MESA_DEBUG
                if (!(f.lose && n == 0))               // fault injection: nothing signals the first
#endif
                mma_commit(&s_full[n & 1]);
                return true;
            };
            ok = swa::wait_bar(bar_k, 0) && scores(0);
            if (ok && steps > 1) ok = scores(1);
            for (int n = 0; n < steps && ok; ++n) {
                ok = swa::wait_bar(&p_ready[n & 1], (n >> 1) & 1);
                if (!ok) break;
                tc_fence_after();
                const uint32_t q = sr + (n % L::kStages) * 2 * L::kPiece, o = q + L::kPiece, t = tm + 128 * (n & 1);
#pragma unroll
                for (int s = 0; s < kSub / 16; ++s)
                    swa::mma_ts(tDv, t + 8 * s, sdesc(o + s * 2048, 8192, 1024), idO, n > 0 || s > 0);
#pragma unroll
                for (int s = 0; s < kSub / 16; ++s)
                    swa::mma_ts(tDk, t + 64 + 8 * s, sdesc(q + s * 2048, 8192, 1024), idO, n > 0 || s > 0);
                mma_commit(&empty[n % L::kStages]);
                if (n + 2 < steps) ok = scores(n + 2);
            }
            mma_commit(done);
            swa::wait_bar(done, 0);
        }
    } else {
        const int grp = warp >> 2, row = (warp & 3) * 32 + lane, j = j0 + row;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const float sc = a.scale * swa::kLog2e;
        for (int n = grp; n < steps; n += 2) {
            const int st = n % L::kStages, q0 = off + ta + (n % per) * kSub;
            ok = swa::wait_bar(&full[st], (n / L::kStages) & 1);             // the statistics
            ok = ok && swa::wait_bar(&s_full[grp], (n >> 1) & 1);
            ok = __all_sync(~0u, ok);                                       // a warp leaves as one
            if (!ok) break;
            tc_fence_after();
            const uint32_t tS = tm + 128 * grp + lanes;
            const float2* stat = reinterpret_cast<const float2*>(smem + L::oStat + st * kSub * 8);
            const bool whole = j0 + kTile - 1 <= q0 && q0 + kSub - 1 - j0 < a.window;
            // queries that see key j: j <= p < j + window, or every later one if j is a sink
            const int lo = j - q0, hi = j < a.sinks ? kSub : j + a.window - q0;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float s[32], dp[32], pk[16], ds[16];
                tmem_ld32_x32(tS + 32 * c, s);
                tmem_ld32_x32(tS + 64 + 32 * c, dp);
                tmem_wait_ld();
                weights32<true>(s, dp, sc, swa::below(hi - 32 * c) & ~swa::below(lo - 32 * c), whole,
                                [&](int e) { return stat[32 * c + e]; }, pk, ds);
                tmem_st32_x16(tS + 16 * c, pk);      // over columns already read
                tmem_st32_x16(tS + 64 + 16 * c, ds);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) swa::mbar_arrive(&p_ready[grp]);
        }
        if (ok && steps > 0) ok = swa::wait_bar(done, 0);
        tc_fence_after();
        // warps 0-3 write dv, warps 4-7 dk
        const uint32_t src = (grp ? tDk : tDv) + lanes;
        const float fct = grp ? a.scale : 1.f;
        const bool in = ok && j < a.S;
        if (j0 == 0 && f.chunks > 1) {
            float* dst = f.parts + ((((size_t)hkv * f.chunks + chunk) * 2 + grp) * kTile + row) * D;
#pragma unroll
            for (int c = 0; c < D; c += 32) {
                float o[32];
                tmem_ld32_x32(src + c, o);
                tmem_wait_ld();
                if (in)
#pragma unroll
                    for (int e = 0; e < 32; e += 4)
                        *reinterpret_cast<float4*>(dst + c + e) =
                            steps > 0 ? make_float4(o[e] * fct, o[e + 1] * fct, o[e + 2] * fct, o[e + 3] * fct)
                                      : make_float4(0.f, 0.f, 0.f, 0.f);
            }
        } else {
            __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(grp ? f.dk : f.dv) + ((size_t)hkv * a.S + j) * D;
            if (steps > 0) {
                store_row<D>(dst, src, 0, D, fct, in);
            } else if (in) {
#pragma unroll
                for (int c = 0; c < D; c += 8) *reinterpret_cast<uint4*>(dst + c) = make_uint4(0, 0, 0, 0);
            }
        }
        tc_fence_before();
    }
    if (!ok) record_error(f.err, kErrTimeout);
    __syncthreads();
    if (warp == 8) tmem_dealloc(tm, 512);
}

// the sink tile's rows from its chunks, added in order
__global__ void swa_sink_reduce_kernel(const float* __restrict__ parts, int chunks, int rows, int S, int D,
                                       __nv_bfloat16* dk, __nv_bfloat16* dv) {
    const int i = blockIdx.x * blockDim.x + threadIdx.x;                 // element of [2][rows][D]
    if (i >= 2 * rows * D) return;
    const int which = i / (rows * D), r = i % (rows * D);
    const float* p = parts + ((size_t)blockIdx.y * chunks * 2 + which) * kTile * D + r;
    float s = 0.f;
    for (int c = 0; c < chunks; ++c) s += p[(size_t)c * 2 * kTile * D];
    (which ? dk : dv)[(size_t)blockIdx.y * S * D + r] = __float2bfloat16_rn(s);
}

// chunk_len: about a window, so that the sink tile's CTAs take as long as the others
int chunks_of(int T, int window, int sinks, int* len) {
    *len = T > 0 ? T : 1;
    if (sinks == 0) return 1;
    long long n = ((long long)window + kTile + kSub - 1) / kSub * kSub;
    const long long least = ((long long)T + kMaxChunks - 1) / kMaxChunks;
    if (n < least) n = (least + kSub - 1) / kSub * kSub;
    if (n >= T) return 1;
    *len = (int)n;
    return (int)((T + n - 1) / n);
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

template <int D>
cudaError_t launch(const SwaBackwardArgs& b, cudaStream_t st) {
    const SwaArgs& a = b.f;
    BwdParams f{};
    f.a = a;
    f.tpad = (a.T + kTile - 1) / kTile * kTile;
    float2* stats = static_cast<float2*>(b.workspace);
    f.stats = stats;
    f.dq = b.dq;
    f.dk = b.dk;
    f.dv = b.dv;
    f.parts = reinterpret_cast<float*>(static_cast<char*>(b.workspace) + up256((size_t)a.B * a.Hq * f.tpad * 8));
    f.chunks = chunks_of(a.T, a.window, a.sinks, &f.chunk_len);
    f.err = error_word_ptr();
    if (!f.err) return cudaErrorUnknown;
    CUtensorMap q128, do128, q64, do64, mk, mv;
    if (!swa::make_map(&q128, a.q, D, a.T, a.B * a.Hq, kTile) || !swa::make_map(&do128, b.dout, D, a.T, a.B * a.Hq, kTile) ||
        !swa::make_map(&q64, a.q, D, a.T, a.B * a.Hq, kSub) || !swa::make_map(&do64, b.dout, D, a.T, a.B * a.Hq, kSub) ||
        !swa::make_map(&mk, a.k, D, a.S, a.B * a.Hkv, kTile) || !swa::make_map(&mv, a.v, D, a.S, a.B * a.Hkv, kTile))
        return cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(swa_tc_dq_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, DqSmem<D>::bytes);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(swa_tc_dkv_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, DkvSmem<D>::bytes);
    if (e != cudaSuccess) return e;
    const int rows = 256 / (D / 8);
    const dim3 grid((f.tpad + rows - 1) / rows, a.B * a.Hq);
    const __nv_bfloat16* dout = static_cast<const __nv_bfloat16*>(b.dout);
    if (swa::few_keys(a.window, a.sinks, a.S)) swa_stats_kernel<D, true><<<grid, 256, 0, st>>>(a, dout, f.tpad, stats);
    else swa_stats_kernel<D, false><<<grid, 256, 0, st>>>(a, dout, f.tpad, stats);
    const int kt = (a.S + kTile - 1) / kTile;
#ifdef MESA_DEBUG
    f.lose = debug_lose_signal();
#endif
    swa_tc_dkv_kernel<D><<<dim3(kt - 1 + f.chunks, a.B * a.Hkv), kThreads, DkvSmem<D>::bytes, st>>>(q64, do64, mk, mv, f);
#ifdef MESA_DEBUG
    f.lose = debug_lose_signal();
#endif
    swa_tc_dq_kernel<D><<<dim3(f.tpad / kTile, a.B * a.Hq), kThreads, DqSmem<D>::bytes, st>>>(q128, do128, mk, mv, f);
    if (f.chunks > 1) {
        const int n = a.S < kTile ? a.S : kTile;
        swa_sink_reduce_kernel<<<dim3((2 * n * D + 255) / 256, a.B * a.Hkv), 256, 0, st>>>(
            f.parts, f.chunks, n, a.S, D, static_cast<__nv_bfloat16*>(f.dk), static_cast<__nv_bfloat16*>(f.dv));
    }
    return cudaGetLastError();
}

}  // namespace

size_t swa_tc_workspace_bytes(int B, int Hq, int Hkv, int T, int d, int sinks) {
    int len;
    const int chunks = chunks_of(T, 1, sinks, &len);                     // the most any window gives
    return up256((size_t)B * Hq * ((T + kTile - 1) / kTile * kTile) * 8) +
           (chunks > 1 ? up256((size_t)B * Hkv * chunks * 2 * kTile * d * 4) : 0);
}

cudaError_t swa_backward_tc(const SwaBackwardArgs& a, cudaStream_t st) {
    LaunchTimer lt(kKindSwaBwd, st);
    return a.f.d == 128 ? launch<128>(a, st) : launch<64>(a, st);
}

}  // namespace mesa
