// swa_tc_forward.cu -- sliding-window attention forward on the tensor cores
// (bf16, d = 64 or 128).
//
// One CTA per SM takes pairs of 128-query tiles in turn and walks the 128-key
// tiles that either may see, from the newest keys back, the sinks last; the
// copies of the next pair run under the products of the present one. The pair
// is two heads that share keys where the group allows it, else two consecutive
// tiles of one head, so that every key tile fetched serves two products. One
// warp issues the tile copies, one the products, and eight warps per query tile
// do the softmax, two threads per row. Tensor memory holds S0, S1, O0, O1 (128
// columns each); P replaces the front half of its S as the bf16 left operand of
// P V.
//
// The products are issued in the order PV0(n) S0(n+1) PV1(n) S1(n+1): while
// one tile's softmax runs, the tensor pipe works for the other. (A warp for each
// tile's products interleaves them and makes both chains longer: 526 us against
// 437.) What bounds the kernel is the chain S -> softmax -> P V -> S of a tile,
// about 3700 cycles, and the issue of the products, 80 cycles each, 2560 for
// both tiles; so the softmax is made short: the maximum m of a row is only a
// reference for the exponents, set on the first tile. Later tiles take their
// exponentials on it without looking for a maximum; a row whose weights of a
// tile add up to more than 2^8 says so, and one barrier with a vote both frees
// the scores for overwriting and tells whether any row did. Only then does such
// a row move its reference and are its O and l rescaled: P stays at most 2^8,
// which costs bf16 and fp32 nothing.
// (64-key tiles with two score buffers take the chain apart, but a product of
// 128 x 64 x 16 takes the tensor pipe as long as one of 128 x 128 x 16.)
// P is rounded to bf16 for its product with v; the sum l adds it unrounded.
// Batch 4, 16 heads, 8192 tokens, d = 128, window 1024, 4 sinks: 425 us by events
// around the kernel, 467 us a pass through the public call, 600 TFLOP/s of
// visible pairs, 0.36 of the measured bf16 rate; tensor pipe 36 %,
// special-function unit 38 % busy. 96 registers a thread, about 140 bytes of them
// spilled.
// Both widths use the same columns: at d = 64 the two O take half of theirs, and
// 128 columns stay unused.
#include "swa_tc.cuh"

namespace mesa {

using namespace tc;

namespace swa {

bool encode_map(CUtensorMap* m, CUtensorMapDataType type, int elem_bytes, const void* base, int x, int y, int z, int bx,
                int by, CUtensorMapSwizzle swizzle) {
    using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static Encode encode = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &r) != cudaSuccess ||
            r != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<Encode>(f);
    }();
    if (!encode) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)x, (cuuint64_t)y, (cuuint64_t)z};
    const cuuint64_t strides[2] = {(cuuint64_t)x * elem_bytes, (cuuint64_t)x * elem_bytes * y};
    const cuuint32_t box[3] = {(cuuint32_t)bx, (cuuint32_t)by, 1}, one[3] = {1, 1, 1};
    auto attempt = [&] {
        return encode(m, type, 3, const_cast<void*>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                      CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    };
    CUresult r = attempt();
    if (r == CUDA_ERROR_INVALID_CONTEXT) {           // a host thread's first call: its device has no context here yet
        int dev;
        if (cudaGetDevice(&dev) != cudaSuccess || cudaSetDevice(dev) != cudaSuccess) return false;
        r = attempt();
    }
    return r == CUDA_SUCCESS;
}

bool make_map(CUtensorMap* m, const void* base, int d, int rows, int heads, int box_rows) {
    return encode_map(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, d, rows, heads, 64, box_rows,
                      CU_TENSOR_MAP_SWIZZLE_128B);
}

}  // namespace swa

namespace {

constexpr int kQ = 128, kK = 128;                    // rows of a query and of a key tile
constexpr int kSoftmaxWarps = 16;
constexpr int kFwdThreads = kSoftmaxWarps * 32 + 64;      // and a warp of copies, a warp of products

template <int D> struct FwdSmem {
    static constexpr int kTile = kQ * D * 2;         // bytes of a query tile
    static constexpr int kPiece = kK * D * 2;        // of a key or value tile
    static constexpr int kBlock = kK * 128;          // of 64 columns of it
    static constexpr int kStages = D == 128 ? 5 : 8;
    static constexpr int oQ = 0;                     // two query tiles
    static constexpr int oRing = 2 * kTile;          // K and V tiles, in turn
    static constexpr int oRow = oRing + kStages * kPiece;    // [2 tiles][128] floats
    static constexpr int oBar = oRow + 1024;
    static constexpr int bytes = oBar + (2 * kStages + 9) * 8 + 16 + 1008;   // + slack to align the base
    static_assert(bytes <= 227 * 1024, "more than a CTA has");
};

struct FwdParams {
    SwaArgs a;
    int pair_heads;      // 1: the two tiles are heads 2 i, 2 i + 1 of one group; 0: consecutive tiles of one head
    int nx, items;       // pairs along the queries, pairs in all
    unsigned* err;
#ifdef MESA_DEBUG
    int lose;
#endif
};

// One query tile of an item as every role of the CTA sees it.
struct QueryTile {
    int head, t0, p0, p1;                            // flat query head, first query, first and last position
    bool live;
    __device__ __forceinline__ QueryTile(const FwdParams& f, int item, int x) {
        const int blk = item % f.nx, y = item / f.nx;
        head = f.pair_heads ? 2 * y + x : y;
        t0 = (f.pair_heads ? blk : 2 * blk + x) * kQ;
        live = t0 < f.a.T;
        p0 = f.a.S - f.a.T + t0;
        p1 = f.a.S - f.a.T + min(t0 + kQ, f.a.T) - 1;
    }
    __device__ __forceinline__ bool uses(int j0, int window, int sinks) const {
        return live && j0 <= p1 && (j0 + kK > p0 - window + 1 || j0 < sinks);
    }
};

// Newest keys first: a query tile begins on its diagonal, where every row sees a
// key (where S - T is no multiple of the tile, at the second step at the latest).
__device__ __forceinline__ int key_tile(const swa::KeyTiles& kt, int i) { return kt.tile(kt.n - 1 - i); }

template <int D>
__global__ void __launch_bounds__(kFwdThreads, 1)
swa_tc_fwd_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                  const __grid_constant__ CUtensorMap mv, const FwdParams f) {
    using L = FwdSmem<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::oBar);
    uint64_t* empty = full + L::kStages;
    uint64_t* bar_q = empty + L::kStages;            // the item's query tiles have landed
    uint64_t* q_free = bar_q + 1;                    // its scores are done
    uint64_t* s_full = q_free + 1;                   // [2] scores of tile x are in tensor memory
    uint64_t* p_full = s_full + 2;                   // [2] weights of tile x are
    uint64_t* o_full = p_full + 2;                   // all products of the item done
    uint64_t* o_free = o_full + 1;                   // every warp is through with the item
    uint32_t* slot = reinterpret_cast<uint32_t*>(o_free + 1);
    float* rows = reinterpret_cast<float*>(smem + L::oRow);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const SwaArgs& a = f.a;
    if (tid == 0) {
        for (int i = 0; i < L::kStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        mbar_init(bar_q, 1);
        mbar_init(q_free, 1);
        mbar_init(o_full, 1);
        mbar_init(o_free, kSoftmaxWarps);
        for (int x = 0; x < 2; ++x) {
            mbar_init(&s_full[x], 1);
            mbar_init(&p_full[x], 8);
        }
        fence_mbar_init();
    }
    if (warp == kSoftmaxWarps) tmem_alloc(slot, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = *slot;
    // scores of tile x: columns 128 x; O of tile x: 256 + 128 x
    bool ok = true;

    if (warp == kSoftmaxWarps) {
        if (lane == 0) {
            // ---- copies: the query tiles, then K and V of every key tile ----
            int st = 0, ph = 1, k = 0;
            for (int w = blockIdx.x; w < f.items && ok; w += gridDim.x, ++k) {
                const QueryTile q0(f, w, 0), q1(f, w, 1);
                const swa::KeyTiles kt(q0.p0, q1.live ? q1.p1 : q0.p1, a.window, a.sinks, kK);
                const int hkv = q0.head / (a.Hq / a.Hkv);            // heads of one sequence follow one another
                ok = swa::wait_bar(q_free, (k & 1) ^ 1);
                if (!ok) break;
                mbar_arrive_expect_tx(bar_q, 2 * L::kTile);
                for (int x = 0; x < 2; ++x)
                    for (int c = 0; c < D / 64; ++c)
                        swa::tma_load(smem + L::oQ + x * L::kTile + c * 16384, &mq, c * 64, x ? q1.t0 : q0.t0,
                                      x ? q1.head : q0.head, bar_q);
                for (int i = 0; i < 2 * kt.n && ok; ++i) {
                    ok = swa::wait_bar(&empty[st], ph);
                    if (!ok) break;
                    mbar_arrive_expect_tx(&full[st], L::kPiece);
                    for (int c = 0; c < D / 64; ++c)
                        swa::tma_load(smem + L::oRing + st * L::kPiece + c * L::kBlock, (i & 1) ? &mv : &mk, c * 64,
                                      key_tile(kt, i >> 1) * kK, hkv, &full[st]);
                    if (++st == L::kStages) st = 0, ph ^= 1;
                }
            }
            // leave only when every copy has landed: the last of each stage and of
            // the query tiles (a parity that was never issued counts as done)
            bool landed = mbar_wait(bar_q, (k & 1) ^ 1);
            for (int i = 0; i < L::kStages && landed; ++i) landed = mbar_wait(&full[i], i < st ? ph ^ 1 : ph);
        }
    } else if (warp > kSoftmaxWarps) {
        if (lane == 0) {
            // ---- products ----
            constexpr uint32_t idS = swa::idesc_bf16(kQ, kK, false, false);
            constexpr uint32_t idO = swa::idesc_bf16(kQ, D, false, true);
            const uint64_t dq = sdesc(smem_addr(smem + L::oQ), 0, 1024);
            const uint64_t dk = sdesc(smem_addr(smem + L::oRing), 0, 1024);
            const uint64_t dv = sdesc(smem_addr(smem + L::oRing), L::kBlock, 1024);
            uint32_t np[2] = {0, 0};                 // weights taken so far, per tile
            bool first[2] = {true, true};            // of the item
            int st = 0, ph = 0;                      // ring stage of the next tile to take, its phase
            auto next_stage = [&]() {
                if (++st == L::kStages) st = 0, ph ^= 1;
            };
            // descriptors count in units of 16 bytes
            auto scores = [&](int x, int stage) {
#pragma unroll
                for (int s = 0; s < D / 16; ++s) {
                    const uint32_t o = ((s / 4) * 16384 + (s % 4) * 32) >> 4;
                    mma_f16(tm + 128 * x, dq + (x * L::kTile >> 4) + o, dk + (stage * L::kPiece >> 4) + o, idS, s > 0);
                }
#ifdef MESA_DEBUG
                if (f.lose && x == 0 && np[0] == 0) return;          // fault injection: nothing signals them
#endif
                mma_commit(&s_full[x]);
            };
            auto values = [&](int x, int stage) {
#pragma unroll
                for (int s = 0; s < kK / 16; ++s)
                    swa::mma_ts(tm + 256 + 128 * x, tm + 128 * x + 8 * s, dv + ((stage * L::kPiece + s * 2048) >> 4), idO,
                                !first[x] || s > 0);
                first[x] = false;
                ++np[x];
            };
            int k = 0;
            for (int w = blockIdx.x; w < f.items && ok; w += gridDim.x, ++k) {
                const QueryTile q0(f, w, 0), q1(f, w, 1);
                const swa::KeyTiles kt(q0.p0, q1.live ? q1.p1 : q0.p1, a.window, a.sinks, kK);
                ok = swa::wait_bar(bar_q, k & 1) && swa::wait_bar(&full[st], ph);
                if (!ok) break;
                bool use[2] = {q0.uses(key_tile(kt, 0) * kK, a.window, a.sinks),
                               q1.uses(key_tile(kt, 0) * kK, a.window, a.sinks)};
                first[0] = first[1] = true;
                // the last item's weights have been taken, in order
                if (use[0]) scores(0, st);
                if (use[1]) scores(1, st);
                mma_commit(&empty[st]);
                next_stage();
                for (int it = 0; it < kt.n && ok; ++it) {
                    const bool more = it + 1 < kt.n;
                    const int jn = key_tile(kt, it + 1) * kK;
                    const bool next[2] = {more && q0.uses(jn, a.window, a.sinks), more && q1.uses(jn, a.window, a.sinks)};
                    const int sv = st;
                    ok = swa::wait_bar(&full[st], ph);
                    next_stage();
                    if (more) ok = ok && swa::wait_bar(&full[st], ph);
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        if (use[x] && ok) {
                            ok = swa::wait_bar(&p_full[x], np[x] & 1);
                            tc_fence_after();
                            if (ok) values(x, sv);
                        }
                        if (x == 1) mma_commit(&empty[sv]);
                        if (next[x] && ok) scores(x, st);
                        use[x] = next[x];
                    }
                    if (more) {
                        mma_commit(&empty[st]);
                        next_stage();
                    }
                }
                mma_commit(q_free);
                // nobody is left an item behind: a parity tells only two phases apart
                if (k > 0 && ok) ok = swa::wait_bar(o_free, (k - 1) & 1);
                mma_commit(o_full);
            }
            // leave only when nothing is in flight any more
            if (k > 0) mbar_wait(o_full, (k - 1) & 1);
        }
    } else {
        // ---- softmax of tile x: columns 64 half .. of a row per thread. A
        // thread that gave up a wait goes on without waiting, so that the
        // others' barriers are met. ----
        const int x = warp >> 3, half = (warp >> 2) & 1;
        const int row = (warp & 3) * 32 + lane;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tS = tm + 128 * x + lanes, tO = tm + 256 + 128 * x + half * (D / 2) + lanes;
        float* shared_row = rows + x * kQ + row;     // between the two threads of a row
        auto exchange = [&](float v, auto combine) { // half 0 hands its value over and takes the result
            if (half == 0) *shared_row = v;
            swa::bar_sync(1 + x, 256);
            if (half == 1) *shared_row = v = combine(*shared_row, v);
            swa::bar_sync(1 + x, 256);
            return half == 0 ? *shared_row : v;
        };
        const float sc = a.scale * swa::kLog2e;
        constexpr float kLimit = 256.f;
        const float2 sc2 = make_float2(sc, sc);
        uint32_t n = 0;
        int k = 0;
        for (int w = blockIdx.x; w < f.items; w += gridDim.x, ++k) {
            const QueryTile q0(f, w, 0), q1(f, w, 1), q(f, w, x);
            const swa::KeyTiles kt(q0.p0, q1.live ? q1.p1 : q0.p1, a.window, a.sinks, kK);
            const int pos = q.p0 + row;
            bool begin = true;                       // the same for all threads of a tile
            float m = -INFINITY;
            float2 l2 = make_float2(0.f, 0.f);
            for (int it = 0; it < kt.n; ++it) {
                const int j0 = key_tile(kt, it) * kK;
                if (!q.uses(j0, a.window, a.sinks)) continue;
                if (ok) ok = swa::wait_bar(&s_full[x], n & 1);
                tc_fence_after();
                float s[2][32], pk[2][16];
                const bool whole = j0 + kK - 1 <= q.p0 && q.p0 + kQ - 1 - j0 < a.window;
                auto fetch = [&]() {
                    tmem_ld32_x32(tS + 64 * half, s[0]);
                    tmem_ld32_x32(tS + 64 * half + 32, s[1]);
                    tmem_wait_ld();
                    if (whole) return;
                    // bit e of a word: column 32 c + e is visible
                    const int c0 = j0 + 64 * half;
                    const int hi = pos - c0, lo = pos - a.window + 1 - c0, sk = a.sinks - c0;
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const uint32_t vis = swa::below(hi + 1 - 32 * c) & (~swa::below(lo - 32 * c) | swa::below(sk - 32 * c));
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (!(vis & (1u << e))) s[c][e] = -INFINITY;
                    }
                };
                fetch();
                float2 sum = make_float2(0.f, 0.f);
                auto weigh = [&](float neg) {
                    const float2 neg2 = make_float2(neg, neg);
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            float2 v = swa::fma2(make_float2(s[c][e], s[c][e + 1]), sc2, neg2);
                            v.x = swa::ex2(v.x);
                            v.y = swa::ex2(v.y);
                            sum = swa::add2(sum, v);
                            pk[c][e / 2] = __uint_as_float(swa::pack_bf16(v.x, v.y));
                        }
                };
                auto row_max = [&]() {
                    float t[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        t[c] = s[c / 2][16 * (c & 1)];
#pragma unroll
                        for (int e = 1; e < 16; ++e) t[c] = fmaxf(t[c], s[c / 2][16 * (c & 1) + e]);
                    }
                    return exchange(fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3])),
                                    [](float u, float v) { return fmaxf(u, v); });
                };
                if (begin) {
                    begin = false;
                    m = row_max();
                    weigh(m == -INFINITY ? 0.f : -m * sc);
                } else {
                    weigh(-m * sc);                  // NaN in a row that has seen no key yet
                    // the tile's threads agree on it, and have all read their scores; a
                    // row moves its reference on its own weights alone
                    const bool passed = !(sum.x + sum.y <= kLimit);
                    if (swa::bar_any(1 + x, 256, passed)) {
                        fetch();                     // the weights took the scores' registers
                        const bool move = exchange(passed ? 1.f : 0.f, [](float u, float v) { return fmaxf(u, v); }) > 0.f;
                        const float top = row_max();
                        float keep = 1.f;
                        if (move && top > m) {
                            keep = swa::ex2((m - top) * sc);
                            m = top;
                        }
                        if (__any_sync(~0u, keep != 1.f)) {
                            // S(n) is complete, so P V(n - 1), issued before it, is too
                            l2.x *= keep;
                            l2.y *= keep;
#pragma unroll
                            for (int c = 0; c < D / 2; c += 16) {
                                float o[16];
                                tmem_ld32_x16(tO + c, o);
                                tmem_wait_ld();
#pragma unroll
                                for (int e = 0; e < 16; ++e) o[e] *= keep;
                                tmem_st32_x16(tO + c, o);
                            }
                        }
                        sum = make_float2(0.f, 0.f);
                        weigh(m == -INFINITY ? 0.f : -m * sc);
                    }
                }
                tmem_st32_x16(tS + 32 * half, pk[0]);
                tmem_st32_x16(tS + 32 * half + 16, pk[1]);
                l2 = swa::add2(l2, sum);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) swa::mbar_arrive(&p_full[x]);
                ++n;
            }
            // ---- output ----
            float l = 1.f;
            if (q.live) l = exchange(l2.x + l2.y, [](float u, float v) { return u + v; });
            // A tile past the last query waits as well: without it its warps would
            // arrive on o_free items ahead and complete phases in the others' place.
            // It waits for the whole item, about 2 us a key tile, so it is given a
            // second for every 2^17 of them.
            if (ok) {
                int more = q.live ? 0 : kt.n >> 17;
                while (!(ok = swa::wait_bar(o_full, k & 1)) && more > 0) --more;
            }
            if (q.live) {
                const float inv = 1.f / l;
                tc_fence_after();
                const int tq = q.t0 + row;
                const bool in = tq < a.T && ok;
                const size_t r = (size_t)q.head * a.T + tq;
#pragma unroll
                for (int c = 0; c < D / 2; c += 32) {
                    float o[32];
                    tmem_ld32_x32(tO + c, o);
                    tmem_wait_ld();
                    if (in) {
                        uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + r * D + half * (D / 2) + c);
#pragma unroll
                        for (int e = 0; e < 32; e += 8)
                            dst[e / 8] = make_uint4(swa::pack_bf16(o[e] * inv, o[e + 1] * inv),
                                                    swa::pack_bf16(o[e + 2] * inv, o[e + 3] * inv),
                                                    swa::pack_bf16(o[e + 4] * inv, o[e + 5] * inv),
                                                    swa::pack_bf16(o[e + 6] * inv, o[e + 7] * inv));
                    }
                }
                if (in && half == 0 && a.lse) a.lse[r] = fmaf(m, a.scale, logf(l));
                tc_fence_before();
            }
            __syncwarp();
            if (lane == 0) swa::mbar_arrive(o_free);
        }
    }
    if (!ok) record_error(f.err, kErrTimeout);
    __syncthreads();
    if (warp == kSoftmaxWarps) tmem_dealloc(tm, 512);
}

template <int D>
cudaError_t launch(const SwaArgs& a, cudaStream_t st) {
    using L = FwdSmem<D>;
    CUtensorMap mq, mk, mv;
    if (!swa::make_map(&mq, a.q, D, a.T, a.B * a.Hq, kQ) || !swa::make_map(&mk, a.k, D, a.S, a.B * a.Hkv, kK) ||
        !swa::make_map(&mv, a.v, D, a.S, a.B * a.Hkv, kK))
        return cudaErrorInvalidValue;
    const int tiles = (a.T + kQ - 1) / kQ, pair_heads = (a.Hq / a.Hkv) % 2 == 0 ? 1 : 0;
    const int nx = pair_heads ? tiles : (tiles + 1) / 2, ny = a.B * a.Hq / (pair_heads ? 2 : 1);
    if ((long long)nx * ny > 0x7fffffffLL) return cudaErrorInvalidValue;
    FwdParams f{a, pair_heads, nx, nx * ny, error_word_ptr()};
#ifdef MESA_DEBUG
    f.lose = debug_lose_signal();
#endif
    if (!f.err) return cudaErrorUnknown;
    cudaError_t e = cudaFuncSetAttribute(swa_tc_fwd_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::bytes);
    if (e != cudaSuccess) return e;
    swa_tc_fwd_kernel<D><<<f.items < 148 ? f.items : 148, kFwdThreads, L::bytes, st>>>(mq, mk, mv, f);
    return cudaGetLastError();
}

}  // namespace

bool swa_tc_supported(int d, mesa_dtype dtype) { return dtype == MESA_BF16 && (d == 64 || d == 128); }

cudaError_t swa_forward_tc(const SwaArgs& a, cudaStream_t st) {
    LaunchTimer lt(kKindSwa, st);
    return a.d == 128 ? launch<128>(a, st) : launch<64>(a, st);
}

}  // namespace mesa
