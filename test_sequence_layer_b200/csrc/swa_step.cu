// swa_step.cu -- one decoded token of sliding-window attention over a rolling
// cache (mesa_swa_step), and the cache after a prompt (mesa_swa_cache_fill).
//
// The cache's bytes bound the step, so its slots are split over many CTAs, each
// warp with its own running maximum, sum and output rows. Two ways of joining:
//   cluster  a cluster of 1 to 16 CTAs shares a head; the parts are joined
//            through distributed shared memory, in one launch.
//   stream   the runs of 64 slots of all sequences and heads, laid end to end,
//            are cut into equal shares, one per resident CTA, whatever the
//            sequences' lengths. A head that one CTA covers is written by it;
//            the parts of the others go to the workspace and a second launch
//            joins them. Few heads over a long cache reach every SM this way,
//            and ragged batches leave none idle.
//
// 64 sequences, 16 over 4 heads, 4100 slots, d = 128: 92 us by shares, 5.1 TB/s
// (0.79 of the measured copy rate), 102 by clusters. Up to 8 MB of cache the
// cluster is as fast or faster: its one launch against two.
//
// bf16 with d = 64 or 128 rounds the softmax weights to bf16 for their product
// with v (sums, maxima and parts stay in fp32), as the forward does: a token
// decoded and the same token in a prompt carry the same roundings. Error
// against 64 bits for the batch above 0.0021, of which the output's own
// rounding is 0.0017.
//
// The fp32 kernel is plain: a thread reads a K row of its own. 64 sequences of
// 4100 slots, 4 heads of 128 columns in fp32: 917 us, 1.2 TB/s; bf16, d = 32:
// 197 us, 0.7 TB/s.
//
// The new token's rows are read from the arguments, not from the cache: their
// slot is written by one CTA while others run, and nobody reads it.
#include <cooperative_groups.h>
#include <math.h>

#include "mesa_common.cuh"
#include "mesa_internal.h"
#include "mixers_internal.h"

namespace cg = cooperative_groups;

namespace mesa {
namespace {

constexpr int kMaxSplits = 16;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ int slot_of(int p, int window, int sinks) {
    return p < sinks ? p : sinks + (p - sinks) % window;
}

// ---- parts of one CTA, joined over the cluster ----
// rows x D outputs with maximum m (in log2 units) and sum l per row
template <int ROWS, int D> struct Part {
    float o[ROWS][D];
    float m[ROWS], l[ROWS];
};

template <typename T> __device__ __forceinline__ T to_out(float v);
template <> __device__ __forceinline__ float to_out<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 to_out<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// out rows [0, rows) of the joined parts; every CTA of the cluster calls it
template <typename T, int ROWS, int D>
__device__ __forceinline__ void join(Part<ROWS, D>& part, int splits, int rank, int rows, T* out) {
    cg::cluster_group cl = cg::this_cluster();
    if (splits > 1) cl.sync(); else __syncthreads();
    for (int i = rank * blockDim.x + threadIdx.x; i < rows * D; i += splits * blockDim.x) {
        const int r = i / D, c = i % D;
        float m = -INFINITY, l = 0.f, o = 0.f;
        for (int s = 0; s < splits; ++s) {
            const Part<ROWS, D>* q = splits > 1 ? cl.map_shared_rank(&part, s) : &part;
            m = fmaxf(m, q->m[r]);
        }
        for (int s = 0; s < splits; ++s) {
            const Part<ROWS, D>* q = splits > 1 ? cl.map_shared_rank(&part, s) : &part;
            const float w = exp2f(q->m[r] - m);            // a part without slots: exp2(-inf) = 0
            l = fmaf(q->l[r], w, l);
            o = fmaf(q->o[r][c], w, o);
        }
        out[i] = to_out<T>(o / l);
    }
    if (splits > 1) cl.sync();                             // no CTA leaves while its part may be read
}

// ---- fp32 on the CUDA cores: any type, d in {16, 32, 64, 128} ----
constexpr int kSimtRows = 8, kSimtThreads = 128;

template <typename T, int D>
__global__ void __launch_bounds__(kSimtThreads) swa_step_simt_kernel(SwaStepArgs p, int splits) {
    constexpr int kParts = kSimtThreads / D;               // threads that share a channel
    __shared__ Part<kSimtRows, D> part;
    __shared__ float sq[kSimtRows][D], sw[kSimtRows][kSimtThreads], keep[kSimtRows];
    __shared__ float so[kParts][kSimtRows][D];
    const int G = p.Hq / p.Hkv, hgroups = (G + kSimtRows - 1) / kSimtRows;
    const int rank = blockIdx.x % splits, b = blockIdx.z, hk = blockIdx.y / hgroups;
    const int h0 = (blockIdx.y % hgroups) * kSimtRows, rows = min(kSimtRows, G - h0);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    T* out = static_cast<T*>(p.out) + ((size_t)b * p.Hq + hk * G + h0) * D;
    const int pos = p.pos[b];
    if (pos < 0) {                                         // the same for the whole cluster
        for (int i = rank * kSimtThreads + tid; i < rows * D; i += splits * kSimtThreads) out[i] = to_out<T>(0.f);
        return;
    }
    const int cap = p.sinks + p.window;
    const unsigned own = slot_of(pos, p.window, p.sinks), n = pos < cap - 1 ? pos + 1 : cap;
    const T* kin = static_cast<const T*>(p.k) + ((size_t)b * p.Hkv + hk) * D;
    const T* vin = static_cast<const T*>(p.v) + ((size_t)b * p.Hkv + hk) * D;
    T* kc = static_cast<T*>(p.kc) + ((size_t)b * p.Hkv + hk) * cap * D;
    T* vc = static_cast<T*>(p.vc) + ((size_t)b * p.Hkv + hk) * cap * D;
    if (rank == 0 && h0 == 0)
        for (int c = tid; c < D; c += kSimtThreads) {
            kc[(size_t)own * D + c] = kin[c];
            vc[(size_t)own * D + c] = vin[c];
        }
    for (int i = tid; i < kSimtRows * D; i += kSimtThreads) {
        const int r = i / D, c = i % D;
        sq[r][c] = r < rows ? ld_in(static_cast<const T*>(p.q), ((size_t)b * p.Hq + hk * G + h0 + r) * D + c) *
                                  (p.scale * kLog2e) : 0.f;
    }
    float o[kSimtRows];
#pragma unroll
    for (int r = 0; r < kSimtRows; ++r) o[r] = 0.f;
    if (tid < kSimtRows) part.m[tid] = -INFINITY, part.l[tid] = 0.f;
    __syncthreads();
    // unsigned: the last step starts below n < 2^31 and ends above it
    for (unsigned s0 = rank * kSimtThreads; s0 < n; s0 += splits * kSimtThreads) {
        float s[kSimtRows];
#pragma unroll
        for (int r = 0; r < kSimtRows; ++r) s[r] = 0.f;
        const unsigned slot = s0 + tid;
        if (slot < n) {
            const T* kr = slot == own ? kin : kc + (size_t)slot * D;
#pragma unroll 4
            for (int c = 0; c < D; ++c) {
                const float kv = ld_in(kr, c);
#pragma unroll
                for (int r = 0; r < kSimtRows; ++r) s[r] = fmaf(sq[r][c], kv, s[r]);
            }
        }
#pragma unroll
        for (int r = 0; r < kSimtRows; ++r) sw[r][tid] = slot < n ? s[r] : -INFINITY;
        __syncthreads();
        for (int r = warp; r < kSimtRows; r += kSimtThreads / 32) {
            float m0 = part.m[r], m = m0, l = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) m = fmaxf(m, sw[r][lane + 32 * i]);
#pragma unroll
            for (int x = 16; x; x >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, x));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float e = exp2f(sw[r][lane + 32 * i] - m);     // slot s0 is in use: m is finite
                sw[r][lane + 32 * i] = e;
                l += e;
            }
#pragma unroll
            for (int x = 16; x; x >>= 1) l += __shfl_xor_sync(~0u, l, x);
            __syncwarp();
            if (lane == 0) {
                keep[r] = exp2f(m0 - m);
                part.m[r] = m;
                part.l[r] = part.l[r] * keep[r] + l;
            }
        }
        __syncthreads();
        const int c = tid % D, first = tid / D, last = min((unsigned)kSimtThreads, n - s0);
#pragma unroll
        for (int r = 0; r < kSimtRows; ++r) o[r] *= keep[r];
        for (int i = first; i < last; i += kParts) {
            const float vv = ld_in(s0 + i == own ? vin : vc + (size_t)(s0 + i) * D, c);
#pragma unroll
            for (int r = 0; r < kSimtRows; ++r) o[r] = fmaf(sw[r][i], vv, o[r]);
        }
        __syncthreads();
    }
#pragma unroll
    for (int r = 0; r < kSimtRows; ++r) so[tid / D][r][tid % D] = o[r];
    __syncthreads();
    for (int i = tid; i < kSimtRows * D; i += kSimtThreads) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kParts; ++w) v += so[w][i / D][i % D];
        part.o[i / D][i % D] = v;
    }
    join<T, kSimtRows, D>(part, splits, rank, rows, out);
}

// ---- bf16, d in {64, 128}: warp-level matrix instructions ----
// Per 16 slots a warp forms S = Q K^T (rows: up to 8 or 16 heads, columns:
// slots) and O += P V with m16n8k16. The contraction over d and the order of
// d in the output may be permuted, so every fragment is a plain 16-byte load
// of a cache row: for S a lane takes pieces c, c + 4, ... of rows g and g + 8
// (g = lane / 4, c = lane % 4), for O piece g of rows 2c, 2c + 1, 2c + 8,
// 2c + 9, whose halves are paired with byte permutes. No shared memory and no
// barrier in the loop; the next 16 slots of K and V are in flight meanwhile.
__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ uint4 ld16(const __nv_bfloat16* p) {
    return *reinterpret_cast<const uint4*>(p);
}

// What a CTA needs to know of one head's cache.
struct Head {
    const __nv_bfloat16* q;      // first of its query heads
    const __nv_bfloat16* kin;    // the token's rows
    const __nv_bfloat16* vin;
    __nv_bfloat16* kc;
    __nv_bfloat16* vc;
    int own, n, rows;            // the token's slot, slots in use, query heads
};

template <int ROWS, int D>
__device__ __forceinline__ Head head_of(const SwaStepArgs& p, int b, int hk, int hg, int pos) {
    using bf = __nv_bfloat16;
    const int G = p.Hq / p.Hkv, cap = p.sinks + p.window, h0 = hg * ROWS;
    const size_t kv = ((size_t)b * p.Hkv + hk) * D;
    Head h;
    h.q = static_cast<const bf*>(p.q) + ((size_t)b * p.Hq + hk * G + h0) * D;
    h.kin = static_cast<const bf*>(p.k) + kv;
    h.vin = static_cast<const bf*>(p.v) + kv;
    h.kc = static_cast<bf*>(p.kc) + kv * cap;
    h.vc = static_cast<bf*>(p.vc) + kv * cap;
    h.own = slot_of(pos, p.window, p.sinks);
    h.n = pos < cap - 1 ? pos + 1 : cap;
    h.rows = min(ROWS, G - h0);
    return h;
}

template <int D> __device__ __forceinline__ void append(const Head& h) {
    if (threadIdx.x < D / 8) {
        reinterpret_cast<uint4*>(h.kc + (size_t)h.own * D)[threadIdx.x] = ld16(h.kin + threadIdx.x * 8);
        reinterpret_cast<uint4*>(h.vc + (size_t)h.own * D)[threadIdx.x] = ld16(h.vin + threadIdx.x * 8);
    }
}

// One warp's part of a head: 16 slots from s0, then every `stride` slots below
// `end`. s0 < end or nothing.
template <int ROWS, int D>
__device__ __forceinline__ void warp_part(const Head& h, float sc, int s0, int stride, int end, Part<ROWS, D>& part) {
    constexpr int kPieces = D / 32;                        // 16-byte pieces of a K row per lane
    constexpr int kSets = D / 64;                          // 64-wide runs of d in a V row
    using bf = __nv_bfloat16;
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    // rows the token's own slot or no token holds come from the arguments (the latter at weight 0)
    auto krow = [&](int slot) { return slot == h.own || slot >= h.n ? h.kin : h.kc + (size_t)slot * D; };
    auto vrow = [&](int slot) { return slot == h.own || slot >= h.n ? h.vin : h.vc + (size_t)slot * D; };
    uint4 kr[2][kPieces], vr[4][kSets];
    auto fetch_k = [&](int s) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const bf* r = krow(s + 8 * t + g);
#pragma unroll
            for (int u = 0; u < kPieces; ++u) kr[t][u] = ld16(r + (c + 4 * u) * 8);
        }
    };
    auto fetch_v = [&](int s) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bf* r = vrow(s + 2 * c + (i & 1) + 8 * (i >> 1));
#pragma unroll
            for (int u = 0; u < kSets; ++u) vr[i][u] = ld16(r + (g + 8 * u) * 8);
        }
    };
    if (s0 < end) {
        fetch_k(s0);
        fetch_v(s0);
    }
    uint4 q0[kPieces], q1[kPieces];
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
        const uint4 z = make_uint4(0, 0, 0, 0);
        const bf* qr = h.q + (c + 4 * u) * 8;
        q0[u] = g < h.rows ? ld16(qr + (size_t)g * D) : z;
        q1[u] = ROWS > 8 && g + 8 < h.rows ? ld16(qr + (size_t)(g + 8) * D) : z;
    }
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    float o[kSets * 8][4];
#pragma unroll
    for (int i = 0; i < kSets * 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
    for (; s0 < end; s0 += stride) {
        float s[2][4];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
#pragma unroll
            for (int e = 0; e < 4; ++e) s[t][e] = 0.f;
#pragma unroll
            for (int u = 0; u < kPieces; ++u) {
                mma_bf16(s[t], q0[u].x, q1[u].x, q0[u].y, q1[u].y, kr[t][u].x, kr[t][u].y);
                mma_bf16(s[t], q0[u].z, q1[u].z, q0[u].w, q1[u].w, kr[t][u].z, kr[t][u].w);
            }
        }
        const bool more = s0 + stride < end;
        if (more) fetch_k(s0 + stride);
        uint32_t pa[4] = {0, 0, 0, 0};
#pragma unroll
        for (int r = 0; r < (ROWS > 8 ? 2 : 1); ++r) {
            float v[4], mx = m[r];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int slot = s0 + 8 * (i >> 1) + 2 * c + (i & 1);
                v[i] = slot < h.n ? s[i >> 1][2 * r + (i & 1)] * sc : -INFINITY;
                mx = fmaxf(mx, v[i]);
            }
            mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 2));
            const float keep = exp2f(m[r] - mx);                     // slot s0 is in use: mx is finite
            if (__any_sync(~0u, mx > m[r])) {
#pragma unroll
                for (int i = 0; i < kSets * 8; ++i) o[i][2 * r] *= keep, o[i][2 * r + 1] *= keep;
                l[r] *= keep;
            }
            m[r] = mx;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[i] = exp2f(v[i] - mx);
                l[r] += v[i];
            }
            pa[r] = pack_bf16(v[0], v[1]);
            pa[2 + r] = pack_bf16(v[2], v[3]);
        }
#pragma unroll
        for (int u = 0; u < kSets; ++u) {
            const uint32_t* v0 = reinterpret_cast<const uint32_t*>(&vr[0][u]);
            const uint32_t* v1 = reinterpret_cast<const uint32_t*>(&vr[1][u]);
            const uint32_t* v2 = reinterpret_cast<const uint32_t*>(&vr[2][u]);
            const uint32_t* v3 = reinterpret_cast<const uint32_t*>(&vr[3][u]);
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                mma_bf16(o[8 * u + 2 * w], pa[0], pa[1], pa[2], pa[3], __byte_perm(v0[w], v1[w], 0x5410),
                         __byte_perm(v2[w], v3[w], 0x5410));
                mma_bf16(o[8 * u + 2 * w + 1], pa[0], pa[1], pa[2], pa[3], __byte_perm(v0[w], v1[w], 0x7632),
                         __byte_perm(v2[w], v3[w], 0x7632));
            }
        }
        if (more) fetch_v(s0 + stride);
    }
    // column n of tile j holds d = 64 u + 8 n + j
#pragma unroll
    for (int r = 0; r < (ROWS > 8 ? 2 : 1); ++r) {
        l[r] += __shfl_xor_sync(~0u, l[r], 1);
        l[r] += __shfl_xor_sync(~0u, l[r], 2);
        const int row = g + 8 * r;
        if (c == 0) part.m[row] = m[r], part.l[row] = l[r];
#pragma unroll
        for (int u = 0; u < kSets; ++u)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int j = 0; j < 8; j += 4)
                    *reinterpret_cast<float4*>(&part.o[row][64 * u + 8 * (2 * c + e) + j]) =
                        make_float4(o[8 * u + j][2 * r + e], o[8 * u + j + 1][2 * r + e],
                                    o[8 * u + j + 2][2 * r + e], o[8 * u + j + 3][2 * r + e]);
    }
}

// Element (r, d) of the sum of `count` parts and, where it is asked for, their
// common maximum and sum. A part without slots has m = -inf and weighs 0.
template <int ROWS, int D, typename At>
__device__ __forceinline__ float join_parts(At at, int count, int r, int d, float& m, float& l) {
    m = -INFINITY;
    for (int w = 0; w < count; ++w) m = fmaxf(m, at(w).m[r]);
    const float ref = m == -INFINITY ? 0.f : m;
    float o = 0.f;
    l = 0.f;
    for (int w = 0; w < count; ++w) {
        const Part<ROWS, D>& p = at(w);
        const float f = exp2f(p.m[r] - ref);
        o = fmaf(p.o[r][d], f, o);
        l = fmaf(p.l[r], f, l);
    }
    return o;
}

constexpr int kMmaWarps = 4, kMmaThreads = kMmaWarps * 32, kRound = kMmaWarps * 16;

// ROWS = 8 or 16 heads of the group per CTA
template <int ROWS, int D>
__global__ void __launch_bounds__(kMmaThreads, 3) swa_step_cluster_kernel(SwaStepArgs p, int splits) {
    using bf = __nv_bfloat16;
    extern __shared__ float4 smem4[];
    Part<ROWS, D>* parts = reinterpret_cast<Part<ROWS, D>*>(smem4);      // one per warp, and their sum
    const int G = p.Hq / p.Hkv, hgroups = (G + ROWS - 1) / ROWS;
    const int rank = blockIdx.x % splits, b = blockIdx.z, hk = blockIdx.y / hgroups, hg = blockIdx.y % hgroups;
    const int tid = threadIdx.x, warp = tid >> 5;
    bf* out = static_cast<bf*>(p.out) + ((size_t)b * p.Hq + hk * G + hg * ROWS) * D;
    const int pos = p.pos[b], rows = min(ROWS, G - hg * ROWS);
    if (pos < 0) {                                         // the same for the whole cluster
        for (int i = rank * kMmaThreads + tid; i < rows * D; i += splits * kMmaThreads) out[i] = to_out<bf>(0.f);
        return;
    }
    const Head h = head_of<ROWS, D>(p, b, hk, hg, pos);
    if (rank == 0 && hg == 0) append<D>(h);
    warp_part<ROWS, D>(h, p.scale * kLog2e, (rank * kMmaWarps + warp) * 16, splits * kRound, h.n, parts[warp]);
    __syncthreads();
    Part<ROWS, D>& sum = parts[kMmaWarps];
    for (int i = tid; i < rows * D; i += kMmaThreads) {
        const int r = i / D, d = i % D;
        float m, l;
        sum.o[r][d] = join_parts<ROWS, D>([&](int w) -> const Part<ROWS, D>& { return parts[w]; }, kMmaWarps, r, d, m, l);
        if (d == 0) sum.m[r] = m, sum.l[r] = l;
    }
    join<bf, ROWS, D>(sum, splits, rank, rows, out);
}

// ---- equal shares of all runs ----
constexpr int kStreamCtas = 3 * 148;                       // all resident at once

// Runs of kRound slots, numbered by sequence, then head, then slot. CTA i of n
// (n at most half their number, so that few parts are short) takes [total i / n,
// total (i + 1) / n). Its first head's part, if it shares it, goes to place 0 of
// its two, its last to place 1.
__device__ __forceinline__ int runs_of(int pos, int cap) {
    return pos < 0 ? 0 : (int)(((long long)min(pos, cap - 1) + kRound) / kRound);
}

__device__ __forceinline__ long long shares(int ctas, long long total) {
    return min((long long)ctas, (total + 1) / 2);
}

// Runs before sequence b and of all sequences (per head), by the whole block
__device__ __forceinline__ void count_runs(const int32_t* pos, int B, int b, int cap, long long& before, long long& total) {
    __shared__ long long s[2][32];
    long long x = 0, y = 0;
    for (int i = threadIdx.x; i < B; i += blockDim.x) {
        const int r = runs_of(pos[i], cap);
        y += r;
        if (i < b) x += r;
    }
#pragma unroll
    for (int k = 16; k; k >>= 1) {
        x += __shfl_xor_sync(~0u, x, k);
        y += __shfl_xor_sync(~0u, y, k);
    }
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s[0][threadIdx.x >> 5] = x, s[1][threadIdx.x >> 5] = y;
    __syncthreads();
    before = total = 0;
    for (int w = 0; w < (int)blockDim.x / 32; ++w) before += s[0][w], total += s[1][w];
}

template <int ROWS, int D>
__global__ void __launch_bounds__(kMmaThreads, 3) swa_step_stream_kernel(SwaStepArgs p, Part<ROWS, D>* places) {
    using bf = __nv_bfloat16;
    extern __shared__ float4 smem4[];
    Part<ROWS, D>* parts = reinterpret_cast<Part<ROWS, D>*>(smem4);
    __shared__ int found[2];
    const int G = p.Hq / p.Hkv, hgroups = (G + ROWS - 1) / ROWS, heads = p.Hkv * hgroups, cap = p.sinks + p.window;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    cudaTriggerProgrammaticLaunchCompletion();
    long long none, total;
    count_runs(p.pos, p.B, 0, cap, none, total);
    total *= heads;
    const long long n = shares(gridDim.x, total);
    if (blockIdx.x >= n) return;
    const long long lo = total * blockIdx.x / n, hi = total * (blockIdx.x + 1) / n;
    // the sequence that holds run lo: warp 0 walks the lengths 32 at a time
    __shared__ long long start;
    if (warp == 0) {
        long long base = 0;
        for (int i = 0; i < p.B; i += 32) {
            const long long r = i + lane < p.B ? (long long)runs_of(p.pos[i + lane], cap) * heads : 0;
            long long inc = r;
#pragma unroll
            for (int k = 1; k < 32; k <<= 1) {
                const long long t = __shfl_up_sync(~0u, inc, k);
                if (lane >= k) inc += t;
            }
            const unsigned hit = __ballot_sync(~0u, base + inc > lo);
            if (hit) {
                if (lane == __ffs(hit) - 1) found[0] = i + lane, start = base + inc - r;
                break;
            }
            base += __shfl_sync(~0u, inc, 31);
        }
    }
    __syncthreads();
    int b = found[0];
    long long at = lo, seq = start;
    int pos = p.pos[b], runs = runs_of(pos, cap);
    while (at < hi) {
        if (at >= seq + (long long)runs * heads) {           // the next sequence that has any
            seq += (long long)runs * heads;
            pos = p.pos[++b];
            runs = runs_of(pos, cap);
            continue;
        }
        const int head = (int)((at - seq) / runs), r0 = (int)((at - seq) % runs);
        const int r1 = (int)min((long long)runs, r0 + (hi - at));
        const int hk = head / hgroups, hg = head % hgroups;
        const Head h = head_of<ROWS, D>(p, b, hk, hg, pos);
        if (hg == 0 && h.own / kRound >= r0 && h.own / kRound < r1) append<D>(h);
        warp_part<ROWS, D>(h, p.scale * kLog2e, r0 * kRound + warp * 16, kRound, min(h.n, r1 * kRound), parts[warp]);
        __syncthreads();
        const bool whole = r0 == 0 && r1 == runs;
        Part<ROWS, D>& place = places[2 * blockIdx.x + (at == lo ? 0 : 1)];
        bf* out = static_cast<bf*>(p.out) + ((size_t)b * p.Hq + hk * G + hg * ROWS) * D;
        for (int i = tid; i < h.rows * D; i += kMmaThreads) {
            const int r = i / D, d = i % D;
            float m, l;
            const float o =
                join_parts<ROWS, D>([&](int w) -> const Part<ROWS, D>& { return parts[w]; }, kMmaWarps, r, d, m, l);
            if (whole) {
                out[i] = to_out<bf>(o / l);
            } else {
                place.o[r][d] = o;
                if (d == 0) place.m[r] = m, place.l[r] = l;
            }
        }
        __syncthreads();
        at += r1 - r0;
    }
}

// The heads that several of the n CTAs share, and zeros for idle rows: one
// block per row, its groups of D threads taking parts in turn.
template <int ROWS, int D, int kJoinThreads>
__global__ void __launch_bounds__(kJoinThreads) swa_step_join_kernel(SwaStepArgs p, const Part<ROWS, D>* places, int ctas) {
    using bf = __nv_bfloat16;
    constexpr int kGroups = kJoinThreads / D;
    __shared__ float weight[kStreamCtas], sum[kGroups][D], red[2][32];
    const int G = p.Hq / p.Hkv, hgroups = (G + ROWS - 1) / ROWS, heads = p.Hkv * hgroups, cap = p.sinks + p.window;
    const int tid = threadIdx.x, b = blockIdx.y, hk = blockIdx.x / G, qh = blockIdx.x % G, r = qh % ROWS;
    const int head = hk * hgroups + qh / ROWS, runs = runs_of(p.pos[b], cap);
    bf* out = static_cast<bf*>(p.out) + ((size_t)b * p.Hq + blockIdx.x) * D;
    long long before, total;
    count_runs(p.pos, p.B, b, cap, before, total);
    if (runs == 0) {
        cudaGridDependencySynchronize();
        if (tid < D) out[tid] = to_out<bf>(0.f);
        return;
    }
    total *= heads;
    const long long n = shares(ctas, total);
    const long long s = before * heads + (long long)head * runs, e = s + runs;
    const long long i0 = ((s + 1) * n - 1) / total, i1 = (e * n - 1) / total;       // the CTAs of its first and last run
    cudaGridDependencySynchronize();                        // the parts are complete
    if (i0 == i1) return;
    const int lead = s == total * i0 / n ? 0 : 1;           // place of the first CTA's part
    const int count = (int)(i1 - i0 + 1);                   // <= ctas = kStreamCtas
    auto part = [&](int w) -> const Part<ROWS, D>& { return places[2 * (i0 + w) + (w == 0 ? lead : 0)]; };
    // every thread holds the maximum and sum of up to kMine parts
    constexpr int kMine = (kStreamCtas + kJoinThreads - 1) / kJoinThreads;
    float pm[kMine], pl[kMine], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
        const int w = tid + i * kJoinThreads;
        pm[i] = w < count ? part(w).m[r] : -INFINITY;
        pl[i] = w < count ? part(w).l[r] : 0.f;
        m = fmaxf(m, pm[i]);
    }
#pragma unroll
    for (int k = 16; k; k >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, k));
    if ((tid & 31) == 0) red[0][tid >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kJoinThreads / 32; ++w) m = fmaxf(m, red[0][w]);           // finite: every run has a slot
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
        const int w = tid + i * kJoinThreads;
        const float f = exp2f(pm[i] - m);
        if (w < count) weight[w] = f;
        l = fmaf(pl[i], f, l);
    }
#pragma unroll
    for (int k = 16; k; k >>= 1) l += __shfl_xor_sync(~0u, l, k);
    if ((tid & 31) == 0) red[1][tid >> 5] = l;
    __syncthreads();
    float o = 0.f;
#pragma unroll 16
    for (int w = tid / D; w < count; w += kGroups) o = fmaf(part(w).o[r][tid % D], weight[w], o);
    sum[tid / D][tid % D] = o;
    __syncthreads();
    if (tid >= D) return;
    l = 0.f, o = 0.f;
    for (int w = 0; w < kJoinThreads / 32; ++w) l += red[1][w];
#pragma unroll
    for (int w = 0; w < kGroups; ++w) o += sum[w][tid];
    out[tid] = to_out<bf>(o / l);
}

// ---- rolling cache of a prompt ----
__global__ void swa_cache_fill_kernel(const uint4* __restrict__ k, const uint4* __restrict__ v, uint4* kc, uint4* vc,
                                      const int32_t* __restrict__ lens, int Hkv, int S, int units, int window,
                                      int sinks, int start) {
    const int bh = blockIdx.y, b = bh / Hkv, cap = sinks + window;
    const int len = lens ? min(max(lens[b], 0), S) : S;
    const int end = start + len;
    const size_t total = (size_t)cap * units;
    for (size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += (size_t)gridDim.x * blockDim.x) {
        const int slot = (int)(i / units), u = (int)(i % units);
        int p = slot;                                     // the last position before end that lives in the slot
        if (slot >= sinks) {
            const int last = end - 1 - slot;              // counted from the slot's first position
            if (last < 0) continue;
            p = slot + last / window * window;
        }
        if (p < start || p >= end) continue;
        const size_t src = ((size_t)bh * S + (p - start)) * units + u;
        kc[(size_t)bh * total + i] = k[src];
        vc[(size_t)bh * total + i] = v[src];
    }
}

// CTAs per head and sequence, in a cluster: doubled while the grid is below
// three CTAs per SM and every CTA's warps still get a run of slots
int splits_for(long long blocks, int slots_per_round, long long slots) {
    int n = 1;
    while (n < kMaxSplits && blocks * n < 3 * 148 && 2LL * n * slots_per_round <= slots) n *= 2;
    return n;
}

template <typename F>
cudaError_t launch_cluster(F* kernel, const SwaStepArgs& a, int hgroups, int slots_per_round, int threads, int smem,
                           cudaStream_t st) {
    const int splits = splits_for((long long)a.B * a.Hkv * hgroups, slots_per_round, (long long)a.sinks + a.window);
    if (splits > 8) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(splits, a.Hkv * hgroups, a.B);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = splits;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = splits > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, a, splits);
}

bool use_mma(const SwaStepArgs& a) { return a.dtype == MESA_BF16 && (a.d == 64 || a.d == 128); }

// Both launches against the cluster's one, events around a call: 15.4 us against
// 13.2 at 4 MB (8 heads of 1028 slots), 15.4 against 12.4 at 7.9 MB (32 heads of
// 504), 15.3 against 16.1 at 8.0 MB (8 heads of 2048), 20 against 30 at 16.8 MB.
bool use_stream(const SwaStepArgs& a) {
    return use_mma(a) && (long long)a.B * a.Hkv * ((long long)a.sinks + a.window) * a.d * 4 >= (8LL << 20);
}

template <int ROWS, int D>
cudaError_t step_mma(const SwaStepArgs& a, cudaStream_t st) {
    const int hgroups = (a.Hq / a.Hkv + ROWS - 1) / ROWS;
    if (!use_stream(a)) {
        constexpr int smem = (int)sizeof(Part<ROWS, D>) * (kMmaWarps + 1);
        static_assert(smem <= 48 * 1024, "no opt-in needed");
        return launch_cluster(swa_step_cluster_kernel<ROWS, D>, a, hgroups, kRound, kMmaThreads, smem, st);
    }
    Part<ROWS, D>* places = static_cast<Part<ROWS, D>*>(a.workspace);
    swa_step_stream_kernel<ROWS, D><<<kStreamCtas, kMmaThreads, sizeof(Part<ROWS, D>) * kMmaWarps, st>>>(a, places);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    // about this many parts a head: a block's threads share long lists of them
    const bool many = kStreamCtas / ((long long)a.B * a.Hkv * hgroups) >= 16;
    const int threads = many ? 1024 : 128;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.Hq, a.B);
    cfg.blockDim = dim3(threads);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, many ? swa_step_join_kernel<ROWS, D, 1024> : swa_step_join_kernel<ROWS, D, 128>, a,
                              static_cast<const Part<ROWS, D>*>(places), kStreamCtas);
}

template <typename T, int D>
cudaError_t step_simt_d(const SwaStepArgs& a, cudaStream_t st) {
    return launch_cluster(swa_step_simt_kernel<T, D>, a, (a.Hq / a.Hkv + kSimtRows - 1) / kSimtRows, kSimtThreads,
                          kSimtThreads, 0, st);
}

// bf16 of 64 and 128 columns never comes here: the matrix instructions take it
cudaError_t step_simt(const SwaStepArgs& a, cudaStream_t st) {
    using bf = __nv_bfloat16;
    if (a.dtype == MESA_BF16) return a.d == 16 ? step_simt_d<bf, 16>(a, st) : step_simt_d<bf, 32>(a, st);
    switch (a.d) {
        case 16: return step_simt_d<float, 16>(a, st);
        case 32: return step_simt_d<float, 32>(a, st);
        case 64: return step_simt_d<float, 64>(a, st);
        default: return step_simt_d<float, 128>(a, st);
    }
}

}  // namespace

size_t swa_step_workspace_bytes(const SwaStepArgs& a) {
    if (!use_stream(a)) return 0;
    const size_t row = (size_t)(a.d + 2) * sizeof(float);
    return 2 * kStreamCtas * (a.Hq / a.Hkv > 8 ? 16 : 8) * row;
}

cudaError_t swa_step(const SwaStepArgs& a, cudaStream_t st) {
    LaunchTimer lt(kKindSwaStep, st);
    if (!use_mma(a)) return step_simt(a, st);
    const bool wide = a.Hq / a.Hkv > 8;
    if (a.d == 128) return wide ? step_mma<16, 128>(a, st) : step_mma<8, 128>(a, st);
    return wide ? step_mma<16, 64>(a, st) : step_mma<8, 64>(a, st);
}

cudaError_t swa_cache_fill(const void* k, const void* v, void* kc, void* vc, const int32_t* lens, int B, int Hkv,
                           int S, int d, int window, int sinks, int start, mesa_dtype dtype, cudaStream_t st) {
    LaunchTimer lt(kKindSwaStep, st);
    const int units = d * (dtype == MESA_F32 ? 4 : 2) / 16;
    const size_t total = (size_t)(sinks + window) * units;
    const unsigned gx = (unsigned)((total + 255) / 256 < 4096 ? (total + 255) / 256 : 4096);
    swa_cache_fill_kernel<<<dim3(gx, B * Hkv), 256, 0, st>>>(static_cast<const uint4*>(k), static_cast<const uint4*>(v),
                                                             static_cast<uint4*>(kc), static_cast<uint4*>(vc), lens, Hkv,
                                                             S, units, window, sinks, start);
    return cudaGetLastError();
}

}  // namespace mesa
