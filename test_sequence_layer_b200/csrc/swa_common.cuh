// swa_common.cuh -- the mask of sliding-window attention and the tile ranges
// that follow from it, shared by its kernels.
//
// Query t sits at position p = S - T + t and sees key j if j <= p and
// (p - j < window or j < sinks). window <= S, so no sum here overflows.
#pragma once

#include <stdint.h>

namespace mesa {
namespace swa {

__device__ __forceinline__ bool visible(int p, int j, int window, int sinks) {
    return j <= p && (p - j < window || j < sinks);
}

// The backward's delta = rowsum(dout o out) takes out as rounded to bf16. With a
// handful of visible keys dP - delta is small against delta, and that rounding
// would show (twice the error of dS's own rounding at two keys, a half at
// eight); up to kFewKeys of them delta is summed from the weights instead,
// sum_j P_j dP_j. Key i of the n that position p sees:
constexpr int kFewKeys = 8;
struct FewKeys {
    int sinks, lo, n, p;
    __device__ __forceinline__ FewKeys(int p_, int window, int all_sinks) : p(p_) {
        lo = p - window + 1 > 0 ? p - window + 1 : 0;
        sinks = all_sinks < lo ? all_sinks : lo;
        n = sinks + p - lo + 1;
    }
    __device__ __forceinline__ int key(int i) const {
        const int j = lo + i - sinks;
        return i < sinks ? i : j < p ? j : p;          // past the last: some key that exists
    }
};
__host__ __forceinline__ bool few_keys(int window, int sinks, int S) {
    return (window + sinks < S ? window + sinks : S) <= kFewKeys;
}

// the n lowest bits of a word
__device__ __forceinline__ uint32_t below(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; }

// The key tiles (of `bn` keys) that queries at positions [p0, p1] may see: the
// sink tiles [0, n_sink) and the window tiles [first, last], without overlap.
struct KeyTiles {
    int n_sink, first, n;                       // n = n_sink + window tiles
    __device__ __forceinline__ KeyTiles(int p0, int p1, int window, int sinks, int bn) {
        const int lo = p0 - window + 1;
        first = lo > 0 ? lo / bn : 0;
        const int s = sinks > p1 + 1 ? p1 + 1 : sinks;
        n_sink = (s + bn - 1) / bn;
        if (n_sink > first) n_sink = first;
        n = n_sink + p1 / bn - first + 1;
    }
    __device__ __forceinline__ int tile(int i) const { return i < n_sink ? i : first + i - n_sink; }
};

// Query indices [t0, t1) that may see a key of [j0, j1]; `far` is whether the
// keys hold a sink, which every later query sees.
__device__ __forceinline__ void query_range(int j0, int j1, int T, int S, int window, int sinks, int& t0, int& t1) {
    const int off = S - T;
    t0 = j0 > off ? j0 - off : 0;
    const int end = j1 - off + window;          // last window query + 1
    t1 = (j0 < sinks || end > T) ? T : end;
    if (t1 < t0) t1 = t0;
}

}  // namespace swa
}  // namespace mesa
