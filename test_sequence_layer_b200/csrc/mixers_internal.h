// mixers_internal.h -- host-side declarations of the gated linear recurrence
// and the sliding-window attention (mesa_mixers.h).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "mesa_mixers.h"

namespace mesa {

constexpr int kLruSave = 64;       // tokens between saved states
constexpr int kLruMaxCluster = 16;  // CTAs that share one sequence's time axis

#ifdef MESA_DEBUG
int debug_lose_signal();           // 1 if the launch at hand is to lose a signal
#endif

struct LruArgs {
    const void* x;
    const void* ga;
    const void* gx;
    const float* lambda;
    int B, T, D;
    mesa_dtype dtype;
    const float* h0;
    void* y;                // nullptr: the states only
    float* hT;
    float* saved;
#ifdef MESA_DEBUG
    int lose = 0;
#endif
};
struct LruBackwardArgs {
    LruArgs f;              // f.saved holds the states (read)
    const void* dy;
    const float* dhT;
    void* dx;
    void* dga;
    void* dgx;
    float* dlambda;
    float* dh0;
    float* partial;         // [lru_backward_rows][D]
};
cudaError_t lru_forward(const LruArgs& a, cudaStream_t st);
cudaError_t lru_backward(const LruBackwardArgs& a, cudaStream_t st);
size_t lru_backward_rows(int B, int T);   // most rows of partial sums of dlambda
cudaError_t lru_step(const void* x, const void* ga, const void* gx, const float* lambda, int B, int D,
                     mesa_dtype dtype, const float* h_in, float* h_out, void* y, cudaStream_t st);

struct SwaArgs {
    const void* q;
    const void* k;
    const void* v;
    int B, Hq, Hkv, T, S, d, window, sinks;   // window <= max(S, 1)
    float scale;
    mesa_dtype dtype;
    void* out;              // written by the forward, read by the backward
    float* lse;             // written by the forward (or nullptr), read by the backward
};
struct SwaBackwardArgs {
    SwaArgs f;
    const void* dout;
    void* dq;
    void* dk;
    void* dv;
    void* workspace;
};
// tensor cores: bf16, d = 64 or 128 (swa_tc_forward.cu)
bool swa_tc_supported(int d, mesa_dtype dtype);
cudaError_t swa_forward_tc(const SwaArgs& a, cudaStream_t st);
cudaError_t swa_forward_simt(const SwaArgs& a, cudaStream_t st);
size_t swa_simt_workspace_bytes(int B, int Hq, int Hkv, int T, int S, int d, int sinks);
cudaError_t swa_backward_simt(const SwaBackwardArgs& a, cudaStream_t st);
// tensor cores (swa_tc_backward.cu)
size_t swa_tc_workspace_bytes(int B, int Hq, int Hkv, int T, int d, int sinks);
cudaError_t swa_backward_tc(const SwaBackwardArgs& a, cudaStream_t st);
// delta [B,Hq,T] = rowsum(dout * out)
cudaError_t swa_delta(const SwaArgs& a, const void* dout, float* delta, cudaStream_t st);

struct SwaStepArgs {
    const void* q;
    const void* k;
    const void* v;
    void* kc;
    void* vc;
    const int32_t* pos;
    int B, Hq, Hkv, d, window, sinks;
    float scale;
    mesa_dtype dtype;
    void* out;
    void* workspace;
};
size_t swa_step_workspace_bytes(const SwaStepArgs& a);        // sizes and type of a matter
cudaError_t swa_step(const SwaStepArgs& a, cudaStream_t st);
cudaError_t swa_cache_fill(const void* k, const void* v, void* kc, void* vc, const int32_t* lens, int B, int Hkv,
                           int S, int d, int window, int sinks, int start, mesa_dtype dtype, cudaStream_t st);

}  // namespace mesa
