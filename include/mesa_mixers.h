/*
 * mesa_mixers.h -- C ABI of the sequence mixers that stand beside the Mesa
 * layer in a hybrid stack (libmesa_b200.so): a gated linear recurrence
 * (mesa_lru_*) and causal sliding-window attention with sink tokens
 * (mesa_swa_*). The MesaNet pages name both beside their layer: the
 * "Hawk-Mesa" hybrid (Architecture) and the sliding-window baseline (Results).
 *
 * Conventions are those of mesa.h: device pointers owned by the caller,
 * contiguous row-major tensors, no allocation inside a call, work enqueued on
 * `stream` without synchronising, status codes, arguments checked on the host
 * before any launch. The calling thread's current device must own the
 * pointers. Outputs must not overlap inputs or each other
 * (MESA_ERR_INVALID_ARG) unless stated otherwise. Every result is
 * bit-reproducible from call to call: no floating-point atomics are used.
 * Make one call on a device before capturing calls into a graph there (the
 * first looks up the device's error word). Several host threads may call at
 * once, with workspaces of their own. A kernel that gives up a bounded
 * wait records MESA_ERR_DEVICE_TIMEOUT for mesa_get_error(); its outputs are
 * then undefined.
 */
#ifndef MESA_MIXERS_H
#define MESA_MIXERS_H

#include "mesa.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Gated linear recurrence (real-gated linear recurrent unit). Per channel c
 * of D, with the learned lambda [D]:
 *     r_t = sigmoid(gate_a_t),  i_t = sigmoid(gate_x_t)
 *     log a_t = -8 softplus(lambda) r_t
 *     h_t = a_t h_{t-1} + sqrt(1 - a_t^2) i_t x_t,     y_t = h_t
 * 1 - a^2 is formed from log a without cancellation, so gates that close
 * (r -> 0, a -> 1) hold the state. gate_a = -inf holds it exactly.
 *
 *   x, gate_a, gate_x   [B,T,D] in `dtype`, aligned to their element.
 *   lambda              float32 [D].
 *   B, T, D             B, D >= 1, T >= 0 (T = 0: only h_T is written, h0 or
 *                       zeros); B*T*D is not limited by 32 bits.
 *   h0                  float32 [B,D] initial state or NULL (zero).
 *   y                   [B,T,D] in `dtype` (the fp32 state rounded once).
 *   h_T                 float32 [B,D] final state or NULL. May be h0 itself.
 *   saved               NULL, or mesa_lru_saved_size() bytes, 4-byte aligned:
 *                       the fp32 state before every 64th token,
 *                       [B, ceil(T/64), D], which mesa_lru_backward takes.
 */
size_t mesa_lru_saved_size(int B, int T, int D);
mesa_status mesa_lru_forward(const void* x, const void* gate_a, const void* gate_x, const float* lambda,
                             int B, int T, int D, mesa_dtype dtype, const float* h0, void* y, float* h_T,
                             float* saved, void* stream);

/*
 * Gradients of mesa_lru_forward. With g_t = dL/dh_t (dy_t plus what later
 * tokens send back, a_{t+1} g_{t+1}; dh_T joins at the last token):
 *     dx = g m i,  dgate_x = g m x i (1 - i)          (m = sqrt(1 - a^2))
 *     dlog a = g (a h_{t-1} - i x a^2 / m),  dgate_a = dlog a log a (1 - r)
 *     dlambda = sigmoid(lambda) / softplus(lambda) sum_{b,t} dlog a log a
 *     dh0 = a_1 g_1
 * The limit log a -> 0 of log a / m is taken as 0.
 *
 *   saved        as mesa_lru_forward left it for the same inputs, or NULL: it
 *                is then recomputed in the workspace from x, the gates and h0.
 *   h0           used only where saved is NULL (NULL: zero).
 *   dy           [B,T,D] in `dtype`.   dh_T  float32 [B,D] or NULL (zero).
 *   dx, dgate_a, dgate_x   [B,T,D] in `dtype`.
 *   dlambda      float32 [D].          dh0   float32 [B,D] or NULL.
 *   workspace    mesa_lru_backward_workspace_size() bytes, 256-byte aligned.
 * T = 0 writes dlambda = 0 and dh0 = dh_T (or zeros).
 */
size_t mesa_lru_backward_workspace_size(int B, int T, int D, mesa_dtype dtype, int have_saved);
mesa_status mesa_lru_backward(const void* x, const void* gate_a, const void* gate_x, const float* lambda,
                              int B, int T, int D, mesa_dtype dtype, const float* h0, const float* saved,
                              const void* dy, const float* dh_T, void* dx, void* dgate_a, void* dgate_x,
                              float* dlambda, float* dh0, void* workspace, size_t ws_bytes, void* stream);

/*
 * One decoded token: h_out = a h_in + m i x, y = h_out in `dtype`.
 * x, gate_a, gate_x, y: [B,D]; h_in, h_out: float32 [B,D], and h_out may be
 * h_in (the state in place).
 */
mesa_status mesa_lru_step(const void* x, const void* gate_a, const void* gate_x, const float* lambda,
                          int B, int D, mesa_dtype dtype, const float* h_in, float* h_out, void* y, void* stream);

/*
 * Causal attention over a sliding window, with the first `sinks` tokens
 * visible to every later one. The T queries are the last T of S positions
 * (query t is position p = S - T + t), and p sees key j if
 *     j <= p  and  (p - j < window  or  j < sinks).
 * out = softmax(scale q k^T) v over the visible keys; lse = their
 * log-sum-exp (natural logarithm). Every query sees at least its own key.
 * Values are finite (not checked, the caller's contract): a hidden key enters
 * the product with v at weight 0, so a NaN or infinity in its row of v also
 * reaches nearby queries that do not see it. A padded row therefore holds any
 * finite value; causality keeps it from the rows before it.
 *
 *   q, out       [B,Hq,T,d] in `dtype`;  k, v [B,Hkv,S,d]; 16-byte aligned.
 *   Hq, Hkv      Hq a multiple of Hkv: query head h reads head h / (Hq/Hkv).
 *   T, S         0 <= T <= S.
 *   d            16, 32, 64 or 128. MESA_BF16 with d = 64 or 128 runs on the
 *                tensor cores (the softmax weights round to bf16 before their
 *                product with v; sums and statistics are fp32), everything
 *                else in fp32 on the CUDA cores.
 *   window       >= 1 (S or more: plain causal attention).
 *   sinks        0..128.
 *   scale        finite, and > 0.
 *   lse          float32 [B,Hq,T] or NULL.
 * B * Hq <= 65535.
 */
mesa_status mesa_swa_forward(const void* q, const void* k, const void* v, int B, int Hq, int Hkv, int T, int S,
                             int d, int window, int sinks, float scale, mesa_dtype dtype, void* out, float* lse,
                             void* stream);

/*
 * Gradients of mesa_swa_forward for the same arguments, from its out and lse:
 *     P = exp(scale q k^T - lse),  dP = dout v^T,  delta = rowsum(dout * out)
 *     dS = scale P (dP - delta),  dq = dS k,  dk = dS^T q,  dv = P^T dout
 * (dk, dv summed over the query heads that share a head).
 *   dq [B,Hq,T,d];  dk, dv [B,Hkv,S,d]; all in `dtype`, rounded once.
 *   workspace    mesa_swa_backward_workspace_size() bytes, 256-byte aligned.
 * MESA_BF16 with d = 64 or 128: P and dS round to bf16 before their products.
 * Keys that no query sees get zero gradients (T < S, or T = 0); where every
 * query of the call sees one key alone (S = 1, or a window of 1 without
 * sinks), dq and dk are exactly zero. In other calls the gradients of a query
 * that sees one key are zero up to the rounding of dP - delta.
 */
size_t mesa_swa_backward_workspace_size(int B, int Hq, int Hkv, int T, int S, int d, int sinks, mesa_dtype dtype);
mesa_status mesa_swa_backward(const void* q, const void* k, const void* v, const void* out, const float* lse,
                              const void* dout, int B, int Hq, int Hkv, int T, int S, int d, int window, int sinks,
                              float scale, mesa_dtype dtype, void* dq, void* dk, void* dv, void* workspace,
                              size_t ws_bytes, void* stream);

/*
 * One decoded token over rolling caches of sinks + window slots: position p
 * lives in slot p while p < sinks, else in slot sinks + (p - sinks) mod
 * window, so the used slots are exactly the positions p may see. For every
 * sequence b with position pos[b] >= 0: k[b], v[b] go into their slot, then
 * out[b] = the attention of q[b] over the used slots (pos[b] + 1 of them, at
 * most sinks + window). pos[b] < 0 marks an idle row: its caches stay as they
 * are and out[b] is zero.
 *
 *   q, out            [B,Hq,d] in `dtype`;  k, v [B,Hkv,d].
 *   k_cache, v_cache  [B,Hkv,sinks+window,d] in `dtype`, updated in place.
 *                     Slots not yet used are not read.
 *   pos               int32 [B], device memory (a captured call follows it).
 *   workspace         mesa_swa_step_workspace_size() bytes, 256-byte aligned
 *                     (that may be 0: then it may be NULL). Calls sharing a
 *                     workspace must not overlap.
 * All others 16-byte aligned (pos 4). d, sinks, scale as above; window >= 1;
 * sinks + window < 2^31; B * Hq <= 65535. MESA_BF16 with d = 64 or 128: the
 * softmax weights round to bf16 before their product with v, as in the forward.
 */
size_t mesa_swa_step_workspace_size(int B, int Hq, int Hkv, int d, int window, int sinks, mesa_dtype dtype);
mesa_status mesa_swa_step(const void* q, const void* k, const void* v, void* k_cache, void* v_cache,
                          const int32_t* pos, int B, int Hq, int Hkv, int d, int window, int sinks, float scale,
                          mesa_dtype dtype, void* out, void* workspace, size_t ws_bytes, void* stream);

/*
 * The rolling caches after the S tokens k, v [B,Hkv,S,d] at positions start,
 * start + 1, ...: every slot receives the last of these positions that maps
 * to it, and slots that none maps to stay as they are. lens: int32 [B] device
 * memory or NULL; sequence b then has min(max(lens[b], 0), S) tokens, and the
 * rows behind are not read. start + S <= 2^31 - 1.
 */
mesa_status mesa_swa_cache_fill(const void* k, const void* v, void* k_cache, void* v_cache, const int32_t* lens,
                                int B, int Hkv, int S, int d, int window, int sinks, int start, mesa_dtype dtype,
                                void* stream);

#ifdef MESA_DEBUG
/*
 * Debug builds only: fault injection for the failure-detection tests. In the
 * next `launches` launches of this file's kernels with bounded waits (the
 * recurrence's forward and backward, the tensor-core attention kernels) one
 * signal per CTA never comes: a tile copy of a cluster's first CTA, or the
 * completion of the first scores. The waits on it run out (about one second of
 * clock cycles each), the kernel records a timeout in the error word, lets its
 * copies and products drain and returns; its outputs are then undefined.
 * Returns MESA_ERR_INVALID_ARG for launches < 0.
 */
mesa_status mesa_debug_lose_signal(int launches);
#endif

#ifdef __cplusplus
}
#endif
#endif /* MESA_MIXERS_H */
