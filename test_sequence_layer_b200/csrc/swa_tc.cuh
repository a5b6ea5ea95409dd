// swa_tc.cuh -- what the tensor-core kernels of sliding-window attention
// share: bf16 products, tensor maps, packed fp32 arithmetic.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>

#include "mesa_common.cuh"
#include "mesa_internal.h"
#include "mixers_internal.h"
#include "swa_common.cuh"
#include "tc_common.cuh"

namespace mesa {
namespace swa {

constexpr float kLog2e = 1.4426950408889634f;

// Instruction descriptor for kind::f16 with bf16 A and B, fp32 accumulator.
__host__ __device__ constexpr uint32_t idesc_bf16(int M, int N, bool a_mn, bool b_mn) {
    return tc::idesc_f16(M, N, a_mn, b_mn) | (1u << 7) | (1u << 10);
}

// D (+)= A * B^T with A in tensor memory (lane = row, each 32-bit column two
// consecutive K elements) and B in shared memory.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred q;\n setp.ne.b32 q, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, q;\n}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Tile copy from a 3-D tensor map (x: element of a row, y: row, z: head).
__device__ __forceinline__ void tma_load(void* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::
            "r"(tc::smem_addr(dst)),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(tc::smem_addr(bar))
        : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(tc::smem_addr(bar)) : "memory");
}

__device__ __forceinline__ float ex2(float v) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(v));
    return y;
}

// two fp32 operations per instruction
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(reinterpret_cast<unsigned long long&>(d))
        : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)),
          "l"(reinterpret_cast<unsigned long long&>(c)));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<unsigned long long&>(d))
        : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)));
    return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("mul.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<unsigned long long&>(d))
        : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)));
    return d;
}

// mbar_wait whose first look costs no clock read
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity) {
    uint32_t done;
    asm volatile("{\n .reg .pred w;\n mbarrier.try_wait.parity.shared::cta.b64 w, [%1], %2;\n selp.u32 %0, 1, 0, w;\n}"
                 : "=r"(done)
                 : "r"(tc::smem_addr(bar)), "r"(parity)
                 : "memory");
    return done || tc::mbar_wait(bar, parity);
}

// barrier of n threads; whether `flag` holds in any of them
__device__ __forceinline__ bool bar_any(int id, int n, bool flag) {
    uint32_t r;
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.or.pred q, %2, %3, p;\n selp.u32 %0, 1, 0, q;\n}"
        : "=r"(r)
        : "r"((uint32_t)flag), "r"(id), "r"(n)
        : "memory");
    return r;
}
__device__ __forceinline__ void bar_sync(int id, int n) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory");
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// A contiguous [z][y][x] tensor as a 3-D map of bx x by tiles; what lies past
// an end reads as zeros.
bool encode_map(CUtensorMap* m, CUtensorMapDataType type, int elem_bytes, const void* base, int x, int y, int z, int bx,
                int by, CUtensorMapSwizzle swizzle);
// bf16 [heads][rows][d] in tiles of 64 x box_rows, 128-byte swizzle
bool make_map(CUtensorMap* m, const void* base, int d, int rows, int heads, int box_rows);

}  // namespace swa
}  // namespace mesa
