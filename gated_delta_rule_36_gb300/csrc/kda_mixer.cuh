// Building blocks shared by the tensor-core mixers (kda_attn.cu, kda_lin_fwd.cu): bounded waits
// that wind a CTA down, bulk-tensor copies, tensor maps and the packed-sequence checks.
#pragma once

#include <cuda.h>

#include "kda_device.cuh"
#include "kda_ops.h"
#include "kda_sm100.cuh"

namespace kda {

// Polls before a wait gives up, after about a second: a poll of a barrier that does not complete lasts
// 4.0 us on GB300 (the hardware suspends the warp that long), one of a word in memory 0.22 us alone and 0.6 with
// 23 warps an SM.  The test build of the timeout path gives up after some milliseconds.
#ifdef KDA_WAIT_TEST
constexpr uint32_t MX_POLLS = 1u << 10, MX_MEMORY_POLLS = 1u << 14;
#else
constexpr uint32_t MX_POLLS = 1u << 18, MX_MEMORY_POLLS = 1u << 22;
#endif

// Shared-memory accesses by window address: they stay shared-memory instructions wherever the
// address comes from.
__device__ __forceinline__ uint32_t lds_u16(uint32_t a) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];\n" : "=h"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ float lds_f32(uint32_t a) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];\n" : "=f"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ float4 lds_f32x4(uint32_t a) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];\n" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ uint4 lds_u128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];\n" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ void sts_f32(uint32_t a, float v) { asm volatile("st.shared.f32 [%0], %1;\n" ::"r"(a), "f"(v) : "memory"); }
__device__ __forceinline__ void sts_u64(uint32_t a, uint32_t x, uint32_t y) {
    asm volatile("st.shared.v2.b32 [%0], {%1,%2};\n" ::"r"(a), "r"(x), "r"(y) : "memory");
}
__device__ __forceinline__ void sts_u128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};\n" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ uint32_t lds_u32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];\n" : "=r"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ void sts_u32(uint32_t a, uint32_t v) { asm volatile("st.shared.u32 [%0], %1;\n" ::"r"(a), "r"(v) : "memory"); }

// try_wait without a time hint suspends the warp in hardware; with one, the compiler builds a
// polling loop, and a CTA's many waiting warps then take half of the issue slots.
__device__ __forceinline__ bool mx_try_wait(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

// Wait for the phase with `parity`; false when the limit expires.  The caller then leaves its
// loop and its CTA reports it, the roles that wait for it run into their own limits, and
// since no named barrier is used every warp reaches the CTA's end.  The body is as small as it
// can be: a CTA's roles run different code on the same schedulers, and what they share of the
// instruction cache limits their pace (a version with a clock and an abort flag in the loop
// cost 10 % of the linear attention forward).
__device__ __forceinline__ bool mx_wait(uint32_t bar, uint32_t parity) {
    uint32_t polls = 0;
    bool ok;
    while (!(ok = mx_try_wait(bar, parity)) && ++polls < MX_POLLS) {}
    return __all_sync(0xffffffffu, ok);
}
// The same for one thread.
__device__ __forceinline__ bool mx_wait_lane(uint32_t bar, uint32_t parity) {
    uint32_t polls = 0;
    bool ok;
    while (!(ok = mx_try_wait(bar, parity)) && ++polls < MX_POLLS) {}
    return ok;
}
// A warp that gave up: time for its CTA's copies in flight to land.
__device__ __forceinline__ void mx_wind_down() {
    for (int i = 0; i < 2000; ++i) __nanosleep(1000);
}

// One arrival for a converged warp whose lanes' earlier work the arrival publishes.
__device__ __forceinline__ void mx_arrive_warp(uint32_t bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
    __syncwarp();
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void* tmap, int c0, int c1, int c2, int c3, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];\n" ::"r"(dst),
        "l"(tmap), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
        : "memory");
}

// A value that is the same in every lane, told so to the compiler: what is computed from it can
// stay in uniform registers, which is where the MMA instruction takes its operands from.
__device__ __forceinline__ int mx_uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }

// One lane of a converged warp (always the same one), as a predicate for the calls below.
__device__ __forceinline__ uint32_t mx_leader() {
    uint32_t e;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(e));
    return e;
}
// D[tmem] (+)= A B by the leader of a converged warp; A from shared memory or Tensor Memory.
__device__ __forceinline__ void mx_mma_ss(uint32_t leader, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p, e;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 e, %5, 0;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(leader)
        : "memory");
}
__device__ __forceinline__ void mx_mma_ts(uint32_t leader, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p, e;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 e, %5, 0;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(leader)
        : "memory");
}
__device__ __forceinline__ void mx_commit(uint32_t leader, uint32_t bar) {
    asm volatile(
        "{\n .reg .pred e;\n setp.ne.b32 e, %1, 0;\n"
        " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(bar), "r"(leader)
        : "memory");
}

// No use of these registers, which a load from Tensor Memory wrote, moves above this point (behind
// its wait).
__device__ __forceinline__ void mx_loaded(uint32_t (&r)[16]) {
    asm volatile("" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                      "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]));
}
__device__ __forceinline__ void mx_loaded(uint32_t (&r)[32]) {
    mx_loaded(reinterpret_cast<uint32_t(&)[16]>(r[0]));
    mx_loaded(reinterpret_cast<uint32_t(&)[16]>(r[16]));
}

// 4 consecutive 32-bit TMEM columns of this thread's lane.
__device__ __forceinline__ void tmem_st4(uint32_t taddr, const uint32_t (&r)[4]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};\n" ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
                 : "memory");
}

__device__ __forceinline__ float mx_u2f(uint32_t x) { return __uint_as_float(x); }

// cuTensorMapEncodeTiled through the runtime's driver entry point (no libcuda link).
typedef CUresult (*MxEncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                               const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                               CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline MxEncodeFn mx_encode_fn() {
    static MxEncodeFn fn = []() -> MxEncodeFn {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return nullptr;
        return reinterpret_cast<MxEncodeFn>(f);
    }();
    return fn;
}

// A bf16 tensor (128 channels, heads, rows, sequences) with strides in elements, read or
// written in boxes of 64 channels x box_heads x box_rows in the 128-byte swizzle.
inline bool mx_encode(CUtensorMap* m, const void* ptr, int64_t heads, int64_t rows, int64_t seqs, int64_t head_stride,
                      int64_t row_stride, int64_t seq_stride, int box_heads, int box_rows) {
    MxEncodeFn fn = mx_encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[4] = {(cuuint64_t)HD, (cuuint64_t)heads, (cuuint64_t)(rows > 0 ? rows : 1), (cuuint64_t)(seqs > 0 ? seqs : 1)};
    const cuuint64_t strides[3] = {(cuuint64_t)head_stride * 2, (cuuint64_t)row_stride * 2,
                                   (cuuint64_t)(seq_stride > 0 ? seq_stride : row_stride) * 2};
    const cuuint32_t box[4] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_rows, 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(ptr), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The same tensor without the sequence dimension, for stores of 64 channels x box_heads x box_rows.
inline bool mx_encode_3d(CUtensorMap* m, const void* ptr, int64_t heads, int64_t rows, int64_t head_stride, int64_t row_stride,
                         int box_heads, int box_rows) {
    MxEncodeFn fn = mx_encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)HD, (cuuint64_t)heads, (cuuint64_t)(rows > 0 ? rows : 1)};
    const cuuint64_t strides[2] = {(cuuint64_t)head_stride * 2, (cuuint64_t)row_stride * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_rows};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(ptr), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace kda
