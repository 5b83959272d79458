// One token of linear attention with a decay for each head:
//   S <- a S + v k^T,  out = scale S q,  a = exp(log_decay).
//
// The state's rows (V index) are independent: out_r = scale (a S_r + v_r k) . q, so one pass
// reads and writes each row once.  Bound by HBM (the state's traffic): 64 sequences x 64 heads with
// fp32 states, 541 MB, take 78 us, 6.9 TB/s; one sequence x 32 heads is a launch's latency.
//
// One CTA of 4 warps per (unit, block of 32 rows); a warp takes 8 rows with all their loads in
// flight, lane l the key channels 4 l .. 4 l + 3.
#include "kda_device.cuh"
#include "kda_ops.h"

namespace kda {
namespace {

constexpr int LD_THREADS = 128, LD_ROWS_PER_WARP = 8, LD_BLOCKS_PER_UNIT = 4;

__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
    const uint2 w = *reinterpret_cast<const uint2*>(p);
    return make_float4(bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y));
}

__global__ void __launch_bounds__(LD_THREADS) lin_decode_kernel(const LinParams p) {
    await_stream();
    const int unit = blockIdx.x / LD_BLOCKS_PER_UNIT, rb = blockIdx.x % LD_BLOCKS_PER_UNIT;
    const int b = unit / p.H, h = unit % p.H;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c0 = 4 * lane;
    const int r0 = rb * 32 + warp * LD_ROWS_PER_WARP;
    const size_t srow0 = ((size_t)unit * HD + r0) * HD + c0;
    float4 s[LD_ROWS_PER_WARP];
#pragma unroll
    for (int i = 0; i < LD_ROWS_PER_WARP; ++i) {
        const size_t off = srow0 + (size_t)i * HD;
        if (p.init_state == nullptr) s[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        else if (p.init_f32) s[i] = *reinterpret_cast<const float4*>(static_cast<const float*>(p.init_state) + off);
        else s[i] = load4(static_cast<const __nv_bfloat16*>(p.init_state) + off);
    }
    const float4 q = load4(p.q.data + b * p.q.row + h * p.q.head + c0);
    const float4 k = load4(p.k.data + b * p.k.row + h * p.k.head + c0);
    const float vr = __bfloat162float(p.v.data[b * p.v.row + h * p.v.head + r0 + (lane & 7)]);
    const float a = expf(p.log_decay[h]);
    float o[LD_ROWS_PER_WARP];
#pragma unroll
    for (int i = 0; i < LD_ROWS_PER_WARP; ++i) {
        const float v = __shfl_sync(0xffffffffu, vr, i);
        s[i].x = fmaf(s[i].x, a, v * k.x);
        s[i].y = fmaf(s[i].y, a, v * k.y);
        s[i].z = fmaf(s[i].z, a, v * k.z);
        s[i].w = fmaf(s[i].w, a, v * k.w);
        o[i] = fmaf(s[i].x, q.x, fmaf(s[i].y, q.y, fmaf(s[i].z, q.z, s[i].w * q.w)));
        if (p.final_state != nullptr) {
            const size_t off = srow0 + (size_t)i * HD;
            if (p.final_f32) *reinterpret_cast<float4*>(static_cast<float*>(p.final_state) + off) = s[i];
            else *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.final_state) + off) =
                     make_uint2(pack_bf16x2(s[i].x, s[i].y), pack_bf16x2(s[i].z, s[i].w));
        }
    }
    // the eight rows' sums over the 32 lanes: halve the rows at each of the first three steps,
    // so that lane l ends with row (l >> 4 & 1) * 4 + (l >> 3 & 1) * 2 + (l >> 2 & 1)
#pragma unroll
    for (int n = 4, bit = 16; n >= 1; n >>= 1, bit >>= 1) {
        const bool up = lane & bit;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const float give = up ? o[i] : o[i + n], keep = up ? o[i + n] : o[i];
            o[i] = keep + __shfl_xor_sync(0xffffffffu, give, bit);
        }
    }
    o[0] += __shfl_xor_sync(0xffffffffu, o[0], 2);
    o[0] += __shfl_xor_sync(0xffffffffu, o[0], 1);
    if ((lane & 3) == 0)
        p.out.data[b * p.out.row + h * p.out.head + r0 + (lane >> 2)] = __float2bfloat16_rn(p.scale * o[0]);
}

}  // namespace

cudaError_t launch_lin_decode(const LinParams& p, cudaStream_t stream) {
    const int64_t blocks = (int64_t)p.nseq * p.H * LD_BLOCKS_PER_UNIT;
    if (blocks == 0) return cudaSuccess;
    return launch_early(lin_decode_kernel, dim3((unsigned)blocks), LD_THREADS, 0, stream, p);
}

}  // namespace kda
