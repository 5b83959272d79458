// Linear attention with a decay for each head over whole prompts:
//   S <- a S + v k^T,  out = scale S q,  a = exp(log_decay), token by token.
//
// One CTA of 4 warps per (sequence, head, block of 32 state rows); a warp keeps 8 rows of the
// state in registers, lane l the key channels 4 l .. 4 l + 3.  Bound by the recurrence's latency.
#include "kda_device.cuh"
#include "kda_ops.h"

namespace kda {
namespace {

constexpr int LF_THREADS = 128, LF_ROWS = 8, LF_BLOCKS = 4;

__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
    const uint2 w = *reinterpret_cast<const uint2*>(p);
    return make_float4(bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y));
}

__global__ void __launch_bounds__(LF_THREADS) lin_fwd_kernel(const LinParams p) {
    if (p.cu_seqlens) {
        bool bad = threadIdx.x == 0 && (p.cu_seqlens[0] != 0 || p.cu_seqlens[p.nseq] > p.T_total);
        for (int i = threadIdx.x; i < p.nseq; i += LF_THREADS) bad |= p.cu_seqlens[i + 1] < p.cu_seqlens[i];
        bad = __syncthreads_or(bad);
        if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = bad ? KDA_DEVERR_CU_SEQLENS : 0u;
        if (bad) return;
    } else if (blockIdx.x == 0 && threadIdx.x == 0) {
        *p.status = 0u;
    }
    if (p.nseq == 0) return;
    const int unit = blockIdx.x / LF_BLOCKS, rb = blockIdx.x % LF_BLOCKS;
    const int n = unit / p.H, h = unit % p.H;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c0 = 4 * lane;
    const int r0 = rb * 32 + warp * LF_ROWS;
    const size_t srow0 = ((size_t)unit * HD + r0) * HD + c0;
    float4 s[LF_ROWS];
#pragma unroll
    for (int i = 0; i < LF_ROWS; ++i) {
        const size_t off = srow0 + (size_t)i * HD;
        if (p.init_state == nullptr) s[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        else if (p.init_f32) s[i] = *reinterpret_cast<const float4*>(static_cast<const float*>(p.init_state) + off);
        else s[i] = load4(static_cast<const __nv_bfloat16*>(p.init_state) + off);
    }
    const int64_t bos = p.cu_seqlens ? p.cu_seqlens[n] : n * p.T, eos = p.cu_seqlens ? p.cu_seqlens[n + 1] : bos + p.T;
    const float a = expf(p.log_decay[h]);
    for (int64_t t = bos; t < eos; ++t) {
        const float4 q = load4(p.q.data + t * p.q.row + h * p.q.head + c0);
        const float4 k = load4(p.k.data + t * p.k.row + h * p.k.head + c0);
        const float vr = __bfloat162float(p.v.data[t * p.v.row + h * p.v.head + r0 + (lane & 7)]);
        float mine = 0.f;
#pragma unroll
        for (int i = 0; i < LF_ROWS; ++i) {
            const float v = __shfl_sync(0xffffffffu, vr, i);
            s[i].x = fmaf(s[i].x, a, v * k.x);
            s[i].y = fmaf(s[i].y, a, v * k.y);
            s[i].z = fmaf(s[i].z, a, v * k.z);
            s[i].w = fmaf(s[i].w, a, v * k.w);
            float o = fmaf(s[i].x, q.x, fmaf(s[i].y, q.y, fmaf(s[i].z, q.z, s[i].w * q.w)));
#pragma unroll
            for (int x = 16; x > 0; x >>= 1) o += __shfl_xor_sync(0xffffffffu, o, x);
            if (lane == i) mine = o;
        }
        if (lane < LF_ROWS) p.out.data[t * p.out.row + h * p.out.head + r0 + lane] = __float2bfloat16_rn(p.scale * mine);
    }
    if (p.final_state == nullptr) return;
#pragma unroll
    for (int i = 0; i < LF_ROWS; ++i) {
        const size_t off = srow0 + (size_t)i * HD;
        if (p.final_f32) *reinterpret_cast<float4*>(static_cast<float*>(p.final_state) + off) = s[i];
        else *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.final_state) + off) =
                 make_uint2(pack_bf16x2(s[i].x, s[i].y), pack_bf16x2(s[i].z, s[i].w));
    }
}

}  // namespace

size_t lin_workspace_bytes(int64_t, int, int) { return 0; }

cudaError_t launch_lin_fwd(const LinParams& p, cudaStream_t stream) {
    const int64_t blocks = (int64_t)p.nseq * p.H * LF_BLOCKS;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    lin_fwd_kernel<<<(unsigned)(blocks > 0 ? blocks : 1), LF_THREADS, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace kda
