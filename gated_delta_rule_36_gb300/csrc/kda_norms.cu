// The norms around a mixer: RMS norm of every head of its output times its activated gate, and the
// norm after a block, its gate and residual scale, the residual sum and the norm before the next block.
#include "kda_device.cuh"
#include "kda_ops.h"

namespace kda {
namespace {

__device__ __forceinline__ void unpack8(const uint4 r, float (&f)[8]) {
    f[0] = bf16_lo(r.x); f[1] = bf16_hi(r.x); f[2] = bf16_lo(r.y); f[3] = bf16_hi(r.y);
    f[4] = bf16_lo(r.z); f[5] = bf16_hi(r.z); f[6] = bf16_lo(r.w); f[7] = bf16_hi(r.w);
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}
__device__ __forceinline__ void load8(const float* p, float (&f)[8]) {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}

// ---------------------------------------------------------------- the norm and gate of a mixer's output
// A half-warp takes a (token, head) row: lane l holds elements 8 l .. 8 l + 7.
constexpr int GN_THREADS = 128, GN_HALVES = GN_THREADS / 16;

template <int kRows>
__global__ void __launch_bounds__(GN_THREADS) gated_norm_kernel(const GatedNormParams p, int groups) {
    await_stream();
    const int lane = threadIdx.x & 15;
    const int64_t item = (int64_t)blockIdx.x * GN_HALVES + (threadIdx.x >> 4);
    const int64_t t = item / groups;
    const int h0 = (int)(item - t * groups) * kRows;
    const int rows = t >= p.tokens ? 0 : min(p.heads - h0, kRows);
    uint4 x[kRows], g[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        x[i] = g[i] = make_uint4(0, 0, 0, 0);
        if (i < rows) {
            x[i] = __ldcs(reinterpret_cast<const uint4*>(p.x.data + t * p.x.row + (h0 + i) * p.x.head + 8 * lane));
            g[i] = __ldcs(reinterpret_cast<const uint4*>(p.gate.data + t * p.gate.row + (h0 + i) * p.gate.head + 8 * lane));
        }
    }
    float w[8];
    if (p.weight) load8(p.weight + 8 * lane, w);
    else {
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = 1.f;
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        float v[8], a[8];
        unpack8(x[i], v);
        unpack8(g[i], a);
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(v[j], v[j], ss);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float r = rsqrtf(ss * (1.f / HD) + p.eps);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float s = rcp_approx(1.f + ex2_approx(-LOG2E * a[j]));
            v[j] *= r * w[j] * (p.silu ? a[j] * s : s);
        }
        if (i < rows) __stcs(reinterpret_cast<uint4*>(p.out.data + t * p.out.row + (h0 + i) * p.out.head + 8 * lane), pack8(v));
    }
}

template <int kRows>
cudaError_t launch_gated(const GatedNormParams& p, cudaStream_t stream) {
    const int groups = (p.heads + kRows - 1) / kRows;
    const int64_t blocks = (p.tokens * groups + GN_HALVES - 1) / GN_HALVES;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    return launch_early(gated_norm_kernel<kRows>, dim3((unsigned)blocks), GN_THREADS, 0, stream, p, groups);
}

// ---------------------------------------------------------------- between two blocks
// kThreads threads take a token's row, each with kChunks groups of 8 elements, and hold it in
// registers from the loads to the stores.
template <int kThreads>
__device__ __forceinline__ float row_sum(float x, float* shared) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    if (kThreads == 32) return x;
    if ((threadIdx.x & 31) == 0) shared[threadIdx.x >> 5] = x;
    __syncthreads();
    x = 0.f;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) x += shared[i];
    return x;
}

template <int kThreads, int kChunks, bool kF32>
__global__ void __launch_bounds__(kThreads < 128 ? 128 : kThreads) residual_norm_kernel(const ResidualNormParams p) {
    __shared__ float shared[2][32];
    constexpr int kRowsHere = kThreads < 128 ? 128 / kThreads : 1;
    await_stream();
    const int tid = threadIdx.x % kThreads;
    const int64_t t = (int64_t)blockIdx.x * kRowsHere + threadIdx.x / kThreads;
    if (t >= p.tokens) return;   // (whole warps, and whole blocks where a row takes more than one)
    float r[kChunks][8], u[kChunks][8];
    float ss = 0.f;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
        const int at = 8 * (tid + c * kThreads);
#pragma unroll
        for (int j = 0; j < 8; ++j) r[c][j] = u[c][j] = 0.f;
        if (at >= p.dim) continue;
        if (kF32) load8(static_cast<const float*>(p.residual) + t * p.residual_row + at, r[c]);
        else unpack8(*reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.residual) + t * p.residual_row + at), r[c]);
        if (p.y) unpack8(*reinterpret_cast<const uint4*>(p.y + t * p.y_row + at), u[c]);
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(u[c][j], u[c][j], ss);
    }
    const float mean = 1.f / (float)p.dim;
    float f = p.scale;
    if (p.post_weight) f *= rsqrtf(row_sum<kThreads>(ss, shared[0]) * mean + p.eps);
    ss = 0.f;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
        const int at = 8 * (tid + c * kThreads);
        if (at >= p.dim) continue;
        if (p.y) {
            float w[8], g[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = g[j] = 1.f;
            if (p.post_weight) load8(p.post_weight + at, w);
            if (p.gate) unpack8(*reinterpret_cast<const uint4*>(p.gate + t * p.gate_row + at), g);
#pragma unroll
            for (int j = 0; j < 8; ++j) r[c][j] = fmaf(u[c][j] * f, w[j] * g[j], r[c][j]);
        }
        if (p.residual_out) {
            if (kF32) {
                float4* o = reinterpret_cast<float4*>(static_cast<float*>(p.residual_out) + t * p.residual_out_row + at);
                o[0] = make_float4(r[c][0], r[c][1], r[c][2], r[c][3]);
                o[1] = make_float4(r[c][4], r[c][5], r[c][6], r[c][7]);
            } else {
                *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.residual_out) + t * p.residual_out_row + at) = pack8(r[c]);
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(r[c][j], r[c][j], ss);
    }
    const float f2 = rsqrtf(row_sum<kThreads>(ss, shared[1]) * mean + p.eps);
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
        const int at = 8 * (tid + c * kThreads);
        if (at >= p.dim) continue;
        float w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = 1.f;
        if (p.pre_weight) load8(p.pre_weight + at, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] *= r[c][j] * f2;
        *reinterpret_cast<uint4*>(p.out + t * p.out_row + at) = pack8(w);
    }
}

template <int kThreads, int kChunks>
cudaError_t launch_residual(const ResidualNormParams& p, cudaStream_t stream) {
    constexpr int block = kThreads < 128 ? 128 : kThreads;
    const int64_t blocks = (p.tokens * kThreads + block - 1) / block;
    return launch_early(p.f32 ? residual_norm_kernel<kThreads, kChunks, true> : residual_norm_kernel<kThreads, kChunks, false>,
                        dim3((unsigned)blocks), block, 0, stream, p);
}

}  // namespace

cudaError_t launch_gated_norm(const GatedNormParams& p, cudaStream_t stream) {
    if (p.tokens == 0) return cudaSuccess;
    if (p.tokens * p.heads >= 152 * 64 * 4) return launch_gated<4>(p, stream);
    return launch_gated<1>(p, stream);
}

cudaError_t launch_residual_norm(const ResidualNormParams& p, cudaStream_t stream) {
    if (p.tokens == 0) return cudaSuccess;
    const int groups = p.dim / 8;
    if (groups <= 32) return launch_residual<32, 1>(p, stream);
    if (groups <= 128) return launch_residual<128, 1>(p, stream);
    if (groups <= 256) return launch_residual<256, 1>(p, stream);
    if (groups <= 512) return launch_residual<512, 1>(p, stream);
    if (groups <= 1024) return launch_residual<512, 2>(p, stream);
    return launch_residual<1024, 2>(p, stream);
}

}  // namespace kda
