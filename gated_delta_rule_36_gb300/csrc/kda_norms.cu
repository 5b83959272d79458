// The norms around a mixer: RMS norm of every head of its output times its activated gate, and the
// norm after a block, its gate and residual scale, the residual sum and the norm before the next block.  Both are
// bound by HBM: each number is read once and written once.
//
// 45,661 tokens x 64 heads (2.24 GB): 327 us, 6.9 TB/s (part of the writes is still in L2 at the end).  A stream of
// 32,768 x 4,096 in bf16 with both norms (1.07 GB): 171 us, 6.3 TB/s; without the next row in flight, a block of 512 threads a row,
// 211 us.  2,024 x 2,304 in fp32 with a gate (65 MB): 12 us, about half of it the start and the last rows.
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
// A block takes a token's row, each thread kChunks groups of 8 elements (where a warp is enough: a warp a row, four of them a
// block), and holds it in registers from the loads to the stores; the next row that it takes is loaded meanwhile.
constexpr int RN_WARP_ROWS = 4;

template <bool kWarp>
__device__ __forceinline__ float row_sum(float x, float* shared) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    if (kWarp) return x;
    if ((threadIdx.x & 31) == 0) shared[threadIdx.x >> 5] = x;
    __syncthreads();
    const int from = threadIdx.x & 15;   // (at most 16 warps; both halves of a warp add them up)
    x = from < (int)(blockDim.x >> 5) ? shared[from] : 0.f;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

template <int kChunks, bool kF32, bool kGate>
struct RawRow {
    uint4 y[kChunks], r[kChunks][kF32 ? 2 : 1], g[kGate ? kChunks : 1];
    __device__ __forceinline__ void load(const ResidualNormParams& p, int64_t t, int tid, int threads) {
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            const int at = 8 * (tid + c * threads);
            y[c] = r[c][0] = make_uint4(0, 0, 0, 0);
            if (kF32) r[c][kF32 ? 1 : 0] = make_uint4(0, 0, 0, 0);
            if (t >= p.tokens || at >= p.dim) continue;
            if (p.y) y[c] = __ldcs(reinterpret_cast<const uint4*>(p.y + t * p.y_row + at));
            if (kF32) {
                const uint4* src = reinterpret_cast<const uint4*>(static_cast<const float*>(p.residual) + t * p.residual_row + at);
                r[c][0] = __ldcs(src);
                r[c][kF32 ? 1 : 0] = __ldcs(src + 1);
            } else {
                r[c][0] = __ldcs(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.residual) + t * p.residual_row + at));
            }
            if (kGate) g[c] = *reinterpret_cast<const uint4*>(p.gate + t * p.gate_row + at);   // (it may be one row for all)
        }
    }
};

template <int kChunks, bool kF32, bool kGate, bool kWarp, int kMost>
__global__ void __launch_bounds__(kMost) residual_norm_kernel(const ResidualNormParams p) {
    __shared__ float shared[3][32];
    await_stream();
    const int threads = kWarp ? 32 : blockDim.x, tid = kWarp ? threadIdx.x & 31 : threadIdx.x;
    const int64_t stride = (int64_t)gridDim.x * (kWarp ? RN_WARP_ROWS : 1);
    int64_t t = kWarp ? (int64_t)blockIdx.x * RN_WARP_ROWS + (threadIdx.x >> 5) : blockIdx.x;
    const float mean = 1.f / (float)p.dim;
    RawRow<kChunks, kF32, kGate> next;
    next.load(p, t, tid, threads);
#pragma unroll 1
    for (int parity = 1; t < p.tokens; t += stride, parity ^= 3) {
        const RawRow<kChunks, kF32, kGate> row = next;
        next.load(p, t + stride, tid, threads);
        float f = p.scale;
        if (p.post_weight) {
            float ss = 0.f;
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
                float u[8];
                unpack8(row.y[c], u);
#pragma unroll
                for (int j = 0; j < 8; ++j) ss = fmaf(u[j], u[j], ss);
            }
            f *= rsqrtf(row_sum<kWarp>(ss, shared[0]) * mean + p.eps);
        }
        float r[kChunks][8];
        float ss = 0.f;
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            const int at = 8 * (tid + c * threads);
            if (kF32) {
                const uint4 a = row.r[c][0], b = row.r[c][kF32 ? 1 : 0];
                r[c][0] = __uint_as_float(a.x); r[c][1] = __uint_as_float(a.y); r[c][2] = __uint_as_float(a.z); r[c][3] = __uint_as_float(a.w);
                r[c][4] = __uint_as_float(b.x); r[c][5] = __uint_as_float(b.y); r[c][6] = __uint_as_float(b.z); r[c][7] = __uint_as_float(b.w);
            } else {
                unpack8(row.r[c][0], r[c]);
            }
            if (at >= p.dim) continue;
            if (p.y) {
                float u[8], w[8], g[8];
                unpack8(row.y[c], u);
#pragma unroll
                for (int j = 0; j < 8; ++j) w[j] = 1.f;
                if (p.post_weight) load8(p.post_weight + at, w);
                if (kGate) {
                    unpack8(row.g[c], g);
#pragma unroll
                    for (int j = 0; j < 8; ++j) w[j] *= g[j];
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) r[c][j] = fmaf(u[j] * f, w[j], r[c][j]);
            }
            if (p.residual_out) {
                if (kF32) {
                    float4* o = reinterpret_cast<float4*>(static_cast<float*>(p.residual_out) + t * p.residual_out_row + at);
                    __stcs(o, make_float4(r[c][0], r[c][1], r[c][2], r[c][3]));
                    __stcs(o + 1, make_float4(r[c][4], r[c][5], r[c][6], r[c][7]));
                } else {
                    __stcs(reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.residual_out) + t * p.residual_out_row + at), pack8(r[c]));
                }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = fmaf(r[c][j], r[c][j], ss);
        }
        const float f2 = rsqrtf(row_sum<kWarp>(ss, shared[parity]) * mean + p.eps);   // (a buffer of its own for two rows in turn)
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            const int at = 8 * (tid + c * threads);
            if (at >= p.dim) continue;
            float w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = 1.f;
            if (p.pre_weight) load8(p.pre_weight + at, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] *= r[c][j] * f2;
            __stcs(reinterpret_cast<uint4*>(p.out + t * p.out_row + at), pack8(w));
        }
    }
}

template <int kChunks, bool kWarp, int kMost>
cudaError_t launch_residual(const ResidualNormParams& p, int sms, cudaStream_t stream) {
    const int groups = p.dim / 8, threads = kWarp ? 32 * RN_WARP_ROWS : (groups + 32 * kChunks - 1) / (32 * kChunks) * 32;
    void (*const kernel)(ResidualNormParams) = p.f32 ? (p.gate ? residual_norm_kernel<kChunks, true, true, kWarp, kMost> : residual_norm_kernel<kChunks, true, false, kWarp, kMost>)
                                                     : (p.gate ? residual_norm_kernel<kChunks, false, true, kWarp, kMost> : residual_norm_kernel<kChunks, false, false, kWarp, kMost>);
    const int64_t blocks = kWarp ? (p.tokens + RN_WARP_ROWS - 1) / RN_WARP_ROWS : p.tokens;
    int per = 1;
    if (blocks > sms) {
        const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kernel, threads, 0);
        if (e != cudaSuccess) return e;
    }
    const int64_t most = (int64_t)sms * per;
    return launch_early(kernel, dim3((unsigned)(blocks < most ? blocks : most)), threads, 0, stream, p);
}

}  // namespace

cudaError_t launch_gated_norm(const GatedNormParams& p, cudaStream_t stream) {
    if (p.tokens == 0) return cudaSuccess;
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    // rows a half-warp takes: four once that still gives every SM eight blocks, else one, for the latency of small calls
    if (p.tokens * p.heads >= (int64_t)sms * 8 * GN_HALVES * 4) return launch_gated<4>(p, stream);
    return launch_gated<1>(p, stream);
}

cudaError_t launch_residual_norm(const ResidualNormParams& p, cudaStream_t stream) {
    if (p.tokens == 0) return cudaSuccess;
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    const int groups = p.dim / 8;
    if (groups <= 32) return launch_residual<1, true, 128>(p, sms, stream);
    if (groups <= 128) return launch_residual<1, false, 128>(p, sms, stream);
    if (groups <= 512) return launch_residual<2, false, 256>(p, sms, stream);
    // two groups a thread and up to 512 threads (8,192 in fp32 with a gate 6.4 TB/s, with four 5.5; bf16 without 6.1 and 5.8),
    // but for bf16 with a gate, where four are faster (4,104 5.4 TB/s, with two 4.2; 8,192 6.1 and 5.7)
    if (groups <= 1024 && (p.f32 || !p.gate)) return launch_residual<2, false, 512>(p, sms, stream);
    return launch_residual<4, false, 512>(p, sms, stream);
}

}  // namespace kda
