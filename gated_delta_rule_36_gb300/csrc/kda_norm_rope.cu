// RMS norm of every query and key head and the rotary rotation, one pass:
//   y = x rsqrt(mean(x^2) + eps) weight;  a' = a cos - b sin, b' = b cos + a sin.
//
// A half-warp takes a (token, head) row: lane l holds elements 8 l .. 8 l + 7 (one 16-byte
// load), the sum of squares is four shuffles, and the partner of a rotated element sits
// rot / 16 lanes away (pairs (i, i + rot/2)) or in the same lane (pairs (2 i, 2 i + 1)).
// It stays with one token for up to kRows heads, loads all their rows at once and reads the
// token's position, table row and weight once for them.
//
// Bound by HBM: each row is read once and written once, past the caches.  What it takes is bytes in
// flight: 28 warps an SM with eight rows a half-warp are 112 KB of loads.  32,768 tokens x 72 heads
// (1.22 GB): 200 us, 6.1 TB/s (blocks of 128 threads, 7 an SM; with 6 218, with 8, which spill,
// 244; 256 threads at 3 an SM 225; plain instead of streaming loads and stores 10 % slower each).
#include "kda_device.cuh"
#include "kda_ops.h"

namespace kda {
namespace {

constexpr int NR_THREADS = 128;
constexpr int NR_HALVES = NR_THREADS / 16;
constexpr int NR_BLOCKS = 7;   // an SM: 72 registers a thread

__device__ __forceinline__ void load8(const float* p, float (&f)[8]) {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}

// groups[i]: groups of kRows heads of q (0) and k (1), the last one possibly partial
template <bool kInterleaved, int kRows>
__global__ void __launch_bounds__(NR_THREADS, NR_BLOCKS) norm_rope_kernel(const NormRopeParams p, int groups_q, int groups) {
    await_stream();
    const int lane = threadIdx.x & 15;
    const int64_t item = (int64_t)blockIdx.x * NR_HALVES + (threadIdx.x >> 4);
    const int64_t t = item / groups;
    const bool active = t < p.tokens;
    const int g = (int)(item - t * groups);
    const int which = g >= groups_q;
    const int h0 = (which ? g - groups_q : g) * kRows;
    const int nrows = !active ? 0 : p.heads[which] - h0 < kRows ? p.heads[which] - h0 : kRows;
    const __nv_bfloat16* x = p.x[which].data + t * p.x[which].row + h0 * p.x[which].head + 8 * lane;
    uint4 raw[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i)
        raw[i] = i < nrows ? __ldcs(reinterpret_cast<const uint4*>(x + i * p.x[which].head)) : make_uint4(0, 0, 0, 0);

    // the token's cosines and sines for this lane's elements: 8 pairs (or 4 adjacent ones)
    const int rl = p.rot / 8, hl = rl / 2;   // lanes that hold rotated elements, and half of them
    float c[8], s[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) c[j] = 1.f, s[j] = 0.f;
    bool bad = false;
    if (p.cos_sin && active) {
        const int64_t pos = p.positions[t];
        bad = pos < 0 || pos >= p.table_rows;
        if (bad) {
            if (p.status && lane == 0) atomicOr(p.status, KDA_DEVERR_POSITION);
#pragma unroll
            for (int j = 0; j < 8; ++j) c[j] = __uint_as_float(0x7fc00000u);
        } else if (lane < rl) {
            const float* row = p.cos_sin + pos * p.rot;
            if (kInterleaved) {
                const float4 cc = *reinterpret_cast<const float4*>(row + 4 * lane);
                const float4 ss = *reinterpret_cast<const float4*>(row + p.rot / 2 + 4 * lane);
                c[0] = cc.x; c[1] = cc.y; c[2] = cc.z; c[3] = cc.w;
                s[0] = ss.x; s[1] = ss.y; s[2] = ss.z; s[3] = ss.w;
            } else {
                const int i0 = 8 * (lane < hl ? lane : lane - hl);
                load8(row + i0, c);
                load8(row + p.rot / 2 + i0, s);
                if (lane < hl) {   // a' = a cos - b sin
#pragma unroll
                    for (int j = 0; j < 8; ++j) s[j] = -s[j];
                }
            }
        }
    }
    float w[8];
    if (p.weight[which]) load8(p.weight[which] + 8 * lane, w);
    else {
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = 1.f;
    }
    const int src = lane < hl ? lane + hl : lane < rl ? lane - hl : lane;
    __nv_bfloat16* y = p.y[which].data + t * p.y[which].row + h0 * p.y[which].head + 8 * lane;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        float v[8] = {bf16_lo(raw[i].x), bf16_hi(raw[i].x), bf16_lo(raw[i].y), bf16_hi(raw[i].y),
                      bf16_lo(raw[i].z), bf16_hi(raw[i].z), bf16_lo(raw[i].w), bf16_hi(raw[i].w)};
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(v[j], v[j], ss);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float r = rsqrtf(ss * (1.f / HD) + p.eps);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] *= r * w[j];
        float o[8];
        if (kInterleaved) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                o[2 * j] = v[2 * j] * c[j] - v[2 * j + 1] * s[j];
                o[2 * j + 1] = v[2 * j + 1] * c[j] + v[2 * j] * s[j];
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float other = __shfl_sync(0xffffffffu, v[j], src, 16);
                o[j] = v[j] * c[j] + other * s[j];
            }
        }
        if (i < nrows)
            __stcs(reinterpret_cast<uint4*>(y + i * p.y[which].head),
                   make_uint4(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]), pack_bf16x2(o[4], o[5]), pack_bf16x2(o[6], o[7])));
    }
}

template <int kRows>
cudaError_t launch(const NormRopeParams& p, cudaStream_t stream) {
    const int gq = (p.heads[0] + kRows - 1) / kRows, groups = gq + (p.heads[1] + kRows - 1) / kRows;
    const int64_t blocks = (p.tokens * groups + NR_HALVES - 1) / NR_HALVES;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    return launch_early(p.interleaved ? norm_rope_kernel<true, kRows> : norm_rope_kernel<false, kRows>, dim3((unsigned)blocks), NR_THREADS, 0, stream, p,
                        gq, groups);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeParams& p, cudaStream_t stream) {
    const int64_t rows = p.tokens * (p.heads[0] + p.heads[1]);
    if (rows == 0) return cudaSuccess;
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    // Rows a half-warp takes: eight once that still gives every SM its seven blocks (32,768 tokens x 72
    // heads: 208 us, against 238 with four and 305 with two), else one, for the latency of small calls.
    if (rows >= (int64_t)sms * NR_BLOCKS * NR_HALVES * 8) return launch<8>(p, stream);
    return launch<1>(p, stream);
}

}  // namespace kda
