// RMS norm of every query and key head and the rotary rotation, one pass:
//   y = x rsqrt(mean(x^2) + eps) weight;  a' = a cos - b sin, b' = b cos + a sin.
//
// A half-warp takes one (token, head) row: lane l holds elements 8 l .. 8 l + 7 (one 16-byte
// load), the sum of squares is four shuffles, and the partner of a rotated element sits
// rot / 16 lanes away (pairs (i, i + rot/2)) or in the same lane (pairs (2 i, 2 i + 1)).
// Bound by HBM: each row is read once and written once.
#include "kda_device.cuh"
#include "kda_ops.h"

namespace kda {
namespace {

constexpr int NR_THREADS = 256;
constexpr int NR_HALVES = NR_THREADS / 16;

template <bool kInterleaved>
__global__ void __launch_bounds__(NR_THREADS) norm_rope_kernel(const NormRopeParams p) {
    const int lane = threadIdx.x & 15;
    const int heads = p.heads[0] + p.heads[1];
    const int64_t row = (int64_t)blockIdx.x * NR_HALVES + (threadIdx.x >> 4);
    const bool active = row < p.tokens * heads;
    const int64_t t = active ? row / heads : 0;
    const int hh = active ? (int)(row % heads) : 0;
    const int which = hh >= p.heads[0];
    const int h = which ? hh - p.heads[0] : hh;
    uint4 w = make_uint4(0, 0, 0, 0);
    if (active) w = *reinterpret_cast<const uint4*>(p.x[which].data + t * p.x[which].row + h * p.x[which].head + 8 * lane);
    float x[8] = {bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y), bf16_lo(w.z), bf16_hi(w.z), bf16_lo(w.w), bf16_hi(w.w)};
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], ss);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float r = rsqrtf(ss * (1.f / HD) + p.eps);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] *= p.weight[which] ? r * p.weight[which][8 * lane + j] : r;
    const int rl = p.rot / 8;   // lanes that hold rotated elements
    int64_t pos = 0;
    bool bad = false;
    if (p.cos_sin && active) {
        pos = p.positions[t];
        bad = pos < 0 || pos >= p.table_rows;
        if (bad && p.status && lane == 0) atomicOr(p.status, KDA_DEVERR_POSITION);
    }
    float y[8];
    if (kInterleaved) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float c = 1.f, s = 0.f;
            if (lane < rl && active && !bad) {
                c = p.cos_sin[pos * p.rot + 4 * lane + j];
                s = p.cos_sin[pos * p.rot + p.rot / 2 + 4 * lane + j];
            }
            y[2 * j] = x[2 * j] * c - x[2 * j + 1] * s;
            y[2 * j + 1] = x[2 * j + 1] * c + x[2 * j] * s;
        }
    } else {
        const int hl = rl / 2;
        const int src = lane < hl ? lane + hl : lane < rl ? lane - hl : lane;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float other = __shfl_sync(0xffffffffu, x[j], src, 16);
            float c = 1.f, s = 0.f;
            if (lane < rl && active && !bad) {
                const int i = 8 * (lane < hl ? lane : lane - hl) + j;
                c = p.cos_sin[pos * p.rot + i];
                s = p.cos_sin[pos * p.rot + p.rot / 2 + i];
            }
            y[j] = x[j] * c + (lane < hl ? -other : other) * s;
        }
    }
    if (bad) {
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = __uint_as_float(0x7fc00000u);
    }
    if (active)
        *reinterpret_cast<uint4*>(p.y[which].data + t * p.y[which].row + h * p.y[which].head + 8 * lane) =
            make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeParams& p, cudaStream_t stream) {
    const int64_t rows = p.tokens * (p.heads[0] + p.heads[1]);
    if (rows == 0) return cudaSuccess;
    const int64_t blocks = (rows + NR_HALVES - 1) / NR_HALVES;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    if (p.interleaved) norm_rope_kernel<true><<<(unsigned)blocks, NR_THREADS, 0, stream>>>(p);
    else norm_rope_kernel<false><<<(unsigned)blocks, NR_THREADS, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace kda
