// New keys and values into a cache held in 4 bits (the row's layout: include/kda.h).
//   zero = min x, scale = bf16((max x - min x) / 15), code = (x - zero) / scale to the nearest, ties to even
// over each 64 channels.  A warp takes a (token, head): its lower half the key, its upper half the value,
// 8 channels a lane; minimum and maximum are three shuffles.
//
// The codes are those of exact arithmetic.  The scale is: two bf16 numbers and a quotient by 15 cannot come
// so close to the middle of two bf16 numbers, without lying on it, that the two fp32 roundings decide.  For
// the codes the quotient rounds right as long as the difference is exact (a scale has 8 bits, a border between
// codes 5, so the border times the scale has 13, and a quotient of 24 bits is never moved onto it).  The
// difference is inexact where the two numbers are more than 16 binades apart; it is then rounded to odd, which
// keeps it on its side of every number of 13 bits.
#include "kda_qcache.cuh"

namespace kda {
namespace {

constexpr int QA_THREADS = 128;

// a + b rounded to odd (exact sums as they are); a + b >= 0
__device__ __forceinline__ float add_to_odd(float a, float b) {
    const float s = a + b, bb = s - a, err = (a - (s - bb)) + (b - bb);
    const int i = __float_as_int(s);
    return err != 0.f && !(i & 1) ? __int_as_float(i + (err > 0.f ? 1 : -1)) : s;
}

__global__ void __launch_bounds__(QA_THREADS) qcache_append_kernel(const QcacheAppendParams p) {
    await_stream();
    const int lane = threadIdx.x & 31, half = lane >> 4;
    const int64_t item = ((int64_t)blockIdx.x * QA_THREADS + threadIdx.x) >> 5;
    // every sequence's lengths, whether it has tokens or not
    const int64_t threads = (int64_t)gridDim.x * QA_THREADS;
    for (int64_t n = (int64_t)blockIdx.x * QA_THREADS + threadIdx.x; n < p.nseq; n += threads) {
        const int64_t c0 = p.cu ? p.cu[n] : n * p.uniform, c1 = p.cu ? p.cu[n + 1] : c0 + p.uniform, s = p.seqlens_k[n];
        const bool bad = c0 < 0 || (n == 0 && c0 != 0) || c1 < c0 || c1 > p.T || s > p.S || s < c1 - c0;
        if (bad && p.status) atomicOr(p.status, KDA_DEVERR_CU_SEQLENS);
    }
    const int64_t t = item / p.Hk;
    const int h = (int)(item - t * p.Hk);
    if (t >= p.T) return;
    const RowsView& in = half ? p.v : p.k;
    const uint4 raw = *reinterpret_cast<const uint4*>(in.data + t * in.row + h * in.head + 8 * (lane & 15));
    int n;
    int64_t c0, c1;
    if (p.cu) {
        n = sequence_of(p.cu, p.nseq, t);
        c0 = p.cu[n];
        c1 = p.cu[n + 1];
    } else {
        n = (int)(t / p.uniform);
        c0 = n * p.uniform;
        c1 = c0 + p.uniform;
    }
    const int64_t s = p.seqlens_k[n];
    if (c0 < 0 || (n == 0 && c0 != 0) || t < c0 || t >= c1 || c1 > p.T || s > p.S || s < c1 - c0) return;
    const int64_t pos = s - (c1 - t);

    float x[8] = {bf16_lo(raw.x), bf16_hi(raw.x), bf16_lo(raw.y), bf16_hi(raw.y), bf16_lo(raw.z), bf16_hi(raw.z), bf16_lo(raw.w), bf16_hi(raw.w)};
    float lo = x[0], hi = x[0];
    bool finite = true;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        lo = fminf(lo, x[j]);
        hi = fmaxf(hi, x[j]);
        finite &= fabsf(x[j]) < INFINITY;
    }
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) {
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    finite = (__ballot_sync(0xffffffffu, finite) >> (lane & 24) & 0xffu) == 0xffu;
    lo += 0.f;   // (-0 and 0 are one zero)
    const bool wide = hi - lo == INFINITY;   // the range passes fp32's: everything halved
    const float f = wide ? 0.5f : 1.f;
    const float range = hi * f - lo * f;
    const uint32_t sz = finite ? pack_bf16x2(wide ? range / 7.5f : range / 15.f, lo) : 0x7fc07fc0u;
    const float scale = bf16_lo(sz), zero = bf16_hi(sz), step = scale * f;
    uint32_t word = 0;
    float y[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float d = add_to_odd(x[j] * f, -lo * f);
        const float c = step > 0.f ? fminf(rintf(d / step), 15.f) : 0.f;
        word |= (uint32_t)c << (4 * j);
        y[j] = fmaf(c, scale, zero);
    }
    uint8_t* row = p.cache.data + n * p.cache.seq + pos * p.cache.row + h * p.cache.head;
    *reinterpret_cast<uint32_t*>(row + 4 * lane) = word;
    if ((lane & 7) == 0) *reinterpret_cast<uint32_t*>(row + QC_NUMBERS + (lane >> 1)) = sz;
    const RowsView& out = half ? p.v_out : p.k_out;
    if (out.data)
        *reinterpret_cast<uint4*>(out.data + t * out.row + h * out.head + 8 * (lane & 15)) =
            make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
}

}  // namespace

cudaError_t launch_qcache_append(const QcacheAppendParams& p, cudaStream_t stream) {
    if (p.nseq == 0) return cudaSuccess;
    const int64_t rows = p.T * p.Hk;
    int64_t blocks = (rows * 32 + QA_THREADS - 1) / QA_THREADS;
    if (blocks == 0) blocks = 1;   // (the lengths are checked all the same)
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    return launch_early(qcache_append_kernel, dim3((unsigned)blocks), QA_THREADS, 0, stream, p);
}

}  // namespace kda
