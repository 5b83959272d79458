// New keys and values into a cache held in 4 bits (the row's layout: include/kda.h).
//   zero = min x, scale = bf16((max x - min x) / 15), code = (x - zero) / scale to the nearest, ties to even
// over each 64 channels.  A warp takes a token's heads, one after another: its lower half the key, its upper half the
// value, 8 channels a lane; minimum and maximum travel together as a pair of bf16 numbers, three shuffles.
//
// The codes are those of exact arithmetic.  The scale is: two bf16 numbers and a quotient by 15 cannot come
// so close to the middle of two bf16 numbers, without lying on it, that the two fp32 roundings decide.  For
// the codes a correctly rounded quotient rounds right as long as the difference is exact (a scale has 8 bits, a border between
// codes 5, so the border times the scale has 13, and a quotient of 24 bits is never moved onto it).  Both quotients are made
// from an approximate reciprocal and one correction by the remainder, which fma gives exactly: what is left then is some 2^-22 of the quotient's
// last place, and a quotient by a number of 8 bits is either on the middle of two neighbours or 2^-9 of a place away from it.
// That asks for scales within 2^-60 and 2^60, and for numbers at most 15 binades below
// the largest, which makes the differences exact.  Other rows go a longer way: division,
// differences rounded to odd (which keeps them on their side of every number of 13 bits), and halves where the
// range passes fp32's.
//
// Bound by the instructions (issue 74 %, 190 for each key and value) about as much as by HBM: 45,661 tokens x 8 heads with the
// values returned (427 MB) 78 us, 5.4 TB/s.  228 us with divisions, rounding to odd for every number and a search for each
// row; 106 with four rows a warp, 93 with packed checks.  Without the values 49 us (56 with their arithmetic left in).  16
// channels a lane, a quarter of a warp a row: 78 as well, but one head 23 us (8 channels 13).
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

// The long way: codes of one lane's eight numbers, one in each four bits, for any finite numbers.
__device__ __noinline__ uint32_t codes_of_any(const uint4 raw, float lo, bool wide, float scale) {
    const float f = wide ? 0.5f : 1.f, step = scale * f;
    const uint32_t in[4] = {raw.x, raw.y, raw.z, raw.w};
    uint32_t word = 0;
#pragma unroll 1
    for (int j = 0; j < 8; ++j) {
        const float x = j & 1 ? bf16_hi(in[j >> 1]) : bf16_lo(in[j >> 1]);
        const float d = add_to_odd(x * f, -lo * f);
        const float c = step > 0.f ? fminf(rintf(d / step), 15.f) : 0.f;
        word |= (uint32_t)c << (4 * j);
    }
    return word;
}

__device__ __noinline__ uint4 values_of(uint32_t word, float scale, float zero) {
    float c[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) c[j] = fmaf((float)(word >> (4 * j) & 15u), scale, zero);
    return make_uint4(pack_bf16x2(c[0], c[1]), pack_bf16x2(c[2], c[3]), pack_bf16x2(c[4], c[5]), pack_bf16x2(c[6], c[7]));
}

__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
    const __nv_bfloat162 m = __hmin2_nan(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&m);
}
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    const __nv_bfloat162 m = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&m);
}

// kHeads: heads of a token that a warp takes, all loaded at once; kValues: what the cache then holds is written too
template <int kHeads, bool kValues>
__global__ void __launch_bounds__(QA_THREADS) qcache_append_kernel(const QcacheAppendParams p) {
    await_stream();
    const int lane = threadIdx.x & 31, half = lane >> 4;
    // every sequence's lengths, whether it has tokens or not
    const int64_t threads = (int64_t)gridDim.x * QA_THREADS;
    for (int64_t n = (int64_t)blockIdx.x * QA_THREADS + threadIdx.x; n < p.nseq && blockIdx.y == 0; n += threads) {
        const int64_t c0 = p.cu ? p.cu[n] : n * p.uniform, c1 = p.cu ? p.cu[n + 1] : c0 + p.uniform, s = p.seqlens_k[n];
        const bool bad = c0 < 0 || (n == 0 && c0 != 0) || c1 < c0 || c1 > p.T || s > p.S || s < c1 - c0;
        if (bad && p.status) atomicOr(p.status, KDA_DEVERR_CU_SEQLENS);
    }
    const int64_t t = (int64_t)blockIdx.x * (QA_THREADS / 32) + (threadIdx.x >> 5);
    if (t >= p.T) return;
    const int h0 = blockIdx.y * kHeads, heads = min(p.Hk - h0, kHeads);
    const RowsView& in = half ? p.v : p.k;
    const __nv_bfloat16* src = in.data + t * in.row + h0 * in.head + 8 * (lane & 15);
    uint4 raws[kHeads];
#pragma unroll
    for (int i = 0; i < kHeads; ++i) raws[i] = i < heads ? __ldcs(reinterpret_cast<const uint4*>(src + i * in.head)) : make_uint4(0, 0, 0, 0);
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
    uint8_t* row = p.cache.data + n * p.cache.seq + (s - (c1 - t)) * p.cache.row + h0 * p.cache.head;
    const RowsView& out = half ? p.v_out : p.k_out;
    __nv_bfloat16* dst = kValues ? out.data + t * out.row + h0 * out.head + 8 * (lane & 15) : nullptr;
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
        if (i >= heads) break;
        const uint4 raw = raws[i];
        const uint32_t l2 = min2(min2(raw.x, raw.y), min2(raw.z, raw.w)), h2 = max2(max2(raw.x, raw.y), max2(raw.z, raw.w));
        // (the smallest, minus the largest) in one register
        uint32_t both = __byte_perm(min2(l2, l2 >> 16), max2(h2, h2 >> 16) ^ 0x8000u, 0x5410);
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) both = min2(both, __shfl_xor_sync(0xffffffffu, both, o));
        const float lo = bf16_lo(both) + 0.f, hi = -bf16_hi(both);   // (-0 and 0 are one zero; a NaN makes both NaN)
        const float most = fmaxf(fabsf(lo), fabsf(hi));
        const bool finite = fabsf(lo) < INFINITY && fabsf(hi) < INFINITY;
        // all eight numbers at least 2^-15 of the largest
        const uint32_t small = min2(min2(raw.x & 0x7fff7fffu, raw.y & 0x7fff7fffu), min2(raw.z & 0x7fff7fffu, raw.w & 0x7fff7fffu));
        const bool near = __hbge2(*reinterpret_cast<const __nv_bfloat162*>(&small), __float2bfloat162_rn(0x1p-15f * most));
        const float range = hi - lo, by15 = range * (1.f / 15.f);
        uint32_t sz = pack_bf16x2(fmaf(fmaf(-by15, 15.f, range), 1.f / 15.f, by15), lo);
        const bool plain = near && finite && bf16_lo(sz) >= 0x1p-60f && bf16_lo(sz) <= 0x1p60f;
        uint32_t word;
        uint4 y;   // the values that the codes stand for
        if (__all_sync(0xffffffffu, plain)) {
            const float scale = bf16_lo(sz), r = rcp_approx(scale);
            const float x[8] = {bf16_lo(raw.x), bf16_hi(raw.x), bf16_lo(raw.y), bf16_hi(raw.y), bf16_lo(raw.z), bf16_hi(raw.z), bf16_lo(raw.w), bf16_hi(raw.w)};
            uint32_t sum = 0;
            float c[8];
#pragma unroll
            for (int j = 7; j >= 0; --j) {
                const float d = x[j] - lo, q0 = d * r, q = fmaf(fmaf(-q0, scale, d), r, q0) + 12582912.f;
                sum = sum * 16 + __float_as_uint(q);   // (2^23 + 2^22: the last bits are the rounded quotient)
                if (kValues) c[j] = fmaf(q - 12582912.f, scale, lo);
            }
            word = sum - 0x4b400000u * 0x11111111u;
            if (kValues) y = make_uint4(pack_bf16x2(c[0], c[1]), pack_bf16x2(c[2], c[3]), pack_bf16x2(c[4], c[5]), pack_bf16x2(c[6], c[7]));
        } else {
            const bool wide = range == INFINITY;   // the range passes fp32's: everything halved
            sz = finite ? pack_bf16x2(wide ? (hi * 0.5f - lo * 0.5f) / 7.5f : range / 15.f, lo) : 0x7fc07fc0u;
            word = codes_of_any(raw, lo, wide, bf16_lo(sz));
            if (kValues) y = values_of(word, bf16_lo(sz), bf16_hi(sz));
        }
        *reinterpret_cast<uint32_t*>(row + i * p.cache.head + 4 * lane) = word;
        if ((lane & 7) == 0) *reinterpret_cast<uint32_t*>(row + i * p.cache.head + QC_NUMBERS + (lane >> 1)) = sz;
        if (kValues) __stcs(reinterpret_cast<uint4*>(dst + i * out.head), y);
    }
}

template <int kHeads>
cudaError_t launch(const QcacheAppendParams& p, cudaStream_t stream) {
    int64_t blocks = (p.T * 32 + QA_THREADS - 1) / QA_THREADS;
    if (blocks == 0) blocks = 1;   // (the lengths are checked all the same)
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    return launch_early(p.k_out.data ? qcache_append_kernel<kHeads, true> : qcache_append_kernel<kHeads, false>,
                        dim3((unsigned)blocks, (unsigned)((p.Hk + kHeads - 1) / kHeads)), QA_THREADS, 0, stream, p);
}

}  // namespace

cudaError_t launch_qcache_append(const QcacheAppendParams& p, cudaStream_t stream) {
    if (p.nseq == 0) return cudaSuccess;
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    // four heads a warp once that still gives every SM 16 warps, else one, for the latency of small calls
    if (p.T * p.Hk >= (int64_t)sms * 16 * 4) return launch<4>(p, stream);
    return launch<1>(p, stream);
}

}  // namespace kda
