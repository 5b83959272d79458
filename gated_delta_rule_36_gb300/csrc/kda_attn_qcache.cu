// Causal softmax attention with grouped heads over a cache held in 4 bits: a plain kernel, one warp for each
// query and head, one pass over the keys with the running maximum and sum.
#include "kda_qcache.cuh"

namespace kda {
namespace {

__global__ void qcache_lengths_kernel(const QcacheAttnParams p) {
    await_stream();
    bool bad = false;
    for (int n = threadIdx.x; n < p.nseq; n += blockDim.x) {
        if (p.cu_q) bad |= p.cu_q[n + 1] < p.cu_q[n] || (n == 0 && p.cu_q[0] != 0) || (n + 1 == p.nseq && p.cu_q[n + 1] > p.Tq);
        bad |= p.seqlens_k[n] < 0 || p.seqlens_k[n] > p.S;
    }
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) *p.status = bad ? KDA_DEVERR_CU_SEQLENS : 0u;
}

__global__ void __launch_bounds__(128) attn_qcache_kernel(const QcacheAttnParams p) {
    await_stream();
    if (*p.status) return;
    const int lane = threadIdx.x & 31;
    const int64_t item = ((int64_t)blockIdx.x * 128 + threadIdx.x) >> 5;
    const int64_t t = item / p.Hq;
    const int h = (int)(item - t * p.Hq);
    if (t >= p.Tq) return;
    const int n = p.cu_q ? sequence_of(p.cu_q, p.nseq, t) : (int)(t / p.uniform_q);
    const int64_t c1 = p.cu_q ? p.cu_q[n + 1] : (n + 1) * p.uniform_q;
    if (t >= c1) return;
    const int64_t keys = p.seqlens_k[n] - (c1 - 1 - t);   // that this query sees
    const uint2 raw = *reinterpret_cast<const uint2*>(p.q.data + t * p.q.row + h * p.q.head + 4 * lane);
    const float c = p.scale * LOG2E;
    const float q[4] = {bf16_lo(raw.x), bf16_hi(raw.x), bf16_lo(raw.y), bf16_hi(raw.y)};
    const uint8_t* row = p.cache.data + n * p.cache.seq + (h / (p.Hq / p.Hk)) * p.cache.head;
    float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
    for (int64_t j = 0; j < keys; ++j, row += p.cache.row) {
        const uint32_t kc = *reinterpret_cast<const uint16_t*>(row + 2 * lane), vc = *reinterpret_cast<const uint16_t*>(row + 64 + 2 * lane);
        const uint32_t kn = *reinterpret_cast<const uint32_t*>(row + QC_NUMBERS + (lane >> 4) * 4);
        const uint32_t vn = *reinterpret_cast<const uint32_t*>(row + QC_NUMBERS + 8 + (lane >> 4) * 4);
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) s = fmaf(q[i], fmaf((float)(kc >> (4 * i) & 15u), bf16_lo(kn), bf16_hi(kn)), s);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
        s *= c;
        if (!(s <= m)) {
            const float f = m == -INFINITY ? 0.f : exp2f(m - s);
            m = s;
            l *= f;
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] *= f;
        }
        const float w = exp2f(s - m);
        l += w;
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = fmaf(w, fmaf((float)(vc >> (4 * i) & 15u), bf16_lo(vn), bf16_hi(vn)), o[i]);
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    *reinterpret_cast<uint2*>(p.out.data + t * p.out.row + h * p.out.head + 4 * lane) =
        make_uint2(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv));
    if (p.lse && lane == 0) p.lse[t * p.Hq + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

}  // namespace

size_t attn_qcache_workspace_bytes(int64_t, int, int, int) { return 0; }

cudaError_t launch_attn_qcache(const QcacheAttnParams& p, cudaStream_t stream) {
    cudaError_t e = launch_early(qcache_lengths_kernel, dim3(1), 256, 0, stream, p);
    const int64_t blocks = (p.Tq * p.Hq + 3) / 4;
    if (e != cudaSuccess || blocks == 0) return e;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    return launch_early(attn_qcache_kernel, dim3((unsigned)blocks), 128, 0, stream, p);
}

}  // namespace kda
