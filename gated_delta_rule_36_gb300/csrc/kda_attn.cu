// Causal softmax attention with grouped heads over packed prompts and caches.
//
// One warp per (query, head): lane l holds channels 4 l .. 4 l + 3 of q and of the output, the
// keys are visited once with the running maximum and sum of the softmax.  Bound by instruction issue.
#include "kda_device.cuh"
#include "kda_ops.h"

namespace kda {
namespace {

constexpr int AT_THREADS = 128;

__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
    const uint2 w = *reinterpret_cast<const uint2*>(p);
    return make_float4(bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y));
}

__global__ void __launch_bounds__(AT_THREADS) attn_kernel(const AttnParams p) {
    bool bad = false;
    for (int i = threadIdx.x; i < p.nseq; i += AT_THREADS) {
        if (p.cu_q) bad |= p.cu_q[i + 1] < p.cu_q[i];
        if (p.cu_k) bad |= p.cu_k[i + 1] < p.cu_k[i];
        if (p.seqlens_k) bad |= p.seqlens_k[i] < 0 || p.seqlens_k[i] > p.Tk;
    }
    if (threadIdx.x == 0) {
        if (p.cu_q) bad |= p.cu_q[0] != 0 || p.cu_q[p.nseq] > p.Tq;
        if (p.cu_k) bad |= p.cu_k[0] != 0 || p.cu_k[p.nseq] > p.Tk;
    }
    bad = __syncthreads_or(bad);
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = bad ? KDA_DEVERR_CU_SEQLENS : 0u;
    if (bad) return;
    const int64_t row = (int64_t)blockIdx.x * (AT_THREADS / 32) + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31, c0 = 4 * lane;
    if (row >= p.Tq * p.Hq) return;
    const int64_t t = row / p.Hq;
    const int h = (int)(row % p.Hq), hk = h / (p.Hq / p.Hk);
    int n = 0;
    int64_t bos, eos;
    if (p.cu_q) {
        if (t >= p.cu_q[p.nseq]) return;
        int lo = 0, hi = p.nseq;   // the last n with cu_q[n] <= t
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (p.cu_q[mid] <= t) lo = mid; else hi = mid;
        }
        n = lo;
        bos = p.cu_q[n];
        eos = p.cu_q[n + 1];
    } else {
        n = (int)(t / p.uniform_q);
        bos = n * p.uniform_q;
        eos = bos + p.uniform_q;
    }
    int64_t kbase = 0, lk = p.Tk;
    if (p.cache) lk = p.seqlens_k[n];
    else if (p.cu_k) kbase = p.cu_k[n], lk = p.cu_k[n + 1] - kbase;
    const __nv_bfloat16* kp = p.k + (p.cache ? n * p.k_seq : 0) + kbase * p.k_row + hk * p.k_head + c0;
    const __nv_bfloat16* vp = p.v + (p.cache ? n * p.v_seq : 0) + kbase * p.v_row + hk * p.v_head + c0;
    int64_t seen = (t - bos) + 1 + lk - (eos - bos);
    const float4 q = load4(p.q.data + t * p.q.row + h * p.q.head + c0);
    const float sc = p.scale * LOG2E;
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int64_t j = 0; j < seen; ++j) {
        const float4 k = load4(kp + j * p.k_row), v = load4(vp + j * p.v_row);
        float s = fmaf(q.x, k.x, fmaf(q.y, k.y, fmaf(q.z, k.z, q.w * k.w)));
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
        s *= sc;
        const float m2 = fmaxf(m, s), f = exp2f(m - m2), e = exp2f(s - m2);
        l = fmaf(l, f, e);
        o.x = fmaf(o.x, f, e * v.x);
        o.y = fmaf(o.y, f, e * v.y);
        o.z = fmaf(o.z, f, e * v.z);
        o.w = fmaf(o.w, f, e * v.w);
        m = m2;
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    *reinterpret_cast<uint2*>(p.out.data + t * p.out.row + h * p.out.head + c0) =
        make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
    if (p.lse && lane == 0) p.lse[t * p.Hq + h] = l > 0.f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

}  // namespace

size_t attn_workspace_bytes(int64_t, int, int) { return 0; }

cudaError_t launch_attn(const AttnParams& p, cudaStream_t stream) {
    const int64_t blocks = (p.Tq * p.Hq + AT_THREADS / 32 - 1) / (AT_THREADS / 32);
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    attn_kernel<<<(unsigned)(blocks > 0 ? blocks : 1), AT_THREADS, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace kda
