// Launch parameters and internal entry points of the token-mixer operators beside KDA
// (include/kda.h: kda_qk_norm_rope, kda_attn_fwd, kda_lin_fwd, kda_lin_decode).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kda.h"

namespace kda {

// A bf16 [rows, heads, 128] view: strides in elements.
struct RowsView {
    __nv_bfloat16* data;
    int64_t row;    // stride of a token (or batch) row
    int64_t head;   // stride of a head
};

struct NormRopeParams {
    RowsView x[2], y[2];        // q, k and their outputs
    const float* weight[2];     // nullptr = 1
    int heads[2];
    const float* cos_sin;       // [table_rows, rot]: rot / 2 cosines, then rot / 2 sines; nullptr = no rotation
    const int64_t* positions;
    int64_t table_rows;
    int64_t tokens;
    uint32_t* status;           // or nullptr
    float eps;
    int rot;
    int interleaved;
};

struct AttnParams {
    RowsView q, out;
    __nv_bfloat16 *k, *v;
    int64_t k_seq, k_row, k_head;   // strides in elements; k_seq = 0 for packed keys
    int64_t v_seq, v_row, v_head;
    float* lse;                     // [Tq, Hq] or nullptr
    const int64_t* cu_q;            // [nseq + 1] or nullptr: uniform_q queries each
    const int64_t* cu_k;            // packed keys: [nseq + 1], or nullptr: one sequence of Tk
    const int64_t* seqlens_k;       // cache: [nseq]
    int64_t uniform_q;
    int64_t Tq, Tk;                 // Tk: packed key rows, or the cache's rows for each sequence
    int nseq, Hq, Hk;
    int cache;
    float scale;
    uint32_t* status;
    void* workspace;                // behind the status word
    int test_skip;                  // the test-only build: the share b that withholds an arrival, -2 - b: that finds itself unsound; -1 for none
};

struct LinParams {
    RowsView q, k, v, out;
    const float* log_decay;
    const void* init_state;         // nullptr = zero state
    void* final_state;              // nullptr = not stored
    const int64_t* cu_seqlens;      // nullptr = batched mode
    int64_t T, T_total;
    int H, nseq;
    int init_f32, final_f32;
    float scale;
    uint32_t* status;
    void* workspace;
    int test_skip;                  // the test-only build: the share b that withholds an arrival, -2 - b: that finds itself unsound; -1 for none
};

cudaError_t launch_norm_rope(const NormRopeParams& p, cudaStream_t stream);
cudaError_t launch_attn(const AttnParams& p, cudaStream_t stream);
size_t attn_workspace_bytes(int64_t Tq, int Hq, int Hk);
cudaError_t launch_lin_fwd(const LinParams& p, cudaStream_t stream);
size_t lin_workspace_bytes(int64_t T_total, int H, int nseq);
cudaError_t launch_lin_decode(const LinParams& p, cudaStream_t stream);

// Launches a kernel that may be set up while the one before it on the stream still ends (2 to 2.5 us of a call: one
// token over 32,767 keys 42.5 -> 39.9 us, 64 x 64 linear steps 80.3 -> 78.1).  Its threads call
// await_stream() before they touch any memory that others write or read.
template <class... P, class... A>
inline cudaError_t launch_early(void (*kernel)(P...), dim3 grid, int threads, size_t shared, cudaStream_t stream, A... args) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = shared;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}
#ifdef __CUDACC__
__device__ __forceinline__ void await_stream() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
#endif

}  // namespace kda
