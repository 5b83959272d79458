// Launch parameters and internal entry points of the token-mixer operators beside KDA
// (include/kda.h: kda_qk_norm_rope, kda_attn_fwd, kda_lin_fwd, kda_lin_decode) and of those around
// them (kda_qcache_append, kda_attn_qcache_fwd, kda_gated_norm, kda_residual_norm).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
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
    // launch_attn_split: queries, keys and values in fp16.  A block of 128 values is v times 2^(top_v - 127 - SPLIT_TOP), one of
    // keys k times 2^(top_k - 127 - SPLIT_KEY), a query q times 2^q_power[token][head]; top[sequence * Hk + head][block] is
    // top_k << 16 | top_v, at least SPLIT_KEY_LEAST and SPLIT_LEAST.  With SPLIT_EACH in it, which says that the block's keys have values
    // of very different size, top_v is each key's own, value_power[sequence * Hk + head][block][128].  16 more channels of both (q_rest[token][head][16] and
    // k_rest[sequence * Hk + head][block][2][128][8]) count in the scores.  Rows of the last block past the sequence's keys hold zeros.
    __half *q_rest, *k_rest;
    const int *q_power, *top;
    const uint8_t* value_power;
    int64_t top_blocks;
    int seq0, seqs;                 // the sequences that this launch answers; all of what is expanded counts from seq0
    int64_t k_seq, k_row, k_head;   // strides in elements; k_seq = 0 for packed keys
    int64_t v_seq, v_row, v_head;
    float* lse;                     // [Tq, Hq] in rows of lse_row, or nullptr
    int64_t lse_row;
    const int64_t* cu_q;            // [nseq + 1] or nullptr: uniform_q queries each
    const int64_t* cu_k;            // packed keys: [nseq + 1], or nullptr: one sequence of Tk
    const int64_t* seqlens_k;       // cache: [nseq]
    int64_t uniform_q;
    int64_t Tq, Tk;                 // Tk: packed key rows, or the cache's rows for each sequence
    int64_t keys;                   // a cache: most keys that a sequence may have
    int keep_status;                // bits are added to the status word (a call of several launches)
    int nseq, Hq, Hk;
    int cache;
    float scale;
    uint32_t* status;
    void* workspace;                // behind the status word
    int test_skip;                  // the test-only build: the share b that withholds an arrival, -2 - b: that finds itself unsound; -1 for none
};

constexpr int SPLIT_TOP = 13, SPLIT_LEAST = 27, SPLIT_KEY = 13, SPLIT_KEY_LEAST = 40, SPLIT_REST = 16;
// Weights are carried as 2^SPLIT_LIFT times what their row's outputs refer to, which they pass by 2^8 at most: the upper
// end of fp16, whose lower end (2^-14 with all bits) is then as far away as it can be.
constexpr int SPLIT_LIFT = 7, SPLIT_EACH = 0x100;
// The values of a block's keys share a power of two if each key's largest is within 2^SPLIT_SPREAD of the block's.
constexpr int SPLIT_SPREAD = 8;

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

// A cache in 4 bits, [sequences, rows, heads, 144] bytes: strides in bytes.
struct QcacheView {
    uint8_t* data;
    int64_t seq, row, head;
};

struct QcacheAppendParams {
    RowsView k, v, k_out, v_out;    // k_out.data, v_out.data: nullptr = not stored
    QcacheView cache;
    const int64_t* seqlens_k;       // [nseq]
    const int64_t* cu;              // [nseq + 1] or nullptr: `uniform` tokens each
    int64_t uniform;
    int64_t T, S;
    int nseq, Hk;
    uint32_t* status;               // or nullptr
};

struct QcacheAttnParams {
    RowsView q, out;
    QcacheView cache;
    float* lse;                     // [Tq, Hq] or nullptr
    const int64_t* cu_q;            // [nseq + 1] or nullptr: uniform_q queries each
    const int64_t* seqlens_k;       // [nseq]
    int64_t uniform_q;
    int64_t Tq, S;
    int nseq, Hq, Hk;
    float scale;
    uint32_t* status;
    void* workspace;                // behind the status word
    int test_skip;                  // the test-only build: few rows, the share b whose first copy never starts; many, as in AttnParams, in the first of its launches
};

struct GatedNormParams {
    RowsView x, gate, out;
    const float* weight;            // nullptr = 1
    int64_t tokens;
    int heads;
    float eps;
    int silu;
};

struct ResidualNormParams {
    const __nv_bfloat16* y;         // nullptr: r = residual
    const __nv_bfloat16* gate;      // nullptr = 1
    const void* residual;
    void* residual_out;             // nullptr = not stored
    __nv_bfloat16* out;
    const float *post_weight, *pre_weight;   // nullptr: no norm after the block; 1
    int64_t y_row, gate_row, residual_row, residual_out_row, out_row;   // strides in elements
    int64_t tokens;
    int dim, f32;                   // f32: the residual stream is fp32
    float scale, eps;
};

cudaError_t launch_qcache_append(const QcacheAppendParams& p, cudaStream_t stream);
cudaError_t launch_attn_qcache(const QcacheAttnParams& p, cudaStream_t stream);
size_t attn_qcache_workspace_bytes(int64_t Tq, int Hq, int Hk, int nseq, int64_t S);
cudaError_t launch_gated_norm(const GatedNormParams& p, cudaStream_t stream);
cudaError_t launch_residual_norm(const ResidualNormParams& p, cudaStream_t stream);
cudaError_t launch_norm_rope(const NormRopeParams& p, cudaStream_t stream);
cudaError_t launch_attn(const AttnParams& p, cudaStream_t stream);
// The same over expanded queries, keys and values (AttnParams: "launch_attn_split").
cudaError_t launch_attn_split(const AttnParams& p, cudaStream_t stream);
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
