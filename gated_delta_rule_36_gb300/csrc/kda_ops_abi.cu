// C ABI of the token-mixer operators beside KDA: argument checks and launches.  Nothing here
// allocates device memory or synchronises.
#include <math.h>
#include <stdarg.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "kda.h"
#include "kda_kernels.h"
#include "kda_ops.h"

namespace {

// The test-only build of the timeout path: the share b that withholds an arrival, or -2 - b: one that
// finds itself unsound (and reports KDA_DEVERR_INTERNAL).
int test_skip() {
#ifdef KDA_WAIT_TEST
    if (const char* sk = getenv("KDA_TEST_SKIP_SHARE")) return atoi(sk);
#endif
    return -1;
}

kda_status fail(kda_status s, const char* fmt, ...) {
    char msg[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(msg, sizeof(msg), fmt, ap);
    va_end(ap);
    kda::set_last_error(msg);
    return s;
}

#define KDA_TRY(call)                        \
    do {                                     \
        const kda_status st_ = (call);       \
        if (st_ != KDA_OK) return st_;       \
    } while (0)

template <class T>
bool present(const T* t) { return t != nullptr && t->data != nullptr; }

size_t elem_size(int32_t dt) { return dt == KDA_F32 ? 4 : dt == KDA_I64 ? 8 : dt == KDA_U8 ? 1 : 2; }

kda_status check_tensor(const char* name, const kda_tensor* t, int32_t dtype, int ndim, const int64_t* shape,
                        size_t align) {
    if (!present(t)) return fail(KDA_ERR_INVALID_ARG, "%s: missing", name);
    if (t->dtype != dtype) return fail(KDA_ERR_INVALID_ARG, "%s: dtype %d, expected %d", name, t->dtype, dtype);
    if (t->ndim != ndim) return fail(KDA_ERR_INVALID_ARG, "%s: ndim %d, expected %d", name, t->ndim, ndim);
    for (int i = 0; i < ndim; ++i)
        if (t->shape[i] != shape[i])
            return fail(KDA_ERR_INVALID_ARG, "%s: dim %d is %lld, expected %lld", name, i, (long long)t->shape[i],
                        (long long)shape[i]);
    if ((uintptr_t)t->data % align != 0)
        return fail(KDA_ERR_INVALID_ARG, "%s: data pointer not %zu-byte aligned", name, align);
    return KDA_OK;
}

// A bf16 view of the given shape (its last dimension the head dim).
kda_status check_view(const char* name, const kda_view* t, int ndim, const int64_t* shape) {
    if (!present(t)) return fail(KDA_ERR_INVALID_ARG, "%s: missing", name);
    if (t->dtype != KDA_BF16) return fail(KDA_ERR_INVALID_ARG, "%s: dtype %d, expected bf16", name, t->dtype);
    if (t->ndim != ndim) return fail(KDA_ERR_INVALID_ARG, "%s: ndim %d, expected %d", name, t->ndim, ndim);
    for (int i = 0; i < ndim; ++i)
        if (t->shape[i] != shape[i])
            return fail(KDA_ERR_INVALID_ARG, "%s: dim %d is %lld, expected %lld", name, i, (long long)t->shape[i],
                        (long long)shape[i]);
    if (t->stride[ndim - 1] != 1) return fail(KDA_ERR_INVALID_ARG, "%s: the innermost stride must be 1", name);
    for (int i = 0; i + 1 < ndim; ++i) {
        if (t->shape[i] <= 1) continue;
        if (t->stride[i] < KDA_HEAD_DIM || t->stride[i] % 8 != 0 || t->stride[i] >= (1LL << 38))
            return fail(KDA_ERR_INVALID_ARG, "%s: stride %lld of dim %d must be a multiple of 8, at least %d", name,
                        (long long)t->stride[i], i, KDA_HEAD_DIM);
        if (t->shape[i] > (1LL << 48) / t->stride[i])
            return fail(KDA_ERR_INVALID_ARG, "%s: dim %d of %lld elements with stride %lld fits no memory", name, i,
                        (long long)t->shape[i], (long long)t->stride[i]);
    }
    if ((uintptr_t)t->data % 16 != 0) return fail(KDA_ERR_INVALID_ARG, "%s: data pointer not 16-byte aligned", name);
    return KDA_OK;
}

// Head dimension and shape of a q-like view, before its dimensions are used.
kda_status check_head_dim(const char* name, const kda_view* t, int ndim) {
    if (!present(t)) return fail(KDA_ERR_INVALID_ARG, "%s: missing", name);
    if (t->ndim != ndim) return fail(KDA_ERR_INVALID_ARG, "%s: ndim %d, expected %d", name, t->ndim, ndim);
    if (t->shape[ndim - 1] != KDA_HEAD_DIM)
        return fail(KDA_ERR_UNSUPPORTED, "%s: head dim %lld: only %d is built", name, (long long)t->shape[ndim - 1],
                    KDA_HEAD_DIM);
    return KDA_OK;
}

// A tensor's elements as bytes: runs of `run` bytes, repeated n[i] times with stride step[i] for each of `dims`
// dimensions, the innermost first (dimensions that continue one another are one).  width[i]: from the first
// to the last byte of what lies below dimension i.
struct Extent {
    int64_t at = 0, run = 0;
    int dims = 0;
    int64_t n[4], step[4], width[5];
};

Extent extent(const void* data, int64_t es, int ndim, const int64_t* shape, const int64_t* stride) {
    Extent e;
    e.at = (int64_t)(uintptr_t)data;
    e.run = es;
    int64_t n[4], step[4];
    int dims = 0;
    for (int i = ndim - 1; i >= 0; --i) {
        if (shape[i] == 0) {
            e.run = 0;
            return e;
        }
        if (shape[i] == 1) continue;
        int at = dims++;
        for (; at > 0 && step[at - 1] > stride[i] * es; --at) n[at] = n[at - 1], step[at] = step[at - 1];
        n[at] = shape[i];
        step[at] = stride[i] * es;
    }
    for (int i = 0; i < dims; ++i) {
        if (e.dims == 0 && step[i] == e.run) {
            e.run *= n[i];
        } else if (e.dims > 0 && step[i] == e.step[e.dims - 1] * e.n[e.dims - 1]) {
            e.n[e.dims - 1] *= n[i];
        } else {
            e.n[e.dims] = n[i];
            e.step[e.dims++] = step[i];
        }
    }
    e.width[0] = e.run;
    for (int i = 0; i < e.dims; ++i) e.width[i + 1] = e.width[i] + (e.n[i] - 1) * e.step[i];
    return e;
}

Extent extent(const kda_view* t) { return extent(t->data, (int64_t)elem_size(t->dtype), t->ndim, t->shape, t->stride); }

Extent extent(const kda_tensor* t) {
    int64_t stride[4], n = 1;
    for (int i = t->ndim - 1; i >= 0; --i) stride[i] = n, n *= t->shape[i];
    return extent(t->data, (int64_t)elem_size(t->dtype), t->ndim, t->shape, stride);
}

// Whether the first i dimensions of a at 0 and the first j of b at `off` may share a byte.  Of the wider step,
// say a's, b is seen from the repetition of a that it starts in: if neither is wider than the step, it meets that one
// and the next, or none.  Parts of one buffer (columns, heads in turn, planes) are told apart like that;
// anything that does not nest counts as meeting.
bool meet(const Extent& a, int i, const Extent& b, int j, int64_t off) {
    if (off >= a.width[i] || -off >= b.width[j]) return false;
    if (i == 0 && j == 0) return true;
    if (i == 0 || (j > 0 && b.step[j - 1] > a.step[i - 1])) return meet(b, j, a, i, -off);
    const int64_t step = a.step[i - 1];
    const int k = j > 0 && b.step[j - 1] == step ? j - 1 : j;
    if (a.width[i - 1] > step || b.width[k] > step) return true;
    const int64_t d = (off % step + step) % step;
    return meet(a, i - 1, b, k, d) || meet(a, i - 1, b, k, d - step);
}

bool overlap(const Extent& a, const Extent& b) {
    return a.run > 0 && b.run > 0 && meet(a, a.dims, b, b.dims, b.at - a.at);
}

// Whether a view may meet itself: a dimension steps by less than what lies below it.  Nothing is written through one.
kda_status check_written(const char* name, const kda_view* t) {
    const Extent e = extent(t);
    for (int i = 0; i < e.dims && e.run > 0; ++i)
        if (e.width[i] > e.step[i]) return fail(KDA_ERR_ALIAS, "%s: its elements overlap one another", name);
    return KDA_OK;
}

bool same_view(const kda_view* a, const kda_view* b) {
    if (a->data != b->data || a->ndim != b->ndim) return false;
    for (int i = 0; i < a->ndim; ++i)
        if (a->shape[i] != b->shape[i] || (a->shape[i] > 1 && a->stride[i] != b->stride[i])) return false;
    return true;
}

// A [rows, heads, 128] view as the kernels take it.  The stride of a dimension of size 1 is
// never used to step and may hold anything: a stride that is valid everywhere stands in.
kda::RowsView rows_view(const kda_view* t, int row_dim) {
    kda::RowsView r;
    r.data = static_cast<__nv_bfloat16*>(t->data);
    r.head = t->shape[row_dim + 1] > 1 ? t->stride[row_dim + 1] : KDA_HEAD_DIM;
    r.row = t->shape[row_dim] > 1 ? t->stride[row_dim] : r.head * t->shape[row_dim + 1];
    return r;
}

kda_status check_state(const char* name, const kda_tensor* t, int64_t nseq, int64_t H) {
    if (!present(t)) return KDA_OK;
    if (t->dtype != KDA_BF16 && t->dtype != KDA_F32)
        return fail(KDA_ERR_INVALID_ARG, "%s: dtype must be bf16 or fp32", name);
    const int64_t shape[4] = {nseq, H, KDA_HEAD_DIM, KDA_HEAD_DIM};
    return check_tensor(name, t, t->dtype, 4, shape, 16);
}

kda_status check_states(const kda_tensor* init, const kda_tensor* fin, int64_t nseq, int64_t H) {
    KDA_TRY(check_state("initial_state", init, nseq, H));
    KDA_TRY(check_state("final_state", fin, nseq, H));
    if (present(init) && present(fin) && overlap(extent(init), extent(fin)) &&
        !(init->data == fin->data && init->dtype == fin->dtype))
        return fail(KDA_ERR_ALIAS, "initial_state and final_state overlap but are not the same buffer and dtype");
    return KDA_OK;
}

kda_status check_i64(const char* name, const kda_tensor* t, int64_t n) {
    const int64_t shape[1] = {n};
    return check_tensor(name, t, KDA_I64, 1, shape, 8);
}

kda_status check_workspace(void* workspace, size_t bytes, size_t need) {
    if (workspace == nullptr || (uintptr_t)workspace % 256 != 0)
        return fail(KDA_ERR_WORKSPACE, "workspace must be a 256-byte aligned device pointer");
    if (bytes < need) return fail(KDA_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", bytes, need);
    return KDA_OK;
}

// A cache in 4 bits, [nseq, S, Hk, 144] bytes.  Its last dimension and rank first, before the others are used.
kda_status check_qcache_rank(const kda_view* t) {
    if (!present(t)) return fail(KDA_ERR_INVALID_ARG, "cache: missing");
    if (t->dtype != KDA_U8) return fail(KDA_ERR_INVALID_ARG, "cache: dtype %d, expected uint8", t->dtype);
    if (t->ndim != 4 || t->shape[3] != KDA_QCACHE_ROW)
        return fail(KDA_ERR_INVALID_ARG, "cache: expected uint8 [N,S,Hk,%d]", KDA_QCACHE_ROW);
    return KDA_OK;
}
kda_status check_qcache(const kda_view* t, int64_t nseq, int64_t Hk) {
    if (t->shape[0] != nseq || t->shape[2] != Hk)
        return fail(KDA_ERR_INVALID_ARG, "cache: [%lld,%lld,%lld,144] for %lld sequences and %lld key heads", (long long)t->shape[0],
                    (long long)t->shape[1], (long long)t->shape[2], (long long)nseq, (long long)Hk);
    if (t->shape[1] < 0) return fail(KDA_ERR_INVALID_ARG, "cache: bad shape");
    if (t->shape[1] > (1 << 30)) return fail(KDA_ERR_UNSUPPORTED, "cache: more than 2^30 rows for a sequence");
    if (t->stride[3] != 1) return fail(KDA_ERR_INVALID_ARG, "cache: the innermost stride must be 1");
    for (int i = 0; i < 3; ++i) {
        if (t->shape[i] <= 1) continue;
        if (t->stride[i] < KDA_QCACHE_ROW || t->stride[i] % 16 != 0 || t->stride[i] >= (1LL << 39))
            return fail(KDA_ERR_INVALID_ARG, "cache: stride %lld of dim %d must be a multiple of 16, at least %d", (long long)t->stride[i],
                        i, KDA_QCACHE_ROW);
        if (t->shape[i] > (1LL << 48) / t->stride[i])
            return fail(KDA_ERR_INVALID_ARG, "cache: dim %d of %lld rows with stride %lld fits no memory", i, (long long)t->shape[i],
                        (long long)t->stride[i]);
    }
    if ((uintptr_t)t->data % 16 != 0) return fail(KDA_ERR_INVALID_ARG, "cache: data pointer not 16-byte aligned");
    return KDA_OK;
}
kda::QcacheView qcache_view(const kda_view* t) {
    kda::QcacheView r;
    r.data = static_cast<uint8_t*>(t->data);
    r.head = t->shape[2] > 1 ? t->stride[2] : KDA_QCACHE_ROW;
    r.row = t->shape[1] > 1 ? t->stride[1] : r.head * t->shape[2];
    r.seq = t->shape[0] > 1 ? t->stride[0] : r.row * t->shape[1];
    return r;
}

// A [T, D] view of rows of 16-byte groups; with `repeat` a token stride of 0 is taken too.
kda_status check_rows(const char* name, const kda_view* t, int32_t dtype, int64_t T, int64_t D, bool repeat, int64_t* row) {
    if (!present(t)) return fail(KDA_ERR_INVALID_ARG, "%s: missing", name);
    if (t->dtype != dtype) return fail(KDA_ERR_INVALID_ARG, "%s: dtype %d, expected %d", name, t->dtype, dtype);
    if (t->ndim != 2 || t->shape[0] != T || t->shape[1] != D)
        return fail(KDA_ERR_INVALID_ARG, "%s: expected [%lld,%lld]", name, (long long)T, (long long)D);
    if (t->stride[1] != 1) return fail(KDA_ERR_INVALID_ARG, "%s: the innermost stride must be 1", name);
    *row = 0;
    if (T > 1 && !(repeat && t->stride[0] == 0)) {
        if (t->stride[0] < D || t->stride[0] % 8 != 0 || T > (1LL << 48) / t->stride[0])
            return fail(KDA_ERR_INVALID_ARG, "%s: token stride %lld must be a multiple of 8, at least %lld", name, (long long)t->stride[0],
                        (long long)D);
        *row = t->stride[0];
    }
    if ((uintptr_t)t->data % 16 != 0) return fail(KDA_ERR_INVALID_ARG, "%s: data pointer not 16-byte aligned", name);
    return KDA_OK;
}

// The sequences of packed tokens: N from cu or from the cache; `uniform` tokens each without cu.
kda_status check_sequences(const char* name, const kda_tensor* cu, const kda_view* cache, int64_t tokens, int64_t* nseq, int64_t* uniform) {
    *nseq = cache->shape[0];
    if (present(cu)) {
        if (cu->ndim != 1 || cu->shape[0] < 1) return fail(KDA_ERR_INVALID_ARG, "%s: expected int64 [N+1]", name);
        *nseq = cu->shape[0] - 1;
    }
    if (*nseq < 0 || *nseq > INT32_MAX / 65536) return fail(KDA_ERR_UNSUPPORTED, "too many sequences");
    if (present(cu)) {
        KDA_TRY(check_i64(name, cu, *nseq + 1));
    } else if (*nseq == 0 ? tokens != 0 : tokens % *nseq != 0) {
        return fail(KDA_ERR_INVALID_ARG, "without %s the %lld tokens must divide into %lld sequences", name, (long long)tokens,
                    (long long)*nseq);
    }
    *uniform = *nseq > 0 ? tokens / *nseq : 0;
    return KDA_OK;
}

// Workspaces start with 256 bytes that hold the device status word.
constexpr size_t kHeaderBytes = 256;

void fill_states(kda::LinParams& p, const kda_tensor* init, const kda_tensor* fin) {
    p.init_state = present(init) ? init->data : nullptr;
    p.init_f32 = present(init) && init->dtype == KDA_F32;
    p.final_state = present(fin) ? fin->data : nullptr;
    p.final_f32 = present(fin) && fin->dtype == KDA_F32;
}

}  // namespace

extern "C" {

kda_status kda_qk_norm_rope(const kda_view* q, const kda_view* k, const kda_tensor* q_weight,
                            const kda_tensor* k_weight, float eps, const kda_tensor* cos_sin,
                            const kda_tensor* positions, const kda_view* q_out, const kda_view* k_out,
                            uint32_t* status, uint32_t flags, kda_stream_t stream) {
    kda::set_last_error("");
    if (flags & ~KDA_FLAG_ROPE_INTERLEAVED)
        return fail(KDA_ERR_INVALID_ARG, "flags: unknown bits 0x%x", flags & ~KDA_FLAG_ROPE_INTERLEAVED);
    if (!isfinite(eps) || eps < 0.f) return fail(KDA_ERR_INVALID_ARG, "eps must be finite and >= 0");
    if ((uintptr_t)status % 4 != 0) return fail(KDA_ERR_INVALID_ARG, "status: not 4-byte aligned");
    const bool has_k = present(k);
    if (has_k != present(k_out)) return fail(KDA_ERR_INVALID_ARG, "k and k_out must both be given, or neither");
    kda::NormRopeParams p;
    memset(&p, 0, sizeof(p));
    const kda_view* in[2] = {q, k};
    const kda_view* out[2] = {q_out, k_out};
    const kda_tensor* weight[2] = {q_weight, k_weight};
    const char* names[2][3] = {{"q", "q_out", "q_weight"}, {"k", "k_out", "k_weight"}};
    for (int i = 0; i < (has_k ? 2 : 1); ++i) {
        KDA_TRY(check_head_dim(names[i][0], in[i], 3));
        const int64_t T = q->shape[0], heads = in[i]->shape[1];
        if (T < 0 || heads < 1) return fail(KDA_ERR_INVALID_ARG, "%s: bad shape [%lld,%lld,128]", names[i][0],
                                            (long long)T, (long long)heads);
        if (T > INT32_MAX || heads > 65535) return fail(KDA_ERR_UNSUPPORTED, "%s: T must be < 2^31 and heads <= 65535", names[i][0]);
        const int64_t shape[3] = {T, heads, KDA_HEAD_DIM};
        KDA_TRY(check_view(names[i][0], in[i], 3, shape));
        KDA_TRY(check_view(names[i][1], out[i], 3, shape));
        const int64_t wshape[1] = {KDA_HEAD_DIM};
        if (present(weight[i])) {
            KDA_TRY(check_tensor(names[i][2], weight[i], KDA_F32, 1, wshape, 16));
            p.weight[i] = static_cast<const float*>(weight[i]->data);
        }
        p.x[i] = rows_view(in[i], 0);
        p.y[i] = rows_view(out[i], 0);
        p.heads[i] = (int)heads;
    }
    if (present(cos_sin) != present(positions))
        return fail(KDA_ERR_INVALID_ARG, "cos_sin and positions must both be given, or neither");
    if (present(cos_sin)) {
        if (cos_sin->dtype != KDA_F32 || cos_sin->ndim != 2) return fail(KDA_ERR_INVALID_ARG, "cos_sin: expected fp32 [P, R]");
        const int64_t R = cos_sin->shape[1];
        if (R < 16 || R > KDA_HEAD_DIM || R % 16 != 0)
            return fail(KDA_ERR_UNSUPPORTED, "cos_sin: R = %lld, must be a multiple of 16 in [16, 128]", (long long)R);
        if (cos_sin->shape[0] < 0 || cos_sin->shape[0] > (1LL << 40))
            return fail(KDA_ERR_INVALID_ARG, "cos_sin: bad shape [%lld,%lld]", (long long)cos_sin->shape[0], (long long)R);
        if ((uintptr_t)cos_sin->data % 16 != 0) return fail(KDA_ERR_INVALID_ARG, "cos_sin: data pointer not 16-byte aligned");
        KDA_TRY(check_i64("positions", positions, q->shape[0]));
        p.cos_sin = static_cast<const float*>(cos_sin->data);
        p.positions = static_cast<const int64_t*>(positions->data);
        p.table_rows = cos_sin->shape[0];
        p.rot = (int)R;
    }
    for (int i = 0; i < (has_k ? 2 : 1); ++i) {
        const Extent o = extent(out[i]);
        for (int j = 0; j < (has_k ? 2 : 1); ++j) {
            if (overlap(o, extent(in[j])) && !(i == j && same_view(in[j], out[i])))
                return fail(KDA_ERR_ALIAS, "%s overlaps %s and is not exactly the same view", names[i][1], names[j][0]);
            if (j > i && overlap(o, extent(out[j]))) return fail(KDA_ERR_ALIAS, "q_out and k_out overlap");
        }
        for (const kda_tensor* t : {q_weight, k_weight, cos_sin, positions})
            if (present(t) && overlap(o, extent(t))) return fail(KDA_ERR_ALIAS, "%s overlaps another tensor", names[i][1]);
    }
    p.tokens = q->shape[0];
    p.status = status;
    p.eps = eps;
    p.interleaved = (flags & KDA_FLAG_ROPE_INTERLEAVED) != 0;
    const cudaError_t e = kda::launch_norm_rope(p, reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return fail(KDA_ERR_CUDA, "norm and rotation launch: %s", cudaGetErrorString(e));
    return KDA_OK;
}

size_t kda_attn_workspace_size(int64_t Tq, int Hq, int Hk) {
    if (Tq < 0 || Hq < 1 || Hk < 1 || Hq % Hk != 0) return 0;
    return kHeaderBytes + kda::attn_workspace_bytes(Tq, Hq, Hk);
}

kda_status kda_attn_fwd(const kda_view* q, const kda_view* k, const kda_view* v, float scale,
                        const kda_view* out, const kda_tensor* lse, const kda_tensor* cu_seqlens_q,
                        const kda_tensor* cu_seqlens_k, const kda_tensor* seqlens_k, void* workspace,
                        size_t workspace_bytes, kda_stream_t stream) {
    kda::set_last_error("");
    if (!isfinite(scale) || scale < 0.f) return fail(KDA_ERR_INVALID_ARG, "scale must be finite and >= 0");
    KDA_TRY(check_head_dim("q", q, 3));
    if (!present(k)) return fail(KDA_ERR_INVALID_ARG, "k: missing");
    if (k->ndim != 3 && k->ndim != 4)
        return fail(KDA_ERR_INVALID_ARG, "k: ndim %d, expected 3 [Tk,Hk,128] or 4 [N,S,Hk,128]", k->ndim);
    const bool cache = k->ndim == 4;
    KDA_TRY(check_head_dim("k", k, k->ndim));
    const int64_t Tq = q->shape[0], Hq = q->shape[1];
    const int64_t Tk = k->shape[cache ? 1 : 0], Hk = k->shape[cache ? 2 : 1];
    if (Tq < 0 || Hq < 1 || Tk < 0 || Hk < 1) return fail(KDA_ERR_INVALID_ARG, "bad q or k shape");
    if (Hq % Hk != 0) return fail(KDA_ERR_INVALID_ARG, "%lld query heads do not divide into %lld key heads", (long long)Hq, (long long)Hk);
    if (Tq > (1 << 30) || Tk > (1 << 30) || Hq > 65535 || Hq / Hk > 128)
        return fail(KDA_ERR_UNSUPPORTED, "Tq and Tk must be <= 2^30, Hq <= 65535 and Hq / Hk <= 128");
    // the sequences
    int64_t nseq = -1;
    if (present(cu_seqlens_q)) {
        if (cu_seqlens_q->ndim != 1 || cu_seqlens_q->shape[0] < 1) return fail(KDA_ERR_INVALID_ARG, "cu_seqlens_q: expected int64 [N+1]");
        nseq = cu_seqlens_q->shape[0] - 1;
    } else if (cache) {
        nseq = k->shape[0];
    } else if (present(cu_seqlens_k)) {
        if (cu_seqlens_k->ndim != 1 || cu_seqlens_k->shape[0] < 1) return fail(KDA_ERR_INVALID_ARG, "cu_seqlens_k: expected int64 [N+1]");
        nseq = cu_seqlens_k->shape[0] - 1;
    } else {
        nseq = 1;
    }
    if (nseq < 0 || nseq > INT32_MAX / 65536) return fail(KDA_ERR_UNSUPPORTED, "too many sequences");
    if (present(cu_seqlens_q)) {
        KDA_TRY(check_i64("cu_seqlens_q", cu_seqlens_q, nseq + 1));
    } else if (nseq == 0 ? Tq != 0 : Tq % nseq != 0) {
        return fail(KDA_ERR_INVALID_ARG, "without cu_seqlens_q the %lld queries must divide into %lld sequences", (long long)Tq, (long long)nseq);
    }
    if (cache) {
        if (present(cu_seqlens_k)) return fail(KDA_ERR_INVALID_ARG, "cu_seqlens_k: not taken with a cache");
        KDA_TRY(check_i64("seqlens_k", seqlens_k, nseq));
    } else {
        if (present(seqlens_k)) return fail(KDA_ERR_INVALID_ARG, "seqlens_k: taken with a cache [N,S,Hk,128] only");
        if (present(cu_seqlens_k)) {
            KDA_TRY(check_i64("cu_seqlens_k", cu_seqlens_k, nseq + 1));
        } else if (present(cu_seqlens_q) && Tk != Tq) {
            return fail(KDA_ERR_INVALID_ARG, "without cu_seqlens_k, k must have the %lld rows of q", (long long)Tq);
        }
    }
    const int64_t qshape[3] = {Tq, Hq, KDA_HEAD_DIM};
    const int64_t kpacked[3] = {Tk, Hk, KDA_HEAD_DIM}, kcache[4] = {nseq, Tk, Hk, KDA_HEAD_DIM};
    KDA_TRY(check_view("q", q, 3, qshape));
    KDA_TRY(check_view("k", k, cache ? 4 : 3, cache ? kcache : kpacked));
    KDA_TRY(check_view("v", v, cache ? 4 : 3, cache ? kcache : kpacked));
    KDA_TRY(check_view("out", out, 3, qshape));
    if (present(lse)) {
        const int64_t lshape[2] = {Tq, Hq};
        KDA_TRY(check_tensor("lse", lse, KDA_F32, 2, lshape, 4));
    }
    for (const kda_view* t : {q, k, v})
        if (overlap(extent(out), extent(t)) || (present(lse) && overlap(extent(lse), extent(t))))
            return fail(KDA_ERR_ALIAS, "out or lse overlaps an input");
    for (const kda_tensor* t : {cu_seqlens_q, cu_seqlens_k, seqlens_k})
        if (present(t) && (overlap(extent(out), extent(t)) || (present(lse) && overlap(extent(lse), extent(t)))))
            return fail(KDA_ERR_ALIAS, "out or lse overlaps the lengths");
    if (present(lse) && overlap(extent(out), extent(lse))) return fail(KDA_ERR_ALIAS, "out and lse overlap");
    KDA_TRY(check_workspace(workspace, workspace_bytes, kda_attn_workspace_size(Tq, (int)Hq, (int)Hk)));

    kda::AttnParams p;
    memset(&p, 0, sizeof(p));
    p.q = rows_view(q, 0);
    p.out = rows_view(out, 0);
    const kda::RowsView kr = rows_view(k, cache ? 1 : 0), vr = rows_view(v, cache ? 1 : 0);
    p.k = kr.data;
    p.k_row = kr.row;
    p.k_head = kr.head;
    p.k_seq = !cache ? 0 : k->shape[0] > 1 ? k->stride[0] : kr.row * Tk;
    p.v = vr.data;
    p.v_row = vr.row;
    p.v_head = vr.head;
    p.v_seq = !cache ? 0 : v->shape[0] > 1 ? v->stride[0] : vr.row * Tk;
    p.lse = present(lse) ? static_cast<float*>(lse->data) : nullptr;
    p.lse_row = Hq;
    p.keys = Tk;
    p.cu_q = present(cu_seqlens_q) ? static_cast<const int64_t*>(cu_seqlens_q->data) : nullptr;
    p.uniform_q = nseq > 0 ? Tq / nseq : 0;
    p.cu_k = cache ? nullptr : present(cu_seqlens_k) ? static_cast<const int64_t*>(cu_seqlens_k->data) : p.cu_q;
    p.seqlens_k = cache ? static_cast<const int64_t*>(seqlens_k->data) : nullptr;
    p.Tq = Tq;
    p.Tk = Tk;
    p.nseq = (int)nseq;
    p.Hq = (int)Hq;
    p.Hk = (int)Hk;
    p.cache = cache;
    p.scale = scale;
    p.status = static_cast<uint32_t*>(workspace);
    p.workspace = static_cast<char*>(workspace) + kHeaderBytes;
    p.test_skip = test_skip();
    const cudaError_t e = kda::launch_attn(p, reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return fail(KDA_ERR_CUDA, "attention launch: %s", cudaGetErrorString(e));
    return KDA_OK;
}

size_t kda_lin_workspace_size(int64_t T_total, int H, int N) {
    if (T_total < 0 || H < 0 || N < 0) return 0;
    return kHeaderBytes + kda::lin_workspace_bytes(T_total, H, N);
}

kda_status kda_lin_fwd(const kda_view* q, const kda_view* k, const kda_view* v, const kda_tensor* log_decay,
                       float scale, const kda_view* out, const kda_tensor* initial_state,
                       const kda_tensor* final_state, const kda_tensor* cu_seqlens, void* workspace,
                       size_t workspace_bytes, kda_stream_t stream) {
    kda::set_last_error("");
    if (!isfinite(scale)) return fail(KDA_ERR_INVALID_ARG, "scale must be finite");
    KDA_TRY(check_head_dim("q", q, 4));
    const int64_t B = q->shape[0], T = q->shape[1], H = q->shape[2];
    if (B < 1 || T < 0 || H < 1) return fail(KDA_ERR_INVALID_ARG, "bad q shape [%lld,%lld,%lld,128]", (long long)B, (long long)T, (long long)H);
    if (B > INT32_MAX || T > INT32_MAX || B * T > (int64_t)INT32_MAX || H > 65535)
        return fail(KDA_ERR_UNSUPPORTED, "B*T must be < 2^31 and H <= 65535");
    const int64_t shape[4] = {B, T, H, KDA_HEAD_DIM};
    const kda_view* views[4] = {q, k, v, out};
    const char* names[4] = {"q", "k", "v", "out"};
    kda::LinParams p;
    memset(&p, 0, sizeof(p));
    kda::RowsView* rows[4] = {&p.q, &p.k, &p.v, &p.out};
    for (int i = 0; i < 4; ++i) {
        KDA_TRY(check_view(names[i], views[i], 4, shape));
        // the batch rows follow each other: token b T + t is row b T + t of one [B T, H, 128] view
        if (B > 1 && T > 1 && views[i]->stride[0] != T * views[i]->stride[1])
            return fail(KDA_ERR_INVALID_ARG, "%s: the batch stride must be T times the token stride", names[i]);
        *rows[i] = rows_view(views[i], 1);
        if (T == 1 && B > 1) rows[i]->row = views[i]->stride[0];
    }
    const int64_t hshape[1] = {H};
    KDA_TRY(check_tensor("log_decay", log_decay, KDA_F32, 1, hshape, 4));
    int64_t nseq = B;
    if (present(cu_seqlens)) {
        if (cu_seqlens->ndim != 1 || cu_seqlens->shape[0] < 1) return fail(KDA_ERR_INVALID_ARG, "cu_seqlens: expected int64 [N+1]");
        if (B != 1) return fail(KDA_ERR_INVALID_ARG, "packed mode (cu_seqlens) requires B == 1");
        nseq = cu_seqlens->shape[0] - 1;
        KDA_TRY(check_i64("cu_seqlens", cu_seqlens, nseq + 1));
    }
    if (nseq > (int64_t)INT32_MAX / 65536) return fail(KDA_ERR_UNSUPPORTED, "too many sequences");
    KDA_TRY(check_states(initial_state, final_state, nseq, H));
    const Extent o = extent(out);
    for (int i = 0; i < 3; ++i)
        if (overlap(o, extent(views[i]))) return fail(KDA_ERR_ALIAS, "out overlaps %s", names[i]);
    for (const kda_tensor* t : {log_decay, initial_state, final_state, cu_seqlens})
        if (present(t) && overlap(o, extent(t))) return fail(KDA_ERR_ALIAS, "out overlaps another tensor");
    if (present(final_state)) {   // (the lengths are read until the last unit is done)
        for (int i = 0; i < 3; ++i)
            if (overlap(extent(final_state), extent(views[i]))) return fail(KDA_ERR_ALIAS, "final_state overlaps %s", names[i]);
        for (const kda_tensor* t : {log_decay, cu_seqlens})
            if (present(t) && overlap(extent(final_state), extent(t)))
                return fail(KDA_ERR_ALIAS, "final_state overlaps log_decay or cu_seqlens");
    }
    KDA_TRY(check_workspace(workspace, workspace_bytes, kda_lin_workspace_size(B * T, (int)H, (int)nseq)));
    p.log_decay = static_cast<const float*>(log_decay->data);
    fill_states(p, initial_state, final_state);
    p.cu_seqlens = present(cu_seqlens) ? static_cast<const int64_t*>(cu_seqlens->data) : nullptr;
    p.T = T;
    p.T_total = B * T;
    p.H = (int)H;
    p.nseq = (int)nseq;
    p.scale = scale;
    p.status = static_cast<uint32_t*>(workspace);
    p.workspace = static_cast<char*>(workspace) + kHeaderBytes;
    p.test_skip = test_skip();
    const cudaError_t e = kda::launch_lin_fwd(p, reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return fail(KDA_ERR_CUDA, "linear attention launch: %s", cudaGetErrorString(e));
    return KDA_OK;
}

kda_status kda_lin_decode(const kda_view* q, const kda_view* k, const kda_view* v, const kda_tensor* log_decay,
                          float scale, const kda_view* out, const kda_tensor* initial_state,
                          const kda_tensor* final_state, kda_stream_t stream) {
    kda::set_last_error("");
    if (!isfinite(scale)) return fail(KDA_ERR_INVALID_ARG, "scale must be finite");
    KDA_TRY(check_head_dim("q", q, 3));
    const int64_t B = q->shape[0], H = q->shape[1];
    if (B < 0 || H < 1) return fail(KDA_ERR_INVALID_ARG, "bad q shape [%lld,%lld,128]", (long long)B, (long long)H);
    if (B > INT32_MAX || H > 65535 || B * H > (int64_t)INT32_MAX / 16) return fail(KDA_ERR_UNSUPPORTED, "B*H too large");
    const int64_t shape[3] = {B, H, KDA_HEAD_DIM};
    const kda_view* views[4] = {q, k, v, out};
    const char* names[4] = {"q", "k", "v", "out"};
    kda::LinParams p;
    memset(&p, 0, sizeof(p));
    kda::RowsView* rows[4] = {&p.q, &p.k, &p.v, &p.out};
    for (int i = 0; i < 4; ++i) {
        KDA_TRY(check_view(names[i], views[i], 3, shape));
        *rows[i] = rows_view(views[i], 0);
    }
    const int64_t hshape[1] = {H};
    KDA_TRY(check_tensor("log_decay", log_decay, KDA_F32, 1, hshape, 4));
    KDA_TRY(check_states(initial_state, final_state, B, H));
    const Extent o = extent(out);
    for (int i = 0; i < 3; ++i) {
        if (overlap(o, extent(views[i]))) return fail(KDA_ERR_ALIAS, "out overlaps %s", names[i]);
        if (present(final_state) && overlap(extent(final_state), extent(views[i])))
            return fail(KDA_ERR_ALIAS, "final_state overlaps %s", names[i]);
    }
    if (present(final_state) && overlap(extent(final_state), extent(log_decay)))
        return fail(KDA_ERR_ALIAS, "final_state overlaps log_decay");
    for (const kda_tensor* t : {log_decay, initial_state, final_state})
        if (present(t) && overlap(o, extent(t))) return fail(KDA_ERR_ALIAS, "out overlaps another tensor");
    p.log_decay = static_cast<const float*>(log_decay->data);
    fill_states(p, initial_state, final_state);
    p.T = 1;
    p.T_total = B;
    p.H = (int)H;
    p.nseq = (int)B;
    p.scale = scale;
    const cudaError_t e = kda::launch_lin_decode(p, reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return fail(KDA_ERR_CUDA, "linear attention step launch: %s", cudaGetErrorString(e));
    return KDA_OK;
}

kda_status kda_qcache_append(const kda_view* k, const kda_view* v, const kda_view* cache, const kda_tensor* seqlens_k,
                             const kda_tensor* cu_seqlens, const kda_view* k_out, const kda_view* v_out, uint32_t* status,
                             kda_stream_t stream) {
    kda::set_last_error("");
    if ((uintptr_t)status % 4 != 0) return fail(KDA_ERR_INVALID_ARG, "status: not 4-byte aligned");
    KDA_TRY(check_head_dim("k", k, 3));
    const int64_t T = k->shape[0], Hk = k->shape[1];
    if (T < 0 || Hk < 1) return fail(KDA_ERR_INVALID_ARG, "k: bad shape [%lld,%lld,128]", (long long)T, (long long)Hk);
    if (T > (1 << 30) || Hk > 65535) return fail(KDA_ERR_UNSUPPORTED, "T must be <= 2^30 and Hk <= 65535");
    const int64_t shape[3] = {T, Hk, KDA_HEAD_DIM};
    KDA_TRY(check_view("k", k, 3, shape));
    KDA_TRY(check_view("v", v, 3, shape));
    KDA_TRY(check_qcache_rank(cache));
    int64_t nseq, uniform;
    KDA_TRY(check_sequences("cu_seqlens", cu_seqlens, cache, T, &nseq, &uniform));
    KDA_TRY(check_qcache(cache, nseq, Hk));
    KDA_TRY(check_i64("seqlens_k", seqlens_k, nseq));
    if (present(k_out) != present(v_out)) return fail(KDA_ERR_INVALID_ARG, "k_out and v_out must both be given, or neither");
    if (present(k_out)) {
        KDA_TRY(check_view("k_out", k_out, 3, shape));
        KDA_TRY(check_view("v_out", v_out, 3, shape));
    }
    const kda_view* written[3] = {cache, k_out, v_out};
    const char* names[3] = {"cache", "k_out", "v_out"};
    for (int i = 0; i < 3; ++i) {
        if (!present(written[i])) continue;
        KDA_TRY(check_written(names[i], written[i]));
        const Extent o = extent(written[i]);
        for (int j = 0; j < 2; ++j)
            if (overlap(o, extent(j ? v : k)) && !(i == j + 1 && same_view(written[i], j ? v : k)))
                return fail(KDA_ERR_ALIAS, "%s overlaps %s", names[i], j ? "v" : "k");
        for (int j = i + 1; j < 3; ++j)
            if (present(written[j]) && overlap(o, extent(written[j]))) return fail(KDA_ERR_ALIAS, "%s and %s overlap", names[i], names[j]);
        for (const kda_tensor* t : {seqlens_k, cu_seqlens})
            if (present(t) && overlap(o, extent(t))) return fail(KDA_ERR_ALIAS, "%s overlaps the lengths", names[i]);
    }
    kda::QcacheAppendParams p;
    memset(&p, 0, sizeof(p));
    p.k = rows_view(k, 0);
    p.v = rows_view(v, 0);
    if (present(k_out)) {
        p.k_out = rows_view(k_out, 0);
        p.v_out = rows_view(v_out, 0);
    }
    p.cache = qcache_view(cache);
    p.seqlens_k = static_cast<const int64_t*>(seqlens_k->data);
    p.cu = present(cu_seqlens) ? static_cast<const int64_t*>(cu_seqlens->data) : nullptr;
    p.uniform = uniform;
    p.T = T;
    p.S = cache->shape[1];
    p.nseq = (int)nseq;
    p.Hk = (int)Hk;
    p.status = status;
    const cudaError_t e = kda::launch_qcache_append(p, reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return fail(KDA_ERR_CUDA, "cache append launch: %s", cudaGetErrorString(e));
    return KDA_OK;
}

size_t kda_attn_qcache_workspace_size(int64_t Tq, int Hq, int Hk, int N, int64_t S) {
    if (Tq < 0 || Tq > (1 << 30) || Hq < 1 || Hk < 1 || Hq % Hk != 0 || N < 0 || S < 0 || S > (1 << 30)) return 0;
    return kHeaderBytes + kda::attn_qcache_workspace_bytes(Tq, Hq, Hk, N, S);
}

kda_status kda_attn_qcache_fwd(const kda_view* q, const kda_view* cache, float scale, const kda_view* out,
                               const kda_tensor* seqlens_k, const kda_tensor* lse, const kda_tensor* cu_seqlens_q,
                               void* workspace, size_t workspace_bytes, kda_stream_t stream) {
    kda::set_last_error("");
    if (!isfinite(scale) || scale < 0.f) return fail(KDA_ERR_INVALID_ARG, "scale must be finite and >= 0");
    KDA_TRY(check_head_dim("q", q, 3));
    KDA_TRY(check_qcache_rank(cache));
    const int64_t Tq = q->shape[0], Hq = q->shape[1], Hk = cache->shape[2];
    if (Tq < 0 || Hq < 1 || Hk < 1) return fail(KDA_ERR_INVALID_ARG, "bad q or cache shape");
    if (Hq % Hk != 0) return fail(KDA_ERR_INVALID_ARG, "%lld query heads do not divide into %lld key heads", (long long)Hq, (long long)Hk);
    if (Tq > (1 << 30) || Hq > 65535 || Hq / Hk > 128)
        return fail(KDA_ERR_UNSUPPORTED, "Tq must be <= 2^30, Hq <= 65535 and Hq / Hk <= 128");
    int64_t nseq, uniform;
    KDA_TRY(check_sequences("cu_seqlens_q", cu_seqlens_q, cache, Tq, &nseq, &uniform));
    KDA_TRY(check_qcache(cache, nseq, Hk));
    KDA_TRY(check_i64("seqlens_k", seqlens_k, nseq));
    const int64_t qshape[3] = {Tq, Hq, KDA_HEAD_DIM};
    KDA_TRY(check_view("q", q, 3, qshape));
    KDA_TRY(check_view("out", out, 3, qshape));
    if (present(lse)) {
        const int64_t lshape[2] = {Tq, Hq};
        KDA_TRY(check_tensor("lse", lse, KDA_F32, 2, lshape, 4));
    }
    KDA_TRY(check_written("out", out));
    for (const kda_view* t : {q, cache})
        if (overlap(extent(out), extent(t)) || (present(lse) && overlap(extent(lse), extent(t))))
            return fail(KDA_ERR_ALIAS, "out or lse overlaps an input");
    for (const kda_tensor* t : {cu_seqlens_q, seqlens_k})
        if (present(t) && (overlap(extent(out), extent(t)) || (present(lse) && overlap(extent(lse), extent(t)))))
            return fail(KDA_ERR_ALIAS, "out or lse overlaps the lengths");
    if (present(lse) && overlap(extent(out), extent(lse))) return fail(KDA_ERR_ALIAS, "out and lse overlap");
    KDA_TRY(check_workspace(workspace, workspace_bytes, kda_attn_qcache_workspace_size(Tq, (int)Hq, (int)Hk, (int)nseq, cache->shape[1])));
    kda::QcacheAttnParams p;
    memset(&p, 0, sizeof(p));
    p.q = rows_view(q, 0);
    p.out = rows_view(out, 0);
    p.cache = qcache_view(cache);
    p.lse = present(lse) ? static_cast<float*>(lse->data) : nullptr;
    p.cu_q = present(cu_seqlens_q) ? static_cast<const int64_t*>(cu_seqlens_q->data) : nullptr;
    p.seqlens_k = static_cast<const int64_t*>(seqlens_k->data);
    p.uniform_q = uniform;
    p.Tq = Tq;
    p.S = cache->shape[1];
    p.nseq = (int)nseq;
    p.Hq = (int)Hq;
    p.Hk = (int)Hk;
    p.scale = scale;
    p.status = static_cast<uint32_t*>(workspace);
    p.workspace = static_cast<char*>(workspace) + kHeaderBytes;
    p.test_skip = test_skip();
    const cudaError_t e = kda::launch_attn_qcache(p, reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return fail(KDA_ERR_CUDA, "attention launch: %s", cudaGetErrorString(e));
    return KDA_OK;
}

kda_status kda_gated_norm(const kda_view* x, const kda_view* gate, const kda_tensor* weight, const kda_view* out, float eps,
                          uint32_t flags, kda_stream_t stream) {
    kda::set_last_error("");
    if (flags & ~KDA_FLAG_GATE_SILU) return fail(KDA_ERR_INVALID_ARG, "flags: unknown bits 0x%x", flags & ~KDA_FLAG_GATE_SILU);
    if (!isfinite(eps) || eps < 0.f) return fail(KDA_ERR_INVALID_ARG, "eps must be finite and >= 0");
    KDA_TRY(check_head_dim("x", x, 3));
    const int64_t T = x->shape[0], H = x->shape[1];
    if (T < 0 || H < 1) return fail(KDA_ERR_INVALID_ARG, "x: bad shape [%lld,%lld,128]", (long long)T, (long long)H);
    if (T > INT32_MAX || H > 65535) return fail(KDA_ERR_UNSUPPORTED, "T must be < 2^31 and H <= 65535");
    const int64_t shape[3] = {T, H, KDA_HEAD_DIM}, wshape[1] = {KDA_HEAD_DIM};
    KDA_TRY(check_view("x", x, 3, shape));
    KDA_TRY(check_view("gate", gate, 3, shape));
    KDA_TRY(check_view("out", out, 3, shape));
    if (present(weight)) KDA_TRY(check_tensor("weight", weight, KDA_F32, 1, wshape, 16));
    KDA_TRY(check_written("out", out));
    const Extent o = extent(out);
    if (overlap(o, extent(x)) && !same_view(out, x)) return fail(KDA_ERR_ALIAS, "out overlaps x and is not exactly the same view");
    if (overlap(o, extent(gate)) && !same_view(out, gate)) return fail(KDA_ERR_ALIAS, "out overlaps gate and is not exactly the same view");
    if (present(weight) && overlap(o, extent(weight))) return fail(KDA_ERR_ALIAS, "out overlaps weight");
    kda::GatedNormParams p;
    memset(&p, 0, sizeof(p));
    p.x = rows_view(x, 0);
    p.gate = rows_view(gate, 0);
    p.out = rows_view(out, 0);
    p.weight = present(weight) ? static_cast<const float*>(weight->data) : nullptr;
    p.tokens = T;
    p.heads = (int)H;
    p.eps = eps;
    p.silu = (flags & KDA_FLAG_GATE_SILU) != 0;
    const cudaError_t e = kda::launch_gated_norm(p, reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return fail(KDA_ERR_CUDA, "gated norm launch: %s", cudaGetErrorString(e));
    return KDA_OK;
}

kda_status kda_residual_norm(const kda_view* y, const kda_view* residual, const kda_tensor* post_weight, const kda_view* gate,
                             float scale, const kda_tensor* pre_weight, const kda_view* residual_out, const kda_view* out,
                             float eps, kda_stream_t stream) {
    kda::set_last_error("");
    if (!isfinite(scale)) return fail(KDA_ERR_INVALID_ARG, "scale must be finite");
    if (!isfinite(eps) || eps < 0.f) return fail(KDA_ERR_INVALID_ARG, "eps must be finite and >= 0");
    if (!present(residual)) return fail(KDA_ERR_INVALID_ARG, "residual: missing");
    if (residual->dtype != KDA_BF16 && residual->dtype != KDA_F32) return fail(KDA_ERR_INVALID_ARG, "residual: dtype must be bf16 or fp32");
    if (residual->ndim != 2) return fail(KDA_ERR_INVALID_ARG, "residual: expected [T,D]");
    const int64_t T = residual->shape[0], D = residual->shape[1];
    if (T < 0 || D < 1) return fail(KDA_ERR_INVALID_ARG, "residual: bad shape [%lld,%lld]", (long long)T, (long long)D);
    if (T > INT32_MAX || D % 8 != 0 || D > KDA_RESIDUAL_MAX_DIM)
        return fail(KDA_ERR_UNSUPPORTED, "T must be < 2^31, and D a multiple of 8 up to %d", KDA_RESIDUAL_MAX_DIM);
    if (!present(y) && (present(post_weight) || present(gate) || present(residual_out)))
        return fail(KDA_ERR_INVALID_ARG, "without y, post_weight, gate and residual_out must be absent too");
    kda::ResidualNormParams p;
    memset(&p, 0, sizeof(p));
    if (present(y)) KDA_TRY(check_rows("y", y, KDA_BF16, T, D, false, &p.y_row));
    KDA_TRY(check_rows("residual", residual, residual->dtype, T, D, false, &p.residual_row));
    if (present(gate)) KDA_TRY(check_rows("gate", gate, KDA_BF16, T, D, true, &p.gate_row));
    if (present(residual_out)) KDA_TRY(check_rows("residual_out", residual_out, residual->dtype, T, D, false, &p.residual_out_row));
    KDA_TRY(check_rows("out", out, KDA_BF16, T, D, false, &p.out_row));
    const int64_t wshape[1] = {D};
    if (present(post_weight)) KDA_TRY(check_tensor("post_weight", post_weight, KDA_F32, 1, wshape, 16));
    if (present(pre_weight)) KDA_TRY(check_tensor("pre_weight", pre_weight, KDA_F32, 1, wshape, 16));
    // every token is read before it is written, by the threads that write it
    const kda_view* written[2] = {out, residual_out};
    const char* names[2] = {"out", "residual_out"};
    for (int i = 0; i < 2; ++i) {
        if (!present(written[i])) continue;
        const Extent o = extent(written[i]);
        const bool over_y = i == 0, over_residual = i == 1 || (!present(residual_out) && residual->dtype == KDA_BF16);
        if (present(y) && overlap(o, extent(y)) && !(over_y && same_view(written[i], y)))
            return fail(KDA_ERR_ALIAS, "%s overlaps y", names[i]);
        if (overlap(o, extent(residual)) && !(over_residual && same_view(written[i], residual)))
            return fail(KDA_ERR_ALIAS, "%s overlaps residual", names[i]);
        if (present(gate)) {
            kda_view g = *gate;
            if (p.gate_row == 0) g.shape[0] = T > 0 ? 1 : 0;   // (one row, repeated)
            if (overlap(o, extent(&g))) return fail(KDA_ERR_ALIAS, "%s overlaps gate", names[i]);
        }
        for (const kda_tensor* t : {post_weight, pre_weight})
            if (present(t) && overlap(o, extent(t))) return fail(KDA_ERR_ALIAS, "%s overlaps a weight", names[i]);
    }
    if (present(residual_out) && overlap(extent(out), extent(residual_out))) return fail(KDA_ERR_ALIAS, "out and residual_out overlap");
    p.y = present(y) ? static_cast<const __nv_bfloat16*>(y->data) : nullptr;
    p.gate = present(gate) ? static_cast<const __nv_bfloat16*>(gate->data) : nullptr;
    p.residual = residual->data;
    p.residual_out = present(residual_out) ? residual_out->data : nullptr;
    p.out = static_cast<__nv_bfloat16*>(out->data);
    p.post_weight = present(post_weight) ? static_cast<const float*>(post_weight->data) : nullptr;
    p.pre_weight = present(pre_weight) ? static_cast<const float*>(pre_weight->data) : nullptr;
    p.tokens = T;
    p.dim = (int)D;
    p.f32 = residual->dtype == KDA_F32;
    p.scale = scale;
    p.eps = eps;
    const cudaError_t e = kda::launch_residual_norm(p, reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return fail(KDA_ERR_CUDA, "residual norm launch: %s", cudaGetErrorString(e));
    return KDA_OK;
}

}  // extern "C"
