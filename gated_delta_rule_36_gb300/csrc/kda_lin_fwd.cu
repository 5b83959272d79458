// Linear attention with a decay for each head over whole prompts, in chunks of C = 128 tokens
// on the 5th-generation tensor cores.  With a = exp(log_decay) and i, j the tokens of a chunk,
//   out_i = scale a^(i+1) S q_i + scale sum_{j <= i} a^(i-j) (q_i . k_j) v_j
//   S     <- a^C S + sum_j (a^(C-1-j) k_j) v_j^T          (kept as K x V: lane k, column v)
// as four products of 128 x 128 x 128 a chunk:
//   W  = Q K^T                    P = W scaled by a^(i-j), masked, in bf16, over W in Tensor Memory
//   O  = Q S                      then each row scaled by scale a^(i+1)
//   KV = K'^T V                   K' = a^(C-1-j) K split into three bf16 terms (24 bits, the width of
//                                 fp32), so that the state is updated to fp32 accuracy
//   O += P V
// The state lives in registers in fp32: KV is a fresh accumulator for each chunk, added with
// rounding to nearest (accumulating a whole sequence in the tensor core would truncate at
// every step).  Its bf16 copy in shared memory is O's operand only.
//
// One persistent CTA per SM takes an equal, contiguous share of all chunks of all (sequence,
// head) units.  A share that starts inside a unit needs the state before it: a first launch
// (kStateOnly) sums v k^T over the share ends that a later share continues, and the second
// starts from their decayed sum.
//
// Warp roles (three warpgroups): warps 0-3 turn W into P, scale O and write the output (thread =
// token row); warps 4-7 make K' and carry the state (thread = key channel); warp 8 loads q, k,
// v by TMA through a ring of two chunks; warp 9 issues the MMAs.  Every wait is bounded.
//
// Bound by HBM: 1,024 bytes a token-head against 4 x 128 x 128 x 2 (+ 2 x the state's extra
// terms) flop; a chunk at HBM speed lasts about 5,700 SM cycles, its MMAs 3,072.
#include "kda_mixer.cuh"

namespace kda {
namespace {

constexpr int LF_C = 128;            // tokens a chunk
constexpr int LF_THREADS = 384;      // three warpgroups, the third with two idle warps
constexpr int LF_MAX_CTAS = 160;     // shares (and partial states) at most
constexpr uint32_t TILE = 128 * 256; // one 128 x 128 bf16 tile: two 64-channel halves of 16 KB
constexpr uint32_t HALF = TILE / 2;
constexpr uint32_t STAGE = 3 * TILE; // q, k, v
constexpr uint32_t OFF_S = 2 * STAGE;
constexpr uint32_t OFF_POW = OFF_S + TILE;       // per warp: a^(31 - j), j < 32; and a short chunk's weights
constexpr uint32_t OFF_BAR = OFF_POW + 12 * 128;
enum { FQ = 0, FK = 2, FV = 4, EQ = 6, EK = 8, EV = 10, KPF = 12, KPE = 14, WF = 16, PF, QSF, OS, OF, OE, KVF, SB, DRAIN, NBAR };
constexpr uint32_t OFF_MISC = OFF_BAR + NBAR * 8;   // tmem address, abort flag, scan scratch
constexpr uint32_t LF_SMEM = OFF_MISC + 128 + 1024;
static_assert(LF_SMEM <= 232448, "one CTA's shared memory");
// Tensor Memory columns: W then P; KV; O; two slots of K' (three terms of 16 columns: 32 tokens)
constexpr uint32_t TM_W = 0, TM_KV = 128, TM_O = 256, TM_KP = 384, KP_SLOT = 48;

struct LinMaps {
    CUtensorMap q, k, v, out;
};

// A chunk: sequence n, head h, chunk c of nc; the sequence's tokens [bos, bos + len).
struct Cursor {
    int n, h, c, nc;
    int64_t bos, len;
};

__device__ __forceinline__ void seq_of(const LinParams& p, int n, int64_t& bos, int64_t& len) {
    if (p.cu_seqlens) {
        bos = p.cu_seqlens[n];
        len = p.cu_seqlens[n + 1] - bos;
    } else {
        bos = n * p.T;
        len = p.T;
    }
}

__device__ __forceinline__ void next_chunk(const LinParams& p, Cursor& u) {
    if (++u.c < u.nc) return;
    u.c = 0;
    if (++u.h < p.H) return;
    u.h = 0;
    do {
        if (++u.n >= p.nseq) return;
        seq_of(p, u.n, u.bos, u.len);
        u.nc = (int)((u.len + LF_C - 1) / LF_C);
    } while (u.nc == 0);
}

__device__ __forceinline__ int chunk_tokens(const Cursor& u) {
    const int64_t left = u.len - (int64_t)u.c * LF_C;
    return left < LF_C ? (int)left : LF_C;
}

// log2 of the decay; -inf (forget everything) as a finite value, so that its 0th power is 1.
__device__ __forceinline__ float log2_decay(const LinParams& p, int h) {
    const float d = p.log_decay[h] * LOG2E;
    return d < -1e30f ? -1e30f : d;
}

struct Share {
    int64_t total, x0, x1;   // chunks of the whole batch; this CTA's share
    Cursor at;               // where it starts
    bool bad;                // cu_seqlens do not describe the tokens
};

__device__ __forceinline__ int64_t share_start(int64_t total, int b, int ctas) {
    return total / ctas * b + total % ctas * b / ctas;
}

// The whole CTA: checks cu_seqlens, counts the chunks and finds the chunk `x0` (of the share's
// start, or with kEnd of its end) among the units in the order (n, h, c).
template <bool kEnd>
__device__ Share find_share(const LinParams& p, int64_t* scratch /* 16 */) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (p.nseq + LF_THREADS - 1) / LF_THREADS;
    const int n0 = min(tid * per, p.nseq), n1 = min(n0 + per, p.nseq);
    int64_t mine = 0;
    bool bad = false;
    for (int n = n0; n < n1; ++n) {
        int64_t bos, len;
        seq_of(p, n, bos, len);
        bad |= len < 0;
        mine += (len + LF_C - 1) / LF_C;
    }
    if (tid == 0 && p.cu_seqlens) bad |= p.cu_seqlens[0] != 0 || p.cu_seqlens[p.nseq] > p.T_total;
    int64_t sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += y;
    }
    if (lane == 31) scratch[warp] = sum;
    bad = __syncthreads_or(bad);
    int64_t before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < LF_THREADS / 32; ++w) {
        before += w < warp ? scratch[w] : 0;
        all += scratch[w];
    }
    before += sum - mine;
    Share s;
    s.bad = bad;
    s.total = bad ? 0 : all * p.H;
    s.x0 = share_start(s.total, blockIdx.x, gridDim.x);
    s.x1 = share_start(s.total, blockIdx.x + 1, gridDim.x);
    const int64_t x = kEnd ? s.x1 : s.x0;
    __syncthreads();
    Cursor* out = reinterpret_cast<Cursor*>(scratch);
    if (!bad && mine > 0 && x >= before * p.H && x < (before + mine) * p.H) {
        int64_t base = before * p.H;
        for (int n = n0; n < n1; ++n) {
            Cursor u;
            u.n = n;
            seq_of(p, n, u.bos, u.len);
            u.nc = (int)((u.len + LF_C - 1) / LF_C);
            if (x < base + (int64_t)u.nc * p.H) {
                u.h = (int)((x - base) / u.nc);
                u.c = (int)((x - base) % u.nc);
                *out = u;
                break;
            }
            base += (int64_t)u.nc * p.H;
        }
    }
    __syncthreads();
    s.at = *out;
    __syncthreads();
    return s;
}

struct Ctx {
    uint32_t base, tmem;
    unsigned char* g;
    volatile uint32_t* abort;
    uint32_t* status;
    int64_t count;   // chunks to do
    __device__ uint32_t bar(int b) const { return base + OFF_BAR + 8u * b; }
    __device__ bool wait(int b, int64_t use) const { return mx_wait(bar(b), (uint32_t)(use & 1), abort, status); }
};

// ---------------------------------------------------------------- warp 8: loads
template <bool kStateOnly>
__device__ void load_warp(const LinParams& p, const LinMaps& maps, const Ctx& x, Cursor u) {
    if ((threadIdx.x & 31) == 0) {
        int64_t i = 0;
        for (; i < x.count; ++i, next_chunk(p, u)) {
            const int s = (int)(i & 1);
            const int t0 = (int)(u.bos + (int64_t)u.c * LF_C);
            auto one = [&](int full, int empty, const CUtensorMap* m, uint32_t off) {
                if (i >= 2) {
                    const uint32_t par = (uint32_t)(((i >> 1) - 1) & 1);
                    const long long c0 = clock64();
                    while (!mbar_try_wait(x.bar(empty + s), par)) {
                        if (*x.abort) return false;
                        if (clock64() - c0 > MX_WAIT_LIMIT) {
                            atomicOr(x.status, KDA_DEVERR_TIMEOUT);
                            *x.abort = 1u;
                            return false;
                        }
                    }
                }
                const uint32_t dst = x.base + s * STAGE + off;
                mbar_arrive_expect_tx(x.bar(full + s), TILE);
                tma_load_4d(dst, m, 0, u.h, t0, 0, x.bar(full + s));
                tma_load_4d(dst + HALF, m, 64, u.h, t0, 0, x.bar(full + s));
                return true;
            };
            if (!one(FK, EK, &maps.k, TILE)) break;
            if (!kStateOnly && !one(FQ, EQ, &maps.q, 0)) break;
            if (!one(FV, EV, &maps.v, 2 * TILE)) break;
        }
        // after a wait gave up: the copies in flight land before the CTA leaves (their phases
        // complete by themselves; a phase not armed is not waited for long)
        if (*x.abort) {
            const long long c0 = clock64();
            while (clock64() - c0 < 2000000LL) __nanosleep(1000);
        }
    }
    __syncwarp();
}

// ---------------------------------------------------------------- warp 9: MMAs
template <bool kStateOnly>
__device__ void mma_warp(const LinParams& p, const Ctx& x) {
    constexpr uint32_t id_kk = make_idesc_bf16_f32(128, 128);          // both operands K-major
    constexpr uint32_t id_mn = make_idesc_bf16_f32(128, 128, true);    // B MN-major
    const uint32_t tm = x.tmem, sS = x.base + OFF_S;
    int64_t i = 0;
    for (; i < x.count; ++i) {
        const int s = (int)(i & 1);
        const int64_t use = i >> 1;
        const uint32_t sQ = x.base + s * STAGE, sK = sQ + TILE, sV = sK + TILE;
        if (!kStateOnly) {
            // W = Q K^T, over the P that the previous chunk's product has read
            if (i > 0 && !x.wait(OF, i - 1)) break;
            if (!x.wait(FK + s, use) || !x.wait(FQ + s, use)) break;
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
                tc_mma_ss_warp(tm + TM_W, make_sdesc_kmajor_sw128(sQ + (kk >> 2) * HALF + (kk & 3) * 32),
                               make_sdesc_kmajor_sw128(sK + (kk >> 2) * HALF + (kk & 3) * 32), id_kk, kk > 0);
            tc_commit_warp(x.bar(WF));
            tc_commit_warp(x.bar(EK + s));
            // O = Q S, once the state is in shared memory and the previous O has been read
            if (!x.wait(SB, i) || (i > 0 && !x.wait(OE, i - 1))) break;
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
                tc_mma_ss_warp(tm + TM_O, make_sdesc_kmajor_sw128(sQ + (kk >> 2) * HALF + (kk & 3) * 32),
                               make_sdesc_mnmajor_sw128(sS + kk * 2048, HALF, 1024), id_mn, kk > 0);
            tc_commit_warp(x.bar(QSF));
        }
        // KV = K'^T V, 32 tokens at a time as warps 4-7 hand them over
        if (!x.wait(FV + s, use)) break;
        bool ok = true;
#pragma unroll 1
        for (int b = 0; b < 4 && ok; ++b) {
            const int slot = b & 1;
            ok = x.wait(KPF + slot, 2 * i + (b >> 1));
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                for (int term = 0; term < 3; ++term)
                    tc_mma_ts_warp(tm + TM_KV, tm + TM_KP + slot * KP_SLOT + term * 16 + kk * 8,
                                   make_sdesc_mnmajor_sw128(sV + (2 * b + kk) * 2048, HALF, 1024), id_mn, b + kk + term > 0);
            tc_commit_warp(x.bar(KPE + slot));
        }
        if (!ok) break;
        tc_commit_warp(x.bar(KVF));
        if (kStateOnly) {
            tc_commit_warp(x.bar(EV + s));
            continue;
        }
        // O += P V
        if (!x.wait(PF, i) || !x.wait(OS, i)) break;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
            tc_mma_ts_warp(tm + TM_O, tm + TM_W + kk * 8, make_sdesc_mnmajor_sw128(sV + kk * 2048, HALF, 1024), id_mn, 1u);
        tc_commit_warp(x.bar(OF));
        tc_commit_warp(x.bar(EV + s));
    }
    // the MMAs in flight finish before the CTA frees Tensor Memory
    tc_commit_warp(x.bar(DRAIN));
    if (!mbar_wait_bounded(x.bar(DRAIN), 0, x.status, KDA_DEVERR_TIMEOUT, MX_WAIT_LIMIT)) *x.abort = 1u;
    __syncwarp();
}

// ---------------------------------------------------------------- warps 0-3: P, O, output
__device__ void out_warps(const LinParams& p, const LinMaps& maps, const Ctx& x, Cursor u) {
    const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) & 3, row = threadIdx.x & 127;
    const uint32_t lanes = (uint32_t)(32 * warp) << 16;
    float* pow = reinterpret_cast<float*>(x.g + OFF_POW + warp * 128);
    float l2 = 0.f, since = 0.f;
    int h = -1;
    int64_t i = 0;
    for (; i < x.count; ++i, next_chunk(p, u)) {
        const int s = (int)(i & 1);
        const int valid = chunk_tokens(u);
        if (u.h != h) {
            h = u.h;
            l2 = log2_decay(p, h);
            __syncwarp();
            pow[lane] = exp2f(l2 * (float)(31 - lane));
            since = p.scale * exp2f(l2 * (float)(row + 1));
            __syncwarp();
        }
        // P: column blocks of 32; the blocks left of this warp's rows factor into a power for the
        // row and one for the column (all exponents >= 0), the diagonal one takes a^(i-j) each
        if (!x.wait(WF, i)) break;
        tc_fence_after();
#pragma unroll 1
        for (int b = 0; b < 4; ++b) {
            uint32_t w[32], o[16];
            if (b < warp) {
                tmem_ld32(x.tmem + lanes + TM_W + 32 * b, w);
                const float f = p.scale * exp2f(l2 * (float)(row - 32 * b - 31));
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 32; j += 4) {
                    const float4 c = *reinterpret_cast<const float4*>(pow + j);
                    o[j / 2] = pack_bf16x2(mx_u2f(w[j]) * (f * c.x), mx_u2f(w[j + 1]) * (f * c.y));
                    o[j / 2 + 1] = pack_bf16x2(mx_u2f(w[j + 2]) * (f * c.z), mx_u2f(w[j + 3]) * (f * c.w));
                }
            } else if (b == warp) {
                tmem_ld32(x.tmem + lanes + TM_W + 32 * b, w);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 32; j += 2) {
                    const float a0 = j <= lane ? mx_u2f(w[j]) * (p.scale * pow[31 - (lane - j)]) : 0.f;
                    const float a1 = j + 1 <= lane ? mx_u2f(w[j + 1]) * (p.scale * pow[31 - (lane - j - 1)]) : 0.f;
                    o[j / 2] = pack_bf16x2(a0, a1);
                }
            } else {
#pragma unroll
                for (int j = 0; j < 16; ++j) o[j] = 0u;
            }
            tmem_st16(x.tmem + lanes + TM_W + 16 * b, o);
        }
        tmem_wait_st();
        tc_fence_before();
        mx_arrive_warp(x.bar(PF));
        // O = Q S, each row scaled by scale a^(i+1)
        if (!x.wait(QSF, i)) break;
        tc_fence_after();
#pragma unroll 1
        for (int b = 0; b < 4; ++b) {
            uint32_t w[32];
            tmem_ld32(x.tmem + lanes + TM_O + 32 * b, w);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 32; ++j) w[j] = __float_as_uint(mx_u2f(w[j]) * since);
            tmem_st32(x.tmem + lanes + TM_O + 32 * b, w);
        }
        tmem_wait_st();
        tc_fence_before();
        mx_arrive_warp(x.bar(OS));
        // the previous chunk's output tile has left its q buffer
        if (i > 0 && lane == 0) {
            bulk_wait_read_all();
            mbar_arrive(x.bar(EQ + (s ^ 1)));
        }
        __syncwarp();
        // the output, through this chunk's q buffer (both products have read it)
        if (!x.wait(OF, i)) break;
        tc_fence_after();
        const int64_t t0 = u.bos + (int64_t)u.c * LF_C;
        unsigned char* tile = x.g + s * STAGE;
#pragma unroll 1
        for (int b = 0; b < 4; ++b) {
            uint32_t w[32];
            tmem_ld32(x.tmem + lanes + TM_O + 32 * b, w);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint4 o = make_uint4(pack_bf16x2(mx_u2f(w[8 * j]), mx_u2f(w[8 * j + 1])), pack_bf16x2(mx_u2f(w[8 * j + 2]), mx_u2f(w[8 * j + 3])),
                                           pack_bf16x2(mx_u2f(w[8 * j + 4]), mx_u2f(w[8 * j + 5])), pack_bf16x2(mx_u2f(w[8 * j + 6]), mx_u2f(w[8 * j + 7])));
                if (valid == LF_C) *reinterpret_cast<uint4*>(tile + sw128_offset(row, 32 * b + 8 * j, 128)) = o;
                else if (row < valid) *reinterpret_cast<uint4*>(p.out.data + (t0 + row) * p.out.row + u.h * p.out.head + 32 * b + 8 * j) = o;
            }
        }
        tc_fence_before();
        mx_arrive_warp(x.bar(OE));
        if (valid == LF_C) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                const uint32_t src = x.base + s * STAGE + 32 * warp * 128;
                tma_store_3d(&maps.out, src, 0, u.h, (int)t0 + 32 * warp);
                tma_store_3d(&maps.out, src + HALF, 64, u.h, (int)t0 + 32 * warp);
                bulk_commit();
            }
            __syncwarp();
        }
    }
    if (lane == 0) bulk_wait_all();
    __syncwarp();
}

// ---------------------------------------------------------------- warps 4-7: K' and the state
// Thread k holds S[k][0 .. 127] (column v).  Global states are [V][K]: the 32 lanes of a warp
// read and write 32 neighbouring k of one v.
__device__ __forceinline__ float state_at(const void* s, int f32, size_t off) {
    return f32 ? __ldg(static_cast<const float*>(s) + off) : __bfloat162float(static_cast<const __nv_bfloat16*>(s)[off]);
}

template <bool kStateOnly>
__device__ void state_warps(const LinParams& p, const Ctx& x, Cursor u, const Share& share) {
    const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) & 3, k = threadIdx.x & 127;
    const uint32_t lanes = (uint32_t)(32 * warp) << 16;
    float* pow = reinterpret_cast<float*>(x.g + OFF_POW + (4 + warp) * 128);
    float* tail = reinterpret_cast<float*>(x.g + OFF_POW + (8 + warp) * 128);
    float S[LF_C];
    float l2 = 0.f, all = 0.f;
    bool fresh = true;   // a unit (or this share) starts
    int64_t i = 0;
    for (; i < x.count; ++i, next_chunk(p, u)) {
        const int s = (int)(i & 1);
        const int valid = chunk_tokens(u);
        const size_t unit = (size_t)u.n * p.H + u.h;
        if (fresh) {
            fresh = false;
            l2 = log2_decay(p, u.h);
            __syncwarp();
            pow[lane] = exp2f(l2 * (float)(31 - lane));
            all = exp2f(l2 * (float)LF_C);
            __syncwarp();
            if (kStateOnly || (u.c == 0 && p.init_state == nullptr)) {
#pragma unroll
                for (int v = 0; v < LF_C; ++v) S[v] = 0.f;
            } else {
                const float f = exp2f(l2 * (float)u.c * (float)LF_C);
                if (p.init_state) {
#pragma unroll
                    for (int v = 0; v < LF_C; ++v) S[v] = f * state_at(p.init_state, p.init_f32, (unit * HD + v) * HD + k);
                } else {
#pragma unroll
                    for (int v = 0; v < LF_C; ++v) S[v] = 0.f;
                }
                // the shares before this one that hold earlier chunks of the unit
                const int64_t first = share.x0 - u.c;
                for (int b = (int)blockIdx.x - 1; u.c > 0 && b >= 0; --b) {
                    const int64_t end = share_start(share.total, b + 1, gridDim.x);
                    if (end <= first) break;
                    if (share_start(share.total, b, gridDim.x) == end) continue;
                    const float g = exp2f(l2 * (float)(share.x0 - end) * (float)LF_C);
                    const float* part = static_cast<const float*>(p.workspace) + (size_t)b * HD * HD + k;
#pragma unroll
                    for (int v = 0; v < LF_C; ++v) S[v] = fmaf(g, __ldg(part + v * HD), S[v]);
                }
            }
        }
        if (!kStateOnly) {
            // the bf16 copy of the state, once the previous product with it is done
            if (i > 0 && !x.wait(QSF, i - 1)) break;
            unsigned char* tile = x.g + OFF_S;
#pragma unroll
            for (int v = 0; v < LF_C; v += 8)
                *reinterpret_cast<uint4*>(tile + sw128_offset(k, v, 128)) =
                    make_uint4(pack_bf16x2(S[v], S[v + 1]), pack_bf16x2(S[v + 2], S[v + 3]), pack_bf16x2(S[v + 4], S[v + 5]), pack_bf16x2(S[v + 6], S[v + 7]));
            fence_proxy_async_smem();
            mx_arrive_warp(x.bar(SB));
        }
        // K': 32 tokens at a time, transposed into lane k, each value as a sum of three bf16
        if (!x.wait(FK + s, i >> 1)) break;
        if (valid < LF_C) {   // rows past the end count for nothing, whatever they hold
            if (!x.wait(FV + s, i >> 1)) break;
            unsigned char* v = x.g + s * STAGE + 2 * TILE;
            for (int r = valid + warp; r < LF_C; r += 4)
                *reinterpret_cast<uint2*>(v + (lane >> 4) * HALF + r * 128 + (lane & 15) * 8) = make_uint2(0u, 0u);
            fence_proxy_async_smem();
        }
        const unsigned char* kt = x.g + s * STAGE + TILE + (k >> 6) * HALF + (k & 7) * 2;
        const int kc = (k >> 3) & 7;
        bool ok = true;
#pragma unroll 1
        for (int b = 0; b < 4; ++b) {
            const int slot = b & 1;
            const int64_t use = 2 * i + (b >> 1);
            if (use > 0) ok = x.wait(KPE + slot, use - 1);
            if (!ok) break;
            tc_fence_after();
            uint32_t raw[16];   // two tokens each
#pragma unroll
            for (int j = 0; j < 32; j += 2) {
                const unsigned char* at = kt + (32 * b + j) * 128;
                raw[j / 2] = *reinterpret_cast<const uint16_t*>(at + ((kc ^ (j & 7)) << 4)) |
                             (uint32_t)*reinterpret_cast<const uint16_t*>(at + 128 + ((kc ^ ((j + 1) & 7)) << 4)) << 16;
            }
            if (valid < LF_C) {
                // weights of a shorter chunk; tokens past the end count for nothing
                __syncwarp();
                tail[lane] = 32 * b + lane < valid ? exp2f(l2 * (float)(valid - 1 - 32 * b - lane)) : 0.f;
                __syncwarp();
#pragma unroll
                for (int j = 0; j < 32; j += 2) {
                    if (32 * b + j >= valid) raw[j / 2] = 0u;
                    else if (32 * b + j + 1 >= valid) raw[j / 2] &= 0xffffu;
                }
            }
            const float f = valid < LF_C ? 1.f : exp2f(l2 * (float)(96 - 32 * b));
            const float* weight = valid < LF_C ? tail : pow;
            uint32_t hi[16], mid[16], lo[16];
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
                const float4 w = *reinterpret_cast<const float4*>(weight + j);
                const float y[4] = {bf16_lo(raw[j / 2]) * (f * w.x), bf16_hi(raw[j / 2]) * (f * w.y),
                                    bf16_lo(raw[j / 2 + 1]) * (f * w.z), bf16_hi(raw[j / 2 + 1]) * (f * w.w)};
#pragma unroll
                for (int e = 0; e < 4; e += 2) {
                    const uint32_t a = pack_bf16x2(y[e], y[e + 1]);
                    const float r0 = y[e] - bf16_lo(a), r1 = y[e + 1] - bf16_hi(a);
                    const uint32_t m = pack_bf16x2(r0, r1);
                    hi[(j + e) / 2] = a;
                    mid[(j + e) / 2] = m;
                    lo[(j + e) / 2] = pack_bf16x2(r0 - bf16_lo(m), r1 - bf16_hi(m));
                }
            }
            const uint32_t kp = x.tmem + lanes + TM_KP + slot * KP_SLOT;
            tmem_st16(kp, hi);
            tmem_st16(kp + 16, mid);
            tmem_st16(kp + 32, lo);
            tmem_wait_st();
            tc_fence_before();
            mx_arrive_warp(x.bar(KPF + slot));
        }
        if (!ok) break;
        mx_arrive_warp(x.bar(EK + s));
        // S <- a^C S + KV
        if (!x.wait(KVF, i)) break;
        tc_fence_after();
        const float ac = valid == LF_C ? all : exp2f(l2 * (float)valid);
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            uint32_t w[32];
            tmem_ld32(x.tmem + lanes + TM_KV + 32 * b, w);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 32; ++j) S[32 * b + j] = fmaf(ac, S[32 * b + j], mx_u2f(w[j]));
        }
        tc_fence_before();
        if (kStateOnly) {
            if (i + 1 == x.count) {
                float* part = static_cast<float*>(p.workspace) + (size_t)blockIdx.x * HD * HD + k;
#pragma unroll
                for (int v = 0; v < LF_C; ++v) part[v * HD] = S[v];
            }
        } else if (u.c + 1 == u.nc) {
            fresh = true;
            if (p.final_state) {
                const size_t off = unit * HD * HD + k;
                if (p.final_f32) {
#pragma unroll
                    for (int v = 0; v < LF_C; ++v) static_cast<float*>(p.final_state)[off + (size_t)v * HD] = S[v];
                } else {
#pragma unroll
                    for (int v = 0; v < LF_C; ++v) static_cast<__nv_bfloat16*>(p.final_state)[off + (size_t)v * HD] = __float2bfloat16_rn(S[v]);
                }
            }
        }
    }
}

// Units of no tokens: the final state is the initial one.
__device__ void empty_units(const LinParams& p) {
    if (!p.final_state) return;
    const int64_t units = (int64_t)p.nseq * p.H;
    for (int64_t u0 = (int64_t)blockIdx.x * LF_THREADS; u0 < units; u0 += (int64_t)gridDim.x * LF_THREADS) {
        for (int j = 0; j < LF_THREADS && u0 + j < units; ++j) {
            const int64_t unit = u0 + j;
            int64_t bos, len;
            seq_of(p, (int)(unit / p.H), bos, len);
            if (len != 0) {   // on to the next sequence's first unit
                j += (int)min((int64_t)LF_THREADS, p.H - 1 - unit % p.H);
                continue;
            }
            for (int e = threadIdx.x; e < HD * HD; e += LF_THREADS) {
                const size_t off = (size_t)unit * HD * HD + e;
                const float v = p.init_state ? state_at(p.init_state, p.init_f32, off) : 0.f;
                if (p.final_f32) static_cast<float*>(p.final_state)[off] = v;
                else static_cast<__nv_bfloat16*>(p.final_state)[off] = __float2bfloat16_rn(v);
            }
        }
    }
}

template <bool kStateOnly>
__global__ void __launch_bounds__(LF_THREADS, 1) lin_fwd_kernel(const LinParams p, const __grid_constant__ LinMaps maps) {
    extern __shared__ unsigned char smem_raw[];
    const int tid = threadIdx.x, warp = tid >> 5;
    Ctx x;
    const uint32_t raw = smem_u32(smem_raw);
    x.base = (raw + 1023u) & ~1023u;
    x.g = smem_raw + (x.base - raw);
    x.abort = reinterpret_cast<volatile uint32_t*>(x.g + OFF_MISC + 4);
    x.status = p.status;
    Share share = find_share<kStateOnly>(p, reinterpret_cast<int64_t*>(x.g + OFF_S));
    if (!kStateOnly && blockIdx.x == 0 && tid == 0) *p.status = share.bad ? KDA_DEVERR_CU_SEQLENS : 0u;
    if (share.bad) return;
    Cursor u = share.at;
    if (kStateOnly) {
        // the share's last chunks, if its end lies inside a unit; u is the chunk after them
        if (share.x1 == share.x0 || share.x1 >= share.total || u.c == 0) return;
        const int64_t own = share.x1 - share.x0;
        x.count = own < u.c ? own : u.c;
        u.c -= (int)x.count;
    } else {
        empty_units(p);
        x.count = share.x1 - share.x0;
        if (x.count == 0) return;
    }
    if (tid == 0) {
        for (int b = 0; b < NBAR; ++b) {
            const bool warps = b == EQ || b == EQ + 1 || b == KPF || b == KPF + 1 || b == PF || b == OS || b == OE || b == SB;
            const bool both = b == EK || b == EK + 1;   // the key tile: W's MMA and the four state warps
            mbar_init(x.bar(b), warps ? 4 : both ? (kStateOnly ? 4 : 5) : 1);
        }
        mbar_fence_init();
        *x.abort = 0u;
        tma_prefetch_desc(&maps.q);
        tma_prefetch_desc(&maps.k);
        tma_prefetch_desc(&maps.v);
        tma_prefetch_desc(&maps.out);
    }
    if (warp == 0) {
        tmem_alloc(x.base + OFF_MISC, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    x.tmem = *reinterpret_cast<volatile uint32_t*>(x.g + OFF_MISC);
    // registers a thread: 168 at launch; 168 + 240 + 96 of the 3 x 168 that the block holds
    if (warp < 4) {
        if (!kStateOnly) out_warps(p, maps, x, u);
    } else if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 240;");
        state_warps<kStateOnly>(p, x, u, share);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 96;");
        if (warp == 8) load_warp<kStateOnly>(p, maps, x, u);
        else if (warp == 9) mma_warp<kStateOnly>(p, x);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(x.tmem, 512);
    }
}

}  // namespace

size_t lin_workspace_bytes(int64_t, int, int) { return (size_t)LF_MAX_CTAS * HD * HD * sizeof(float); }

cudaError_t launch_lin_fwd(const LinParams& p, cudaStream_t stream) {
    LinMaps maps;
    if (!mx_encode(&maps.q, p.q.data, p.H, p.T_total, 1, p.q.head, p.q.row, 0, 1, LF_C) ||
        !mx_encode(&maps.k, p.k.data, p.H, p.T_total, 1, p.k.head, p.k.row, 0, 1, LF_C) ||
        !mx_encode(&maps.v, p.v.data, p.H, p.T_total, 1, p.v.head, p.v.row, 0, 1, LF_C) ||
        !mx_encode_3d(&maps.out, p.out.data, p.H, p.T_total, p.out.head, p.out.row, 32))
        return cudaErrorInvalidValue;
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    const int64_t most = (p.T_total / LF_C + p.nseq) * p.H;   // chunks at most
    int ctas = sms < LF_MAX_CTAS ? sms : LF_MAX_CTAS;
    if (most < ctas) ctas = most > 0 ? (int)most : 1;
    for (auto k : {lin_fwd_kernel<true>, lin_fwd_kernel<false>}) {
        e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)LF_SMEM);
        if (e != cudaSuccess) return e;
        k<<<ctas, LF_THREADS, LF_SMEM, stream>>>(p, maps);
    }
    return cudaGetLastError();
}

}  // namespace kda
