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
// every step).  Its bf16 copy in shared memory is O's operand only, as P is in bf16 with V's type:
// against 64 bits the output is off by 0.0023 of its norm, 0.0017 of which is its own rounding.
//
// One persistent CTA per SM takes a contiguous share of all chunks of all (sequence, head)
// units, in the order (n, h, c); the shares are equal in chunks plus `extra` for each unit that
// starts there (reading and writing an fp32 state is a chunk's traffic, and changing units costs
// about another one).  A share that starts inside a unit needs the state before
// it.  Where the unit lies in two shares, the first one takes its part of that unit first of all
// and publishes the state, and the second one takes its part last of all, when the state has
// long been there: no chunk is read twice and nobody waits.  Units that lie in more than two
// shares (few heads, long prompts) would make a chain of waits; there every share first sums k v^T
// over its last chunks, if the unit goes on behind them (kSum: keys and values only, and K' made by
// two more groups), publishes that, and starts its own chunks from the decayed sums before it.  All of them
// read the unit's initial state in their own time, and the last one writes the final state: where that
// takes the initial one's place, the share that begins the unit copies it before it publishes its sum, and
// they read the copy.
//
// Warp roles: warps 0-3 turn W into P and scale O (thread = token row); warps 4-7 write the
// output out; warps 8-11 carry the state (thread = key channel); warps 12-15 and 16-19 make K',
// alternate parts of 32 tokens; warp 20 loads q, k, v by TMA through a ring of two chunks; warp
// 21 issues the products W, O and P V, warp 22 those of KV.  Each scheduler of the SM then runs
// one warp of every role, and the chunk lasts as long as the busiest role's chain of dependent
// instructions; that is why K' is spread over two groups.  Every wait is bounded.
//
// Bound by HBM: 1,024 bytes a token-head against 4 x 128 x 128 x 2 (+ 2 x the state's extra
// terms) flop; a chunk at HBM speed lasts about 5,700 SM cycles, its MMAs 3,072.  Measured: eight
// prompts of 63 to 9,088 tokens, 64 heads, fp32 states: 552 to 589 us (the latter with new inputs
// each time), 5.5 to 5.2 TB/s; prompts of 300, 700 and 1,024 tokens, 96 heads: 66 us, of which 7 pass
// between two calls (a cooperative launch and a memset), 4 until the share is found, and the shares
// end between 39 and 58; one prompt of 32,768, 32 heads: 302 to 316 us (305 with a state in place), about 95 of it for the sums, which read the keys and
// values once more (a 225 us floor for this way; a chain of waits would read nothing twice but
// leave four of five SMs waiting).
//
// Why so: 128 tokens fill an MMA's rows and make the state's update, whose cost does not depend on
// the chunk, cheap; K' from Tensor Memory in three terms costs 8 more MMAs a term but no
// rounding that a plain fp32 evaluation would not have; one group more for the output (seven in
// all) leaves too few registers each: 75 and 703 us for the first two at the time, against 78 and 575.
#include "kda_mixer.cuh"

namespace kda {
namespace {

constexpr int LF_C = 128;            // tokens a chunk
constexpr int LF_THREADS = 768;      // six warpgroups, the last with an idle warp
constexpr int LF_MAX_CTAS = 160;     // shares (and partial states) at most
constexpr uint32_t TILE = 128 * 256; // one 128 x 128 bf16 tile: two 64-channel halves of 16 KB
constexpr uint32_t HALF = TILE / 2;
constexpr uint32_t STAGE = 3 * TILE; // q, k, v
constexpr uint32_t OFF_S = 2 * STAGE;
// powers a^(31 - j), j < 32: for each of warps 0-3 followed by 32 zeros, for each of warps 12-19
// alone (a short chunk puts its own weights there)
constexpr uint32_t OFF_POW = OFF_S + TILE, OFF_KPOW = OFF_POW + 4 * 256;
constexpr uint32_t OFF_BAR = OFF_KPOW + 8 * 128;
// (the barriers; then as many for the chunks that are only summed)
enum { FQ = 0, FK = 2, FV = 4, EQ = 6, EK = 8, EV = 10, KPF = 12, KPE = 16, VR = 20, WF = 22, PF, QSF, OS, OF, OE, KVF, KVE, SB, DRAIN, DRAIN2, NBAR };
constexpr uint32_t OFF_TMEM = OFF_BAR + 2 * NBAR * 8, OFF_SEG = OFF_TMEM + 8;
constexpr uint32_t LF_SMEM = OFF_SEG + 5 * 24;   // no room to align the base: it has to be (and is checked to be) 1 KB aligned
static_assert(LF_SMEM <= 232448, "one CTA's shared memory");
// Tensor Memory columns (all are allocated, so that its address is 0): W then P; KV; O; two slots of K' (32 tokens: three terms of 16 columns)
constexpr uint32_t TM_W = 0, TM_KV = 128, TM_O = 256, TM_KP = 384, KP_SLOT = 48;

// Summing alone needs no W: its place takes two more slots, for two more groups.
__device__ __forceinline__ uint32_t kp_slot(int s) { return s < 2 ? TM_KP + s * KP_SLOT : TM_W + (s - 2) * KP_SLOT; }

struct LinMaps {
    CUtensorMap q, k, v, out;
};

// A chunk: sequence n, head h, chunk c of nc; the sequence's tokens [bos, bos + len).
struct Cursor {
    int n, h, c, nc;
    int bos, len;
};

// (all tokens are fewer than 2^31; what cu_seqlens holds beyond that is refused before it is used)
__device__ __forceinline__ void seq_of(const LinParams& p, int n, int& bos, int& len) {
    if (p.cu_seqlens) {
        bos = (int)p.cu_seqlens[n];
        len = (int)p.cu_seqlens[n + 1] - bos;
    } else {
        len = (int)p.T;
        bos = n * len;
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
        u.nc = (u.len + LF_C - 1) / LF_C;
    } while (u.nc == 0);
}

__device__ __forceinline__ int chunk_tokens(const Cursor& u) {
    const int left = u.len - u.c * LF_C;
    return left < LF_C ? left : LF_C;
}

// log2 of the decay; -inf (forget everything) as a finite value, so that its 0th power is 1.
__device__ __forceinline__ float log2_decay(const LinParams& p, int h) {
    const float d = p.log_decay[h] * LOG2E;
    return d < -1e30f ? -1e30f : d;
}

// Where, by weight, share b of `ctas` equal ones starts (recip = 2^64 / ctas, rounded up: no division).
__device__ __forceinline__ int64_t share_start(int64_t total, int b, int ctas, uint64_t recip) {
    return b >= ctas ? total : b <= 0 ? 0 : (int64_t)__umul64hi((uint64_t)total * (uint64_t)b, recip);
}

struct Share {
    int64_t total;        // weight of the whole batch
    int64_t x0, x1;       // the share's chunks, counted over the whole batch
    int64_t unit;         // where, by weight, the chunks of x0's unit start
    Cursor first, end;    // the chunk x0; the chunk x1 (if there is one)
    bool bad;             // cu_seqlens do not describe the tokens
    bool head, tail;      // x0 / x1 lies inside a unit that has no other share than the two there
    bool cut;             // x1 lies inside a unit
    bool empties;         // there are sequences of no tokens
};

// The whole CTA: checks cu_seqlens, counts the chunks and finds the share's ends.  Every CTA
// starts with this: one pass over the lengths and two block-wide exchanges.
__device__ Share find_share(const LinParams& p, uint64_t recip, int64_t* scratch /* 64 */) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (p.nseq + LF_THREADS - 1) / LF_THREADS;
    const int n0 = min(tid * per, p.nseq), n1 = min(n0 + per, p.nseq);
    // sequences that are not empty (upper 20 bits) and chunks (lower 44)
    Cursor u{};
    int64_t mine = 0;
    int what = 0;   // 1: bad, 2: a sequence of no tokens
#pragma unroll 1
    for (int n = n0; n < n1; ++n) {
        // nondecreasing from 0 to at most T_total: every entry is then in range
        if (p.cu_seqlens && (p.cu_seqlens[n + 1] < p.cu_seqlens[n] || (n == 0 && p.cu_seqlens[0] != 0) ||
                             (n + 1 == p.nseq && p.cu_seqlens[n + 1] > p.T_total)))
            what |= 1;
        seq_of(p, n, u.bos, u.len);
        u.n = n;
        u.nc = (u.len + LF_C - 1) / LF_C;
        if (u.len == 0) what |= 2;
        else mine += (1LL << 44) + u.nc;
    }
    int64_t sum = mine;
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += y;
    }
    if (lane == 31) scratch[warp] = sum;
    Share s{};
    s.bad = __syncthreads_or(what & 1);
    if (s.bad) return s;
    s.empties = __syncthreads_or(what & 2);
    int64_t before = sum - mine, all = 0;
#pragma unroll
    for (int w = 0; w < LF_THREADS / 32; ++w) {
        before += w < warp ? scratch[w] : 0;
        all += scratch[w];
    }
    // (0, 1, 2 and 3 with fp32 states: three prompts 64.7, 64.5, 66.5 and 69.5 us, eight long ones, 64 short units
    // among theirs, 657, 556, 544 and 544)
    const int extra = 1 + (p.init_state != nullptr || p.final_state != nullptr);
    auto weight = [&](int64_t v) { return ((v & ((1LL << 44) - 1)) + (v >> 44) * extra) * p.H; };
    const int64_t total = s.total = weight(all);
    const int b = blockIdx.x, ctas = gridDim.x;
    const int64_t y0 = share_start(total, b, ctas, recip), y1 = share_start(total, b + 1, ctas, recip);
    struct Place {
        Cursor at;
        int64_t x, unit;
    };
    Place* place = reinterpret_cast<Place*>(scratch + 32);   // [2]
    if (tid == 0) place[1].x = (all & ((1LL << 44) - 1)) * p.H;   // the end of the last share
    __syncthreads();
#pragma unroll 1
    for (int e = 0; e < 2; ++e) {
        int64_t at = (e ? y1 : y0) - weight(before), done = (before & ((1LL << 44) - 1)) * p.H;
        if (at < 0 || at >= weight(mine)) continue;
        if (n1 - n0 > 1)
            for (u.n = n0;; ++u.n) {
                seq_of(p, u.n, u.bos, u.len);
                u.nc = (u.len + LF_C - 1) / LF_C;
                const int64_t w = u.nc > 0 ? (int64_t)(u.nc + extra) * p.H : 0;
                if (at < w) break;
                at -= w;
                done += (int64_t)u.nc * p.H;
            }
        const int w = u.nc + extra;
        u.h = (int)((float)at / (float)w);   // (within one of the quotient, which is below 2^16)
        at -= (int64_t)u.h * w;
        if (at < 0) --u.h, at += w;
        else if (at >= w) ++u.h, at -= w;
        u.c = at > extra ? (int)at - extra : 0;
        place[e] = Place{u, done + (int64_t)u.h * u.nc + u.c, (e ? y1 : y0) - at + extra};
    }
    __syncthreads();
    s.first = place[0].at;
    s.end = place[1].at;
    s.x0 = y0 < total ? place[0].x : place[1].x;
    s.x1 = place[1].x;
    s.unit = place[0].unit;
    const int64_t end_unit = place[1].unit;
    __syncthreads();
    // (chunks of a unit, by weight: [unit, unit + nc))
    s.cut = y1 < total && s.x1 > s.x0 && s.end.c > 0;
    s.tail = s.cut && end_unit >= y0 && end_unit + s.end.nc <= share_start(total, b + 2, ctas, recip);
    s.head = s.x1 > s.x0 && s.first.c > 0 && s.unit >= share_start(total, b - 1, ctas, recip) && s.unit + s.first.nc <= y1;
    return s;
}

template <bool kSum>
struct Ctx {
    uint32_t base;         // shared-window address
    int count;             // chunks to do (a GPU's memory holds fewer than 2^31 in all)
    // in this order: nA chunks of the unit that the next share ends, then up to nAB, then the rest of
    // the unit that the share before began
    int nA, nAB;
    int kept;              // the chunk that starts a unit whose initial state the sums keep in the workspace, or -1
    const Cursor* seg;     // where the three parts start (in shared memory)
    __device__ uint32_t bar(int b) const { return base + OFF_BAR + 8u * (b + (kSum ? NBAR : 0)); }
    __device__ bool wait(int b, int use) const { return mx_wait(bar(b), (uint32_t)use & 1u); }
};

template <bool kSum>
__device__ __forceinline__ Cursor first_chunk(const Ctx<kSum>& x) { return x.seg[x.nA > 0 ? 0 : x.nAB > 0 ? 1 : 2]; }
// From chunk i of the share to chunk i + 1.
template <bool kSum>
__device__ __forceinline__ void advance(const LinParams& p, const Ctx<kSum>& x, Cursor& u, int i) {
    if (i + 1 == x.nA || i + 1 == x.nAB) u = x.seg[i + 1 < x.nAB ? 1 : 2];
    else next_chunk(p, u);
}

// Workspace: a flag for each share (right behind the status word's 256 bytes: one launch clears them all), then
// a partial or published state for each share and a kept initial state for every second one (shares that begin a
// unit of more than two shares are never neighbours).
constexpr size_t LF_STATES = LF_MAX_CTAS + LF_MAX_CTAS / 2, LF_FLAG_BYTES = LF_MAX_CTAS * sizeof(uint32_t);
static_assert(LF_FLAG_BYTES % 16 == 0, "the states are read and written in 16 bytes");
__host__ __device__ __forceinline__ uint32_t* share_flag(const LinParams& p, int b) { return static_cast<uint32_t*>(p.workspace) + b; }
__device__ __forceinline__ float* share_state(const LinParams& p, int b) {
    return reinterpret_cast<float*>(share_flag(p, LF_MAX_CTAS)) + (size_t)b * HD * HD;
}
__device__ __forceinline__ void* kept_state(const LinParams& p, int b) { return share_state(p, LF_MAX_CTAS + (b >> 1)); }
__device__ __forceinline__ bool in_place(const LinParams& p) { return p.init_state != nullptr && p.init_state == p.final_state; }

// ---------------------------------------------------------------- warp 20: loads
template <bool kSum>
__device__ bool load_warp(const LinParams& p, const LinMaps& maps, const Ctx<kSum>& x) {
    bool ok = true;
    if ((threadIdx.x & 31) == 0) {
        Cursor u = first_chunk(x);
        auto one = [&](int i, int full, int empty, const CUtensorMap* m, uint32_t off) {
            const int s = i & 1;
            if (i >= 2 && !mx_wait_lane(x.bar(empty + s), (uint32_t)((i >> 1) - 1) & 1u)) return false;
            const uint32_t dst = x.base + s * STAGE + off;
            const int t0 = u.bos + u.c * LF_C;
            mbar_arrive_expect_tx(x.bar(full + s), TILE);
            tma_load_4d(dst, m, 0, u.h, t0, 0, x.bar(full + s));
            tma_load_4d(dst + HALF, m, 64, u.h, t0, 0, x.bar(full + s));
            return true;
        };
        for (int i = 0; i < x.count && ok; advance(p, x, u, i), ++i) {
            if (!kSum && u.c == 0 && p.init_state) {   // the state warps will want it soon
                const uint32_t bytes = HD * HD * (p.init_f32 ? 4 : 2);
                const char* from = static_cast<const char*>(p.init_state) + ((size_t)u.n * p.H + u.h) * bytes;
                asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(from), "r"(bytes) : "memory");
            }
            ok = one(i, FK, EK, &maps.k, TILE);
            if (!kSum) ok = ok && one(i, FQ, EQ, &maps.q, 0);
            ok = ok && one(i, FV, EV, &maps.v, 2 * TILE);
        }
    }
    return __all_sync(0xffffffffu, ok);
}

// ---------------------------------------------------------------- warps 21 and 22: MMAs
// Descriptors: a slice of 16 along K is 32 bytes further in a K-major tile (64 of K to a half
// tile), 2 KB further in an MN-major one.
constexpr uint64_t K_STEP = 32 >> 4, K_HALF = HALF >> 4, MN_STEP = 2048 >> 4, D_STAGE = STAGE >> 4;
constexpr uint32_t ID_KK = make_idesc_bf16_f32(128, 128);          // both operands K-major
constexpr uint32_t ID_MN = make_idesc_bf16_f32(128, 128, true);    // B MN-major

// the MMAs in flight finish before the CTA frees Tensor Memory
template <bool kSum>
__device__ __forceinline__ bool drain_mma(const Ctx<kSum>& x, uint32_t lead, int bar) {
    __syncwarp();
    mx_commit(lead, x.bar(bar));
    return x.wait(bar, 0);
}

__device__ bool mma_out_warp(const Ctx<false>& x) {
    const uint32_t lead = mx_leader();
    const int count = mx_uniform(x.count);
    const uint64_t dQ = make_sdesc_kmajor_sw128(x.base), dS = make_sdesc_mnmajor_sw128(x.base + OFF_S, HALF, 1024);
    const uint64_t dV = make_sdesc_mnmajor_sw128(x.base + 2 * TILE, HALF, 1024);
    bool ok = true;
    for (int i = 0; i < count; ++i) {
        const int s = i & 1;
        const uint32_t use = (uint32_t)i >> 1, par = i & 1;
        const uint64_t q = dQ + s * D_STAGE, k = q + (TILE >> 4), v = dV + s * D_STAGE;
        // W = Q K^T, over the P that the previous chunk's product has read
        ok = mx_wait_lane(x.bar(FK + s), use & 1u) && mx_wait_lane(x.bar(FQ + s), use & 1u) && (i == 0 || mx_wait_lane(x.bar(OF), par ^ 1u));
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
            mx_mma_ss(lead, TM_W, q + (kk >> 2) * K_HALF + (kk & 3) * K_STEP, k + (kk >> 2) * K_HALF + (kk & 3) * K_STEP, ID_KK, kk > 0);
        mx_commit(lead, x.bar(WF));
        mx_commit(lead, x.bar(EK + s));
        // O = Q S, once the state is in shared memory and the previous O has been read
        ok = mx_wait_lane(x.bar(SB), par) && (i == 0 || mx_wait_lane(x.bar(OE), par ^ 1u));
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
            mx_mma_ss(lead, TM_O, q + (kk >> 2) * K_HALF + (kk & 3) * K_STEP, dS + kk * MN_STEP, ID_MN, kk > 0);
        mx_commit(lead, x.bar(QSF));
        // O += P V
        ok = mx_wait_lane(x.bar(VR + s), use & 1u) && mx_wait_lane(x.bar(PF), par) && mx_wait_lane(x.bar(OS), par);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) mx_mma_ts(lead, TM_O, TM_W + kk * 8, v + kk * MN_STEP, ID_MN, 1u);
        mx_commit(lead, x.bar(OF));
        mx_commit(lead, x.bar(EV + s));
    }
    return drain_mma(x, lead, DRAIN) && ok;
}

// KV = K'^T V, 32 tokens at a time as the key warps hand them over
template <bool kSum>
__device__ bool mma_state_warp(const Ctx<kSum>& x) {
    const uint32_t lead = mx_leader();
    const int count = mx_uniform(x.count);
    const uint64_t dV = make_sdesc_mnmajor_sw128(x.base + 2 * TILE, HALF, 1024);
    bool ok = true;
    for (int i = 0; i < count; ++i) {
        const int s = i & 1;
        ok = mx_wait_lane(x.bar(VR + s), (uint32_t)(i >> 1) & 1u) && (i == 0 || mx_wait_lane(x.bar(KVE), (uint32_t)(i - 1) & 1u));
        if (!ok) break;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const int slot = kSum ? b : b & 1;
            ok = ok && mx_wait_lane(x.bar(KPF + slot), kSum ? i & 1u : (uint32_t)(b >> 1));
            if (!ok) break;
            tc_fence_after();
            const uint64_t v = dV + s * D_STAGE + 2 * b * MN_STEP;
#pragma unroll
            for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                for (int term = 0; term < 3; ++term)
                    mx_mma_ts(lead, TM_KV, kp_slot(slot) + term * 16 + 8 * kk, v + kk * MN_STEP, ID_MN, b + kk + term > 0);
            mx_commit(lead, x.bar(KPE + slot));
        }
        if (!ok) break;
        mx_commit(lead, x.bar(KVF));
        mx_commit(lead, x.bar(EV + s));
    }
    return drain_mma(x, lead, DRAIN2) && ok;
}

// ---------------------------------------------------------------- warps 0-3: P and the scale of O
__device__ bool score_warps(const LinParams& p, const Ctx<false>& x) {
    Cursor u = first_chunk(x);
    const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) & 3, row = threadIdx.x & 127;
    const uint32_t lanes = (uint32_t)(32 * warp) << 16;
    const uint32_t pow = x.base + OFF_POW + warp * 256;
    sts_f32(pow + 128 + 4 * lane, 0.f);
    float since = 0.f, left = 0.f, hop = 0.f;
    int h = -1;
    for (int i = 0; i < x.count; advance(p, x, u, i), ++i) {
        if (u.h != h) {
            h = u.h;
            const float l2 = log2_decay(p, h);
            __syncwarp();
            sts_f32(pow + 4 * lane, exp2f(l2 * (float)(31 - lane)));
            __syncwarp();
            since = p.scale * exp2f(l2 * (float)(row + 1));
            // the row's factor for the block just left of the diagonal one, and from block to block
            left = p.scale * exp2f(l2 * (float)(lane + 1));
            hop = exp2f(l2 * 32.f);
        }
        // P, in blocks of 32 columns (its 16 registers a block go over columns of W that have been
        // read): left of the diagonal block a^(i-j) is a power for the row times one for the column, all
        // exponents >= 0; in the diagonal block it is looked up; right of it P is zero
        if (!x.wait(WF, i)) return false;
        tc_fence_after();
        uint32_t w[32], y[16];
#pragma unroll 1
        for (int b = 0; b < warp; ++b) {
            tmem_ld32(lanes + TM_W + 32 * b, w);
            const int e = warp - 1 - b;
            const float f = e == 0 ? left : e == 1 ? left * hop : left * hop * hop;
            const float2 f2 = make_float2(f, f);
            tmem_wait_ld();
            mx_loaded(w);
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
                const float4 c = lds_f32x4(pow + 4 * j);
                const float2 y0 = __fmul2_rn(make_float2(mx_u2f(w[j]), mx_u2f(w[j + 1])), __fmul2_rn(f2, make_float2(c.x, c.y)));
                const float2 y1 = __fmul2_rn(make_float2(mx_u2f(w[j + 2]), mx_u2f(w[j + 3])), __fmul2_rn(f2, make_float2(c.z, c.w)));
                y[j / 2] = pack_bf16x2(y0.x, y0.y);
                y[j / 2 + 1] = pack_bf16x2(y1.x, y1.y);
            }
            tmem_st16(lanes + TM_W + 16 * b, y);
        }
        tmem_ld32(lanes + TM_W + 32 * warp, w);
        tmem_wait_ld();
        mx_loaded(w);
#pragma unroll
        for (int j = 0; j < 32; j += 2) {   // a^(lane - j) is power 31 - lane + j of the table, zeros follow
            const float a0 = mx_u2f(w[j]) * (p.scale * lds_f32(pow + 4 * (31 + j) - 4 * lane));
            const float a1 = mx_u2f(w[j + 1]) * (p.scale * lds_f32(pow + 4 * (32 + j) - 4 * lane));
            y[j / 2] = pack_bf16x2(j <= lane ? a0 : 0.f, j < lane ? a1 : 0.f);   // whatever W holds there
        }
        tmem_st16(lanes + TM_W + 16 * warp, y);
#pragma unroll
        for (int j = 0; j < 16; ++j) y[j] = 0u;
#pragma unroll 1
        for (int b = warp + 1; b < 4; ++b) tmem_st16(lanes + TM_W + 16 * b, y);
        tmem_wait_st();
        tc_fence_before();
        mx_arrive_warp(x.bar(PF));
        // O = Q S, each row scaled by scale a^(i+1)
        if (!x.wait(QSF, i)) return false;
        tc_fence_after();
        const float2 s2 = make_float2(since, since);
#pragma unroll 1
        for (int b = 0; b < 4; ++b) {
            uint32_t w[32];
            tmem_ld32(lanes + TM_O + 32 * b, w);
            tmem_wait_ld();
            mx_loaded(w);
#pragma unroll
            for (int j = 0; j < 32; j += 2) {
                const float2 y = __fmul2_rn(make_float2(mx_u2f(w[j]), mx_u2f(w[j + 1])), s2);
                w[j] = __float_as_uint(y.x);
                w[j + 1] = __float_as_uint(y.y);
            }
            tmem_st32(lanes + TM_O + 32 * b, w);
        }
        tmem_wait_st();
        tc_fence_before();
        mx_arrive_warp(x.bar(OS));
    }
    return true;
}

// ---------------------------------------------------------------- warps 4-7: the output
__device__ bool out_warps(const LinParams& p, const LinMaps& maps, const Ctx<false>& x) {
    Cursor u = first_chunk(x);
    const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) & 3, row = threadIdx.x & 127;
    const uint32_t lanes = (uint32_t)(32 * warp) << 16;
    for (int i = 0; i < x.count; advance(p, x, u, i), ++i) {
        const int s = i & 1;
        const int valid = chunk_tokens(u);
        if (!x.wait(OF, i)) return false;
        tc_fence_after();
        // through this chunk's q buffer (both products have read it); a short chunk's rows go
        // straight to memory
        const int64_t t0 = u.bos + (int64_t)u.c * LF_C;
        const bool full = valid == LF_C;
        const uint32_t tile = x.base + s * STAGE + row * 128;
        __nv_bfloat16* direct = p.out.data + (t0 + row) * p.out.row + u.h * p.out.head;
        const bool mine = row < valid;
#pragma unroll 1
        for (int b = 0; b < 4; ++b) {
            uint32_t w[32];
            tmem_ld32(lanes + TM_O + 32 * b, w);
            tmem_wait_ld();
            mx_loaded(w);
            uint32_t o[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) o[j] = pack_bf16x2(mx_u2f(w[2 * j]), mx_u2f(w[2 * j + 1]));
            if (full) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    sts_u128(tile + (b >> 1) * HALF + (((4 * (b & 1) + j) ^ (row & 7)) << 4), o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
            } else if (mine) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    *reinterpret_cast<uint4*>(direct + 32 * b + 8 * j) = make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
            }
        }
        tc_fence_before();
        mx_arrive_warp(x.bar(OE));
        if (full) {
            fence_proxy_async_smem();
            __syncwarp();
        }
        if (lane == 0) {
            if (full) {
                const uint32_t src = x.base + s * STAGE + 32 * warp * 128;
                tma_store_3d(&maps.out, src, 0, u.h, (int)t0 + 32 * warp);
                tma_store_3d(&maps.out, src + HALF, 64, u.h, (int)t0 + 32 * warp);
                bulk_commit();
                bulk_wait_read_all();
            }
            mbar_arrive(x.bar(EQ + s));
        }
        __syncwarp();
    }
    if (lane == 0) bulk_wait_all();
    __syncwarp();
    return true;
}

// ---------------------------------------------------------------- warps 8-11: the state
// Thread k holds S[k][0 .. 127] (column v).  Global states are [V][K]: the 32 lanes of a warp
// read and write 32 neighbouring k of one v.  (Not by way of the read-only cache: a state that is updated in
// place is written by the same kernel, after it has been read.)
template <class T>
__device__ __forceinline__ void load_state(const T* s, float2 (&S)[LF_C / 2]) {
#pragma unroll
    for (int v = 0; v < LF_C / 2; ++v) S[v] = make_float2((float)__ldcg(s + (2 * v) * HD), (float)__ldcg(s + (2 * v + 1) * HD));
}

template <bool kSum>
__device__ bool state_warps(const LinParams& p, const Ctx<kSum>& x, const Share& share, uint64_t recip) {
    Cursor u = first_chunk(x);
    const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) & 3, k = threadIdx.x & 127;
    const uint32_t lanes = (uint32_t)(32 * warp) << 16;
    float2 S[LF_C / 2];
    float l2 = 0.f, all = 0.f;
    bool fresh = true;      // a unit or a part of one starts
    bool publish = false;   // this share's part of a unit is written but not yet announced
    auto announce = [&]() {
#ifdef KDA_WAIT_TEST
        if ((int)blockIdx.x == p.test_skip) return;
#endif
        __threadfence();
        __syncwarp();
        if (lane == 0) asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(share_flag(p, blockIdx.x)) : "memory");
        publish = false;
    };
    auto published = [&](int b) {   // by all four warps of share b
        const uint32_t* flag = share_flag(p, b);
        uint32_t seen = 0, polls = 0;
        while (seen != 4 && ++polls < MX_MEMORY_POLLS) asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(seen) : "l"(flag) : "memory");
        return (bool)__all_sync(0xffffffffu, seen == 4);
    };
    for (int i = 0; i < x.count; advance(p, x, u, i), ++i) {
        const int valid = chunk_tokens(u);
        const size_t unit = (size_t)u.n * p.H + u.h;
        if (fresh) {
            fresh = false;
            l2 = log2_decay(p, u.h);
            all = exp2f(l2 * (float)LF_C);
            if (!kSum && u.c > 0 && i >= x.nAB) {
                // the share before published this unit's state
                if (!published(blockIdx.x - 1)) return false;
                const float* s = share_state(p, blockIdx.x - 1) + k;
#pragma unroll
                for (int v = 0; v < LF_C / 2; ++v) S[v] = make_float2(__ldcg(s + (2 * v) * HD), __ldcg(s + (2 * v + 1) * HD));
            } else {
                size_t off = unit * HD * HD + k;
                const void* init = p.init_state;
                if (kSum && i == x.kept) {
                    const size_t bytes = HD * HD * (p.init_f32 ? 4 : 2);
                    const uint4* from = reinterpret_cast<const uint4*>(static_cast<const char*>(init) + unit * bytes) + k;
                    uint4* to = static_cast<uint4*>(kept_state(p, blockIdx.x)) + k;
#pragma unroll 1
                    for (int n = 0; n < (int)(bytes / 16); n += 16 * 128) {
                        uint4 r[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) r[e] = __ldcg(from + n + 128 * e);
#pragma unroll
                        for (int e = 0; e < 16; ++e) to[n + 128 * e] = r[e];
                    }
                } else if (!kSum && i == x.kept) {
                    init = kept_state(p, blockIdx.x);
                    off = k;
                } else if (!kSum && u.c > 0 && in_place(p)) {   // the share that begins the unit has a copy
                    int b = (int)blockIdx.x - 1;
                    while (share_start(share.total, b, gridDim.x, recip) > share.unit) --b;
                    if (!published(b)) return false;
                    init = kept_state(p, b);
                    off = k;
                }
                if (kSum || init == nullptr) {
#pragma unroll
                    for (int v = 0; v < LF_C / 2; ++v) S[v] = make_float2(0.f, 0.f);
                } else if (p.init_f32) {
                    load_state(static_cast<const float*>(init) + off, S);
                } else {
                    load_state(static_cast<const __nv_bfloat16*>(init) + off, S);
                }
                if (!kSum && u.c > 0) {
                    // decayed to here, plus what the shares before this one summed over the unit's chunks
                    const float f = exp2f(l2 * (float)u.c * (float)LF_C);
#pragma unroll
                    for (int v = 0; v < LF_C / 2; ++v) S[v].x *= f, S[v].y *= f;
#pragma unroll 1
                    for (int b = (int)blockIdx.x - 1; b >= 0; --b) {
                        const int64_t end = share_start(share.total, b + 1, gridDim.x, recip) - share.unit;   // chunks up to there
                        if (end <= 0) break;
                        if (share_start(share.total, b, gridDim.x, recip) - share.unit == end) continue;
                        if (!published(b)) return false;
                        const float g = exp2f(l2 * (float)(u.c - end) * (float)LF_C);
                        const float* part = share_state(p, b) + k;
#pragma unroll
                        for (int v = 0; v < LF_C / 2; ++v) {
                            S[v].x = fmaf(g, __ldcg(part + (2 * v) * HD), S[v].x);
                            S[v].y = fmaf(g, __ldcg(part + (2 * v + 1) * HD), S[v].y);
                        }
                    }
                }
            }
        }
        if (!kSum) {
            // the bf16 copy of the state, once the previous product with it is done
            if (i > 0 && !x.wait(QSF, i - 1)) return false;
            const uint32_t tile = x.base + OFF_S + k * 128;
#pragma unroll
            for (int c = 0; c < 16; ++c)
                sts_u128(tile + (c >> 3) * HALF + (((c & 7) ^ (k & 7)) << 4), pack_bf16x2(S[4 * c].x, S[4 * c].y),
                         pack_bf16x2(S[4 * c + 1].x, S[4 * c + 1].y), pack_bf16x2(S[4 * c + 2].x, S[4 * c + 2].y),
                         pack_bf16x2(S[4 * c + 3].x, S[4 * c + 3].y));
            fence_proxy_async_smem();
            mx_arrive_warp(x.bar(SB));
        }
        // S <- a^C S + KV
        if (!x.wait(KVF, i)) return false;
        tc_fence_after();
        const float ac = valid == LF_C ? all : exp2f(l2 * (float)valid);
        const float2 ac2 = make_float2(ac, ac);
#pragma unroll
        for (int b = 0; b < 8; ++b) {
            uint32_t w[16];
            tmem_ld16(lanes + TM_KV + 16 * b, w);
            tmem_wait_ld();
            mx_loaded(w);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                S[8 * b + j] = __ffma2_rn(ac2, S[8 * b + j], make_float2(mx_u2f(w[2 * j]), mx_u2f(w[2 * j + 1])));
        }
        tc_fence_before();
        mx_arrive_warp(x.bar(KVE));
        if (!kSum && publish) announce();   // a chunk later: its stores have long been done
        if (kSum ? i + 1 == x.count : i + 1 == x.nA) {
            // this share's part of a unit that the next share goes on with
            float* part = share_state(p, blockIdx.x) + k;
#pragma unroll
            for (int v = 0; v < LF_C / 2; ++v) {
                part[(2 * v) * HD] = S[v].x;
                part[(2 * v + 1) * HD] = S[v].y;
            }
            publish = true;
            fresh = true;
        } else if (!kSum && i + 1 == x.nAB && u.c + 1 < u.nc) {
            fresh = true;   // (the shares behind go on from the sums; here the last part follows)
        } else if (!kSum && u.c + 1 == u.nc) {
            fresh = true;
            if (p.final_state) {
                const size_t off = unit * HD * HD + k;
                if (p.final_f32) {
                    float* f = static_cast<float*>(p.final_state) + off;
#pragma unroll
                    for (int v = 0; v < LF_C / 2; ++v) {
                        f[(2 * v) * HD] = S[v].x;
                        f[(2 * v + 1) * HD] = S[v].y;
                    }
                } else {
                    __nv_bfloat16* f = static_cast<__nv_bfloat16*>(p.final_state) + off;
#pragma unroll
                    for (int v = 0; v < LF_C / 2; ++v) {
                        f[(2 * v) * HD] = __float2bfloat16_rn(S[v].x);
                        f[(2 * v + 1) * HD] = __float2bfloat16_rn(S[v].y);
                    }
                }
            }
        }
    }
    if (publish) announce();
    return true;
}

// ---------------------------------------------------------------- warps 12-19: K'
// Thread k reads column k of the key tile, weighs it by a^(C-1-j) and leaves each value as a
// sum of three bf16 in lane k of Tensor Memory, 32 tokens at a time; group g takes the parts
// g and g + 2 of each chunk and owns slot g.  (While chunks are only summed, the warps of the
// scores and of the output are groups 2 and 3, and each group takes one part.)
__device__ __forceinline__ float2 unpack2(uint32_t w) { return make_float2(bf16_lo(w), bf16_hi(w)); }

template <bool kSum>
__device__ bool key_warps(const LinParams& p, const Ctx<kSum>& x, int g) {
    Cursor u = first_chunk(x);
    const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) & 3, k = threadIdx.x & 127;
    const uint32_t kp = ((uint32_t)(32 * warp) << 16) + kp_slot(g);
    const uint32_t pow = x.base + (g < 2 ? OFF_KPOW : OFF_POW) + (4 * (g & 1) + warp) * 128;
    const int kc = (k >> 3) & 7;
    const float2 minus = make_float2(-1.f, -1.f);
    float l2 = 0.f, hop = 0.f;
    int h = -1;
    for (int i = 0; i < x.count; advance(p, x, u, i), ++i) {
        const int s = i & 1;
        const int valid = chunk_tokens(u);
        const bool full = valid == LF_C;
        if (u.h != h || !full) {
            h = u.h;
            l2 = log2_decay(p, h);
            __syncwarp();
            sts_f32(pow + 4 * lane, exp2f(l2 * (float)(31 - lane)));   // (a short chunk puts its own weights there)
            __syncwarp();
            hop = exp2f(l2 * 32.f);
            if (!full) h = -1;
        }
        if (!x.wait(FK + s, i >> 1)) return false;
        if (g == 0) {
            // v is ready once it has landed and, in a short chunk, the values past its end are
            // zeros: they count for nothing, whatever they hold.  (Every chunk waits here, so that
            // this barrier never gets ahead of the value tile's use.)
            if (!x.wait(FV + s, i >> 1)) return false;
            if (!full) {
                const uint32_t v = x.base + s * STAGE + 2 * TILE;
                for (int r = valid + warp; r < LF_C; r += 4) sts_u64(v + (lane >> 4) * HALF + r * 128 + (lane & 15) * 8, 0u, 0u);
                fence_proxy_async_smem();
            }
            mx_arrive_warp(x.bar(VR + s));
        }
        bool ok = true;
#pragma unroll 1
        for (int b = g; b < 4; b += kSum ? 4 : 2) {
            const int use = kSum ? i : 2 * i + (b >> 1);
            uint32_t kt = x.base + s * STAGE + TILE + (k >> 6) * HALF + (k & 7) * 2 + 32 * b * 128;
            float f = b == 3 ? 1.f : b == 2 ? hop : b == 1 ? hop * hop : hop * hop * hop;   // a^(96 - 32 b)
            if (!full) {
                f = 1.f;
                const int t = 32 * b + lane;
                __syncwarp();
                sts_f32(pow + 4 * lane, t < valid ? exp2f(l2 * (float)(valid - 1 - t)) : 0.f);
                __syncwarp();
            }
            const float2 f2 = make_float2(f, f);
            if (use > 0) ok = x.wait(KPE + g, use - 1);
            if (!ok) return false;
            tc_fence_after();
#pragma unroll 1
            for (int q = 0; q < 2; ++q, kt += 16 * 128) {
                uint32_t raw[16];   // bf16 bits in the upper half
#pragma unroll
                for (int j = 0; j < 16; ++j) raw[j] = lds_u16(kt + j * 128 + ((kc ^ (j & 7)) << 4)) << 16;
                if (!full) {   // keys past the end: zeros, whatever they hold
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        if (32 * b + 16 * q + j >= valid) raw[j] = 0u;
                }
                uint32_t hi[8], mid[8], lo[8];
#pragma unroll
                for (int j = 0; j < 16; j += 4) {
                    const float4 w4 = lds_f32x4(pow + 4 * (16 * q + j));
#pragma unroll
                    for (int d = 0; d < 4; d += 2) {
                        const float2 w = __fmul2_rn(f2, d ? make_float2(w4.z, w4.w) : make_float2(w4.x, w4.y));
                        const float2 y = __fmul2_rn(make_float2(mx_u2f(raw[j + d]), mx_u2f(raw[j + d + 1])), w);
                        const uint32_t a = pack_bf16x2(y.x, y.y);
                        const float2 r = __ffma2_rn(unpack2(a), minus, y);
                        const uint32_t m = pack_bf16x2(r.x, r.y);
                        const float2 t = __ffma2_rn(unpack2(m), minus, r);
                        hi[(j + d) / 2] = a;
                        mid[(j + d) / 2] = m;
                        lo[(j + d) / 2] = pack_bf16x2(t.x, t.y);
                    }
                }
                tmem_st8(kp + 8 * q, hi);
                tmem_st8(kp + 16 + 8 * q, mid);
                tmem_st8(kp + 32 + 8 * q, lo);
            }
            tmem_wait_st();
            tc_fence_before();
            mx_arrive_warp(x.bar(KPF + g));
        }
        if (!ok) return false;
        mx_arrive_warp(x.bar(EK + s));
    }
    return true;
}

// Units of no tokens: the final state is the initial one.
__device__ void empty_units(const LinParams& p) {
    if (!p.final_state) return;
    for (int n = blockIdx.x; n < p.nseq; n += gridDim.x) {
        int bos, len;
        seq_of(p, n, bos, len);
        if (len != 0) continue;
        for (size_t e = threadIdx.x; e < (size_t)p.H * HD * HD; e += LF_THREADS) {
            const size_t off = (size_t)n * p.H * HD * HD + e;
            const float v = !p.init_state ? 0.f : p.init_f32 ? static_cast<const float*>(p.init_state)[off]
                                                             : __bfloat162float(static_cast<const __nv_bfloat16*>(p.init_state)[off]);
            if (p.final_f32) static_cast<float*>(p.final_state)[off] = v;
            else static_cast<__nv_bfloat16*>(p.final_state)[off] = __float2bfloat16_rn(v);
        }
    }
}

template <bool kSum>
__device__ __forceinline__ void init_barriers(const Ctx<kSum>& x, int lane) {
    for (int b = lane; b < NBAR; b += 32) {
        const bool warps = b == EQ || b == EQ + 1 || (b >= KPF && b < KPF + 4) || b == VR || b == VR + 1 || b == PF || b == OS || b == OE || b == SB || b == KVE;
        const bool both = b == EK || b == EK + 1;   // the key tile: W's MMA and the key warps
        const bool twice = b == EV || b == EV + 1;  // the value tile: KV's and P V's MMAs
        mbar_init(x.bar(b), warps ? 4 : both ? (kSum ? 16 : 9) : twice ? (kSum ? 1 : 2) : 1);
    }
}

__global__ void __launch_bounds__(LF_THREADS, 1) lin_fwd_kernel(const LinParams p, const __grid_constant__ LinMaps maps, uint64_t recip) {
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    const int tid = threadIdx.x, warp = mx_uniform(tid >> 5);
    Ctx<false> x;   // the share's chunks
    Ctx<true> y;    // those that are summed before
    x.base = y.base = smem_u32(smem_raw);
    if (warp == 20) {
        init_barriers(x, tid & 31);
        init_barriers(y, tid & 31);
        mbar_fence_init();
        if ((tid & 31) == 0) {
            tma_prefetch_desc(&maps.q);
            tma_prefetch_desc(&maps.k);
            tma_prefetch_desc(&maps.v);
            tma_prefetch_desc(&maps.out);
        }
        __syncwarp();
        tmem_alloc(x.base + OFF_TMEM, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    const Share share = find_share(p, recip, reinterpret_cast<int64_t*>(smem_raw + OFF_S));
    if (share.empties && !share.bad) empty_units(p);
    Cursor* seg = reinterpret_cast<Cursor*>(smem_raw + OFF_SEG);
    x.seg = seg;
    y.seg = seg + 2;   // (its one part is number 1; number 2 is only read)
    x.count = (int)(share.x1 - share.x0);
    x.nA = share.tail ? share.end.c : 0;
    x.nAB = x.count - (share.head ? share.first.nc - share.first.c : 0);
    // the share's last chunks, of a unit in more than two shares
    y.nA = 0;
    y.nAB = y.count = share.cut && !share.tail ? min(x.count, share.end.c) : 0;
    // a summed unit that begins here and whose state is updated in place
    const bool keep = in_place(p) && y.count > 0 && y.count == share.end.c;
    x.kept = keep ? x.nAB - y.count : -1;
    y.kept = keep ? 0 : -1;
    if (tid == 0) {
        seg[0] = share.end, seg[0].c = 0;
        seg[1] = seg[2] = share.first;
        if (share.head) {
            seg[1].c = seg[1].nc - 1;
            if (x.nAB > x.nA) next_chunk(p, seg[1]);
        }
        seg[3] = share.end, seg[3].c -= y.count;
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = lds_u32(x.base + OFF_TMEM);
    bool sound = tmem == 0 && x.base % 1024 == 0;   // (the tiles' swizzle counts from 1 KB boundaries)
#ifdef KDA_WAIT_TEST
    sound = sound && p.test_skip != -2 - (int)blockIdx.x;
#endif
    if (tid == 0) {
        if (share.bad) atomicOr(p.status, KDA_DEVERR_CU_SEQLENS);
        if (!sound) atomicOr(p.status, KDA_DEVERR_INTERNAL);
    }
    if (!sound) x.count = y.count = 0;   // (bad lengths have no chunks)
    bool ok = true;
    // registers a thread: 80 at launch; of the 6 x 80 that the block holds 72 + 72 + 144 + 72 + 72 + 48
    // while it only sums, then 64 + 56 + 168 + 72 + 72 + 48.  (The last group keeps its 48: with 40 first and
    // an increase after, the compiler gave its loops fewer, and eight prompts of 1k to 9k took 579 us, not 547.)
    if (y.count > 0) {
        if (warp < 8) {
            asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
            ok = key_warps<true>(p, y, 2 + (warp >> 2));
        } else if (warp < 12) {
            asm volatile("setmaxnreg.inc.sync.aligned.u32 144;");
            ok = state_warps<true>(p, y, share, recip);
        } else if (warp < 20) {
            asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
            ok = key_warps<true>(p, y, (warp - 12) >> 2);
        } else {
            asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
            if (warp == 20) ok = load_warp<true>(p, maps, y);
            else if (warp == 22) ok = mma_state_warp<true>(y);
        }
        tc_fence_before();
        ok = __syncthreads_and(ok);
        tc_fence_after();
        if (!ok) x.count = 0;
    }
    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        ok = score_warps(p, x) && ok;
    } else if (warp < 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        ok = out_warps(p, maps, x) && ok;
    } else if (warp < 12) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 168;");
        ok = state_warps<false>(p, x, share, recip) && ok;
    } else if (warp < 20) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        ok = key_warps<false>(p, x, (warp - 12) >> 2) && ok;
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
        if (warp == 20) ok = load_warp<false>(p, maps, x) && ok;
        else if (warp == 21) ok = mma_out_warp(x) && ok;
        else if (warp == 22) ok = mma_state_warp<false>(x) && ok;
    }
    if (!ok) {
        atomicOr(p.status, KDA_DEVERR_TIMEOUT);
        mx_wind_down();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 20) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

}  // namespace

size_t lin_workspace_bytes(int64_t, int, int) { return LF_FLAG_BYTES + LF_STATES * HD * HD * sizeof(float); }

cudaError_t launch_lin_fwd(const LinParams& p, cudaStream_t stream) {
    LinMaps maps;
    if (!mx_encode(&maps.q, p.q.data, p.H, p.T_total, 1, p.q.head, p.q.row, 0, 1, LF_C) ||
        !mx_encode(&maps.k, p.k.data, p.H, p.T_total, 1, p.k.head, p.k.row, 0, 1, LF_C) ||
        !mx_encode(&maps.v, p.v.data, p.H, p.T_total, 1, p.v.head, p.v.row, 0, 1, LF_C) ||
        !mx_encode_3d(&maps.out, p.out.data, p.H, p.T_total, p.out.head, p.out.row, 1, 32))
        return cudaErrorInvalidValue;
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    const int64_t most = (p.T_total / LF_C + p.nseq) * p.H;   // chunks at most
    int ctas = sms < LF_MAX_CTAS ? sms : LF_MAX_CTAS;
    if (most < ctas) ctas = most > 0 ? (int)most : 1;
    const uint64_t recip = ctas > 1 ? ~0ull / (uint64_t)ctas + 1 : 0;
    e = cudaFuncSetAttribute(lin_fwd_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)LF_SMEM);
    // the status word and the flags: before the kernel, so that no share's report can be overwritten
    char* cleared = reinterpret_cast<char*>(p.status);
    if (e == cudaSuccess) e = cudaMemsetAsync(cleared, 0, (size_t)(reinterpret_cast<char*>(share_flag(p, ctas)) - cleared), stream);
    if (e != cudaSuccess) return e;
    // cooperative: a share may wait for what the shares before it publish, so all of them are resident
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(LF_THREADS);
    cfg.dynamicSmemBytes = LF_SMEM;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, lin_fwd_kernel, p, maps, recip);
}

}  // namespace kda
