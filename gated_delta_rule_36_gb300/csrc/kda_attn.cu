// Causal softmax attention with grouped heads over packed prompts and caches, on the
// 5th-generation tensor cores: one pass over the keys with the running maximum and sum.
//
// A query tile is 128 rows of (token, head) pairs that share a key/value head: floor(128 / G)
// tokens with all G heads of the group.  A CTA works on two neighbouring tiles at a time and on
// blocks of 128 keys:
//   S_t = Q_t K^T   (128 x 128 x 128 each)     P_t = exp2(c S_t - c m) in bf16, over S_t in Tensor Memory
//   O_t += P_t V                               l_t += row sums of P_t in fp32
// The maximum m that the exponents refer to moves only when a row's maximum has grown by more
// than 2^8 (then O and l are rescaled): P stays below 2^8 and the sums in fp32's range, and most
// blocks skip the rescaling.  P is rounded to bf16, the type of V in the same MMA; l sums the
// unrounded weights in fp32.  The roundings are independent: against 64 bits the output is off by 0.0020
// of its norm, 0.0016 of which is its own rounding to bf16.
//
// All (sequence, key head, tile pair, key block) steps are one line that is cut into equal
// shares, one for each SM: long prompts, ragged batches and single tokens over a long cache
// all come out even.  What a pair costs by itself (its queries' way in, its results' way out, a
// softmax that waits for its first scores) counts as PIECE steps in front of it.  A pair that lies in more than one share leaves unnormalised partial rows in
// the workspace, and a second, small kernel joins them in the order of the keys.
//
// A pair of at most one tile's rows (single tokens, short prompts) alternates its one tile between
// the two places for scores, so that the next block's scores are there when this one's are done.
// (Those blocks have barriers of their own, SX and PX: a warp that counts a barrier's phases has to
// wait for every one of them.)
//
// Warp roles: warps 0-3 and 4-7 are the softmax of the two tiles (thread = row) and write the
// results; warp 8 loads q, k and v by TMA (a ring of four 32 KB tiles); warp 9 issues the MMAs,
// alternating between the tiles so that one is multiplied while the other is exponentiated.
//
// Bound by the tensor cores for prompts (4 x 128 x 128 x 128 flop, 1,024 SM cycles, a tile and
// key block), by HBM for single tokens.  Measured: one prompt of 8,192 tokens, 64 heads on 8: 680 to
// 735 us (the latter with new inputs each time, 1.50 PFLOP/s; a pair's step lasts about 2,800 cycles for its 2,048 of MMAs: the
// softmax of one tile, a chain of 1,250 cycles and more, does not fit under the other's products, but
// 400 cycles less of it gained 1 %: the plain product sustains 1.71 PFLOP/s on this card);
// 32 single tokens over caches of 67 to 8,189, 32 heads on 8: 99 us (5.4 TB/s: about 7 us until
// the first block has arrived and 8 us for the join, HBM speed between); one token over 32,767:
// 40 us; prompts of 300, 700 and 1,024 tokens: 30 us.
//
// Why so: two tiles a CTA share every key block, which halves the traffic from L2 and lets one
// tile's products hide the other's exponentials; a second warp for the MMAs fell into step with
// the first (984 against 890 us at the time).  Joining inside this kernel (the last of a pair's
// shares) was slower than the second launch: 59 against 46 us for one token, since the code
// that writes and joins is cold.  The maximum of half the scores while the other half loads:
// 704 against 696 us.  Two threads a row, each with half of the keys: 784 against 677 us; an
// exponential with its scaling, sum and packing takes 7.3 cycles from one warp of a scheduler and 5.5 from
// two, so that halves gain less than exchanging their maxima costs.
//
// Split keys (kSplit, launch_attn_split): all operands are in fp16 and scaled by powers of two, the values and keys for each block,
// the queries for each row.  A block's scores take the powers in their scale, so m counts in steps of base 2.  What the keys' 11 bits
// do not hold comes as 16 more channels, one MMA on top of eight.  The weights take their values' powers with them, and what
// a row of outputs refers to follows the largest product of a weight and its values' power, not the largest power: fp16 ends
// at 2^-24, and a large value without weight (or one that the mask hides) must not push the others' weights below that.  A block whose
// keys' powers lie further apart than 2^SPLIT_SPREAD has them key by key, and its sums of weights are made by themselves
// (prompts of 1,024, 517 and 33 behind 16,384, 8,484 and 15,967 over one set of inputs: 546 us; such keys in one block of four 667, in all 1,090).
#include <cuda_fp16.h>
#include <string.h>

#include "kda_mixer.cuh"

namespace kda {
namespace {

constexpr int AT_MAX_CTAS = 160;
constexpr int KB = 128;                       // keys a block
constexpr int AT_THREADS = 384;
constexpr uint32_t TILE = 128 * 256, HALF = TILE / 2;
// A pair's own weight, in steps.  With 0, 1, 2 and 3: long prompt 803, 733, 705 and 710 us, 32 single
// tokens 128, 105, 105 and 106 us.
constexpr int PIECE = 2;
constexpr uint32_t OFF_RING = 2 * TILE;       // behind the two query tiles
constexpr int RING = 4;                        // tiles: k and v of two blocks
enum { FULL = 0, EMPTY = RING, QF = 2 * RING, QE, SF, PF = SF + 2, OF = PF + 4, SX = OF + 2, PX, PV = PX + 2, VZ, DRAIN, NBAR };
// Split keys: the rest of the queries' and keys' channels (16 more, without swizzle) has tiles of its own, which leaves no room
// for staged results.
constexpr uint32_t REST = 128 * 2 * SPLIT_REST;
template <bool kSplit>
struct Layout {
    static constexpr uint32_t OFF_STAGE = OFF_RING + RING * TILE;           // 4 KB for each softmax warp: 32 rows of 128 bytes
    static constexpr uint32_t OFF_K_REST = OFF_RING + RING * TILE;          // one for each tile of the ring
    static constexpr uint32_t OFF_Q_REST = OFF_K_REST + RING * REST;
    // The search for the shares works here: its ordinary stores must not meet a tile's bulk loads, which
    // nothing but a proxy fence would order behind them.
    static constexpr uint32_t OFF_SCRATCH = kSplit ? OFF_Q_REST + 2 * REST : OFF_STAGE;
    static constexpr uint32_t OFF_BAR = kSplit ? OFF_SCRATCH + 512 : OFF_STAGE + 8 * 4096;
    static constexpr uint32_t OFF_TMEM = OFF_BAR + NBAR * 8;
    static constexpr uint32_t SMEM = OFF_TMEM + 8;
    static_assert(OFF_SCRATCH >= (kSplit ? OFF_Q_REST + 2 * REST : OFF_RING + RING * TILE) && OFF_SCRATCH + 48 * 8 <= OFF_BAR, "outside what bulk loads fill");
    static_assert(SMEM <= 232448, "one CTA's shared memory");
};
// Tensor Memory (all 512 columns, so that its address is 0): two tiles of 128 columns each; P over
// the first 64 of S
constexpr uint32_t TM_S = 0, TM_O = 256;

struct AttnMaps {
    CUtensorMap q, k, v;
    CUtensorMap q_rest; // split keys: boxes of eight channels
    CUtensorMap out;   // boxes of a warp's 32 rows (used when G divides 32)
};

// What a share leaves for the join: the pair that it starts in and how far into it, and its status bits.
struct Cut {
    int j, nb;          // starts at block j of nb (j = 0: between two pairs; nb = 0: an empty share)
    int q0, lq, kh, pair;
    uint32_t status;
    int pad;
};
// Partial results: two for each share, of 256 rows each.
struct Partials {
    Cut* cut;     // [shares]
    float2* ml;   // [2 * shares][256]: reference exponent (base 2) and sum
    float4* o;    // [2 * shares][32][256]: four channels of every row, not normalised (a warp of rows writes 512 bytes together)
};
constexpr size_t CUT_BYTES = AT_MAX_CTAS * sizeof(Cut), ML_BYTES = (size_t)2 * AT_MAX_CTAS * 256 * sizeof(float2);
__device__ __forceinline__ Partials partials(void* ws) {
    char* at = static_cast<char*>(ws);
    return Partials{reinterpret_cast<Cut*>(at), reinterpret_cast<float2*>(at + CUT_BYTES), reinterpret_cast<float4*>(at + CUT_BYTES + ML_BYTES)};
}

// How a sequence's steps are laid out: tiles of tq tokens in pairs; pair j sees blocks(j) key blocks.
struct Seq {
    int q0, lq, k0, lk;   // first query row and queries, first key row and keys
};

__device__ __forceinline__ Seq seq_of(const AttnParams& p, int n) {
    Seq s;
    if (p.cu_q) {
        s.q0 = (int)p.cu_q[n];
        s.lq = (int)p.cu_q[n + 1] - s.q0;
    } else {
        s.lq = (int)p.uniform_q;
        s.q0 = n * s.lq;
    }
    if (p.cache) {
        s.k0 = 0;
        s.lk = (int)p.seqlens_k[n];
    } else if (p.cu_k) {
        s.k0 = (int)p.cu_k[n];
        s.lk = (int)p.cu_k[n + 1] - s.k0;
    } else {
        s.k0 = 0;
        s.lk = (int)p.Tk;
    }
    return s;
}

// Key blocks that the first `tokens` queries of a sequence see together (at least one: a query
// that sees no key still has an answer to write).
__device__ __forceinline__ int blocks_seen(const Seq& s, int tokens) {
    const int seen = s.lk - (s.lq - min(tokens, s.lq));
    return seen <= KB ? 1 : (seen - 1) / KB + 1;
}

// A sequence's pairs are taken from both ends in turn, 0, m - 1, 1, m - 2, ...: the number of blocks
// grows with the pair, and two neighbours then have about as many as any others, so that shares of
// a few whole pairs come out alike (three prompts 39.6 -> 34.7 us, the long one 705 -> 695 us).
__device__ __forceinline__ int pairs_of(const Seq& s, int tp) { return (s.lq + tp - 1) / tp; }
__device__ __forceinline__ int pair_in_turn(int i, int m) { return i & 1 ? m - 1 - (i >> 1) : i >> 1; }

// Weight of the sequence's first m pairs, m below pairs_of: the sum of PIECE + blocks_seen((j + 1) tp),
// in closed form from the sum of residues modulo 128, which repeat after 128 / gcd(tp, 128) pairs.
__device__ __noinline__ int64_t weight_before(int lq, int lk, int m, int tp) {
    const int d = lk - lq;
    int ones = d > KB ? 0 : (KB - d) / tp;   // pairs that see one block
    ones = min(ones, m);
    const int n = m - ones;
    if (n == 0) return ones + m * (int64_t)PIECE;
    const int b = (ones + 1) * tp + d + KB - 1;   // floor((b + i tp) / 128), i < n
    const int g = min(tp & -tp, KB), bits = 7 - (__ffs(g) - 1), per = 1 << bits;
    int64_t residues = (int64_t)(n >> bits) * (per * (b & (g - 1)) + g * per * (per - 1) / 2);
#pragma unroll 1
    for (int i = 0, r = b; i < (n & (per - 1)); ++i, r += tp) residues += r & (KB - 1);
    return ones + m * (int64_t)PIECE + (((int64_t)b * n + tp * ((int64_t)n * (n - 1) / 2) - residues) >> 7);
}
__device__ __forceinline__ int64_t weight_of(const Seq& s, int tp) {
    const int m = pairs_of(s, tp);
    return m == 0 ? 0 : weight_before(s.lq, s.lk, m - 1, tp) + PIECE + blocks_seen(s, s.lq);
}

// ... of the first i in turn; `all` is the weight of all m.
__device__ __noinline__ int64_t weight_in_turn(int lq, int lk, int i, int tp, int m, int64_t all) {
    const int64_t front = weight_before(lq, lk, (i + 1) >> 1, tp);
    return i < 2 ? front : front + all - weight_before(lq, lk, m - (i >> 1), tp);
}

// Where share b of `ctas` equal ones starts (recip = 2^64 / ctas, rounded up: no division).
__device__ __forceinline__ int64_t share_start(int64_t total, int b, int ctas, uint64_t recip) {
    return b == ctas ? total : (int64_t)__umul64hi((uint64_t)total * (uint64_t)b, recip);
}

// A step: pair `pair` (the turn-th to be taken) of key head kh of sequence n, key block j.
struct Cursor {
    int n, kh, turn, pair, j;
    Seq s;
};

// The whole block: checks the lengths, counts the steps and finds where share b starts and ends
// among them, in the order (sequence, key head, pair, key block).  Every CTA starts with this, so
// it is short in latency: one pass over the lengths, two block-wide exchanges, one parallel search.
struct Found {
    int64_t at, each;   // how far into its sequence; the weight of one key head there
    int n;
    Seq s;
};
struct Share {
    int64_t weight;
    Cursor at;          // where it starts
    bool bad;           // lengths that contradict the tensors
};
template <bool kSplit>
__device__ Share find_share(const AttnParams& p, int tq, int G, uint64_t recip, int64_t* scratch /* 48 */) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, tp = 2 * tq;
    const int per = (p.nseq + AT_THREADS - 1) / AT_THREADS;
    const int n0 = min(tid * per, p.nseq), n1 = min(n0 + per, p.nseq);
    Seq s{};
    int64_t mine = 0, each = 0;
    Share r{};
    auto weight = [&](int n) { return kSplit && (n < p.seq0 || n >= p.seq0 + p.seqs) ? (int64_t)0 : weight_of(s, tp); };   // of sequence n, which s holds
    bool bad = false;
#pragma unroll 1
    for (int n = n0; n < n1; ++n) {   // nothing is computed from bad lengths
        bool b = false;
        if (p.cu_q) b |= p.cu_q[n + 1] < p.cu_q[n] || (n == 0 && p.cu_q[0] != 0) || (n + 1 == p.nseq && p.cu_q[n + 1] > p.Tq);
        if (p.cu_k) b |= p.cu_k[n + 1] < p.cu_k[n] || (n == 0 && p.cu_k[0] != 0) || (n + 1 == p.nseq && p.cu_k[n + 1] > p.Tk);
        if (p.seqlens_k) b |= p.seqlens_k[n] < 0 || p.seqlens_k[n] > p.keys;
        bad |= b;
        s = seq_of(p, n);
        each = b ? 0 : weight(n);
        mine += each * p.Hk;
    }
    int64_t sum = mine;
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += y;
    }
    if (lane == 31) scratch[warp] = sum;
    int* best = reinterpret_cast<int*>(scratch + 16);   // [2]
    int64_t* start = scratch + 18;                      // [2]
    Found* found = reinterpret_cast<Found*>(scratch + 20);   // [2]: the start, the end
    if (tid < 2) best[tid] = 0, start[tid] = 0;
    r.bad = __syncthreads_or(bad);
    if (r.bad) return r;
    int64_t total = 0, before = sum - mine;
#pragma unroll
    for (int w = 0; w < AT_THREADS / 32; ++w) {
        before += w < warp ? scratch[w] : 0;
        total += scratch[w];
    }
    const int64_t x0 = share_start(total, blockIdx.x, gridDim.x, recip), x1 = share_start(total, blockIdx.x + 1, gridDim.x, recip);
    if (x0 >= total) return r;
#pragma unroll 1
    for (int e = 0; e < 2; ++e) {
        const int64_t x = e ? x1 : x0;
        if (x < before || x >= before + mine) continue;
        int64_t base = before;
        int n = n1 - 1;
        if (n > n0)
            for (n = n0;; ++n) {
                s = seq_of(p, n);
                each = weight(n);
                if (x < base + each * p.Hk) break;
                base += each * p.Hk;
            }
        found[e] = Found{x - base, each, n, s};
    }
    __syncthreads();
    // half of the threads for each end: the key head and the step within it; then the last pair that
    // starts at or before that step, of which every thread tries some
    const int e = tid >= AT_THREADS / 2;
    const bool open = e && x1 >= total;   // the last share's end needs no search
    const Found f = found[open ? 0 : e];
    Cursor u;
    u.n = f.n;
    u.s = f.s;
    int64_t at = f.at;
    u.kh = (int)((float)at / (float)f.each);   // (within one of the quotient, which is below 2^16)
    at -= u.kh * f.each;
    if (at < 0) --u.kh, at += f.each;
    else if (at >= f.each) ++u.kh, at -= f.each;
    const int m = open ? 1 : pairs_of(u.s, tp);
    int lo = 0, width = m;
#pragma unroll 1
    while (__syncthreads_or(width > 1)) {   // narrow [lo, lo + width)
        const int step = (width + AT_THREADS / 2 - 1) / (AT_THREADS / 2), c = lo + (tid % (AT_THREADS / 2)) * step;
        const int64_t st = width > 1 && c < lo + width ? weight_in_turn(u.s.lq, u.s.lk, c, tp, m, f.each) : at + 1;
        if (st <= at) atomicMax(best + e, c);
        __syncthreads();
        const int b = best[e];
        if (c == b && st <= at) start[e] = st;
        if (width > 1) width = min(step, lo + width - b), lo = b;
    }
    u.turn = lo;
    u.pair = pair_in_turn(lo, m);
    const int from = open ? 0 : (int)(at - start[e]);   // the pair's own weight is at its front
    u.j = max(from - PIECE, 0);
    // A cut near the end of a pair moves there: a pair that is cut costs its rows' partial results,
    // written and read again (about six steps' time for 256 rows; with the steps and the join of split keys two: 100 tokens
    // behind 900, 32 heads on 8, 27 us instead of 33).  Both neighbours find the same.
    int64_t x = (e ? x1 : x0) - (u.j > 0 ? 0 : from);
    const int nb = blocks_seen(u.s, (u.pair + 1) * tp), near = (kSplit ? 2 : 6) * min(min(u.s.lq - u.pair * tp, tp) * G, 256) >> 8;
    bool over = false;
    if (u.j > 0 && !open) {
        if (u.j <= near && u.j <= nb - u.j) x -= from, u.j = 0;
        else if (nb - u.j <= near) x += nb - u.j, over = true;
    }
    if (over) {   // the next pair
        u.j = 0;
        if (++u.turn < m) {
            u.pair = pair_in_turn(u.turn, m);
        } else {
            u.turn = u.pair = 0;
            if (++u.kh == p.Hk) {
                u.kh = 0;
                while (++u.n < p.nseq) {
                    u.s = seq_of(p, u.n);
                    if (u.s.lq > 0) break;
                }
            }
        }
    }
    __syncthreads();
    Cursor* place = reinterpret_cast<Cursor*>(scratch + 20);
    if (tid == 0) *place = u, start[0] = x;
    if (tid == AT_THREADS / 2) start[1] = x;
    __syncthreads();
    r.at = *place;
    r.weight = start[1] - start[0];
    return r;
}

// A share's next piece: the blocks [j0, j1) of one pair.
struct Piece {
    int j0, j1, nb;     // of nb
    int weight;
    int e0;             // the first tile's blocks end here (at most j1)
    bool two;           // the second tile has tokens
    bool whole;         // the share holds the whole pair
};

struct Ctx {
    uint32_t base, bars;
    int64_t weight;     // of this share
    int tq, tp, G;      // tokens of a tile and of a pair, heads of a group
    __device__ uint32_t bar(int b) const { return bars + 8u * b; }
    __device__ bool wait(int b, uint32_t use) const { return mx_wait(bar(b), use & 1u); }
};

__device__ __forceinline__ Piece piece_at(const Ctx& x, const Cursor& u, int64_t left) {
    Piece r;
    r.nb = blocks_seen(u.s, (u.pair + 1) * x.tp);
    r.j0 = u.j;
    const int own = u.j == 0 ? PIECE : 0;
    r.j1 = left - own < r.nb - u.j ? u.j + (int)left - own : r.nb;
    r.weight = r.j1 - u.j + own;
    r.two = u.pair * x.tp + x.tq < u.s.lq;
    r.e0 = r.two ? min(r.j1, blocks_seen(u.s, u.pair * x.tp + x.tq)) : r.j1;
    r.e0 = max(r.e0, r.j0);
    r.whole = r.j0 == 0 && r.j1 == r.nb;
    return r;
}

__device__ __forceinline__ void next_pair(const AttnParams& p, const Ctx& x, Cursor& u) {
    u.j = 0;
    const int m = pairs_of(u.s, x.tp);
    u.pair = pair_in_turn(++u.turn, m);
    if (u.turn < m) return;
    u.turn = u.pair = 0;
    if (++u.kh < p.Hk) return;
    u.kh = 0;
    do {
        if (++u.n >= p.nseq) return;
        u.s = seq_of(p, u.n);
    } while (u.s.lq == 0);
}

// ---------------------------------------------------------------- warp 8: loads
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(dst), "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}
template <bool kSplit>
__device__ bool load_warp(const AttnParams& p, const AttnMaps& maps, const Ctx& x, Cursor u) {
    bool ok = true;
    if ((threadIdx.x & 31) == 0) {
        int slot = 0;
        uint32_t lap = 0, pieces = 0;
        auto tile = [&](const CUtensorMap* m, int kh, int row, int n, const __half* rest) {
            if (lap > 0 && !mx_wait_lane(x.bar(EMPTY + slot), (lap - 1) & 1u)) return false;
            const uint32_t dst = x.base + OFF_RING + slot * TILE, full = x.bar(FULL + slot);
            if (p.Tk == 0) {   // no row to read: every key is masked and the values are set to zero
                mbar_arrive(full);
            } else {
                mbar_arrive_expect_tx(full, rest ? TILE + REST : TILE);
                if (rest) bulk_load(x.base + Layout<kSplit>::OFF_K_REST + slot * REST, rest, REST, full);
                tma_load_4d(dst, m, 0, kh, row, n, full);
                tma_load_4d(dst + HALF, m, 64, kh, row, n, full);
            }
            if (++slot == RING) slot = 0, ++lap;
            return true;
        };
        for (int64_t left = x.weight; left > 0 && ok; next_pair(p, x, u), ++pieces) {
            const Piece r = piece_at(x, u, left);
            left -= r.weight;
            const int n = kSplit ? u.n - p.seq0 : p.cache ? u.n : 0;
            for (int j = r.j0; j < r.j1 && ok; ++j) {
                const __half* rest = kSplit ? p.k_rest + (((int64_t)n * p.Hk + u.kh) * p.top_blocks + j) * (REST / 2) : nullptr;
                ok = tile(&maps.k, u.kh, u.s.k0 + j * KB, n, rest) && tile(&maps.v, u.kh, u.s.k0 + j * KB, n, nullptr);
                if (j > r.j0 || !ok) continue;
                // the queries, once the last scores of the piece before are done
                if (pieces > 0) ok = mx_wait_lane(x.bar(QE), (pieces - 1) & 1u);
                if (!ok) break;
                const int t0 = u.s.q0 + u.pair * x.tp;
                const uint32_t bytes = (uint32_t)(x.tq * x.G) * (256u + (kSplit ? 2 * SPLIT_REST : 0));
                mbar_arrive_expect_tx(x.bar(QF), r.two ? 2 * bytes : bytes);
                for (int t = 0; t < (r.two ? 2 : 1); ++t) {
                    tma_load_4d(x.base + t * TILE, &maps.q, 0, u.kh * x.G, t0 + t * x.tq, 0, x.bar(QF));
                    tma_load_4d(x.base + t * TILE + HALF, &maps.q, 64, u.kh * x.G, t0 + t * x.tq, 0, x.bar(QF));
                    if (!kSplit) continue;
                    const uint32_t rest_q = x.base + Layout<kSplit>::OFF_Q_REST + t * REST;   // eight channels: 128 rows of 16 bytes
                    tma_load_4d(rest_q, &maps.q_rest, 0, u.kh * x.G, t0 + t * x.tq, 0, x.bar(QF));
                    tma_load_4d(rest_q + REST / 2, &maps.q_rest, 8, u.kh * x.G, t0 + t * x.tq, 0, x.bar(QF));
                }
            }
        }
    }
    return __all_sync(0xffffffffu, ok);
}

// ---------------------------------------------------------------- warp 9: MMAs
constexpr uint64_t K_STEP = 32 >> 4, K_HALF = HALF >> 4, MN_STEP = 2048 >> 4, D_TILE = TILE >> 4;
constexpr uint32_t ID_KK = make_idesc_bf16_f32(128, 128), ID_MN = make_idesc_bf16_f32(128, 128, true);
constexpr uint32_t F16 = ~(1u << 7 | 1u << 10);   // both operands in fp16

// One warp for both tiles, strictly in turn: for each block P V of tile 0, the next scores of tile
// 0 (over P: the MMAs of a thread go in order), P V of tile 1, the next scores of tile 1.  (Two
// warps, one a tile, fall into step and leave the tensor core idle while both tiles are
// exponentiated: 984 against 890 us on 8,192 tokens x 64 heads.)  MMAs with both
// operands in shared memory are issued one by one as they execute, those with A in Tensor Memory
// queue up; so the waits stand behind the latter where they can.
template <bool kSplit>
__device__ bool mma_warp(const AttnParams& p, const Ctx& x, Cursor u) {
    const int lane = threadIdx.x & 31;
    const uint32_t lead = mx_leader();
    const uint64_t dQ = make_sdesc_kmajor_sw128(x.base), dK = make_sdesc_kmajor_sw128(x.base + OFF_RING);
    const uint64_t dV = make_sdesc_mnmajor_sw128(x.base + OFF_RING, HALF, 1024);
    const uint64_t dQR = make_sdesc_kmajor_noswizzle(x.base + Layout<kSplit>::OFF_Q_REST, REST / 2, 128);
    const uint64_t dKR = make_sdesc_kmajor_noswizzle(x.base + Layout<kSplit>::OFF_K_REST, REST / 2, 128);
    uint32_t it = 0;              // tiles of the ring before this piece: k and v alternate
    uint32_t pieces = 0, n0 = 0, n1 = 0, nX = 0, nZ = 0;
    // A wait's verdict is the lane's own (a vote each time would cost 3.5 % of a long prompt), so within a piece
    // nothing that the whole warp has to reach follows; the warp agrees at the piece's end.
    bool ok = true;
    // tile i of the piece has landed; its slot
    auto landed = [&](uint32_t i) { return mx_wait_lane(x.bar(FULL + (it + i) % RING), (it + i) / RING & 1u); };
    auto slot = [&](uint32_t i) { return (int)((it + i) % RING); };
    auto scores = [&](int q, int t, int j, int done) {   // of query tile q with the keys of block j, into place t
        const uint64_t a = dQ + q * D_TILE, k = dK + slot(2 * j) * D_TILE;
        constexpr uint32_t id = kSplit ? ID_KK & F16 : ID_KK;
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
            mx_mma_ss(lead, TM_S + 128 * t, a + (kk >> 2) * K_HALF + (kk & 3) * K_STEP, k + (kk >> 2) * K_HALF + (kk & 3) * K_STEP, id, kk > 0);
        if (kSplit) mx_mma_ss(lead, TM_S + 128 * t, dQR + q * (REST >> 4), dKR + slot(2 * j) * (REST >> 4), id, 1);
        mx_commit(lead, x.bar(done));
    };
    auto values = [&](int o, int t, int s, int half, bool first) {   // weights in place t, onto output o
        const uint64_t v = dV + s * D_TILE;
#pragma unroll
        for (int kk = 4 * half; kk < 4 * half + 4; ++kk)
            mx_mma_ts(lead, TM_O + 128 * o, TM_S + 128 * t + kk * 8, v + kk * MN_STEP, kSplit ? ID_MN & F16 : ID_MN, kk > 0 || !first);
    };
    // (half of) the weights are in place, for the n-th time
    auto weights = [&](int done, uint32_t n) {
        const bool r = mx_wait_lane(x.bar(done), n & 1u);
        tc_fence_after();
        return r;
    };
    u.n = mx_uniform(u.n), u.kh = mx_uniform(u.kh), u.turn = mx_uniform(u.turn), u.pair = mx_uniform(u.pair), u.j = mx_uniform(u.j);
    for (int64_t left = x.weight; left > 0; next_pair(p, x, u), ++pieces) {
        u.s.lq = mx_uniform(u.s.lq), u.s.lk = mx_uniform(u.s.lk);
        Piece r = piece_at(x, u, left);
        r.j0 = mx_uniform(r.j0), r.j1 = mx_uniform(r.j1), r.e0 = mx_uniform(r.e0);
        left -= r.weight;
        const int count = r.j1 - r.j0, c0 = r.e0 - r.j0;   // blocks; the first tile's
        // the values of block j have landed; those past the sequence's keys count for nothing,
        // whatever they hold
        auto next_values = [&](int j) {
            if (!landed(2 * j + 1)) return false;
            const int valid = u.s.lk - (r.j0 + j) * KB;
            if (!kSplit && valid < KB) {   // (split keys and values: their rows are zeros there)
                const uint32_t at = x.base + OFF_RING + slot(2 * j + 1) * TILE;
#pragma unroll 1
                for (int row = max(valid, 0); row < KB; ++row) sts_u64(at + (lane >> 4) * HALF + row * 128 + (lane & 15) * 8, 0u, 0u);
                fence_proxy_async_smem();
                mbar_arrive(x.bar(VZ));
                return mx_wait_lane(x.bar(VZ), nZ++ & 1u);
            }
            return true;
        };
        // the keys of block j are used; after the last ones the queries are too
        auto scored = [&](int j) {
            mx_commit(lead, x.bar(EMPTY + slot(2 * j)));
            if (j + 1 == count) mx_commit(lead, x.bar(QE));
        };
        ok = x.wait(QF, pieces) && __all_sync(0xffffffffu, landed(0));
        if (!ok) break;
        if (!r.two) {
            // one tile: its scores alternate between the two places, so that the next block's are there
            // when the tile's softmax has done with this one's
            scores(0, 0, 0, SF);
            scored(0);
            if (count > 1) {
                ok = landed(2);
                if (!ok) break;
                scores(0, 1, 1, SX);
                scored(1);
            }
#pragma unroll 1
            for (int j = 0; j < count; ++j) {
                const int t = j & 1;
                const uint32_t n = t ? nX++ : n0++;
                const int done = t ? PX : PF;
                ok = next_values(j) && weights(done, n);
                if (!ok) break;
                values(0, t, slot(2 * j + 1), 0, j == 0);
                ok = weights(done + 1, n);
                if (!ok) break;
                values(0, t, slot(2 * j + 1), 1, j == 0);
                mx_commit(lead, x.bar(j + 1 == count ? OF : PV));
                mx_commit(lead, x.bar(EMPTY + slot(2 * j + 1)));
                if (j + 2 < count) {
                    ok = landed(2 * j + 4);
                    if (!ok) break;
                    scores(0, t, j + 2, t ? SX : SF);
                    scored(j + 2);
                }
            }
        } else {
            if (c0 > 0) scores(0, 0, 0, SF);
            scores(1, 1, 0, SF + 1);
            scored(0);
            ok = next_values(0);
#pragma unroll 1
            for (int j = 0; ok; ++j) {
                const bool more = j + 1 < count;
                const int vs = slot(2 * j + 1);
                if (j < c0) {
                    ok = weights(PF, n0);
                    if (!ok) break;
                    values(0, 0, vs, 0, j == 0);
                    ok = weights(PF + 1, n0++);
                    if (!ok) break;
                    values(0, 0, vs, 1, j == 0);
                    if (j + 1 == c0) mx_commit(lead, x.bar(OF));
                }
                if (more) {
                    ok = landed(2 * j + 2);
                    if (!ok) break;
                    if (j + 1 < c0) scores(0, 0, j + 1, SF);
                }
                ok = weights(PF + 2, n1);
                if (!ok) break;
                values(1, 1, vs, 0, j == 0);
                ok = weights(PF + 3, n1++);
                if (!ok) break;
                values(1, 1, vs, 1, j == 0);
                mx_commit(lead, x.bar(EMPTY + vs));
                if (!more) {
                    mx_commit(lead, x.bar(OF + 1));
                    break;
                }
                ok = next_values(j + 1);
                if (!ok) break;
                scores(1, 1, j + 1, SF + 1);
                scored(j + 1);
            }
        }
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        it += 2 * count;
    }
    __syncwarp();
    mx_commit(lead, x.bar(DRAIN));
    return x.wait(DRAIN, 0) && ok;
}

// ---------------------------------------------------------------- warps 0-7: softmax and results
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// x 2^e, e within 2 x (-126 .. 127)
__device__ __forceinline__ float times_power(float x, int e) {
    const int half = e >> 1;
    return x * __uint_as_float((uint32_t)(127 + half) << 23) * __uint_as_float((uint32_t)(127 + e - half) << 23);
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

template <bool kSplit>
__device__ bool softmax_warps(const AttnParams& p, const AttnMaps& maps, const Ctx& x, Cursor u, int t) {
    const int row = threadIdx.x & 127;
    const uint32_t lanes = (uint32_t)(row & ~31) << 16, tO = lanes + TM_O + 128 * t;
    const int lane = threadIdx.x & 31;
    const uint32_t stage = x.base + Layout<kSplit>::OFF_STAGE + (threadIdx.x >> 5) * 4096;
    const float c = kSplit ? p.scale * LOG2E : fmaxf(p.scale * LOG2E, 1e-30f);   // (a scale of 0 must not turn a masked -inf into NaN)
    const Partials part = partials(p.workspace);
    const int tok = row / x.G, head = row - tok * x.G;
    uint32_t nS = 0, nX = 0, nO = 0, nV = 0;   // uses so far of SF, SX, OF and PV
    bool first_piece = true;
    for (int64_t left = x.weight; left > 0; next_pair(p, x, u), first_piece = false) {
        const Piece r = piece_at(x, u, left);
        left -= r.weight;
        if (t == 1 && !r.two) continue;
        const int end = t ? r.j1 : r.e0;
        bool other = false;   // this block's scores are in the other tile's place
        const int i = u.pair * x.tp + t * x.tq + tok;                  // query within the sequence
        const bool mine = tok < x.tq && i < u.s.lq;
        // the last key it sees; a row that is no query's is left as it is, nothing reads its results
        const int last = mine ? i + u.s.lk - u.s.lq : 0x7fffffff;
        float m = -INFINITY, l = 0.f;
        // split: a block's values are scaled by a power of two of their own (top[j], or one for each key); the output refers to
        // 2^(m + ref), where powers count from -127 as in a float.  m and ref are whole numbers, so that they move without rounding
        const int64_t unit_0 = kSplit ? ((int64_t)(u.n - p.seq0) * p.Hk + u.kh) * p.top_blocks : 0;
        // (at least 18 once a key is seen, since powers are SPLIT_LEAST and more)
        float ref = 20.f, neg = 0.f;   // neg: -m
        // ... and its keys and this query too: the exponents' scale is the block's, and m counts in steps of base 2
        const int power_q = kSplit && mine ? __ldg(p.q_power + (u.s.q0 + i) * (int64_t)p.Hq + u.kh * x.G + head) - 127 - SPLIT_KEY : 0;
        const float unit = kSplit ? 1.f : c;
        for (int j = r.j0; j < end; ++j) {
            const int tops_j = kSplit ? __ldg(p.top + unit_0 + j) : 0;
            float cj = kSplit ? fminf(fmaxf(times_power(c, power_q + (tops_j >> 16)), 1e-30f), 3e38f) : c;
            if (!x.wait(other ? SX : SF + t, other ? nX++ : nS++)) return false;
            tc_fence_after();
            const uint32_t tS = lanes + TM_S + 128 * (t + other);
            uint32_t s[128];
#pragma unroll
            for (int b = 0; b < 4; ++b) tmem_ld32(tS + 32 * b, reinterpret_cast<uint32_t(&)[32]>(s[32 * b]));
            tmem_wait_ld();
#pragma unroll
            for (int b = 0; b < 4; ++b) mx_loaded(reinterpret_cast<uint32_t(&)[32]>(s[32 * b]));
            const int seen = last - j * KB;   // columns 0 .. seen
            if (__any_sync(0xffffffffu, seen < KB - 1)) {
#pragma unroll
                for (int k = 0; k < 128; ++k) s[k] = k <= seen ? s[k] : 0xff800000u;
            }
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int k = 0; k < 128; k += 8)
#pragma unroll
                for (int e = 0; e < 4; ++e) mx[e] = max3(mx[e], mx_u2f(s[k + 2 * e]), mx_u2f(s[k + 2 * e + 1]));
            const float most = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])), top = kSplit ? most * cj : most;
            // the output has to hold all earlier products before it is scaled: with two tiles these scores
            // came after them; with one they did not, and the product before has a barrier of its own
            if (!r.two && j > r.j0 && !x.wait(PV, nV++)) return false;
            auto scale_output = [&](float f) {
                const float2 f2 = make_float2(f, f);
#pragma unroll 1
                for (int b = 0; b < 8; ++b) {
                    uint32_t o[16];
                    tmem_ld16(tO + 16 * b, o);
                    tmem_wait_ld_regs(o);
#pragma unroll
                    for (int k = 0; k < 16; k += 2) {
                        const float2 y = __fmul2_rn(make_float2(mx_u2f(o[k]), mx_u2f(o[k + 1])), f2);
                        o[k] = __float_as_uint(y.x);
                        o[k + 1] = __float_as_uint(y.y);
                    }
                    tmem_st16(tO + 16 * b, o);
                }
            };
            float mc, power = 0.f;   // what the exponents take; of it, what is not m's
            if constexpr (kSplit) {
                // (a comparison with m = -inf holds whenever a key is seen)
                float power_v = (float)(tops_j & 0xff);
                const bool each = tops_j & SPLIT_EACH, grown = mine && top - m > 8.f;
                mc = neg;
                if (each || __any_sync(0xffffffffu, grown || (mine && top - m + power_v > ref + 8.f) || fabsf(neg) > 0x1p20f)) {
                    if (grown) {
                        const float to = ceilf(top);
                        l *= exp2f(m - to);
                        if (m != -INFINITY) ref -= to - m;
                        m = to;
                        neg = -to;
                    }
                    float high = top + neg + power_v;   // the largest product of a weight and its value's power, as ref counts
                    mc = neg;
                    if (each) {
                        const uint4* powers = reinterpret_cast<const uint4*>(p.value_power + (unit_0 + j) * KB);
                        float sum[2] = {0.f, 0.f}, far[2] = {-INFINITY, -INFINITY};
#pragma unroll
                        for (int b = 0; b < 8; ++b) {
                            const uint4 w = __ldg(powers + b);
                            const uint32_t of[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                            for (int k = 0; k < 16; ++k) {
                                const float z = __fadd_rn(__fmul_rn(mx_u2f(s[16 * b + k]), cj), mc);
                                sum[k & 1] += ex2_approx(z);
                                const float y = z + (float)(of[k >> 2] >> 8 * (k & 3) & 255u);
                                far[k & 1] = fmaxf(far[k & 1], y);
                                s[16 * b + k] = __float_as_uint(y);
                            }
                        }
                        l += sum[0] + sum[1];
                        high = fmaxf(far[0], far[1]);
                        power_v = mc = 0.f;
                        cj = 1.f;
                    } else if (__any_sync(0xffffffffu, fabsf(mc) > 0x1p20f)) {   // so large that the scores have to be rounded as the maximum was
#pragma unroll
                        for (int k = 0; k < 128; ++k) s[k] = __float_as_uint(__fadd_rn(__fmul_rn(mx_u2f(s[k]), cj), mc));
                        cj = 1.f;
                        mc = 0.f;
                    }
                    const bool moved = mine && high > ref + 8.f;
                    float f = 1.f;
                    if (moved) {
                        const float to = ceilf(high);
                        f = exp2f(ref - to);
                        ref = to;
                    }
                    if (__any_sync(0xffffffffu, moved) && j > r.j0) scale_output(f);
                }
                power = power_v + (SPLIT_LIFT - ref);
                if (!each) power = fmaxf(power, -60.f);   // (weights far below that are nothing, and l is made from them)
                mc += power;
            } else {
                const bool grown = mine && (top - m) * unit > 8.f;   // (m = -inf: whenever a key is seen)
                if (__any_sync(0xffffffffu, grown)) {
                    const float f = grown ? exp2f((m - top) * unit) : 1.f;
                    if (grown) m = top;
                    l *= f;
                    if (j > r.j0) scale_output(f);
                }
                mc = m == -INFINITY ? 0.f : -m * unit;
            }
            const float2 c2 = make_float2(cj, cj), mc2 = make_float2(mc, mc);
            float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                uint32_t y[16];
#pragma unroll
                for (int k = 0; k < 32; k += 2) {
                    const float2 a = __ffma2_rn(make_float2(mx_u2f(s[32 * b + k]), mx_u2f(s[32 * b + k + 1])), c2, mc2);
                    const float2 e = make_float2(ex2_approx(a.x), ex2_approx(a.y));
                    sum[(k >> 1) & 1] = __fadd2_rn(sum[(k >> 1) & 1], e);
                    y[k / 2] = kSplit ? pack_half2(e.x, e.y) : pack_bf16x2(e.x, e.y);
                }
                tmem_st16(tS + 16 * b, y);
                if (b & 1) {   // half of P: the tensor core can start on it
                    tmem_wait_st();
                    tc_fence_before();
#ifdef KDA_WAIT_TEST
                    if ((int)blockIdx.x == p.test_skip) continue;
#endif
                    mx_arrive_warp(x.bar((other ? PX : PF + 2 * t) + (b >> 1)));
                }
            }
            const float all = (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
            if (!kSplit) l += all;
            else if (!(tops_j & SPLIT_EACH)) l += times_power(all, -(int)power);
            other = !r.two && !other;
        }
        const int64_t q = u.s.q0 + i;
        const int h = u.kh * x.G + head;
        const size_t part_slot = 2 * blockIdx.x + (first_piece ? 0 : 1);
        const int part_row = 128 * t + row;
        const uint32_t mask = __ballot_sync(0xffffffffu, mine);
        if (end > r.j0) {
            if (!x.wait(OF + t, nO)) return false;
            ++nO;
            tc_fence_after();
            const float back = kSplit ? times_power(1.f, (int)ref - 127 - SPLIT_TOP - SPLIT_LIFT) : 1.f;   // to 2^m
            if (!r.whole) {
                float4* o = part.o + part_slot * 32 * 256 + part_row;
#pragma unroll 1
                for (int b = mask ? 0 : 4; b < 4; ++b) {
                    uint32_t w[32];
                    tmem_ld32(tO + 32 * b, w);
                    tmem_wait_ld();
                    mx_loaded(w);
                    if (mine) {
                        if (kSplit) {
#pragma unroll
                            for (int k = 0; k < 32; ++k) w[k] = __float_as_uint(back * mx_u2f(w[k]));
                        }
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            o[(8 * b + k) * 256] = make_float4(mx_u2f(w[4 * k]), mx_u2f(w[4 * k + 1]), mx_u2f(w[4 * k + 2]), mx_u2f(w[4 * k + 3]));
                    }
                    __syncwarp();
                }
            } else {
                // 64 channels at a time through the warp's stage; then one tensor store of the warp's rows
                // if they are whole tokens and all there, or eight lanes a row
                const float inv = l == 0.f ? 0.f : kSplit ? back / l : 1.f / l;
                const float2 inv2 = make_float2(inv, inv);
                const bool tensor = !kSplit && mask == 0xffffffffu && x.G <= 32 && (x.G & (x.G - 1)) == 0;
                const unsigned long long dst = reinterpret_cast<unsigned long long>(p.out.data + q * p.out.row + h * p.out.head);
#pragma unroll 1
                for (int b = mask ? 0 : 4; b < 4; ++b) {
                    uint32_t w[32];
                    tmem_ld32(tO + 32 * b, w);
                    tmem_wait_ld();
                    mx_loaded(w);
#pragma unroll
                    for (int k = 0; k < 32; k += 2) {
                        const float2 y = __fmul2_rn(make_float2(mx_u2f(w[k]), mx_u2f(w[k + 1])), inv2);
                        w[k / 2] = pack_bf16x2(y.x, y.y);
                    }
                    if constexpr (kSplit) {   // (no room for a stage: each thread its own row)
                        if (mine) {
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                *reinterpret_cast<uint4*>(dst + 64 * b + 16 * k) = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
                        }
                    } else {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            sts_u128(stage + lane * 128 + (((4 * (b & 1) + k) ^ (lane & 7)) << 4), w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
                        if (!(b & 1)) continue;
                        if (tensor) {
                            fence_proxy_async_smem();
                            __syncwarp();
                            if (lane == 0) {
                                tma_store_3d(&maps.out, stage, 32 * (b - 1), u.kh * x.G, (int)q);
                                bulk_commit();
                                bulk_wait_read_all();
                            }
                        } else {
                            __syncwarp();
#pragma unroll 1
                            for (int k = 0; k < 8; ++k) {
                                const int from = 4 * k + (lane >> 3);   // this lane's row in turn
                                const unsigned long long d = __shfl_sync(0xffffffffu, dst, from);
                                const uint4 y = lds_u128(stage + from * 128 + (((lane & 7) ^ (from & 7)) << 4));
                                if (mask >> from & 1u) *reinterpret_cast<uint4*>(d + (b >> 1) * 128 + (lane & 7) * 16) = y;
                            }
                        }
                    }
                    __syncwarp();
                }
            }
            tc_fence_before();
        }
        if (mine) {
            if (!r.whole) part.ml[part_slot * 256 + part_row] = make_float2(m * unit, l);
            else if (p.lse) p.lse[q * p.lse_row + h] = l == 0.f ? -INFINITY : (m * unit + log2f(l)) * 0.6931471805599453f;
        }
    }
    if (lane == 0) bulk_wait_all();
    __syncwarp();
    return true;
}

template <bool kSplit>
__global__ void __launch_bounds__(AT_THREADS, 1) attn_kernel(const AttnParams p, const __grid_constant__ AttnMaps maps, uint64_t recip) {
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    const int tid = threadIdx.x, warp = mx_uniform(tid >> 5);
    asm volatile("griddepcontrol.launch_dependents;");
    using L = Layout<kSplit>;
    Ctx x;
    x.base = smem_u32(smem_raw);
    x.bars = x.base + L::OFF_BAR;
    x.G = p.Hq / p.Hk;
    x.tq = 128 / x.G;
    x.tp = 2 * x.tq;
    if (warp == 8) {
        if ((tid & 31) == 0) {
            for (int b = 0; b < NBAR; ++b) mbar_init(x.bar(b), b == VZ ? 32 : (b >= PF && b < PF + 4) || b == PX || b == PX + 1 ? 4 : 1);
            mbar_fence_init();
            tma_prefetch_desc(&maps.q);
            tma_prefetch_desc(&maps.k);
            tma_prefetch_desc(&maps.v);
            tma_prefetch_desc(&maps.out);
        }
        __syncwarp();
        tmem_alloc(x.base + L::OFF_TMEM, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    await_stream();
    const Share share = find_share<kSplit>(p, x.tq, x.G, recip, reinterpret_cast<int64_t*>(smem_raw + L::OFF_SCRATCH));
    const Cursor u = share.at;
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = lds_u32(x.base + L::OFF_TMEM);
    bool sound = tmem == 0 && x.base % 1024 == 0;   // (the tiles' swizzle counts from 1 KB boundaries)
#ifdef KDA_WAIT_TEST
    sound = sound && p.test_skip != -2 - (int)blockIdx.x;
#endif
    x.weight = sound ? share.weight : 0;                  // (bad lengths have none)
    if (tid == 0) {
        Cut c{};
        if (x.weight > 0) c = Cut{u.j, blocks_seen(u.s, (u.pair + 1) * x.tp), u.s.q0, u.s.lq, u.kh, u.pair};
        c.status = (share.bad ? KDA_DEVERR_CU_SEQLENS : 0u) | (sound ? 0u : KDA_DEVERR_INTERNAL);
        partials(p.workspace).cut[blockIdx.x] = c;
    }
    bool ok = true;
    // registers a thread: 168 at launch; 208 + 208 + 88 of the 3 x 168 that the block holds
    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        ok = softmax_warps<kSplit>(p, maps, x, u, warp >> 2);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
        if (warp == 8) ok = load_warp<kSplit>(p, maps, x, u);
        else if (warp == 9) ok = mma_warp<kSplit>(p, x, u);
    }
    if (!ok) mx_wind_down();
    tc_fence_before();
    ok = __syncthreads_and(ok);
    if (!ok && tid == 0) atomicOr(&partials(p.workspace).cut[blockIdx.x].status, KDA_DEVERR_TIMEOUT);
    if (warp == 8) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Joins the partial rows of the pairs that several shares hold (and, the last block, the shares' status bits: one store,
// so that none is lost).  Block (b, y) takes 32 rows of the
// pair that share b + 1 starts in, if that is the pair's first cut; a warp takes four of them, lane l
// their channels 4 l .. 4 l + 3.  Bound by latency: little code (it is fetched cold) and few loads
// in a row.
constexpr int JOIN_THREADS = 256, JOIN_ROWS = 32;
// The parts of the pair that share `first` starts in, if that is the pair's first cut: share b's last piece (or its first one: `same`),
// then the first pieces of the shares before `end`, empty ones between.
struct Parts {
    Cut c;
    int b, end;
    bool same;
    __device__ size_t slot(int s) const { return (size_t)(2 * s + (s == b && !same ? 1 : 0)); }
};
__device__ __forceinline__ bool find_parts(const Partials& part, int first, int ctas, Parts& r) {
    const int lane = threadIdx.x & 31;
    r.c = part.cut[first];
    Cut before = part.cut[first - 1];
    Cut e = part.cut[min(first + lane, ctas - 1)];
    if (r.c.j == 0) return false;                // between two pairs, or nothing to do
    // the share before it that is not empty starts at or before the pair, or that cut was the first
    r.b = first - 1;
    while (r.b > 0 && before.nb == 0) before = part.cut[--r.b];
    auto inside = [&](const Cut& a) { return a.q0 == r.c.q0 && a.lq == r.c.lq && a.kh == r.c.kh && a.pair == r.c.pair; };
    r.same = inside(before);
    if (r.same && before.j > 0) return false;
    r.end = first;
    for (;;) {
        const uint32_t past = __ballot_sync(0xffffffffu, r.end + lane >= ctas || (e.nb != 0 && (e.j == 0 || !inside(e))));
        if (past) {
            r.end += __ffs(past) - 1;
            return true;
        }
        r.end += 32;
        e = part.cut[min(r.end + lane, ctas - 1)];
    }
}
// The shares' status bits.
__device__ __forceinline__ void join_status(const AttnParams& p, const Partials& part, int ctas) {
    const int lane = threadIdx.x & 31;
    uint32_t status = 0;
    for (int s = lane; s < ctas; s += 32) status |= part.cut[s].status;
    status = __reduce_or_sync(0xffffffffu, status);
    if (lane == 0) *p.status = p.keep_status ? *p.status | status : status;
}

__global__ void __launch_bounds__(JOIN_THREADS) attn_join_kernel(const AttnParams p, int ctas) {
    const int first = blockIdx.x + 1, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int G = p.Hq / p.Hk, tq = 128 / G;
    const Partials part = partials(p.workspace);
    await_stream();
    if (first == ctas) {
        if (blockIdx.y == 0 && warp == 0) join_status(p, part, ctas);
        return;
    }
    Parts r;
    if (!find_parts(part, first, ctas, r)) return;
    const Cut c = r.c;
    const int b = r.b, end = r.end;
    auto slot = [&](int s) { return r.slot(s); };
#pragma unroll 1
    for (int k = 0; k < JOIN_ROWS / 8; ++k) {
        const int row = blockIdx.y * JOIN_ROWS + 8 * k + warp;
        const int t = row >> 7, tok = (row & 127) / G, head = (row & 127) - tok * G;
        const int i = (2 * c.pair + t) * tq + tok;
        if (tok >= tq || i >= c.lq) continue;
        float m = -INFINITY, l = 0.f;   // this lane's parts; then all
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
        for (int s0 = b; s0 < end; s0 += 32) {   // (more than 32 parts: the sums so far are rescaled)
            const int s = s0 + lane;
            float2 ml = make_float2(-INFINITY, 0.f);
            if (s < end && (s == b || part.cut[s].nb != 0)) ml = part.ml[slot(s) * 256 + row];
            float top = ml.y != 0.f ? ml.x : -INFINITY;   // a part that saw no key has a sum of 0 (a NaN goes on into the results)
#pragma unroll 1
            for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            top = fmaxf(top, m);
            const float old = m == -INFINITY ? 0.f : exp2f(m - top);
            m = top;
            const float w = ml.y != 0.f ? exp2f(ml.x - m) : 0.f;
            l = fmaf(l, old, w * ml.y);
            o.x *= old, o.y *= old, o.z *= old, o.w *= old;
            const int n = min(32, end - s0);
#pragma unroll 1
            for (int a = 0; a < n; a += 8) {
                float4 y[8];
                float f[8];
#pragma unroll
                for (int d = 0; d < 8; ++d) {   // (the rows of a part that saw no key may not even be written)
                    f[d] = __shfl_sync(0xffffffffu, w, (a + d) & 31);
                    if (a + d >= n) f[d] = 0.f;
                    y[d] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (f[d] != 0.f) y[d] = __ldcg(part.o + (slot(s0 + a + d) * 32 + lane) * 256 + row);
                }
#pragma unroll
                for (int d = 0; d < 8; ++d) {
                    o.x = fmaf(f[d], y[d].x, o.x);
                    o.y = fmaf(f[d], y[d].y, o.y);
                    o.z = fmaf(f[d], y[d].z, o.z);
                    o.w = fmaf(f[d], y[d].w, o.w);
                }
            }
        }
#pragma unroll 1
        for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const int64_t q = c.q0 + i;
        const int h = c.kh * G + head;
        *reinterpret_cast<uint2*>(p.out.data + q * p.out.row + h * p.out.head + 4 * lane) =
            make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
        if (p.lse && lane == 0) p.lse[q * p.lse_row + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
    }
}

// The same for pairs of many rows: a thread takes a row, block (b, y) its channels 16 y .. 16 y + 15, so that a
// warp reads 512 bytes together, as they were written; two parts are asked for at once.  (Continued prompts 740 -> 703 us at the
// time; the join above took some 40.  Eight channels and four parts: 1,000 over 5,000, 32 heads on 8, 83.5 us, now 81.7; two parts
// 83.7; 32 channels 104.)
constexpr int JOIN_PARTS = 2, JOIN_GROUPS = 4;
__global__ void __launch_bounds__(JOIN_THREADS, 4) attn_join_rows_kernel(const AttnParams p, int ctas) {
    const int first = blockIdx.x + 1, row = threadIdx.x, G = p.Hq / p.Hk, tq = 128 / G;
    const Partials part = partials(p.workspace);
    await_stream();
    if (first == ctas) {
        if (blockIdx.y == 0 && row < 32) join_status(p, part, ctas);
        return;
    }
    Parts r;
    if (!find_parts(part, first, ctas, r)) return;
    const int t = row >> 7, tok = (row & 127) / G, head = (row & 127) - tok * G, i = (2 * r.c.pair + t) * tq + tok;
    if (tok >= tq || i >= r.c.lq) return;
    float m = -INFINITY, l = 0.f;
    float4 o[JOIN_GROUPS] = {};
#pragma unroll 1
    for (int s0 = r.b; s0 < r.end; s0 += JOIN_PARTS) {
        float2 ml[JOIN_PARTS];
        float4 y[JOIN_PARTS][JOIN_GROUPS];
#pragma unroll
        for (int d = 0; d < JOIN_PARTS; ++d) {
            const int s = s0 + d;
            ml[d] = make_float2(-INFINITY, 0.f);
            if (s < r.end && (s == r.b || part.cut[s].nb != 0)) {
                ml[d] = __ldcg(part.ml + r.slot(s) * 256 + row);
#pragma unroll
                for (int k = 0; k < JOIN_GROUPS; ++k) y[d][k] = __ldcg(part.o + (r.slot(s) * 32 + JOIN_GROUPS * blockIdx.y + k) * 256 + row);
            }
        }
        float top = m;
#pragma unroll
        for (int d = 0; d < JOIN_PARTS; ++d) top = ml[d].y != 0.f ? fmaxf(top, ml[d].x) : top;   // a part that saw no key has a sum of 0 (a NaN goes on into the results)
        const float old = m == -INFINITY ? 0.f : exp2f(m - top);
        m = top;
        l *= old;
#pragma unroll
        for (int k = 0; k < JOIN_GROUPS; ++k) o[k].x *= old, o[k].y *= old, o[k].z *= old, o[k].w *= old;
#pragma unroll
        for (int d = 0; d < JOIN_PARTS; ++d) {
            if (ml[d].y == 0.f) continue;   // (its rows may not even be written)
            const float w = exp2f(ml[d].x - m);
            l = fmaf(w, ml[d].y, l);
#pragma unroll
            for (int k = 0; k < JOIN_GROUPS; ++k) {
                o[k].x = fmaf(w, y[d][k].x, o[k].x);
                o[k].y = fmaf(w, y[d][k].y, o[k].y);
                o[k].z = fmaf(w, y[d][k].z, o[k].z);
                o[k].w = fmaf(w, y[d][k].w, o[k].w);
            }
        }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const int64_t q = r.c.q0 + i;
    const int h = r.c.kh * G + head;
#pragma unroll
    for (int k = 0; k < JOIN_GROUPS; k += 2)
        *reinterpret_cast<uint4*>(p.out.data + q * p.out.row + h * p.out.head + 4 * (JOIN_GROUPS * blockIdx.y + k)) =
            make_uint4(pack_bf16x2(o[k].x * inv, o[k].y * inv), pack_bf16x2(o[k].z * inv, o[k].w * inv), pack_bf16x2(o[k + 1].x * inv, o[k + 1].y * inv),
                       pack_bf16x2(o[k + 1].z * inv, o[k + 1].w * inv));
    if (p.lse && blockIdx.y == 0) p.lse[q * p.lse_row + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

}  // namespace

size_t attn_workspace_bytes(int64_t, int, int) {
    return CUT_BYTES + ML_BYTES + (size_t)2 * AT_MAX_CTAS * 256 * HD * sizeof(float);
}

template <bool kSplit>
static cudaError_t launch(const AttnParams& p, cudaStream_t stream) {
    const int G = p.Hq / p.Hk, tq = 128 / G;
    AttnMaps maps;
    memset(&maps, 0, sizeof(maps));
    const int seqs = kSplit ? p.seqs : p.cache ? p.nseq : 1;
    if (!mx_encode(&maps.q, p.q.data, p.Hq, p.Tq, 1, p.q.head, p.q.row, 0, G, tq) ||
        !mx_encode(&maps.k, p.k, p.Hk, p.Tk, seqs, p.k_head, p.k_row, p.k_seq, 1, KB) ||
        (kSplit && !mx_encode(&maps.q_rest, p.q_rest, p.Hq, p.Tq, 1, SPLIT_REST, (int64_t)SPLIT_REST * p.Hq, 0, G, tq, SPLIT_REST, 8)) ||
        !mx_encode(&maps.v, p.v, p.Hk, p.Tk, seqs, p.v_head, p.v_row, p.v_seq, 1, KB) ||
        !mx_encode_3d(&maps.out, p.out.data, p.Hq, p.Tq, p.out.head, p.out.row, G <= 32 ? G : 1, G <= 32 ? 32 / G : 1))
        return cudaErrorInvalidValue;
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(attn_kernel<kSplit>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Layout<kSplit>::SMEM);
    if (e != cudaSuccess) return e;
    const int ctas = sms < AT_MAX_CTAS ? sms : AT_MAX_CTAS;
    e = launch_early(attn_kernel<kSplit>, dim3((unsigned)ctas), AT_THREADS, Layout<kSplit>::SMEM, stream, p, maps,
                     ctas > 1 ? ~0ull / (uint64_t)ctas + 1 : (uint64_t)0);
    if (e != cudaSuccess) return e;
    if constexpr (kSplit) return launch_early(attn_join_rows_kernel, dim3((unsigned)ctas, HD / (4 * JOIN_GROUPS)), JOIN_THREADS, 0, stream, p, ctas);
    return launch_early(attn_join_kernel, dim3((unsigned)ctas, 256 / JOIN_ROWS), JOIN_THREADS, 0, stream, p, ctas);
}

cudaError_t launch_attn(const AttnParams& p, cudaStream_t stream) { return launch<false>(p, stream); }
cudaError_t launch_attn_split(const AttnParams& p, cudaStream_t stream) { return launch<true>(p, stream); }

}  // namespace kda
