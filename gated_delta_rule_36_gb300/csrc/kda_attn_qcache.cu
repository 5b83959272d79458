// Causal softmax attention with grouped heads over a cache held in 4 bits.  Few rows (single tokens, drafts): one pass
// over the keys with the running maximum and sum, mma.sync on codes that never leave registers.  Many rows (prompts that
// continue): at the end of this file.
//
// A tile is 8 kN rows of (token, head) pairs that share a key head, a slice 32 keys (4,608 bytes).  A warp takes
// every eighth slice by bulk copies into its own small ring and waits for no other warp until the tile is done:
//   A_h = Y_h Q_h^T       (keys x queries) for the two halves h of the channels, Y the codes
//   s = sum_h scale_h A_h + zero_h sum_c q_c     in fp32
//   p = exp2(c s - m),  l += p,  R_h = bf16(p scale'_h),  z_h += p (zero'_h + 7.5 scale'_h)   (the values' numbers)
//   O_h += Y'_h^T R_h,  u_h += 1^T R_h
//   out_h = (O_h - 7.5 u_h + z_h) / l
// so that codes count from their middle (7.5): a weight's rounding to bf16, at most 2^-8 of it, then moves the output by that
// share of what the value deviates from its group's middle, and the middle itself is summed in fp32.  Against 64 bits the
// output is off by 0.0021 to 0.0024 of its norm, 0.0017 of which is its own rounding to bf16.  One term for a weight, as
// attention over a bf16 cache has: with a second one (its rest) the output's own rounding is all that remains, but one token over 32,767
// takes 20.5 instead of 18.9 us, 32 tokens 44.4 instead of 38.7, 24 x 4 drafts 51.6 instead of 42 (16 long ones 85 both).
//
// A code becomes a bf16 operand by a mask alone: in the lowest eight bits (seven of the fraction and one of the
// exponent, whose first step continues the subnormal numbers) bf16 counts linearly, so four bits there are
// code 2^-133 or, four places higher, code 2^-129.  The other operands carry the powers of two that bring the
// products back: q 2^64 against the first and 2^60 against the second, weights 2^60.  (A shift and a mask for
// two codes, 1 + code / 16, is 8 instead of 5 instructions for eight codes, on the pipe that bounds the slices;
// e4m3, where a byte 0 .. 15 is code 2^-9, would be 3, but its mma.sync is no single instruction here: 30 % more in all.)
// The maximum m that the exponents refer to moves only when a score exceeds it by more than 8 (base 2), so that
// most slices need no exchange between lanes.
//
// All (sequence, key head, tile, slice) steps are one line that is cut into equal shares, two for each SM (one with tiles of 16
// rows); a tile that lies in more than one share leaves unnormalised partial rows in the workspace, and a second, small kernel
// joins them in the order of the keys.  What a tile costs by itself counts as PIECE slices in front of it (32 tokens with
// 6, 10, 14, 20: 56, 47, 42, 42 us; drafts with 14, 20, 32, 44 on tiles of 16 rows: 67, 55, 48, 50).
//
// Bound by HBM between a start of about 2 us (the lengths, the search), some 3 us a tile (queries, the warps' results)
// and the join (3 us): 32 single tokens over caches of 67 to 8,189, 32 heads on 8: 39 us (3.9 TB/s; 6.4 in the slices);
// 16 over 5,002 to 32,767, 64 heads on 8, heads inside the rows: 83 to 88 us, where the 144 bytes of a head bring 21 %
// of others with them (heads outside: 72 us, 4.8 TB/s); one token over 32,767: 19 us, over 2,000 9.7;
// 24 x 4 drafts: 42 us, bound by latency with eight warps an SM.

#include <cuda_fp16.h>
#include <string.h>

#include "kda_mixer.cuh"
#include "kda_qcache.cuh"

namespace kda {
namespace {

constexpr int QS_WARPS[3] = {0, 8, 8};             // by kN (16 rows: ten and twelve warps spill, 81 and 101 us against 48 on drafts)
constexpr int QS_MAX_CTAS = 320;
constexpr int SLICE = 32;                          // keys
constexpr uint32_t SLICE_BYTES = SLICE * QC_ROW;
constexpr int QS_MAX_ROWS = 16;                    // of a tile of 8 rows for the heads that go together (16 rows: 32)
constexpr int PIECE[3] = {0, 18, 34};              // a tile's own weight, in slices, by kN
// Weights are carried as p 2^60, and pass that by 2^8 at most: with scales and zeros below 2^40 a lane's sums of their
// products (2^68 2^43.1 each) stay in fp32's range for 2^15 keys, 4 million of a share; with scales from 2^-40 on the
// products with codes (2^-73) are normal numbers.
constexpr float LIFT = 60.f;
constexpr float NO_KEY = -3e38f;                   // (finite, so that a masked -inf less this is -inf)
constexpr float UNLIFT = 0x1p-60f, CODE = 0x1p73f; // a product of a value's code and a weight, brought back
constexpr float KEY_CODE = 0x1p-69f;               // a product of a key's code and a query, of 1 and 1

// What a share leaves for the join: the tile that it starts in and how far into it, and its status bits.
struct QsCut {
    int j, some;        // starts at slice j (0: between two tiles); not an empty share
    int n, kh, tile;
    int q0, lq;
    uint32_t status;
};
struct QsPartials {
    QsCut* cut;         // [shares]
    float2* ml;         // [2 * shares][kN * QS_MAX_ROWS]: reference exponent (base 2) and sum
    float* o;           // [2 * shares][kN * QS_MAX_ROWS][128], not normalised
};
constexpr size_t QS_CUT_BYTES = QS_MAX_CTAS * sizeof(QsCut), QS_ML_BYTES = (size_t)2 * QS_MAX_CTAS * QS_MAX_ROWS * sizeof(float2);
__device__ __forceinline__ QsPartials qs_partials(void* ws) {
    char* at = static_cast<char*>(ws);
    return QsPartials{reinterpret_cast<QsCut*>(at), reinterpret_cast<float2*>(at + QS_CUT_BYTES), reinterpret_cast<float*>(at + QS_CUT_BYTES + QS_ML_BYTES)};
}

struct QsSeq {
    int q0, lq, lk;
};
__device__ __forceinline__ QsSeq qs_seq(const QcacheAttnParams& p, int n) {
    QsSeq s;
    if (p.cu_q) {
        s.q0 = (int)p.cu_q[n];
        s.lq = (int)p.cu_q[n + 1] - s.q0;
    } else {
        s.lq = (int)p.uniform_q;
        s.q0 = n * s.lq;
    }
    s.lk = (int)p.seqlens_k[n];
    return s;
}
__device__ __forceinline__ int qs_tiles(const QsSeq& s, int G, int rows) { return (int)(((int64_t)s.lq * G + rows - 1) / rows); }
__device__ __forceinline__ int qs_slices(const QsSeq& s) { return (s.lk + SLICE - 1) / SLICE; }

// A step: slice j of tile `tile` of the 2^hg key heads from kh << hg on, of sequence n.
struct QsCursor {
    int n, kh, tile, j;
    QsSeq s;
};
struct QsShare {
    QsCursor at;
    int64_t weight;
    bool bad;
};

// Where share b of `shares` equal ones starts.
__device__ __forceinline__ int64_t qs_share_start(int64_t total, int b, int shares) {
    if (b >= shares) return total;
    if (total < (1LL << 22)) return (int64_t)((uint32_t)total * (uint32_t)b / (uint32_t)shares);   // (b < 2^10)
    return total / shares * b + total % shares * b / shares;
}

// Sequence n's lengths contradict the tensors.
__device__ __forceinline__ bool qs_bad(const QcacheAttnParams& p, int n) {
    bool b = p.seqlens_k[n] < 0 || p.seqlens_k[n] > p.S;
    if (p.cu_q) b |= p.cu_q[n + 1] < p.cu_q[n] || (n == 0 && p.cu_q[0] != 0) || (n + 1 == p.nseq && p.cu_q[n + 1] > p.Tq);
    return b;
}
template <int kN, int kHg>
__device__ __forceinline__ int64_t qs_weight(const QcacheAttnParams& p, const QsSeq& s, int G) {
    constexpr int own = PIECE[kN] >> kHg;
    return (int64_t)qs_tiles(s, G, 8 * kN) * (p.Hk >> kHg) * (qs_slices(s) + own);
}
// Step `at` of sequence n.  A cut inside a tile's own weight, which is at its front, moves to the tile's start: by `back` steps.
template <int kN, int kHg>
__device__ __forceinline__ QsCursor qs_cursor(const QsSeq& s, int n, int64_t at, int G, int& back) {
    constexpr int own = PIECE[kN] >> kHg;
    const int w = qs_slices(s) + own, tiles = qs_tiles(s, G, 8 * kN);
    const bool small = (at >> 31) == 0;   // (64-bit divisions take long)
    const int64_t unit = small ? (int64_t)((uint32_t)at / (uint32_t)w) : at / w;
    const int head = tiles == 1 ? (int)unit : small ? (int)((uint32_t)unit / (uint32_t)tiles) : (int)(unit / tiles);
    const int from = (int)(at - unit * w), j = max(from - own, 0);
    back = j > 0 ? 0 : from;
    return QsCursor{n, head, (int)(unit - (int64_t)head * tiles), j, s};
}

// Checks the lengths, counts the steps and finds where share b starts and ends among them.  At most 32 sequences: every warp by itself.
template <int kN, int kHg>
__device__ QsShare qs_find_share_by_warp(const QcacheAttnParams& p, int G) {
    const int lane = threadIdx.x & 31;
    const bool mine = lane < p.nseq;
    QsSeq s{};
    QsShare r{};
    if (mine) s = qs_seq(p, lane);
    r.bad = __any_sync(0xffffffffu, mine && qs_bad(p, lane));
    if (r.bad) return r;
    const int64_t weight = mine ? qs_weight<kN, kHg>(p, s, G) : 0;
    int64_t end = weight;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, end, o);
        if (lane >= o) end += y;
    }
    const int64_t total = __shfl_sync(0xffffffffu, end, 31);
    const int shares = (int)min((int64_t)gridDim.x, max(total / (QS_WARPS[kN] >> kHg), (int64_t)1));
    const int64_t x0 = qs_share_start(total, blockIdx.x, shares), x1 = qs_share_start(total, blockIdx.x + 1, shares);
    if (x0 >= total) return r;
    const uint32_t first = __ffs(__ballot_sync(0xffffffffu, x0 < end)) - 1, last = __ffs(__ballot_sync(0xffffffffu, x1 < end)) - 1;   // (-1: none)
    int back0 = 0, back1 = 0;
    QsCursor u{};
    if (lane == first) u = qs_cursor<kN, kHg>(s, lane, x0 - (end - weight), G, back0);
    if (lane == last) qs_cursor<kN, kHg>(s, lane, x1 - (end - weight), G, back1);
    auto of = [](int x, uint32_t l) { return __shfl_sync(0xffffffffu, x, l); };
    r.at = QsCursor{(int)first, of(u.kh, first), of(u.tile, first), of(u.j, first), QsSeq{of(s.q0, first), of(s.lq, first), of(s.lk, first)}};
    r.weight = x1 - (last == ~0u ? 0 : of(back1, last)) - (x0 - of(back0, first));
    return r;
}
// ... the whole block.
template <int kN, int kHg>
__device__ QsShare qs_find_share(const QcacheAttnParams& p, int G, int64_t* scratch /* 32 */) {
    constexpr int warps = QS_WARPS[kN], threads = 32 * warps;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (p.nseq + threads - 1) / threads;
    const int n0 = min(tid * per, p.nseq), n1 = min(n0 + per, p.nseq);
    QsSeq s{};
    int64_t mine = 0, each = 0;
    bool bad = false;
#pragma unroll 1
    for (int n = n0; n < n1; ++n) {   // nothing is computed from bad lengths
        const bool b = qs_bad(p, n);
        bad |= b;
        s = qs_seq(p, n);
        each = b ? 0 : qs_weight<kN, kHg>(p, s, G);
        mine += each;
    }
    int64_t sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += y;
    }
    if (lane == 31) scratch[warp] = sum;
    QsShare r{};
    r.bad = __syncthreads_or(bad);
    if (r.bad) return r;
    int64_t total = 0, before = sum - mine;
#pragma unroll
    for (int w = 0; w < warps; ++w) {
        before += w < warp ? scratch[w] : 0;
        total += scratch[w];
    }
    // (fewer shares than CTAs where a share would not give every warp a slice)
    const int shares = (int)min((int64_t)gridDim.x, max(total / (warps >> kHg), (int64_t)1));
    const int64_t x0 = qs_share_start(total, blockIdx.x, shares), x1 = qs_share_start(total, blockIdx.x + 1, shares);
    QsCursor* place = reinterpret_cast<QsCursor*>(scratch + 20);
    if (tid == 0) scratch[16] = x0, scratch[17] = x1;
    __syncthreads();
#pragma unroll 1
    for (int e = 0; e < 2; ++e) {
        const int64_t x = e ? x1 : x0;
        if (x < before || x >= before + mine) continue;
        int64_t base = before;
        int n = n1 - 1;
        if (n > n0)
            for (n = n0;; ++n) {
                s = qs_seq(p, n);
                each = qs_weight<kN, kHg>(p, s, G);
                if (x < base + each) break;
                base += each;
            }
        int back;
        const QsCursor c = qs_cursor<kN, kHg>(s, n, x - base, G, back);
        scratch[16 + e] = x - back;
        if (e == 0) *place = c;
    }
    __syncthreads();
    if (x0 < total) {
        r.at = *place;
        r.weight = scratch[17] - scratch[16];
    }
    return r;
}

template <int kHg>
__device__ __forceinline__ void qs_next_tile(const QcacheAttnParams& p, int G, int rows, QsCursor& u) {
    u.j = 0;
    if (++u.tile < qs_tiles(u.s, G, rows)) return;
    u.tile = 0;
    if (++u.kh < p.Hk >> kHg) return;
    u.kh = 0;
    do {
        if (++u.n >= p.nseq) return;
        u.s = qs_seq(p, u.n);
    } while (u.s.lq == 0);
}

// A share's next piece: the slices [j0, j1) of one tile.
struct QsPiece {
    int j0, j1, nb, weight;
};
template <int kN, int kHg>
__device__ __forceinline__ QsPiece qs_piece(const QsCursor& u, int64_t left) {
    QsPiece r;
    r.nb = qs_slices(u.s);
    r.j0 = u.j;
    constexpr int piece = PIECE[kN] >> kHg;
    const int own = u.j == 0 ? piece : 0;
    r.j1 = left - own < r.nb - u.j ? u.j + (int)left - own : r.nb;
    r.weight = r.j1 - u.j + own;
    return r;
}

// Codes 2 e and 2 e + 1 (e: byte) of both halves of x, as bf16 numbers code 2^-133 and code 2^-129.
struct Codes {
    uint32_t y[4];
    __device__ __forceinline__ explicit Codes(uint32_t x) {
        const uint32_t z = x >> 8;
        y[0] = x & 0x000f000fu;
        y[1] = x & 0x00f000f0u;
        y[2] = z & 0x000f000fu;
        y[3] = z & 0x00f000f0u;
    }
};
__device__ __forceinline__ uint32_t transposed(uint32_t x) {   // of an 8 x 8 matrix of 16-bit numbers
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
// Row of a slice's 16 keys that row i of an operand stands for: neighbouring rows of 144 bytes lie four banks
// apart, these eight.  key_row(i + 8) = key_row(i) + 8, key_row(2 i + 1) = key_row(2 i) + 2.
__device__ __forceinline__ int key_row(int i) { return (i & 8) | (i & 3) << 1 | (i >> 2 & 1); }

// D = A B + C; without `volatile`, so that the compiler may order them (a C of zeros costs no registers).
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, float c0, float c1, float c2, float c3) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};\n"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    mma_bf16(d, a, b0, b1, d[0], d[1], d[2], d[3]);
}
// Both numbers of a pair times 2^n.
template <int n>
__device__ __forceinline__ uint32_t lifted(uint32_t x) {
    const __nv_bfloat162 f = __float2bfloat162_rn((float)(1ull << n));
    const __nv_bfloat162 y = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&x), f);
    return *reinterpret_cast<const uint32_t*>(&y);
}

// Where a row's 16-byte groups are kept among the warps' results: with rows 2 t and 2 t + 1 from lane (g, t), groups 2 g and
// 2 g + 1, bits 0 and 2 of the group's number spread the four t, bit 1 the neighbouring g.
__device__ __forceinline__ int row_swizzle(int row) { return (row >> 1 & 1) | (row & 4); }

constexpr int QS_STAGES = 2;
template <int kN>
struct QsLayout {
    static constexpr uint32_t ROWS = 8 * kN, WARPS = QS_WARPS[kN], THREADS = 32 * WARPS;
    static constexpr uint32_t OFF_SUMS = WARPS * QS_STAGES * SLICE_BYTES;          // [warps][rows][128] fp32
    static constexpr uint32_t OFF_ML = OFF_SUMS + WARPS * ROWS * 512;              // [piece & 1][warps][rows] float2
    static constexpr uint32_t OFF_BAR = OFF_ML + 2 * WARPS * ROWS * 8;
    static constexpr uint32_t OFF_SCRATCH = OFF_BAR + WARPS * QS_STAGES * 8;
    static constexpr uint32_t BYTES = OFF_SCRATCH + 32 * 8;
};

template <int kN, int kHg>
__global__ void __launch_bounds__(QsLayout<kN>::THREADS, kN == 1 ? 2 : 1) attn_qcache_kernel(const QcacheAttnParams p, const __grid_constant__ CUtensorMap map) {
    using L = QsLayout<kN>;
    constexpr int WARPS = L::WARPS;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    const uint32_t base = smem_u32(smem_raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = mx_uniform(tid >> 5), g = lane >> 2, t = lane & 3;
    const int G = p.Hq / p.Hk, rows = L::ROWS;
    asm volatile("griddepcontrol.launch_dependents;");
    // this warp's head of those that go together, and its slices of it
    constexpr int heads = (1 << kHg) - 1, step = WARPS >> kHg;
    const int mine = warp & heads, from = warp >> kHg;
    const uint32_t ring = base + warp * QS_STAGES * SLICE_BYTES, bars = base + L::OFF_BAR + warp * QS_STAGES * 8;
    if (lane == 0) {
        for (int i = 0; i < QS_STAGES; ++i) mbar_init(bars + 8 * i, 1);
        mbar_fence_init();
        tma_prefetch_desc(&map);
    }
    __syncwarp();
    await_stream();
    const QsShare share = p.nseq <= 32 ? qs_find_share_by_warp<kN, kHg>(p, G)
                                       : qs_find_share<kN, kHg>(p, G, reinterpret_cast<int64_t*>(smem_raw + L::OFF_SCRATCH));
    QsPartials part = qs_partials(p.workspace);
    QsCursor u = share.at;
    if (tid == 0) {
        QsCut c{};
        if (share.weight > 0) c = QsCut{u.j, 1, u.n, u.kh, u.tile, u.s.q0, u.s.lq, 0};
        c.status = share.bad ? KDA_DEVERR_CU_SEQLENS : 0u;
        part.cut[blockIdx.x] = c;
    }
    if (share.weight == 0) {   // (an empty share may lie between the parts of a tile)
        if (tid < kN * QS_MAX_ROWS) part.ml[(size_t)2 * blockIdx.x * kN * QS_MAX_ROWS + tid] = make_float2(-INFINITY, 0.f);
        return;
    }
    // the warp's slices: loads run QS_STAGES ahead within a piece, and the next piece's first ones are under way while
    // the warps put this one's results together
    uint32_t used = 0;
    auto load = [&](int kh, int n, int j, uint32_t count) {   // slice j, the count-th of this warp
#ifdef KDA_WAIT_TEST
        if (warp == 0 && count == 0 && (int)blockIdx.x == p.test_skip) return;
#endif
        if (lane == 0) {
            const uint32_t stage = count % QS_STAGES;
            mbar_arrive_expect_tx(bars + 8 * stage, SLICE_BYTES);
            tma_load_4d(ring + stage * SLICE_BYTES, &map, 0, kh, j * SLICE, n, bars + 8 * stage);
        }
    };
    auto load_first = [&](const QsCursor& v, const QsPiece& r) {
#pragma unroll
        for (int i = 0; i < QS_STAGES; ++i)
            if (r.j0 + from + i * step < r.j1) load((v.kh << kHg) + mine, v.n, r.j0 + from + i * step, used + i);
    };
    int64_t left = share.weight;
    QsPiece r{};
    if (left > 0) {
        r = qs_piece<kN, kHg>(u, left);
        load_first(u, r);
    }

    // what turns s into an exponent of base 2 (a scale of 0 must not turn a masked -inf into NaN, nor one past fp32 a score of 0)
    const float cq = fminf(fmaxf(p.scale * LOG2E / KEY_CODE, 1.2e-38f), 3e38f);
    // this lane's keys and its values' codes in a slice
    const unsigned char* krow = smem_raw + warp * QS_STAGES * SLICE_BYTES + key_row(g) * QC_ROW;
    const unsigned char* vrow = smem_raw + warp * QS_STAGES * SLICE_BYTES + key_row(2 * t) * QC_ROW + 64 + 4 * g;
    bool ok = true, first_piece = true, odd = false;
#pragma unroll 1
    while (left > 0) {
        const int kh = (u.kh << kHg) + mine;
        // ---- the tile's queries: lane (g, t) holds channels 16 t .. 16 t + 15 of both halves of row g
        uint32_t q[kN][8][2];            // pairs (e, e + 4) of each eight, the order in which the codes come
        uint32_t qz[kN];                 // sums over the halves' channels, each as three bf16 terms
        // the tile's first row is (token, head) (tok0, head0); row i is head (head0 + i) % G of (head0 + i) / G tokens on
        const int64_t total = (int64_t)u.s.lq * G, row0 = (int64_t)u.tile * rows;
        const int tok0 = (int)(row0 / G);
        const uint32_t head0 = (uint32_t)(row0 - (int64_t)tok0 * G);
        const int have = (int)min((int64_t)rows, total - row0);   // rows that are there
#pragma unroll
        for (int b = 0; b < kN; ++b) {
            const uint32_t on = (head0 + 8 * b + g) / (uint32_t)G, head = head0 + 8 * b + g - on * G;
            const __nv_bfloat16* src = p.q.data + ((int64_t)u.s.q0 + tok0 + on) * p.q.row + ((int64_t)kh * G + head) * p.q.head + 16 * t;
            float sum[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint4 x[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
                if (8 * b + g < have) {
                    x[0] = *reinterpret_cast<const uint4*>(src + 64 * h);
                    x[1] = *reinterpret_cast<const uint4*>(src + 64 * h + 8);
                }
                sum[h] = 0.f;
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    sum[h] += (bf16_lo(x[w].x) + bf16_hi(x[w].x)) + (bf16_lo(x[w].y) + bf16_hi(x[w].y)) +
                              ((bf16_lo(x[w].z) + bf16_hi(x[w].z)) + (bf16_lo(x[w].w) + bf16_hi(x[w].w)));
                    q[b][4 * h + 2 * w][0] = lifted<60>(lifted<4>(__byte_perm(x[w].x, x[w].z, 0x5410)));       // channels 0, 4
                    q[b][4 * h + 2 * w][1] = lifted<60>(__byte_perm(x[w].x, x[w].z, 0x7632));                  // 1, 5
                    q[b][4 * h + 2 * w + 1][0] = lifted<60>(lifted<4>(__byte_perm(x[w].y, x[w].w, 0x5410)));   // 2, 6
                    q[b][4 * h + 2 * w + 1][1] = lifted<60>(__byte_perm(x[w].y, x[w].w, 0x7632));              // 3, 7
                }
                sum[h] += __shfl_xor_sync(0xffffffffu, sum[h], 1);
                sum[h] += __shfl_xor_sync(0xffffffffu, sum[h], 2);
                sum[h] *= KEY_CODE;
            }
            qz[b] = 0;
#pragma unroll
            for (int i = 0; i < 3; ++i) {   // lane t takes the terms number t
                const uint32_t term = pack_bf16x2(sum[0], sum[1]);
                if (t == i) qz[b] = term;
                sum[0] -= bf16_lo(term);
                sum[1] -= bf16_hi(term);
            }
        }
        const int all_see = tok0 + u.s.lk - u.s.lq;   // the last key that the tile's first row sees

        float o[kN][2][4][4];            // [half][tile of channels]: channels 8 g + i and 8 g + 4 + i of the half, rows 2 t and 2 t + 1
        float ones[kN][2][4], z[kN][2][2], l[kN][2], low[kN][2];   // low: what the exponents refer to, less LIFT
#pragma unroll
        for (int b = 0; b < kN; ++b)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                low[b][i] = NO_KEY;
                l[b][i] = 0.f;
                z[b][0][i] = z[b][1][i] = 0.f;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    ones[b][i][e] = 0.f;
#pragma unroll
                    for (int f = 0; f < 4; ++f) o[b][i][f][e] = 0.f;
                }
            }
#pragma unroll 1
        for (int j = ok ? r.j0 + from : r.j1; j < r.j1; j += step) {
            const uint32_t stage = used % QS_STAGES;
            // (a warp whose wait ran out starts no more copies: their arrivals could meet a phase that is still open)
            if (!mx_wait(bars + 8 * stage, (used / QS_STAGES) & 1)) {
                ok = false;
                break;
            }
            const unsigned char* kat = krow + stage * SLICE_BYTES;
            const unsigned char* vat = vrow + stage * SLICE_BYTES;
            float s[kN][2][4];
            uint2 num[2][2];             // the values' numbers of rows g and g + 8 of each 16 keys
#pragma unroll
            for (int a = 0; a < 2; ++a) {
                uint2 w[2][2];           // [row g, g + 8][half]
                uint2 n[2];              // their scales and zeros
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const unsigned char* row = kat + (16 * a + 8 * i) * QC_ROW;
                    const uint4 x = *reinterpret_cast<const uint4*>(row + QC_NUMBERS);
                    n[i] = make_uint2(x.x, x.y);
                    num[a][i] = make_uint2(x.z, x.w);
                    w[i][0] = *reinterpret_cast<const uint2*>(row + 8 * t);
                    w[i][1] = *reinterpret_cast<const uint2*>(row + 8 * t + 32);
                }
                float acc[kN][2][4], zero[kN][4];
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int v = 0; v < 2; ++v) {
                        const uint32_t x0 = v ? w[0][h].y : w[0][h].x, x1 = v ? w[1][h].y : w[1][h].x;
                        const Codes c0(x0), c1(x1);
                        const uint32_t ya[4] = {c0.y[0], c1.y[0], c0.y[1], c1.y[1]}, yb[4] = {c0.y[2], c1.y[2], c0.y[3], c1.y[3]};
#pragma unroll
                        for (int b = 0; b < kN; ++b) {
                            if (v == 0) mma_bf16(acc[b][h], ya, q[b][4 * h][0], q[b][4 * h][1], 0.f, 0.f, 0.f, 0.f);
                            else mma_bf16(acc[b][h], ya, q[b][4 * h + 2][0], q[b][4 * h + 2][1]);
                            mma_bf16(acc[b][h], yb, q[b][4 * h + 2 * v + 1][0], q[b][4 * h + 2 * v + 1][1]);
                        }
                    }
                // the zeros of row g and g + 8, for each of the three terms of the channels' sums
                const uint32_t z[4] = {__byte_perm(n[0].x, n[0].y, 0x7632), __byte_perm(n[1].x, n[1].y, 0x7632), 0u, 0u};
#pragma unroll
                for (int b = 0; b < kN; ++b) {
                    mma_bf16(zero[b], z, qz[b], 0u, 0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            s[b][a][2 * i + e] = fmaf(bf16_lo(n[i].x), acc[b][0][2 * i + e], fmaf(bf16_lo(n[i].y), acc[b][1][2 * i + e], zero[b][2 * i + e]));
                }
            }
            if (SLICE * j + SLICE - 1 > all_see) {
#pragma unroll
                for (int b = 0; b < kN; ++b)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int last = min(tok0 + (int)((head0 + 8 * b + 2 * t + e) / (uint32_t)G), u.s.lq - 1) + u.s.lk - u.s.lq;
#pragma unroll
                        for (int a = 0; a < 2; ++a)
#pragma unroll
                            for (int i = 0; i < 2; ++i)
                                if (SLICE * j + 16 * a + key_row(g + 8 * i) > last) s[b][a][2 * i + e] = -INFINITY;
                    }
#pragma unroll
                for (int a = 0; a < 2; ++a)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int key = SLICE * j + 16 * a + key_row(g + 8 * i);
                        if (key >= u.s.lk) num[a][i] = make_uint2(0u, 0u);   // whatever such a row holds
                    }
            }
            // ---- the maximum, when a score has passed it by far
            bool grown = false;
            float top[kN][2];
#pragma unroll
            for (int b = 0; b < kN; ++b)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    top[b][e] = cq * fmaxf(fmaxf(s[b][0][e], s[b][0][2 + e]), fmaxf(s[b][1][e], s[b][1][2 + e]));
                    grown |= top[b][e] - low[b][e] > LIFT + 8.f;
                }
            if (__any_sync(0xffffffffu, grown)) {
#pragma unroll
                for (int b = 0; b < kN; ++b)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float x = top[b][e];
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
                        x = fmaxf(x - LIFT, low[b][e]);
                        const float f = ex2_approx(low[b][e] - x);
                        low[b][e] = x;
                        l[b][e] *= f;
                        z[b][0][e] *= f;
                        z[b][1][e] *= f;
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            ones[b][h][e] *= f;
                            ones[b][h][2 + e] *= f;
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                o[b][h][i][e] *= f;
                                o[b][h][i][2 + e] *= f;
                            }
                        }
                    }
            }
            // ---- weights, and the values
#pragma unroll
            for (int a = 0; a < 2; ++a) {
                uint32_t x[2][2][2];         // the words of keys 2 t and 2 t + 1 and of eight keys on: [half][i][key]
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int k = 0; k < 2; ++k) x[h][i][k] = *reinterpret_cast<const uint32_t*>(vat + (16 * a + 8 * i + 2 * k) * QC_ROW + 32 * h);
                uint32_t rw[kN][2][2];       // [half][keys 0-7, 8-15]: weights times scale, transposed
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float s0 = bf16_lo(num[a][i].x), s1 = bf16_lo(num[a][i].y);
                    const float m0 = fmaf(7.5f, s0, bf16_hi(num[a][i].x)), m1 = fmaf(7.5f, s1, bf16_hi(num[a][i].y));
#pragma unroll
                    for (int b = 0; b < kN; ++b) {
                        float w[2];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            w[e] = ex2_approx(__fsub_rn(__fmul_rn(cq, s[b][a][2 * i + e]), low[b][e]));   // (rounded as the maximum was: scores may be large)
                            l[b][e] += w[e];
                            z[b][0][e] = fmaf(w[e], m0, z[b][0][e]);
                            z[b][1][e] = fmaf(w[e], m1, z[b][1][e]);
                        }
                        rw[b][0][i] = transposed(pack_bf16x2(w[0] * s0, w[1] * s0));
                        rw[b][1][i] = transposed(pack_bf16x2(w[0] * s1, w[1] * s1));
                    }
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    // codes 0-3 and 4-7 of the two keys' words
                    const Codes l0(__byte_perm(x[h][0][0], x[h][0][1], 0x5410)), h0(__byte_perm(x[h][0][0], x[h][0][1], 0x7632));
                    const Codes l1(__byte_perm(x[h][1][0], x[h][1][1], 0x5410)), h1(__byte_perm(x[h][1][0], x[h][1][1], 0x7632));
                    const uint32_t one[4] = {0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u};
#pragma unroll
                    for (int b = 0; b < kN; ++b) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint32_t y[4] = {l0.y[i], h0.y[i], l1.y[i], h1.y[i]};
                            mma_bf16(o[b][h][i], y, rw[b][h][0], rw[b][h][1]);
                        }
                        mma_bf16(ones[b][h], one, rw[b][h][0], rw[b][h][1]);
                    }
                }
            }
            __syncwarp();
            if (j + QS_STAGES * step < r.j1) load(kh, u.n, j + QS_STAGES * step, used + QS_STAGES);
            ++used;
        }
        // ---- on to the next piece, whose loads start here
        const bool whole = r.j0 == 0 && r.j1 == r.nb;
        const int q0 = u.s.q0, kh0 = u.kh << kHg;
        left -= r.weight;
        if (left > 0) {
            qs_next_tile<kHg>(p, G, rows, u);
            r = qs_piece<kN, kHg>(u, left);
            if (ok) load_first(u, r);
        }
        // ---- the warps' results: reference and sum of every row, then the rows themselves
        // (two places for the references: a warp without a slice of the next piece writes its own there while others still read these;
        // the rows are written behind a barrier that those reach after)
        float2* ml = reinterpret_cast<float2*>(smem_raw + L::OFF_ML) + (odd ? WARPS * rows : 0);
        odd = !odd;
        float* sums = reinterpret_cast<float*>(smem_raw + L::OFF_SUMS);
#pragma unroll
        for (int b = 0; b < kN; ++b)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) {
                    l[b][e] += __shfl_xor_sync(0xffffffffu, l[b][e], d);
                    z[b][0][e] += __shfl_xor_sync(0xffffffffu, z[b][0][e], d);
                    z[b][1][e] += __shfl_xor_sync(0xffffffffu, z[b][1][e], d);
                }
                if (g == 0) ml[warp * rows + 8 * b + 2 * t + e] = make_float2(l[b][e] == 0.f ? -INFINITY : low[b][e] + LIFT, UNLIFT * l[b][e]);
            }
        __syncthreads();
#pragma unroll
        for (int b = 0; b < kN; ++b)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int row = 8 * b + 2 * t + e;
                float top = -INFINITY;
#pragma unroll
                for (int w = 0; w < step; ++w) top = fmaxf(top, ml[((w << kHg) + mine) * rows + row].x);   // (this head's warps)
                const float f = l[b][e] == 0.f ? 0.f : ex2_approx(low[b][e] + LIFT - top);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float y[8];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {   // (codes 1 and 3 were four places higher)
                        const float back = i & 1 ? CODE / 16.f : CODE, rest = UNLIFT * fmaf(-7.5f, ones[b][h][e], z[b][h][e]);
                        y[i] = f * fmaf(back, o[b][h][i][e], rest);
                        y[4 + i] = f * fmaf(back, o[b][h][i][2 + e], rest);
                    }
                    // (eight lanes that store together store to different banks: see row_swizzle)
                    float4* dst = reinterpret_cast<float4*>(sums + (warp * rows + row) * 128);
                    dst[(16 * h + 2 * g) ^ row_swizzle(row)] = make_float4(y[0], y[1], y[2], y[3]);
                    dst[(16 * h + 2 * g + 1) ^ row_swizzle(row)] = make_float4(y[4], y[5], y[6], y[7]);
                }
            }
        __syncthreads();
        const size_t slot = (size_t)(2 * blockIdx.x + (first_piece ? 0 : 1)) * kN * QS_MAX_ROWS;
#pragma unroll 1
        for (int i = warp; i < rows << kHg; i += WARPS) {   // a warp takes a row of a head, a lane four channels
            const int hh = i & heads, row = i >> kHg;
            if (row >= have) break;
            float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
            float top = -INFINITY, sum = 0.f;
#pragma unroll
            for (int w = 0; w < step; ++w) {
                const float4 x = reinterpret_cast<const float4*>(sums + (((w << kHg) + hh) * rows + row) * 128)[lane ^ row_swizzle(row)];
                y.x += x.x, y.y += x.y, y.z += x.z, y.w += x.w;
                top = fmaxf(top, ml[((w << kHg) + hh) * rows + row].x);
            }
#pragma unroll
            for (int w = 0; w < step; ++w) {
                const float2 x = ml[((w << kHg) + hh) * rows + row];
                sum += x.x == -INFINITY ? 0.f : x.y * ex2_approx(x.x - top);
            }
            if (!whole) {
                *reinterpret_cast<float4*>(part.o + (slot + i) * 128 + 4 * lane) = y;
                if (lane == 0) part.ml[slot + i] = make_float2(top, sum);
            } else {
                const uint32_t on = (head0 + row) / (uint32_t)G;
                const int64_t tok = (int64_t)q0 + tok0 + on, head = (int64_t)(kh0 + hh) * G + (head0 + row - on * G);
                const float inv = sum == 0.f ? 0.f : 1.f / sum;
                *reinterpret_cast<uint2*>(p.out.data + tok * p.out.row + head * p.out.head + 4 * lane) =
                    make_uint2(pack_bf16x2(y.x * inv, y.y * inv), pack_bf16x2(y.z * inv, y.w * inv));
                if (p.lse && lane == 0) p.lse[tok * p.Hq + head] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
            }
        }
        first_piece = false;
    }
    if (!ok) {
        mx_wind_down();
        if (lane == 0) atomicOr(&part.cut[blockIdx.x].status, KDA_DEVERR_TIMEOUT);
    }
}

// Joins the partial rows of the tiles that several shares hold (and, the last block, the shares' status bits: one
// store, so that none is lost).  Block (b, y) takes eight rows of the tile that share b + 1 starts in, if that is the tile's first
// cut; a warp takes a row of a head, lane l its channels 4 l .. 4 l + 3.  Bound by latency: what it needs of the shares is asked for
// at once, then kParts parts at once, and blocks are few and small (one for each row: 2 to 7 us more; one for a tile's 32 rows:
// 24 x 4 drafts 2.3 us more; 16 warps, two for a row, with eight parts each: 1.3 us more for one token; 32: 4 us).
constexpr int QJ_WARPS = 8;
template <int kParts>
__global__ void __launch_bounds__(32 * QJ_WARPS, 2) attn_qcache_join_kernel(const QcacheAttnParams p, int ctas, int rows, int hg) {
    const int first = blockIdx.x + 1, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, G = p.Hq / p.Hk;
    const QsPartials part = qs_partials(p.workspace);
    await_stream();
    if (first == ctas) {
        if (warp != 0 || blockIdx.y != 0) return;
        uint32_t status = 0;
        for (int s = lane; s < ctas; s += 32) status |= part.cut[s].status;
        status = __reduce_or_sync(0xffffffffu, status);
        if (lane == 0) *p.status = status;
        return;
    }
    const QsCut c = part.cut[first];
    QsCut before = part.cut[max(first - 1 - lane, 0)], e = part.cut[min(first + 1 + lane, ctas - 1)];
    if (c.j == 0) return;   // between two tiles, or nothing to do
    auto inside = [&](const QsCut& a) { return a.n == c.n && a.kh == c.kh && a.tile == c.tile; };
    // the share before it that is not empty: it holds the tile's part before this one
    int b = first - 1;
    bool same = false;
    for (;;) {
        const uint32_t some = __ballot_sync(0xffffffffu, b - lane >= 0 && before.some);
        if (some) {
            const int d = __ffs(some) - 1;
            b -= d;
            same = __shfl_sync(0xffffffffu, (int)inside(before), d);
            if (same && __shfl_sync(0xffffffffu, before.j, d) > 0) return;   // an earlier cut's
            break;
        }
        b -= 32;
        if (b < 0) return;   // (there is one)
        before = part.cut[max(b - lane, 0)];
    }
    // the parts: share b's last piece, then the first pieces of the shares that start inside the tile (empty ones between, which
    // have left sums of zero)
    int end = first + 1;
    for (int base = first + 1;; base += 32) {
        const bool part_of = base + lane < ctas && e.some && e.j > 0 && inside(e);
        const uint32_t past = __ballot_sync(0xffffffffu, base + lane >= ctas || (e.some && !part_of));
        const uint32_t parts = __ballot_sync(0xffffffffu, part_of) & (past ? (past & -past) - 1u : 0xffffffffu);
        if (parts) end = base + 32 - __clz(parts);
        if (past) break;
        e = part.cut[min(base + 32 + lane, ctas - 1)];
    }
    const int count = 1 + end - first;
    const int i = QJ_WARPS * blockIdx.y + warp, row = i >> hg;
    const int64_t at = (int64_t)c.tile * rows + row;
    if (at >= (int64_t)c.lq * G) return;
    auto slot = [&](int k) {
        return (size_t)(k == 0 ? 2 * b + (same ? 0 : 1) : 2 * (first + k - 1)) * (rows / 8) * QS_MAX_ROWS + i;
    };
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int k0 = 0; k0 < count; k0 += kParts) {
        float2 ml[kParts];
        float4 y[kParts];
#pragma unroll
        for (int d = 0; d < kParts; ++d) {
            const int k = k0 + d;
            ml[d] = make_float2(-INFINITY, 0.f);
            if (k < count) {
                ml[d] = __ldcg(part.ml + slot(k));
                y[d] = __ldcg(reinterpret_cast<const float4*>(part.o + slot(k) * 128 + 4 * lane));
            }
        }
        float top = m;
#pragma unroll
        for (int d = 0; d < kParts; ++d) top = fmaxf(top, ml[d].x);
        const float old = m == -INFINITY ? 0.f : ex2_approx(m - top);
        m = top;
        l *= old;
        o.x *= old, o.y *= old, o.z *= old, o.w *= old;
#pragma unroll
        for (int d = 0; d < kParts; ++d) {
            if (ml[d].x == -INFINITY) continue;   // a part that saw no key, or an empty share
            const float w = ex2_approx(ml[d].x - m);
            l = fmaf(w, ml[d].y, l);
            o.x = fmaf(w, y[d].x, o.x);
            o.y = fmaf(w, y[d].y, o.y);
            o.z = fmaf(w, y[d].z, o.z);
            o.w = fmaf(w, y[d].w, o.w);
        }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const int64_t tok = c.q0 + at / G, head = (int64_t)((c.kh << hg) + (i & ((1 << hg) - 1))) * G + at % G;
    *reinterpret_cast<uint2*>(p.out.data + tok * p.out.row + head * p.out.head + 4 * lane) =
        make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
    if (p.lse && lane == 0) p.lse[tok * p.Hq + head] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

// The cache in boxes of 144 bytes x 1 head x `rows` rows.
bool encode_cache(CUtensorMap* m, const QcacheAttnParams& p, int rows) {
    MxEncodeFn fn = mx_encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[4] = {(cuuint64_t)QC_ROW, (cuuint64_t)p.Hk, (cuuint64_t)(p.S > 0 ? p.S : 1), (cuuint64_t)(p.nseq > 0 ? p.nseq : 1)};
    const cuuint64_t strides[3] = {(cuuint64_t)p.cache.head, (cuuint64_t)p.cache.row, (cuuint64_t)(p.cache.seq > 0 ? p.cache.seq : QC_ROW)};
    const cuuint32_t box[4] = {(cuuint32_t)QC_ROW, 1, (cuuint32_t)rows, 1}, estr[4] = {1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, p.cache.data, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
              CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int kN, int kHg>
cudaError_t launch(const QcacheAttnParams& p, int sms, cudaStream_t stream) {
    CUtensorMap map;
    if (!encode_cache(&map, p, SLICE)) return cudaErrorInvalidValue;
    const int ctas = min(sms * (kN == 1 ? 2 : 1), QS_MAX_CTAS / kN);
    cudaError_t e = cudaFuncSetAttribute(attn_qcache_kernel<kN, kHg>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)QsLayout<kN>::BYTES);
    if (e == cudaSuccess) e = launch_early(attn_qcache_kernel<kN, kHg>, dim3((unsigned)ctas), QsLayout<kN>::THREADS, QsLayout<kN>::BYTES, stream, p, map);
    // parts asked for at once: 16 where there are few units (one token over 32,767: 19.1 us; four 21, 20 20.7), else four
    // (16 tokens over 5,002 to 32,767, rows order, 82.7 us; eight 83.6)
    const bool many = ctas > 4 * (int64_t)p.nseq * (p.Hk >> kHg);
    if (e == cudaSuccess)
        e = launch_early(many ? attn_qcache_join_kernel<16> : attn_qcache_join_kernel<4>, dim3((unsigned)ctas, (8 * kN << kHg) / QJ_WARPS), 32 * QJ_WARPS, 0, stream, p, ctas, 8 * kN, kHg);
    return e;
}

// ---------------------------------------------------------------- many rows: expanded once, then the tensor cores
// Many rows read a block of keys many times (a pair of query tiles each), so the codes are expanded once, for some key
// heads at a time, into the workspace, and the kernel of kda_attn.cu runs on that.
//   keys     y = scale (code - 8) in fp16, which is exact (8 bits times 4 with a sign, of which 8 is a power of two), and
//            zero + 8 scale, constant over 64 channels: what it adds to a score is (zero + 8 scale) sum q, the sum in three terms
//            of fp16, so 12 more channels hold zero and 8 scale of both halves against them.  (Keys rounded
//            once to bf16 move the results by 0.0034 of their norm and lse by 1e-4.)
//   values   in fp16, as are the weights that meet them (11 bits instead of 8: both roundings vanish beside the output's)
//   queries  in fp16, which holds bf16's eight bits
// all scaled by powers of two: a block of 128 keys and one of values each, so that its largest is below 2^(SPLIT_KEY + 1) and
// 2^(SPLIT_TOP + 1), a query to below 2^9, so that 64 of them are below 2^15.  Where the keys of a block have values of very
// different size, each has its own power.  fp16 holds all bits down to 2^-27 of the largest (queries: 2^-22) and is off by 2^-38 (2^-33)
// of it below: keys and queries lose by that what only products of 2^20 and more would show, a key's values what is that
// small beside its own largest channel (or 2^-SPLIT_SPREAD of that).
// A CTA takes a block of keys of a head: half a warp a row, a lane eight channels of the key and of the value; or 64 rows of
// queries.  Bound by HBM (144 bytes read and 544 written, 545 at most, for each key and head).  Prompts of 1,024, 517 and 33 behind 16,384,
// 8,484 and 15,967, 64 heads on 8: 580 us; 700 with the keys as two terms of bf16, both multiplied with the queries (three products a
// block instead of two and an eighth, and 768 bytes), 1,328 with codes expanded in the other kernel by four more warps.
constexpr int EX_THREADS = 256, EX_BLOCK = 128, EX_ROWS = EX_BLOCK * 16 / EX_THREADS;   // rows of a thread
constexpr int EX_QUERIES = 4;   // its rows of queries
constexpr int QUERY_TOP = 8, QUERY_LEAST = 35;

struct ExpandParams {
    QcacheView cache;
    const int64_t* seqlens_k;
    int64_t S;
    int seq0, head0, heads, blocks; // blocks of a sequence
    __half *k, *v;                  // [sequences][heads][blocks * 128][128]
    __half* k_rest;                 // [sequences][heads][blocks][2][128][8]
    int* top;                       // [sequences][heads][blocks]
    uint8_t* value_power;           // [sequences][heads][blocks][128], of the blocks that have them
    RowsView q;
    int64_t query_rows, query_blocks;   // tokens times query heads of these key heads
    int query_heads;
    __half *q_to, *q_rest;          // [tokens][query_heads][128 and 16]
    int* q_power;
};

__device__ __forceinline__ uint32_t half2_of(float lo, float hi) {
    const __half2 y = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&y);
}
__device__ __forceinline__ float half_round(float x) { return __half2float(__float2half_rn(x)); }

__device__ __forceinline__ void expand_queries(const ExpandParams& p, int64_t block) {
    const int lane = threadIdx.x & 15;
    const int64_t row0 = block * (EX_QUERIES * EX_THREADS / 16) + (threadIdx.x >> 4);
    uint4 x[EX_QUERIES];
#pragma unroll
    for (int i = 0; i < EX_QUERIES; ++i) {
        const int64_t row = row0 + i * (EX_THREADS / 16), t = row / p.query_heads;
        x[i] = make_uint4(0, 0, 0, 0);
        if (row < p.query_rows) x[i] = *reinterpret_cast<const uint4*>(p.q.data + t * p.q.row + (row - t * p.query_heads) * p.q.head + 8 * lane);
    }
#pragma unroll
    for (int i = 0; i < EX_QUERIES; ++i) {
        const int64_t row = row0 + i * (EX_THREADS / 16);
        const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
        uint32_t big = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) big = max(big, max(w[e] & 0x7fffu, w[e] >> 16 & 0x7fffu));   // (bf16's order is that of its bits)
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) big = max(big, __shfl_xor_sync(0xffffffffu, big, o));
        const int top = max((int)(big >> 7), QUERY_LEAST);
        const float lift = __uint_as_float((uint32_t)(127 + QUERY_TOP + 127 - top) << 23);
        uint32_t y[4];
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float a = lift * bf16_lo(w[e]), b = lift * bf16_hi(w[e]);
            y[e] = half2_of(a, b);
            sum += a + b;
        }
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        const float other = __shfl_xor_sync(0xffffffffu, sum, 8);   // lanes 0 .. 7 and 8 .. 15: a half each
        if (row >= p.query_rows) continue;
        *reinterpret_cast<uint4*>(p.q_to + row * HD + 8 * lane) = make_uint4(y[0], y[1], y[2], y[3]);
        if (lane == 0) {
            const float a1 = half_round(sum), a2 = half_round(sum - a1), a3 = sum - a1 - a2;
            const float b1 = half_round(other), b2 = half_round(other - b1), b3 = other - b1 - b2;
            uint4* rest = reinterpret_cast<uint4*>(p.q_rest + row * SPLIT_REST);
            rest[0] = make_uint4(half2_of(a1, a2), half2_of(a3, a1), half2_of(a2, a3), half2_of(b1, b2));
            rest[1] = make_uint4(half2_of(b3, b1), half2_of(b2, b3), 0, 0);
            p.q_power[row] = top - 127 - QUERY_TOP;
        }
    }
}

__device__ __forceinline__ float code_at(uint32_t x, int bit) { return __uint_as_float((x >> bit & 15u) | 0x4b000000u) - 8388608.f; }

__global__ void __launch_bounds__(EX_THREADS, 4) qcache_expand_kernel(const ExpandParams p) {
    __shared__ uint3 most[EX_THREADS / 32];
    await_stream();
    const int block = blockIdx.x, h = blockIdx.y, n = blockIdx.z;
    if (block >= p.blocks) {
        const int64_t b = ((int64_t)(block - p.blocks) * gridDim.z + n) * gridDim.y + h;
        if (b < p.query_blocks) expand_queries(p, b);
        return;
    }
    const int64_t lk = min(max(p.seqlens_k[p.seq0 + n], (int64_t)0), p.S);
    if (block > 0 && (int64_t)block * EX_BLOCK >= lk) return;   // (block 0 is read even if there are no keys)
    const int lane = threadIdx.x & 15, row0 = threadIdx.x >> 4;
    const uint8_t* src = p.cache.data + (int64_t)(p.seq0 + n) * p.cache.seq + (int64_t)(p.head0 + h) * p.cache.head;
    uint32_t kc[EX_ROWS], vc[EX_ROWS], kn[EX_ROWS], vn[EX_ROWS];   // codes; scale and zero of this lane's half
#pragma unroll
    for (int i = 0; i < EX_ROWS; ++i) {
        const int64_t key = (int64_t)block * EX_BLOCK + row0 + i * (EX_THREADS / 16);
        kc[i] = vc[i] = kn[i] = vn[i] = 0;
        if (key < lk) {
            const uint8_t* at = src + key * p.cache.row;
            kc[i] = __ldcs(reinterpret_cast<const uint32_t*>(at) + lane);
            vc[i] = __ldcs(reinterpret_cast<const uint32_t*>(at + 64) + lane);
            kn[i] = *reinterpret_cast<const uint32_t*>(at + QC_NUMBERS + (lane >> 3) * 4);
            vn[i] = *reinterpret_cast<const uint32_t*>(at + QC_NUMBERS + (lane >> 3) * 4 + 8);
        }
    }
    auto largest = [](float most, uint32_t w) { return fmaxf(most, fmaxf(fabsf(bf16_hi(w)), fabsf(fmaf(15.f, bf16_lo(w), bf16_hi(w))))); };
    // the largest of a row's values, which lie in both halves of its lanes
    auto row_value = [&](uint32_t w) {
        const float x = largest(0.f, w);
        return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
    };
    float big_k = 0.f, big_v = 0.f, least_v = INFINITY;   // (a row of zeros has no size)
#pragma unroll
    for (int i = 0; i < EX_ROWS; ++i) {
        big_k = largest(big_k, kn[i]);
        const float v = row_value(vn[i]);
        big_v = fmaxf(big_v, v);
        if (v > 0.f) least_v = fminf(least_v, v);
    }
    uint32_t all_k = __reduce_max_sync(0xffffffffu, __float_as_uint(big_k)), all_v = __reduce_max_sync(0xffffffffu, __float_as_uint(big_v));
    uint32_t all_least = __reduce_min_sync(0xffffffffu, __float_as_uint(least_v));
    if ((threadIdx.x & 31) == 0) most[threadIdx.x >> 5] = make_uint3(all_k, all_v, all_least);
    __syncthreads();
#pragma unroll
    for (int w = 0; w < EX_THREADS / 32; ++w) all_k = max(all_k, most[w].x), all_v = max(all_v, most[w].y), all_least = min(all_least, most[w].z);
    const int top_k = max((int)(all_k >> 23), SPLIT_KEY_LEAST), top_v = max((int)(all_v >> 23), SPLIT_LEAST);
    const bool each = top_v - max((int)(all_least >> 23), SPLIT_LEAST) > SPLIT_SPREAD;
    const int64_t unit = ((int64_t)n * p.heads + h) * p.blocks + block;
    if (threadIdx.x == 0) p.top[unit] = top_k << 16 | (each ? SPLIT_EACH : 0) | top_v;
    const float lift_k = __uint_as_float((uint32_t)(127 + SPLIT_KEY + 127 - top_k) << 23);
    const float lift_block = __uint_as_float((uint32_t)(127 + SPLIT_TOP + 127 - top_v) << 23);
#pragma unroll
    for (int i = 0; i < EX_ROWS; ++i) {
        const int row = row0 + i * (EX_THREADS / 16);
        const int64_t at = (unit * EX_BLOCK + row) * HD + 8 * lane;
        float lift_v = lift_block;
        if (each) {
            const int top = max((int)(__float_as_uint(row_value(vn[i])) >> 23), SPLIT_LEAST);
            lift_v = __uint_as_float((uint32_t)(127 + SPLIT_TOP + 127 - top) << 23);
            if (lane == 0) p.value_power[unit * EX_BLOCK + row] = (uint8_t)top;
        }
        const float ks = lift_k * bf16_lo(kn[i]), k8 = -8.f * ks, vs = lift_v * bf16_lo(vn[i]), vz = lift_v * bf16_hi(vn[i]);
        uint32_t k[4], v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            k[e] = half2_of(fmaf(code_at(kc[i], 8 * e), ks, k8), fmaf(code_at(kc[i], 8 * e + 4), ks, k8));
            v[e] = half2_of(fmaf(code_at(vc[i], 8 * e), vs, vz), fmaf(code_at(vc[i], 8 * e + 4), vs, vz));
        }
        *reinterpret_cast<uint4*>(p.k + at) = make_uint4(k[0], k[1], k[2], k[3]);
        *reinterpret_cast<uint4*>(p.v + at) = make_uint4(v[0], v[1], v[2], v[3]);
        const uint32_t other = __shfl_xor_sync(0xffffffffu, kn[i], 8);
        if (lane < 2) {   // the channels against a query's sums: zero three times, 8 scale three times, for both halves
            const float s0 = -k8, z0 = lift_k * bf16_hi(kn[i]), s1 = 8.f * lift_k * bf16_lo(other), z1 = lift_k * bf16_hi(other);
            const uint4 first = make_uint4(half2_of(z0, z0), half2_of(z0, s0), half2_of(s0, s0), half2_of(z1, z1));
            const uint4 second = make_uint4(half2_of(z1, s1), half2_of(s1, s1), 0, 0);
            *reinterpret_cast<uint4*>(p.k_rest + ((unit * 2 + lane) * EX_BLOCK + row) * 8) = lane ? second : first;
        }
    }
}

}  // namespace

// Few rows: this file's kernel; many: that of kda_attn.cu on expanded keys and values.  With 64 rows for a key head and with 128,
// few and many: 24 sequences over 71 to 8,098 131 and 205, 245 and 210 us; four over 16,000 86 and 137, 155 and 139; one over
// 32,767 49 and 84, 85 and 86: they meet between 104 and 128 rows.  Where there is room for few keys only, three launches and the
// expansion cost more than they bring (100 queries over up to 1,000 keys, 8 heads on one, 13 and 32 us; 128 over up to 512, 32 heads
// on 8, 18 and 23; but 300 over up to 300 30 and 23, and four times 100 over up to 400 40 and 29).
static bool few_rows(int64_t Tq, int Hq, int Hk, int nseq, int64_t S) {
    return Tq * (Hq / Hk) <= 112 * (int64_t)nseq || (double)Tq * Hq * S <= 1 << 21;
}

// Expanded keys and values: of all sequences, for as many key heads at a time as fit into 1 GB, one at least.  Where one
// head of all sequences would pass 4 GB (the room counts, whether used or not), some sequences at a time, with as many heads
// as fit into 4 GB: a turn costs three launches, however little there is in it, so turns are not made smaller before that.
constexpr int64_t EX_MOST = 1LL << 30, EX_HEAD_MOST = 1LL << 32;
constexpr int64_t EX_QUERY_BYTES = (HD + SPLIT_REST) * 2 + 4;   // of an expanded query
struct Expanded {
    int64_t blocks, unit;   // of a sequence; bytes of one (sequence, head)
    int heads, seqs;        // at a time
};
static Expanded expanded(int64_t S, int Hk, int nseq) {
    Expanded x;
    x.blocks = S > 0 ? (S + EX_BLOCK - 1) / EX_BLOCK : 1;
    x.unit = x.blocks * (EX_BLOCK * (2 * HD + SPLIT_REST) * 2 + EX_BLOCK + 16);   // (keys' powers, a byte each; 16: a block's, with what keeps the arrays aligned)
    auto within = [](int64_t n, int64_t most) { return (int)(n < 1 ? 1 : n < most ? n : most); };
    const int all = nseq > 0 ? nseq : 1;
    const int64_t units = EX_HEAD_MOST / x.unit;
    x.heads = within(units >= all ? EX_MOST / x.unit / all : units, Hk);
    x.seqs = within(units / x.heads, all);
    return x;
}

size_t attn_qcache_workspace_bytes(int64_t Tq, int Hq, int Hk, int nseq, int64_t S) {
    if (few_rows(Tq, Hq, Hk, nseq, S)) return QS_CUT_BYTES + QS_ML_BYTES + (size_t)2 * QS_MAX_CTAS * QS_MAX_ROWS * HD * sizeof(float);   // (16 rows a tile: half as many CTAs)
    const Expanded x = expanded(S, Hk, nseq);
    const int64_t query_rows = Tq * (Hq / Hk) * x.heads;
    return attn_workspace_bytes(Tq, Hq, Hk) + 256 + (size_t)(x.unit * x.seqs * x.heads + query_rows * EX_QUERY_BYTES);
}

static cudaError_t launch_many_rows(const QcacheAttnParams& p, cudaStream_t stream) {
    const Expanded x = expanded(p.S, p.Hk, p.nseq);
    const int G = p.Hq / p.Hk;
    char* ex = static_cast<char*>(p.workspace) + attn_workspace_bytes(p.Tq, p.Hq, p.Hk);
    ex += -(uintptr_t)ex & 255;
    const int64_t rows = x.blocks * EX_BLOCK, units = (int64_t)x.seqs * x.heads;
    for (int h0 = 0, n0 = 0; h0 < p.Hk;) {
        const int heads = min(x.heads, p.Hk - h0), seqs = min(x.seqs, p.nseq - n0);
        ExpandParams e;
        memset(&e, 0, sizeof(e));
        e.cache = p.cache;
        e.seqlens_k = p.seqlens_k;
        e.S = p.S;
        e.seq0 = n0;
        e.head0 = h0;
        e.heads = heads;
        e.blocks = (int)x.blocks;
        e.k = reinterpret_cast<__half*>(ex);
        e.v = e.k + units * rows * HD;
        e.k_rest = e.v + units * rows * HD;
        e.q = p.q;
        e.q.data += (int64_t)h0 * G * p.q.head;
        e.query_heads = heads * G;
        e.query_rows = p.Tq * e.query_heads;
        if (n0 == 0) e.query_blocks = (e.query_rows + EX_QUERIES * EX_THREADS / 16 - 1) / (EX_QUERIES * EX_THREADS / 16);
        e.value_power = reinterpret_cast<uint8_t*>(e.k_rest + units * rows * SPLIT_REST);
        e.q_to = reinterpret_cast<__half*>(e.value_power + units * rows);
        e.q_rest = e.q_to + e.query_rows * HD;
        e.q_power = reinterpret_cast<int*>(e.q_rest + e.query_rows * SPLIT_REST);
        e.top = e.q_power + e.query_rows;
        if (seqs > 0) {
            const int64_t more = (e.query_blocks + (int64_t)heads * seqs - 1) / ((int64_t)heads * seqs);
            const cudaError_t err = launch_early(qcache_expand_kernel, dim3((unsigned)(x.blocks + more), (unsigned)heads, (unsigned)seqs), EX_THREADS, 0, stream, e);
            if (err != cudaSuccess) return err;
        }
        AttnParams a;
        memset(&a, 0, sizeof(a));
        a.q = RowsView{reinterpret_cast<__nv_bfloat16*>(e.q_to), (int64_t)HD * e.query_heads, HD};
        a.out = p.out;
        a.out.data += (int64_t)h0 * G * p.out.head;
        a.k = reinterpret_cast<__nv_bfloat16*>(e.k);
        a.v = reinterpret_cast<__nv_bfloat16*>(e.v);
        a.q_rest = e.q_rest;
        a.k_rest = e.k_rest;
        a.q_power = e.q_power;
        a.top = e.top;
        a.value_power = e.value_power;
        a.top_blocks = x.blocks;
        a.seq0 = n0;
        a.seqs = seqs;
        a.k_row = a.v_row = HD;
        a.k_head = a.v_head = rows * HD;
        a.k_seq = a.v_seq = rows * HD * heads;
        a.lse = p.lse ? p.lse + h0 * G : nullptr;
        a.lse_row = p.Hq;
        a.cu_q = p.cu_q;
        a.seqlens_k = p.seqlens_k;
        a.uniform_q = p.uniform_q;
        a.Tq = p.Tq;
        a.Tk = rows;
        a.keys = p.S;
        a.keep_status = h0 > 0 || n0 > 0;
        a.nseq = p.nseq;
        a.Hq = heads * G;
        a.Hk = heads;
        a.cache = 1;
        a.scale = p.scale;
        a.status = p.status;
        a.workspace = p.workspace;
        a.test_skip = h0 == 0 && n0 == 0 ? p.test_skip : -1;
        const cudaError_t err = launch_attn_split(a, stream);
        if (err != cudaSuccess) return err;
        n0 += x.seqs;
        if (n0 >= p.nseq) n0 = 0, h0 += x.heads;
    }
    return cudaSuccess;
}

cudaError_t launch_attn_qcache(const QcacheAttnParams& p, cudaStream_t stream) {
    if (!few_rows(p.Tq, p.Hq, p.Hk, p.nseq, p.S)) return launch_many_rows(p, stream);
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    const bool single = p.Tq * (p.Hq / p.Hk) <= 8 * (int64_t)p.nseq;
    // Two key heads together where the heads lie inside the rows (their bytes come with one another: 16 single tokens over up to
    // 32,767, 102 -> 89 us) or a tile has 16 rows (half as many pieces: 24 x 4 drafts 47 -> 44 us), once there are enough
    // (sequence, head) units that cutting them does not cost more (one token over 32,767: 23 -> 27 us; 8 over up to
    // 16,000 28 -> 33; 128 units even)
    if ((p.cache.head < p.cache.row || !single) && p.Hk % 2 == 0 && (int64_t)p.nseq * p.Hk >= 128)
        return single ? launch<1, 1>(p, sms, stream) : launch<2, 1>(p, sms, stream);
    return single ? launch<1, 0>(p, sms, stream) : launch<2, 0>(p, sms, stream);
}

}  // namespace kda
