// paged_attn.cu -- causal attention of new tokens over a paged cache.
//
// One pass over the keys with the running maximum and sum of the softmax:
// with x_j = scale log2(e) q . k_j, m a reference near the largest x so far,
// l = sum 2^(x_j - m) and o = sum 2^(x_j - m) v_j; a larger m rescales l and
// o by 2^(m_old - m).  The reference follows the maximum only when that has
// grown by more than kSlack, so o (in tensor memory) is seldom touched; the
// largest weight then lies between 2^kShift = 2^8 and 2^(kShift + kSlack) =
// 2^14, inside fp16, and all keep full precision down to 2^-22 of the largest
// and are lost from 2^-33 of it on.  Weights of 16 bits because the tensor
// cores want both operands of one kind, and V is fp16: TF32 would double V's
// and P's room and halve the rate of half the products.  What it costs is
// 2^-11 of a weight, and in the mean over keys less than the result's own
// rounding to fp16 (2.3-2.9e-4 of the outputs' norm in all, against 2.0-2.1e-4
// with weights of 32 bits).
//
// Both products run on the tensor cores with M = 128 rows.  The rows of a
// tile are (token, query head) pairs that read the same key/value head:
// tok = 128 / group tokens by group heads, so a verify block of K + 1
// positions uses the rows that a single token would leave empty, and its
// keys are read once.  Per 128 keys: S = Q K^T (Q and K from shared memory,
// both K-major as TMA lays the pages down), softmax in registers, the
// weights back into S's tensor-memory columns as fp16, O += P V (P from
// tensor memory, V from shared memory, N along the rows of 64 elements).
//
// Pages: a TMA box is one page (at most 128 tokens) of one head, laid down
// as 8-token groups of [64-element block][8 tokens][128 bytes] with the
// 128-byte swizzle.  Groups of different pages are then the same distance
// apart as groups of one page, so a tile gathered from up to 16 pages is one
// operand of one descriptor, K-major for K and N-major for V.
//
// Work: the unit is one tile's 128 keys; a row tile counts kPartCost more for
// what it costs beside its keys (its epilogue, its first scores).  All units
// in order (sequence, key/value head, row tile, keys) are dealt out evenly to
// one CTA per SM, so a long context at one row tile and a causal triangle of
// many both fill the GPU.  A CTA's range may begin and end inside a tile; such
// a part leaves o, m and l in the workspace (at most two parts a CTA), and a
// second kernel joins them, each boundary's CTAs a share of the tile's rows.
// The lengths are on the device, so each CTA finds its own range by a scan
// over the sequences.  With batch invariance the unit is a fixed range of
// keys, every one a part of its own: which keys meet in one running sum then
// depends on the row alone.
//
// A weight of 0 does not hide a value that is not finite (0 x inf is NaN),
// and within a tile some rows see keys that others must not.  Where a tile
// holds such keys, a warp looks their values over before the product and
// clears what is not finite; the rows that do see it add it in the epilogue.
// A drafted token that overflowed thus spoils no position before it.
//
// Roles (12 warps): 0 producer (the CTA's parts, which it hands on through a
// ring in shared memory, page ids, TMA), 1 issuer of Q K^T, 2 issuer of P V,
// 3 guard (the looking over, a tile ahead of the issuer) and tensor-memory
// owner, 4-7 and 8-11 softmax.  S and P have buffers of their own, so Q K^T
// runs ahead (two tiles; one for heads of 256, whose O leaves room for one S)
// and waits only until the scores are in registers.  An issuer is held up by
// its MMAs' execution and in between by its own waits and loop; with two,
// one's MMAs run meanwhile (with one issuer for both, the 8192-token prompt
// took a fifth longer).  The two softmax groups take alternate key tiles, a
// thread a whole row; what passes between them is the rows' reference.
//
// Code size is part of the design: the roles run through most of the code
// once per tile or once per part, and what falls out of the instruction
// caches is fetched again.  So each loop body is there once, conditions that
// hold for a whole call are arithmetic instead of branches (the compiler
// copies a loop for either side of those), waits are a few instructions and
// the schedule is worked out by one warp.  The 8192-token prompt went from
// 537 to 441 us with 138 -> 77 KB of code, and when the kernel had grown
// again from 272 to 257 with 94 -> 78.
//
// Measured (one GB300, device time of a call; in brackets first the
// batch-invariant form's, which writes and reads back a part for every 512 keys
// or more of a row tile; bound: the cached keys' and values' bytes at 6.67 TB/s
// or the products at 1905 TFLOP/s):
//   1 token over 1000, 20 heads on 4 of 128              9.9 us (11.6; bound 0.3: latency)
//   16 tokens over 32,781, 16 heads on 4 of 256         34.4 us (41.6; bound 20.2: bytes)
//   8 x 21 tokens over up to 9000, 20 heads of 128      70.4 us (97; bound 60.8: bytes; 5.8 TB/s)
//   32 x up to 40 tokens, window 1000, 20 on 4 of 64    23.6 us (31; bound 3.9: bytes)
//   4 x up to 1500 tokens over 12,000, 16 on 4 of 256    225 us (534; bound 173: 1465 TFLOP/s)
//   8192 tokens, 20 heads of 128                         253 us (672; bound 180: 1357 TFLOP/s)
// The short ones are a chain of latencies.  By the clock, us from the end of
// the kernel before, one token over 1000: place found 1.0, page ids 1.9, first
// scores 3.2, weights 4.4, product 5.0, part stored 5.5, CTAs ended 6.4, second
// kernel under way 7.2, joined 9.0.  16 tokens over 32,781: 1.8, 2.1, 5.6, 6.5,
// the last product 26.1 (so 24 us from the first load to the last product, 5.6
// TB/s), part stored 28.2, ended 28.4, second kernel 29.2, joined 34.3.
// Prompts are bound by a row's softmax between its two products (maximum 340
// cycles, powers 910, loads and stores 350 of 1500 a tile and group, the
// tensor pipe 61-71% active).
#include <algorithm>
#include <climits>

#include "runtime.h"
#include "sm103_ptx.cuh"

namespace w4v {
namespace {

constexpr int kKeyBits = 7, kKeys = 1 << kKeyBits;       // keys per tile
constexpr int kRows = 128;                      // rows per tile
constexpr int kThreads = 384;
constexpr int kWarpProd = 0, kWarpScores = 1, kWarpOut = 2, kWarpGuard = 3, kWarpSoft = 4;
// Ring of parts (three, with room for it made, changed nothing; the softmax
// groups count on two).
constexpr int kParts = 2;
constexpr int kPartReaders = 11;                // every warp but the producer
constexpr uint32_t kTmemCols = 512;
// Tensor memory: S in one or two buffers of 128 columns, P in two of 64, O.
constexpr uint32_t kPcols = kKeys / 2;
constexpr float kShift = 8.f, kSlack = 6.f;
constexpr float kLn2 = 0.6931471805599453f;
// What a row tile costs beside its keys, in key tiles.  The time of 3; with 0
// the CTAs that hold the short rows of prompts end last: 272 -> 314 us for
// 8192 tokens, 245 -> 338 for prompts in chunks; 6 costs up to 2% more.
constexpr int kPartCost = 3;
constexpr int kInvBits = 2;                     // least tiles of a batch-invariant part (2^this)
constexpr int kInvParts = 32;                   // most parts of a row tile

template <int D>
struct Plan {
    static constexpr int kBlocks = D / 64;                       // 64-element blocks of a head
    static constexpr int kStageBlocks = D >= 128 ? 2 : 1;
    static constexpr int kHalves = kBlocks / kStageBlocks;       // stages per tile of K (or V)
    static constexpr int kGroupBytes = kStageBlocks * 1024;      // 8 tokens of a stage
    static constexpr int kStageBytes = kKeys / 8 * kGroupBytes;
    static constexpr int kQBytes = kBlocks * kRows * 128;
    static constexpr int kStagesK = D == 64 ? 5 : 3, kStagesV = D == 64 ? 5 : D == 128 ? 3 : 2;
    static constexpr int kStages = kStagesK + kStagesV;          // rings of their own, each with one reader
    static constexpr int kBar = kQBytes + kStages * kStageBytes;
    static constexpr int kScores = D >= 256 ? 1 : 2;             // S buffers, and tiles that Q K^T runs ahead
    static constexpr bool kOwn = D <= 64;                        // an O for each softmax group
    static constexpr uint32_t kPcol = kScores * kKeys, kOcol = kPcol + 2 * kPcols;
    static constexpr int kNumBars = 2 + 2 * kStages + 12 + 4 + 8 + 8 + 2 * kParts;
    static constexpr int kMisc = kBar + 8 * kNumBars;
    static constexpr int kRing = (kMisc + 16 + 15) & ~15;
    static constexpr int kRef = kRing + kParts * 48;             // float[kRows]: the rows' references
    static constexpr int kSums = kRef + kRows * 4;               // float2[2][kRows]: a group's m and l, by part
    static constexpr int kBytes = kSums + 2 * kRows * 8;
    static_assert(kOcol + (kOwn ? 2 : 1) * D <= kTmemCols, "tensor memory plan");
    static_assert(kBytes <= 227 * 1024, "shared memory plan");
};

// Rows [r0, r1) of a row tile that an entry's CTAs of the second kernel join
// from n parts (n = 0: nothing).  Default: entry c is for the tile that range c
// begins inside of, its parts in slot 2 first + 1 and then 2 (first + i);
// batch-invariant: entry u for unit u, slots in a row.  What needs a division
// is worked out here, where there is time.
struct __align__(16) Share {
    int row0, kvh;              // the tile's first token
    int rows;                   // r0, and in the upper half r1
    int slot0, n;
    int n_mul;                  // 2^20 / n, rounded up: k * n_mul >> 20 is k / n for k < 1024
    int block;                  // rows that are fetched at a time
    int count;                  // batch-invariant, entry 0: how many entries there are (default: one per range)
};
template <int D>
constexpr int kHeld = D == 256 ? 40 : 12288 / (2 * D);      // rows of parts that it holds at a time

struct Args {
    __half *out;
    float *lse;
    float *part_o;              // [slots][slot_rows][D]
    float2 *part_ml;            // [slots][slot_rows]: m (log2), l
    const __half *v;            // the cache's values (rows that must be looked at again)
    const int32_t *table, *lengths, *offsets;
    uint32_t *status;
    int n_tokens, q_heads, kv_heads, group, tok;   // query heads per key/value head, tokens per tile
    uint64_t tok_mul;           // 2^tok_shift / tok, rounded up; 2^tok_shift is 2^31 times tok or more,
    int group_mul;              // 2^16 / group, rounded up: row * group_mul >> 16 is row / group for rows of a tile
    int tok_shift;              // so that x * tok_mul >> tok_shift is x / tok for 31-bit x
    int wide;                   // out is 32-byte aligned
    int B, width, n_pages, page_bits, slot_rows;   // 2^page_bits tokens a page
    int back;                   // keys that a row sees before its own (INT_MAX: all)
    int invariant;              // batch-invariant: a part is one unit
    int unit_bits, part_cost;   // 2^unit_bits tiles per unit; units for the work beside a row tile's keys
    uint32_t max_units;         // of one key/value head: what the workspace (batch-invariant) and 32 bits hold
    struct Share *shares;       // what the second kernel joins
    float scale_log2;
};

// ------------------------------------------------------------------ schedule
struct Seq {
    int first, n, len;          // its rows, their count, cached tokens
};
__device__ __forceinline__ Seq seq_of(const Args &p, int b) {
    Seq s;
    s.first = min(max(p.offsets[b], 0), p.n_tokens);
    s.n = max(min(max(p.offsets[b + 1], 0), p.n_tokens) - s.first, 0);
    s.len = min(max(p.lengths[b], 0), p.width << p.page_bits);
    return s;
}

// Key tiles that row tile qt reads, and its units: one per key tile (one where
// there are none), and in the default schedule kPartCost more, last, that
// stand for the work beside the keys.  (Without branches on the mode: the
// compiler makes a copy of a loop for each side of those.)
struct Extent {
    int lo, hi, units;          // tiles [lo, hi)
};
__device__ __forceinline__ Extent extent_of(const Args &p, const Seq &s, int qt) {
    const int t0 = qt * p.tok, t1 = min(s.n, t0 + p.tok) - 1;
    const int p0 = max(s.len - s.n + t0, 0), p1 = max(s.len - s.n + t1, -1);
    Extent e;
    e.lo = max(p0 - p.back, 0) >> kKeyBits;
    e.hi = (p1 >> kKeyBits) + 1;
    e.units = max(((e.hi - 1) >> p.unit_bits) - (e.lo >> p.unit_bits) + 1, 1) + p.part_cost;
    return e;
}

// Row tiles of n new tokens: n / tok rounded up, by a multiplication.
__device__ __forceinline__ int row_tiles(const Args &p, int n) {
    return int(uint64_t(uint32_t(n + p.tok - 1)) * p.tok_mul >> p.tok_shift);
}

// Units of one key/value head of 32 sequences, one per lane (0 past the end).
// A lane counts a few row tiles by itself; the warp together those of a
// sequence with more.
__device__ __forceinline__ int lane_units(const Args &p, int b) {
    constexpr int kFew = 4;
    const int lane = threadIdx.x & 31;
    Seq s{0, 0, 0};
    if (b < p.B) s = seq_of(p, b);
    const int tiles = row_tiles(p, s.n);
    uint32_t many = __ballot_sync(0xFFFFFFFFu, tiles > kFew);
    Seq o = s;
    int u = 0, src = lane, qt = 0, end = min(tiles, kFew), step = 1;
#pragma unroll 1
    for (bool own = true;; own = false) {        // the loop's body is there once
        int sum = 0;
#pragma unroll 1
        for (; qt < end; qt += step) sum += extent_of(p, o, qt).units;
        if (!own) sum = __reduce_add_sync(0xFFFFFFFFu, sum);
        if (lane == src) u += sum;
        if (many == 0) break;
        src = __ffs(many) - 1;
        many &= many - 1;
        o = Seq{0, __shfl_sync(0xFFFFFFFFu, s.n, src), __shfl_sync(0xFFFFFFFFu, s.len, src)};
        qt = kFew + lane;
        end = __shfl_sync(0xFFFFFFFFu, tiles, src);
        step = 32;
    }
    return u;
}

// The same value in every lane, as one that the compiler knows to be so.
__device__ __forceinline__ int warp_uniform(int x) { return __reduce_max_sync(0xFFFFFFFFu, x); }

__device__ __forceinline__ int warp_scan(int x) {
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xFFFFFFFFu, x, d);
        if ((threadIdx.x & 31) >= d) x += y;
    }
    return x;
}

// An even split of `units` over at most `ctas` ranges, none of them empty.
struct Split {
    int ranges = 0, each = 0, more = 0;          // the first `more` ranges hold one unit more than `each`
    __device__ __forceinline__ Split() {}
    __device__ __forceinline__ Split(int units, int ctas) {
        ranges = min(units, ctas);
        each = ranges > 0 ? units / ranges : 0;
        more = units - each * ranges;
    }
    __device__ __forceinline__ int begin(int c) const { return c * each + min(c, more); }
    __device__ __forceinline__ int owner(int u) const {
        const int past = u - more * (each + 1);
        return past < 0 ? u / (each + 1) : more + past / each;
    }
};

struct Place {
    int b, kvh, qt, u;          // unit u of a row tile
};
// All units, how they are split, and the place of the first one of range cta
// (one warp).  Two passes over the sequences, 32 at a time; with 32 or fewer
// the second one has the first one's counts.  The host has seen that rows
// counted once fit; offsets that go up and down count rows again and again, so
// the sum is looked at here, and too large a one leaves nothing to do (false).
__device__ __forceinline__ bool schedule(const Args &p, int cta, int ctas, Place &w, int &all, Split &split) {
    const int lane = threadIdx.x & 31;
    int u = 0, at = 0;
    uint32_t mine = 0;                           // this lane's sequences, no further than 2^31 - 1
    all = 0;
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
#pragma unroll 1
        for (int b0 = 0; b0 < p.B; b0 += 32) {
            if (pass == 0 || p.B > 32) u = lane_units(p, b0 + lane);
            if (pass == 0) {
                mine = min(mine + uint32_t(u), 0x7FFFFFFFu);
                continue;
            }
            const int upto = warp_scan(u * p.kv_heads);
            const uint32_t past = __ballot_sync(0xFFFFFFFFu, upto > at);
            if (past == 0) {
                at -= __shfl_sync(0xFFFFFFFFu, upto, 31);
                continue;
            }
            const int src = __ffs(past) - 1;
            const int su = __shfl_sync(0xFFFFFFFFu, u, src);
            at -= __shfl_sync(0xFFFFFFFFu, upto, src) - su * p.kv_heads;
            w.b = b0 + src;
            w.kvh = at / su;
            int rest = at - w.kvh * su;
            const Seq s = seq_of(p, w.b);
            const int tiles = row_tiles(p, s.n);
#pragma unroll 1
            for (int q0 = 0;; q0 += 32) {
                const int tile = q0 + lane < tiles ? extent_of(p, s, q0 + lane).units : 0;
                const int sum = warp_scan(tile);
                const uint32_t over = __ballot_sync(0xFFFFFFFFu, sum > rest);
                if (over != 0 || q0 >= tiles) {
                    const int l = over != 0 ? __ffs(over) - 1 : 0;
                    w.qt = q0 + l;
                    w.u = rest - __shfl_sync(0xFFFFFFFFu, sum - tile, l);
                    break;
                }
                rest -= __shfl_sync(0xFFFFFFFFu, sum, 31);
            }
            break;
        }
        if (pass == 0) {
            const uint64_t sum = (uint64_t(__reduce_add_sync(0xFFFFFFFFu, mine >> 16)) << 16) +
                                 __reduce_add_sync(0xFFFFFFFFu, mine & 0xFFFFu);
            if (sum > p.max_units) return false;
            all = int(sum) * p.kv_heads;
            split = Split(all, ctas);
            if (cta >= split.ranges) break;
            at = split.begin(cta);
        }
    }
    return true;
}

// A run of units of one row tile.
struct Part {
    int nt, kt0;                // key tiles (-1: no more parts), the first one
    int row0, rows;             // the first row's token, rows in use
    int pos0, keys_end;         // its position; keys that any of the rows sees end here
    int b, kvh;
    int slot;                   // where its partial result goes, -1: it is the whole
    int u, units;               // its first unit, the row tile's (without kPartCost)
};
static_assert(sizeof(Part) <= 48, "ring of parts");
struct Cursor {
    Place w;
    int unit, left;             // index of the next unit, units left in the range
    Seq s;
    __device__ __forceinline__ void load(const Args &p) { s = seq_of(p, w.b); }
    // The next part, and the index of its first unit.
    __device__ __forceinline__ bool next(const Args &p, int cta, Part &g, int &first) {
        for (int take = 0; take == 0;) {
            if (left <= 0) return false;
            const Extent e = extent_of(p, s, w.qt);
            const int t0 = w.qt * p.tok, toks = min(p.tok, s.n - t0);
            g.row0 = s.first + t0;
            g.rows = toks * p.group;
            g.pos0 = s.len - s.n + t0;
            g.keys_end = max(g.pos0 + toks, 0);
            g.b = w.b;
            g.kvh = w.kvh;
            g.u = w.u;
            g.units = e.units;
            first = unit;
            const int step = min(e.units - w.u, p.invariant ? 1 : left);
            g.units -= p.part_cost;
            take = max(min(g.units - w.u, step), 0);         // none: a range may begin past the keys
            const int c = ((e.lo >> p.unit_bits) + w.u) << p.unit_bits;
            g.kt0 = max(e.lo, c);
            g.nt = max(min(e.hi, c + (take << p.unit_bits)) - g.kt0, 0);
            g.slot = p.invariant ? unit : 2 * cta + (w.u == 0);
            if (take == g.units) g.slot = -1;
            w.u += step;
            unit += step;
            left -= step;
            if (w.u == e.units) {
                w.u = 0;
                if ((w.qt + 1) * p.tok < s.n) {
                    ++w.qt;
                } else {
                    w.qt = 0;
                    if (++w.kvh == p.kv_heads) {
                        w.kvh = 0;
                        if (left > 0)
#pragma unroll 1
                        do {
                            ++w.b;
                            load(p);
                        } while (s.n == 0 && w.b < p.B - 1);
                    }
                }
            }
        }
        return true;
    }
};

// 0 if none of eight fp16 values is infinite or NaN (exponent all ones).
__device__ __forceinline__ uint32_t not_finite(const uint4 &v) {
    auto carry = [](uint32_t w) { return (w & 0x7C007C00u) + 0x04000400u; };
    return (carry(v.x) | carry(v.y) | carry(v.z) | carry(v.w)) & 0x80008000u;
}
__device__ __forceinline__ void clear_not_finite(uint4 &v) {
    auto clear = [](uint32_t w) {
        const uint32_t c = ((w & 0x7C007C00u) + 0x04000400u) & 0x80008000u;
        return w & ~((c >> 15) * 0xFFFFu);
    };
    v.x = clear(v.x);
    v.y = clear(v.y);
    v.z = clear(v.z);
    v.w = clear(v.w);
}

// Whether a tile's values are looked over before the product: some row does
// not see some key of it (the first row sees those up to pos0, the last one
// those from keys_end - window on), or its last step has spare keys.
__device__ __forceinline__ bool guarded(const Args &p, int key, int keys_end, int pos0) {
    const int seen = min(keys_end - key, kKeys);
    return seen % 16 != 0 || pos0 + 1 - key < seen || (keys_end - 1 - p.back > key);
}

// A whole warp's wait for a phase, in as few instructions as it takes: they
// are at two dozen places (with a look at the clock in the loop the kernel was
// 2-7% slower throughout).  A try suspends the warp for up to kSuspendHintNs,
// so the limit is seconds.  A role that gave up leaves; those that wait for it
// give up in turn.
constexpr int kWaitTries = 1 << 17;
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity) {
    bool done = mbar_test_wait(bar, parity);
#pragma unroll 1
    for (int n = 0; n < kWaitTries; ++n) {
        if (__all_sync(0xFFFFFFFFu, done)) return true;
        done = mbar_try_wait(bar, parity);
    }
    return false;
}

// ---------------------------------------------------------------- the kernel
template <int D>
__global__ void __launch_bounds__(kThreads, 1)
paged_attn_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                  const __grid_constant__ CUtensorMap vmap, const Args p) {
    using P = Plan<D>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t base = smem_u32(smem);
    const uint32_t bar0 = base + P::kBar;
    const uint32_t q_full = bar0, q_empty = bar0 + 8u;
    auto kv_full = [&](int s) { return bar0 + 16u + 8u * s; };   // K's stages, then V's
    auto kv_empty = [&](int s) { return bar0 + 16u + 8u * (P::kStages + s); };
    const uint32_t rest = bar0 + 16u + 16u * P::kStages;
    auto s_full = [&](int i) { return rest + 8u * i; };          // by softmax group
    auto p_full = [&](int i) { return rest + 16u + 8u * i; };
    // Four phases apart: who has seen tile t - 4's product may wait for any of
    // t - 3 .. t without taking one phase for the next but one.
    auto pv_done = [&](int tile) { return rest + 32u + 8u * (tile & 3); };
    auto pv_phase = [&](int tile) { return uint32_t(tile >> 2) & 1u; };
    auto s_empty = [&](int i) { return rest + 64u + 8u * i; };
    auto v_ask = [&](int n) { return rest + 80u + 8u * (n & 1); };          // by guarded tile
    auto v_ready = [&](int n) { return rest + 96u + 8u * (n & 1); };
    const uint32_t o_empty = rest + 112u, done_bar = rest + 120u;
    auto turn = [&](int quad, int i) { return rest + 128u + 16u * quad + 8u * i; };
    auto pair = [&](int quad, int i) { return rest + 192u + 16u * quad + 8u * i; };
    auto part_full = [&](int i) { return rest + 256u + 8u * i; };
    auto part_empty = [&](int i) { return rest + 256u + 8u * (kParts + i); };
    uint32_t *misc = reinterpret_cast<uint32_t *>(smem + P::kMisc);    // [0] tmem, [2..3] below
    volatile uint32_t *spoilt = misc + 2;                    // [i & 1]: part i (from 1) had values cleared
    Part *ring = reinterpret_cast<Part *>(smem + P::kRing);
    float *ref = reinterpret_cast<float *>(smem + P::kRef);
    float2 *sums = reinterpret_cast<float2 *>(smem + P::kSums);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        for (int s = 0; s < P::kStages; ++s) {
            mbar_init(kv_full(s), 1);
            mbar_init(kv_empty(s), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(s_full(i), 1);
            mbar_init(p_full(i), 4);             // the warps of one softmax group
            mbar_init(s_empty(i), 4);
        }
        for (int i = 0; i < 4; ++i) mbar_init(pv_done(i), 2);    // the MMAs, and the issuer's own arrival
        for (int i = 0; i < 2; ++i) {
            mbar_init(v_ask(i), 1);
            mbar_init(v_ready(i), 1);
        }
        mbar_init(o_empty, 4);                   // the group that ends a part
        mbar_init(done_bar, 2);                  // both issuers
        for (int q = 0; q < 4; ++q) {
            mbar_init(turn(q, 0), 1);
            mbar_init(turn(q, 1), 1);
            mbar_init(pair(q, 0), 1);            // the group that does not end a part
            mbar_init(pair(q, 1), 1);
        }
        for (int i = 0; i < kParts; ++i) {
            mbar_init(part_full(i), 1);
            mbar_init(part_empty(i), kPartReaders);
        }
        misc[2] = misc[3] = 0;
        fence_barrier_init();
    }
    if (warp == kWarpGuard) {
        tmem_alloc(smem_u32(&misc[0]), kTmemCols);
        tmem_relinquish();
    }
    if (warp == kWarpProd && lane == 0) {
        prefetch_tensormap(&qmap);
        prefetch_tensormap(&kmap);
        prefetch_tensormap(&vmap);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = warp_uniform(misc[0]);
    grid_dep_wait();
    grid_dep_launch();
    bool ok = (base & 1023u) == 0u;              // the operands' swizzle needs it

    // The next part (its number in the ring is `i`); the warp gives it back
    // with release() once it has read what it needs.
    auto part_of = [&](int i) -> const Part & { return ring[i % kParts]; };
    auto acquire = [&](int i) {
        ok = ok && wait(part_full(i % kParts), (i / kParts) & 1);
        return ok && part_of(i).nt >= 0;
    };
    auto release = [&](int i) {
        __syncwarp();
        if (lane == 0) mbar_arrive(part_empty(i % kParts));
    };

    // registers from the four single warps to the softmax groups: 128 x 88 +
    // 256 x 208 of the 384 x 168 that the CTA was launched with
    if (warp < kWarpSoft) set_max_registers_down<88>();
    if (warp == kWarpProd) {
        int all = 0;
        Split split;
        Cursor cur{};
        if (!schedule(p, blockIdx.x, gridDim.x, cur.w, all, split) && blockIdx.x == 0 && lane == 0)
            atomicOr(p.status, 1u << kStatusShape);
        if (int(blockIdx.x) < split.ranges) {
            cur.unit = split.begin(blockIdx.x);
            cur.left = split.begin(blockIdx.x + 1) - cur.unit;
            cur.load(p);
        }
        const int box_bits = min(p.page_bits, 7);            // 2^box_bits tokens per TMA box
        const uint32_t box_bytes = P::kGroupBytes << (box_bits - 3);
        const int boxes = kKeys >> box_bits;                 // of a key tile
        const int group_bits = p.page_bits - 3;              // 8-token groups of a page
        // this lane's box within a stage, and the stages to fill next
        const uint32_t box_at = base + P::kQBytes + lane * box_bytes;
        struct Stage {
            int s;
            uint32_t phase;
        } sk{0, 0}, sv{0, 0};
        int nq = 0;
        for (int i = 0; ok; ++i) {
            Part g{};
            int unit = 0;
            if (!cur.next(p, blockIdx.x, g, unit)) g.nt = -1;
            if (i >= kParts) ok = wait(part_empty(i % kParts), (i / kParts - 1) & 1);
            if (!ok) break;
            if (lane == 0) {
                ring[i % kParts] = g;
                mbar_arrive(part_full(i % kParts));
            }
            if (g.nt > 0) {
                // Page ids of the part's boxes, 32 at a time, one per lane: three
                // such batches at hand, so that each is loaded long before its use
                // and V's, which runs behind K's, is still there.
                const int32_t *row = p.table + size_t(g.b) * p.width;
                const int box0 = (g.kt0 * kKeys) >> box_bits;
                const int all_boxes = ((g.keys_end - 1) >> box_bits) + 1;
                auto batch = [&](int n) -> int {
                    const int at = box0 + 32 * n + lane;
                    return at < all_boxes ? row[at >> (p.page_bits - box_bits)] : -1;
                };
                int ids0 = batch(0), ids1 = batch(1), ids2 = -1;
                // this lane's box of key tile j: its first 8-token group (that of
                // no page is one past the cache, which TMA fills with zeros)
                auto group_of = [&](int j) -> int {
                    const int e = j * boxes, n = (e >> 5) % 3;
                    const int id = __shfl_sync(0xFFFFFFFFu, n == 0 ? ids0 : n == 1 ? ids1 : ids2, (e + lane) & 31);
                    const int at = id >= 0 && id < p.n_pages ? id * p.kv_heads + g.kvh : p.n_pages * p.kv_heads;
                    return (at << group_bits) + (((box0 + e + lane) << (box_bits - 3)) & ((1 << group_bits) - 1));
                };
                auto load = [&](const CUtensorMap *map, int j, int first, int depth, Stage &st) {
                    const int grp = group_of(j);
                    const int n = min(all_boxes - (box0 + j * boxes), boxes);
#pragma unroll 1
                    for (int h = 0; h < P::kHalves && ok; ++h) {
                        const int s = first + st.s;
                        ok = wait(kv_empty(s), st.phase ^ 1);    // the first time round: passes
                        if (!ok) break;
                        if (lane == 0) mbar_arrive_expect_tx(kv_full(s), n * box_bytes);
                        __syncwarp();
                        if (lane < n)
                            tma_load_4d(box_at + s * P::kStageBytes, map, 0, 0, h * P::kStageBlocks, grp, kv_full(s));
                        if (++st.s == depth) {
                            st.s = 0;
                            st.phase ^= 1;
                        }
                    }
                };
                if (nq > 0) ok = wait(q_empty, (nq - 1) & 1);
                if (ok) {
                    if (lane == 0) mbar_arrive_expect_tx(q_full, P::kBlocks * p.tok * p.group * 128u);
                    __syncwarp();
                    if (lane < P::kBlocks)
                        tma_load_4d(base + lane * kRows * 128, &qmap, 0, g.kvh * p.group, g.row0, lane, q_full);
                    ++nq;
                }
                // K runs kScores tiles ahead of V, in the issuers' order
                for (int j = 0; j < g.nt + P::kScores && ok; ++j) {
                    const int e = j * boxes;
                    if ((e & 31) == 0 && e > 0) {                // K enters a batch: on its way, the next one
                        const int n = (e >> 5) + 1;
                        const int next = n % 3;
                        if (next == 0) ids0 = batch(n);
                        else if (next == 1) ids1 = batch(n);
                        else ids2 = batch(n);
                    }
                    if (j < g.nt) load(&kmap, j, 0, P::kStagesK, sk);
                    if (j >= P::kScores) load(&vmap, j - P::kScores, P::kStagesK, P::kStagesV, sv);
                }
            }
            // the share of this range's first row tile, or of every unit's
            // (here, behind the loads, for the second kernel alone reads it)
            if (lane == 0 && (p.invariant ? g.nt >= 0 || all == 0 : i == 0)) {
                Share e{g.row0, g.kvh, 0, unit - g.u, 0, 0, 1, p.invariant ? all : int(gridDim.x)};
                int share = g.u, shares = g.units;
                if (p.invariant) {
                    e.n = g.units > 1 ? g.units : 0;
                } else if (g.nt >= 0 && g.u > 0) {
                    const int first = split.owner(unit - g.u);
                    e.n = split.owner(unit - g.u + g.units - 1) - first + 1;
                    e.slot0 = 2 * first + 1;
                    share = int(blockIdx.x) - first - 1;
                    shares = e.n - 1;
                }
                if (e.n > 0) {
                    e.rows = share * g.rows / shares | (share + 1) * g.rows / shares << 16;
                    e.n_mul = (1 << 20) / e.n + 1;
                    e.block = max(kHeld<D> / e.n, 1);
                }
                p.shares[p.invariant ? unit : int(blockIdx.x)] = e;
            }
            if (g.nt < 0) break;
        }
        // A range that was given up leaves nothing to join.
        if (!ok)
            for (int e = (p.invariant ? split.begin(blockIdx.x) : int(blockIdx.x)) + lane;
                 e < (p.invariant ? min(split.begin(blockIdx.x + 1), max(all, 1)) : int(blockIdx.x) + 1); e += 32) {
                p.shares[e].n = 0;
                p.shares[e].count = all;
            }
        // Every copy has landed before the CTA ends, also where its reader gave
        // up.  (A stage that was never filled passes, as the phase before the first.)
#pragma unroll 1
        for (int s = 0; s < P::kStages; ++s) {
            const Stage st = s < P::kStagesK ? sk : Stage{P::kStagesK + sv.s, sv.phase};
            ok = wait(kv_full(s), st.phase ^ (s < st.s ? 0 : 1)) && ok;
        }
        if (nq > 0) ok = wait(q_full, (nq - 1) & 1) && ok;
    } else if (warp == kWarpScores) {
        // S = Q K^T.  Descriptors: the high words are constants, and the low
        // ones (address / 16) grow by constants from one per operand.  (Put
        // together from the address for each MMA they cost more to issue than
        // the MMA runs.)  What steers the loops goes through a warp-wide vote
        // or reduction: their results are uniform to the compiler, so stage
        // numbers and descriptors stay in uniform registers.
        constexpr uint32_t idesc = idesc_f16_f32(kRows, kKeys);
        constexpr uint64_t kHighQ = uint64_t(sdesc_high(1024)) << 32, kHighK = uint64_t(sdesc_high(P::kGroupBytes)) << 32;
        const uint32_t q_low = sdesc_low(base, 16), k_low = sdesc_low(base + P::kQBytes, 16);
        int it = 0, nq = 0, t = 0;                           // stages, parts, tiles so far
        for (int i = 0; __any_sync(0xFFFFFFFFu, acquire(i)); ++i) {
            const int nt = warp_uniform(part_of(i).nt);
            release(i);
            if (nt == 0) continue;
            ok = wait(q_full, nq & 1);
            ++nq;
            const int end = t + nt;
            for (; t < end && ok; ++t) {
                const int b = t % P::kScores, u = t / P::kScores;
                if (u > 0) ok = wait(s_empty(b), (u - 1) & 1);
#pragma unroll 1
                for (int h = 0; h < P::kHalves && ok; ++h, ++it) {
                    const int s = it % P::kStagesK;
                    ok = wait(kv_full(s), (it / P::kStagesK) & 1);
                    if (!ok) break;
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int k = 0; k < 4 * P::kStageBlocks; ++k)
                            mma_f16_ss(tmem + b * kKeys,
                                       kHighQ | (q_low + h * (P::kStageBlocks * kRows * 128 / 16) +
                                                 ((k >> 2) * (kRows * 128) + (k & 3) * 32) / 16),
                                       kHighK | (k_low + s * (P::kStageBytes / 16) + ((k >> 2) * 1024 + (k & 3) * 32) / 16),
                                       idesc, h > 0 || k > 0);
                        mma_commit(kv_empty(s));
                        if (h + 1 == P::kHalves) {
                            mma_commit(s_full(t & 1));       // by group: each waits for its own tiles alone
                            if (t + 1 == end) mma_commit(q_empty);
                        }
                    }
                    __syncwarp();
                }
            }
        }
        if (elect_one()) mma_commit(done_bar);
        __syncwarp();
        mbar_wait_bounded(done_bar, 0);
        __syncwarp();
    } else if (warp == kWarpOut) {
        // O += P V, over the keys that some row sees
        constexpr uint32_t idesc = idesc_f16_f32(kRows, 64 * P::kStageBlocks) | kIdescBMnMajor;
        constexpr uint64_t kHighV = uint64_t(sdesc_high(P::kGroupBytes)) << 32;
        const uint32_t v_low = sdesc_low(base + P::kQBytes + P::kStagesK * P::kStageBytes, 1024);
        int it = 0, nq = 0, t = 0;                           // stages, parts, tiles so far
        int asked = 0, looked = 0;                           // guarded tiles that the guard was asked for, and has done
        auto ask = [&](bool look) {
            if (look && elect_one()) mbar_arrive(v_ask(asked));
            asked += look;
            __syncwarp();
        };
        for (int i = 0; __any_sync(0xFFFFFFFFu, acquire(i)); ++i) {
            const int nt = warp_uniform(part_of(i).nt), pos0 = warp_uniform(part_of(i).pos0);
            const int key0 = warp_uniform(part_of(i).kt0 * kKeys), keys_end = warp_uniform(part_of(i).keys_end);
            release(i);
            if (nt == 0) continue;
            bool look = guarded(p, key0, keys_end, pos0);
            ask(look);
            for (int j = 0; j < nt && ok; ++j, ++t) {
                const int key = key0 + j * kKeys;
                // The guard works one tile ahead where that tile's stages were
                // last filled before this one's: waiting for their next fill
                // it then cannot take the one before for it.
                const bool next = j + 1 < nt && guarded(p, key + kKeys, keys_end, pos0);
                if (P::kStagesV >= 2 * P::kHalves) ask(next);
                if (j == 0 && nq++ > 0) ok = wait(o_empty, nq & 1);          // the part before is read
                ok = ok && wait(p_full(t & 1), (t >> 1) & 1);
                if (ok && look) {
                    ok = wait(v_ready(looked), (looked >> 1) & 1);
                    ++looked;
                }
                look = next;
                const int steps = min((keys_end - key + 15) / 16, kKeys / 16);
#pragma unroll 1
                for (int h = 0; h < P::kHalves && ok; ++h, ++it) {
                    const int s = it % P::kStagesV;
                    ok = wait(kv_full(P::kStagesK + s), (it / P::kStagesV) & 1);
                    if (!ok) break;
                    tc_fence_after();
                    if (elect_one()) {
                        const uint32_t d = tmem + P::kOcol + (P::kOwn ? (t & 1) * D : 0) + h * 64 * P::kStageBlocks, a = tmem + P::kPcol + (t & 1) * kPcols;
                        const uint32_t low = v_low + s * (P::kStageBytes / 16);
#pragma unroll
                        for (int k = 0; k < kKeys / 16; ++k)
                            if (k < steps)
                                mma_f16_ts(d, a + 8 * k, kHighV | (low + k * (2 * P::kGroupBytes / 16)), idesc,
                                           j > (P::kOwn ? 1 : 0) || k > 0);
                        mma_commit(kv_empty(P::kStagesK + s));
                        if (h + 1 == P::kHalves) {
                            mma_commit(pv_done(t));
                            mbar_arrive(pv_done(t));         // passes the guard's findings on
                        }
                    }
                    __syncwarp();
                }
                if (P::kStagesV < 2 * P::kHalves) ask(ok && next);
            }
        }
        if (elect_one()) mma_commit(done_bar);
        __syncwarp();
        mbar_wait_bounded(done_bar, 0);
        __syncwarp();
    } else if (warp == kWarpGuard) {
        // In guarded tiles, what the last 16 keys hold past those that some
        // row sees (other tokens, nothing at all) is cleared, and so is what
        // is not finite among keys that only some rows see.
        constexpr int kPieces = P::kStageBlocks * 8;         // 16-byte pieces of a token in a stage
        int it = 0, np = 0, looked = 0;
        for (int i = 0; acquire(i); ++i) {
            const Part g = part_of(i);
            release(i);
            if (g.nt == 0) continue;
            ++np;
            bool found = false;
            for (int j = 0; j < g.nt && ok; ++j) {
                const int key = (g.kt0 + j) * kKeys;
                if (!guarded(p, key, g.keys_end, g.pos0)) {
                    it += P::kHalves;
                    continue;
                }
                // the issuer has seen the stages' fill before this one
                ok = wait(v_ask(looked), (looked >> 1) & 1);
                const int seen = min(g.keys_end - key, kKeys), cleared = (seen + 15) / 16 * 16;
                const int above = min(max(g.pos0 + 1 - key, 0), seen);
                const int below = min(max(g.keys_end - 1 - p.back, 0) - key, above);
#pragma unroll 1
                for (int h = 0; h < P::kHalves && ok; ++h, ++it) {
                    const int s = P::kStagesK + it % P::kStagesV;
                    ok = wait(kv_full(s), (it / P::kStagesV) & 1);
                    if (!ok) break;
                    uint8_t *st = smem + P::kQBytes + s * P::kStageBytes;
                    // A first look at the 8-token groups that hold such keys, in
                    // the order of the addresses: 0 x v is 0 or, if v is not
                    // finite, NaN, and a NaN stays in the sum.
                    constexpr int kLoads = 8;                                // 512 bytes each
                    static_assert(kLoads * 512 % P::kGroupBytes == 0 && P::kStageBytes % (kLoads * 512) == 0, "whole groups");
                    __half2 sum[2] = {__float2half2_rn(0.f), __float2half2_rn(0.f)};
                    const int end = (seen + 7) / 8 * P::kGroupBytes;
#pragma unroll 1
                    for (int a = below > 0 ? 0 : above / 8 * P::kGroupBytes & ~(kLoads * 512 - 1); a < end; a += kLoads * 512) {
                        uint4 v[kLoads];
#pragma unroll
                        for (int k = 0; k < kLoads; ++k) v[k] = *reinterpret_cast<const uint4 *>(st + a + 512 * k + 16 * lane);
#pragma unroll
                        for (int k = 0; k < kLoads; ++k) {
                            const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                sum[e & 1] = __hfma2(*reinterpret_cast<const __half2 *>(&w[e]), __float2half2_rn(0.f), sum[e & 1]);
                        }
                    }
                    const bool some = __any_sync(0xFFFFFFFFu, ((h2_as_u32(sum[0]) | h2_as_u32(sum[1])) & 0x7FFF7FFFu) != 0u);
                    // a lane's 16-byte column, of every kStep'th token
                    constexpr int kStep = 32 / kPieces;
                    uint8_t *col = st + (lane % kPieces / 8) * 1024 + (lane % 8) * 16;
                    const int first = lane / kPieces;
                    auto piece = [&](int tok) {
                        return reinterpret_cast<uint4 *>(col + (tok / 8) * P::kGroupBytes + (tok % 8) * 128);
                    };
#pragma unroll 1
                    for (int k = first; some && k < seen; k += kStep) {
                        uint4 v = *piece(k);
                        if ((k >= below && k < above) || not_finite(v) == 0u) continue;
                        found = true;
                        clear_not_finite(v);
                        *piece(k) = v;
                    }
#pragma unroll 1
                    for (int k = seen + first; k < cleared; k += kStep) *piece(k) = make_uint4(0, 0, 0, 0);
                    fence_proxy_async_shared();
                }
                if (found) spoilt[np & 1] = np;
                __syncwarp();
                if (ok && lane == 0) mbar_arrive(v_ready(looked));
                ++looked;
            }
        }
    } else {
        set_max_registers_up<208>();
        const int half = (warp - kWarpSoft) >> 2, quad = warp & 3, row = 32 * quad + lane;
        const int row_tok = row / p.group, row_head = row - row_tok * p.group;
        const uint32_t lanes = uint32_t(32 * quad) << 16;
        const float c = p.scale_log2;
        int t = 0, np = 0;                                   // tiles and parts (with keys) so far
        int use = 0, pairs = 0;                              // references handed on, parts ended by this pair of warps
        for (int i = 0; acquire(i); ++i) {
            const int nt = part_of(i).nt, rows = part_of(i).rows, kt0 = part_of(i).kt0;
            np += nt > 0;
            const bool mine = row < rows;
            const bool busy = 32 * quad < rows;              // some row of this warp is in use
            const int pos = part_of(i).pos0 + row_tok;
            const int from = max(max(pos, 0) - p.back, 0);
            // every key of [sure_lo, sure_hi] is seen by all of the warp's rows
            const int sure_hi = __reduce_min_sync(0xFFFFFFFFu, mine ? pos : 0x7FFFFFFF);
            const int sure_lo = __reduce_max_sync(0xFFFFFFFFu, mine ? from : 0);
            float m = -INFINITY, l = 0.f;                    // reference (in units of q . k), this group's sum by it
            for (int j = 0; j < nt; ++j, ++t, ++use) {
                if ((t & 1) != half) continue;               // the other group's tile
                const int sb = t % P::kScores;
                ok = wait(s_full(t & 1), (t >> 1) & 1);
                if (!ok) break;
                if (!busy) {
                    // Nothing to do but keep the pace: a phase is told from
                    // the next but one only by who waited for the one between,
                    // and a second arrival within a phase would stand in for a
                    // warp that still works.
                    if (lane == 0) mbar_arrive(s_empty(sb));
                    if (t > 1) ok = wait(pv_done(t - 2), pv_phase(t - 2));
                    if (!ok) break;
                    if (lane == 0) mbar_arrive(p_full(t & 1));
                    continue;
                }
                tc_fence_after();
                uint32_t x[4][32];
                const int key = (kt0 + j) * kKeys;
#pragma unroll
                for (int k = 0; k < 4; ++k) tmem_ld_32x32b_x32(tmem + lanes + sb * kKeys + 32 * k, x[k]);
#pragma unroll
                for (int k = 0; k < 4; ++k) tc_wait_ld_keep<32>(x[k]);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(s_empty(sb));     // the scores are in registers
                if (key + kKeys - 1 > sure_hi || key < sure_lo) {
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        const int hi = pos - key - 32 * b, lo = from - key - 32 * b;         // keys lo .. hi are seen
                        const uint32_t seen = (hi < 0 ? 0u : 0xFFFFFFFFu >> (31 - min(hi, 31))) &
                                              (lo > 31 ? 0u : 0xFFFFFFFFu << max(lo, 0));
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            if ((seen & (1u << k)) == 0u) x[b][k] = 0xFF800000u;             // -inf
                    }
                }
                float top4[4];
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    top4[b] = __uint_as_float(x[b][0]);
#pragma unroll
                    for (int k = 1; k < 31; k += 2)
                        top4[b] = max3(top4[b], __uint_as_float(x[b][k]), __uint_as_float(x[b][k + 1]));
                    top4[b] = fmaxf(top4[b], __uint_as_float(x[b][31]));
                }
                const float top = fmaxf(max3(top4[0], top4[1], top4[2]), top4[3]);
                // The reference that the tile before left (of this group's own
                // tiles, or with one O of all), raised if need be
                float was = m;
                if (!P::kOwn) {
                    if (use > 0) ok = wait(turn(quad, (use - 1) & 1), ((use - 1) >> 1) & 1);
                    if (!ok) break;
                    was = j > 0 ? ref[row] : -INFINITY;
                }
                const bool raise = mine && top > was && (was == -INFINITY || (top - was) * c > kSlack);
                const float now = raise ? top : was;
                if (!P::kOwn) {
                    ref[row] = now;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(turn(quad, use & 1));
                }
                l = __fmul_rn(l, now == m ? 1.f : ex2((m - now) * c));   // m = -inf: l is 0 and stays
                m = now;
                // P's buffer: tile t - 2's product has read it
                if (t > 1) ok = wait(pv_done(t - 2), pv_phase(t - 2));
                if (!ok) break;
                tc_fence_after();
                if (__any_sync(0xFFFFFFFFu, raise && j > (P::kOwn ? 1 : 0))) {
                    // O by the new reference, once the tile before is added in
                    if (!P::kOwn) ok = wait(pv_done(t - 1), pv_phase(t - 1));
                    if (!ok) break;
                    tc_fence_after();
                    const float a = raise ? ex2((was - now) * c) : 1.f;
                    const uint32_t ocol = tmem + lanes + P::kOcol + (P::kOwn ? half * D : 0);
#pragma unroll 1
                    for (int o = 0; o < D; o += 32) {
                        uint32_t r[32];
                        tmem_ld_32x32b_x32(ocol + o, r);
                        tc_wait_ld_keep<32>(r);
#pragma unroll
                        for (int k = 0; k < 32; ++k) r[k] = __float_as_uint(__uint_as_float(r[k]) * a);
                        tmem_st_32x32b_x32(ocol + o, r);
                        tc_wait_st();
                        tc_keep_alive<32>(r);
                    }
                }
                const float off = m == -INFINITY ? 0.f : kShift - m * c;
                const float2 cc = make_float2(c, c), oo = make_float2(off, off);
                float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                uint32_t w[2][32];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
#pragma unroll
                    for (int k = 0; k < 32; ++k) {
                        const int e = 64 * h + 2 * k;
                        float2 y = __ffma2_rn(make_float2(__uint_as_float(x[e >> 5][e & 31]),
                                                          __uint_as_float(x[e >> 5][(e & 31) + 1])), cc, oo);
                        y.x = ex2(y.x);
                        y.y = ex2(y.y);
                        sum[k & 1] = __fadd2_rn(sum[k & 1], y);
                        w[h][k] = h2_as_u32(__float22half2_rn(y));
                    }
                    tmem_st_32x32b_x32(tmem + lanes + P::kPcol + (t & 1) * kPcols + 32 * h, w[h]);
                }
                tc_wait_st();
                tc_keep_alive<32>(w[0]);
                tc_keep_alive<32>(w[1]);
                const float2 all = __fadd2_rn(sum[0], sum[1]);
                l = __fadd_rn(l, __fadd_rn(all.x, all.y));
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full(t & 1));
            }
            if (!ok) break;
            // The group that had the part's last tile ends it (a part without
            // keys: the first group); the other leaves its sums and goes on to
            // the next part.
            if (!busy) use -= nt;                            // a pair that skips a part hands nothing on
            float2 *shared_sums = sums + (np & 1) * kRows + row;
            float weight = 1.f, weight2 = 0.f;
            if (nt > 0 ? ((t - 1) & 1) != half : half != 0) {
                if (busy && nt > 0) {
                    *shared_sums = make_float2(m, l);
                    __syncwarp();
                    // (it runs ahead by one part at most, for the ring holds two)
                    if (lane == 0) mbar_arrive(pair(quad, pairs & 1));
                    ++pairs;
                }
                release(i);
                continue;
            }
            if (nt > 0) ok = wait(pv_done(t - 1), pv_phase(t - 1));
            if (!ok) break;
            tc_fence_after();
            if (!busy) {
                if (nt > 0 && lane == 0) mbar_arrive(o_empty);
                release(i);
                continue;
            }
            if (nt > 0) {
                ok = wait(pair(quad, pairs & 1), (pairs >> 1) & 1);
                ++pairs;
                if (!ok) break;
                // Both groups' sums.  With one O by this group's reference, the
                // last; with two by the larger, and the O's with them.  Each
                // product is rounded by itself, here and in the loop above:
                // which group has the even key tiles, and which the last one,
                // depends on the CTA's work before and on the tile's other
                // rows, and a row's sum must not.
                const float2 other = *shared_sums;
                if (P::kOwn) {
                    const float both = fmaxf(m, other.x);
                    weight = m == both ? 1.f : ex2((m - both) * c);
                    weight2 = other.x == both ? 1.f : ex2((other.x - both) * c);
                    l = __fadd_rn(__fmul_rn(l, weight), __fmul_rn(other.y, weight2));    // a group without keys: 0
                    if (both == -INFINITY) weight = weight2 = 0.f;
                    m = both;
                } else {
                    l = __fadd_rn(l, other.x == m ? other.y : __fmul_rn(other.y, ex2((other.x - m) * c)));
                }
            }
            const bool fix = nt > 0 && spoilt[np & 1] == np;
            const Part g = part_of(i);
            const bool whole = g.slot < 0;
            const float inv = nt > 0 && l != 0.f ? 1.f / l : 0.f;
            const float m2 = m * c - kShift;
            const size_t orow = size_t(g.row0 + row_tok) * p.q_heads + g.kvh * p.group + row_head;
            const size_t srow = size_t(whole ? 0 : g.slot) * p.slot_rows + row;
            if (mine) {
                if (!whole) p.part_ml[srow] = make_float2(m2, l);
                else if (p.lse != nullptr) p.lse[orow] = nt > 0 ? (m2 + log2f(l)) * kLn2 : -INFINITY;
            }
            __syncwarp();
            __half *out = p.out + orow * D;
            float *part = p.part_o + srow * D;
#pragma unroll 1
            for (int o = 0; o < D; o += 32) {
                uint32_t r[32];
                tmem_ld_32x32b_x32(tmem + lanes + P::kOcol + (P::kOwn ? half * D : 0) + o, r);
                tc_wait_ld_keep<32>(r);
                if (P::kOwn && nt > 1) {
                    uint32_t q[32];
                    tmem_ld_32x32b_x32(tmem + lanes + P::kOcol + (half ^ 1) * D + o, q);
                    tc_wait_ld_keep<32>(q);
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        r[k] = __float_as_uint(__fadd_rn(__fmul_rn(__uint_as_float(r[k]), weight),
                                                         __fmul_rn(__uint_as_float(q[k]), weight2)));
                }
                if (mine && whole) {
                    uint32_t w[16];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint32_t h[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float2 y = make_float2(__uint_as_float(r[8 * k + 2 * e]), __uint_as_float(r[8 * k + 2 * e + 1]));
                            h[e] = inv != 0.f ? h2_as_u32(__floats2half2_rn(y.x * inv, y.y * inv)) : 0u;
                        }
                        w[4 * k] = h[0];
                        w[4 * k + 1] = h[1];
                        w[4 * k + 2] = h[2];
                        w[4 * k + 3] = h[3];
                    }
                    if (p.wide) {
                        stg_256(out + o, w);
                        stg_256(out + o + 16, w + 8);
                    } else {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            reinterpret_cast<uint4 *>(out + o)[k] = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
                    }
                } else if (mine) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) stg_256(part + o + 8 * k, r + 8 * k);
                }
                __syncwarp();
            }
            tc_fence_before();
            __syncwarp();
            if (nt > 0 && lane == 0) mbar_arrive(o_empty);
            if (fix && mine) {
                // the values that were cleared, for a row that sees them: the
                // weight is above 0, so they make the sum what they are
                const int below = max(g.keys_end - 1 - p.back, 0);
                const int last = min((kt0 + nt) * kKeys - 1, pos);
#pragma unroll 1
                for (int k = max(kt0 * kKeys, from); k <= last; ++k) {
                    if (k >= below && k <= g.pos0) k = g.pos0 + 1;       // seen by every row: not cleared
                    if (k > last) break;
                    const int id = p.table[size_t(g.b) * p.width + (k >> p.page_bits)];
                    if (id < 0 || id >= p.n_pages) continue;
                    const size_t slot = ((size_t(id) * p.kv_heads + g.kvh) << p.page_bits) + (k & ((1 << p.page_bits) - 1));
                    const __half *v = p.v + slot * D;
#pragma unroll 1
                    for (int o = 0; o < D; ++o) {
                        const float y = __half2float(v[o]);
                        if (isfinite(y)) continue;
                        if (whole) out[o] = __float2half_rn(__half2float(out[o]) + y);
                        else part[o] += y;
                    }
                }
            }
            release(i);
        }
    }

    if (!ok && lane == 0) atomicOr(p.status, 1u << kStatusTimeout);
    tc_fence_before();
    __syncthreads();
    if (warp == kWarpGuard) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// ---------------------------------------------------------- joining the parts
constexpr int kJoinThreads = 256;
// A share has at most rows / (n - 1) + 1 rows of n parts, and kJoinSplit CTAs.
constexpr int kJoinSplit = 4;
constexpr int kJoinWeights = 3 * kRows + 2 * kMaxCtas;

// o = sum 2^(m_i - M) o_i / sum 2^(m_i - M) l_i over a row's parts, M the
// largest m_i.  Latency bounds it: a warp fetches its rows' statistics and all
// fetch o's parts, both to shared memory, before anything is waited for, and
// the weights are worked out while the latter come in.  Sums run over the
// parts in order, so that parts of which a row sees no key (o = 0) change
// nothing.  A weight too small for fp32 still multiplies, so that it does not
// hide what is not finite.
template <int D>
__global__ void __launch_bounds__(kJoinThreads)
paged_attn_join_kernel(const Args p) {
    __shared__ float2 ml[kJoinWeights];          // m, l; then the part's weight, its share of the sum
    __shared__ float scale[kRows];
    constexpr int kLanes = D / 4, kLines = kJoinThreads / kLanes;    // threads per row, four columns each
    __shared__ __align__(16) float4 parts[kHeld<D> * kLanes];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int col = int(threadIdx.x) % kLanes, line = int(threadIdx.x) / kLanes;
    grid_dep_wait();
    grid_dep_launch();
    const int count = p.invariant ? p.shares[0].count : int(gridDim.x);
#pragma unroll 1
    for (int e = blockIdx.x; e < count; e += gridDim.x) {
        const Share g = p.shares[e];
        const int n = g.n;
        if (n == 0) continue;
        const int s0 = g.rows & 0xFFFF, s1 = g.rows >> 16;
        const int r0 = s0 + int(blockIdx.y) * (s1 - s0) / kJoinSplit;
        const int rows = s0 + int(blockIdx.y + 1) * (s1 - s0) / kJoinSplit - r0;
        auto at = [&](int i, int r) {            // part i's row
            const int slot = p.invariant ? g.slot0 + i : i == 0 ? g.slot0 : g.slot0 - 1 + 2 * i;
            return size_t(slot) * p.slot_rows + r0 + r;
        };
        auto row_out = [&](int r) {
            const int tok = (r0 + r) * p.group_mul >> 16;
            return size_t(g.row0 + tok) * p.q_heads + g.kvh * p.group + (r0 + r - tok * p.group);
        };
        const int held = min(n, kHeld<D>);          // parts at a time (all of them, or those of one row)
        __syncthreads();                         // the entry before is done with
        // rows to warps: of a few parts a row is a lane's, else a warp's
        const int wide = n <= 4 ? 0 : 31;        // lanes per row - 1
        const int first = wide != 0 ? warp : int(threadIdx.x), step = wide != 0 ? kJoinThreads / 32 : kJoinThreads;
#pragma unroll 1
        for (int r = first; r < rows; r += step)
#pragma unroll 1
            for (int i = lane & wide; i < n; i += wide + 1) cp_async<8>(smem_u32(&ml[r * n + i]), &p.part_ml[at(i, r)], 8);
        cp_async_commit();
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
        for (int b = 0; b < rows; b += g.block) {
            const int here = min(g.block, rows - b);
#pragma unroll 1
            for (int i0 = 0; i0 < n; i0 += held) {
                const int m = min(held, n - i0);
                if (b + i0 > 0) __syncthreads(); // what was there before is done with
#pragma unroll 2
                for (int k = line; k < here * m; k += kLines) {
                    const int r = m == n ? k * g.n_mul >> 20 : 0, i = k - r * m;
                    cp_async_16(smem_u32(&parts[k * kLanes + col]), p.part_o + at(i0 + i, b + r) * D + 4 * col);
                }
                cp_async_commit();
                if (b + i0 == 0) {
                    cp_async_wait<1>();
                    __syncwarp();
#pragma unroll 1
                    for (int r = first; r < rows; r += step) {
                        float2 *x = ml + r * n;
                        float top = -INFINITY, l = 0.f;
#pragma unroll 1
                        for (int i = lane & wide; i < n; i += wide + 1) top = fmaxf(top, x[i].x);
                        if (wide != 0)
#pragma unroll
                            for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
#pragma unroll 1
                        for (int i = lane & wide; i < n; i += wide + 1) {
                            const float2 y = x[i];
                            const float w = top == -INFINITY ? 0.f : ex2(y.x - top);
                            x[i] = make_float2(w, y.y != 0.f ? w * y.y : 0.f);
                        }
                        if (wide != 0) __syncwarp();
#pragma unroll 4
                        for (int i = 0; i < n; ++i) l += x[i].y;
                        if ((lane & wide) == 0) {
                            scale[r] = l != 0.f ? 1.f / l : 0.f;
                            if (p.lse != nullptr) p.lse[row_out(r)] = l != 0.f ? (top + log2f(l)) * kLn2 : -INFINITY;
                        }
                    }
                }
                cp_async_wait<0>();
                __syncthreads();
#pragma unroll 1
                for (int r = line; r < here; r += kLines) {
                    if (i0 == 0) o = make_float4(0.f, 0.f, 0.f, 0.f);
                    const float2 *x = ml + (b + r) * n + i0;
                    const float4 *v = parts + r * m * kLanes + col;
#pragma unroll 4
                    for (int i = 0; i < m; ++i) {
                        const float w = x[i].x;
                        const float4 y = v[i * kLanes];
                        o = make_float4(fmaf(w, y.x, o.x), fmaf(w, y.y, o.y), fmaf(w, y.z, o.z), fmaf(w, y.w, o.w));
                    }
                    if (i0 + m < n) continue;
                    const float inv = scale[b + r];
                    uint2 h = make_uint2(0u, 0u);
                    if (inv != 0.f) {
                        h.x = h2_as_u32(__floats2half2_rn(o.x * inv, o.y * inv));
                        h.y = h2_as_u32(__floats2half2_rn(o.z * inv, o.w * inv));
                    }
                    *reinterpret_cast<uint2 *>(p.out + row_out(b + r) * D + 4 * col) = h;
                }
            }
        }
    }
}

// -------------------------------------------------------------------- the host
int tokens_per_tile(int q_heads, int kv_heads) { return kRows / (q_heads / kv_heads); }

// Tiles of a batch-invariant part (2^this): by the table's size alone, so that
// it is the same in every call on a cache.  (By the keys' positions, 16 parts
// in every doubling, it would not depend on the table either, but parts of
// unequal length are dealt out unevenly: 16 tokens over 32,781 took 54.5 us
// against 41.5.)
int inv_tile_bits(int max_context) {
    const long long tiles = ((long long)max_context + kKeys - 1) / kKeys;
    int bits = kInvBits;
    while (tiles > (long long)kInvParts << bits) ++bits;
    return bits;
}

struct Slots {
    size_t count;
    int rows;
};
Slots slots_of(int n_tokens, int B, int q_heads, int kv_heads, int max_context, bool invariant) {
    const int tok = tokens_per_tile(q_heads, kv_heads);
    Slots s;
    s.rows = std::min(tok, std::max(n_tokens, 1)) * (q_heads / kv_heads);
    if (!invariant) {
        s.count = 2 * size_t(kMaxCtas);
    } else {
        const size_t tiles = size_t(kv_heads) * (size_t(n_tokens) / tok + std::min(B, n_tokens) + 1);
        const size_t keys = size_t(kKeys) << inv_tile_bits(max_context);
        s.count = tiles * ((size_t(max_context) + keys - 1) / keys + 1);
    }
    return s;
}

template <int D>
w4v_status launch(const CUtensorMap &qmap, const CUtensorMap &kmap, const CUtensorMap &vmap, const Args &a, int grid,
                  cudaStream_t stream) {
    static int configured_for = -1;
    int dev = 0;
    cudaGetDevice(&dev);
    if (configured_for != dev) {
        if (cudaFuncSetAttribute(paged_attn_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 Plan<D>::kBytes) != cudaSuccess) {
            cudaGetLastError();
            return W4V_ERR_CUDA;
        }
        configured_for = dev;
    }
    if (launch_pdl(paged_attn_kernel<D>, dim3(grid), dim3(kThreads), Plan<D>::kBytes, stream, qmap, kmap, vmap, a) !=
            cudaSuccess ||
        launch_pdl(paged_attn_join_kernel<D>, dim3(grid, kJoinSplit), dim3(kJoinThreads), 0, stream, a) != cudaSuccess) {
        cudaGetLastError();
        return W4V_ERR_CUDA;
    }
    return W4V_OK;
}

}  // namespace

size_t paged_attn_ws_bytes(int n_tokens, int B, int q_heads, int kv_heads, int head_dim, int max_context,
                           bool invariant) {
    const Slots s = slots_of(n_tokens, B, q_heads, kv_heads, max_context, invariant);
    return s.count * (s.rows * (size_t(head_dim) * sizeof(float) + sizeof(float2)) + sizeof(Share)) + 256;
}

w4v_status launch_paged_attn(const w4v_kv_t &kv, const uint16_t *q, long long q_stride, int n_tokens, int q_heads,
                             float scale, int window, uint16_t *out, float *lse, void *ws, bool invariant,
                             cudaStream_t stream) {
    const DeviceInfo *info = nullptr;
    w4v_status st = device_info(&info);
    if (st != W4V_OK) return st;
    const int D = kv.head_dim, group = q_heads / kv.kv_heads;
    const Slots slots = slots_of(n_tokens, kv.B, q_heads, kv.kv_heads, kv.table_width * kv.page, invariant);
    Args a;
    a.out = reinterpret_cast<__half *>(out);
    a.lse = lse;
    a.wide = (reinterpret_cast<uintptr_t>(out) & 31u) == 0u;
    a.part_o = reinterpret_cast<float *>((reinterpret_cast<uintptr_t>(ws) + 31u) & ~uintptr_t(31));
    a.part_ml = reinterpret_cast<float2 *>(a.part_o + slots.count * slots.rows * D);
    a.shares = reinterpret_cast<Share *>((reinterpret_cast<uintptr_t>(a.part_ml + slots.count * slots.rows) + 15u) & ~uintptr_t(15));
    a.v = reinterpret_cast<const __half *>(kv.v);
    a.table = kv.table;
    a.lengths = kv.lengths;
    a.offsets = kv.offsets;
    a.status = info->status;
    a.n_tokens = n_tokens;
    a.q_heads = q_heads;
    a.kv_heads = kv.kv_heads;
    a.group = group;
    a.tok = tokens_per_tile(q_heads, kv.kv_heads);
    a.group_mul = 65536 / group + 1;
    a.tok_shift = 31;
    while (1 << (a.tok_shift - 31) < a.tok) ++a.tok_shift;
    a.tok_mul = ((uint64_t(1) << a.tok_shift) + a.tok - 1) / a.tok;
    a.B = kv.B;
    a.width = kv.table_width;
    a.n_pages = kv.n_pages;
    a.page_bits = 0;
    while (1 << a.page_bits < kv.page) ++a.page_bits;
    a.back = window > 0 ? window - 1 : INT_MAX;
    a.slot_rows = slots.rows;
    a.invariant = invariant;
    a.unit_bits = invariant ? inv_tile_bits(kv.table_width * kv.page) : 0;
    a.part_cost = invariant ? 0 : kPartCost;
    a.max_units = uint32_t(std::min(invariant ? slots.count : size_t(INT_MAX), size_t(INT_MAX)) / kv.kv_heads);
    a.scale_log2 = scale * 1.4426950408889634f;
    // K and V as (64 elements, 8 tokens, blocks of a head, 8-token groups):
    // a box is a page's groups of one stage's blocks
    CUtensorMap qmap, kmap, vmap;
    const uint64_t row = uint64_t(D) * 2;
    const uint64_t kv_dims[4] = {64, 8, uint64_t(D) / 64, uint64_t(kv.n_pages) * kv.kv_heads * (kv.page / 8)};
    const uint64_t kv_strides[3] = {row, 128, 8 * row};
    const uint32_t kv_box[4] = {64, 8, D >= 128 ? 2u : 1u, uint32_t(std::min(kv.page, kKeys) / 8)};
    // Q as (64 elements, heads, tokens, blocks): a box is one block of a tile's rows
    const uint64_t q_dims[4] = {64, uint64_t(q_heads), uint64_t(n_tokens), uint64_t(D) / 64};
    const uint64_t q_strides[3] = {row, uint64_t(q_stride) * 2, 128};
    const uint32_t q_box[4] = {64, uint32_t(group), uint32_t(a.tok), 1};
    st = encode_tmap_sw128(&qmap, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, q, q_dims, q_strides, q_box);
    if (st == W4V_OK)
        st = encode_tmap_sw128(&kmap, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, kv.k, kv_dims, kv_strides, kv_box);
    if (st == W4V_OK)
        st = encode_tmap_sw128(&vmap, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, kv.v, kv_dims, kv_strides, kv_box);
    if (st != W4V_OK) return st;
    const int grid = std::min(info->sm_count, kMaxCtas);
    return D == 64 ? launch<64>(qmap, kmap, vmap, a, grid, stream)
                   : D == 128 ? launch<128>(qmap, kmap, vmap, a, grid, stream)
                              : launch<256>(qmap, kmap, vmap, a, grid, stream);
}

}  // namespace w4v
