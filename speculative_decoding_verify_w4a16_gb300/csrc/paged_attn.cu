// paged_attn.cu -- causal attention of new tokens over a paged cache.
//
// One pass over the keys with the running maximum and sum of the softmax:
// with x_j = scale log2(e) q . k_j, m a reference near the largest x so far,
// l = sum 2^(x_j - m) and o = sum 2^(x_j - m) v_j; a larger m rescales l and
// o by 2^(m_old - m).  The reference follows the maximum only when that has
// grown by more than kSlack, so o (in tensor memory) is seldom touched; the
// weights then reach 2^(kShift + kSlack) = 2^14, inside fp16, and keep full
// precision down to 2^-22 of the largest.
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
// Work: the unit is one tile's 128 keys.  All units in order (sequence,
// key/value head, row tile, keys) are dealt out evenly to one CTA per SM, so
// a long context at one row tile and a causal triangle of many both fill the
// GPU.  A CTA's range may begin and end inside a tile; such a part leaves o,
// m and l in the workspace (at most two parts a CTA), and a second kernel
// joins them, each boundary's CTA a share of the tile's rows.  The lengths
// are on the device, so each CTA finds its own range by a scan over the
// sequences.  With batch invariance the unit is a fixed range of keys, every
// one a part of its own: which keys meet in one running sum then depends on
// the row alone.
//
// A weight of 0 does not hide a value that is not finite (0 x inf is NaN),
// and within a tile some rows see keys that others must not.  Where a tile
// holds such keys, the issuer looks their values over before the product and
// clears what is not finite; the rows that do see it add it in the epilogue.
// A drafted token that overflowed thus spoils no position before it.
//
// Roles (12 warps): 0 producer (page ids, TMA), 1 MMA issuer, 2 schedule and
// tensor-memory owner, 3 idle, 4-11 softmax.  Softmax warps w and w + 4
// share 32 rows, 64 of the 128 columns each, and agree on the maximum
// through shared memory.  S is double buffered: the next tile's Q K^T runs
// under this one's softmax.
#include <algorithm>

#include "runtime.h"
#include "sm103_ptx.cuh"

namespace w4v {
namespace {

constexpr int kKeys = 128;                      // keys per tile
constexpr int kRows = 128;                      // rows per tile
constexpr int kThreads = 384;
constexpr int kWarpProd = 0, kWarpMma = 1, kWarpPlan = 2, kWarpSoft = 4;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kOcol = 256;                 // S buffers at columns 0 and 128
constexpr float kShift = 8.f, kSlack = 6.f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kInvTiles = 4;                    // least tiles of a batch-invariant part
constexpr int kInvParts = 32;                   // most parts of a row tile

template <int D>
struct Plan {
    static constexpr int kBlocks = D / 64;                       // 64-element blocks of a head
    static constexpr int kStageBlocks = D >= 128 ? 2 : 1;
    static constexpr int kHalves = kBlocks / kStageBlocks;       // stages per tile of K (or V)
    static constexpr int kGroupBytes = kStageBlocks * 1024;      // 8 tokens of a stage
    static constexpr int kStageBytes = kKeys / 8 * kGroupBytes;
    static constexpr int kQBytes = kBlocks * kRows * 128;
    static constexpr int kStages = D == 64 ? 11 : D == 128 ? 6 : 5;
    static constexpr int kBar = kQBytes + kStages * kStageBytes;
    static constexpr int kNumBars = 2 + 2 * kStages + 2 + 2 + 2 + 1;
    static constexpr int kMisc = kBar + 256;
    static constexpr int kMax = kBar + 512;                      // float[2][2][kRows]
    static constexpr int kBytes = kMax + 2 * 2 * kRows * 4;
    static_assert(8 * kNumBars <= 256 && kBytes <= 227 * 1024, "shared memory plan");
};

struct Args {
    __half *out;
    float *lse;
    float *part_o;              // [slots][slot_rows][D]
    float2 *part_ml;            // [slots][slot_rows]: m (log2), l
    const __half *v;            // the cache's values (rows that must be looked at again)
    const int32_t *table, *lengths, *offsets;
    uint32_t *status;
    int n_tokens, q_heads, kv_heads, group, tok;   // query heads per key/value head, tokens per tile
    int B, width, n_pages, page, window, slot_rows;
    int inv;                    // 0, or tiles per batch-invariant part
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
    s.len = min(max(p.lengths[b], 0), p.width * p.page);
    return s;
}

// Key tiles that row tile qt reads, and its units.
struct Extent {
    int lo, hi, units;          // tiles [lo, hi); a tile without keys is one unit
};
__device__ __forceinline__ Extent extent_of(const Args &p, const Seq &s, int qt) {
    const int t0 = qt * p.tok, t1 = min(s.n, t0 + p.tok) - 1;
    const int p0 = s.len - s.n + t0, p1 = s.len - s.n + t1;
    Extent e{0, 0, 1};
    if (p1 < 0) return e;
    e.lo = p.window > 0 ? max(0, p0 - p.window + 1) / kKeys : 0;
    e.hi = p1 / kKeys + 1;
    e.units = p.inv == 0 ? e.hi - e.lo : (e.hi - 1) / p.inv - e.lo / p.inv + 1;
    return e;
}

// Units of one key/value head of 32 sequences, one per lane (0 past the end).
__device__ int lane_units(const Args &p, int b) {
    const int lane = threadIdx.x & 31;
    Seq s{0, 0, 0};
    if (b < p.B) s = seq_of(p, b);
    const int tiles = (s.n + p.tok - 1) / p.tok;
    int u = tiles == 1 ? extent_of(p, s, 0).units : 0;
    for (uint32_t many = __ballot_sync(0xFFFFFFFFu, tiles > 1); many != 0; many &= many - 1) {
        const int src = __ffs(many) - 1;
        const Seq o{0, __shfl_sync(0xFFFFFFFFu, s.n, src), __shfl_sync(0xFFFFFFFFu, s.len, src)};
        const int ot = __shfl_sync(0xFFFFFFFFu, tiles, src);
        int sum = 0;
        for (int qt = lane; qt < ot; qt += 32) sum += extent_of(p, o, qt).units;
        sum = __reduce_add_sync(0xFFFFFFFFu, sum);
        if (lane == src) u = sum;
    }
    return u;
}

template <typename T>
__device__ __forceinline__ T warp_scan(T x) {
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const T y = __shfl_up_sync(0xFFFFFFFFu, x, d);
        if ((threadIdx.x & 31) >= d) x += y;
    }
    return x;
}

__device__ long long all_units(const Args &p) {
    long long sum = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) sum += lane_units(p, b0 + (threadIdx.x & 31));
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
    return sum * p.kv_heads;
}

struct Place {
    int b, kvh, qt, u;          // unit u of a row tile
};
// The place of unit `at` (one warp; at < all_units).
__device__ Place place_of(const Args &p, long long at) {
    const int lane = threadIdx.x & 31;
    Place w{0, 0, 0, 0};
    for (int b0 = 0; b0 < p.B; b0 += 32) {
        const int u = lane_units(p, b0 + lane);
        const long long upto = warp_scan((long long)u * p.kv_heads);
        const uint32_t past = __ballot_sync(0xFFFFFFFFu, upto > at);
        if (past == 0) {
            at -= __shfl_sync(0xFFFFFFFFu, upto, 31);
            continue;
        }
        const int src = __ffs(past) - 1;
        const int su = __shfl_sync(0xFFFFFFFFu, u, src);
        at -= __shfl_sync(0xFFFFFFFFu, upto, src) - (long long)su * p.kv_heads;
        w.b = b0 + src;
        w.kvh = int(at / su);
        int rest = int(at % su);
        const Seq s = seq_of(p, w.b);
        for (int q0 = 0;; q0 += 32) {
            const bool in = q0 + lane < (s.n + p.tok - 1) / p.tok;
            const int mine = in ? extent_of(p, s, q0 + lane).units : 0;
            const int sum = warp_scan(mine);
            const uint32_t over = __ballot_sync(0xFFFFFFFFu, sum > rest);
            if (over != 0 || q0 >= s.n) {
                const int l = over != 0 ? __ffs(over) - 1 : 0;
                w.qt = q0 + l;
                w.u = rest - __shfl_sync(0xFFFFFFFFu, sum - mine, l);
                break;
            }
            rest -= __shfl_sync(0xFFFFFFFFu, sum, 31);
        }
        break;
    }
    return w;
}

// A run of units of one row tile.
struct Part {
    Seq s;
    int b, kvh, t0, rows;       // first token, rows in use
    int kt0, nt;                // first key tile, key tiles
    int keys_end;               // keys that any of its rows sees end here
    int u, take, units;         // units [u, u + take) of the row tile's
};
struct Cursor {
    Place w;
    long long unit, left;       // index of the next unit, units left in the range
    Seq s;
    __device__ __forceinline__ void load(const Args &p) { s = seq_of(p, w.b); }
    __device__ __forceinline__ bool next(const Args &p, Part &g) {
        if (left <= 0) return false;
        const Extent e = extent_of(p, s, w.qt);
        g.s = s;
        g.b = w.b;
        g.kvh = w.kvh;
        g.t0 = w.qt * p.tok;
        const int toks = min(p.tok, s.n - g.t0);
        g.rows = toks * p.group;
        g.keys_end = max(s.len - s.n + g.t0 + toks, 0);
        g.u = w.u;
        g.units = e.units;
        if (p.inv == 0) {
            g.take = int(min((long long)(e.units - w.u), left));
            g.kt0 = e.lo + w.u;
            g.nt = e.hi > e.lo ? g.take : 0;
        } else {
            g.take = 1;
            const int c = (e.lo / p.inv + w.u) * p.inv;
            g.kt0 = max(e.lo, c);
            g.nt = max(min(e.hi, c + p.inv) - g.kt0, 0);
        }
        w.u += g.take;
        unit += g.take;
        left -= g.take;
        if (w.u == e.units) {
            w.u = 0;
            if ((w.qt + 1) * p.tok < s.n) {
                ++w.qt;
            } else {
                w.qt = 0;
                if (++w.kvh == p.kv_heads) {
                    w.kvh = 0;
                    if (left > 0) do {
                        ++w.b;
                        load(p);
                    } while (s.n == 0 && w.b < p.B - 1);
                }
            }
        }
        return true;
    }
};

// Whether none of eight fp16 values is infinite or NaN (exponent all ones).
__device__ __forceinline__ bool finite_halves(const uint4 &v) {
    auto carry = [](uint32_t w) { return (w & 0x7C007C00u) + 0x04000400u; };
    return ((carry(v.x) | carry(v.y) | carry(v.z) | carry(v.w)) & 0x80008000u) == 0u;
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
    auto kv_full = [&](int s) { return bar0 + 16u + 8u * s; };
    auto kv_empty = [&](int s) { return bar0 + 16u + 8u * (P::kStages + s); };
    const uint32_t tail = bar0 + 16u + 16u * P::kStages;
    auto s_full = [&](int i) { return tail + 8u * i; };
    auto p_full = [&](int i) { return tail + 16u + 8u * i; };
    auto pv_done = [&](int i) { return tail + 32u + 8u * i; };
    const uint32_t done_bar = tail + 48u;
    uint32_t *misc = reinterpret_cast<uint32_t *>(smem + P::kMisc);    // [0] tmem, [1] abort, [2..3] below
    volatile uint32_t *spoilt = misc + 2;                    // [i & 1]: part i (from 1) had values cleared
    volatile Cursor *start = reinterpret_cast<volatile Cursor *>(smem + P::kMisc + 16);
    float *xmax = reinterpret_cast<float *>(smem + P::kMax);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    AbortState ab{reinterpret_cast<volatile uint32_t *>(&misc[1]), p.status};

    if (threadIdx.x == 0) {
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        for (int s = 0; s < P::kStages; ++s) {
            mbar_init(kv_full(s), 1);
            mbar_init(kv_empty(s), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(s_full(i), 1);
            mbar_init(p_full(i), 8);             // the softmax warps
            mbar_init(pv_done(i), 2);            // the MMAs, and the issuer's own writes
        }
        mbar_init(done_bar, 1);
        misc[1] = misc[2] = misc[3] = 0;
        fence_barrier_init();
    }
    if (warp == kWarpPlan) {
        tmem_alloc(smem_u32(&misc[0]), kTmemCols);
        tmem_relinquish();
    }
    if (warp == kWarpProd && lane == 0) {
        prefetch_tensormap(&qmap);
        prefetch_tensormap(&kmap);
        prefetch_tensormap(&vmap);
    }
    grid_dep_wait();
    grid_dep_launch();
    if (warp == kWarpPlan) {
        const long long all = all_units(p);
        const long long ctas = min((long long)gridDim.x, all);
        Cursor c{};
        if (blockIdx.x < ctas) {
            c.unit = split_begin(blockIdx.x, all, ctas);
            c.left = split_begin(blockIdx.x + 1, all, ctas) - c.unit;
            c.w = place_of(p, c.unit);
        }
        if (lane == 0) {
            start->unit = c.unit;
            start->left = c.left;
            start->w.b = c.w.b;
            start->w.kvh = c.w.kvh;
            start->w.qt = c.w.qt;
            start->w.u = c.w.u;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = misc[0];
    Cursor cur;
    cur.unit = start->unit;
    cur.left = start->left;
    cur.w.b = start->w.b;
    cur.w.kvh = start->w.kvh;
    cur.w.qt = start->w.qt;
    cur.w.u = start->w.u;
    if (cur.left > 0) cur.load(p);
    Part g;
    bool ok = (base & 1023u) == 0u;              // the operands' swizzle needs it
    if (!ok && threadIdx.x == 0) raise_abort(ab);

    if (warp == kWarpProd) {
        const int box = min(p.page, kKeys);                  // tokens per TMA box
        const uint32_t box_bytes = uint32_t(box / 8) * P::kGroupBytes;
        const int boxes = kKeys / box;
        const int groups = p.page / 8;                       // 8-token groups of a page
        int it = 0, nq = 0;
        // this lane's page (box) of tile kt: its first 8-token group, or one
        // past the cache, which TMA fills with zeros
        auto group_of = [&](const Part &g, int kt) -> int {
            const int key = kt * kKeys + lane * box;
            if (lane >= boxes || key >= g.keys_end) return -1;
            const int id = p.table[size_t(g.b) * p.width + key / p.page];
            if (id < 0 || id >= p.n_pages) return p.n_pages * p.kv_heads * groups;
            return (id * p.kv_heads + g.kvh) * groups + (key % p.page) / 8;
        };
        auto load = [&](const CUtensorMap *map, int grp) {
            const uint32_t n = __popc(__ballot_sync(0xFFFFFFFFu, grp >= 0));
            for (int h = 0; h < P::kHalves && ok; ++h, ++it) {
                const int s = it % P::kStages;
                if (it >= P::kStages) ok = warp_wait(kv_empty(s), (it / P::kStages - 1) & 1, ab);
                if (!ok) break;
                if (lane == 0) mbar_arrive_expect_tx(kv_full(s), n * box_bytes);
                __syncwarp();
                if (grp >= 0)
                    tma_load_4d(base + P::kQBytes + s * P::kStageBytes + lane * box_bytes, map, 0, 0,
                                h * P::kStageBlocks, grp, kv_full(s));
            }
        };
        while (ok && cur.next(p, g)) {
            if (g.nt == 0) continue;
            int now = group_of(g, g.kt0), soon = g.nt > 1 ? group_of(g, g.kt0 + 1) : -1;
            if (nq > 0) ok = warp_wait(q_empty, (nq - 1) & 1, ab);
            if (!ok) break;
            if (lane == 0) mbar_arrive_expect_tx(q_full, P::kBlocks * p.tok * p.group * 128u);
            __syncwarp();
            if (lane < P::kBlocks)
                tma_load_4d(base + lane * kRows * 128, &qmap, 0, g.kvh * p.group, g.s.first + g.t0, lane, q_full);
            ++nq;
            load(&kmap, now);
            for (int j = 0; j < g.nt && ok; ++j) {
                const int after = j + 2 < g.nt ? group_of(g, g.kt0 + j + 2) : -1;
                if (j + 1 < g.nt) load(&kmap, soon);
                load(&vmap, now);
                now = soon;
                soon = after;
            }
        }
        if (*ab.flag) {                                      // copies in flight land before the CTA ends
            for (int i = max(0, it - P::kStages); i < it; ++i)
                mbar_wait_bounded(kv_full(i % P::kStages), (i / P::kStages) & 1);
            if (nq > 0) mbar_wait_bounded(q_full, (nq - 1) & 1);
        }
    } else if (warp == kWarpMma) {
        constexpr uint32_t idesc_s = idesc_f16_f32(kRows, kKeys);
        constexpr uint32_t idesc_o = idesc_f16_f32(kRows, 64 * P::kStageBlocks) | kIdescBMnMajor;
        const uint32_t st0 = base + P::kQBytes;
        int it = 0, nq = 0, t = 0;                           // stages, parts and tiles so far
        auto scores = [&](int tile) {                        // S[tile & 1] = Q K^T
            for (int h = 0; h < P::kHalves && ok; ++h, ++it) {
                const int s = it % P::kStages;
                ok = warp_wait(kv_full(s), (it / P::kStages) & 1, ab);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < 4 * P::kStageBlocks; ++k)
                    mma_f16_ss_lane0(tmem + (tile & 1) * kKeys,
                                     sdesc_sw128(base + (h * P::kStageBlocks + (k >> 2)) * (kRows * 128) + (k & 3) * 32),
                                     sdesc_sw128_stride(st0 + s * P::kStageBytes + (k >> 2) * 1024 + (k & 3) * 32,
                                                        P::kGroupBytes),
                                     idesc_s, h > 0 || k > 0);
                mma_commit_lane0(kv_empty(s));
            }
            if (ok) mma_commit_lane0(s_full(tile & 1));
        };
        while (ok && cur.next(p, g)) {
            if (g.nt == 0) continue;
            ok = warp_wait(q_full, nq & 1, ab);
            if (!ok) break;
            ++nq;
            tc_fence_after();
            scores(t);
            if (ok && g.nt == 1) mma_commit_lane0(q_empty);
            for (int j = 0; j < g.nt && ok; ++j, ++t) {
                if (j + 1 < g.nt) {
                    scores(t + 1);
                    if (ok && j + 2 == g.nt) mma_commit_lane0(q_empty);
                }
                // O += P V over the keys that some row sees.  While the
                // softmax runs: what the last 16 of them hold past those keys
                // (other tokens, nothing at all) is cleared, and so is what
                // is not finite among keys that only some rows see.
                const int key = (g.kt0 + j) * kKeys, seen = min(g.keys_end - key, kKeys), steps = (seen + 15) / 16;
                const int above = max(g.s.len - g.s.n + g.t0 + 1 - key, 0);          // the first row sees those before
                const int below = p.window > 0 ? min(g.keys_end - p.window - key, seen) : 0;   // the last row, those from
                if (seen < 16 * steps || above < seen || below > 0) {
                    bool found = false;
                    for (int h = 0; h < P::kHalves && ok; ++h) {
                        const int s = (it + h) % P::kStages;
                        const uint32_t st = st0 + s * P::kStageBytes;
                        ok = warp_wait(kv_full(s), ((it + h) / P::kStages) & 1, ab);
                        if (!ok) break;
                        constexpr int kPieces = P::kStageBlocks * 8;                 // 16-byte pieces of a token
                        auto piece = [&](int tok, int i) {
                            return st + (tok / 8) * P::kGroupBytes + (i / 8) * 1024 + (tok % 8) * 128 + (i % 8) * 16;
                        };
                        auto look = [&](int a, int b) {
                            for (int i = a * kPieces + lane; i < b * kPieces; i += 32) {
                                const uint32_t at = piece(i / kPieces, i % kPieces);
                                uint4 v = lds128(at);
                                if (finite_halves(v)) continue;
                                clear_not_finite(v);
                                sts_f32x4(at, __uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z),
                                          __uint_as_float(v.w));
                                found = true;
                            }
                        };
                        if (above < seen) look(above, seen);
                        if (below > 0) look(0, min(below, above));
                        for (int i = seen * kPieces + lane; i < 16 * steps * kPieces; i += 32)
                            sts_f32x4(piece(i / kPieces, i % kPieces), 0.f, 0.f, 0.f, 0.f);
                        fence_proxy_async_shared();
                    }
                    if (__any_sync(0xFFFFFFFFu, found)) spoilt[nq & 1] = nq;
                }
                if (ok) ok = warp_wait(p_full(t & 1), (t >> 1) & 1, ab);
                if (!ok) break;
                tc_fence_after();
                for (int h = 0; h < P::kHalves && ok; ++h, ++it) {
                    const int s = it % P::kStages;
                    const uint32_t st = st0 + s * P::kStageBytes;
                    ok = warp_wait(kv_full(s), (it / P::kStages) & 1, ab);
                    if (!ok) break;
                    tc_fence_after();
                    for (int k = 0; k < steps; ++k)
                        mma_f16_ts_lane0(tmem + kOcol + h * 64 * P::kStageBlocks, tmem + (t & 1) * kKeys + 8 * k,
                                         sdesc_sw128_mn(st + 2 * k * P::kGroupBytes, 1024, P::kGroupBytes), idesc_o,
                                         j > 0 || k > 0);
                    mma_commit_lane0(kv_empty(s));
                }
                if (ok) mma_commit_lane0(pv_done(t & 1));
                if (ok && lane == 0) mbar_arrive(pv_done(t & 1));
            }
        }
        mma_commit_lane0(done_bar);
        mbar_wait_bounded(done_bar, 0);
        __syncwarp();
    } else if (warp >= kWarpSoft) {
        const int half = (warp - kWarpSoft) >> 2, quad = warp & 3, row = 32 * quad + lane;
        const uint32_t lanes = uint32_t(32 * quad) << 16;
        const float c = p.scale_log2;
        constexpr int kCols = D / 2;                         // this warp's columns of O
        const uint32_t ocol = tmem + lanes + kOcol + half * kCols;
        int t = 0, np = 0;                                   // tiles and parts (with keys) so far
        while (ok && cur.next(p, g)) {
            np += g.nt > 0;
            const bool mine = row < g.rows;
            const bool busy = 32 * quad < g.rows;            // some row of this warp is in use
            const int tok = g.t0 + row / p.group;
            const int head = g.kvh * p.group + row % p.group;
            const int pos = g.s.len - g.s.n + tok;
            const int from = p.window > 0 ? pos - p.window + 1 : 0;
            // every key of [sure_lo, sure_hi] is seen by all of the warp's rows
            const int sure_hi = __reduce_min_sync(0xFFFFFFFFu, mine ? pos : 0x7FFFFFFF);
            const int sure_lo = __reduce_max_sync(0xFFFFFFFFu, mine ? from : 0);
            float m = -INFINITY, l = 0.f;                    // reference (in units of q . k), sum of this warp's half
            for (int j = 0; j < g.nt; ++j, ++t) {
                // tile t - 2's product is done by now (its MMAs were issued
                // before this tile's); seeing its phase keeps the later waits
                // on pv_done, two phases a barrier, unambiguous
                ok = warp_wait(s_full(t & 1), (t >> 1) & 1, ab) &&
                     (t < 2 || warp_wait(pv_done(t & 1), ((t >> 1) - 1) & 1, ab));
                if (!ok) break;
                if (!busy) {
                    if (lane == 0) mbar_arrive(p_full(t & 1));
                    continue;
                }
                tc_fence_after();
                uint32_t x[2][32];
                const uint32_t scol = tmem + lanes + (t & 1) * kKeys + half * 64;
                tmem_ld_32x32b_x32(scol, x[0]);
                tmem_ld_32x32b_x32(scol + 32, x[1]);
                tc_wait_ld_keep<32>(x[0]);
                tc_wait_ld_keep<32>(x[1]);
                const int key = (g.kt0 + j) * kKeys + half * 64;
                if (key + 63 > sure_hi || key < sure_lo) {
#pragma unroll
                    for (int i = 0; i < 64; ++i)
                        if (key + i > pos || key + i < from) x[i >> 5][i & 31] = 0xFF800000u;   // -inf
                }
                float top = -INFINITY;
#pragma unroll
                for (int i = 0; i < 64; ++i) top = fmaxf(top, __uint_as_float(x[i >> 5][i & 31]));
                // the row's maximum over both halves; past the barrier both
                // warps hold their scores in registers, so P may overwrite S
                xmax[((t & 1) * 2 + half) * kRows + row] = top;
                tc_fence_before();
                named_bar_sync(1 + quad, 64);
                tc_fence_after();
                top = fmaxf(top, xmax[((t & 1) * 2 + (half ^ 1)) * kRows + row]);
                if (*ab.flag) {
                    ok = false;
                    break;
                }
                const bool raise = mine && top > m && (m == -INFINITY || (top - m) * c > kSlack);
                if (__any_sync(0xFFFFFFFFu, raise)) {
                    const float a = raise ? ex2((m - top) * c) : 1.f;
                    if (raise) m = top;
                    l *= a;
                    if (j > 0) {
                        ok = warp_wait(pv_done((t - 1) & 1), ((t - 1) >> 1) & 1, ab);
                        if (!ok) break;
                        tc_fence_after();
#pragma unroll 1
                        for (int o = 0; o < kCols; o += 32) {
                            uint32_t r[32];
                            tmem_ld_32x32b_x32(ocol + o, r);
                            tc_wait_ld_keep<32>(r);
#pragma unroll
                            for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * a);
                            tmem_st_32x32b_x32(ocol + o, r);
                            tc_wait_st();
                            tc_keep_alive<32>(r);
                        }
                    }
                }
                const float off = m == -INFINITY ? 0.f : kShift - m * c;
                uint32_t w[32];
                float sum0 = 0.f, sum1 = 0.f;
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const float p0 = ex2(fmaf(__uint_as_float(x[(2 * i) >> 5][(2 * i) & 31]), c, off));
                    const float p1 = ex2(fmaf(__uint_as_float(x[(2 * i + 1) >> 5][(2 * i + 1) & 31]), c, off));
                    sum0 += p0;
                    sum1 += p1;
                    w[i] = h2_as_u32(__floats2half2_rn(p0, p1));
                }
                l += sum0 + sum1;
                tmem_st_32x32b_x32(tmem + lanes + (t & 1) * kKeys + half * 32, w);
                tc_wait_st();
                tc_keep_alive<32>(w);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full(t & 1));
            }
            if (!ok) {
                if (busy) named_bar_arrive(1 + quad, 64);    // the partner may wait there; it sees the flag after
                break;
            }
            if (g.nt > 0) {
                ok = warp_wait(pv_done((t - 1) & 1), ((t - 1) >> 1) & 1, ab);
                if (ok) tc_fence_after();
                if (busy) {
                    // the row's sum, lower half first
                    xmax[half * kRows + row] = l;
                    named_bar_sync(1 + quad, 64);
                    l = xmax[row] + xmax[kRows + row];
                    named_bar_sync(1 + quad, 64);            // read before the next tile's maxima are written
                    if (*ab.flag) ok = false;
                }
                if (!ok) break;
            }
            if (!busy) continue;
            const bool fix = g.nt > 0 && spoilt[np & 1] == np;
            const bool whole = g.take == g.units;
            const float inv = g.nt > 0 && l != 0.f ? 1.f / l : 0.f;
            const float m2 = m * c - kShift;
            const size_t slot = p.inv ? size_t(cur.unit - g.take) : 2 * size_t(blockIdx.x) + (g.u == 0);
            const size_t orow = size_t(g.s.first + tok) * p.q_heads + head;
            const size_t srow = slot * p.slot_rows + row;
            if (mine && half == 0) {
                if (!whole) p.part_ml[srow] = make_float2(m2, l);
                else if (p.lse != nullptr) p.lse[orow] = g.nt > 0 ? (m2 + log2f(l)) * kLn2 : -INFINITY;
            }
            __syncwarp();
#pragma unroll 1
            for (int o = 0; o < kCols; o += 32) {
                uint32_t r[32];
                if (g.nt > 0) {
                    tmem_ld_32x32b_x32(ocol + o, r);
                    tc_wait_ld_keep<32>(r);
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) r[i] = 0u;
                }
                if (fix && mine) {
                    // the values that were cleared, for a row that sees them
                    const int k0 = max(g.kt0 * kKeys, from), k1 = min((g.kt0 + g.nt) * kKeys - 1, pos);
                    const int above = g.s.len - g.s.n + g.t0 + 1, below = p.window > 0 ? g.keys_end - p.window : 0;
                    for (int k = k0; k <= k1; ++k) {
                        if (k >= below && k < above) k = above;          // seen by every row: not cleared
                        if (k > k1) break;
                        const int id = p.table[size_t(g.b) * p.width + k / p.page];
                        if (id < 0 || id >= p.n_pages) continue;
                        const uint16_t *v = reinterpret_cast<const uint16_t *>(p.v) +
                                            ((size_t(id) * p.kv_heads + g.kvh) * p.page + k % p.page) * D + half * kCols + o;
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if ((v[i] & 0x7C00u) == 0x7C00u)
                                r[i] = __float_as_uint(__uint_as_float(r[i]) + __half2float(__ushort_as_half(v[i])));
                    }
                }
                if (mine && whole) {
                    uint4 *dst = reinterpret_cast<uint4 *>(p.out + orow * D + half * kCols + o);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t h[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            h[e] = h2_as_u32(__floats2half2_rn(l != 0.f ? __uint_as_float(r[8 * i + 2 * e]) * inv : 0.f,
                                                              l != 0.f ? __uint_as_float(r[8 * i + 2 * e + 1]) * inv : 0.f));
                        dst[i] = make_uint4(h[0], h[1], h[2], h[3]);
                    }
                } else if (mine) {
                    uint4 *dst = reinterpret_cast<uint4 *>(p.part_o + srow * D + half * kCols + o);
#pragma unroll
                    for (int i = 0; i < 8; ++i) dst[i] = make_uint4(r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
                }
                __syncwarp();
            }
            tc_fence_before();
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == kWarpPlan) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// ---------------------------------------------------------- joining the parts
constexpr int kJoinThreads = 256;

// Rows [r0, r1) of a row tile from its parts, in order: slot(i), i < n.
template <int D, typename Slot>
__device__ void join_rows(const Args &p, const Part &g, int r0, int r1, int n, Slot slot, float *weights) {
    __syncthreads();                                         // weights may still be read
    for (int r = r0 + int(threadIdx.x >> 5); r < r1; r += kJoinThreads / 32) {
        const int lane = threadIdx.x & 31;
        float top = -INFINITY, l = 0.f;
        for (int i = lane; i < n; i += 32) top = fmaxf(top, __ldcg(&p.part_ml[slot(i) * p.slot_rows + r]).x);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
        for (int i0 = 0; i0 < n; i0 += 32) {
            const int i = i0 + lane;
            float w = 0.f, wl = 0.f;
            if (i < n) {
                const float2 ml = __ldcg(&p.part_ml[slot(i) * p.slot_rows + r]);
                w = top == -INFINITY ? 0.f : ex2(ml.x - top);
                wl = ml.y == 0.f ? 0.f : w * ml.y;
            }
            // in order, so that parts which add nothing change nothing
            for (int k = 0; k < min(32, n - i0); ++k) l += __shfl_sync(0xFFFFFFFFu, wl, k);
            if (i < n) weights[(r - r0) * n + i] = w;
        }
        const float inv = l != 0.f ? 1.f / l : 0.f;
        if (lane == 0) {
            weights[(r1 - r0) * n + (r - r0)] = inv;
            if (p.lse != nullptr)
                p.lse[size_t(g.s.first + g.t0 + r / p.group) * p.q_heads + g.kvh * p.group + r % p.group] =
                    l != 0.f ? (top + log2f(l)) * kLn2 : -INFINITY;
        }
    }
    __syncthreads();
    constexpr int kLanes = D / 4;                            // threads per row, four columns each
    for (int r = r0 + int(threadIdx.x) / kLanes; r < r1; r += kJoinThreads / kLanes) {
        const int col = 4 * (int(threadIdx.x) % kLanes);
        const float *w = weights + (r - r0) * n;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        constexpr int kAhead = 8;
        for (int i0 = 0; i0 < n; i0 += kAhead) {
            float4 v[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                if (i0 + k < n)
                    v[k] = __ldcg(reinterpret_cast<const float4 *>(p.part_o + (slot(i0 + k) * p.slot_rows + r) * D + col));
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                if (i0 + k < n && w[i0 + k] != 0.f) {
                    o.x = fmaf(w[i0 + k], v[k].x, o.x);
                    o.y = fmaf(w[i0 + k], v[k].y, o.y);
                    o.z = fmaf(w[i0 + k], v[k].z, o.z);
                    o.w = fmaf(w[i0 + k], v[k].w, o.w);
                }
        }
        const float inv = weights[(r1 - r0) * n + (r - r0)];
        const size_t orow = size_t(g.s.first + g.t0 + r / p.group) * p.q_heads + g.kvh * p.group + r % p.group;
        uint2 h;
        h.x = h2_as_u32(inv != 0.f ? __floats2half2_rn(o.x * inv, o.y * inv) : __floats2half2_rn(0.f, 0.f));
        h.y = h2_as_u32(inv != 0.f ? __floats2half2_rn(o.z * inv, o.w * inv) : __floats2half2_rn(0.f, 0.f));
        *reinterpret_cast<uint2 *>(p.out + orow * D + col) = h;
    }
}

// One CTA per boundary between two ranges (batch invariance: the same ranges
// of units), each a share of the rows of the tile that it cuts.
template <int D>
__global__ void __launch_bounds__(kJoinThreads)
paged_attn_join_kernel(const Args p, int ranges) {
    // rows of a share times parts, and a factor per row: at most
    // (rows / (n - 1) + 1) (n + 1) with n >= 2 parts
    __shared__ float weights[3 * kRows + 3 + 2 * kMaxCtas];
    __shared__ Cursor start;
    __shared__ long long total;
    grid_dep_launch();
    // the sequences' sizes were final before the kernel in front of this one began
    if (threadIdx.x < 32) {
        const long long all = all_units(p);
        const long long ctas = min((long long)ranges, all);
        const long long c = blockIdx.x + (p.inv ? 0 : 1);
        Cursor s{};
        if (c < ctas) {
            s.unit = split_begin(c, all, ctas);
            s.left = split_begin(c + 1, all, ctas) - s.unit;
            s.w = place_of(p, s.unit);
        }
        if (threadIdx.x == 0) {
            start = s;
            total = all;
        }
    }
    __syncthreads();
    Cursor cur = start;
    if (cur.left > 0) cur.load(p);
    grid_dep_wait();                                         // every CTA: who waits for this grid waits for the one before
    if (cur.left <= 0) return;
    Part g;
    if (p.inv == 0) {
        const long long ctas = min((long long)ranges, total);
        const long long at = cur.unit;
        cur.next(p, g);
        if (g.u == 0) return;                                // the boundary lies between two tiles
        const int first = split_owner(at - g.u, total, ctas), last = split_owner(at - g.u + g.units - 1, total, ctas);
        const int m = last - first, i = int(blockIdx.x) + 1 - first - 1;
        join_rows<D>(p, g, i * g.rows / m, (i + 1) * g.rows / m, m + 1,
                     [&](int k) { return 2 * size_t(first + k) + (k == 0); }, weights);
    } else {
        while (cur.next(p, g)) {
            if (g.units == 1) continue;
            const size_t s0 = size_t(cur.unit - 1 - g.u);
            join_rows<D>(p, g, g.u * g.rows / g.units, (g.u + 1) * g.rows / g.units, g.units,
                         [&](int k) { return s0 + k; }, weights);
        }
    }
}

// -------------------------------------------------------------------- the host
int tokens_per_tile(int q_heads, int kv_heads) { return kRows / (q_heads / kv_heads); }

// Tiles of a batch-invariant part: by the table's width alone, so that it is
// the same in every call on a cache.
int inv_tiles(int max_context) {
    const int tiles = (max_context + kKeys - 1) / kKeys;
    return std::max(kInvTiles, (tiles + kInvParts - 1) / kInvParts);
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
        const int keys = inv_tiles(max_context) * kKeys;
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
        launch_pdl(paged_attn_join_kernel<D>, dim3(a.inv ? grid : std::max(grid - 1, 1)), dim3(kJoinThreads), 0,
                   stream, a, grid) != cudaSuccess) {
        cudaGetLastError();
        return W4V_ERR_CUDA;
    }
    return W4V_OK;
}

}  // namespace

size_t paged_attn_ws_bytes(int n_tokens, int B, int q_heads, int kv_heads, int head_dim, int max_context,
                           bool invariant) {
    const Slots s = slots_of(n_tokens, B, q_heads, kv_heads, max_context, invariant);
    return s.count * s.rows * (size_t(head_dim) * sizeof(float) + sizeof(float2)) + 256;
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
    a.part_o = static_cast<float *>(ws);
    a.part_ml = reinterpret_cast<float2 *>(a.part_o + slots.count * slots.rows * D);
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
    a.B = kv.B;
    a.width = kv.table_width;
    a.n_pages = kv.n_pages;
    a.page = kv.page;
    a.window = window;
    a.slot_rows = slots.rows;
    a.inv = invariant ? inv_tiles(kv.table_width * kv.page) : 0;
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
