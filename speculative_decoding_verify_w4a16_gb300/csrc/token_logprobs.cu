// token_logprobs.cu -- log probabilities of given tokens, the rows' entropy
// and their most likely tokens, from the lm_head's logits.
//
// With y_v = (x_v - m) log2(e) / temperature, m a reference near a row's largest
// logit,
//     s = sum_v 2^y_v,  t = sum_v y_v 2^y_v:
//     log p_v = (x_v - m) / temperature - ln s,   entropy = ln s - ln 2 t / s.
// (t in the exponents' unit: in the logits' own, large ones overflow it.)
// One pass: each logit is read once.  A thread has its own reference, the
// largest of its first 16 logits, which it raises (s and t rescaled) when a
// logit is more than a factor 2^kSlack above it, so nothing waits for a
// maximum, and ln s stays so small that log probabilities near 0 keep their
// digits.  The references meet at the end: t becomes w (t + y s), y the
// exponent of w.
// Sums of 64 terms a thread are added up with what each addition rounds off
// (Kahan), so that their error does not grow with V (equal terms, whose roundings
// do not average out, were off by 7e-5 of s at 2^26 logits; for it 2048 rows of
// 151,936 with five alternatives take 194 us against 191).
//
// A row is one CTA's, or with few rows cut over the CTAs of a cluster, joined
// by the first of them through distributed shared memory: no workspace, no
// second launch, no atomics between CTAs.
//
// The `top` largest, ties to the lower index, without sorting.  The threads in
// 64 groups: the top-th largest of the groups' largest logits is a bound that
// at least `top` logits reach, and few exceed where they lie without order.
// A CTA's first loads give such a bound.  From then on a thread looks whether
// its 16 next logits' largest, which it has anyway, is above it (a logit equal
// to it comes too late, by its index), and if so notes the batch; CTAs of 128
// threads, whose first loads are few, take a closer bound whenever the logits
// seen have doubled.  At the end the groups' largest of all logits give the last
// bound; the noted batches that reach it, some 25, are read once more, and the
// logits that reach it count how many are above them.  (Collecting logits on the
// way instead of notes cost 100 instructions a batch.)  Where more come than
// there is room for (a row in ascending order, one of few different values), the
// row is gone through once more, a batch of every thread at a time.
//
// Measured (one GB300, device time; bound: the logits' bytes at 6.78 TB/s):
//   1 row of 151,936                          4.7 us (0.1: latency); with 20 alternatives 9.3
//   300 rows of 50,001 fp16, masked, 20       15.3 us (4.4: latency of a row's ends)
//   2048 rows of 151,936, 5                   194 us (184: bytes, 6.4 TB/s); none 172, 20 200
// What bounds it: the bytes.  The powers, at 16 a clock and SM, take a third of
// the time that 4-byte logits take from HBM.
#include <climits>

#include "runtime.h"
#include "sm103_ptx.cuh"

namespace w4v {
namespace {

constexpr int kBatch = 16;                      // logits of a thread that are looked at together
constexpr float kSlack = 2.f, kLn2 = 0.6931471805599453f;
constexpr int kGroups = 64;
constexpr int kMost = kLogprobsMaxTop;
static_assert(kMost <= kGroups, "the bound is a group's largest");
constexpr int kMaxCluster = 8;
// CTAs of 128 threads, eight an SM, for vocabularies up to kSmall (2048 rows of
// 1024: 14 us against 51) and from kManyRows rows an SM on, where the others'
// loads cover what a CTA does at a row's ends (2048 rows of 151,936 with five
// alternatives 194 against 208 us; 700 rows with twenty 91 against 84).  With
// fewer rows CTAs of 512, two an SM.
constexpr int kSmall = 8192, kManyRows = 8;

struct Args {
    const void *logits;
    long long stride;
    const int32_t *tokens;
    float *logprobs, *entropy, *top_logprobs;
    int32_t *top_ids;
    int V, n, top, cluster_bits;
    float heat, heat_log2;                      // 1 / temperature, and times log2(e)
    float slack;                                // kSlack in units of the logits
};

// Larger for a larger logit, then for a lower index; NaN counts as -inf and -0
// as 0, as in the argmax.  0 is below every key.
__device__ __forceinline__ uint64_t key_of(float x, int index) {
    if (!(x > -INFINITY)) x = -INFINITY;
    if (x == 0.f) x = 0.f;
    const uint32_t b = __float_as_uint(x);
    return uint64_t(b & 0x80000000u ? ~b : b | 0x80000000u) << 32 | uint32_t(~uint32_t(index));
}
__device__ __forceinline__ float logit_of(uint64_t key) {
    const uint32_t u = uint32_t(key >> 32);
    return __uint_as_float(u & 0x80000000u ? u & 0x7FFFFFFFu : ~u);
}
__device__ __forceinline__ int index_of(uint64_t key) { return int(~uint32_t(key)); }

__device__ __forceinline__ uint64_t ld_cluster_u64(uint32_t addr) {
    uint64_t v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
    return v;
}

// Sums by a reference: m the largest logit, s and t by it (0 where m = -inf).
struct Sums {
    float m, s, t;
};
__device__ __forceinline__ Sums join(const Sums &a, const Sums &b, float heat_log2) {
    const float m = fmaxf(a.m, b.m);
    Sums r{m, 0.f, 0.f};
    // Without a logit above -inf a side is s = t = 0, or NaN, which stays.  A
    // weight of 0 leaves t's term out: the exponent may be infinite.
    auto add = [&](const Sums &x) {
        const float y = (x.m - m) * heat_log2, w = x.m == -INFINITY ? 1.f : ex2(y);
        r.s += w * x.s;
        if (x.m > -INFINITY && w != 0.f) r.t += w * (x.t + y * x.s);
    };
    add(a);
    add(b);
    return r;
}

// Long sums s and t, and what their last additions rounded off, which the next
// ones make up for (Kahan): however many terms follow, they are off by little more
// than their last bit.
struct __align__(16) Long {
    float s, s_rest, t, t_rest;
    __device__ __forceinline__ void add(float ds, float dt) {
        const float ys = __fadd_rn(ds, s_rest), yt = __fadd_rn(dt, t_rest);
        const float next_s = __fadd_rn(s, ys), next_t = __fadd_rn(t, yt);
        s_rest = __fsub_rn(ys, __fsub_rn(next_s, s));
        t_rest = __fsub_rn(yt, __fsub_rn(next_t, t));
        s = next_s;
        t = next_t;
    }
};

template <typename T>
struct Vec;                                     // 16 bytes of logits
template <>
struct Vec<float> {
    static constexpr int kCount = 4;
    static constexpr uint32_t kLowest = 0xFF800000u;             // -inf
    static __device__ __forceinline__ void get(const uint4 &w, float *x) {
        x[0] = __uint_as_float(w.x);
        x[1] = __uint_as_float(w.y);
        x[2] = __uint_as_float(w.z);
        x[3] = __uint_as_float(w.w);
    }
    static __device__ __forceinline__ float one(const float *p) { return *p; }
};
template <>
struct Vec<__half> {
    static constexpr int kCount = 8;
    static constexpr uint32_t kLowest = 0xFC00FC00u;
    static __device__ __forceinline__ void get(const uint4 &w, float *x) {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(u32_as_h2(u[i]));
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    }
    static __device__ __forceinline__ float one(const __half *p) { return __half2float(*p); }
};

// A batch whose largest logit may be among the row's `top`.
struct Note {
    float most;
    int first;                                  // see collect()
};
template <int kThreads>
struct __align__(16) Shared {
    static constexpr int kLanes = kThreads / kGroups, kWarps = kThreads / 32;
    static constexpr int kTies = kThreads < 256 ? kThreads : 256;
    // What a batch of every thread may add: all of 31 groups, what is equal to
    // the bound, what was there.
    static constexpr int kList = ((kMost - 1) * kLanes * kBatch + kTies + kMost + 127) / 128 * 128;
    static constexpr int kKeys = 2 * kThreads, kNotes = kList - kKeys;
    union {
        uint64_t list[kList];
        struct {
            uint64_t keys[kKeys];               // (the list's begin)
            Note notes[kNotes];
        };
    };
    uint64_t ties[kTies];
    uint64_t best[kMost];                       // the CTA's largest, in order (0: none)
    uint64_t group_key[kGroups], bound_key;
    float group[2][kGroups], bound[2];          // by turns
    Long sums[kThreads >= 512 ? kThreads : 1];  // see token_logprobs_kernel()
    Sums warp[kWarps], all;
    // Keys in the list, those equal to a bound, noted batches.  Counted up by
    // whoever adds one, cleared by thread 0; they are read only behind a barrier
    // that follows the last write, and written again only behind one that follows
    // the reads.  How long the list is goes on as a value from there.
    int n, n_ties, n_notes;
    int scan[kWarps];
};
static_assert(sizeof(Shared<512>) <= 48 * 1024 && sizeof(Note) == sizeof(uint64_t), "static shared memory");

// Of the groups' values, how many are larger than this thread's group's, and
// how many as large (the lanes of a group share the work).
template <int kLanes, typename K>
__device__ __forceinline__ int2 groups_above(const K *group, K mine) {
    int2 n = make_int2(0, 0);
#pragma unroll
    for (int k = 0; k < kGroups; k += kLanes) {
        const K o = group[k + int(threadIdx.x) % kLanes];
        n.x += o > mine;
        n.y += o >= mine;
    }
#pragma unroll
    for (int d = 1; d < kLanes; d <<= 1) {
        n.x += __shfl_xor_sync(0xFFFFFFFFu, n.x, d);
        n.y += __shfl_xor_sync(0xFFFFFFFFu, n.y, d);
    }
    return n;
}

// The top-th largest of the groups' largest logits, `most` this thread's.
// Every thread calls it, with another `turn` than the last time; two barriers.
template <int kThreads>
__device__ __forceinline__ float bound_of_groups(Shared<kThreads> &sh, float most, int top, int turn) {
    constexpr int kLanes = Shared<kThreads>::kLanes;
#pragma unroll
    for (int d = 1; d < kLanes; d <<= 1) most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, d));
    if (threadIdx.x % kLanes == 0) sh.group[turn][threadIdx.x / kLanes] = most;
    __syncthreads();
    const int2 n = groups_above<kLanes>(sh.group[turn], most);
    if (n.x < top && top <= n.y) sh.bound[turn] = most;          // (several groups: the same value)
    __syncthreads();
    return sh.bound[turn];
}

// sh.best: the `top` largest of sh.list[0 .. n), in order; n < top: all, then 0.
// Begins and ends with a barrier.
template <int kThreads>
__device__ __noinline__ void best_of_list(Shared<kThreads> &sh, int top, int n) {
    constexpr int kLanes = Shared<kThreads>::kLanes;
    const int tid = threadIdx.x;
    __syncthreads();
    const uint64_t *list = sh.list;
    if (n > 4 * kMost) {
        // those that reach the top-th of the groups' largest
        uint64_t g = 0;
        for (int i = tid; i < n; i += kThreads) g = max(g, sh.list[i]);
#pragma unroll
        for (int d = 1; d < kLanes; d <<= 1) g = max(g, __shfl_xor_sync(0xFFFFFFFFu, g, d));
        if (tid % kLanes == 0) sh.group_key[tid / kLanes] = g;
        if (tid == 0) sh.n_ties = 0;             // (collect()'s was read before this function's first barrier)
        __syncthreads();
        const int2 above = groups_above<kLanes>(sh.group_key, g);
        if (above.x < top && top <= above.y) sh.bound_key = g;
        __syncthreads();
        const uint64_t bound = sh.bound_key;
        if (g >= bound)
            for (int i = tid; i < n; i += kThreads) {
                const uint64_t key = sh.list[i];
                if (key < bound || key == 0) continue;
                const int at = atomicAdd(&sh.n_ties, 1);
                if (at < Shared<kThreads>::kTies) sh.ties[at] = key;
            }
        __syncthreads();                         // every tie is counted; the last barrier parts this read from collect()
        if (sh.n_ties <= Shared<kThreads>::kTies) {
            list = sh.ties;
            n = sh.n_ties;
        }
    }
    if (n < top) {                               // else every place is written
        if (tid < kMost) sh.best[tid] = 0;
        __syncthreads();
    }
    // each counts those above it, two threads a key
    for (int i = tid / 2; i < (n + 15) / 16 * 16; i += kThreads / 2) {       // (whole warps)
        const uint64_t key = i < n ? list[i] : 0;
        int place = 0;
        for (int o = tid & 1; o < n; o += 2) place += list[o] > key;
        place += __shfl_xor_sync(0xFFFFFFFFu, place, 1);
        if (i < n && (tid & 1) == 0 && place < top) sh.best[place] = key;
    }
    __syncthreads();
}

// The first `want` of the batch's logits that equal `value`, in order of their
// index, to sh.list[n ...]; returns how many (x, first, limit: see collect()).
// Every thread calls it; ends with a barrier.
template <int W, int kThreads>
__device__ __forceinline__ int in_order(Shared<kThreads> &sh, const float (&x)[kBatch], float value, int first, int limit,
                                        int n, int want) {
    constexpr int kWarps = Shared<kThreads>::kWarps;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto index_of_logit = [&](int k) { return first + k / W * (kThreads * W) + k % W; };
    auto equal = [&](int k) {
        const int i = index_of_logit(k);
        return i >= 0 && i < limit && (value == -INFINITY ? !(x[k] > -INFINITY) : x[k] == value);
    };
    int found = 0;
#pragma unroll
    for (int r = 0; r < kBatch; r += W) {
        if (found >= want) continue;                             // the same for all threads
        int mine = 0;
#pragma unroll
        for (int j = 0; j < W; ++j) mine += equal(r + j);
        int upto = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(0xFFFFFFFFu, upto, d);
            if (lane >= d) upto += y;
        }
        __syncthreads();
        if (lane == 31) sh.scan[warp] = upto;
        __syncthreads();
        int at = found + upto - mine, all = 0;
        for (int o = 0; o < kWarps; ++o) {
            if (o < warp) at += sh.scan[o];
            all += sh.scan[o];
        }
#pragma unroll
        for (int j = 0; j < W; ++j)
            if (equal(r + j)) {
                if (at < want) sh.list[n + at] = key_of(x[r + j], index_of_logit(r + j));
                ++at;
            }
        found += all;
    }
    __syncthreads();
    return min(found, want);
}

// A batch of every thread: logit k of a thread has index first + k / W * kThreads
// * W + k % W, and is there at all where that is in [0, limit) (else it reads
// -inf).  Those that may be among the `top` largest go behind the sh.n keys in
// sh.list; returns how many are there then, to every thread (sh.n is not kept up).
// Every thread calls it; begins and ends with a barrier.
template <int W, int kThreads>
__device__ __noinline__ int collect(Shared<kThreads> &sh, const float (&x)[kBatch], float most, int first, int limit, int top) {
    const int tid = threadIdx.x;
    if (tid == 0) sh.n_ties = 0;                 // (last read before best_of_list()'s last barrier)
    __syncthreads();
    const float bound = bound_of_groups(sh, most, top, 0);
    const int before = sh.n;                     // written before the barriers above
    __syncthreads();                             // read by all: from here on it grows
    if (most >= bound && most > -INFINITY)
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            if (!(x[k] >= bound) || !(x[k] > -INFINITY)) continue;
            const uint64_t key = key_of(x[k], first + k / W * (kThreads * W) + k % W);
            if (x[k] > bound) {
                sh.list[atomicAdd(&sh.n, 1)] = key;
            } else {
                const int at = atomicAdd(&sh.n_ties, 1);
                if (at < Shared<kThreads>::kTies) sh.ties[at] = key;
            }
        }
    __syncthreads();                             // all are counted
    const int n = sh.n;
    int add = sh.n_ties;
    if (add <= Shared<kThreads>::kTies && bound > -INFINITY) {
        if (tid < add) sh.list[n + tid] = sh.ties[tid];
    } else {
        add = in_order<W>(sh, x, bound, first, limit, n, max(top - (n - before), 0));
    }
    __syncthreads();
    return n + add;
}

template <typename T, bool kTop, int kThreads>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads)
token_logprobs_kernel(const Args p) {
    using Sh = Shared<kThreads>;
    __shared__ Sh sh;
    constexpr int W = Vec<T>::kCount, kRows = kBatch / W;        // vectors of a batch
    // 16-byte loads of a thread in flight.  More of them spill with alternatives
    // (2048 rows: 208 us with 4, 220 with 8; without 186 and 176).
    constexpr int kLoads = kTop ? 4 : 8;
    constexpr int kWarps = Sh::kWarps;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cluster = 1 << p.cluster_bits, rank = int(blockIdx.x) & (cluster - 1), row = int(blockIdx.x) >> p.cluster_bits;
    grid_dep_wait();
    grid_dep_launch();
    // Vectors of 16 bytes from the boundary at or before the row's first logit:
    // vector v holds logits v W - shift ...  Whole ones are dealt out; the few
    // logits at the row's ends are a thread's each, of the first CTA.
    const T *x0 = static_cast<const T *>(p.logits) + row * p.stride;
    const int shift = int(reinterpret_cast<uintptr_t>(x0) & 15u) / int(sizeof(T));
    const uint4 *base = reinterpret_cast<const uint4 *>(x0 - shift);
    const int whole0 = shift > 0, whole1 = max(int((unsigned(p.V) + shift) / W), whole0);    // whole vectors: [whole0, whole1)
    const int each = (whole1 - whole0 + cluster - 1) >> p.cluster_bits;
    const int begin = min(whole0 + rank * each, whole1), end = min(begin + each, whole1);
    const int limit = end * W - shift;                           // the dealt logits of this CTA end here
    const int head = min(whole0 * W - whole0 * shift, p.V), tail = max(whole1 * W - shift, head);
    const int at_end = rank == 0 ? (tid < head ? tid : tail + tid - head < p.V ? tail + tid - head : -1) : -1;

    Sums mine{-INFINITY, 0.f, 0.f};
    // s and t of this thread: of the last kFold rounds of loads, here, and of all before
    constexpr int kFold = 8 * kRows / kLoads;    // (64 additions in a chain)
    float2 s = make_float2(0.f, 0.f), t = make_float2(0.f, 0.f);
    // (fp16 logits with alternatives, 512 threads: in shared memory, for in registers
    // they spill where it counts, 300 masked rows 17.3 us against 14.5; elsewhere in
    // registers, 400 rows of 151,936 55.4 against 56.3)
    constexpr bool kFar = kTop && kThreads >= 512 && sizeof(T) == 2;
    Long here;
    Long &all = kFar ? sh.sums[kFar ? tid : 0] : here;
    all = Long{0.f, 0.f, 0.f, 0.f};
    auto fold = [&] {
        Long x = all;
        x.add(s.x + s.y, t.x + t.y);
        all = x;
        s = t = make_float2(0.f, 0.f);
    };
    // The thread's sums by a larger reference (none so far: they are 0, or NaN, which
    // stays).  This rounds without making up for it: what was there shrinks to a
    // quarter or less, so it happens few times to sums that still count.
    auto raise = [&](float to) {
        if (mine.m > -INFINITY) {
            const Long x = all;
            const float old_s = x.s + (s.x + s.y + x.s_rest), old_t = x.t + (t.x + t.y + x.t_rest);
            const float y = (mine.m - to) * p.heat_log2, a = ex2(y);
            all = Long{a * old_s, 0.f, a == 0.f ? 0.f : a * (old_t + y * old_s), 0.f};
            s = t = make_float2(0.f, 0.f);
        }
        mine.m = to;
    };
    float bound = -INFINITY, most = -INFINITY;
    bool again = false;                          // the row once more, every batch collected by all
    int listed = p.top;                          // keys in sh.list at the end (gone through again: each batch leaves top)
    // Where the loop next stops for what is not done every round: folding the sums,
    // and for CTAs of 128 threads a closer bound after 2, 4, 8, ... rounds.  (One
    // comparison for both: a second one cost 3% of a round.)
    constexpr int kRound = kThreads * kLoads;
    constexpr bool kRenew = kTop && kThreads < 512;
    int pause = begin + (kRenew ? 2 : kFold) * kRound, turn = 1;
    const float edge = at_end >= 0 ? Vec<T>::one(x0 + at_end) : -INFINITY;
    if (kTop) {
        if (tid == 0) sh.n = sh.n_notes = 0;
        __syncthreads();                         // the counts are 0 before anyone adds
    }
    for (;;) {
        if (kTop && at_end >= 0) sh.list[atomicAdd(&sh.n, 1)] = key_of(edge, at_end);          // (14 at most)
        // (a vector's room is filled again as soon as it is done with)
        uint4 w[kLoads];
        auto fetch = [&](int v) {
            return v < end ? base[v] : make_uint4(Vec<T>::kLowest, Vec<T>::kLowest, Vec<T>::kLowest, Vec<T>::kLowest);
        };
#pragma unroll
        for (int i = 0; i < kLoads; ++i) w[i] = fetch(begin + i * kThreads + tid);
        for (int v0 = begin; v0 == begin || v0 < end; v0 += kRound) {
            const bool opening = kTop && !again && v0 == begin;
            if (opening) {
                float x[W];
#pragma unroll
                for (int i = 0; i < kLoads; ++i) {
                    Vec<T>::get(w[i], x);
#pragma unroll
                    for (int k = 0; k < W; k += 2) most = max3(most, x[k], x[k + 1]);
                }
                bound = bound_of_groups(sh, most, p.top, 0);
            }
            if (v0 == pause) {                   // (never in the second pass: every one was met in the first)
                fold();
                const int rounds = (v0 - begin) / kRound;
                pause += (kRenew ? min(rounds, kFold) : kFold) * kRound;
                if (kRenew && (rounds & (rounds - 1)) == 0) {
                    bound = bound_of_groups(sh, most, p.top, turn);
                    turn ^= 1;
                }
            }
#pragma unroll
            for (int b = 0; b < kLoads; b += kRows) {
                if (b > 0 && v0 + b * kThreads >= end) break;
                float x[kBatch];
#pragma unroll
                for (int i = 0; i < kRows; ++i) Vec<T>::get(w[b + i], x + i * W);
                auto refill = [&] {
#pragma unroll
                    for (int i = 0; i < kRows; ++i) w[b + i] = fetch(v0 + (kLoads + b + i) * kThreads + tid);
                };
                float top = x[0];
#pragma unroll
                for (int k = 1; k < kBatch - 1; k += 2) top = max3(top, x[k], x[k + 1]);
                top = max3(top, x[kBatch - 1], -INFINITY);
                const int first = (v0 + b * kThreads + tid) * W - shift;
                if (kTop && (again || (opening && b == 0 && bound == -INFINITY))) {
                    float y[kBatch];                             // (a copy, so that x itself stays in registers)
#pragma unroll
                    for (int k = 0; k < kBatch; ++k) y[k] = x[k];
                    if (again) {
                        best_of_list(sh, p.top, collect<W>(sh, y, top, first, limit, p.top));
                        if (tid < p.top) sh.list[tid] = sh.best[tid];
                        if (tid == 0) sh.n = p.top;          // for the next collect(), whose barriers come before its read
                        refill();
                        continue;
                    }
                    // Few groups hold a token above -inf, so the first batch has
                    // all those of -inf that may be wanted (or it is all there is).
                    const int before = sh.n;                 // the row's ends, counted before the bound's barriers
                    __syncthreads();
                    const int n = in_order<W>(sh, y, -INFINITY, first, limit, before, p.top);
                    if (tid == 0) sh.n = before + n;         // (next used behind the last bound's barriers)
                }
                if (kTop) {
                    most = fmaxf(most, top);
                    if (top > bound || (opening && top == bound && bound > -INFINITY)) {
                        const int at = atomicAdd(&sh.n_notes, 1);
                        if (at < Sh::kNotes) sh.notes[at] = Note{top, first};
                    }
                }
                if (top > mine.m + p.slack || (mine.m == -INFINITY && top > -INFINITY)) raise(top);
                const float ref = mine.m == -INFINITY ? 0.f : mine.m;
                const float2 minus = make_float2(-ref, -ref), by = make_float2(p.heat_log2, p.heat_log2);
#pragma unroll
                for (int k = 0; k < kBatch; k += 2) {
                    float2 y = __fmul2_rn(__fadd2_rn(make_float2(x[k], x[k + 1]), minus), by);
                    const float2 e = make_float2(ex2(y.x), ex2(y.y));
                    s = __fadd2_rn(s, e);
                    y.x = fmaxf(y.x, -3e38f);                    // 0 times -inf is 0 (a NaN is in s already)
                    y.y = fmaxf(y.y, -3e38f);
                    t = __ffma2_rn(e, y, t);
                }
                refill();
            }
        }
        if (!kTop || again) break;
        const float second = bound_of_groups(sh, most, p.top, turn);     // (and every note is there)
        const int notes = sh.n_notes;
        if (notes <= Sh::kNotes) {
            for (int i = tid; i < notes * kRows; i += kThreads) {
                const Note note = sh.notes[i / kRows];
                const int first = note.first + i % kRows * (kThreads * W), v = (first + shift) / W;
                if (note.most < second || v >= end) continue;
                float x[W];
                Vec<T>::get(base[v], x);
#pragma unroll
                for (int j = 0; j < W; ++j)
                    if (x[j] >= second && x[j] > -INFINITY) {
                        const int at = atomicAdd(&sh.n, 1);
                        if (at < Sh::kKeys) sh.keys[at] = key_of(x[j], first + j);
                    }
            }
            __syncthreads();                     // every key is counted
            listed = sh.n;
            if (listed <= Sh::kKeys) break;
        }
        __syncthreads();                         // both counts are read by all
        if (tid == 0) sh.n = 0;
        listed = p.top;
        __syncthreads();
        again = true;
    }
    // The count as a value: after a row gone through again sh.n is thread 0's
    // last write, which no barrier has parted from this.
    if (kTop) best_of_list(sh, p.top, listed);
    if (at_end >= 0 && (edge > -INFINITY || edge != edge)) {
        if (edge > mine.m) raise(edge);
        const float y = (edge - (mine.m == -INFINITY ? 0.f : mine.m)) * p.heat_log2, e2 = ex2(y);
        s.x += e2;
        t.x += e2 * fmaxf(y, -3e38f);
    }
    const Long last = all;
    mine.s = last.s + (s.x + s.y + last.s_rest);
    mine.t = last.t + (t.x + t.y + last.t_rest);

    // the warp's sums by its largest reference, the CTA's, then the cluster's
    {
        float m = mine.m;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
        mine = join(mine, Sums{m, 0.f, 0.f}, p.heat_log2);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) {
            mine.s += __shfl_xor_sync(0xFFFFFFFFu, mine.s, d);
            mine.t += __shfl_xor_sync(0xFFFFFFFFu, mine.t, d);
        }
    }
    if (lane == 0) sh.warp[warp] = mine;
    __syncthreads();
    if (warp == 0) {
        Sums a = lane < kWarps ? sh.warp[lane] : Sums{-INFINITY, 0.f, 0.f};
#pragma unroll
        for (int d = kWarps / 2; d > 0; d >>= 1) {
            const Sums o{__shfl_xor_sync(0xFFFFFFFFu, a.m, d), __shfl_xor_sync(0xFFFFFFFFu, a.s, d),
                         __shfl_xor_sync(0xFFFFFFFFu, a.t, d)};
            a = join(a, o, p.heat_log2);
        }
        if (lane == 0) sh.all = a;
    }
    cluster_sync_all();
    if (rank == 0) {
        Sums a = sh.all;
        for (int c = 1; c < cluster; ++c) {
            const uint32_t o = mapa_shared(smem_u32(&sh.all), c);
            a = join(a, Sums{ld_cluster_f32(o), ld_cluster_f32(o + 4), ld_cluster_f32(o + 8)}, p.heat_log2);
        }
        const float log_s = logf(a.s);
        // nothing above -inf: no token has a probability
        auto logprob = [&](float x) { return a.s == 0.f ? -INFINITY : p.heat * (x - a.m) - log_s; };
        if (tid == 0 && p.entropy != nullptr) p.entropy[row] = a.s == 0.f ? 0.f : log_s - kLn2 * a.t / a.s;
        for (int i = tid; i < p.n; i += kThreads) {
            const int at = p.tokens[size_t(row) * p.n + i];
            p.logprobs[size_t(row) * p.n + i] = at >= 0 && at < p.V ? logprob(Vec<T>::one(x0 + at)) : -INFINITY;
        }
        if (kTop) {
            if (cluster > 1) {
                const int n = p.top << p.cluster_bits;
                for (int i = tid; i < n; i += kThreads)
                    sh.list[i] = ld_cluster_u64(mapa_shared(smem_u32(&sh.best[i >> p.cluster_bits]), i & (cluster - 1)));
                best_of_list(sh, p.top, n);
            }
            if (tid < p.top) {
                const uint64_t key = sh.best[tid];
                p.top_ids[size_t(row) * p.top + tid] = index_of(key);
                p.top_logprobs[size_t(row) * p.top + tid] = logprob(logit_of(key));
            }
        }
    }
    cluster_sync_all();                          // no CTA leaves while its shared memory is read
}

template <typename T, bool kTop, int kThreads>
w4v_status launch(const Args &a, int M, cudaStream_t stream) {
    if (launch_pdl_cluster(token_logprobs_kernel<T, kTop, kThreads>, dim3(unsigned(M) << a.cluster_bits), dim3(kThreads),
                           0, stream, 1 << a.cluster_bits, a) != cudaSuccess) {
        cudaGetLastError();
        return W4V_ERR_CUDA;
    }
    return W4V_OK;
}

template <typename T, bool kTop>
w4v_status launch(const Args &a, int M, bool small, cudaStream_t stream) {
    return small ? launch<T, kTop, 128>(a, M, stream) : launch<T, kTop, 512>(a, M, stream);
}

}  // namespace

w4v_status launch_token_logprobs(const void *logits, bool half, long long stride, int M, int V, const int32_t *tokens,
                                 int n, float temperature, float *logprobs, float *entropy, int top, int32_t *top_ids,
                                 float *top_logprobs, cudaStream_t stream) {
    const DeviceInfo *info = nullptr;
    const w4v_status st = device_info(&info);
    if (st != W4V_OK) return st;
    Args a;
    a.logits = logits;
    a.stride = stride;
    a.tokens = tokens;
    a.logprobs = logprobs;
    a.entropy = entropy;
    a.top_ids = top_ids;
    a.top_logprobs = top_logprobs;
    a.V = V;
    a.n = n;
    a.top = top;
    a.heat = 1.f / temperature;
    a.heat_log2 = 1.4426950408889634f / temperature;
    a.slack = kSlack / a.heat_log2;
    const bool small = V <= kSmall || M >= kManyRows * info->sm_count;
    // Rows are cut while there are fewer CTAs than the GPU holds at a time and a
    // piece has more logits than its threads take at once.
    a.cluster_bits = 0;
    while (1 << a.cluster_bits < kMaxCluster && (long long)M << a.cluster_bits <= info->sm_count &&
           V > (small ? 128 : 512) * kBatch << a.cluster_bits)
        ++a.cluster_bits;
    if (half) return top > 0 ? launch<__half, true>(a, M, small, stream) : launch<__half, false>(a, M, small, stream);
    return top > 0 ? launch<float, true>(a, M, small, stream) : launch<float, false>(a, M, small, stream);
}

}  // namespace w4v
