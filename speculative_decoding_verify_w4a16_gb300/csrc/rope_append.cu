// rope_append.cu -- rotary positions of the new tokens, and their keys and
// values into the paged cache.
//
// Pair i of a head turns by p f_i at position p.  The host gives f_i as the
// fraction of a full turn per position, scaled by 2^64 (F_i), so the angle
// past whole turns is p F_i mod 2^64 -- one wrapping integer product, exact
// for any position -- and sincospif takes its top 32 bits as a fraction.
// (p f_i in fp32 would be off by 2^-24 p f_i radians: 6e-3 at 100,000.)
//
// The work is a copy with a few operations in between: (q_heads + 2 kv_heads)
// head_dim fp16 read and written once per token.  HBM bounds many tokens, a
// chain of latencies (sequence, length, page) a few; in between it is
// instructions, so they are kept off the pieces.  One CTA takes one token.  A
// thread owns one 16-byte piece of a head, the same of every head it serves,
// so the piece's cosines and sines stay in its registers and nothing is
// divided; in the half layout it reads the partner piece too (from L1) and
// writes its own alone.  The first heads' pieces are on the way while the CTA
// finds the token's sequence and slot.  (With pairs as items, numbered over
// the heads, 8192 rows of 24 x 256 took 48.6 us, half of it in divisions.)
//
// With norms (norm_rope_append) every head of q and k is first divided by its
// root mean square and weighted: y = x w / sqrt(mean x^2 + eps).  The pieces of
// a head lie in neighbouring lanes, so its sum of squares is one butterfly of
// log2(D / 8) shuffles.  Weight and rotation are both linear in x, so element i
// becomes r (x_i (w_i c_i) + x_j (w_j s_i)), j its partner: the products in
// brackets are worked out once per CTA and lie in shared memory by piece, and
// r, the head's factor, multiplies last.  Measured (device time): 16 rows of 28 x
// 128 2.9 us, 660 rows of 60 x 128 6.7 (bound 3.4: bytes), 8192 rows of 24 x 256
// 38.1 (29.7; 5.3 TB/s), interleaved 37.2; pair by pair (rot 50) 96, and 5.5 for
// 16 rows of 28 x 128: 2-byte loads and stores.
#include <algorithm>

#include "runtime.h"
#include "sm103_ptx.cuh"

namespace w4v {
namespace {

struct Args {
    const __half *q, *k, *v;
    long long q_stride, k_stride, v_stride;
    __half *q_out, *k_cache, *v_cache;
    const int32_t *table, *lengths, *offsets, *positions;
    const uint64_t *phases;
    int n_tokens, q_heads, kv_heads, head_dim, rot;
    int B, table_width, n_pages, page_bits;      // 2^page_bits tokens a page
    float mul;
    const __half *q_weight, *k_weight;           // norms: [head_dim] or null (all ones)
    float eps, centre;                           // centre: added to the weights
};

union Piece {
    uint4 u;
    __half2 h[4];
};

constexpr int kAhead = 3;                       // heads of a thread whose pieces are loaded together

// kVec: rot is a multiple of 16 (half layout) or 8 (interleaved), so pairs
// and copied elements fall into whole 16-byte pieces.  Otherwise elements are
// moved pair by pair, with a division each: the same bytes, but 88 us instead of
// 35 for 8192 rows of 24 x 256 (rot 242), 31 instead of 16 for 28 x 64 (rot 50),
// 6.0 instead of 3.1 for 16 rows.  The bound is 48 registers, 40 warps an SM;
// the half layout spills 44 bytes under it.
template <bool kInter, bool kVec, int kThreads>
__global__ void __launch_bounds__(kThreads, 1280 / kThreads)
rope_append_kernel(const Args p) {
    __shared__ float2 cs[128];
    __shared__ int seq;
    const int t = blockIdx.x, D = p.head_dim, tid = threadIdx.x;
    if (tid == 0) seq = -1;
    grid_dep_wait();
    grid_dep_launch();
    const __half *qs = p.q + t * p.q_stride, *ks = p.k + t * p.k_stride, *vs = p.v + t * p.v_stride;
    // this thread's piece, and its heads: first, first + step, ... of the
    // query heads, then the key heads, then the value heads
    const int e = 8 * (tid & (D / 8 - 1)), first = tid / (D / 8), step = kThreads / (D / 8);
    const int turned = p.q_heads + p.kv_heads, heads = turned + p.kv_heads;
    const bool turn = e < p.rot, upper = !kInter && e >= p.rot / 2;
    const int partner = upper ? -p.rot / 2 : p.rot / 2;
    Piece a[kAhead], z[kAhead];
    auto load = [&](int h0) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int h = h0 + u * step;
            if (h >= heads) continue;
            const __half *src = (h < p.q_heads ? qs + h * D : h < turned ? ks + (h - p.q_heads) * D : vs + (h - turned) * D) + e;
            a[u].u = *reinterpret_cast<const uint4 *>(src);
            if (!kInter && turn && h < turned) z[u].u = *reinterpret_cast<const uint4 *>(src + partner);
        }
    };
    if (kVec) load(first);

    __syncthreads();
    for (int b = tid; b < p.B; b += kThreads)
        if (p.offsets[b] <= t && t < p.offsets[b + 1]) seq = b;
    __syncthreads();
    const int b = seq;
    if (b < 0) return;
    const int end = min(p.offsets[b + 1], p.n_tokens);
    const int cap = p.table_width << p.page_bits, last = (1 << p.page_bits) - 1;
    const int at = min(max(p.lengths[b], 0), cap) - end + t;      // may be negative: the row has no slot
    const int pos = p.positions != nullptr ? p.positions[t] : at;
    for (int i = tid; i < p.rot / 2; i += kThreads) {
        const uint32_t part = uint32_t((uint64_t(int64_t(pos)) * p.phases[i]) >> 32);
        float s, c;
        sincospif(float(int32_t(part)) * (1.f / 2147483648.f), &s, &c);   // 2 pi part / 2^32
        cs[i] = make_float2(c * p.mul, s * p.mul);
    }
    long long slot = -1;                                         // head 0's elements of this token
    if (at >= 0) {
        const int id = p.table[size_t(b) * p.table_width + (at >> p.page_bits)];
        if (id >= 0 && id < p.n_pages) slot = (((long long)id * p.kv_heads << p.page_bits) + (at & last)) * D;
    }
    const long long hop = (long long)D << p.page_bits;           // from head to head within a page
    __half *qd = p.q_out + size_t(t) * p.q_heads * D;
    __syncthreads();

    if (kVec) {
        // element i of the piece: x c + y s (half layout; the lower partner
        // subtracts), or pairs within the piece (interleaved)
        float c[8], s[8];
        if (turn) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 v = cs[kInter ? e / 2 + i / 2 : (upper ? e - p.rot / 2 : e) + i];
                c[i] = v.x;
                s[i] = kInter ? ((i & 1) ? v.y : -v.y) : (upper ? v.y : -v.y);
            }
        }
        for (int h0 = first, pass = 0; pass * kAhead * step < heads; h0 += kAhead * step, ++pass) {
            if (pass > 0) {
                load(h0);
                __syncthreads();                                 // q_out may be q: both partners read before either is written
            }
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int h = h0 + u * step;
                if (h >= heads || (h >= p.q_heads && slot < 0)) continue;
                __half *dst = (h < p.q_heads ? qd + h * D
                                             : h < turned ? p.k_cache + slot + (h - p.q_heads) * hop
                                                          : p.v_cache + slot + (h - turned) * hop) + e;
                if (turn && h < turned) {
                    Piece o;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 x = __half22float2(a[u].h[i]);
                        const float2 y = kInter ? make_float2(x.y, x.x) : __half22float2(z[u].h[i]);
                        o.h[i] = __floats2half2_rn(x.x * c[2 * i] + y.x * s[2 * i], x.y * c[2 * i + 1] + y.y * s[2 * i + 1]);
                    }
                    a[u].u = o.u;
                }
                *reinterpret_cast<uint4 *>(dst) = a[u].u;
            }
        }
    } else {
        const int pairs = p.rot / 2, each = pairs + D - p.rot;
        for (int i = tid; i < (p.q_heads + (slot >= 0 ? p.kv_heads : 0)) * each; i += kThreads) {
            const int h = i / each, j = i % each;
            const bool isq = h < p.q_heads;
            const __half *src = isq ? qs + h * D : ks + (h - p.q_heads) * D;
            __half *dst = isq ? qd + h * D : p.k_cache + slot + (h - p.q_heads) * hop;
            if (j >= pairs) {
                dst[p.rot + j - pairs] = src[p.rot + j - pairs];
            } else {
                const int f = kInter ? 2 * j : j, g = kInter ? 2 * j + 1 : j + pairs;
                const float x = __half2float(src[f]), y = __half2float(src[g]);
                dst[f] = __float2half_rn(x * cs[j].x - y * cs[j].y);
                dst[g] = __float2half_rn(y * cs[j].x + x * cs[j].y);
            }
        }
        if (slot >= 0)
            for (int h = first; h < p.kv_heads; h += step)
                *reinterpret_cast<uint4 *>(p.v_cache + slot + h * hop + e) = *reinterpret_cast<const uint4 *>(vs + h * D + e);
    }
}

// The sums of a head's squares, lane by lane in, in every lane of the head out
// (`lanes` neighbouring lanes, a power of two).
template <int n>
__device__ __forceinline__ void head_sums(float (&x)[n], int lanes) {
#pragma unroll 1
    for (int d = 1; d < lanes; d <<= 1)
#pragma unroll
        for (int u = 0; u < n; ++u) x[u] += __shfl_xor_sync(0xFFFFFFFFu, x[u], d);
}

// The same with norms.  kVec as above; without it a warp takes a head, pair by
// pair.  Partner pieces come from their lanes by shuffles: read again from L1
// they held 12 registers more across the waits, 49.7 us against 44.8 for 8192
// rows of 24 x 256.  Two heads a thread ahead: 660 rows of 60 x 128 6.7 us
// (three 7.2), 16 rows of 28 x 128 2.9 (3.2).
constexpr int kNormAhead = 2;
template <bool kInter, bool kVec, int kThreads>
__global__ void __launch_bounds__(kThreads, 1280 / kThreads)
norm_rope_append_kernel(const Args p) {
    // Elements 2j and 2j + 1 of piece c of q (0) or k (1) are r (x coef.xy +
    // x_partner coef.zw), coef[.][j][c].
    __shared__ float4 coef[2][4][32];
    __shared__ int seq;
    const int t = blockIdx.x, D = p.head_dim, tid = threadIdx.x;
    if (tid == 0) seq = -1;
    grid_dep_wait();
    grid_dep_launch();
    const __half *qs = p.q + t * p.q_stride, *ks = p.k + t * p.k_stride, *vs = p.v + t * p.v_stride;
    const int e = 8 * (tid & (D / 8 - 1)), first = tid / (D / 8), step = kThreads / (D / 8);
    const int turned = p.q_heads + p.kv_heads, heads = turned + p.kv_heads;
    // The lane that holds the partner piece (half layout), or this one.  (What is
    // not rotated has itself for a partner in both layouts, by a factor of 0: an
    // infinity then spoils no other element.)
    const int partner = kInter || e >= p.rot ? int(threadIdx.x & 31) : int(threadIdx.x & 31) + (e >= p.rot / 2 ? -p.rot / 16 : p.rot / 16);
    Piece a[kNormAhead];
    auto load = [&](int h0) {
#pragma unroll
        for (int u = 0; u < kNormAhead; ++u) {
            const int h = h0 + u * step;
            a[u].u = make_uint4(0u, 0u, 0u, 0u);
            if (h < heads)
                a[u].u = *reinterpret_cast<const uint4 *>((h < p.q_heads ? qs + h * D : h < turned ? ks + (h - p.q_heads) * D
                                                                                                   : vs + (h - turned) * D) + e);
        }
    };
    if (kVec) load(first);

    // This thread's pairs (then single elements) f, g and their weights of q and k
    constexpr int kItems = 256 / kThreads;
    const int pairs = p.rot / 2, items = D - pairs;
    auto places = [&](int i, int &f, int &g) {
        f = i >= pairs ? pairs + i : kInter ? 2 * i : i;
        g = i >= pairs ? f : kInter ? f + 1 : f + pairs;
    };
    float w[kItems][2][2];
#pragma unroll
    for (int n = 0; n < kItems; ++n) {
        int f, g;
        places(min(tid + n * kThreads, items - 1), f, g);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const __half *src = x == 0 ? p.q_weight : p.k_weight;
            w[n][x][0] = src != nullptr ? __half2float(src[f]) + p.centre : 1.f;
            w[n][x][1] = src != nullptr ? __half2float(src[g]) + p.centre : 1.f;
        }
    }
    __syncthreads();
    for (int b = tid; b < p.B; b += kThreads)
        if (p.offsets[b] <= t && t < p.offsets[b + 1]) seq = b;
    __syncthreads();
    const int b = seq;
    if (b < 0) return;
    const int end = min(p.offsets[b + 1], p.n_tokens);
    const int cap = p.table_width << p.page_bits, last = (1 << p.page_bits) - 1;
    const int at = min(max(p.lengths[b], 0), cap) - end + t;      // may be negative: the row has no slot
    const int pos = p.positions != nullptr ? p.positions[t] : at;
    auto at_element = [&](int x, int i) {        // its own factor; two on its partner's
        return reinterpret_cast<float *>(&coef[x][i / 2 & 3][i / 8]) + (i & 1);
    };
    auto put = [&](int x, int i, float own, float other) {
        float *m = at_element(x, i);
        m[0] = own;
        m[2] = other;
    };
#pragma unroll
    for (int n = 0; n < kItems; ++n) {
        const int i = tid + n * kThreads;
        if (i >= items) continue;
        int f, g;
        places(i, f, g);
        float s = 0.f, c = 1.f;
        if (i < pairs) {
            const uint32_t part = uint32_t((uint64_t(int64_t(pos)) * p.phases[i]) >> 32);
            sincospif(float(int32_t(part)) * (1.f / 2147483648.f), &s, &c);   // 2 pi part / 2^32
            s *= p.mul;
            c *= p.mul;
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            if (i < pairs) put(x, g, w[n][x][1] * c, w[n][x][0] * s);
            // (a single element's own is +0, as in the kernel below: -0 would give zeros another sign)
            put(x, f, w[n][x][0] * c, i < pairs ? -w[n][x][1] * s : 0.f);
        }
    }
    long long slot = -1;                                         // head 0's elements of this token
    if (at >= 0) {
        const int id = p.table[size_t(b) * p.table_width + (at >> p.page_bits)];
        if (id >= 0 && id < p.n_pages) slot = (((long long)id * p.kv_heads << p.page_bits) + (at & last)) * D;
    }
    const long long hop = (long long)D << p.page_bits;           // from head to head within a page
    __half *qd = p.q_out + size_t(t) * p.q_heads * D;
    const float mean = 1.f / float(D);                           // D is a power of two
    __syncthreads();

    if (kVec) {
        for (int h0 = first, pass = 0; pass * kNormAhead * step < heads; h0 += kNormAhead * step, ++pass) {
            if (pass > 0) load(h0);
            float sum[kNormAhead];
#pragma unroll
            for (int u = 0; u < kNormAhead; ++u) {
                float2 q = make_float2(0.f, 0.f);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 x = __half22float2(a[u].h[i]);
                    q = __ffma2_rn(x, x, q);
                }
                sum[u] = q.x + q.y;
            }
            head_sums(sum, D / 8);
#pragma unroll
            for (int u = 0; u < kNormAhead; ++u) {
                const int h = h0 + u * step;
                const bool normed = h < turned;
                if (__any_sync(0xFFFFFFFFu, normed)) {
                    const float r = rsqrtf(sum[u] * mean + p.eps);
                    Piece o;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float4 m = coef[h < p.q_heads ? 0 : 1][i][e / 8];
                        const uint32_t w = h2_as_u32(a[u].h[i]);
                        const float2 x = __half22float2(a[u].h[i]);
                        const float2 y = kInter ? e < p.rot ? make_float2(x.y, x.x) : x
                                                : __half22float2(u32_as_h2(__shfl_sync(0xFFFFFFFFu, w, partner)));
                        const float2 v = __ffma2_rn(y, make_float2(m.z, m.w), __fmul2_rn(x, make_float2(m.x, m.y)));
                        o.h[i] = __float22half2_rn(__fmul2_rn(v, make_float2(r, r)));
                    }
                    if (normed) a[u].u = o.u;
                }
                if (h >= heads || (h >= p.q_heads && slot < 0)) continue;
                __half *dst = (h < p.q_heads ? qd + h * D
                                             : h < turned ? p.k_cache + slot + (h - p.q_heads) * hop
                                                          : p.v_cache + slot + (h - turned) * hop) + e;
                *reinterpret_cast<uint4 *>(dst) = a[u].u;
            }
        }
    } else {
        const int warp = tid / 32, lane = tid & 31;
        for (int h = warp; h < p.q_heads + (slot >= 0 ? p.kv_heads : 0); h += kThreads / 32) {
            const bool isq = h < p.q_heads;
            const __half *src = isq ? qs + h * D : ks + (h - p.q_heads) * D;
            __half *dst = isq ? qd + h * D : p.k_cache + slot + (h - p.q_heads) * hop;
            float sum[1] = {0.f};
            if (lane < D / 8) {
                Piece x;
                x.u = *reinterpret_cast<const uint4 *>(src + 8 * lane);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 y = __half22float2(x.h[i]);
                    sum[0] = fmaf(y.x, y.x, fmaf(y.y, y.y, sum[0]));
                }
            }
            head_sums(sum, 32);
            const float r = rsqrtf(sum[0] * mean + p.eps);
            for (int i = lane; i < items; i += 32) {
                int f, g;
                places(i, f, g);
                const float *m = at_element(isq ? 0 : 1, f), *l = at_element(isq ? 0 : 1, g);
                const float x = __half2float(src[f]), y = __half2float(src[g]);
                if (i < pairs) dst[g] = __float2half_rn((y * l[0] + x * l[2]) * r);
                dst[f] = __float2half_rn(i < pairs ? (x * m[0] + y * m[2]) * r : x * m[0] * r);
            }
        }
        if (slot >= 0)
            for (int h = first; h < p.kv_heads; h += step)
                *reinterpret_cast<uint4 *>(p.v_cache + slot + h * hop + e) = *reinterpret_cast<const uint4 *>(vs + h * D + e);
    }
}

// The same for many tokens in whole pieces.  There the instructions count (45 us
// for 8192 rows of 24 x 256 with 78% of the issue slots in use), so a warp takes
// a token: the factors of its pieces lie in registers for all heads, and there
// is no barrier; 5039 -> 2810 instructions a token.  kAheadMany passes over 256
// / D heads are loaded ahead; more of them cost more in warps at a time than
// they bring (8192 rows, by passes ahead and CTAs an SM: 2 and 7 38.2 us, 5.3
// TB/s, 2 and 8 38.4, 3 and 7 40.8, 1 and 8 43.9, 4 and 5 48.5; 24 x 128 27.3 of
// 31.7, 36 x 64 19.0 of 26.7 with a CTA a token).  From 24 rows an SM on: 2560
// rows take 13.3 us like this and 12.1 with a CTA each, some 4100 21.2 and 22.1.
constexpr int kWarpThreads = 128, kAheadMany = 2, kWarpRows = 24;
template <bool kInter, int D>
__global__ void __launch_bounds__(kWarpThreads, 7)
norm_rope_append_warp_kernel(const Args p) {
    constexpr int kLanes = D / 8, kHeads = 32 / kLanes;          // lanes a head, heads a pass
    __shared__ float2 cs[kWarpThreads / 32][D / 2];
    const int lane = threadIdx.x & 31, warp = int(threadIdx.x) >> 5, t = blockIdx.x * (kWarpThreads / 32) + warp;
    grid_dep_wait();
    grid_dep_launch();
    if (t >= p.n_tokens) return;
    const __half *qs = p.q + t * p.q_stride, *ks = p.k + t * p.k_stride, *vs = p.v + t * p.v_stride;
    const int e = 8 * (lane % kLanes), sub = lane / kLanes;
    const int turned = p.q_heads + p.kv_heads, heads = turned + p.kv_heads, passes = (heads + kHeads - 1) / kHeads;
    const bool turn = e < p.rot, upper = !kInter && e >= p.rot / 2;
    // The lane that holds the partner piece (half layout), or this one.
    const int partner = kInter || !turn ? lane : lane + (upper ? -p.rot / 16 : p.rot / 16);
    Piece a[kAheadMany];
    auto load = [&](int pass) {
        const int h = pass * kHeads + sub;
        const __half *src = h < p.q_heads ? qs + h * D : h < turned ? ks + (h - p.q_heads) * D : vs + (h - turned) * D;
        return h < heads ? *reinterpret_cast<const uint4 *>(src + e) : make_uint4(0u, 0u, 0u, 0u);
    };
#pragma unroll
    for (int u = 0; u < kAheadMany; ++u) a[u].u = load(u);

    int b = -1;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
        const bool here = b0 + lane < p.B && p.offsets[b0 + lane] <= t && t < p.offsets[b0 + lane + 1];
        const uint32_t some = __ballot_sync(0xFFFFFFFFu, here);
        if (some != 0) b = b0 + __ffs(some) - 1;
    }
    if (b < 0) return;
    const int end = min(p.offsets[b + 1], p.n_tokens);
    const int cap = p.table_width << p.page_bits, last = (1 << p.page_bits) - 1;
    const int at = min(max(p.lengths[b], 0), cap) - end + t;      // may be negative: the row has no slot
    const int pos = p.positions != nullptr ? p.positions[t] : at;
    for (int i = lane; i < p.rot / 2; i += 32) {
        const uint32_t part = uint32_t((uint64_t(int64_t(pos)) * p.phases[i]) >> 32);
        float s, c;
        sincospif(float(int32_t(part)) * (1.f / 2147483648.f), &s, &c);   // 2 pi part / 2^32
        cs[warp][i] = make_float2(c * p.mul, s * p.mul);
    }
    long long slot = -1;                                         // head 0's elements of this token
    if (at >= 0) {
        const int id = p.table[size_t(b) * p.table_width + (at >> p.page_bits)];
        if (id >= 0 && id < p.n_pages) slot = (((long long)id * p.kv_heads << p.page_bits) + (at & last)) * D;
    }
    __syncwarp();
    // Elements 2i and 2i + 1 of the piece are r (x own + x_partner other).
    float2 own[4], other[4];
    auto factors = [&](const __half *weight) {
        Piece w, z;
        if (weight != nullptr) w.u = *reinterpret_cast<const uint4 *>(weight + e);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float2 x = make_float2(1.f, 1.f);
            if (weight != nullptr) {
                x = __half22float2(w.h[i]);
                x = make_float2(x.x + p.centre, x.y + p.centre);
            }
            own[i] = x;
            other[i] = make_float2(0.f, 0.f);
        }
        if (!turn) return;
        if (weight != nullptr && !kInter) z.u = *reinterpret_cast<const uint4 *>(weight + (upper ? e - p.rot / 2 : e + p.rot / 2));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float2 y = make_float2(own[i].y, own[i].x);          // the partners' weights
            if (!kInter) {
                y = make_float2(1.f, 1.f);
                if (weight != nullptr) {
                    y = __half22float2(z.h[i]);
                    y = make_float2(y.x + p.centre, y.y + p.centre);
                }
            }
            const float2 v0 = cs[warp][kInter ? e / 2 + i : (upper ? e - p.rot / 2 : e) + 2 * i];
            const float2 v1 = kInter ? v0 : cs[warp][(upper ? e - p.rot / 2 : e) + 2 * i + 1];
            own[i] = make_float2(own[i].x * v0.x, own[i].y * v1.x);
            other[i] = make_float2(y.x * (upper ? v0.y : -v0.y), y.y * (kInter || upper ? v1.y : -v1.y));
        }
    };
    factors(p.q_weight);
    const long long hop = (long long)D << p.page_bits;           // from head to head within a page
    __half *qd = p.q_out + size_t(t) * p.q_heads * D + e, *kd = p.k_cache + slot + e, *vd = p.v_cache + slot + e;
    const int k_pass = p.q_heads / kHeads;                       // the first pass with a key head
    auto finish = [&](const Piece &x) {
        float2 q = make_float2(0.f, 0.f), f[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[i] = __half22float2(x.h[i]);
            q = __ffma2_rn(f[i], f[i], q);
        }
        float sum = q.x + q.y;
#pragma unroll
        for (int d = 1; d < kLanes; d <<= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
        const float r = rsqrtf(sum * (1.f / D) + p.eps);
        Piece o;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float2 y = turn ? make_float2(f[i].y, f[i].x) : f[i];
            if (!kInter) y = __half22float2(u32_as_h2(__shfl_sync(0xFFFFFFFFu, h2_as_u32(x.h[i]), partner)));
            const float2 z = __ffma2_rn(y, other[i], __fmul2_rn(f[i], own[i]));
            o.h[i] = __float22half2_rn(__fmul2_rn(z, make_float2(r, r)));
        }
        return o.u;
    };
    // The query heads, and what shares a pass with them; then key heads by
    // their own factors; then values as they are.
#pragma unroll 1
    for (int pass0 = 0; pass0 < passes; pass0 += kAheadMany) {
#pragma unroll
        for (int u = 0; u < kAheadMany; ++u) {
            const int pass = pass0 + u, h = pass * kHeads + sub;
            if (pass >= passes) break;                           // the same for all lanes
            Piece x;
            x.u = a[u].u;
            a[u].u = load(pass + kAheadMany);
            uint4 out = x.u;
            if (pass * kHeads < p.q_heads) out = finish(x);
            if (h < p.q_heads) *reinterpret_cast<uint4 *>(qd + h * D) = out;
            if (pass < k_pass) continue;
            if (pass == k_pass) factors(p.k_weight);             // (its key heads are done again with them)
            if (pass * kHeads < turned) out = finish(x);
            if (slot < 0) continue;
            if (h >= p.q_heads && h < turned) *reinterpret_cast<uint4 *>(kd + (h - p.q_heads) * hop) = out;
            if (h >= turned && h < heads) *reinterpret_cast<uint4 *>(vd + (h - turned) * hop) = x.u;
        }
    }
}

// CTAs of 256 threads for a few tokens, of 128 for many, where twice as many
// tokens side by side count for more than each one's own time (one GB300: 16
// rows of 28 x 128 2.8 against 3.1 us, 8192 rows of 24 x 256 39.7 against
// 34.8 us, 5.8 TB/s; measured at these two ends, not where they cross).
template <bool kInter, bool kVec>
w4v_status launch(const Args &a, bool norm, int sms, cudaStream_t stream) {
    const bool many = a.n_tokens >= 16 * sms;
    if (norm && kVec && a.n_tokens >= kWarpRows * sms) {
        const auto kernel = a.head_dim == 64 ? norm_rope_append_warp_kernel<kInter, 64>
                            : a.head_dim == 128 ? norm_rope_append_warp_kernel<kInter, 128>
                                                : norm_rope_append_warp_kernel<kInter, 256>;
        constexpr int kTokens = kWarpThreads / 32;
        if (launch_pdl(kernel, dim3((a.n_tokens + kTokens - 1) / kTokens), dim3(kWarpThreads), 0, stream, a) != cudaSuccess) {
            cudaGetLastError();
            return W4V_ERR_CUDA;
        }
        return W4V_OK;
    }
    const auto kernel = norm ? many ? norm_rope_append_kernel<kInter, kVec, 128> : norm_rope_append_kernel<kInter, kVec, 256>
                             : many ? rope_append_kernel<kInter, kVec, 128> : rope_append_kernel<kInter, kVec, 256>;
    if (launch_pdl(kernel, dim3(a.n_tokens), dim3(many ? 128 : 256), 0, stream, a) != cudaSuccess) {
        cudaGetLastError();
        return W4V_ERR_CUDA;
    }
    return W4V_OK;
}

}  // namespace

w4v_status launch_rope_append(const w4v_kv_t &kv, const uint16_t *q, const uint16_t *k, const uint16_t *v,
                              long long q_stride, long long k_stride, long long v_stride, int n_tokens, int q_heads,
                              const int32_t *positions, const uint64_t *phases, int rot, float mul, bool interleaved,
                              const HeadNorm *norm, uint16_t *q_out, cudaStream_t stream) {
    const DeviceInfo *info = nullptr;
    w4v_status st = device_info(&info);
    if (st != W4V_OK) return st;
    Args a;
    a.q = reinterpret_cast<const __half *>(q);
    a.k = reinterpret_cast<const __half *>(k);
    a.v = reinterpret_cast<const __half *>(v);
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.q_out = reinterpret_cast<__half *>(q_out);
    a.k_cache = reinterpret_cast<__half *>(kv.k);
    a.v_cache = reinterpret_cast<__half *>(kv.v);
    a.table = kv.table;
    a.lengths = kv.lengths;
    a.offsets = kv.offsets;
    a.positions = positions;
    a.phases = phases;
    a.n_tokens = n_tokens;
    a.q_heads = q_heads;
    a.kv_heads = kv.kv_heads;
    a.head_dim = kv.head_dim;
    a.rot = rot;
    a.B = kv.B;
    a.table_width = kv.table_width;
    a.n_pages = kv.n_pages;
    a.page_bits = 0;
    while (1 << a.page_bits < kv.page) ++a.page_bits;
    a.mul = mul;
    a.q_weight = norm != nullptr ? reinterpret_cast<const __half *>(norm->q_weight) : nullptr;
    a.k_weight = norm != nullptr ? reinterpret_cast<const __half *>(norm->k_weight) : nullptr;
    a.eps = norm != nullptr ? norm->eps : 0.f;
    a.centre = norm != nullptr && norm->zero_centred ? 1.f : 0.f;
    const bool whole = rot % (interleaved ? 8 : 16) == 0, n = norm != nullptr;
    const int sms = info->sm_count;
    if (interleaved) return whole ? launch<true, true>(a, n, sms, stream) : launch<true, false>(a, n, sms, stream);
    return whole ? launch<false, true>(a, n, sms, stream) : launch<false, false>(a, n, sms, stream);
}

}  // namespace w4v
