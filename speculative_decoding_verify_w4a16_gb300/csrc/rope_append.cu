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

// CTAs of 256 threads for a few tokens, of 128 for many, where twice as many
// tokens side by side count for more than each one's own time (one GB300: 16
// rows of 28 x 128 2.8 against 3.1 us, 8192 rows of 24 x 256 39.7 against
// 34.8 us, 5.8 TB/s; measured at these two ends, not where they cross).
template <bool kInter, bool kVec>
w4v_status launch(const Args &a, int sms, cudaStream_t stream) {
    const bool many = a.n_tokens >= 16 * sms;
    if (launch_pdl(many ? rope_append_kernel<kInter, kVec, 128> : rope_append_kernel<kInter, kVec, 256>,
                   dim3(a.n_tokens), dim3(many ? 128 : 256), 0, stream, a) != cudaSuccess) {
        cudaGetLastError();
        return W4V_ERR_CUDA;
    }
    return W4V_OK;
}

}  // namespace

w4v_status launch_rope_append(const w4v_kv_t &kv, const uint16_t *q, const uint16_t *k, const uint16_t *v,
                              long long q_stride, long long k_stride, long long v_stride, int n_tokens, int q_heads,
                              const int32_t *positions, const uint64_t *phases, int rot, float mul, bool interleaved,
                              uint16_t *q_out, cudaStream_t stream) {
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
    if (interleaved) return rot % 8 == 0 ? launch<true, true>(a, info->sm_count, stream) : launch<true, false>(a, info->sm_count, stream);
    return rot % 16 == 0 ? launch<false, true>(a, info->sm_count, stream) : launch<false, false>(a, info->sm_count, stream);
}

}  // namespace w4v
