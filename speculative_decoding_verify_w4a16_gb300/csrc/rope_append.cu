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
// head_dim fp16 read and written once per token, so HBM bounds it.  One CTA
// takes one token: rot/2 threads form the token's cosines and sines once for
// all heads, then every thread moves 16-byte pieces.
#include <algorithm>

#include "runtime.h"
#include "sm103_ptx.cuh"

namespace w4v {
namespace {

constexpr int kThreads = 256;

struct Args {
    const __half *q, *k, *v;
    long long q_stride, k_stride, v_stride;
    __half *q_out, *k_cache, *v_cache;
    const int32_t *table, *lengths, *offsets, *positions;
    const uint64_t *phases;
    int n_tokens, q_heads, kv_heads, head_dim, rot;
    int B, table_width, n_pages, page;
    float mul;
};

union Piece {
    uint4 u;
    __half2 h[4];
};

// Two pieces of eight elements whose elements pair up (half layout).
__device__ __forceinline__ void turn_half(Piece &a, Piece &b, const float2 *cs) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 x = __half22float2(a.h[i]), y = __half22float2(b.h[i]);
        const float2 c0 = cs[2 * i], c1 = cs[2 * i + 1];
        a.h[i] = __floats2half2_rn(x.x * c0.x - y.x * c0.y, x.y * c1.x - y.y * c1.y);
        b.h[i] = __floats2half2_rn(y.x * c0.x + x.x * c0.y, y.y * c1.x + x.y * c1.y);
    }
}
// One piece of four adjacent pairs (interleaved layout).
__device__ __forceinline__ void turn_inter(Piece &a, const float2 *cs) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 x = __half22float2(a.h[i]);
        a.h[i] = __floats2half2_rn(x.x * cs[i].x - x.y * cs[i].y, x.y * cs[i].x + x.x * cs[i].y);
    }
}

// kVec: rot is a multiple of 16 (half layout) or 8 (interleaved), so pairs
// and copied elements fall into whole 16-byte pieces.  Otherwise elements
// are moved pair by pair (twice the instructions, the same bytes).
template <bool kInter, bool kVec>
__global__ void __launch_bounds__(kThreads)
rope_append_kernel(const Args p) {
    __shared__ float2 cs[128];
    __shared__ int seq;
    grid_dep_wait();
    grid_dep_launch();
    const int t = blockIdx.x, D = p.head_dim;
    if (threadIdx.x == 0) seq = -1;
    __syncthreads();
    for (int b = threadIdx.x; b < p.B; b += kThreads)
        if (p.offsets[b] <= t && t < p.offsets[b + 1]) seq = b;
    __syncthreads();
    const int b = seq;
    if (b < 0) return;
    const int end = min(p.offsets[b + 1], p.n_tokens);
    const int cap = p.table_width * p.page;
    const int at = min(max(p.lengths[b], 0), cap) - end + t;      // may be negative: the row has no slot
    const int pos = p.positions != nullptr ? p.positions[t] : at;
    for (int i = threadIdx.x; i < p.rot / 2; i += kThreads) {
        const uint32_t turn = uint32_t((uint64_t(int64_t(pos)) * p.phases[i]) >> 32);
        float s, c;
        sincospif(float(int32_t(turn)) * (1.f / 2147483648.f), &s, &c);   // 2 pi turn / 2^32
        cs[i] = make_float2(c * p.mul, s * p.mul);
    }
    __half *kd = nullptr, *vd = nullptr;                         // head 0's slot of this token
    if (at >= 0) {
        const int id = p.table[size_t(b) * p.table_width + at / p.page];
        if (id >= 0 && id < p.n_pages) {
            const size_t off = (size_t(id) * p.kv_heads * p.page + at % p.page) * D;
            kd = p.k_cache + off;
            vd = p.v_cache + off;
        }
    }
    const size_t hop = size_t(p.page) * D;                        // from head to head within a page
    const __half *qs = p.q + t * p.q_stride, *ks = p.k + t * p.k_stride, *vs = p.v + t * p.v_stride;
    __half *qd = p.q_out + size_t(t) * p.q_heads * D;
    __syncthreads();

    const int turned = p.q_heads + (kd != nullptr ? p.kv_heads : 0);
    if (kVec) {
        // items of a head: its pairs' pieces (two at once in the half layout), then the copied pieces
        const int np = kInter ? p.rot / 8 : p.rot / 16, per = np + (D - p.rot) / 8;
        for (int i = threadIdx.x; i < turned * per; i += kThreads) {
            const int h = i / per, j = i % per;
            const bool isq = h < p.q_heads;
            const __half *src = isq ? qs + h * D : ks + (h - p.q_heads) * D;
            __half *dst = isq ? qd + h * D : kd + (h - p.q_heads) * hop;
            Piece a;
            if (j >= np) {
                const int e = p.rot + 8 * (j - np);
                *reinterpret_cast<uint4 *>(dst + e) = *reinterpret_cast<const uint4 *>(src + e);
            } else if (kInter) {
                a.u = *reinterpret_cast<const uint4 *>(src + 8 * j);
                turn_inter(a, cs + 4 * j);
                *reinterpret_cast<uint4 *>(dst + 8 * j) = a.u;
            } else {
                Piece z;
                a.u = *reinterpret_cast<const uint4 *>(src + 8 * j);
                z.u = *reinterpret_cast<const uint4 *>(src + p.rot / 2 + 8 * j);
                turn_half(a, z, cs + 8 * j);
                *reinterpret_cast<uint4 *>(dst + 8 * j) = a.u;
                *reinterpret_cast<uint4 *>(dst + p.rot / 2 + 8 * j) = z.u;
            }
        }
    } else {
        const int np = p.rot / 2, per = np + D - p.rot;
        for (int i = threadIdx.x; i < turned * per; i += kThreads) {
            const int h = i / per, j = i % per;
            const bool isq = h < p.q_heads;
            const __half *src = isq ? qs + h * D : ks + (h - p.q_heads) * D;
            __half *dst = isq ? qd + h * D : kd + (h - p.q_heads) * hop;
            if (j >= np) {
                dst[p.rot + j - np] = src[p.rot + j - np];
            } else {
                const int a = kInter ? 2 * j : j, z = kInter ? 2 * j + 1 : j + np;
                const float x = __half2float(src[a]), y = __half2float(src[z]);
                dst[a] = __float2half_rn(x * cs[j].x - y * cs[j].y);
                dst[z] = __float2half_rn(y * cs[j].x + x * cs[j].y);
            }
        }
    }
    if (vd != nullptr)
        for (int i = threadIdx.x; i < p.kv_heads * (D / 8); i += kThreads) {
            const int h = i / (D / 8), e = 8 * (i % (D / 8));
            *reinterpret_cast<uint4 *>(vd + h * hop + e) = *reinterpret_cast<const uint4 *>(vs + h * D + e);
        }
}

template <bool kInter, bool kVec>
w4v_status launch(const Args &a, cudaStream_t stream) {
    if (launch_pdl(rope_append_kernel<kInter, kVec>, dim3(a.n_tokens), dim3(kThreads), 0, stream, a) != cudaSuccess) {
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
    a.page = kv.page;
    a.mul = mul;
    if (interleaved) return rot % 8 == 0 ? launch<true, true>(a, stream) : launch<true, false>(a, stream);
    return rot % 16 == 0 ? launch<false, true>(a, stream) : launch<false, false>(a, stream);
}

}  // namespace w4v
