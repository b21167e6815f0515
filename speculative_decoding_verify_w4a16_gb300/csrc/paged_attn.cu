// paged_attn.cu -- causal attention of new tokens over a paged cache.
//
// One pass over the keys with the running maximum and sum of the softmax:
// with x_j = scale log2(e) q . k_j, m the largest x so far, l = sum 2^(x_j - m)
// and o = sum 2^(x_j - m) v_j, a larger x rescales l and o by 2^(m_old - m).
//
// The plain form of it: a warp takes one row (token, query head), its lanes
// the head's elements, one key after the other.
#include "runtime.h"
#include "sm103_ptx.cuh"

namespace w4v {
namespace {

constexpr int kWarps = 8;

struct Args {
    const __half *q, *k, *v;
    __half *out;
    float *lse;
    const int32_t *table, *lengths, *offsets;
    long long q_stride;
    int n_tokens, q_heads, kv_heads, B, width, n_pages, page, window;
    float scale_log2;
};

template <int D>
__global__ void __launch_bounds__(32 * kWarps)
paged_attn_kernel(const Args p) {
    grid_dep_wait();
    grid_dep_launch();
    constexpr int kPer = D / 32;
    const int lane = threadIdx.x & 31;
    const long long row = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (row >= (long long)p.n_tokens * p.q_heads) return;
    const int t = int(row / p.q_heads), h = int(row % p.q_heads), kh = h / (p.q_heads / p.kv_heads);
    int b = -1;
    for (int i = lane; i < p.B; i += 32)
        if (p.offsets[i] <= t && t < p.offsets[i + 1]) b = i;
    b = __reduce_max_sync(0xFFFFFFFFu, b);
    if (b < 0) return;
    const int len = min(max(p.lengths[b], 0), p.width * p.page);
    const int pos = len - min(p.offsets[b + 1], p.n_tokens) + t;
    float q[kPer], o[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        q[i] = __half2float(p.q[t * p.q_stride + h * D + lane + 32 * i]) * p.scale_log2;
        o[i] = 0.f;
    }
    float m = -INFINITY, l = 0.f;
    for (int j = p.window > 0 ? max(0, pos - p.window + 1) : 0; j <= pos; ++j) {
        const int id = p.table[size_t(b) * p.width + j / p.page];
        const bool ok = id >= 0 && id < p.n_pages;
        const size_t at = ((size_t(ok ? id : 0) * p.kv_heads + kh) * p.page + j % p.page) * D + lane;
        float x = 0.f, v[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            x += ok ? q[i] * __half2float(p.k[at + 32 * i]) : 0.f;
            v[i] = ok ? __half2float(p.v[at + 32 * i]) : 0.f;
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, d);
        const float top = fmaxf(m, x), a = m == top ? 1.f : exp2f(m - top), w = exp2f(x - top);
        l = l * a + w;
#pragma unroll
        for (int i = 0; i < kPer; ++i) o[i] = o[i] * a + w * v[i];
        m = top;
    }
    const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) p.out[row * D + lane + 32 * i] = __float2half_rn(o[i] * inv);
    if (p.lse != nullptr && lane == 0) p.lse[row] = (m + log2f(l)) * 0.6931471805599453f;
}

}  // namespace

size_t paged_attn_ws_bytes(int, int, int, int, int, int, bool) { return 256; }

w4v_status launch_paged_attn(const w4v_kv_t &kv, const uint16_t *q, long long q_stride, int n_tokens, int q_heads,
                             float scale, int window, uint16_t *out, float *lse, void *ws, bool invariant,
                             cudaStream_t stream) {
    (void)ws;
    (void)invariant;
    const DeviceInfo *info = nullptr;
    w4v_status st = device_info(&info);
    if (st != W4V_OK) return st;
    Args a;
    a.q = reinterpret_cast<const __half *>(q);
    a.k = reinterpret_cast<const __half *>(kv.k);
    a.v = reinterpret_cast<const __half *>(kv.v);
    a.out = reinterpret_cast<__half *>(out);
    a.lse = lse;
    a.table = kv.table;
    a.lengths = kv.lengths;
    a.offsets = kv.offsets;
    a.q_stride = q_stride;
    a.n_tokens = n_tokens;
    a.q_heads = q_heads;
    a.kv_heads = kv.kv_heads;
    a.B = kv.B;
    a.width = kv.table_width;
    a.n_pages = kv.n_pages;
    a.page = kv.page;
    a.window = window;
    a.scale_log2 = scale * 1.4426950408889634f;
    const long long rows = (long long)n_tokens * q_heads;
    const dim3 grid(unsigned((rows + kWarps - 1) / kWarps)), block(32 * kWarps);
    auto kernel = kv.head_dim == 64 ? paged_attn_kernel<64>
                                    : kv.head_dim == 128 ? paged_attn_kernel<128> : paged_attn_kernel<256>;
    if (launch_pdl(kernel, grid, block, 0, stream, a) != cudaSuccess) {
        cudaGetLastError();
        return W4V_ERR_CUDA;
    }
    return W4V_OK;
}

}  // namespace w4v
