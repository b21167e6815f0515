// token_logprobs.cu -- log probabilities of given tokens, the rows' entropy
// and their most likely tokens, from the lm_head's logits.
//
// With d_v = x_v - m, m a row's largest logit, and h = 1 / temperature,
//     s = sum_v e^(h d_v),  t = sum_v d_v e^(h d_v):
//     log p_v = h d_v - ln s,   entropy = ln s - h t / s
// (both terms of the entropy are positive, so nothing cancels).  One pass:
// the logits are read once, into registers, 40 a thread.  A thread takes its
// own largest one as reference, so the powers need no wait; s and t are brought
// to a common reference by 2^(h (m_thread - m)), t as w (t + (m_thread - m) s).
//
// A row is cut over the CTAs of a cluster, each of which holds its piece whole
// (up to 20,480 logits), and joined by the first one through distributed shared
// memory: no workspace, no second launch, no atomics between CTAs.
//
// The `top` largest, ties to the lower index, without sorting: 128 groups of
// four threads have a largest logit each, and the top-th largest of those is a
// bound that at least `top` logits reach and few exceed (31 groups' at most:
// 4960, but some 25 where logits lie without order).  Those are collected and
// each counts how many are above it.  Logits equal to the bound that are too many to
// collect, and those of a row that has fewer than `top` tokens above -inf, are
// taken in order of their index by a scan.
#include <climits>

#include "runtime.h"
#include "sm103_ptx.cuh"

namespace w4v {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kHeldLogits = 40;                 // of a thread
constexpr int kPiece = kThreads * kHeldLogits;  // of a CTA at a time
constexpr int kGroups = 128, kGroupLanes = kThreads / kGroups;
constexpr int kMost = kLogprobsMaxTop;
constexpr int kAbove = 4960, kTies = 512;       // keys that are collected: above the bound, equal to it
static_assert((kMost - 1) * kGroupLanes * kHeldLogits <= kAbove, "every logit of the groups above the bound fits");
static_assert(kMost <= kGroups, "the bound is a group's largest logit");
constexpr int kMaxCluster = 8;

struct Args {
    const void *logits;
    long long stride;
    const int32_t *tokens;
    float *logprobs, *entropy, *top_logprobs;
    int32_t *top_ids;
    int V, n, top, cluster_bits;
    float heat, heat_log2;                      // 1 / temperature, and times log2(e)
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
    // weight of 0 leaves t's term out: the distance may be infinite.
    auto add = [&](const Sums &x) {
        const float d = x.m - m, w = x.m == -INFINITY ? 1.f : ex2(d * heat_log2);
        r.s += w * x.s;
        if (x.m > -INFINITY && w != 0.f) r.t += w * (x.t + d * x.s);
    };
    add(a);
    add(b);
    return r;
}

struct __align__(8) Shared {
    uint64_t above[kAbove], ties[kTies + kMost];
    uint64_t best[kMost];                       // the CTA's largest, in order
    float group[kGroups];
    Sums warp[kWarps], all;
    float bound;
    int n_above, n_ties;
    int scan[kWarps];
};

template <typename T>
struct Vec;                                     // 16 bytes of logits
template <>
struct Vec<float> {
    static constexpr int kCount = 4;
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

template <typename T, bool kTop>
__global__ void __launch_bounds__(kThreads, 2)
token_logprobs_kernel(const Args p) {
    __shared__ Shared sh;
    constexpr int W = Vec<T>::kCount, kVecs = kHeldLogits / W;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cluster = 1 << p.cluster_bits, rank = int(blockIdx.x) & (cluster - 1), row = int(blockIdx.x) >> p.cluster_bits;
    grid_dep_wait();
    grid_dep_launch();
    // Vectors of 16 bytes from the boundary at or before the row's first
    // logit: vector v holds logits v W - shift ...
    const T *x0 = static_cast<const T *>(p.logits) + row * p.stride;
    const int shift = int(reinterpret_cast<uintptr_t>(x0) & 15u) / int(sizeof(T));
    const T *base = x0 - shift;
    const int vecs = int((unsigned(p.V) + shift + W - 1) / W);
    const int each = (vecs + cluster - 1) >> p.cluster_bits;
    const int begin = min(rank * each, vecs), end = min(begin + each, vecs);

    Sums mine{-INFINITY, 0.f, 0.f};
    int carried = 0;
    for (int v0 = begin; v0 == begin || v0 < end; v0 += kThreads * kVecs) {
        float x[kHeldLogits];
        uint4 w[kVecs];
        // whole vectors all at once; what lies at the row's ends one by one
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const int v = v0 + i * kThreads + tid, first = v * W - shift;
            if (v < end && first >= 0 && first <= p.V - W) w[i] = *reinterpret_cast<const uint4 *>(base + size_t(v) * W);
        }
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const int v = v0 + i * kThreads + tid, first = v * W - shift;
            if (v >= end) continue;
            if (first >= 0 && first <= p.V - W) {
                Vec<T>::get(w[i], x + i * W);
            } else {
#pragma unroll
                for (int j = 0; j < W; ++j)
                    x[i * W + j] = first + j >= 0 && first + j < p.V ? Vec<T>::one(x0 + (first + j)) : -INFINITY;
            }
#pragma unroll
            for (int j = 0; j < W; j += 2) top = max3(top, x[i * W + j], x[i * W + j + 1]);
        }
        // s and t by this thread's largest
        const float ref = top == -INFINITY ? 0.f : top;
        float2 s2 = make_float2(0.f, 0.f), t2 = make_float2(0.f, 0.f);
        const float2 minus = make_float2(-ref, -ref), by = make_float2(p.heat_log2, p.heat_log2);
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            if (v0 + i * kThreads + tid >= end) continue;
#pragma unroll
            for (int j = 0; j < W; j += 2) {
                const float2 d = __fadd2_rn(make_float2(x[i * W + j], x[i * W + j + 1]), minus);
                float2 e = __fmul2_rn(d, by);
                e.x = ex2(e.x);
                e.y = ex2(e.y);
                s2 = __fadd2_rn(s2, e);
                t2 = __ffma2_rn(e, d, t2);
            }
        }
        Sums here{top, s2.x + s2.y, t2.x + t2.y};
        if (here.t != here.t && here.s == here.s) {              // 0 times -inf: a logit of -inf
            here.t = 0.f;
#pragma unroll
            for (int k = 0; k < kHeldLogits; ++k)
                if (v0 + k / W * kThreads + tid < end) {
                    const float d = x[k] - ref;
                    if (d > -INFINITY) here.t = fmaf(ex2(d * p.heat_log2), d, here.t);
                }
        }
        mine = join(mine, here, p.heat_log2);

        if (kTop) {
            float g = top;
#pragma unroll
            for (int d = 1; d < kGroupLanes; d <<= 1) g = fmaxf(g, __shfl_xor_sync(0xFFFFFFFFu, g, d));
            if (tid % kGroupLanes == 0) sh.group[tid / kGroupLanes] = g;
            if (tid == 0) {
                sh.n_above = 0;
                sh.n_ties = carried;
            }
            if (tid < carried) sh.ties[tid] = sh.best[tid];
            __syncthreads();
            // the groups' largest: how many are above this one (a part for each lane)
            constexpr int kShare = kGroups / kGroupLanes;
            int above = 0;
#pragma unroll 8
            for (int k = 0; k < kShare; ++k) {
                const int o = k * kGroupLanes + tid % kGroupLanes;
                above += sh.group[o] > g || (sh.group[o] == g && o < tid / kGroupLanes);
            }
#pragma unroll
            for (int d = 1; d < kGroupLanes; d <<= 1) above += __shfl_xor_sync(0xFFFFFFFFu, above, d);
            if (above == p.top - 1 && tid % kGroupLanes == 0) sh.bound = g;
            __syncthreads();
            const float bound = sh.bound;
            if (top >= bound && top > -INFINITY) {
#pragma unroll
                for (int k = 0; k < kHeldLogits; ++k) {
                    const int v = v0 + k / W * kThreads + tid;
                    if (v >= end || !(x[k] >= bound) || !(x[k] > -INFINITY)) continue;
                    const uint64_t key = key_of(x[k], v * W - shift + k % W);
                    if (x[k] > bound) {
                        sh.above[atomicAdd(&sh.n_above, 1)] = key;
                    } else {
                        const int at = atomicAdd(&sh.n_ties, 1);
                        if (at < kTies + kMost) sh.ties[at] = key;
                    }
                }
            }
            __syncthreads();
            int n_above = sh.n_above, n_ties = sh.n_ties;
            if (n_ties > kTies + kMost || bound == -INFINITY) {
                // those equal to the bound in order of their index (the first
                // vectors of all threads, then the second ones ...)
                const int want = p.top - n_above;
                int found = 0;
#pragma unroll
                for (int i = 0; i < kVecs; ++i) {
                    const int v = v0 + i * kThreads + tid;
                    if (found >= want || v0 + i * kThreads >= end) continue;             // the same for all
                    int here_n = 0;
#pragma unroll
                    for (int j = 0; j < W; ++j) {
                        const int index = v * W - shift + j;
                        const bool is = v < end && index >= 0 && index < p.V &&
                                        (bound == -INFINITY ? !(x[i * W + j] > -INFINITY) : x[i * W + j] == bound);
                        here_n += is;
                    }
                    int upto = here_n;
#pragma unroll
                    for (int d = 1; d < 32; d <<= 1) {
                        const int y = __shfl_up_sync(0xFFFFFFFFu, upto, d);
                        if (lane >= d) upto += y;
                    }
                    __syncthreads();
                    if (lane == 31) sh.scan[warp] = upto;
                    __syncthreads();
                    int at = found + upto - here_n, all = 0;
#pragma unroll
                    for (int o = 0; o < kWarps; ++o) {
                        if (o < warp) at += sh.scan[o];
                        all += sh.scan[o];
                    }
#pragma unroll
                    for (int j = 0; j < W; ++j) {
                        const int index = v * W - shift + j;
                        const bool is = v < end && index >= 0 && index < p.V &&
                                        (bound == -INFINITY ? !(x[i * W + j] > -INFINITY) : x[i * W + j] == bound);
                        if (is && at < want) sh.ties[carried + at] = key_of(x[i * W + j], index);
                        at += is;
                    }
                    found += all;
                }
                n_ties = carried + min(found, max(want, 0));
                __syncthreads();
            }
            // in order: each key counts those above it
            if (tid < kMost) sh.best[tid] = 0;
            __syncthreads();
            const int n = n_above + n_ties;
            for (int i = tid; i < n; i += kThreads) {
                const uint64_t key = i < n_above ? sh.above[i] : sh.ties[i - n_above];
                int place = 0;
                for (int o = 0; o < n_above; ++o) place += sh.above[o] > key;
                for (int o = 0; o < n_ties; ++o) place += sh.ties[o] > key;
                if (place < p.top) sh.best[place] = key;
            }
            __syncthreads();
            carried = p.top;
        }
    }

    // the CTA's sums, then the cluster's
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        const Sums o{__shfl_xor_sync(0xFFFFFFFFu, mine.m, d), __shfl_xor_sync(0xFFFFFFFFu, mine.s, d),
                     __shfl_xor_sync(0xFFFFFFFFu, mine.t, d)};
        mine = join(mine, o, p.heat_log2);
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
        if (tid == 0 && p.entropy != nullptr) p.entropy[row] = a.s == 0.f ? 0.f : log_s - p.heat * a.t / a.s;
        for (int i = tid; i < p.n; i += kThreads) {
            const int at = p.tokens[size_t(row) * p.n + i];
            p.logprobs[size_t(row) * p.n + i] = at >= 0 && at < p.V ? logprob(Vec<T>::one(x0 + at)) : -INFINITY;
        }
        if (kTop) {
            const int n = p.top << p.cluster_bits;
            for (int i = tid; i < n; i += kThreads)
                sh.above[i] = ld_cluster_u64(mapa_shared(smem_u32(&sh.best[i >> p.cluster_bits]), i & (cluster - 1)));
            __syncthreads();
            for (int i = tid; i < n; i += kThreads) {
                const uint64_t key = sh.above[i];
                int place = 0;
                for (int o = 0; o < n; ++o) place += sh.above[o] > key;
                if (place < p.top && key != 0) {
                    p.top_ids[size_t(row) * p.top + place] = index_of(key);
                    p.top_logprobs[size_t(row) * p.top + place] = logprob(logit_of(key));
                }
            }
        }
    }
    cluster_sync_all();                          // no CTA leaves while its shared memory is read
}

template <typename T, bool kTop>
w4v_status launch(const Args &a, int M, cudaStream_t stream) {
    if (launch_pdl_cluster(token_logprobs_kernel<T, kTop>, dim3(unsigned(M) << a.cluster_bits), dim3(kThreads), 0, stream,
                           1 << a.cluster_bits, a) != cudaSuccess) {
        cudaGetLastError();
        return W4V_ERR_CUDA;
    }
    return W4V_OK;
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
    // A row in one piece a CTA, as far as a cluster goes; few rows in smaller ones.
    a.cluster_bits = 0;
    while (1 << a.cluster_bits < kMaxCluster &&
           (V > (long long)kPiece << a.cluster_bits ||
            ((long long)M << a.cluster_bits < info->sm_count && V > 4096 << a.cluster_bits)))
        ++a.cluster_bits;
    if (half) return top > 0 ? launch<__half, true>(a, M, stream) : launch<__half, false>(a, M, stream);
    return top > 0 ? launch<float, true>(a, M, stream) : launch<float, false>(a, M, stream);
}

}  // namespace w4v
