// kv_pages.cu -- bookkeeping of a paged key/value cache on the device: pages
// handed out, given back, shared, moved down and copied.
//
// The lengths that drive it (accepted drafts) are on the device, so nothing
// here goes through the host.  Which pages are free follows from refs alone
// (refs[p] == 0): there is no free list to keep in order, and "lowest id
// first" is one scan of refs, which makes every result independent of the
// order in which threads run.
//
// Each call is one CTA that decides (block scans over refs and over the
// sequences) and, where data moves or many table entries change, a grid-wide
// kernel after it that applies what the first one wrote into the workspace.
// The decisions are latency (a few dependent passes over arrays of some
// KB); the copies run at HBM speed: pieces of 16 KB, a CTA each, so that a
// page of a few KB in many planes and one of a megabyte fill the GPU alike.
//
// Measured (one GB300, device time): 16 tokens more for 8 sequences and some
// of them taken back, 6.5 us for the two calls; 32 sequences dropped and
// forked anew, 32 pages of 16 x 64 KB copied, 15.5 us (8 of them the decision,
// 10 the copies' bound); 2048 of 4096 pages of 16 x 16 KB moved down, 87 us
// (75.2 for the copies, 6.7 TB/s; 8.6 the decision).  What grows: the decision
// passes over all pages up to the last one it hands out (8 sequences a page
// each, the lower 95 % of the pool live: 10 us at 2^12 pages, 24 at 2^16, 115 at
// 2^19), and holders of one partly filled page take their copies in turn, in one
// thread, 0.2 to 0.4 us each (8 sequences 13 us, 256 74 us, 4096 1.8 ms, against 11, 16
// and 107 us with pages of their own).
#include <algorithm>

#include "runtime.h"
#include "sm103_ptx.cuh"

namespace w4v {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kCopyThreads = 256;
constexpr uint32_t kCopyPiece = 16384;          // bytes of one plane's page that a CTA takes at a time

// Workspace: header, then ints.  Every call writes what it reads of it, so one
// workspace may serve pools of different sizes, whose arrays lie elsewhere.
struct Header {
    int copies;                                  // pairs in src/dst
    int ok;                                      // whether the second kernel has anything to apply
};
struct Work {
    Header *head;
    int32_t *list;        // [n_pages] free pages, lowest first; compact: new id of every page
    int32_t *src, *dst;   // [n_pages] copies
    int32_t *need;        // [S] kv_extend: pages a sequence needs
    int32_t *base;        // [S] kv_extend: first of them in list; kv_fork: rank of a fork's partial page, or -1
    int32_t *marks;       // [S] kv_extend: the last page is replaced by a copy; kv_fork: named as a child
};
__host__ __device__ inline size_t work_ints(int n_pages, int S) { return 4 + 3 * size_t(n_pages) + 3 * size_t(S); }

struct Args {
    void *pool;
    int32_t *refs, *table, *lengths;
    size_t page_bytes;
    int planes, n_pages, S, width, page;
    const int32_t *want;                         // new lengths
    const int32_t *parents, *children;
    int n;
    int32_t *short_out;
    int32_t *refs_out, *table_out;
    Work w;
};

// Sum over the block of one value a thread, and the sum of the threads before.
template <typename T>
__device__ __forceinline__ T block_scan(T v, T &before, T *warp_sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    T x = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const T y = __shfl_up_sync(0xFFFFFFFFu, x, d);
        if (lane >= d) x += y;
    }
    __syncthreads();                             // warp_sums may still be read from the last call
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    if (warp == 0) {
        T s = warp_sums[lane];
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const T y = __shfl_up_sync(0xFFFFFFFFu, s, d);
            if (lane >= d) s += y;
        }
        warp_sums[lane] = s;
    }
    __syncthreads();
    before = x - v + (warp > 0 ? warp_sums[warp - 1] : 0);
    return warp_sums[kPlanWarps - 1];
}
static_assert(kPlanWarps == 32, "one warp scans the warps' sums");

// The first `most` free pages into list; returns how many
// there are (a count of at least `most` may stop short of all).
__device__ int find_free(const Args &p, int most, int *warp_sums) {
    int found = 0;
    for (int p0 = 0; p0 < p.n_pages && found < most; p0 += 4 * kPlanThreads) {
        const int i = p0 + 4 * threadIdx.x;
        bool free[4];
        int mine = 0, before;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            free[j] = i + j < p.n_pages && p.refs[i + j] <= 0;
            mine += free[j];
        }
        const int all = block_scan(mine, before, warp_sums);
        int r = found + before;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (free[j] && r < most) p.w.list[r++] = i + j;
        found += all;
    }
    __syncthreads();
    return found;
}

__device__ __forceinline__ bool id_ok(int id, const Args &p) { return id >= 0 && id < p.n_pages; }
__device__ __forceinline__ int length_of(int s, const Args &p) { return min(max(p.lengths[s], 0), p.width * p.page); }
__device__ __forceinline__ int pages_of(int len, const Args &p) { return (len + p.page - 1) / p.page; }

__global__ void __launch_bounds__(kPlanThreads)
kv_extend_kernel(const Args p) {
    __shared__ int warp_sums[kPlanWarps];
    __shared__ long long wide_sums[kPlanWarps];  // sums of needs may pass 32 bits
    __shared__ int shared_last, bad, copies;
    grid_dep_wait();
    grid_dep_launch();
    if (threadIdx.x == 0) shared_last = bad = copies = 0;
    __syncthreads();
    // What each sequence needs: whole new pages, and one in place of a partly
    // filled last page that others hold too (marks).
    for (int s = threadIdx.x; s < p.S; s += kPlanThreads) {
        const int len = length_of(s, p), want = p.want[s];
        int need = 0, mark = 0;
        if (want > len) {
            if (want > p.width * p.page) {
                bad = 1;
            } else {
                need = pages_of(want, p) - pages_of(len, p);
                if (len % p.page != 0) {
                    const int id = p.table[size_t(s) * p.width + len / p.page];
                    if (id_ok(id, p) && p.refs[id] > 1) mark = shared_last = 1;
                }
            }
        }
        p.w.need[s] = need;
        p.w.marks[s] = mark;
    }
    __syncthreads();
    if (shared_last && threadIdx.x == 0) {
        // Sequences that hold the same last page take copies in ascending
        // order until one holder is left, which keeps the page: in turn,
        // since each decides on what the ones before it left.
        for (int s = 0; s < p.S; ++s) {
            if (!p.w.marks[s]) continue;
            const int id = p.table[size_t(s) * p.width + length_of(s, p) / p.page];
            if (p.refs[id] > 1) {
                p.refs[id] -= 1;
                p.w.need[s] += 1;
            } else {
                p.w.marks[s] = 0;
            }
        }
    }
    __syncthreads();
    long long total = 0;
    for (int s0 = 0; s0 < p.S; s0 += kPlanThreads) {
        const int s = s0 + threadIdx.x;
        long long before;
        const long long all = block_scan<long long>(s < p.S ? p.w.need[s] : 0, before, wide_sums);
        if (s < p.S) p.w.base[s] = int32_t(total + before);     // used only if total <= n_pages
        total += all;
    }
    const int most = int(min(total, (long long)p.n_pages + 1));
    const long long lack = bad ? 0 : total - find_free(p, most, warp_sums);
    const bool ok = !bad && lack <= 0;
    if (ok) {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        for (int s = warp; s < p.S; s += kPlanWarps) {
            int need = p.w.need[s];
            if (p.want[s] > length_of(s, p)) {
                const int len = length_of(s, p);
                int32_t *row = p.table + size_t(s) * p.width;
                int from = p.w.base[s], at = pages_of(len, p);
                if (shared_last && p.w.marks[s]) {
                    if (lane == 0) {
                        const int id = p.w.list[from], c = atomicAdd(&copies, 1);
                        p.w.src[c] = row[len / p.page];
                        p.w.dst[c] = id;
                        p.refs[id] = 1;
                        row[len / p.page] = id;
                    }
                    ++from;
                    --need;
                }
                for (int i = lane; i < need; i += 32) {
                    const int id = p.w.list[from + i];
                    p.refs[id] = 1;
                    row[at + i] = id;
                }
                __syncwarp();
                if (lane == 0) p.lengths[s] = p.want[s];
            }
        }
    } else if (shared_last) {
        __syncthreads();
        if (threadIdx.x == 0)
            for (int s = 0; s < p.S; ++s)
                if (p.w.marks[s]) p.refs[p.table[size_t(s) * p.width + length_of(s, p) / p.page]] += 1;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        p.w.head->copies = ok ? copies : 0;
        *p.short_out = ok ? 0 : bad ? -1 : int(min(lack, 0x7FFFFFFFll));
    }
}

// One warp per sequence; references are given back by atomics (integers, so
// their order does not matter).
__global__ void __launch_bounds__(kCopyThreads)
kv_truncate_kernel(const Args p) {
    grid_dep_wait();
    grid_dep_launch();
    const int s = blockIdx.x * (kCopyThreads / 32) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (s >= p.S) return;
    const int len = length_of(s, p), want = max(p.want[s], 0);
    if (want >= len) return;
    int32_t *row = p.table + size_t(s) * p.width;
    for (int i = pages_of(want, p) + lane; i < pages_of(len, p); i += 32) {
        const int id = row[i];
        if (id_ok(id, p)) atomicSub(p.refs + id, 1);
        row[i] = -1;
    }
    __syncwarp();
    if (lane == 0) p.lengths[s] = want;
}

__global__ void __launch_bounds__(kPlanThreads)
kv_fork_kernel(const Args p) {
    __shared__ int warp_sums[kPlanWarps];
    __shared__ int bad;
    grid_dep_wait();
    grid_dep_launch();
    if (threadIdx.x == 0) bad = 0;
    for (int i = threadIdx.x; i < p.n; i += kPlanThreads) {
        const int a = p.parents[i], c = p.children[i];
        if (a >= 0 && a < p.S) p.w.marks[a] = 0;
        if (c >= 0 && c < p.S) p.w.marks[c] = 0;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < p.n; i += kPlanThreads) {
        const int a = p.parents[i], c = p.children[i];
        if (a < 0 || a >= p.S || c < 0 || c >= p.S || p.lengths[c] > 0 || atomicExch(p.w.marks + c, 1) != 0) bad = 1;
    }
    __syncthreads();
    // a child that is a parent too would be read while it is written
    for (int i = threadIdx.x; i < p.n; i += kPlanThreads)
        if (p.parents[i] >= 0 && p.parents[i] < p.S && p.w.marks[p.parents[i]] != 0) bad = 1;
    __syncthreads();
    int total = 0, lack = 0;
    if (!bad) {
        // base: forks with a partly filled last page, in order (a child may
        // be named by fork i only, so base has room for every fork: n <= S)
        for (int i0 = 0; i0 < p.n; i0 += kPlanThreads) {
            const int i = i0 + threadIdx.x;
            int before;
            const bool part = i < p.n && length_of(p.parents[i], p) % p.page != 0;
            const int all = block_scan(int(part), before, warp_sums);
            if (i < p.n) p.w.base[i] = part ? total + before : -1;
            total += all;
        }
        lack = total - find_free(p, total, warp_sums);
        if (lack <= 0)
            for (int i = threadIdx.x; i < p.n; i += kPlanThreads) {
                const int r = p.w.base[i];
                if (r >= 0) {
                    const int len = length_of(p.parents[i], p);
                    p.w.src[r] = p.table[size_t(p.parents[i]) * p.width + len / p.page];
                    p.w.dst[r] = p.w.list[r];
                    p.refs[p.w.list[r]] = 1;
                }
            }
    }
    if (threadIdx.x == 0) {
        const bool ok = !bad && lack <= 0;
        p.w.head->copies = ok ? total : 0;
        p.w.head->ok = ok;
        *p.short_out = bad ? -1 : max(lack, 0);
    }
}

__global__ void __launch_bounds__(kPlanThreads)
kv_compact_kernel(const Args p) {
    __shared__ int warp_sums[kPlanWarps];
    grid_dep_wait();
    grid_dep_launch();
    int live = 0;
    for (int p0 = 0; p0 < p.n_pages; p0 += 4 * kPlanThreads) {
        const int i = p0 + 4 * threadIdx.x;
        int mine = 0, before;
#pragma unroll
        for (int j = 0; j < 4; ++j) mine += i + j < p.n_pages && p.refs[i + j] > 0;
        live += block_scan(mine, before, warp_sums);
    }
    // src: live pages from `live` on; dst: free pages below it (as many)
    int moves = 0, holes = 0;
    for (int p0 = 0; p0 < p.n_pages; p0 += 4 * kPlanThreads) {
        const int i = p0 + 4 * threadIdx.x;
        int mine = 0, before, ref[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            ref[j] = i + j < p.n_pages ? p.refs[i + j] : 0;
            // a piece of four may hold both kinds: counted in two halves of one int
            if (i + j < p.n_pages) mine += i + j >= live ? (ref[j] > 0 ? 0x10000 : 0) : (ref[j] > 0 ? 0 : 1);
        }
        const int all = block_scan(mine, before, warp_sums);
        int m = moves + (before >> 16), h = holes + (before & 0xFFFF);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (i + j >= p.n_pages) continue;
            p.w.list[i + j] = i + j;
            if (p.refs_out != p.refs) p.refs_out[i + j] = ref[j];
            if (i + j >= live && ref[j] > 0) p.w.src[m++] = i + j;
            if (i + j < live && ref[j] <= 0) p.w.dst[h++] = i + j;
        }
        moves += all >> 16;
        holes += all & 0xFFFF;
    }
    __syncthreads();
    for (int r = threadIdx.x; r < moves; r += kPlanThreads) {
        const int from = p.w.src[r], to = p.w.dst[r];
        const int ref = p.refs[from];
        p.w.list[from] = to;
        p.refs_out[to] = ref;
        p.refs_out[from] = 0;
    }
    if (threadIdx.x == 0) p.w.head->copies = moves;
}

struct CopyArgs {
    uint8_t *pool;
    size_t page_bytes;
    int planes, n_pages;
    const int32_t *src, *dst;
    const int *count;                            // null: n
    int n;
};

// Every copied page of every plane in pieces of 16 KB, a CTA each; four
// 16-byte loads of a thread are in flight together.
__device__ __forceinline__ void copy_pages(const CopyArgs &c) {
    const int n = c.count != nullptr ? *c.count : c.n;
    const uint32_t pieces = uint32_t((c.page_bytes + kCopyPiece - 1) / kCopyPiece);
    const long long items = (long long)n * c.planes * pieces;
    for (long long it = blockIdx.x; it < items; it += gridDim.x) {
        const uint32_t piece = uint32_t(it % pieces);
        const long long rest = it / pieces;
        const int plane = int(rest % c.planes), i = int(rest / c.planes);
        const int a = c.src[i], z = c.dst[i];
        if (a < 0 || a >= c.n_pages || z < 0 || z >= c.n_pages) continue;
        uint8_t *base = c.pool + size_t(plane) * c.n_pages * c.page_bytes + size_t(piece) * kCopyPiece;
        const uint4 *from = reinterpret_cast<const uint4 *>(base + size_t(a) * c.page_bytes);
        uint4 *to = reinterpret_cast<uint4 *>(base + size_t(z) * c.page_bytes);
        const size_t left = c.page_bytes - size_t(piece) * kCopyPiece;
        const int m = int((left < kCopyPiece ? left : kCopyPiece) / 16);
        uint4 v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int e = threadIdx.x + j * kCopyThreads;
            if (e < m) v[j] = from[e];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int e = threadIdx.x + j * kCopyThreads;
            if (e < m) to[e] = v[j];
        }
    }
}
static_assert(kCopyPiece == 4 * 16 * kCopyThreads, "four 16-byte loads a thread cover one piece");

__global__ void __launch_bounds__(kCopyThreads)
kv_copy_kernel(const CopyArgs c) {
    grid_dep_wait();
    grid_dep_launch();
    copy_pages(c);
}

// The forks' table rows and references, and the copies of partial pages.
__global__ void __launch_bounds__(kCopyThreads)
kv_fork_apply_kernel(const Args p, const CopyArgs c) {
    grid_dep_wait();
    grid_dep_launch();
    if (!p.w.head->ok) return;
    for (int i = blockIdx.x; i < p.n; i += gridDim.x) {
        const int len = length_of(p.parents[i], p), full = len / p.page, r = p.w.base[i];
        const int32_t *from = p.table + size_t(p.parents[i]) * p.width;
        int32_t *row = p.table + size_t(p.children[i]) * p.width;
        for (int e = threadIdx.x; e < p.width; e += kCopyThreads) {
            int id = -1;
            if (e < full) {
                id = from[e];
                if (id_ok(id, p)) atomicAdd(p.refs + id, 1);
            } else if (e == full && r >= 0) {
                id = p.w.dst[r];
            }
            row[e] = id;
        }
        if (threadIdx.x == 0) p.lengths[p.children[i]] = len;
    }
    copy_pages(c);
}

// Tables through the pages' new ids, and the moved pages.
__global__ void __launch_bounds__(kCopyThreads)
kv_compact_apply_kernel(const Args p, const CopyArgs c) {
    grid_dep_wait();
    grid_dep_launch();
    for (int s = blockIdx.x; s < p.S; s += gridDim.x) {
        const int n = pages_of(length_of(s, p), p);
        const size_t row = size_t(s) * p.width;
        for (int e = threadIdx.x; e < p.width; e += kCopyThreads) {
            const int id = p.table[row + e];
            p.table_out[row + e] = e < n && id_ok(id, p) ? p.w.list[id] : id;
        }
    }
    copy_pages(c);
}

Args make_args(const w4v_pages_t &g, void *ws) {
    Args a = {};
    a.pool = g.pool;
    a.refs = g.refs;
    a.table = g.table;
    a.lengths = g.lengths;
    a.page_bytes = g.page_bytes;
    a.planes = g.planes;
    a.n_pages = g.n_pages;
    a.S = g.S;
    a.width = g.table_width;
    a.page = g.page;
    if (ws != nullptr) {
        int32_t *w = static_cast<int32_t *>(ws);
        a.w.head = reinterpret_cast<Header *>(w);
        a.w.list = w + 4;
        a.w.src = a.w.list + g.n_pages;
        a.w.dst = a.w.src + g.n_pages;
        a.w.need = a.w.dst + g.n_pages;
        a.w.base = a.w.need + g.S;
        a.w.marks = a.w.base + g.S;
    }
    return a;
}

CopyArgs copy_args(const Args &a) {
    return CopyArgs{static_cast<uint8_t *>(a.pool), a.page_bytes, a.planes, a.n_pages, a.w.src, a.w.dst,
                    &a.w.head->copies, 0};
}

w4v_status launched(cudaError_t e) {
    if (e == cudaSuccess) return W4V_OK;
    cudaGetLastError();
    return W4V_ERR_CUDA;
}

}  // namespace

size_t kv_pages_ws_bytes(int n_pages, int S) { return work_ints(n_pages, S) * sizeof(int32_t); }

w4v_status launch_kv_extend(const w4v_pages_t &g, const int32_t *want, int32_t *short_out, void *ws,
                            cudaStream_t stream) {
    const DeviceInfo *info = nullptr;
    w4v_status st = device_info(&info);
    if (st != W4V_OK) return st;
    Args a = make_args(g, ws);
    a.want = want;
    a.short_out = short_out;
    st = launched(launch_pdl(kv_extend_kernel, dim3(1), dim3(kPlanThreads), 0, stream, a));
    if (st != W4V_OK) return st;
    return launched(launch_pdl(kv_copy_kernel, dim3(4 * info->sm_count), dim3(kCopyThreads), 0, stream, copy_args(a)));
}

w4v_status launch_kv_truncate(const w4v_pages_t &g, const int32_t *want, cudaStream_t stream) {
    const DeviceInfo *info = nullptr;
    w4v_status st = device_info(&info);
    if (st != W4V_OK) return st;
    Args a = make_args(g, nullptr);
    a.want = want;
    constexpr int kPer = kCopyThreads / 32;
    return launched(
        launch_pdl(kv_truncate_kernel, dim3((g.S + kPer - 1) / kPer), dim3(kCopyThreads), 0, stream, a));
}

w4v_status launch_kv_fork(const w4v_pages_t &g, const int32_t *parents, const int32_t *children, int n,
                          int32_t *short_out, void *ws, cudaStream_t stream) {
    const DeviceInfo *info = nullptr;
    w4v_status st = device_info(&info);
    if (st != W4V_OK) return st;
    Args a = make_args(g, ws);
    a.parents = parents;
    a.children = children;
    a.n = n;
    a.short_out = short_out;
    st = launched(launch_pdl(kv_fork_kernel, dim3(1), dim3(kPlanThreads), 0, stream, a));
    if (st != W4V_OK) return st;
    return launched(launch_pdl(kv_fork_apply_kernel, dim3(4 * info->sm_count), dim3(kCopyThreads), 0, stream, a,
                               copy_args(a)));
}

w4v_status launch_kv_compact(const w4v_pages_t &g, int32_t *refs_out, int32_t *table_out, void *ws,
                             cudaStream_t stream) {
    const DeviceInfo *info = nullptr;
    w4v_status st = device_info(&info);
    if (st != W4V_OK) return st;
    Args a = make_args(g, ws);
    a.refs_out = refs_out;
    a.table_out = table_out;
    st = launched(launch_pdl(kv_compact_kernel, dim3(1), dim3(kPlanThreads), 0, stream, a));
    if (st != W4V_OK) return st;
    return launched(launch_pdl(kv_compact_apply_kernel, dim3(4 * info->sm_count), dim3(kCopyThreads), 0, stream, a,
                               copy_args(a)));
}

w4v_status launch_kv_copy(void *pool, int planes, int n_pages, size_t page_bytes, const int32_t *src,
                          const int32_t *dst, int n, cudaStream_t stream) {
    const DeviceInfo *info = nullptr;
    w4v_status st = device_info(&info);
    if (st != W4V_OK) return st;
    const CopyArgs c{static_cast<uint8_t *>(pool), page_bytes, planes, n_pages, src, dst, nullptr, n};
    return launched(launch_pdl(kv_copy_kernel, dim3(4 * info->sm_count), dim3(kCopyThreads), 0, stream, c));
}

}  // namespace w4v
