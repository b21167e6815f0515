// api.cpp -- the C ABI: argument validation (before anything touches the
// GPU), workspace sizing, the host int4 packer, and dispatch to launchers.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "runtime.h"

namespace {

constexpr int kGroup = 128;
constexpr int kTile = 128;
constexpr int kBlockBytes = kTile * kGroup / 2;
// Nibble i of a packed word holds the code of k offset kNibbleK[i].
constexpr int kNibbleK[8] = {0, 2, 4, 6, 1, 3, 5, 7};

inline size_t packed_offset(int t, int g, int n_groups, int r, int j) {
    return (size_t(t) * n_groups + g) * kBlockBytes + (size_t(j) * kTile + r) * 16;
}

bool pack_shape_ok(int N, int K) { return N > 0 && K > 0 && K % kGroup == 0 && N % 8 == 0; }

}  // namespace

extern "C" {

const char *w4v_status_string(w4v_status s) {
    switch (s) {
        case W4V_OK: return "ok";
        case W4V_ERR_ARG: return "invalid argument (null pointer or bad flag)";
        case W4V_ERR_SHAPE: return "unsupported shape";
        case W4V_ERR_ALIGN: return "pointer not 16-byte aligned";
        case W4V_ERR_WORKSPACE: return "workspace missing or too small";
        case W4V_ERR_ARCH: return "current device is not sm_103 (GB300) or the library was built for another GPU";
        case W4V_ERR_CUDA: return "CUDA runtime or launch error";
        case W4V_ERR_TIMEOUT: return "a kernel abandoned a bounded wait";
    }
    return "unknown status";
}

size_t w4v_packed_bytes(int N, int K) {
    if (!pack_shape_ok(N, K)) return 0;
    const size_t tiles = (size_t(N) + kTile - 1) / kTile;
    return tiles * size_t(K / kGroup) * kBlockBytes;
}

w4v_status w4v_pack_int4(const uint8_t *q, int N, int K, void *out) {
    if (q == nullptr || out == nullptr) return W4V_ERR_ARG;
    if (!pack_shape_ok(N, K)) return W4V_ERR_SHAPE;
    const int n_groups = K / kGroup;
    const int n_tiles = (N + kTile - 1) / kTile;
    uint8_t *o = static_cast<uint8_t *>(out);
    for (int t = 0; t < n_tiles; ++t)
        for (int g = 0; g < n_groups; ++g)
            for (int r = 0; r < kTile; ++r) {
                const int n = t * kTile + r;
                for (int j = 0; j < 4; ++j) {
                    uint8_t *chunk = o + packed_offset(t, g, n_groups, r, j);
                    for (int w = 0; w < 4; ++w) {
                        const int k0 = g * kGroup + 32 * j + 8 * w;
                        uint32_t word = 0;
                        for (int i = 0; i < 8; ++i) {
                            const uint32_t code = n < N ? (q[size_t(n) * K + k0 + kNibbleK[i]] & 15u) : 8u;
                            word |= code << (4 * i);
                        }
                        for (int b = 0; b < 4; ++b) chunk[4 * w + b] = uint8_t(word >> (8 * b));
                    }
                }
            }
    return W4V_OK;
}

w4v_status w4v_unpack_int4(const void *packed, int N, int K, uint8_t *q) {
    if (q == nullptr || packed == nullptr) return W4V_ERR_ARG;
    if (!pack_shape_ok(N, K)) return W4V_ERR_SHAPE;
    const int n_groups = K / kGroup;
    const uint8_t *p = static_cast<const uint8_t *>(packed);
    for (int n = 0; n < N; ++n) {
        const int t = n / kTile, r = n % kTile;
        for (int g = 0; g < n_groups; ++g)
            for (int j = 0; j < 4; ++j) {
                const uint8_t *chunk = p + packed_offset(t, g, n_groups, r, j);
                for (int w = 0; w < 4; ++w) {
                    uint32_t word = 0;
                    for (int b = 0; b < 4; ++b) word |= uint32_t(chunk[4 * w + b]) << (8 * b);
                    const int k0 = g * kGroup + 32 * j + 8 * w;
                    for (int i = 0; i < 8; ++i) q[size_t(n) * K + k0 + kNibbleK[i]] = uint8_t((word >> (4 * i)) & 15u);
                }
            }
    }
    return W4V_OK;
}

size_t w4a16_workspace_bytes(int M, int N, int K) {
    if (M < 0 || !pack_shape_ok(N, K)) return 0;
    // M > 32: enough for the prefill kernel and for the 32-row blocks of
    // the batch-invariant path, whichever the call takes
    if (M > w4v::kDecodeMaxRows)
        return std::max(w4v::w4a16_prefill_ws_bytes(M, N, K), w4v::w4a16_decode_ws_bytes(w4v::kDecodeMaxRows, N, K));
    return w4v::w4a16_decode_ws_bytes(M, N, K);
}

w4v_status w4a16_gemm(const uint16_t *A, const void *Bq, const uint16_t *scales, const uint8_t *zeros, int group,
                      uint16_t *C, int M, int N, int K, void *ws, size_t ws_bytes, w4v_stream_t stream) {
    return w4a16_gemm_ex(A, Bq, scales, zeros, group, C, M, N, K, ws, ws_bytes, 0u, stream);
}

w4v_status w4a16_gemm_ex(const uint16_t *A, const void *Bq, const uint16_t *scales, const uint8_t *zeros,
                         int group, uint16_t *C, int M, int N, int K, void *ws, size_t ws_bytes, unsigned flags,
                         w4v_stream_t stream) {
    if ((flags & ~unsigned(W4V_STATIC_WEIGHTS | W4V_BATCH_INVARIANT)) != 0u) return W4V_ERR_ARG;
    if (M < 0 || N <= 0 || K <= 0) return W4V_ERR_SHAPE;
    if (group != kGroup && group != 32) return W4V_ERR_SHAPE;
    if (K % kGroup != 0 || N % 8 != 0) return W4V_ERR_SHAPE;
    if (zeros != nullptr && N % 16 != 0) return W4V_ERR_SHAPE;
    if (M == 0) return W4V_OK;
    if (A == nullptr || Bq == nullptr || scales == nullptr || C == nullptr) return W4V_ERR_ARG;
    if (!w4v::aligned16(A) || !w4v::aligned16(Bq) || !w4v::aligned16(scales) ||
        (zeros != nullptr && !w4v::aligned16(zeros)))
        return W4V_ERR_ALIGN;
    if (ws == nullptr || ws_bytes < w4a16_workspace_bytes(M, N, K)) return W4V_ERR_WORKSPACE;
    if (!w4v::aligned16(ws)) return W4V_ERR_ALIGN;
    const bool static_w = (flags & W4V_STATIC_WEIGHTS) != 0u;
    if (M > w4v::kDecodeMaxRows && (flags & W4V_BATCH_INVARIANT) != 0u) {
        // Blocks of 32 rows through the verify-sized kernel, in order on the
        // stream (each leaves the workspace zeroed for the next): every row
        // gets the arithmetic it gets in a call of 1..32 rows.
        for (int m0 = 0; m0 < M; m0 += w4v::kDecodeMaxRows) {
            const int mb = std::min(w4v::kDecodeMaxRows, M - m0);
            const w4v_status st = w4v::launch_w4a16_decode(A + size_t(m0) * K, Bq, scales, zeros, group,
                                                           C + size_t(m0) * N, mb, N, K, ws, static_w,
                                                           reinterpret_cast<cudaStream_t>(stream));
            if (st != W4V_OK) return st;
        }
        return W4V_OK;
    }
    if (M > w4v::kDecodeMaxRows)
        return w4v::launch_w4a16_prefill(A, Bq, scales, zeros, group, C, M, N, K, ws,
                                         reinterpret_cast<cudaStream_t>(stream));
    return w4v::launch_w4a16_decode(A, Bq, scales, zeros, group, C, M, N, K, ws, static_w,
                                    reinterpret_cast<cudaStream_t>(stream));
}

size_t w4a16_grouped_plan_bytes(int n_problems) {
    if (n_problems < 1 || n_problems > w4v::kGroupedMaxProblems) return 0;
    return w4v::w4a16_grouped_table_bytes(n_problems);
}

w4v_status w4a16_grouped_plan(const w4a16_problem *problems, int n, int M, int group, void *plan,
                              size_t plan_bytes, w4a16_grouped_t *handle, w4v_stream_t stream) {
    if (n < 1 || n > w4v::kGroupedMaxProblems || M < 1 || M > w4v::kDecodeMaxRows) return W4V_ERR_SHAPE;
    if (group != kGroup && group != 32) return W4V_ERR_SHAPE;
    if (problems == nullptr || plan == nullptr || handle == nullptr) return W4V_ERR_ARG;
    const bool zeros = problems[0].zeros != nullptr;
    for (int i = 0; i < n; ++i) {
        const w4a16_problem &q = problems[i];
        if (q.N <= 0 || q.K <= 0 || q.K % kGroup != 0 || q.N % 8 != 0) return W4V_ERR_SHAPE;
        if (zeros && q.N % 16 != 0) return W4V_ERR_SHAPE;
        if ((q.zeros != nullptr) != zeros) return W4V_ERR_ARG;
        if (q.A == nullptr || q.Bq == nullptr || q.scales == nullptr || q.C == nullptr) return W4V_ERR_ARG;
        if (!w4v::aligned16(q.A) || !w4v::aligned16(q.Bq) || !w4v::aligned16(q.scales) ||
            (q.zeros != nullptr && !w4v::aligned16(q.zeros)) || !w4v::aligned16(q.C))
            return W4V_ERR_ALIGN;
    }
    if (plan_bytes < w4v::w4a16_grouped_table_bytes(n)) return W4V_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(plan) & 63u) return W4V_ERR_ALIGN;
    cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
    if (cudaStreamIsCapturing(reinterpret_cast<cudaStream_t>(stream), &cap) != cudaSuccess) {
        cudaGetLastError();
        return W4V_ERR_CUDA;
    }
    if (cap != cudaStreamCaptureStatusNone) return W4V_ERR_ARG;
    const w4v::DeviceInfo *info = nullptr;
    w4v_status st = w4v::device_info(&info);
    if (st != W4V_OK) return st;
    return w4v::build_w4a16_grouped(problems, n, M, group, plan, handle, reinterpret_cast<cudaStream_t>(stream));
}

size_t w4a16_grouped_workspace_bytes(const w4a16_grouped_t *handle) {
    if (handle == nullptr || !w4v::w4a16_grouped_handle_ok(*handle)) return 0;
    return w4v::w4a16_grouped_ws_bytes(*handle);
}

w4v_status w4a16_gemm_grouped(const w4a16_grouped_t *handle, void *ws, size_t ws_bytes, unsigned flags,
                              w4v_stream_t stream) {
    if ((flags & ~unsigned(W4V_STATIC_WEIGHTS)) != 0u) return W4V_ERR_ARG;
    if (handle == nullptr || !w4v::w4a16_grouped_handle_ok(*handle)) return W4V_ERR_ARG;
    if (ws == nullptr || ws_bytes < w4v::w4a16_grouped_ws_bytes(*handle)) return W4V_ERR_WORKSPACE;
    if (!w4v::aligned16(ws)) return W4V_ERR_ALIGN;
    return w4v::launch_w4a16_grouped(*handle, ws, (flags & W4V_STATIC_WEIGHTS) != 0u,
                                     reinterpret_cast<cudaStream_t>(stream));
}

size_t w8_lmhead_argmax_workspace_bytes(int M, int V) {
    if (M < 0 || M > 128 || V <= 0) return 0;
    return w4v::w8_lmhead_ws_bytes(M, V);
}

w4v_status w8_lmhead_argmax(const uint16_t *X, const int8_t *W, const uint16_t *scale, int M, int K,
                            int V, int32_t *argmax_out, float *maxlogit, float *logits_debug,
                            void *ws, size_t ws_bytes, w4v_stream_t stream) {
    return w8_lmhead_argmax_ex(X, W, scale, M, K, V, argmax_out, maxlogit, logits_debug, ws, ws_bytes, 0u, stream);
}

namespace {
// The rows in blocks of at most 32, one launch each, in order on the stream
// (each leaves the workspace cleared for the next): every row gets the
// arithmetic of a call with 1..32 rows.
w4v_status lmhead_row_blocks(const uint16_t *X, const int8_t *W, const uint16_t *scale, int M, int K, int V,
                             int32_t *argmax_out, float *maxlogit, float *logits, void *ws, cudaStream_t stream) {
    for (int m0 = 0; m0 < M; m0 += w4v::kDecodeMaxRows) {
        const int mb = std::min(w4v::kDecodeMaxRows, M - m0);
        const w4v_status st = w4v::launch_w8_lmhead_argmax(
            X + size_t(m0) * K, W, scale, mb, K, V, argmax_out + m0, maxlogit != nullptr ? maxlogit + m0 : nullptr,
            logits != nullptr ? logits + size_t(m0) * V : nullptr, ws, stream);
        if (st != W4V_OK) return st;
    }
    return W4V_OK;
}
}  // namespace

w4v_status w8_lmhead_argmax_ex(const uint16_t *X, const int8_t *W, const uint16_t *scale, int M, int K,
                               int V, int32_t *argmax_out, float *maxlogit, float *logits_debug,
                               void *ws, size_t ws_bytes, unsigned flags, w4v_stream_t stream) {
    if ((flags & ~unsigned(W4V_BATCH_INVARIANT)) != 0u) return W4V_ERR_ARG;
    if (M < 0 || M > 128 || K <= 0 || V <= 0 || K % 128 != 0 || V % 8 != 0) return W4V_ERR_SHAPE;
    if (M == 0) return W4V_OK;
    if (X == nullptr || W == nullptr || scale == nullptr || argmax_out == nullptr) return W4V_ERR_ARG;
    if (!w4v::aligned16(X) || !w4v::aligned16(W) || !w4v::aligned16(scale)) return W4V_ERR_ALIGN;
    if ((reinterpret_cast<uintptr_t>(argmax_out) & 3u) || (reinterpret_cast<uintptr_t>(maxlogit) & 3u) ||
        (reinterpret_cast<uintptr_t>(logits_debug) & 3u))
        return W4V_ERR_ALIGN;
    if (ws == nullptr || ws_bytes < w4v::w8_lmhead_ws_bytes(M, V)) return W4V_ERR_WORKSPACE;
    if (!w4v::aligned16(ws)) return W4V_ERR_ALIGN;
    if (M > w4v::kDecodeMaxRows && (flags & W4V_BATCH_INVARIANT) != 0u)
        return lmhead_row_blocks(X, W, scale, M, K, V, argmax_out, maxlogit, logits_debug, ws,
                                 reinterpret_cast<cudaStream_t>(stream));
    return w4v::launch_w8_lmhead_argmax(X, W, scale, M, K, V, argmax_out, maxlogit, logits_debug, ws,
                                        reinterpret_cast<cudaStream_t>(stream));
}

w4v_status w8_lmhead_argmax_accept(const uint16_t *X, const int8_t *W, const uint16_t *scale, int B, int n_draft,
                                   int K, int V, const int32_t *draft, int32_t *argmax_out, int32_t *n_accepted,
                                   int32_t *out_tokens, float *maxlogit, void *ws, size_t ws_bytes,
                                   w4v_stream_t stream) {
    return w8_lmhead_argmax_accept_ex(X, W, scale, B, n_draft, K, V, draft, argmax_out, n_accepted, out_tokens,
                                      maxlogit, ws, ws_bytes, 0u, stream);
}

w4v_status w8_lmhead_argmax_accept_ex(const uint16_t *X, const int8_t *W, const uint16_t *scale, int B,
                                      int n_draft, int K, int V, const int32_t *draft, int32_t *argmax_out,
                                      int32_t *n_accepted, int32_t *out_tokens, float *maxlogit, void *ws,
                                      size_t ws_bytes, unsigned flags, w4v_stream_t stream) {
    if ((flags & ~unsigned(W4V_BATCH_INVARIANT)) != 0u) return W4V_ERR_ARG;
    if (B < 0 || n_draft < 0 || K <= 0 || V <= 0 || K % 128 != 0 || V % 8 != 0) return W4V_ERR_SHAPE;
    if (B > 128 || long(B) * (n_draft + 1) > 128) return W4V_ERR_SHAPE;
    if (B == 0) return W4V_OK;
    const int M = B * (n_draft + 1);
    if (X == nullptr || W == nullptr || scale == nullptr || argmax_out == nullptr || n_accepted == nullptr ||
        (n_draft > 0 && draft == nullptr))
        return W4V_ERR_ARG;
    if (!w4v::aligned16(X) || !w4v::aligned16(W) || !w4v::aligned16(scale)) return W4V_ERR_ALIGN;
    if ((reinterpret_cast<uintptr_t>(argmax_out) & 3u) || (reinterpret_cast<uintptr_t>(maxlogit) & 3u) ||
        (reinterpret_cast<uintptr_t>(draft) & 3u) || (reinterpret_cast<uintptr_t>(n_accepted) & 3u) ||
        (reinterpret_cast<uintptr_t>(out_tokens) & 3u))
        return W4V_ERR_ALIGN;
    if (ws == nullptr || ws_bytes < w4v::w8_lmhead_ws_bytes(M, V)) return W4V_ERR_WORKSPACE;
    if (!w4v::aligned16(ws)) return W4V_ERR_ALIGN;
    if (M > w4v::kDecodeMaxRows && (flags & W4V_BATCH_INVARIANT) != 0u) {
        // the row blocks' tokens, then the acceptance of every sequence over them
        const w4v_status st = lmhead_row_blocks(X, W, scale, M, K, V, argmax_out, maxlogit, nullptr, ws,
                                                reinterpret_cast<cudaStream_t>(stream));
        if (st != W4V_OK) return st;
        return w4v::launch_spec_accept(argmax_out, draft, B, n_draft, n_accepted, out_tokens,
                                       reinterpret_cast<cudaStream_t>(stream));
    }
    const w4v::LmAccept acc{draft, B, n_draft, n_accepted, out_tokens};
    return w4v::launch_w8_lmhead_argmax(X, W, scale, M, K, V, argmax_out, maxlogit, nullptr, ws,
                                        reinterpret_cast<cudaStream_t>(stream), &acc);
}

size_t ngram_draft_workspace_bytes(int B) {
    if (B < 0 || B > 65535) return 0;
    return w4v::ngram_ws_bytes(B);
}

w4v_status ngram_draft(const int32_t *context, const int32_t *lengths, int B, int ld, int n_min, int n_max, int K,
                       int32_t *drafts, int32_t *match_len, void *ws, size_t ws_bytes, w4v_stream_t stream) {
    if (B < 0 || B > 65535 || ld < 1 || n_min < 1 || n_max < n_min || n_max > w4v::kNgramMax || K < 0 || K > 1024)
        return W4V_ERR_SHAPE;
    if (B == 0) return W4V_OK;
    if (context == nullptr || lengths == nullptr || (K > 0 && drafts == nullptr)) return W4V_ERR_ARG;
    if ((reinterpret_cast<uintptr_t>(context) & 3u) || (reinterpret_cast<uintptr_t>(lengths) & 3u) ||
        (reinterpret_cast<uintptr_t>(drafts) & 3u) || (reinterpret_cast<uintptr_t>(match_len) & 3u))
        return W4V_ERR_ALIGN;
    if (ws == nullptr || ws_bytes < w4v::ngram_ws_bytes(B)) return W4V_ERR_WORKSPACE;
    if (!w4v::aligned16(ws)) return W4V_ERR_ALIGN;
    return w4v::launch_ngram_draft(context, lengths, B, ld, n_min, n_max, K, drafts, match_len, ws,
                                   reinterpret_cast<cudaStream_t>(stream));
}

namespace {
w4v_status gdn_check(const float *state, const uint16_t *k, const uint16_t *v, const float *alpha,
                     const float *beta, int B, int T, int H, int dk, int dv) {
    if (B < 0 || B > 65535 || T < 1 || T > w4v::kGdnMaxT || H < 1 || H > 65535 || dk != w4v::kGdnDk || dv < 32 ||
        dv % 32 != 0 || dv > 4096)
        return W4V_ERR_SHAPE;
    if (B == 0) return W4V_OK;
    if (state == nullptr || k == nullptr || v == nullptr || alpha == nullptr || beta == nullptr) return W4V_ERR_ARG;
    if (!w4v::aligned16(state) || !w4v::aligned16(k) || !w4v::aligned16(v) ||
        (reinterpret_cast<uintptr_t>(alpha) & 3u) || (reinterpret_cast<uintptr_t>(beta) & 3u))
        return W4V_ERR_ALIGN;
    return W4V_OK;
}
}  // namespace

w4v_status gdn_verify(const float *state, const uint16_t *q, const uint16_t *k, const uint16_t *v,
                      const float *alpha, const float *beta, int B, int T, int H, int dk, int dv, uint16_t *o,
                      w4v_stream_t stream) {
    w4v_status st = gdn_check(state, k, v, alpha, beta, B, T, H, dk, dv);
    if (st != W4V_OK || B == 0) return st;
    if (q == nullptr || o == nullptr) return W4V_ERR_ARG;
    if (!w4v::aligned16(q) || !w4v::aligned16(o)) return W4V_ERR_ALIGN;
    return w4v::launch_gdn(false, const_cast<float *>(state), q, k, v, alpha, beta, nullptr, o, B, T, H, dv,
                           reinterpret_cast<cudaStream_t>(stream));
}

w4v_status gdn_commit(float *state, const uint16_t *k, const uint16_t *v, const float *alpha, const float *beta,
                      const int32_t *n_accepted, int B, int T, int H, int dk, int dv, w4v_stream_t stream) {
    w4v_status st = gdn_check(state, k, v, alpha, beta, B, T, H, dk, dv);
    if (st != W4V_OK || B == 0) return st;
    if (n_accepted == nullptr) return W4V_ERR_ARG;
    if (reinterpret_cast<uintptr_t>(n_accepted) & 3u) return W4V_ERR_ALIGN;
    return w4v::launch_gdn(true, state, nullptr, k, v, alpha, beta, n_accepted, nullptr, B, T, H, dv,
                           reinterpret_cast<cudaStream_t>(stream));
}

w4v_status gdn_step(float *state, const uint16_t *k_prev, const uint16_t *v_prev, const float *alpha_prev,
                    const float *beta_prev, const int32_t *n_prev, int T_prev, const uint16_t *q, const uint16_t *k,
                    const uint16_t *v, const float *alpha, const float *beta, int B, int T, int H, int dk, int dv,
                    uint16_t *o, w4v_stream_t stream) {
    w4v_status st = gdn_check(state, k, v, alpha, beta, B, T, H, dk, dv);
    if (st != W4V_OK) return st;
    if (T_prev < 0 || T_prev > w4v::kGdnMaxT) return W4V_ERR_SHAPE;
    if (B == 0) return W4V_OK;
    if (q == nullptr || o == nullptr) return W4V_ERR_ARG;
    if (!w4v::aligned16(q) || !w4v::aligned16(o)) return W4V_ERR_ALIGN;
    if (T_prev > 0) {
        st = gdn_check(state, k_prev, v_prev, alpha_prev, beta_prev, B, T_prev, H, dk, dv);
        if (st != W4V_OK) return st;
        if (n_prev == nullptr) return W4V_ERR_ARG;
        if (reinterpret_cast<uintptr_t>(n_prev) & 3u) return W4V_ERR_ALIGN;
    }
    return w4v::launch_gdn_step(state, k_prev, v_prev, alpha_prev, beta_prev, n_prev, T_prev, q, k, v, alpha, beta,
                                o, B, T, H, dv, reinterpret_cast<cudaStream_t>(stream));
}

w4v_status spec_accept(const int32_t *target, const int32_t *draft, int B, int K, int32_t *n_accepted,
                       int32_t *out_tokens, w4v_stream_t stream) {
    if (B < 0 || K < 0 || K > 1024) return W4V_ERR_SHAPE;
    if (B == 0) return W4V_OK;
    if (target == nullptr || n_accepted == nullptr || (K > 0 && draft == nullptr)) return W4V_ERR_ARG;
    if ((reinterpret_cast<uintptr_t>(target) & 3u) || (reinterpret_cast<uintptr_t>(draft) & 3u) ||
        (reinterpret_cast<uintptr_t>(n_accepted) & 3u) || (reinterpret_cast<uintptr_t>(out_tokens) & 3u))
        return W4V_ERR_ALIGN;
    return w4v::launch_spec_accept(target, draft, B, K, n_accepted, out_tokens,
                                   reinterpret_cast<cudaStream_t>(stream));
}

namespace {
bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
}  // namespace

w4v_status token_logprobs(const void *logits, long long row_stride, int M, int V, const int32_t *tokens, int n,
                          float temperature, float *logprobs, float *entropy, int top, int32_t *top_ids,
                          float *top_logprobs, unsigned flags, w4v_stream_t stream) {
    if ((flags & ~unsigned(W4V_LOGITS_FP16)) != 0u) return W4V_ERR_ARG;
    const bool half = (flags & W4V_LOGITS_FP16) != 0u;
    if (M < 0 || M > 1 << 24 || V < 1 || V > 1 << 28 || n < 0 || n > 1 << 20 || top < 0 || top > w4v::kLogprobsMaxTop ||
        top > V || row_stride < V || row_stride >= 1ll << 38)
        return W4V_ERR_SHAPE;
    if (!(temperature > 0.f) || !std::isfinite(temperature) || !std::isfinite(1.4426951f / temperature)) return W4V_ERR_ARG;
    if (M == 0) return W4V_OK;
    if (logits == nullptr || (n > 0 && (tokens == nullptr || logprobs == nullptr)) ||
        (top > 0 && (top_ids == nullptr || top_logprobs == nullptr)))
        return W4V_ERR_ARG;
    if ((reinterpret_cast<uintptr_t>(logits) & (half ? 1u : 3u)) != 0u || !aligned4(tokens) || !aligned4(logprobs) ||
        !aligned4(entropy) || !aligned4(top_ids) || !aligned4(top_logprobs))
        return W4V_ERR_ALIGN;
    return w4v::launch_token_logprobs(logits, half, row_stride, M, V, tokens, n, temperature, logprobs, entropy, top,
                                      top_ids, top_logprobs, reinterpret_cast<cudaStream_t>(stream));
}

namespace {
bool page_ok(int page) { return page >= 8 && page <= 256 && (page & (page - 1)) == 0; }

// The cache, and the rows that go with it (after n_tokens == 0 returned).
w4v_status kv_check(const w4v_kv_t *kv, int n_tokens, int q_heads) {
    if (kv == nullptr) return W4V_ERR_ARG;
    const int D = kv->head_dim;
    if (n_tokens < 0 || q_heads < 1 || kv->B < 0 || kv->table_width < 1 || kv->n_pages < 1 || kv->kv_heads < 1 ||
        !page_ok(kv->page) || (D != 64 && D != 128 && D != 256))
        return W4V_ERR_SHAPE;
    if ((long long)kv->table_width * kv->page >= 1ll << 31) return W4V_ERR_SHAPE;
    if ((long long)kv->n_pages * kv->kv_heads >= (1ll << 34) / kv->page) return W4V_ERR_SHAPE;
    if (n_tokens == 0 || kv->B == 0) return W4V_OK;
    if (kv->k == nullptr || kv->v == nullptr || kv->table == nullptr || kv->lengths == nullptr ||
        kv->offsets == nullptr)
        return W4V_ERR_ARG;
    if (!w4v::aligned16(kv->k) || !w4v::aligned16(kv->v) || !aligned4(kv->table) || !aligned4(kv->lengths) ||
        !aligned4(kv->offsets))
        return W4V_ERR_ALIGN;
    return W4V_OK;
}
bool stride_ok(long long stride, int heads, int head_dim) {
    return stride % 8 == 0 && stride >= (long long)heads * head_dim && stride < 1ll << 38;
}
}  // namespace

namespace {
// rope_append and, with norms, norm_rope_append.
w4v_status append(const w4v_kv_t *kv, const uint16_t *q, const uint16_t *k, const uint16_t *v, long long q_stride,
                  long long k_stride, long long v_stride, int n_tokens, int q_heads, const w4v::HeadNorm *norm,
                  const int32_t *positions, const uint64_t *phases, int rot, float mul, bool interleaved,
                  uint16_t *q_out, w4v_stream_t stream) {
    const w4v_status st = kv_check(kv, n_tokens, q_heads);
    if (st != W4V_OK) return st;
    const int D = kv->head_dim, Hk = kv->kv_heads;
    if (rot < 0 || rot > D || rot % 2 != 0 || !stride_ok(q_stride, q_heads, D) || !stride_ok(k_stride, Hk, D) ||
        !stride_ok(v_stride, Hk, D))
        return W4V_ERR_SHAPE;
    if (norm != nullptr && (!(norm->eps >= 0.f) || !std::isfinite(norm->eps))) return W4V_ERR_ARG;
    if (n_tokens == 0 || kv->B == 0) return W4V_OK;
    if (q == nullptr || k == nullptr || v == nullptr || q_out == nullptr || (rot > 0 && phases == nullptr))
        return W4V_ERR_ARG;
    if (q_out == q && q_stride != (long long)q_heads * D) return W4V_ERR_ARG;
    if (!w4v::aligned16(q) || !w4v::aligned16(k) || !w4v::aligned16(v) || !w4v::aligned16(q_out) ||
        !aligned4(positions) || (reinterpret_cast<uintptr_t>(phases) & 7u) != 0u)
        return W4V_ERR_ALIGN;
    if (norm != nullptr && (!w4v::aligned16(norm->q_weight) || !w4v::aligned16(norm->k_weight))) return W4V_ERR_ALIGN;
    return w4v::launch_rope_append(*kv, q, k, v, q_stride, k_stride, v_stride, n_tokens, q_heads, positions, phases,
                                   rot, mul, interleaved, norm, q_out, reinterpret_cast<cudaStream_t>(stream));
}
}  // namespace

w4v_status rope_append(const w4v_kv_t *kv, const uint16_t *q, const uint16_t *k, const uint16_t *v,
                       long long q_stride, long long k_stride, long long v_stride, int n_tokens, int q_heads,
                       const int32_t *positions, const uint64_t *phases, int rot, float mul, unsigned flags,
                       uint16_t *q_out, w4v_stream_t stream) {
    if ((flags & ~unsigned(W4V_ROPE_INTERLEAVED)) != 0u) return W4V_ERR_ARG;
    return append(kv, q, k, v, q_stride, k_stride, v_stride, n_tokens, q_heads, nullptr, positions, phases, rot, mul,
                  (flags & W4V_ROPE_INTERLEAVED) != 0u, q_out, stream);
}

w4v_status norm_rope_append(const w4v_kv_t *kv, const uint16_t *q, const uint16_t *k, const uint16_t *v,
                            long long q_stride, long long k_stride, long long v_stride, int n_tokens, int q_heads,
                            const uint16_t *q_weight, const uint16_t *k_weight, float eps, const int32_t *positions,
                            const uint64_t *phases, int rot, float mul, unsigned flags, uint16_t *q_out,
                            w4v_stream_t stream) {
    if ((flags & ~unsigned(W4V_ROPE_INTERLEAVED | W4V_NORM_ZERO_CENTRED)) != 0u) return W4V_ERR_ARG;
    const w4v::HeadNorm norm{q_weight, k_weight, eps, (flags & W4V_NORM_ZERO_CENTRED) != 0u};
    return append(kv, q, k, v, q_stride, k_stride, v_stride, n_tokens, q_heads, &norm, positions, phases, rot, mul,
                  (flags & W4V_ROPE_INTERLEAVED) != 0u, q_out, stream);
}

w4v_status rope_phases(int rot, double base, int scaling, const double *params, uint64_t *phases, float *mul_out) {
    if (scaling < W4V_ROPE_PLAIN || scaling > W4V_ROPE_BANDED || phases == nullptr || mul_out == nullptr ||
        (scaling != W4V_ROPE_PLAIN && params == nullptr))
        return W4V_ERR_ARG;
    if (rot < 2 || rot % 2 != 0 || rot > 256 || !(base > 1.0) || !std::isfinite(base)) return W4V_ERR_SHAPE;
    const double factor = scaling != W4V_ROPE_PLAIN ? params[0] : 1.0;
    if (!(factor >= 1.0) || !std::isfinite(factor)) return W4V_ERR_SHAPE;
    constexpr double kTurn = 6.283185307179586476925286766559;
    double lo = 0.0, hi = 1.0, context = 0.0;
    *mul_out = 1.f;
    if (scaling == W4V_ROPE_NTK) {
        if (rot == 2) return W4V_ERR_SHAPE;
        base *= std::pow(factor, double(rot) / (rot - 2));
    } else if (scaling == W4V_ROPE_YARN) {
        context = params[1];
        const double fast = params[2], slow = params[3];
        if (!(context > 0.0) || !(slow > 0.0) || !(fast > slow)) return W4V_ERR_SHAPE;
        // the pair index that turns b times in `context` positions
        auto pair = [&](double b) { return rot * std::log(context / (b * kTurn)) / (2.0 * std::log(base)); };
        lo = std::max(std::floor(pair(fast)), 0.0);
        hi = std::min(std::ceil(pair(slow)), rot - 1.0);
        *mul_out = float(0.1 * std::log(factor) + 1.0);
    } else if (scaling == W4V_ROPE_BANDED) {
        lo = params[1];
        hi = params[2];
        context = params[3];
        if (!(context > 0.0) || !(lo > 0.0) || !(hi > lo)) return W4V_ERR_SHAPE;
    }
    for (int i = 0; i < rot / 2; ++i) {
        double f = std::pow(base, -2.0 * i / rot);
        if (scaling == W4V_ROPE_LINEAR) f /= factor;
        if (scaling == W4V_ROPE_YARN) {
            const double slow_part = std::min(std::max((i - lo) / std::max(hi - lo, 0.001), 0.0), 1.0);
            f = f / factor * slow_part + f * (1.0 - slow_part);
        }
        if (scaling == W4V_ROPE_BANDED) {
            const double kept = std::min(std::max((context * f / kTurn - lo) / (hi - lo), 0.0), 1.0);
            f = f / factor * (1.0 - kept) + f * kept;
        }
        phases[i] = uint64_t(std::ldexp(f / kTurn, 64));      // f <= 1 radian: below 2^62
    }
    return W4V_OK;
}

size_t paged_attn_workspace_bytes(int n_tokens, int B, int q_heads, int kv_heads, int head_dim, int max_context,
                                  unsigned flags) {
    if (n_tokens < 0 || B < 0 || q_heads < 1 || kv_heads < 1 || q_heads % kv_heads != 0 ||
        q_heads / kv_heads > w4v::kAttnMaxGroup || (head_dim != 64 && head_dim != 128 && head_dim != 256) ||
        max_context < 0 || (flags & ~unsigned(W4V_BATCH_INVARIANT)) != 0u)
        return 0;
    return w4v::paged_attn_ws_bytes(n_tokens, B, q_heads, kv_heads, head_dim, max_context,
                                    (flags & W4V_BATCH_INVARIANT) != 0u);
}

w4v_status paged_attn(const w4v_kv_t *kv, const uint16_t *q, long long q_stride, int n_tokens, int q_heads,
                      float scale, int window, uint16_t *out, float *lse, void *ws, size_t ws_bytes, unsigned flags,
                      w4v_stream_t stream) {
    return paged_attn_sinks(kv, q, q_stride, n_tokens, q_heads, scale, window, 0, out, lse, ws, ws_bytes, flags, stream);
}

namespace {
// What paged_attn_sinks and paged_attn_shared check alike; `sizes`: whether what
// they have apart is in range.  *done: nothing to compute.
w4v_status attention_check(const w4v_kv_t *kv, const uint16_t *q, long long q_stride, int n_tokens, int q_heads, float scale,
                           bool sizes, int groups, const uint16_t *out, const float *lse, bool *done) {
    *done = false;
    const w4v_status st = kv_check(kv, n_tokens, q_heads);
    if (st != W4V_OK) return st;
    if (q_heads % kv->kv_heads != 0 || q_heads / kv->kv_heads > w4v::kAttnMaxGroup || !sizes ||
        !stride_ok(q_stride, q_heads, kv->head_dim))
        return W4V_ERR_SHAPE;
    // row tiles times key tiles of a whole table row (and the units that stand
    // for a row tile's other work): counted in 32 bits
    const int tok = w4v::kAttnMaxGroup / (q_heads / kv->kv_heads);
    double tiles = n_tokens / tok + std::min(kv->B, n_tokens);
    if (groups > 0) tiles += n_tokens / tok + std::min(groups, n_tokens);
    if (tiles * kv->kv_heads * (double(kv->table_width) * kv->page / 128 + 5) >= 2147483648.0) return W4V_ERR_SHAPE;
    if (!(scale > 0.f) || !std::isfinite(scale)) return W4V_ERR_ARG;
    *done = n_tokens == 0 || kv->B == 0;
    if (*done) return W4V_OK;
    if (q == nullptr || out == nullptr) return W4V_ERR_ARG;
    if (!w4v::aligned16(q) || !w4v::aligned16(out) || !aligned4(lse)) return W4V_ERR_ALIGN;
    return W4V_OK;
}
}  // namespace

w4v_status paged_attn_sinks(const w4v_kv_t *kv, const uint16_t *q, long long q_stride, int n_tokens, int q_heads,
                            float scale, int window, int sinks, uint16_t *out, float *lse, void *ws, size_t ws_bytes,
                            unsigned flags, w4v_stream_t stream) {
    if ((flags & ~unsigned(W4V_BATCH_INVARIANT)) != 0u) return W4V_ERR_ARG;
    bool done;
    const w4v_status st =
        attention_check(kv, q, q_stride, n_tokens, q_heads, scale, window >= 0 && sinks >= 0, 0, out, lse, &done);
    if (st != W4V_OK || done) return st;
    const bool inv = (flags & W4V_BATCH_INVARIANT) != 0u;
    if (ws == nullptr || ws_bytes < w4v::paged_attn_ws_bytes(n_tokens, kv->B, q_heads, kv->kv_heads, kv->head_dim,
                                                             kv->table_width * kv->page, inv))
        return W4V_ERR_WORKSPACE;
    if (!w4v::aligned16(ws)) return W4V_ERR_ALIGN;
    // (first tokens past the table's are all that a row can see)
    return w4v::launch_paged_attn(*kv, q, q_stride, n_tokens, q_heads, scale, window,
                                  std::min(sinks, kv->table_width * kv->page), nullptr, out, lse, ws, inv,
                                  reinterpret_cast<cudaStream_t>(stream));
}

size_t paged_attn_shared_workspace_bytes(int n_tokens, int B, int n_groups, int q_heads, int kv_heads, int head_dim) {
    if (n_groups < 0 || paged_attn_workspace_bytes(n_tokens, B, q_heads, kv_heads, head_dim, 0, 0u) == 0) return 0;
    return w4v::paged_attn_shared_ws_bytes(n_tokens, q_heads, kv_heads, head_dim);
}

w4v_status paged_attn_shared(const w4v_kv_t *kv, const uint16_t *q, long long q_stride, int n_tokens, int q_heads,
                             float scale, const int32_t *groups, const int32_t *prefix, int n_groups, uint16_t *out,
                             float *lse, void *ws, size_t ws_bytes, unsigned flags, w4v_stream_t stream) {
    if (flags != 0u) return W4V_ERR_ARG;
    bool done;
    const bool sizes = n_groups >= 0 && (kv == nullptr || kv->B == 0 || n_groups <= kv->B);
    const w4v_status st = attention_check(kv, q, q_stride, n_tokens, q_heads, scale, sizes, n_groups, out, lse, &done);
    if (st != W4V_OK || done) return st;
    if (n_groups > 0 && (groups == nullptr || prefix == nullptr)) return W4V_ERR_ARG;
    if (!aligned4(groups) || !aligned4(prefix)) return W4V_ERR_ALIGN;
    if (ws == nullptr || ws_bytes < w4v::paged_attn_shared_ws_bytes(n_tokens, q_heads, kv->kv_heads, kv->head_dim))
        return W4V_ERR_WORKSPACE;
    if (!w4v::aligned16(ws)) return W4V_ERR_ALIGN;
    const w4v::PrefixGroups shared{groups, prefix, n_groups};
    return w4v::launch_paged_attn(*kv, q, q_stride, n_tokens, q_heads, scale, 0, 0, &shared, out, lse, ws, false,
                                  reinterpret_cast<cudaStream_t>(stream));
}

size_t kv_workspace_bytes(int n_pages, int S) {
    if (n_pages < 1 || n_pages > 1 << 24 || S < 0 || S > 65535) return 0;
    return w4v::kv_pages_ws_bytes(n_pages, S);
}

namespace {
w4v_status pages_check(const w4v_pages_t *g, bool copies) {
    if (g == nullptr) return W4V_ERR_ARG;
    if (g->n_pages < 1 || g->n_pages > 1 << 24 || g->S < 0 || g->S > 65535 || g->table_width < 1 ||
        !page_ok(g->page) || (long long)g->table_width * g->page >= 1ll << 31)
        return W4V_ERR_SHAPE;
    if (copies && (g->planes < 0 || g->page_bytes % 16 != 0 || g->page_bytes >= size_t(1) << 31)) return W4V_ERR_SHAPE;
    if (g->S == 0) return W4V_OK;
    if (g->refs == nullptr || g->table == nullptr || g->lengths == nullptr ||
        (copies && g->planes > 0 && g->pool == nullptr))
        return W4V_ERR_ARG;
    if (!aligned4(g->refs) || !aligned4(g->table) || !aligned4(g->lengths) || (copies && !w4v::aligned16(g->pool)))
        return W4V_ERR_ALIGN;
    return W4V_OK;
}
w4v_status pages_ws_check(const w4v_pages_t *g, const void *ws, size_t ws_bytes) {
    if (ws == nullptr || ws_bytes < w4v::kv_pages_ws_bytes(g->n_pages, g->S)) return W4V_ERR_WORKSPACE;
    return w4v::aligned16(ws) ? W4V_OK : W4V_ERR_ALIGN;
}
}  // namespace

w4v_status kv_extend(const w4v_pages_t *pages, const int32_t *new_lengths, int32_t *short_out, void *ws,
                     size_t ws_bytes, w4v_stream_t stream) {
    w4v_status st = pages_check(pages, true);
    if (st != W4V_OK || pages->S == 0) return st;
    if (new_lengths == nullptr || short_out == nullptr) return W4V_ERR_ARG;
    if (!aligned4(new_lengths) || !aligned4(short_out)) return W4V_ERR_ALIGN;
    st = pages_ws_check(pages, ws, ws_bytes);
    if (st != W4V_OK) return st;
    return w4v::launch_kv_extend(*pages, new_lengths, short_out, ws, reinterpret_cast<cudaStream_t>(stream));
}

w4v_status kv_truncate(const w4v_pages_t *pages, const int32_t *new_lengths, w4v_stream_t stream) {
    const w4v_status st = pages_check(pages, false);
    if (st != W4V_OK || pages->S == 0) return st;
    if (new_lengths == nullptr) return W4V_ERR_ARG;
    if (!aligned4(new_lengths)) return W4V_ERR_ALIGN;
    return w4v::launch_kv_truncate(*pages, new_lengths, reinterpret_cast<cudaStream_t>(stream));
}

w4v_status kv_fork(const w4v_pages_t *pages, const int32_t *parents, const int32_t *children, int n,
                   int32_t *short_out, void *ws, size_t ws_bytes, w4v_stream_t stream) {
    w4v_status st = pages_check(pages, true);
    if (st != W4V_OK) return st;
    if (n < 0 || n > pages->S) return W4V_ERR_SHAPE;
    if (pages->S == 0) return W4V_OK;
    if ((n > 0 && (parents == nullptr || children == nullptr)) || short_out == nullptr) return W4V_ERR_ARG;
    if (!aligned4(parents) || !aligned4(children) || !aligned4(short_out)) return W4V_ERR_ALIGN;
    st = pages_ws_check(pages, ws, ws_bytes);
    if (st != W4V_OK) return st;
    return w4v::launch_kv_fork(*pages, parents, children, n, short_out, ws, reinterpret_cast<cudaStream_t>(stream));
}

w4v_status kv_compact(const w4v_pages_t *pages, int32_t *refs_out, int32_t *table_out, void *ws, size_t ws_bytes,
                      w4v_stream_t stream) {
    w4v_status st = pages_check(pages, true);
    if (st != W4V_OK || pages->S == 0) return st;
    if (refs_out == nullptr || table_out == nullptr) return W4V_ERR_ARG;
    if (!aligned4(refs_out) || !aligned4(table_out)) return W4V_ERR_ALIGN;
    st = pages_ws_check(pages, ws, ws_bytes);
    if (st != W4V_OK) return st;
    return w4v::launch_kv_compact(*pages, refs_out, table_out, ws, reinterpret_cast<cudaStream_t>(stream));
}

w4v_status kv_copy(void *pool, int planes, int n_pages, size_t page_bytes, const int32_t *src, const int32_t *dst,
                   int n, w4v_stream_t stream) {
    if (planes < 1 || n_pages < 1 || n_pages > 1 << 24 || page_bytes == 0 || page_bytes % 16 != 0 ||
        page_bytes >= size_t(1) << 31 || n < 0)
        return W4V_ERR_SHAPE;
    if (n == 0) return W4V_OK;
    if (pool == nullptr || src == nullptr || dst == nullptr) return W4V_ERR_ARG;
    if (!w4v::aligned16(pool) || !aligned4(src) || !aligned4(dst)) return W4V_ERR_ALIGN;
    return w4v::launch_kv_copy(pool, planes, n_pages, page_bytes, src, dst, n,
                               reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
