// C-ABI entry points of the serving operators (declared in include/spa.h): rotary
// positions, tree attention, accumulated attention weight, eviction. Host-side
// argument validation and dispatch to the launchers of serve.h.
#include <math.h>
#include <stdio.h>

#include "serve.h"

#define SPA_API extern "C" __attribute__((visibility("default")))

namespace spa {
namespace {

spa_status fail(spa_status st, const char *msg) {
    record_last_error(msg);
    return st;
}

spa_status launched(cudaError_t e, const char *what) {
    if (e == cudaSuccess) return SPA_OK;
    if (e == cudaErrorNotSupported) return fail(SPA_ERR_UNSUPPORTED, "tensor map encoding unavailable");
    char msg[256];
    snprintf(msg, sizeof msg, "%s: %s", what, cudaGetErrorString(e));
    return fail(SPA_ERR_CUDA, msg);
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

spa_strides strides_or_dense(const spa_strides *s, int H, int L, int d) {
    if (s) return *s;
    return spa_strides{(int64_t)H * L * d, (int64_t)L * d, d};
}

// Whether [a, a + na) and [b, b + nb) share a byte.
bool overlap(const void *a, size_t na, const void *b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

// Whether the rows of an output are each its own (no broadcast stride).
bool own_rows(const spa_strides &s, int B, int H, int L) {
    return (B == 1 || s.b) && (H == 1 || s.h) && (L == 1 || s.l);
}

bool block_ok(int block) { return block == 16 || block == 32 || block == 64 || block == 128; }

spa_status check_rope(const RopeCall &c, spa_dtype dt, int Hq, int Hkv, spa_rope_layout layout) {
    if (!c.t[0].x || !c.t[0].y || !c.freqs) return fail(SPA_ERR_INVALID, "null pointer");
    if (c.B <= 0 || Hq <= 0 || c.L <= 0 || c.d <= 0 || (c.t[1].x && Hkv <= 0))
        return fail(SPA_ERR_INVALID, "sizes must be positive");
    if (dt != SPA_F32 && dt != SPA_BF16) return fail(SPA_ERR_INVALID, "unknown dtype");
    if (layout != SPA_ROPE_HALF && layout != SPA_ROPE_INTERLEAVED)
        return fail(SPA_ERR_INVALID, "unknown rotary layout");
    if (c.rot < 2 || c.rot % 2 || c.rot > c.d)
        return fail(SPA_ERR_INVALID, "rot must be even, at least 2 and at most d");
    if (!isfinite(c.mscale)) return fail(SPA_ERR_INVALID, "mscale must be finite");
    for (int i = 0; i < c.rot / 2 && i < kRopeMaxPairs; ++i)
        if (!isfinite(c.freqs[i])) return fail(SPA_ERR_INVALID, "freqs must be finite");
    if ((long long)c.pos0 + c.L - 1 > 0x7fffffffll)
        return fail(SPA_ERR_INVALID, "positions must fit 32 bits");
    const uintptr_t mask = dt == SPA_BF16 ? 1 : 3;
    for (const RopeTensor &t : c.t)
        if ((reinterpret_cast<uintptr_t>(t.x) | reinterpret_cast<uintptr_t>(t.y)) & mask)
            return fail(SPA_ERR_INVALID, "tensors must be aligned to their elements");
    if (c.d > 2 * kRopeMaxPairs) return fail(SPA_ERR_UNSUPPORTED, "d must be at most 256");
    if ((long long)Hq + 2ll * Hkv > 65535) return fail(SPA_ERR_UNSUPPORTED, "too many heads");
    if ((long long)c.B * c.L > (1ll << 30)) return fail(SPA_ERR_UNSUPPORTED, "too many tokens");
    return SPA_OK;
}

}  // namespace
}  // namespace spa

using namespace spa;

SPA_API spa_status spa_rope_frequencies(int rot, double base, spa_rope_scaling scaling,
                                        double factor, double trained, double fast, double slow,
                                        double *freqs, float *mscale) {
    record_last_error("");
    if (!freqs || !mscale) return fail(SPA_ERR_INVALID, "null pointer");
    if (rot < 2 || rot % 2 || rot > 2 * kRopeMaxPairs)
        return fail(SPA_ERR_INVALID, "rot must be even and in [2, 256]");
    if (!(base > 1.0) || !isfinite(base)) return fail(SPA_ERR_INVALID, "base must be > 1");
    if (scaling < SPA_ROPE_NONE || scaling > SPA_ROPE_PARTS)
        return fail(SPA_ERR_INVALID, "unknown scaling");
    if (scaling != SPA_ROPE_NONE && (!(factor >= 1.0) || !isfinite(factor)))
        return fail(SPA_ERR_INVALID, "factor must be >= 1");
    if (scaling == SPA_ROPE_NTK && rot < 4) return fail(SPA_ERR_INVALID, "this scaling needs rot >= 4");
    if (scaling == SPA_ROPE_PARTS &&
        (!(trained > 0.0) || !isfinite(trained) || !(slow > 0.0) || !(fast > slow) || !isfinite(fast)))
        return fail(SPA_ERR_INVALID, "need trained > 0 and fast > slow > 0");
    const int n = rot / 2;
    if (scaling == SPA_ROPE_NTK) base *= pow(factor, (double)rot / (rot - 2));
    *mscale = 1.f;
    double lo = 0.0, hi = 0.0;
    if (scaling == SPA_ROPE_PARTS) {
        // the pair that turns `r` times over the trained length: trained * f_c = 2 pi r
        constexpr double kTwoPi = 6.283185307179586476925286766559;
        const auto pair_at = [&](double r) { return rot * log(trained / (r * kTwoPi)) / (2.0 * log(base)); };
        lo = fmax(floor(pair_at(fast)), 0.0);
        hi = fmin(ceil(pair_at(slow)), (double)rot - 1.0);
        *mscale = (float)(0.1 * log(factor) + 1.0);
    }
    for (int c = 0; c < n; ++c) {
        double f = pow(base, -2.0 * c / rot);
        if (scaling == SPA_ROPE_LINEAR) f /= factor;
        if (scaling == SPA_ROPE_PARTS) {
            const double ramp = fmin(fmax((c - lo) / fmax(hi - lo, 0.001), 0.0), 1.0);
            f = f * (1.0 - ramp) + f / factor * ramp;
        }
        freqs[c] = f;
    }
    return SPA_OK;
}

SPA_API spa_status spa_rope(const void *q, const spa_strides *q_str, void *q_out,
                            const spa_strides *qo_str, const void *k, const spa_strides *k_str,
                            void *k_out, const spa_strides *ko_str, spa_dtype dt, int B, int Hq,
                            int Hkv, int L, int d, int rot, spa_rope_layout layout,
                            const double *freqs, float mscale, const int32_t *pos, int pos0,
                            int backward, spa_stream stream) {
    record_last_error("");
    if (!k != !k_out) return fail(SPA_ERR_INVALID, "k and k_out go together");
    if (backward != 0 && backward != 1) return fail(SPA_ERR_INVALID, "backward must be 0 or 1");
    RopeCall c;
    c.t[0] = {q, q_out, strides_or_dense(q_str, Hq, L, d), strides_or_dense(qo_str, Hq, L, d), Hq};
    if (k) c.t[1] = {k, k_out, strides_or_dense(k_str, Hkv, L, d), strides_or_dense(ko_str, Hkv, L, d), Hkv};
    c.bf16 = dt == SPA_BF16;
    c.B = B; c.L = L; c.d = d; c.rot = rot;
    c.interleaved = layout == SPA_ROPE_INTERLEAVED;
    c.backward = backward != 0;
    c.freqs = freqs;
    c.mscale = mscale;
    c.pos = pos;
    c.pos0 = pos0;
    const spa_status st = check_rope(c, dt, Hq, k ? Hkv : 0, layout);
    if (st != SPA_OK) return st;
    if (q_out == k_out || !own_rows(c.t[0].ys, B, Hq, L) || (k && !own_rows(c.t[1].ys, B, Hkv, L)))
        return fail(SPA_ERR_INVALID, "the rows of the outputs must not overlap");
    return launched(launch_rope(c, static_cast<cudaStream_t>(stream)), "rope launch");
}

SPA_API spa_status spa_rope_append(const void *q, const spa_strides *q_str, void *q_out,
                                   const spa_strides *qo_str, const void *k,
                                   const spa_strides *k_str, const void *v,
                                   const spa_strides *v_str, void *kc, void *vc, spa_dtype dt,
                                   int B, int Hq, int Hkv, int L, int T, int d, int rot,
                                   spa_rope_layout layout, const double *freqs, float mscale,
                                   const int32_t *pos, const int32_t *rows, int row0,
                                   spa_stream stream) {
    record_last_error("");
    if (!k || !v || !kc || !vc) return fail(SPA_ERR_INVALID, "null pointer");
    if (T <= 0) return fail(SPA_ERR_INVALID, "sizes must be positive");
    if (!rows && (row0 < 0 || (long long)row0 + L > T))
        return fail(SPA_ERR_INVALID, "rows [row0, row0 + L) must lie in [0, T)");
    RopeCall c;
    const spa_strides cache = strides_or_dense(nullptr, Hkv, T, d);
    c.t[0] = {q, q_out, strides_or_dense(q_str, Hq, L, d), strides_or_dense(qo_str, Hq, L, d), Hq};
    c.t[1] = {k, kc, strides_or_dense(k_str, Hkv, L, d), cache, Hkv};
    c.t[2] = {v, vc, strides_or_dense(v_str, Hkv, L, d), cache, Hkv};
    c.bf16 = dt == SPA_BF16;
    c.B = B; c.L = L; c.d = d; c.rot = rot;
    c.interleaved = layout == SPA_ROPE_INTERLEAVED;
    c.append = true;
    c.T = T;
    c.freqs = freqs;
    c.mscale = mscale;
    c.pos = pos;
    c.rows = rows;
    c.pos0 = rows ? 0 : row0;
    const spa_status st = check_rope(c, dt, Hq, Hkv, layout);
    if (st != SPA_OK) return st;
    const size_t cache_bytes = (size_t)B * Hkv * T * d * (c.bf16 ? 2 : 4);
    if (overlap(kc, cache_bytes, vc, cache_bytes) || !own_rows(c.t[0].ys, B, Hq, L))
        return fail(SPA_ERR_INVALID, "the rows of the outputs must not overlap");
    c.err = device_error_word();
    if (!c.err) return fail(SPA_ERR_CUDA, "device error word unavailable");
    return launched(launch_rope(c, static_cast<cudaStream_t>(stream)), "rope launch");
}

SPA_API size_t spa_tree_workspace_bytes(int B, int Hq, int Hkv, int n, int T, int d, int block) {
    if (B <= 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv || n < 1 || n > 128 || T < n ||
        (d != 64 && d != 128) || !block_ok(block) || Hq / Hkv > 16)
        return 0;
    return tree_workspace_bytes(B, Hq, Hkv, n, T, d, block);
}

SPA_API spa_status spa_sparse_attn_tree(const void *q, const void *kc, const void *vc, spa_dtype dt,
                                        int B, int Hq, int Hkv, int n, int T, int d, int block,
                                        const int32_t *parents, const int32_t *lens,
                                        const int32_t *idx, int cap, const int32_t *count,
                                        float scale, void *workspace, size_t workspace_bytes,
                                        void *out, float *lse, spa_stream stream) {
    record_last_error("");
    if (!q || !kc || !vc || !parents || !workspace || !out) return fail(SPA_ERR_INVALID, "null pointer");
    if (!idx != !count) return fail(SPA_ERR_INVALID, "idx and count go together");
    if (B <= 0 || Hq <= 0 || Hkv <= 0 || n <= 0 || T <= 0 || d <= 0 || block <= 0)
        return fail(SPA_ERR_INVALID, "sizes must be positive");
    if (Hq % Hkv) return fail(SPA_ERR_INVALID, "Hq must be a multiple of Hkv");
    if (T < n) return fail(SPA_ERR_INVALID, "the cache holds the n nodes: T must be >= n");
    if (!(scale > 0.f) || !isfinite(scale)) return fail(SPA_ERR_INVALID, "scale must be > 0");
    if (idx && cap < (T + block - 1) / block) return fail(SPA_ERR_INVALID, "cap must be >= nb");
    if (!aligned16(q) || !aligned16(kc) || !aligned16(vc) || !aligned16(out) || !aligned16(workspace))
        return fail(SPA_ERR_INVALID, "tensors must be 16-byte aligned");
    if (dt != SPA_BF16) return fail(SPA_ERR_UNSUPPORTED, "tree attention is bf16 only");
    if (d != 64 && d != 128) return fail(SPA_ERR_UNSUPPORTED, "d must be 64 or 128");
    if (!block_ok(block)) return fail(SPA_ERR_UNSUPPORTED, "block must be 16, 32, 64 or 128");
    if (n > 128) return fail(SPA_ERR_UNSUPPORTED, "at most 128 nodes");
    if (Hq / Hkv > 16) return fail(SPA_ERR_UNSUPPORTED, "at most 16 query heads per kv-head");
    if ((long long)B * Hkv * T > 0x7fffffffll || (long long)B * Hq * n > 0x7fffffffll || B * (long long)Hkv > 65535)
        return fail(SPA_ERR_UNSUPPORTED, "too many rows");
    if (workspace_bytes < tree_workspace_bytes(B, Hq, Hkv, n, T, d, block))
        return fail(SPA_ERR_INVALID, "workspace smaller than spa_tree_workspace_bytes");
    int *err = device_error_word();
    if (!err) return fail(SPA_ERR_CUDA, "device error word unavailable");
    const TreeCall c{q, kc, vc, B, Hq, Hkv, n, T, d, block, cap, parents, lens, idx, count,
                     scale, workspace, out, lse, err};
    return launched(launch_tree(c, static_cast<cudaStream_t>(stream)), "tree attention launch");
}

SPA_API size_t spa_attn_weight_workspace_bytes(int B, int Hkv, int Lq, int T, int block) {
    if (B <= 0 || Hkv <= 0 || Lq <= 0 || T < Lq || (block != 0 && !block_ok(block))) return 0;
    return weight_workspace_bytes(B, Hkv, Lq, T, block);
}

SPA_API spa_status spa_attn_weight(const void *q, const void *k, spa_dtype dt, int B, int Hq,
                                   int Hkv, int Lq, int T, int d, const float *lse,
                                   const int32_t *lens, int block, const int32_t *idx, int cap,
                                   const int32_t *count, float scale, const float *prev,
                                   float decay, void *workspace, size_t workspace_bytes,
                                   float *out, spa_stream stream) {
    record_last_error("");
    if (!q || !k || !lse || !workspace || !out) return fail(SPA_ERR_INVALID, "null pointer");
    if (!idx != !count) return fail(SPA_ERR_INVALID, "idx and count go together");
    if (B <= 0 || Hq <= 0 || Hkv <= 0 || Lq <= 0 || T <= 0 || d <= 0)
        return fail(SPA_ERR_INVALID, "sizes must be positive");
    if (Hq % Hkv) return fail(SPA_ERR_INVALID, "Hq must be a multiple of Hkv");
    if (Lq > T) return fail(SPA_ERR_INVALID, "the queries are the sequence's last: Lq must be <= T");
    if (!(scale > 0.f) || !isfinite(scale)) return fail(SPA_ERR_INVALID, "scale must be > 0");
    if (!isfinite(decay)) return fail(SPA_ERR_INVALID, "decay must be finite");
    if (!aligned16(q) || !aligned16(k) || !aligned16(workspace))
        return fail(SPA_ERR_INVALID, "q, k and the workspace must be 16-byte aligned");
    if (!aligned4(lse) || !aligned4(prev) || !aligned4(out))
        return fail(SPA_ERR_INVALID, "tensors must be aligned to their elements");
    if (dt != SPA_BF16) return fail(SPA_ERR_UNSUPPORTED, "the accumulated weight is bf16 only");
    if (d != 64 && d != 128) return fail(SPA_ERR_UNSUPPORTED, "d must be 64 or 128");
    if (Hq / Hkv > 16) return fail(SPA_ERR_UNSUPPORTED, "at most 16 query heads per kv-head");
    if ((long long)B * Hkv * T > 0x7fffffffll || (long long)B * Hq * Lq > 0x7fffffffll || B * (long long)Hkv > 65535)
        return fail(SPA_ERR_UNSUPPORTED, "too many rows");
    // (128-key tile, query tile of at least 16 positions) pairs per CTA: a 32-bit count
    if (((long long)B * Hkv * T / 128 + 1) * (Lq / 16ll + 1) / 148 > 0x7fffffffll)
        return fail(SPA_ERR_UNSUPPORTED, "too many queries and keys");
    if (idx) {
        if (block <= 0) return fail(SPA_ERR_INVALID, "sizes must be positive");
        if (!block_ok(block)) return fail(SPA_ERR_UNSUPPORTED, "block must be 16, 32, 64 or 128");
        if (cap < (T + block - 1) / block) return fail(SPA_ERR_INVALID, "cap must be >= nb");
        if (T / block > kMaxMarkBlocks) return fail(SPA_ERR_UNSUPPORTED, "too many blocks");
        if (lens && Lq != 1) return fail(SPA_ERR_INVALID, "lists of several queries need lens = NULL");
    }
    if (workspace_bytes < weight_workspace_bytes(B, Hkv, Lq, T, idx ? block : 0))
        return fail(SPA_ERR_INVALID, "workspace smaller than spa_attn_weight_workspace_bytes");
    const size_t out_bytes = (size_t)B * Hkv * T * sizeof(float);
    if (prev && prev != out && overlap(prev, out_bytes, out, out_bytes))
        return fail(SPA_ERR_INVALID, "out may be prev, but not overlap it otherwise");
    int *err = device_error_word();
    if (!err) return fail(SPA_ERR_CUDA, "device error word unavailable");
    const WeightCall c{q, k, B, Hq, Hkv, Lq, T, d, idx ? block : 128, cap, lse, lens, idx, count,
                       scale, decay, prev, workspace, out, err};
    return launched(launch_weight(c, static_cast<cudaStream_t>(stream)), "attention weight launch");
}

SPA_API spa_status spa_evict_select(const float *score, const int32_t *lens, int B, int Hkv, int T,
                                    int n_keep, int n_sink, int n_recent, int32_t *keep,
                                    int32_t *count, spa_stream stream) {
    record_last_error("");
    if (!score || !keep || !count) return fail(SPA_ERR_INVALID, "null pointer");
    if (B <= 0 || Hkv <= 0 || T <= 0 || n_keep <= 0)
        return fail(SPA_ERR_INVALID, "sizes must be positive");
    if (n_sink < 0 || n_recent < 0 || (long long)n_sink + n_recent > n_keep)
        return fail(SPA_ERR_INVALID, "need n_sink, n_recent >= 0 and n_sink + n_recent <= n_keep");
    if ((long long)B * Hkv > (1 << 27)) return fail(SPA_ERR_UNSUPPORTED, "too many heads");
    if (T > 0x7fffffff - 63) return fail(SPA_ERR_UNSUPPORTED, "too many keys");   // T is rounded up in 32 bits
    int *err = device_error_word();
    if (!err) return fail(SPA_ERR_CUDA, "device error word unavailable");
    return launched(launch_evict_select(score, lens, B, Hkv, T, n_keep, n_sink, n_recent, keep, count,
                                        err, static_cast<cudaStream_t>(stream)),
                    "eviction launch");
}

SPA_API spa_status spa_cache_gather(const void *kc, const void *vc, const float *score,
                                    spa_dtype dt, int B, int Hkv, int T, int d,
                                    const int32_t *keep, int n_keep, const int32_t *count,
                                    int T_out, void *k_out, void *v_out, float *score_out,
                                    spa_stream stream) {
    record_last_error("");
    if (!kc || !vc || !keep || !k_out || !v_out) return fail(SPA_ERR_INVALID, "null pointer");
    if (!score != !score_out) return fail(SPA_ERR_INVALID, "score and score_out go together");
    if (B <= 0 || Hkv <= 0 || T <= 0 || d <= 0 || n_keep <= 0)
        return fail(SPA_ERR_INVALID, "sizes must be positive");
    if (T_out < n_keep) return fail(SPA_ERR_INVALID, "T_out must be >= n_keep");
    if (dt != SPA_F32 && dt != SPA_BF16) return fail(SPA_ERR_INVALID, "unknown dtype");
    if (!aligned16(kc) || !aligned16(vc) || !aligned16(k_out) || !aligned16(v_out))
        return fail(SPA_ERR_INVALID, "tensors must be 16-byte aligned");
    const int row_bytes = d * (dt == SPA_BF16 ? 2 : 4);
    if (row_bytes % 16) return fail(SPA_ERR_UNSUPPORTED, "rows must be a multiple of 16 bytes");
    if ((long long)B * Hkv * n_keep * (row_bytes / 16) > (1ll << 39))
        return fail(SPA_ERR_UNSUPPORTED, "too many rows");
    const size_t rows_in = (size_t)B * Hkv * T, rows_out = (size_t)B * Hkv * T_out;
    const size_t in = rows_in * row_bytes, out = rows_out * row_bytes;
    if (overlap(kc, in, k_out, out) || overlap(kc, in, v_out, out) || overlap(vc, in, k_out, out) ||
        overlap(vc, in, v_out, out) || (overlap(k_out, out, v_out, out) && (kc != vc || k_out != v_out)) ||
        (score && overlap(score, rows_in * sizeof(float), score_out, rows_out * sizeof(float))))
        return fail(SPA_ERR_INVALID, "the smaller cache must not overlap the cache, nor its parts one another");
    int *err = device_error_word();
    if (!err) return fail(SPA_ERR_CUDA, "device error word unavailable");
    return launched(launch_cache_gather(kc, vc, score, B, Hkv, T, row_bytes, keep, n_keep, count, T_out,
                                        k_out, v_out, score_out, err, static_cast<cudaStream_t>(stream)),
                    "gather launch");
}
