// Eviction from a KV cache by accumulated attention weight: the choice of the keys that
// stay, and the move of their rows to a smaller cache.
#include <cooperative_groups.h>

#include "serve.h"

namespace cg = cooperative_groups;

namespace spa {
namespace {

// ------------------------------------------------------------------ the choice
// The n-th largest score of each (b, kv-head) by radix selection: four rounds, each
// fixing the next 8 bits of the threshold's order-preserving 32-bit key from a histogram
// of the keys that agree with it so far. A cluster of CTAs owns one (b, kv-head);
// each holds a slice of the keys in shared memory (read from HBM once), and the
// histograms of a round are added over the cluster through distributed shared memory
// (two in turn, so a round needs one cluster barrier). The kept set is then written in
// ascending order from the counts of the CTAs and warps before.
constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kSliceMax = 48 * 1024;      // keys of a slice held in shared memory

// Unsigned order of the floats; NaN below all, -0 and +0 equal.
__device__ __forceinline__ uint32_t order_key(float f) {
    if (f != f) return 0u;
    const uint32_t b = __float_as_uint(f + 0.f);   // -0 + 0 = +0
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

struct EvictArgs {
    const float *score;
    const int32_t *lens;
    int Hkv, T, n_keep, n_sink, n_recent, slice, cached;
    int32_t *keep, *count;
    int *err;
};

__global__ void __launch_bounds__(kThreads) evict_select_kernel(EvictArgs a) {
    extern __shared__ uint32_t keys_s[];           // [slice] when it is held
    __shared__ int hist[2][256];
    __shared__ int wgt[kWarps], weq[kWarps];
    __shared__ int mine[2];                        // this CTA's keys above and at the threshold
    __shared__ uint32_t sh_digit;
    __shared__ int sh_left;
    cg::cluster_group cl = cg::this_cluster();
    const int C = (int)cl.num_blocks(), rank = (int)cl.block_rank();
    const int bg = blockIdx.x / C, b = bg / a.Hkv;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    int len = a.lens ? a.lens[b] : a.T;
    if (len < 0 || len > a.T) {
        if (tid == 0) set_error(a.err, SPA_DEVERR_BAD_COUNT);
        len = len < 0 ? 0 : a.T;
    }
    const int total = min(len, a.n_keep);
    int32_t *keep = a.keep + (size_t)bg * a.n_keep;
    if (rank == 0 && tid == 0 && bg % a.Hkv == 0) a.count[b] = total;
    const int gtid = rank * kThreads + tid, gthreads = C * kThreads;
    if (len <= a.n_keep) {                         // uniform over the cluster
        for (int i = gtid; i < a.n_keep; i += gthreads) keep[i] = i < len ? i : -1;
        return;
    }
    // here len > n_keep >= n_sink + n_recent
    const int c_lo = a.n_sink, c_hi = len - a.n_recent;   // the candidates
    const int need = a.n_keep - a.n_sink - a.n_recent;
    for (int i = gtid; i < a.n_sink; i += gthreads) keep[i] = i;
    for (int i = gtid; i < a.n_recent; i += gthreads) keep[a.n_keep - a.n_recent + i] = c_hi + i;

    const int n = c_hi - c_lo;
    const int per = ((n + C - 1) / C + 31) & ~31;  // keys per CTA, <= slice
    const int lo = min(n, rank * per), cnt = min(n, lo + per) - lo;
    const float *src = a.score + (size_t)bg * a.T + c_lo + lo;
    if (a.cached)
        for (int i = tid; i < cnt; i += kThreads) keys_s[i] = order_key(src[i]);
    auto key_at = [&](int i) -> uint32_t { return a.cached ? keys_s[i] : order_key(src[i]); };

    uint32_t prefix = 0;
    int left = need, gt_mine = 0;
    for (int round = 0; round < 4; ++round) {
        const int sh = 24 - 8 * round;
        int *hs = hist[round & 1];
        for (int i = tid; i < 256; i += kThreads) hs[i] = 0;
        __syncthreads();
        for (int i0 = 0; i0 < cnt; i0 += kThreads) {
            const int i = i0 + tid;
            const uint32_t k = i < cnt ? key_at(i) : 0u;
            const bool in = i < cnt && (round == 0 || (k >> (sh + 8)) == prefix);
            const unsigned act = __ballot_sync(0xffffffffu, in);
            if (in) {                               // equal digits of a warp count once
                const uint32_t dg = (k >> sh) & 255u;
                const unsigned same = __match_any_sync(act, dg);
                if (lane == __ffs(same) - 1) atomicAdd(&hs[dg], __popc(same));
            }
        }
        cl.sync();
        if (tid < 256) {
            int sum = 0;
            for (int r = 0; r < C; ++r) sum += cl.map_shared_rank(hs, r)[tid];
            // digit: the largest d with (keys of digits >= d) >= left
            int suf = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_down_sync(0xffffffffu, suf, o);
                if (lane + o < 32) suf += y;
            }
            if (lane == 0) weq[warp] = suf;
            asm volatile("bar.sync 1, 256;" ::: "memory");
            int above = 0;
            for (int w = warp + 1; w < 8; ++w) above += weq[w];
            const int incl = suf + above, excl = incl - sum;
            if (left > 0 ? (incl >= left && excl < left) : tid == 255) {
                sh_digit = (uint32_t)tid;
                sh_left = left - excl;
            }
        }
        __syncthreads();
        const uint32_t dg = sh_digit;
        if (warp == 0) {                            // this CTA's keys above the digit
            int g = 0;
            for (int i = lane; i < 256; i += 32) g += i > (int)dg ? hs[i] : 0;
#pragma unroll
            for (int o = 16; o; o >>= 1) g += __shfl_xor_sync(0xffffffffu, g, o);
            gt_mine += g;
            if (round == 3 && lane == 0) {
                mine[0] = gt_mine;
                mine[1] = hs[dg];
            }
        }
        left = sh_left;
        prefix = (prefix << 8) | dg;
    }
    // need == 0: the threshold is above every key's digit path; take nothing
    cl.sync();
    int gt_before = 0, eq_before = 0;
    for (int r = 0; r < rank; ++r) {
        gt_before += cl.map_shared_rank(mine, r)[0];
        eq_before += cl.map_shared_rank(mine, r)[1];
    }
    const uint32_t thr = prefix;
    const int need_eq = left;
    if (need > 0) {
        // each warp owns a run of 32-key steps; counts first, then the ordered write
        const int steps = (cnt + 31) / 32, wsteps = (steps + kWarps - 1) / kWarps;
        const int s_lo = min(steps, warp * wsteps), s_hi = min(steps, s_lo + wsteps);
        int g = 0, q = 0;
        for (int st = s_lo; st < s_hi; ++st) {
            const int i = st * 32 + lane;
            const uint32_t k = i < cnt ? key_at(i) : 0u;
            g += __popc(__ballot_sync(0xffffffffu, i < cnt && k > thr));
            q += __popc(__ballot_sync(0xffffffffu, i < cnt && k == thr));
        }
        if (lane == 0) {
            wgt[warp] = g;
            weq[warp] = q;
        }
        __syncthreads();
        for (int w = 0; w < warp; ++w) {
            gt_before += wgt[w];
            eq_before += weq[w];
        }
        for (int st = s_lo; st < s_hi; ++st) {
            const int i = st * 32 + lane;
            const uint32_t k = i < cnt ? key_at(i) : 0u;
            const bool is_g = i < cnt && k > thr, is_q = i < cnt && k == thr;
            const unsigned bg_ = __ballot_sync(0xffffffffu, is_g), bq = __ballot_sync(0xffffffffu, is_q);
            const unsigned below = (1u << lane) - 1u;
            const int gb = gt_before + __popc(bg_ & below), qb = eq_before + __popc(bq & below);
            if (is_g || (is_q && qb < need_eq)) keep[a.n_sink + gb + min(qb, need_eq)] = c_lo + lo + i;
            gt_before += __popc(bg_);
            eq_before += __popc(bq);
        }
    }
    cl.sync();                                      // mine[] is read by the others until here
}

// ------------------------------------------------------------------ the move
// One thread per 16 bytes of a kept row, K and V together; reads follow the list,
// writes are contiguous. Bound by HBM.
struct GatherArgs {
    const uint4 *k, *v;
    const float *score;
    const int32_t *keep, *count;
    int Hkv, T, T_out, n_keep, nv;       // nv: 16-byte vectors per row
    long long total;                     // B * Hkv * n_keep * nv
    uint4 *ko, *vo;
    float *so;
    int *err;
};

__global__ void __launch_bounds__(256) gather_kernel(GatherArgs a) {
    const long long id = (long long)blockIdx.x * 256 + threadIdx.x;
    if (id >= a.total) return;
    const long long row = id / a.nv;
    const int c = (int)(id - row * a.nv);
    const long long bg = row / a.n_keep;
    const int i = (int)(row - bg * a.n_keep);
    if (a.count) {
        const int cn = a.count[bg / a.Hkv];
        if ((cn < 0 || cn > a.n_keep) && i == 0 && c == 0) set_error(a.err, SPA_DEVERR_BAD_COUNT);
        if (i >= cn) return;
    }
    const int t = __ldg(a.keep + row);
    if (t < 0 || t >= a.T) {
        if (c == 0) set_error(a.err, SPA_DEVERR_BAD_INDEX);
        return;
    }
    const long long s = (bg * a.T + t) * a.nv + c, o = (bg * a.T_out + i) * a.nv + c;
    const uint4 x = __ldg(a.k + s), y = __ldg(a.v + s);
    a.ko[o] = x;
    a.vo[o] = y;
    if (a.so && c == 0) a.so[bg * a.T_out + i] = __ldg(a.score + bg * a.T + t);
}

}  // namespace

cudaError_t launch_evict_select(const float *score, const int32_t *lens, int B, int Hkv, int T,
                                int n_keep, int n_sink, int n_recent, int32_t *keep,
                                int32_t *count, int *err, cudaStream_t s) {
    EvictArgs a{score, lens, Hkv, T, n_keep, n_sink, n_recent, 0, 0, keep, count, err};
    // CTAs per (b, kv-head): one per 4096 keys (4 rounds over 4 keys a thread), at most 8
    int C = 1;
    while (C < kMaxCluster && (long long)C * 4096 < T) C *= 2;
    const int per = ((T + C - 1) / C + 31) & ~31;
    a.cached = per <= kSliceMax;
    a.slice = per;
    const size_t smem = a.cached ? (size_t)per * 4 : 0;
    cudaError_t e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((size_t)B * Hkv * C));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)C;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, evict_select_kernel, a);
}

cudaError_t launch_cache_gather(const void *kc, const void *vc, const float *score, int B, int Hkv,
                                int T, int row_bytes, const int32_t *keep, int n_keep,
                                const int32_t *count, int T_out, void *k_out, void *v_out,
                                float *score_out, int *err, cudaStream_t s) {
    GatherArgs a;
    a.k = static_cast<const uint4 *>(kc);
    a.v = static_cast<const uint4 *>(vc);
    a.score = score;
    a.keep = keep;
    a.count = count;
    a.Hkv = Hkv; a.T = T; a.T_out = T_out; a.n_keep = n_keep;
    a.nv = row_bytes / 16;
    a.total = (long long)B * Hkv * n_keep * a.nv;
    a.ko = static_cast<uint4 *>(k_out);
    a.vo = static_cast<uint4 *>(v_out);
    a.so = score_out;
    a.err = err;
    gather_kernel<<<(unsigned)((a.total + 255) / 256), 256, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace spa
