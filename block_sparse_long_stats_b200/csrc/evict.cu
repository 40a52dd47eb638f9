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
// by one warp (two histograms in turn, so a round needs one cluster barrier). The kept
// set is then written in ascending order from the counts of the CTAs and warps before.
// Bound by the rounds' latencies: 17 us for eight heads of 32K keys, 10 for 128 of up to 4000.
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
    int Hkv, T, n_keep, n_sink, n_recent, cached;
    int32_t *keep, *count;
    int *err;
};

__global__ void __launch_bounds__(kThreads) evict_select_kernel(EvictArgs a) {
    extern __shared__ __align__(16) uint32_t keys_s[];   // the slice, when it is held
    __shared__ __align__(16) int hist[2][256];
    __shared__ int wgt[kWarps], weq[kWarps];
    __shared__ int mine[2];                        // this CTA's keys above and at the threshold
    __shared__ uint32_t sh_digit;
    __shared__ int sh_left;
    cg::cluster_group cl = cg::this_cluster();
    const int C = (int)cl.num_blocks(), rank = (int)cl.block_rank();
    const int bg = blockIdx.x / C, b = bg / a.Hkv;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid < 512) hist[tid >> 8][tid & 255] = 0;
    grid_wait();

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
    const int per = ((n + C - 1) / C + 31) & ~31;  // keys per CTA
    const int lo = min(n, rank * per), cnt = min(n, lo + per) - lo;
    const float *src = a.score + (size_t)bg * a.T + c_lo + lo;
    // keys i0 + 4 lane .. + 3 (anything from cnt on); returns the first one's number
    auto quad = [&](int i0, uint32_t (&k)[4]) -> int {
        const int i = i0 + 4 * lane;
        if (a.cached) {
            *reinterpret_cast<uint4 *>(k) = *reinterpret_cast<const uint4 *>(keys_s + i);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) k[e] = i + e < cnt ? order_key(__ldg(src + i + e)) : 0u;
        }
        return i;
    };
    // one more key with digit dg: those that share the first lane's count once (scores that
    // are all alike), the others each (a match over the whole warp took most of the time)
    auto add = [&](int *hs, bool in, uint32_t dg) {
        const unsigned act = __ballot_sync(0xffffffffu, in);
        if (!act) return;
        const int lead = __ffs(act) - 1;
        const uint32_t d0 = __shfl_sync(0xffffffffu, dg, lead);
        const unsigned same = __ballot_sync(0xffffffffu, in && dg == d0);
        if (lane == lead) atomicAdd(&hs[d0], __popc(same));
        else if (in && dg != d0) atomicAdd(&hs[dg], 1);
    };
    __syncthreads();                               // the histograms are zero

    uint32_t prefix = 0;
    int left = need, gt_mine = 0;
    for (int round = 0; round < 4; ++round) {
        const int sh = 24 - 8 * round;
        int *hs = hist[round & 1];
        if (round == 0) {                          // the keys come in with their first digit counted
            constexpr int kAhead = 16;             // loads in flight per thread
            for (int i0 = tid; i0 - tid < cnt; i0 += kAhead * kThreads) {
                float f[kAhead];
#pragma unroll
                for (int j = 0; j < kAhead; ++j) f[j] = i0 + j * kThreads < cnt ? __ldg(src + i0 + j * kThreads) : 0.f;
#pragma unroll
                for (int j = 0; j < kAhead; ++j) {
                    const int i = i0 + j * kThreads;
                    if (i - tid >= cnt) break;     // uniform
                    const uint32_t k = order_key(f[j]);
                    if (a.cached && i < cnt) keys_s[i] = k;
                    add(hs, i < cnt, k >> 24);
                }
            }
        } else {                                   // few keys agree with the threshold so far
            for (int i0 = warp * 128; i0 < cnt; i0 += kWarps * 128) {
                uint32_t k[4];
                const int i = quad(i0, k);
                bool in[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) in[e] = i + e < cnt && (k[e] >> (sh + 8)) == prefix;
                if (__any_sync(0xffffffffu, in[0] || in[1] || in[2] || in[3])) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) add(hs, in[e], (k[e] >> sh) & 255u);
                }
            }
        }
        if (C > 1) cl.sync(); else __syncthreads();
        if (warp == 0) {
            // lane: digits 8 lane .. 8 lane + 7, over the cluster and of this CTA
            int sum[8], own[8];
            *reinterpret_cast<int4 *>(own) = *reinterpret_cast<const int4 *>(hs + 8 * lane);
            *reinterpret_cast<int4 *>(own + 4) = *reinterpret_cast<const int4 *>(hs + 8 * lane + 4);
#pragma unroll
            for (int e = 0; e < 8; ++e) sum[e] = own[e];
            // (in fours: every load of a group on its way before the first is used)
            for (int r0 = 1; r0 < C; r0 += 4) {
                int4 x[4], y[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int4 *o = reinterpret_cast<const int4 *>(
                        cl.map_shared_rank(hs, r0 + j < C ? (rank + r0 + j) % C : rank) + 8 * lane);
                    x[j] = o[0];
                    y[j] = o[1];
                }
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (r0 + j < C) {
                        sum[0] += x[j].x; sum[1] += x[j].y; sum[2] += x[j].z; sum[3] += x[j].w;
                        sum[4] += y[j].x; sum[5] += y[j].y; sum[6] += y[j].z; sum[7] += y[j].w;
                    }
            }
            int mine_all = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) mine_all += sum[e];
            int suf = mine_all;                     // keys of this lane's digits and above
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_down_sync(0xffffffffu, suf, o);
                if (lane + o < 32) suf += y;
            }
            // the digit: the largest with (keys of it and above) >= left
            int above = suf - mine_all, dg = -1, rest = 0;
#pragma unroll
            for (int e = 7; e >= 0; --e) {
                if (dg < 0 && above < left && above + sum[e] >= left) {
                    dg = 8 * lane + e;
                    rest = left - above;
                }
                above += sum[e];
            }
            const unsigned who = __ballot_sync(0xffffffffu, dg >= 0);
            if (left <= 0) {                        // nothing to take: a threshold above every key
                dg = 255;
                rest = 0;
            } else {
                const int from = __ffs(who) - 1;
                dg = __shfl_sync(0xffffffffu, dg, from);
                rest = __shfl_sync(0xffffffffu, rest, from);
            }
            int g = 0, q = 0;                       // this CTA's keys above the digit, and of it
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                g += 8 * lane + e > dg ? own[e] : 0;
                q += 8 * lane + e == dg ? own[e] : 0;
            }
            gt_mine += __reduce_add_sync(0xffffffffu, g);
            q = __reduce_add_sync(0xffffffffu, q);
            if (lane == 0) {
                sh_digit = (uint32_t)dg;
                sh_left = rest;
                if (round == 3) {
                    mine[0] = gt_mine;
                    mine[1] = q;
                }
            }
        } else if (tid < 288) {                     // the next round's histogram
            hist[(round + 1) & 1][tid - 32] = 0;
        }
        __syncthreads();
        left = sh_left;
        prefix = (prefix << 8) | sh_digit;
    }
    if (C > 1) cl.sync(); else __syncthreads();
    int gt_before = 0, eq_before = 0;
    for (int r = 0; r < rank; ++r) {
        gt_before += cl.map_shared_rank(mine, r)[0];
        eq_before += cl.map_shared_rank(mine, r)[1];
    }
    const uint32_t thr = prefix;
    const int need_eq = left;
    if (need > 0) {
        // each warp owns a run of 128-key steps, four keys a lane; counts first, then the
        // ordered write (counts above and at the threshold in the halves of a word)
        const int steps = (cnt + 127) / 128, wsteps = (steps + kWarps - 1) / kWarps;
        const int s_lo = min(steps, warp * wsteps), s_hi = min(steps, s_lo + wsteps);
        auto count = [&](int st, bool (&is_g)[4], bool (&is_q)[4], int &i) -> uint32_t {
            uint32_t k[4], c = 0;
            i = quad(st * 128, k);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                is_g[e] = i + e < cnt && k[e] > thr;
                is_q[e] = i + e < cnt && k[e] == thr;
                c += (is_g[e] ? 1u : 0u) + (is_q[e] ? 0x10000u : 0u);
            }
            return c;
        };
        bool is_g[4], is_q[4];
        int i;
        int g = 0, q = 0;
        for (int st = s_lo; st < s_hi; ++st) {
            const uint32_t c = count(st, is_g, is_q, i);
            g += c & 0xffffu;
            q += c >> 16;
        }
        g = __reduce_add_sync(0xffffffffu, g);
        q = __reduce_add_sync(0xffffffffu, q);
        if (lane == 0) {
            wgt[warp] = g;
            weq[warp] = q;
        }
        __syncthreads();
        const int bw = lane < warp ? wgt[lane] : 0, be = lane < warp ? weq[lane] : 0;
        gt_before += __reduce_add_sync(0xffffffffu, bw);
        eq_before += __reduce_add_sync(0xffffffffu, be);
        for (int st = s_lo; st < s_hi; ++st) {
            const uint32_t c = count(st, is_g, is_q, i);
            if (!__any_sync(0xffffffffu, c != 0u)) continue;
            uint32_t inc = c;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t y = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += y;
            }
            int gb = gt_before + (int)((inc - c) & 0xffffu), qb = eq_before + (int)((inc - c) >> 16);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (is_g[e] || (is_q[e] && qb < need_eq))
                    keep[a.n_sink + gb + min(qb, need_eq)] = c_lo + lo + i + e;
                gb += is_g[e] ? 1 : 0;
                qb += is_q[e] ? 1 : 0;
            }
            const uint32_t all = __shfl_sync(0xffffffffu, inc, 31);
            gt_before += all & 0xffffu;
            eq_before += all >> 16;
        }
    }
    if (C > 1) cl.sync();                           // mine[] is read by the others until here
}

// ------------------------------------------------------------------ the move
// One thread per 16 bytes of a kept row, K and V together; reads follow the list,
// writes are contiguous. Bound by HBM: 128 heads of up to 1000 rows (117 MB read and written) in 21 us, 5.5 TB/s.
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
    grid_wait();
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
    EvictArgs a{score, lens, Hkv, T, n_keep, n_sink, n_recent, 0, keep, count, err};
    // CTAs per (b, kv-head): one per 8192 keys while the GPU has SMs left (a second round of
    // clusters costs more than it splits: 32 heads of 32K keys take 18.5 us with four CTAs
    // each, 56 with eight; one head's 32K keys 31 us with one CTA, 18 with four), and as many
    // as hold the keys in shared memory; at most 8
    int C = 1;
    const auto slice = [&](int c) { return ((T + c - 1) / c + 31) & ~31; };
    while (C < kMaxCluster &&
           (slice(C) > kSliceMax || ((long long)C * 8192 < T && (long long)B * Hkv * C * 2 <= 148)))
        C *= 2;
    const int per = slice(C);
    a.cached = per <= kSliceMax;
    const size_t smem = a.cached ? (size_t)((per + 127) & ~127) * 4 : 0;   // whole steps of 128 keys
    const cudaError_t e = allow_smem<evict_select_kernel>((size_t)kSliceMax * 4 + 512);
    if (e != cudaSuccess) return e;
    void *args[] = {&a};
    return launch_early(reinterpret_cast<const void *>(evict_select_kernel), dim3((unsigned)((size_t)B * Hkv * C)),
                        dim3(kThreads), smem, args, s, (unsigned)C);
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
    void *args[] = {&a};
    return launch_early(reinterpret_cast<const void *>(gather_kernel), dim3((unsigned)((a.total + 255) / 256)), dim3(256),
                        0, args, s);
}

}  // namespace spa
