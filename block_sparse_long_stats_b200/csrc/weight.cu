// Attention weight that every cached key receives (bf16), on the sm_100a tensor cores.
//
//   w_t = sum_c exp(s q_c.k_t - lse_c) over the queries c of the key's kv-head that see t
//
// The score tile is taken transposed, S^T = K Q^T: 128 keys are the rows (TMEM lanes)
// and up to 256 queries the columns, so a thread owns one key and its sum runs over its
// own registers, with no reduction between threads. The log-sum-exp is an input, so
// one pass over K is enough. Decode (a few queries) is bound by reading K once (256
// bytes per key at d = 128); with some hundred queries and more the exponentials bound it
// (16 a cycle and SM).
//
// A query tile holds `pc` positions of all G heads of the group (so that a causal
// border cuts few tiles). Work is counted in (key tile, query tile) pairs, key tiles
// outside; tiles the causal border leaves nothing of are not counted. The pairs of all
// (b, kv-head) are cut into equal runs, one per CTA and SM. A key tile whose pairs lie in
// several runs leaves a partial sum per run in the workspace (at most the first and the last
// tile of a run do), and a second kernel adds them in order: no atomics, so a call repeats
// bit for bit.
//
// Warp roles: warps 0-15: four warpgroups; up to 128 columns they take the pairs in turn,
// each with a score tile of its own in tensor memory, with more (STREAM) two of them
// share a tile of 256 columns, 128 each (the N = 256 product runs at the full rate, 128
// cycles a step, where N = 128 takes 102-118, and half as many pairs pass the issuing
// thread); warps 16, 18: TMA producers (query tiles, and a half of every key tile each);
// warp 17: TMEM allocator and tcgen05.mma issuer.
//
// Measured (B200): a decode step's weight over four 128K caches with three quarters of the
// blocks kept 142 us (5.9 TB/s, 90 % of the measured copy bandwidth; weight_few_kernel),
// 128 queries over 32K keys 54 us, all queries of a 4K prompt 99 us (53 and 98 before the
// columns of queries that saw nothing were masked; carrying whether there are any on the
// barrier of the columns' lse took as long). In the last two ex2 is busy 54-57 % of
// the time and a scheduler issues 37 %: what is left is the latency of the
// sums. Tried, against 53 and 98: a product of N = 128 for each warpgroup of a score tile, begun as soon as its own
// half is read (59 us for the window: the products take longer than what the early start
// gains), the columns' lse in two buffers with one barrier instead of two (53.4 and 99), all four
// warpgroups on one score tile, 64 columns each, the other tile multiplied meanwhile (61 and
// 113; with a warp of its own for the lse 56 and 101), a quarter of the exponentials as
// polynomials on the FMA pipes (with the last 55 and 102: ex2 is not what bounds it).
#include <math.h>

#include "serve.h"

namespace spa {
namespace {

constexpr int kCtas = 148;             // one per SM
constexpr int kGroups = 4;             // consumer warpgroups
constexpr int kConsumers = kGroups * 128;
constexpr int kThreads = kConsumers + 96;
constexpr int kTile = 128;             // keys
constexpr int kUnits = 8;              // key tiles whose sums may be open at once: 7 at most (with
                                       // two score tiles no warpgroup is more than 6 pairs ahead)
constexpr int kMarkChunk = 512;        // blocks per CTA of the mark kernel
constexpr float kLog2e = 1.4426950408889634f;

struct WeightArgs {
    const int32_t *lens;
    const void *q, *k;
    const float *lse, *prev;
    const uint16_t *marks;             // [B, Hkv, nq, nbp] head masks of the kept blocks, or null
    float *out, *parts;                // parts [2 kCtas][kTile]
    int B, Hq, Hkv, G, Lq, T, block, nq, nbp;
    int pc, nqt;                       // positions per query tile, query tiles
    float scale_log2, decay;
    int *err;
};

template <int D, int NC, bool STREAM>
struct Cfg {
    static constexpr int HALVES = D / 64;
    static constexpr int K_HALF = kTile * 128;
    static constexpr int K_SLOT = HALVES * K_HALF;
    static constexpr int Q_HALF = NC * 128;
    static constexpr int Q_SLOT = HALVES * Q_HALF;
    // streams of query tiles want a deep query ring, a stream of key tiles a deep key ring
    static constexpr int NK = STREAM ? 2 : (D == 64 ? 8 : 4);
    static constexpr int NQ = 2;
    static constexpr int SHARE = STREAM ? 2 : 1;           // warpgroups per score tile
    static constexpr int BUFS = kGroups / SHARE;           // score tiles in tensor memory
    static constexpr int COLS = NC / SHARE;                // columns of a warpgroup
    static constexpr int OFF_Q = NK * K_SLOT;
    static constexpr int SMEM = OFF_Q + NQ * Q_SLOT + 1024;
    static constexpr uint32_t IDESC = idesc_bf16(128, NC, false);
};

__device__ __forceinline__ int seq_len(const WeightArgs &a, int b) {
    const int n = a.lens ? __ldg(a.lens + b) : a.T;
    return min(max(n, a.Lq), a.T);
}
// First query tile that sees key tile kt (off: position of the first query).
__device__ __forceinline__ int first_tile(const WeightArgs &a, int kt, int off) {
    const int t0 = kt * kTile - off;
    return t0 > 0 ? t0 / a.pc : 0;
}
// Pairs of one (b, kv-head), summed by a warp.
__device__ __forceinline__ long long pairs_of(const WeightArgs &a, int b) {
    const int len = seq_len(a, b), nt = (len + kTile - 1) / kTile, off = len - a.Lq;
    long long s = (long long)nt * a.nqt;
    if (a.nqt == 1) return s;
    long long skip = 0;
    for (int kt = max(0, off / kTile) + (int)(threadIdx.x & 31); kt < nt; kt += 32) skip += first_tile(a, kt, off);
#pragma unroll
    for (int o = 16; o; o >>= 1) skip += __shfl_xor_sync(0xffffffffu, skip, o);
    return s - skip;
}
__device__ __forceinline__ long long run_total(const WeightArgs &a) {
    if (!a.lens) return (long long)a.B * a.Hkv * pairs_of(a, 0);
    long long s = 0;
    if (a.nqt == 1) {
        for (int b = threadIdx.x & 31; b < a.B; b += 32) s += (seq_len(a, b) + kTile - 1) / kTile;
#pragma unroll
        for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    } else {
        for (int b = 0; b < a.B; ++b) s += pairs_of(a, b);
    }
    return s * a.Hkv;
}
__device__ __forceinline__ long long run_chunk(long long total) {
    const long long c = (total + kCtas - 1) / kCtas;
    return c < 1 ? 1 : c;
}

// A pair: sequence and kv-head, key tile, query tile. Advances in the runs' order.
struct Pair {
    int b, bg, kt, qi, nt, off;
    __device__ void at_head(const WeightArgs &a) {
        const int len = seq_len(a, b);
        nt = (len + kTile - 1) / kTile;
        off = len - a.Lq;
    }
    // Returns whether the key tile changed; new_head whether the (b, kv-head) did.
    __device__ bool next(const WeightArgs &a, bool &new_head) {
        new_head = false;
        if (++qi < a.nqt) return false;
        if (++kt >= nt) {
            kt = 0;
            ++bg;
            new_head = true;
            if (bg % a.Hkv == 0 && ++b < a.B) at_head(a);
        }
        qi = first_tile(a, kt, off);
        return true;
    }
};

// The pair at position pos of the runs; every lane of a warp calls it together.
__device__ __forceinline__ Pair locate(const WeightArgs &a, long long pos) {
    const int lane = threadIdx.x & 31;
    Pair p;
    p.b = 0;
    long long per = 0;
    if (!a.lens) {
        per = pairs_of(a, 0);
        p.bg = (int)(pos / per);
        p.b = p.bg / a.Hkv;
        pos -= per * p.bg;
    } else {
        for (;; ++p.b) {
            per = pairs_of(a, p.b);
            if (pos < per * a.Hkv || p.b + 1 >= a.B) break;
            pos -= per * a.Hkv;
        }
        const int g = (int)(pos / per);
        p.bg = p.b * a.Hkv + g;
        pos -= per * g;
    }
    p.at_head(a);
    if (a.nqt == 1) {
        p.kt = (int)pos;
        p.qi = 0;
        return p;
    }
    for (int k0 = 0;; k0 += 32) {                  // 32 key tiles a step
        const int kt = k0 + lane;
        const int np = kt < p.nt ? a.nqt - first_tile(a, kt, p.off) : 0;
        long long inc = np;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += y;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, inc > pos);
        if (hit || k0 + 32 >= p.nt) {
            const int src = hit ? __ffs(hit) - 1 : 0;
            p.kt = k0 + src;
            const long long rest = pos - (__shfl_sync(0xffffffffu, inc, src) - __shfl_sync(0xffffffffu, np, src));
            p.qi = first_tile(a, p.kt, p.off) + (int)rest;
            return p;
        }
        pos -= __shfl_sync(0xffffffffu, inc, 31);
    }
}

// -lse in log2 units, so that exp2(s log2e q.k + it) is the weight: 0 for a row of -inf.
__device__ __forceinline__ float minus_log2(float lse) { return lse == -INFINITY ? -INFINITY : -lse * kLog2e; }

// Sets bits [lo, hi) of a 128-bit mask.
__device__ __forceinline__ void set_range(uint32_t (&m)[4], int lo, int hi) {
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        const int l = min(max(lo - 32 * w, 0), 32), h = min(max(hi - 32 * w, 0), 32);
        const uint32_t below_h = h == 32 ? 0xffffffffu : (1u << h) - 1u;
        const uint32_t below_l = l == 32 ? 0xffffffffu : (1u << l) - 1u;
        m[w] |= below_h & ~below_l;
    }
}

template <int D, int NC, bool STREAM>
__global__ void __launch_bounds__(kThreads, 1)
    weight_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                  const __grid_constant__ WeightArgs a) {
    using C = Cfg<D, NC, STREAM>;
    constexpr int NK = C::NK, NQ = C::NQ, BUFS = C::BUFS, COLS = C::COLS;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *smem = reinterpret_cast<unsigned char *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ uint64_t full_k[NK], empty_k[NK], full_q[NQ], empty_q[NQ], s_full[BUFS], s_empty[BUFS];
    __shared__ uint32_t tmem_slot;
    __shared__ Pair sh_pair;
    __shared__ long long sh_total;
    __shared__ __align__(16) float nl_s[kGroups][COLS]; // -lse of the columns, log2 units
    __shared__ __align__(16) uint32_t dead_s[kGroups][4];   // columns of queries that saw nothing
    __shared__ float red[STREAM ? kUnits : 1][kGroups][kTile];   // sums of the last key tiles
    __shared__ int arrived[STREAM ? kUnits : 1][4];              // warps that have brought theirs

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int s = 0; s < NK; ++s) { mbar_init(&full_k[s], 2); mbar_init(&empty_k[s], 1); }
        for (int s = 0; s < NQ; ++s) { mbar_init(&full_q[s], 1); mbar_init(&empty_q[s], 1); }
        for (int w = 0; w < BUFS; ++w) { mbar_init(&s_full[w], 1); mbar_init(&s_empty[w], 128 * C::SHARE); }
        for (int w = 0; STREAM && w < kUnits * 4; ++w) arrived[w >> 2][w & 3] = 0;
        fence_mbar_init();
    }
    // query rows that no copy fills stay zero (finite scores; their columns count nothing)
    for (int x = tid; x < NQ * C::Q_SLOT / 16; x += kThreads)
        reinterpret_cast<uint4 *>(smem + C::OFF_Q)[x] = make_uint4(0, 0, 0, 0);
    fence_async_shared();
    if (warp == 16 && lane == 0) {
        prefetch_tmap(&tq);
        prefetch_tmap(&tk);
    }
    // tensor memory only after the wait: taken earlier it could be what a kernel that this one
    // waits for is waiting for
    grid_wait();
    if (warp == 17) tmem_alloc(&tmem_slot, 512);
    if (warp == 0) {
        const long long t = run_total(a), pos = (long long)blockIdx.x * run_chunk(t);
        if (lane == 0) sh_total = t;
        Pair p = {0, 0, 0, 0, 1, 0};             // a run without a pair: not used
        if (pos < t) p = locate(a, pos);
        if (lane == 0) sh_pair = p;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    const long long chunk = run_chunk(sh_total), pos0 = (long long)blockIdx.x * chunk;
    const int jobs = (int)max(0ll, min(sh_total, pos0 + chunk) - pos0);   // below 2^31: checked by the API
    const bool gq1 = a.nq == 1;

    if (warp == 16 || warp == 18) {
        // ---------------------------------------------------- producers
        // warp 16 copies the query tiles; of a key tile each copies a part: a 64-column half
        // (d = 128), or every other block
        bool ok = true;
        const int part = warp == 18;
        int nk = 0, nqs = 0;
        Pair p = sh_pair;
        bool new_k = true, new_q = true;
        const int per = kTile / a.block;
        int kept = 0, kept_at = -1;      // lane i: kept blocks of key tile kept_at + i
        for (int m = 0; m < jobs && ok; ++m) {
            if (new_q && lane == 0 && part == 0) {
                const int s = nqs % NQ;
                ok = mbar_wait(&empty_q[s], ((nqs / NQ) & 1) ^ 1, a.err);
                if (ok) {
                    mbar_arrive_expect_tx(&full_q[s], (uint32_t)(a.pc * a.G * D * 2));
                    const int head = p.b * a.Hq + (p.bg % a.Hkv) * a.G;
#pragma unroll
                    for (int hf = 0; hf < C::HALVES; ++hf)
                        asm volatile(
                            "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                            " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
                                smem_u32(smem + C::OFF_Q + s * C::Q_SLOT + hf * C::Q_HALF)),
                            "l"(&tq), "r"(smem_u32(&full_q[s])), "r"(hf * 64), "r"(p.qi * a.pc), "r"(head)
                            : "memory");
                }
            }
            if (new_q) ++nqs;
            if (new_k) {
                int want = (1 << per) - 1;
                if (a.marks && gq1) {    // one list per head: blocks that no head keeps are not read
                    if (kept_at < 0 || p.kt >= kept_at + 32 || p.kt < kept_at || p.kt == 0) {
                        kept_at = p.kt;
                        kept = 0;
                        const int kt = p.kt + lane;
                        if (kt < p.nt)
                            for (int e = 0; e < per; ++e) {
                                const int j = kt * per + e;
                                if (j < a.nbp && a.marks[(size_t)p.bg * a.nbp + j]) kept |= 1 << e;
                            }
                    }
                    want = __shfl_sync(0xffffffffu, kept, p.kt - kept_at);
                }
                if (D == 64) want &= part ? 0xaa : 0x55;
                if (lane == 0 && ok) {
                    const int s = nk % NK;
                    ok = mbar_wait(&empty_k[s], ((nk / NK) & 1) ^ 1, a.err);
                    if (ok) {
                        mbar_arrive_expect_tx(&full_k[s], (uint32_t)(__popc(want) * a.block * 128));
                        const int hf = D == 128 ? part : 0, row = p.bg * a.T + p.kt * kTile;
                        unsigned char *dst = smem + s * C::K_SLOT + hf * C::K_HALF;
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            if ((want >> e) & 1)
                                tma_load_2d(dst + e * a.block * 128, &tk, &full_k[s], hf * 64, row + e * a.block);
                    }
                }
                ++nk;
            }
            ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
            bool head;
            new_k = p.next(a, head);
            new_q = head || a.nqt > 1;
        }
        if (lane == 0 && !ok) {
            drain_ring<NK>(full_k, nk);
            if (part == 0) drain_ring<NQ>(full_q, nqs);
        }
    } else if (warp == 17) {
        // ---------------------------------------------------- products
        if (lane == 0) {
            // With one query tile per head two key tiles are multiplied together, step by step
            // in turn: a narrow product's steps wait for one another (some 100 cycles each)
            constexpr int TWO = STREAM ? 1 : 2;
            bool ok = true, new_k = true, new_q = true;
            int nk = 0, nqs = 0;
            Pair p = sh_pair;
            for (int m = 0; m < jobs && ok; m += TWO) {
                uint32_t kb[TWO], qb[TWO];
                int k_used[TWO], q_used[TWO], free_q[TWO];
                const int n = TWO == 1 || m + 1 == jobs ? 1 : 2;
#pragma unroll
                for (int i = 0; i < TWO; ++i) {
                    free_q[i] = 0;
                    if (i >= n || !ok) continue;
                    if (new_k) { ok = mbar_wait(&full_k[nk % NK], (nk / NK) & 1, a.err); ++nk; }
                    if (new_q && ok) ok = mbar_wait(&full_q[nqs % NQ], (nqs / NQ) & 1, a.err);
                    if (new_q) ++nqs;
                    if (ok) ok = mbar_wait(&s_empty[(m + i) % BUFS], (uint32_t)(((m + i) / BUFS) & 1) ^ 1u, a.err);
                    k_used[i] = (nk - 1) % NK;
                    q_used[i] = (nqs - 1) % NQ;
                    kb[i] = smem_u32(smem + k_used[i] * C::K_SLOT);
                    qb[i] = smem_u32(smem + C::OFF_Q + q_used[i] * C::Q_SLOT);
                    bool head;
                    new_k = p.next(a, head);
                    new_q = head || a.nqt > 1;
                    free_q[i] = new_q;
                }
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t ko = (kk >> 2) * C::K_HALF + (kk & 3) * 32, qo = (kk >> 2) * C::Q_HALF + (kk & 3) * 32;
#pragma unroll
                    for (int i = 0; i < TWO; ++i)
                        if (i < n)
                            tc_mma_ss(tmem + (m + i) % BUFS * (512 / BUFS), sw128_desc(kb[i] + ko, 16, 1024),
                                      sw128_desc(qb[i] + qo, 16, 1024), C::IDESC, kk > 0 ? 1u : 0u);
                }
#pragma unroll
                for (int i = 0; i < TWO; ++i) {
                    if (i >= n) continue;
                    tc_commit(&s_full[(m + i) % BUFS]);
                    if (!STREAM || new_k) tc_commit(&empty_k[k_used[i]]);
                    if (free_q[i]) tc_commit(&empty_q[q_used[i]]);
                }
            }
        }
    } else {
        // ---------------------------------------------------- sums
        const int wg = warp >> 2, r = tid & 127;
        const int buf = wg / C::SHARE, col0 = wg % C::SHARE * COLS;
        const uint32_t t_s = tmem + wg * 128 + ((uint32_t)((warp & 3) * 32) << 16);
        const int ch = (col0 + r) / a.pc, ci = col0 + r - ch * a.pc;   // this thread's column: head, position
        const bool col = r < COLS && ch < a.G;
        // keys behind every sequence: no weight
        for (int bg = blockIdx.x; bg < a.B * a.Hkv; bg += gridDim.x) {
            const int b = bg / a.Hkv, t0 = (seq_len(a, b) + kTile - 1) / kTile * kTile;
            if (a.lens && tid == 0 && bg % a.Hkv == 0) {
                const int n = __ldg(a.lens + b);
                if (n < a.Lq || n > a.T) set_error(a.err, SPA_DEVERR_BAD_COUNT);
            }
            for (int t = t0 + tid; t < a.T; t += kConsumers) {
                const size_t o = (size_t)bg * a.T + t;
                a.out[o] = a.prev ? a.decay * a.prev[o] : 0.f;
            }
        }
        Pair p = sh_pair;
        // the log-sum-exp of this thread's column of a pair's query tile; no row there: as if
        // it saw nothing
        auto column = [&](const Pair &x) -> float {
            if (!col || x.qi * a.pc + ci >= a.Lq) return -INFINITY;
            return __ldg(a.lse + ((size_t)x.bg * a.G + ch) * a.Lq + x.qi * a.pc + ci);
        };
        // The key tile's sum over the groups: each brings its own once (zero where it had no
        // pair), and of the four warps with the same keys the last one adds them up, in the
        // groups' order. No group waits for another; the score tiles keep them within a few jobs.
        auto bring = [&](const Pair &x, int unit, bool whole, bool first, float value) {
            const int slot = unit % kUnits, rows32 = warp & 3;
            red[slot][wg][r] = value;
            __threadfence_block();
            __syncwarp();
            int before = 0;
            if (lane == 0) before = atomicAdd(&arrived[slot][rows32], 1);
            if (__shfl_sync(0xffffffffu, before, 0) != kGroups - 1) return;
            __threadfence_block();
            if (lane == 0) arrived[slot][rows32] = 0;
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < kGroups; ++w) s += *reinterpret_cast<volatile float *>(&red[slot][w][r]);
            const int t = x.kt * kTile + r;
            if (t >= x.off + a.Lq) s = 0.f;
            if (t >= a.T) return;
            if (whole) {
                const size_t o = (size_t)x.bg * a.T + t;
                a.out[o] = a.prev ? fmaf(a.decay, a.prev[o], s) : s;
            } else {
                a.parts[((size_t)blockIdx.x * 2 + (first ? 0 : 1)) * kTile + r] = s;
            }
        };
        // this group walks over the run by its own pairs: p is pair m; a key tile that ends (or
        // is cut by the run's end) on the way is handed to `ended`
        int m = 0, units = 0, unit_first = 0;
        bool from_start = jobs > 0 && p.qi == first_tile(a, p.kt, p.off);
        auto advance = [&](int steps, auto &&ended) -> bool {
            for (;;) {
                const int rest = a.nqt - p.qi, left = jobs - m;      // pairs of the key tile, of the run
                if (steps < min(rest, left)) {
                    p.qi += steps;
                    m += steps;
                    return true;
                }
                ended(from_start && rest <= left, unit_first == 0);
                if (rest >= left) return false;
                m += rest;
                steps -= rest;
                ++units;
                unit_first = m;
                from_start = true;
                p.qi = a.nqt - 1;
                bool head;
                p.next(a, head);
            }
        };
        bool ok = true, more = jobs > 0;
        if (more)
            more = advance(buf, [&](bool whole, bool first) {
                if (STREAM) bring(p, units, whole, first, 0.f);
            });
        float sum = 0.f, nl_next = more && a.nqt > 1 ? column(p) : 0.f;
        int bg_cols = -1;                      // whose columns nl_s holds (one query tile per head)
        while (more) {
            // this pair, and where the next one lies (the columns' lse a pair ahead)
            const Pair at = p;
            const int mc = m;
            const float nl = nl_next;
            const bool fresh = a.nqt > 1 || at.bg != bg_cols;
            bg_cols = at.bg;
            int unit = -1;
            bool unit_whole = false, unit_begins = false;
            more = advance(BUFS, [&](bool whole, bool first) {
                if (!STREAM) return;
                if (unit < 0) {            // this pair's key tile: once its sum is there
                    unit = units;
                    unit_whole = whole;
                    unit_begins = first;
                } else {
                    bring(p, units, whole, first, 0.f);
                }
            });
            if (more && a.nqt > 1) nl_next = column(p);
            const int t = at.kt * kTile + r;
            const size_t o = (size_t)at.bg * a.T + t;
            float before = 0.f;
            if (!STREAM && a.prev && t < a.T) before = a.prev[o];
            uint32_t see[4];
            bool masked = false;
            const int q0 = at.off + at.qi * a.pc;        // position of the tile's first query
            const int lim = t - q0;                    // positions from lim on see the key
            if (a.marks) {
                masked = true;
#pragma unroll
                for (int c = 0; c < 4; ++c) see[c] = 0u;
                const int blk = t / a.block, qb0 = at.off / a.block;
                if (t < a.T) {
                    const uint16_t *mk = a.marks + (size_t)at.bg * a.nq * a.nbp + blk;
                    {
                        const int q_end = min(a.Lq, (at.qi + 1) * a.pc) + at.off;
                        for (int qb = q0 / a.block; qb * a.block < q_end; ++qb) {
                            const uint32_t hm = mk[(size_t)(qb - qb0) * a.nbp];
                            const int lo = max(max(qb * a.block - q0, 0), lim);
                            const int hi = min((qb + 1) * a.block, q_end) - q0;
                            if (lo < hi)
                                for (int h = 0; h < a.G; ++h)
                                    if ((hm >> h) & 1u) set_range(see, h * a.pc + lo - col0, h * a.pc + hi - col0);
                        }
                    }
                }
            } else if (at.kt * kTile + kTile - 1 > q0) {        // the causal border
                masked = true;
#pragma unroll
                for (int c = 0; c < 4; ++c) see[c] = 0u;
                if (lim < a.pc)
                    for (int h = 0; h < a.G; ++h) set_range(see, h * a.pc + max(lim, 0) - col0, (h + 1) * a.pc - col0);
            }
            if (fresh) {
                named_bar_sync(2 + wg, 128);           // the group is done with the last columns
                const float lse = a.nqt > 1 ? nl : column(at);
                const unsigned dead =
                    __ballot_sync(0xffffffffu, col && at.qi * a.pc + ci < a.Lq && lse == -INFINITY);
                if (r < COLS) nl_s[wg][r] = minus_log2(lse);
                if (lane == 0) dead_s[wg][warp & 3] = dead;
                named_bar_sync(2 + wg, 128);
            }
            // a query that saw nothing may hold anything (columns without a row hold zeros)
            const uint4 dead = *reinterpret_cast<const uint4 *>(dead_s[wg]);
            if ((dead.x | dead.y | dead.z | dead.w) != 0u) {
                if (!masked) see[0] = see[1] = see[2] = see[3] = 0xffffffffu;
                masked = true;
                see[0] &= ~dead.x;
                see[1] &= ~dead.y;
                see[2] &= ~dead.z;
                see[3] &= ~dead.w;
            }
            ok = __all_sync(0xffffffffu, ok && mbar_wait(&s_full[buf], (uint32_t)((mc / BUFS) & 1), a.err));
            if (ok) {
                tc_fence_after();
                uint64_t acc[2] = {0ull, 0ull};
                const uint64_t scale2 = f32x2(a.scale_log2, a.scale_log2);
                float x[2][16];
                tmem_ld16f(t_s, x[0]);
#pragma unroll
                for (int c0 = 0; c0 < COLS; c0 += 16) {
                    tc_wait_ld();
                    float *y = x[(c0 / 16) & 1];
                    if (c0 + 16 < COLS) {
                        tmem_ld16f(t_s + c0 + 16, x[(c0 / 16 + 1) & 1]);
                    } else {                       // all read: the next product may begin
                        tc_fence_before();
                        mbar_arrive(&s_empty[buf]);
                    }
                    // a key no one keeps may hold anything: select (few tiles have a mask:
                    // __any_sync keeps this a branch; as selects it took as long as the sums)
                    if (__any_sync(0xffffffffu, masked)) {
                        const uint32_t bits = see[c0 >> 5] >> (c0 & 16);
#pragma unroll
                        for (int e = 0; e < 16; ++e) y[e] = (bits >> e) & 1u ? y[e] : -INFINITY;
                    }
#pragma unroll
                    for (int e = 0; e < 16; e += 4) {
                        const float4 n4 = *reinterpret_cast<const float4 *>(&nl_s[wg][c0 + e]);
                        float y0, y1, y2, y3;
                        f32x2_split(fma_f32x2(f32x2(y[e], y[e + 1]), scale2, f32x2(n4.x, n4.y)), y0, y1);
                        f32x2_split(fma_f32x2(f32x2(y[e + 2], y[e + 3]), scale2, f32x2(n4.z, n4.w)), y2, y3);
                        acc[0] = add_f32x2(acc[0], f32x2(fast_exp2(y0), fast_exp2(y1)));
                        acc[1] = add_f32x2(acc[1], f32x2(fast_exp2(y2), fast_exp2(y3)));
                    }
                }
                float s0, s1;
                f32x2_split(add_f32x2(acc[0], acc[1]), s0, s1);
                sum += s0 + s1;
            }
            if (!STREAM) {                              // the key tile's only pair
                if (t < a.T) {
                    const bool in = t < at.off + a.Lq;
                    a.out[o] = a.prev ? fmaf(a.decay, before, in ? sum : 0.f) : (in ? sum : 0.f);
                }
                sum = 0.f;
            }
            if (STREAM && unit >= 0) {
                bring(at, unit, unit_whole, unit_begins, sum);
                sum = 0.f;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 17) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ---------------------------------------------------------------- a few queries
// Up to 16 query rows per kv-head (decode), bound by HBM: each key is read once. Neither
// tcgen05.mma nor TMA pays here: a product step over 128 keys takes over 100 cycles
// however few its columns (1300 a tile in all, where the tile's bytes leave 1050), and a
// copy box of a 16-key block some 90 (measured: 185 us, 4.5 TB/s, for a decode step over four
// 128K caches with mma.sync on TMA tiles). So a warp loads 16 keys straight into the
// fragments of mma.sync (keys as the 16 rows, queries as 8 or 16 columns): the features of a
// product step may be taken in any order, as long as keys and queries agree, so a lane's 16
// bytes of a key serve two steps and a quad reads 64 bytes together. The next 16 keys are
// on their way meanwhile. A quad holds a key's row and adds its weights. Equal runs of 16-key
// slabs over all warps.
constexpr int kSlab = 16;
constexpr int kFar = 1;                      // slabs behind the next one that are brought into L2
                                             // (decode step below: none 161 us, 1 142, 2 143, 4 152, 8 193)
constexpr int kFewThreads = 256, kFewCtas = 2 * kCtas;

template <int D, int NT>
__global__ void __launch_bounds__(kFewThreads, 2) weight_few_kernel(const __grid_constant__ WeightArgs a) {
    constexpr int KB = D / 32;                   // two product steps (32 features) each
    const int lane = threadIdx.x & 31, gq = lane >> 2, tq = lane & 3;
    const int wid = blockIdx.x * (kFewThreads / 32) + (threadIdx.x >> 5), warps = gridDim.x * (kFewThreads / 32);
    const int rows = a.G * a.Lq;
    grid_wait();
    // keys behind every sequence: no weight
    for (int bg = blockIdx.x; bg < a.B * a.Hkv; bg += gridDim.x) {
        const int b = bg / a.Hkv, t0 = (seq_len(a, b) + kSlab - 1) / kSlab * kSlab;
        if (a.lens && threadIdx.x == 0 && bg % a.Hkv == 0) {
            const int n = __ldg(a.lens + b);
            if (n < a.Lq || n > a.T) set_error(a.err, SPA_DEVERR_BAD_COUNT);
        }
        for (int t = t0 + threadIdx.x; t < a.T; t += kFewThreads) {
            const size_t o = (size_t)bg * a.T + t;
            a.out[o] = a.prev ? a.decay * a.prev[o] : 0.f;
        }
    }
    // this warp's run of slabs
    auto slabs = [&](int b) -> int { return (seq_len(a, b) + kSlab - 1) / kSlab; };
    long long total;
    if (a.lens) {
        int s = 0;
        for (int b = lane; b < a.B; b += 32) s += slabs(b);
        total = (long long)__reduce_add_sync(0xffffffffu, s) * a.Hkv;
    } else {
        total = (long long)a.B * a.Hkv * slabs(0);
    }
    long long pos = total * wid / warps;
    int left = (int)(total * (wid + 1) / warps - pos);
    if (left <= 0) return;
    int b = 0, ns = slabs(0);
    if (a.lens) {
        while (pos >= (long long)ns * a.Hkv) {
            pos -= (long long)ns * a.Hkv;
            ns = slabs(++b);
        }
    } else {
        b = (int)(pos / ((long long)ns * a.Hkv));
        pos -= (long long)b * ns * a.Hkv;
    }
    int bg = b * a.Hkv + (int)(pos / ns), sl = (int)(pos % ns), off = seq_len(a, b) - a.Lq;

    // the columns of this lane: position and head
    int ci[NT][2], ch[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int c = t * 8 + 2 * tq + e;
            ch[t][e] = c / a.Lq;
            ci[t][e] = c - ch[t][e] * a.Lq;
        }
    const bool one = a.marks && a.nq == 1;       // one list per head: the slab's heads as a mask
    // head masks of 32 slabs ahead, one per lane
    uint32_t ahead = 0xffffu;
    int ahead_at = -1;
    auto heads_of = [&](int bg_, int s_) -> uint32_t {
        if (!one) return 0xffffu;
        if (ahead_at < 0 || s_ < ahead_at || s_ >= ahead_at + 32) {
            ahead_at = s_;
            const int blk = (s_ + lane) * kSlab / a.block;
            ahead = blk < a.nbp ? a.marks[(size_t)bg_ * a.nbp + blk] : 0u;
        }
        return __shfl_sync(0xffffffffu, ahead, s_ - ahead_at);
    };
    const uint4 *k4 = static_cast<const uint4 *>(a.k);
    uint4 kr[2][KB][2];                          // [now, next][32 features][keys gq, gq + 8]
    float pr[2][2];
    uint32_t hm[2];
    auto load = [&](int bg_, int s_, uint32_t heads, uint4 (&r)[KB][2], float (&pv)[2]) {
        const int t = s_ * kSlab + gq;
        // slabs end inside the cache's rows or are cut at T
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const bool in = t + 8 * h < a.T;
            const size_t row = (size_t)bg_ * a.T + (in ? t + 8 * h : 0);
            if (heads) {
#pragma unroll
                for (int kb = 0; kb < KB; ++kb) r[kb][h] = __ldg(k4 + row * (D / 8) + kb * 4 + tq);
            }
            pv[h] = a.prev && in && tq == 0 ? a.prev[row] : 0.f;
        }
    };
    uint32_t qf[NT][KB][4];
    float nl[NT][2];
    uint32_t saw = 0;                            // bit 2 t + e: that column's query saw a key
    bool fresh = true;
    hm[0] = heads_of(bg, sl);
    load(bg, sl, hm[0], kr[0], pr[0]);
    for (;;) {
#pragma unroll
        for (int now = 0; now < 2; ++now) {      // unrolled so that the two buffers stay registers
            if (fresh) {                         // a new (b, kv-head): its rows lie together in q and lse
                fresh = false;
                saw = 0;
                const size_t row0 = (size_t)bg * rows;
                const uint4 *q4 = static_cast<const uint4 *>(a.q);
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const bool in = t * 8 + gq < rows;
#pragma unroll
                    for (int kb = 0; kb < KB; ++kb) {
                        const uint4 v = in ? __ldg(q4 + (row0 + t * 8 + gq) * (D / 8) + kb * 4 + tq)
                                           : make_uint4(0u, 0u, 0u, 0u);
                        qf[t][kb][0] = v.x;
                        qf[t][kb][1] = v.y;
                        qf[t][kb][2] = v.z;
                        qf[t][kb][3] = v.w;
                    }
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int c = t * 8 + 2 * tq + e;
                        const float lse = c < rows ? __ldg(a.lse + row0 + c) : -INFINITY;
                        nl[t][e] = minus_log2(lse);
                        if (lse != -INFINITY) saw |= 1u << (2 * t + e);
                    }
                }
            }
            // the next slab
            int bg2 = bg, sl2 = sl + 1, off2 = off, ns2 = ns;
            bool head2 = false;
            if (left > 1) {
                if (sl2 >= ns) {
                    sl2 = 0;
                    ++bg2;
                    head2 = true;
                    ahead_at = -1;
                    if (bg2 % a.Hkv == 0) {
                        off2 = seq_len(a, bg2 / a.Hkv) - a.Lq;
                        ns2 = slabs(bg2 / a.Hkv);
                    }
                }
                hm[now ^ 1] = heads_of(bg2, sl2);
                load(bg2, sl2, hm[now ^ 1], kr[now ^ 1], pr[now ^ 1]);
                // and the slabs after it into L2, a line per lane (a cut slab: its rows in the cache)
                const int far = sl2 + kFar;
                if (far < ns2 && (far - sl2) < left) {
                    const int at = one ? far - ahead_at : 0;
                    const int lines = min(kSlab, a.T - far * kSlab) * (D * 2 / 128);
                    if (at < 32 && (!one || __shfl_sync(0xffffffffu, ahead, at)) && lane < lines)
                        asm volatile("prefetch.global.L2 [%0];" ::"l"(
                            reinterpret_cast<const char *>(k4) + (((size_t)bg2 * a.T + far * kSlab) * D * 2 + lane * 128)));
                }
            }
            // this one
            const int t0 = sl * kSlab + gq, t1 = t0 + 8;
            const size_t o = (size_t)bg * a.T;
            float w0 = 0.f, w1 = 0.f;
            if (hm[now]) {
                float c[NT][2][4];               // two chains per column tile
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) c[t][0][e] = c[t][1][e] = 0.f;
#pragma unroll
                for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                    for (int t = 0; t < NT; ++t)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const uint4 x = kr[now][kb][0], y = kr[now][kb][1];
                            asm volatile(
                                "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
                                "{%8,%9}, {%0,%1,%2,%3};"
                                : "+f"(c[t][i][0]), "+f"(c[t][i][1]), "+f"(c[t][i][2]), "+f"(c[t][i][3])
                                : "r"(i ? x.z : x.x), "r"(i ? y.z : y.x), "r"(i ? x.w : x.y), "r"(i ? y.w : y.y),
                                  "r"(qf[t][kb][2 * i]), "r"(qf[t][kb][2 * i + 1]));
                        }
                const uint16_t *mk = a.marks && !one ? a.marks + (size_t)bg * a.nq * a.nbp + sl * kSlab / a.block : nullptr;
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int at = off + ci[t][e];               // the column's position
                        uint32_t heads = hm[now];
                        if (mk)
                            heads = ci[t][e] < a.Lq && ch[t][e] < a.G
                                        ? mk[(size_t)(at / a.block - off / a.block) * a.nbp] : 0u;
                        const bool in = (heads >> ch[t][e]) & (saw >> (2 * t + e)) & 1u;
                        // keys behind the sequence and queries that saw nothing may hold anything: select
                        const float y0 = fmaf(c[t][0][e] + c[t][1][e], a.scale_log2, nl[t][e]);
                        const float y1 = fmaf(c[t][0][2 + e] + c[t][1][2 + e], a.scale_log2, nl[t][e]);
                        w0 += in && t0 <= at ? fast_exp2(y0) : 0.f;
                        w1 += in && t1 <= at ? fast_exp2(y1) : 0.f;
                    }
                w0 += __shfl_xor_sync(0xffffffffu, w0, 1);
                w1 += __shfl_xor_sync(0xffffffffu, w1, 1);
                w0 += __shfl_xor_sync(0xffffffffu, w0, 2);
                w1 += __shfl_xor_sync(0xffffffffu, w1, 2);
            }
            if (tq == 0) {
                if (t0 < a.T) a.out[o + t0] = a.prev ? fmaf(a.decay, pr[now][0], w0) : w0;
                if (t1 < a.T) a.out[o + t1] = a.prev ? fmaf(a.decay, pr[now][1], w1) : w1;
            }
            if (--left == 0) return;
            bg = bg2;
            sl = sl2;
            off = off2;
            ns = ns2;
            fresh = head2;
        }
    }
}

// Adds the partial sums of the key tiles that lie in several runs: CTA c looks after the
// tile that run c begins inside of, if that tile began in run c - 1 or before and no
// run between begins inside of it too.
__global__ void __launch_bounds__(kTile) weight_join_kernel(const __grid_constant__ WeightArgs a) {
    grid_wait();
    const int r = threadIdx.x;
    const long long total = run_total(a), chunk = run_chunk(total);
    const long long pos = (long long)blockIdx.x * chunk;
    if (blockIdx.x == 0 || pos >= total) return;
    const Pair p = locate(a, pos);
    const int first = first_tile(a, p.kt, p.off);
    if (p.qi == first) return;                                       // run c begins with a tile
    const long long t_pos = pos - (p.qi - first), t_end = t_pos + (a.nqt - first);
    const int c0 = (int)(t_pos / chunk), c1 = (int)((t_end - 1) / chunk);
    if ((int)blockIdx.x != c0 + 1) return;                            // the first run that continues it
    const int t = p.kt * kTile + r;
    if (t >= a.T) return;
    float s = 0.f;
    for (int c = c0; c <= c1; ++c) {
        const bool begins = c == c0 && t_pos != (long long)c0 * chunk;
        s += a.parts[((size_t)c * 2 + (begins ? 1 : 0)) * kTile + r];
    }
    const size_t o = (size_t)p.bg * a.T + t;
    a.out[o] = a.prev ? fmaf(a.decay, a.prev[o], s) : s;
}

// Head masks of the kept blocks, [B, Hkv, nq, nbp]: CTA ((b, kv-head, query block), chunk
// of blocks).
__global__ void __launch_bounds__(256) mark_kernel(const int32_t *__restrict__ idx, const int32_t *__restrict__ count,
                                                   int Hkv, int G, int nq, int nb, int nbp, int cap,
                                                   uint16_t *__restrict__ marks, int *err) {
    __shared__ __align__(16) uint16_t mk[kMarkChunk];
    const int unit = blockIdx.x, bg = unit / nq, qb = unit % nq, j_lo = blockIdx.y * kMarkChunk;
    const int j_hi = min(nbp, j_lo + kMarkChunk), warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    grid_wait();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    for (int x = threadIdx.x; x < kMarkChunk / 8; x += 256) reinterpret_cast<uint4 *>(mk)[x] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    for (int h = warp & 3; h < G; h += 4) {                 // two warps per head
        const size_t u = (((size_t)bg * G) + h) * nq + qb;
        int cnt = __ldg(count + u);
        if (cnt < 0 || cnt > cap) {
            set_error(err, SPA_DEVERR_BAD_COUNT);
            cnt = cnt < 0 ? 0 : cap;
        }
        const int32_t *list = idx + u * cap;
        // lists shorter than a chunk are read whole, longer ones from a 32-way search on
        int lo = 0, hi = cnt;
        while (hi - lo > 1024) {
            const int step = (hi - lo + 31) / 32, q = lo + (lane + 1) * step - 1;
            const bool less = q < hi && __ldg(list + q) < j_lo;
            const int k = __popc(__ballot_sync(0xffffffffu, less));
            const int nlo = min(hi, lo + k * step);
            hi = max(nlo, min(hi, lo + (k + 1) * step - 1));
            lo = nlo;
        }
        for (int e0 = lo + (warp >> 2) * 128; e0 < cnt; e0 += 256) {
            int j[4], before[4];
            bool past = true;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int e = e0 + i * 32 + lane;
                j[i] = e < cnt ? __ldg(list + e) : 0x7fffffff;
                before[i] = e < cnt && e > 0 ? __ldg(list + e - 1) : -1;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (e0 + i * 32 + lane >= cnt) continue;
                if (j[i] < 0 || j[i] >= nb || before[i] >= j[i]) {
                    set_error(err, SPA_DEVERR_BAD_INDEX);
                    past = false;
                    continue;
                }
                past = past && j[i] >= j_hi;
                if (j[i] >= j_lo && j[i] < j_hi) {
                    const int x = j[i] - j_lo;
                    atomicOr(reinterpret_cast<unsigned int *>(mk + (x & ~1)), (unsigned)(1u << h) << ((x & 1) * 16));
                }
            }
            if (__all_sync(0xffffffffu, past)) break;
        }
    }
    __syncthreads();
    uint4 *dst = reinterpret_cast<uint4 *>(marks + (size_t)unit * nbp + j_lo);
    for (int x = threadIdx.x; x < (j_hi - j_lo) / 8; x += 256) dst[x] = reinterpret_cast<const uint4 *>(mk)[x];
}

bool make_maps(CUtensorMap *mq, CUtensorMap *mk, const WeightCall &c, int pc) {
    EncodeTiledFn enc = encode_tiled_fn();
    if (!enc) return false;
    const cuuint32_t one[3] = {1, 1, 1};
    const cuuint64_t qd[3] = {(cuuint64_t)c.d, (cuuint64_t)c.Lq, (cuuint64_t)c.B * c.Hq};
    const cuuint64_t qs[2] = {(cuuint64_t)c.d * 2, (cuuint64_t)c.Lq * c.d * 2};
    const cuuint32_t qb[3] = {64, (cuuint32_t)pc, (cuuint32_t)(c.Hq / c.Hkv)};
    const cuuint64_t kd[2] = {(cuuint64_t)c.d, (cuuint64_t)c.B * c.Hkv * c.T};
    const cuuint64_t ks[1] = {(cuuint64_t)c.d * 2};
    const cuuint32_t kb[2] = {64, (cuuint32_t)c.block};
    return enc(mq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(c.q), qd, qs, qb, one,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS &&
           enc(mk, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(c.k), kd, ks, kb, one,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int NC, bool STREAM>
cudaError_t launch_cfg(const WeightCall &c, WeightArgs &a, cudaStream_t s) {
    using C = Cfg<D, NC, STREAM>;
    CUtensorMap mq, mk;
    if (!make_maps(&mq, &mk, c, a.pc)) return cudaErrorNotSupported;
    const void *kern = reinterpret_cast<const void *>(weight_kernel<D, NC, STREAM>);
    cudaError_t e = allow_smem<weight_kernel<D, NC, STREAM>>(C::SMEM);
    if (e != cudaSuccess) return e;
    const long long most = (long long)c.B * c.Hkv * ((c.T + kTile - 1) / kTile) * a.nqt;
    void *args[] = {&mq, &mk, &a};
    e = launch_early(kern, dim3((unsigned)(most < kCtas ? most : kCtas)), dim3(kThreads), C::SMEM, args, s);
    if (e != cudaSuccess || a.nqt == 1) return e;      // one pair per key tile: no partial sums
    void *jargs[] = {&a};
    return launch_early(reinterpret_cast<const void *>(weight_join_kernel), dim3(kCtas), dim3(kTile), 0, jargs, s);
}

template <int D, int NT>
cudaError_t launch_few(const WeightCall &c, WeightArgs &a, cudaStream_t s) {
    const long long most = (long long)c.B * c.Hkv * ((c.T + kSlab - 1) / kSlab);
    const long long ctas = (most + kFewThreads / 32 - 1) / (kFewThreads / 32);
    void *args[] = {&a};
    return launch_early(reinterpret_cast<const void *>(weight_few_kernel<D, NT>),
                        dim3((unsigned)(ctas < kFewCtas ? ctas : kFewCtas)), dim3(kFewThreads), 0, args, s);
}

template <int D>
cudaError_t launch_d(const WeightCall &c, WeightArgs &a, cudaStream_t s) {
    // query tiles of up to 256 rows, in a stream; or one tile as narrow as the rows allow
    if (a.G * a.pc > 128) return launch_cfg<D, 256, true>(c, a, s);
    const int rows = a.G * a.pc;
    if (rows <= 8) return launch_few<D, 1>(c, a, s);
    if (rows <= 16) return launch_few<D, 2>(c, a, s);
    if (rows <= 64) return launch_cfg<D, 64, false>(c, a, s);
    return launch_cfg<D, 128, false>(c, a, s);
}

int query_blocks(int Lq, int T, int block) { return (T - 1) / block - (T - Lq) / block + 1; }
constexpr size_t kPartBytes = (size_t)2 * kCtas * kTile * sizeof(float);

}  // namespace

// Partial sums of the runs, then (with lists: block > 0) the head masks.
size_t weight_workspace_bytes(int B, int Hkv, int Lq, int T, int block) {
    size_t n = kPartBytes;
    if (block > 0) {
        const size_t nbp = ((size_t)((T + block - 1) / block) + 7) & ~size_t(7);
        n += (size_t)B * Hkv * query_blocks(Lq, T, block) * nbp * sizeof(uint16_t);
    }
    return n;
}

cudaError_t launch_weight(const WeightCall &c, cudaStream_t s) {
    WeightArgs a;
    a.q = c.q; a.k = c.k;
    a.lens = c.lens; a.lse = c.lse; a.prev = c.prev;
    a.out = c.out;
    a.parts = static_cast<float *>(c.workspace);
    a.B = c.B; a.Hq = c.Hq; a.Hkv = c.Hkv; a.G = c.Hq / c.Hkv; a.Lq = c.Lq; a.T = c.T; a.block = c.block;
    a.pc = 256 / a.G < c.Lq ? 256 / a.G : c.Lq;
    a.nqt = (c.Lq + a.pc - 1) / a.pc;
    a.scale_log2 = c.scale * kLog2e;
    a.decay = c.decay;
    a.err = c.err;
    a.marks = nullptr;
    a.nq = query_blocks(c.Lq, c.T, c.block);
    a.nbp = 0;
    if (c.idx) {
        const int nb = (c.T + c.block - 1) / c.block;
        a.nbp = (nb + 7) & ~7;
        uint16_t *marks = reinterpret_cast<uint16_t *>(static_cast<unsigned char *>(c.workspace) + kPartBytes);
        a.marks = marks;
        const dim3 grid((unsigned)(c.B * c.Hkv * a.nq), (unsigned)((a.nbp + kMarkChunk - 1) / kMarkChunk));
        int Hkv = c.Hkv, nb_ = nb, cap = c.cap;
        const int32_t *idx = c.idx, *count = c.count;
        int *err = c.err;
        void *args[] = {&idx, &count, &Hkv, &a.G, &a.nq, &nb_, &a.nbp, &cap, &marks, &err};
        const cudaError_t e = launch_early(reinterpret_cast<const void *>(mark_kernel), grid, dim3(256), 0, args, s);
        if (e != cudaSuccess) return e;
    }
    return c.d == 64 ? launch_d<64>(c, a, s) : launch_d<128>(c, a, s);
}

}  // namespace spa
