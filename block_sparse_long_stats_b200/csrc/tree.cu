// Attention of a tree of drafted tokens over the kept blocks of a KV cache (bf16), on
// the sm_100a tensor cores.
//
//   out_i = sum_u softmax_u(s q_i.k_u) v_u over the kept cached keys and the ancestors
//
// The rows of a problem are the G n queries of a (b, kv-head): they lie next to each
// other in q, and all of them read the same keys. A CTA has 128 of them, a row tile. Decode
// with a few drafted tokens is bound by the bytes of K and V (512 per key at d = 128 against
// 4 G n d flops); from about 200 rows on the tensor cores and the exponentials take as long.
//
// Work is counted in tiles of 128 keys of text (the tree itself is the last tile of its
// sequence). The tiles of all (b, kv-head) units in a row are cut into equal runs, whatever
// the sequences' lengths: a run may end inside a unit and go on in the next one. Of its
// stretch of text a run reads the kept blocks alone, closed up to tiles again, so its
// work is what the lists keep there: with blocks kept at random 61 tiles at most where
// the mean is 56 (16 nodes below), 14 where it is 10.5 (64 nodes), and further apart the
// more the kept blocks cluster. A run is a CTA per row tile; these stand next to each other in
// the grid and read the same K and V at the same time, so that they cross HBM once. A unit
// that lies in several runs leaves one (m, l, O) state per run in the workspace, and a
// second kernel joins them.
//
// Two CTAs per SM (96 KB of tiles and half of tensor memory each): a CTA's chain of
// S = Q K^T, softmax, O += P V is serial (P lies over S), and the SM works on one CTA's
// products and copies during the other's softmax. Warp roles:
//   warps 0-3 : softmax; thread r owns row r = TMEM lane r
//   warp 4    : TMA producer (Q per unit; K and V tiles)
//   warp 5    : TMEM allocator and tcgen05.mma issuer
//
// P is rounded to bf16 for the second product, as in prefill: V is bf16, and both operands
// of a product have one type. Against fp64 the output is then off by 2.1e-3 (7 nodes) to
// 2.3e-3 of its norm, 1.66e-3 of which is its own rounding. P as the sum of two bf16 halves
// (twice the products) left 1.66e-3 and took 280 us a call where this takes 227 (16 nodes,
// long runs), and 66 against 57 (64 nodes).
//
// Measured (B200, main kernel, ten calls one after another; in brackets alone and cold):
// 16 nodes, 32/8 heads over four 128K caches, half of the 16-key blocks kept: 200 us, 5.4
// TB/s of kept K and V (up to 30 more in long runs under the power cap: half of the products'
// rows are empty). 64 nodes over 32K: 49 us (52); 33 nodes, 40/8 heads over eight ragged
// caches with 343 MB of K and V: 106 us (114); there a tile takes 4600 cycles with two CTAs
// on the SM: 2500 of softmax, 2000 for the products, which wait for one another.
// Tried: runs of two and four blocks copied in boxes of their own too (210 us for the first
// case: the longer issuing loop costs more than the fewer boxes save), one CTA per SM with two
// softmax warpgroups and deeper rings (107 us for the last case with one MMA warp, 117 with
// two), and halves of 64 keys with a score tile each, so that a warpgroup's softmax
// overlaps its own products (134 us: a step with N = 64 takes nearly as long as one with
// N = 128).
#include <math.h>

#include "serve.h"

namespace spa {
namespace {

constexpr int kCtas = 296;             // two per SM
constexpr int kThreads = 192;
constexpr int kTile = 128;             // keys
constexpr int kRange = 1536;           // blocks whose list is held in shared memory
constexpr int kShortList = 1024;       // entries up to which a list is read whole
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescaleThreshold = 8.0f;   // log2 units

struct TreeArgs {
    const int32_t *parents, *lens, *idx, *count;
    __nv_bfloat16 *out;
    float *lse, *ws_o, *ws_ml;
    int B, Hq, Hkv, G, n, T, cap;
    int nrt, runs;                       // row tiles per (b, kv-head), runs (CTAs per row tile)
    float scale_log2;
    int *err;
};

template <int D, int BLK>
struct Cfg {
    static constexpr int PER = kTile / BLK;            // blocks per tile
    static constexpr int HALVES = D / 64;              // 64-column halves (128-byte swizzle)
    static constexpr int HALF = kTile * 128;           // bytes of one
    static constexpr int SLOT = HALVES * HALF;         // a K or V tile, the Q tile
    static constexpr int ST = D == 64 ? 2 : 1;         // K and V tiles in flight
    static constexpr int OFF_K = SLOT;
    static constexpr int OFF_V = OFF_K + ST * SLOT;
    static constexpr int OFF_LIST = OFF_V + ST * SLOT; // uint32 [kRange]: head mask, block
    static constexpr int OFF_MARK = OFF_LIST + kRange * 4;   // uint16 [kRange]
    static constexpr int SMEM = OFF_MARK + kRange * 2 + 1024;
    static constexpr uint32_t IDESC_S = idesc_bf16(128, kTile, false);
    static constexpr uint32_t IDESC_O = idesc_bf16(128, D, true);
};

// Text length before the tree, clamped to the cache.
__device__ __forceinline__ int text_len(const TreeArgs &a, int b) {
    const int p = a.lens ? __ldg(a.lens + b) : a.T - a.n;
    return min(max(p, 0), a.T - a.n);
}
__device__ __forceinline__ int tiles_of(const TreeArgs &a, int b) {
    return (text_len(a, b) + kTile - 1) / kTile + 1;
}

// The runs: tiles in all (below 2^31: the rows of the caches are), tiles per CTA, and
// where a tile lies. Every lane of a warp calls these together.
struct Where {
    int b, unit, t;      // sequence, unit (b-major, then kv-head), tile of the unit
};
__device__ __forceinline__ int run_total(const TreeArgs &a) {
    const int lane = threadIdx.x & 31, upb = a.Hkv;
    if (!a.lens) return a.B * upb * tiles_of(a, 0);
    int s = 0;
    for (int b = lane; b < a.B; b += 32) s += tiles_of(a, b);
    return __reduce_add_sync(0xffffffffu, s) * upb;
}
__device__ __forceinline__ int run_chunk(const TreeArgs &a, int total) {
    return (total + a.runs - 1) / a.runs;
}
__device__ __forceinline__ Where locate(const TreeArgs &a, int pos) {
    const int lane = threadIdx.x & 31, upb = a.Hkv;
    Where w;
    if (!a.lens) {
        const int tb = tiles_of(a, 0);
        w.unit = pos / tb;
        w.t = pos - w.unit * tb;
        w.b = w.unit / upb;
        return w;
    }
    int before = 0;
    for (int b0 = 0;; b0 += 32) {
        const int b = b0 + lane;
        const int tb = b < a.B ? tiles_of(a, b) : 0;
        int inc = tb * upb;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += y;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, b < a.B && before + inc > pos);
        if (hit) {                        // always: pos < run_total
            const int src = __ffs(hit) - 1;
            const int tbs = __shfl_sync(0xffffffffu, tb, src);
            const int base = before + __shfl_sync(0xffffffffu, inc, src) - tbs * upb;
            w.b = b0 + src;
            const int k = (pos - base) / tbs;
            w.unit = w.b * upb + k;
            w.t = pos - base - k * tbs;
            return w;
        }
        before += __shfl_sync(0xffffffffu, inc, 31);
    }
}

// First entry of an ascending list that is >= j: 32 probes a step.
__device__ __forceinline__ int lower_bound(const int32_t *list, int cnt, int j) {
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = cnt;                       // the answer lies in [lo, hi]
    while (hi - lo > 0) {
        const int step = (hi - lo + 31) / 32;
        const int p = lo + (lane + 1) * step - 1;
        const bool less = p < hi && __ldg(list + p) < j;
        const int k = __popc(__ballot_sync(0xffffffffu, less));
        const int nlo = min(hi, lo + k * step);
        hi = min(hi, lo + (k + 1) * step - 1);
        lo = nlo;
        if (hi < lo) hi = lo;
    }
    return lo;
}

// What a CTA's roles share about the segment (the part of a run inside one unit) and the
// stretch of its list they are at. It stays in shared memory and is read where it is
// needed: the softmax holds 128 scores in registers and has none to spare.
struct Segment {
    int pos, end;                       // the run's next tile, its end
    int b, unit, P, more;
    int t_hi, whole, with_tree;         // the unit's tiles end; all of them, the tree here
    int j_hi;                           // blocks of the text end
    int s_lo, nu, ntile, tree_here;     // the stretch: first block, kept blocks, tiles
    int clean;                          // tiles of PER whole blocks, ahead of the others
    int tu, segs;                       // key tiles, segments so far
    int had;                            // key tiles of this segment
};

template <int D, int BLK>
__global__ void __launch_bounds__(kThreads, 2)
    tree_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                const __grid_constant__ CUtensorMap tv, const __grid_constant__ CUtensorMap tk1,
                const __grid_constant__ CUtensorMap tv1, const __grid_constant__ TreeArgs a) {
    using C = Cfg<D, BLK>;
    constexpr int PER = C::PER, ST = C::ST;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *smem = reinterpret_cast<unsigned char *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint32_t *ulist = reinterpret_cast<uint32_t *>(smem + C::OFF_LIST);
    uint16_t *mark = reinterpret_cast<uint16_t *>(smem + C::OFF_MARK);
    __shared__ uint64_t bar_q, full_k[ST], empty_k[ST], full_v[ST], empty_v[ST], s_full, p_ready, o_done;
    __shared__ uint32_t tmem_slot;
    __shared__ Segment sg;
    __shared__ int par[kTile];
    __shared__ uint32_t nmask[kTile][4];          // ancestors and self; all zero: unused
    __shared__ int wcount[kThreads / 32];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        mbar_init(&bar_q, 1);
        for (int s = 0; s < ST; ++s) {
            mbar_init(&full_k[s], 1);
            mbar_init(&empty_k[s], 1);
            mbar_init(&full_v[s], 1);
            mbar_init(&empty_v[s], 1);
        }
        mbar_init(&s_full, 1);
        mbar_init(&p_ready, 128);
        mbar_init(&o_done, 1);
        fence_mbar_init();
        fence_async_shared();
    }
    if (warp == 4 && lane == 0) {
        prefetch_tmap(&tq);
        prefetch_tmap(&tk);
        prefetch_tmap(&tv);
    }
    // tensor memory only after the wait: taken earlier it could be what a kernel that this one
    // waits for is waiting for
    grid_wait();
    if (warp == 5) tmem_alloc(&tmem_slot, 256);
    if (warp == 0) {
        const int total = run_total(a), chunk = run_chunk(a, total);
        if (lane == 0) {
            sg.pos = blockIdx.x / a.nrt * chunk;
            sg.end = min(total, sg.pos + chunk);
            sg.tu = 0;
            sg.segs = -1;
        }
    }
    const int row0 = blockIdx.x % a.nrt * 128;     // this CTA's rows of every (b, kv-head)
    // Up to 64 rows fill two of the softmax warps. The SM's second CTA (the grid's second
    // 148) takes the other two lane quarters, whose warps issue on the SM's other two
    // sub-partitions.
    const int shift = a.G * a.n - row0 <= 64 && blockIdx.x >= kCtas / 2 ? 64 : 0;
    bool ok = true;                    // cleared by a wait that ran out: no more work, no waits
    tc_fence_before();
    __syncthreads();
    tc_fence_after();

    for (;;) {
        // ------------------------------------------------ the segment
        if (warp == 0) {
            __syncwarp();
            const int pos = sg.pos;
            const bool more = pos < sg.end;
            Where w = {0, 0, 0};
            if (more) w = locate(a, pos);
            if (lane == 0) {
                sg.more = more;
                if (more) {
                    const int P = text_len(a, w.b), tiles = (P + kTile - 1) / kTile + 1;
                    sg.b = w.b;
                    sg.unit = w.unit;
                    sg.P = P;
                    sg.t_hi = min(tiles, w.t + sg.end - pos);
                    sg.with_tree = sg.t_hi == tiles;
                    sg.whole = w.t == 0 && sg.with_tree;
                    sg.s_lo = w.t * PER;
                    sg.j_hi = min((P + BLK - 1) / BLK, sg.t_hi * PER);
                    sg.pos = pos + sg.t_hi - w.t;
                    sg.had = 0;
                    ++sg.segs;
                    if (a.lens && w.unit % a.Hkv == 0 && sg.with_tree) {
                        const int p = __ldg(a.lens + w.b);
                        if (p < 0 || p > a.T - a.n) set_error(a.err, SPA_DEVERR_BAD_COUNT);
                    }
                }
            }
        }
        __syncthreads();
        if (!sg.more) break;
        if (warp == 4 && lane == 0 && ok) {
            mbar_arrive_expect_tx(&bar_q, C::SLOT);
            const int qrow = sg.unit * a.G * a.n + row0 - shift;   // rows before q: zero-filled
#pragma unroll
            for (int hf = 0; hf < C::HALVES; ++hf) tma_load_2d(smem + hf * C::HALF, &tq, &bar_q, hf * 64, qrow);
        }
        if (tid < a.n) par[tid] = __ldg(a.parents + (size_t)sg.b * a.n + tid);
        if (a.idx)
            for (int x = tid; x < kRange / 2; x += kThreads) reinterpret_cast<uint32_t *>(mark)[x] = 0u;
        __syncthreads();
        if (tid < kTile) {
            uint32_t m0 = 0, m1 = 0, m2 = 0, m3 = 0;
            int j = tid < a.n ? tid : -2;
            while (j >= 0) {
                const uint32_t bit = 1u << (j & 31);
                if (j < 32) m0 |= bit; else if (j < 64) m1 |= bit; else if (j < 96) m2 |= bit; else m3 |= bit;
                const int p = par[j];
                if (p >= j) {
                    set_error(a.err, SPA_DEVERR_BAD_INDEX);
                    j = -2;
                } else {
                    j = max(p, -2);
                }
            }
            if (j == -2) m0 = m1 = m2 = m3 = 0;
            nmask[tid][0] = m0;
            nmask[tid][1] = m1;
            nmask[tid][2] = m2;
            nmask[tid][3] = m3;
        }

        float m_used = -INFINITY, l = 0.f;
        int started = 0;                             // MMA: a product is in O
        for (;;) {
            // ---------------------------------------- kept blocks of the stretch
            if (a.idx) {
                const int s_lo = sg.s_lo, s_hi = min(sg.j_hi, s_lo + kRange), nr = max(0, s_hi - s_lo);
                const int nb_all = (a.T + BLK - 1) / BLK;
                // warps and heads in turn; a list's stretch is found by a 32-way search unless
                // the whole list is short
                constexpr int kW = kThreads / 32;
                const int h_lo = row0 / a.n, nh = (min(a.G * a.n, row0 + 128) - 1) / a.n + 1 - h_lo;
                const int share = max(1, kW / nh);                         // warps per head
                for (int k = warp; k < nh * share; k += kW) {
                    const int hh = h_lo + k % nh, part = k / nh;
                    const size_t u = (size_t)sg.unit * a.G + hh;
                    const int32_t *list = a.idx + u * a.cap;
                    int cnt = __ldg(a.count + u);
                    if (cnt < 0 || cnt > a.cap) {
                        if (lane == 0) set_error(a.err, SPA_DEVERR_BAD_COUNT);
                        cnt = cnt < 0 ? 0 : a.cap;
                    }
                    int lo = 0, hi = cnt;
                    if (cnt > kShortList) {
                        lo = lower_bound(list, cnt, s_lo);
                        hi = lower_bound(list, cnt, s_hi);
                        if (lane == 0 && part == 0 && sg.with_tree && __ldg(list + cnt - 1) >= nb_all)
                            set_error(a.err, SPA_DEVERR_BAD_INDEX);
                    }
                    constexpr int kAhead = 8;                              // loads in flight per lane
                    for (int p0 = lo + part * 32; p0 < hi; p0 += share * 32 * kAhead) {
                        int j[kAhead], before[kAhead];
#pragma unroll
                        for (int i = 0; i < kAhead; ++i) {
                            const int p = p0 + i * share * 32 + lane;
                            j[i] = p < hi ? __ldg(list + p) : s_hi;
                            before[i] = p < hi && p > 0 ? __ldg(list + p - 1) : -1;
                        }
#pragma unroll
                        for (int i = 0; i < kAhead; ++i) {
                            if (p0 + i * share * 32 + lane >= hi) continue;
                            if (j[i] < 0 || j[i] >= nb_all || before[i] >= j[i]) {
                                set_error(a.err, SPA_DEVERR_BAD_INDEX);
                                continue;
                            }
                            const int x = j[i] - s_lo;
                            if (x >= 0 && x < nr)
                                atomicOr(reinterpret_cast<unsigned int *>(mark + (x & ~1)),
                                         (unsigned)(1u << hh) << ((x & 1) * 16));
                        }
                    }
                }
                __syncthreads();
                // close up: each warp a stretch, behind the blocks of the warps before
                const int steps = (nr + 31) / 32, per = (steps + kW - 1) / kW;
                const int x_lo = min(nr, warp * per * 32), x_hi = min(nr, x_lo + per * 32);
                int c = 0;
                for (int x = x_lo; x < x_hi; x += 32)
                    c += __popc(__ballot_sync(0xffffffffu, x + lane < x_hi && mark[x + lane] != 0));
                if (lane == 0) wcount[warp] = c;
                __syncthreads();
                int at = 0;
                for (int w = 0; w < warp; ++w) at += wcount[w];
                for (int x = x_lo; x < x_hi; x += 32) {
                    const uint32_t m = x + lane < x_hi ? mark[x + lane] : 0u;
                    const unsigned bal = __ballot_sync(0xffffffffu, m != 0);
                    if (m) ulist[at + __popc(bal & ((1u << lane) - 1u))] = (m << 16) | (uint32_t)(x + lane);
                    at += __popc(bal);
                }
            }
            if (a.idx) __syncthreads();
            if (tid == 0) {
                int nu;
                if (a.idx) {
                    nu = 0;
                    for (int w = 0; w < kThreads / 32; ++w) nu += wcount[w];
                    sg.tree_here = sg.with_tree && sg.s_lo + kRange >= sg.j_hi;
                } else {
                    nu = max(0, sg.j_hi - sg.s_lo);
                    sg.tree_here = sg.with_tree;
                }
                // Lists ascend: only the last block can be one that the text ends in.
                const int last_blk = nu > 0 ? (a.idx ? sg.s_lo + (int)(ulist[nu - 1] & 0xffffu) : sg.s_lo + nu - 1) : 0;
                sg.clean = nu > 0 && nu % PER == 0 && (last_blk + 1) * BLK > sg.P ? nu / PER - 1 : nu / PER;
                sg.nu = nu;
                sg.ntile = (nu + PER - 1) / PER + (sg.tree_here ? 1 : 0);
                sg.had += sg.ntile;
            }
            __syncthreads();
            const bool last = !a.idx || sg.s_lo + kRange >= sg.j_hi;
            // block x of the stretch's list: its number in the sequence, the heads that keep it
            auto block_at = [&](int x, uint32_t &heads) -> int {
                if (!a.idx) {
                    heads = 0xffffu;
                    return sg.s_lo + x;
                }
                const uint32_t w = ulist[x];
                heads = w >> 16;
                return sg.s_lo + (int)(w & 0xffffu);
            };

            if (warp == 4) {
                // ------------------------------------ producer
                if (lane == 0 && ok) {
                    const int kv_row0 = sg.unit * a.T, ntile = sg.ntile, nu = sg.nu;
                    for (int u = 0; u < ntile && ok; ++u) {
                        const int tt = sg.tu + u, s = tt % ST;
                        const bool tree = sg.tree_here && u == ntile - 1;
                        const int nblk = tree ? (a.n + BLK - 1) / BLK : min(PER, nu - u * PER);
                        int rw[PER];                     // read together, ahead of the copies
#pragma unroll
                        for (int e = 0; e < PER; ++e) {
                            uint32_t hm;
                            rw[e] = kv_row0 + (tree ? sg.P + e * BLK : block_at(min(u * PER + e, nu - 1), hm) * BLK);
                        }
                        // (lists ascend) a tile of blocks that follow one another: one box. With every
                        // 16-key block of four 128K caches kept 344 us against 357, 6.2 TB/s.
                        const bool side_by_side = nblk == PER && rw[PER - 1] - rw[0] == (PER - 1) * BLK;
#pragma unroll
                        for (int kv = 0; kv < 2; ++kv) {
                            uint64_t *full = kv ? &full_v[s] : &full_k[s];
                            if (!mbar_wait(kv ? &empty_v[s] : &empty_k[s], ((tt / ST) & 1) ^ 1, a.err)) {
                                ok = false;
                                break;
                            }
                            mbar_arrive_expect_tx(full, (uint32_t)(nblk * BLK * D * 2));
                            unsigned char *dst = smem + (kv ? C::OFF_V : C::OFF_K) + s * C::SLOT;
                            if (PER > 1 && side_by_side) {
#pragma unroll
                                for (int hf = 0; hf < C::HALVES; ++hf)
                                    tma_load_2d(dst + hf * C::HALF, kv ? &tv1 : &tk1, full, hf * 64, rw[0]);
                                continue;
                            }
#pragma unroll
                            for (int e = 0; e < PER; ++e)
                                if (e < nblk) {
#pragma unroll
                                    for (int hf = 0; hf < C::HALVES; ++hf)
                                        tma_load_2d(dst + hf * C::HALF + e * BLK * 128, kv ? &tv : &tk, full, hf * 64,
                                                    rw[e]);
                                }
                        }
                    }
                }
            } else if (warp == 5) {
                // ------------------------------------ products
                if (lane == 0 && ok) {
                    const uint32_t t_s = tmem_slot, qb = smem_u32(smem);
                    const int ntile = sg.ntile, tu = sg.tu;
                    ok = mbar_wait(&bar_q, sg.segs & 1, a.err);
                    auto issue_s = [&](int u) -> bool {
                        const int s = u % ST;
                        if (!mbar_wait(&full_k[s], (u / ST) & 1, a.err)) return false;
                        tc_fence_after();
                        const uint32_t kb = smem_u32(smem + C::OFF_K + s * C::SLOT);
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk) {
                            const uint32_t off = (kk >> 2) * C::HALF + (kk & 3) * 32;
                            tc_mma_ss(t_s, sw128_desc(qb + off, 16, 1024), sw128_desc(kb + off, 16, 1024),
                                      C::IDESC_S, kk > 0 ? 1u : 0u);
                        }
                        tc_commit(&s_full);
                        tc_commit(&empty_k[s]);
                        return true;
                    };
                    if (ok && ntile > 0) ok = issue_s(tu);
                    for (int u = tu; u < tu + ntile && ok; ++u) {
                        const int s = u % ST;
                        ok = mbar_wait(&p_ready, u & 1, a.err) && mbar_wait(&full_v[s], (u / ST) & 1, a.err);
                        if (!ok) break;
                        tc_fence_after();
                        const uint32_t vb = smem_u32(smem + C::OFF_V + s * C::SLOT);
#pragma unroll
                        for (int kk = 0; kk < kTile / 16; ++kk)
                            tc_mma_ts(t_s + 128, t_s + kk * 8, sw128_desc(vb + kk * 2048, C::HALF, 1024), C::IDESC_O,
                                      (kk > 0 || started) ? 1u : 0u);
                        started = 1;
                        tc_commit(&empty_v[s]);
                        if (u + 1 < tu + ntile) ok = issue_s(u + 1);
                    }
                    if (last && ok) tc_commit(&o_done);
                }
            } else {
                // ------------------------------------ softmax
                const int r = tid, row = row0 + max(r - shift, 0), node = row % a.n, head = row / a.n & 15;
                const bool live = r >= shift && row < a.G * a.n &&
                                  (nmask[node][0] | nmask[node][1] | nmask[node][2] | nmask[node][3]) != 0u;
                const bool warp_live = __any_sync(0xffffffffu, live);
                const uint32_t t_s = tmem_slot + ((uint32_t)(warp * 32) << 16), t_o = t_s + 128;
                const int ntile = sg.ntile, tu = sg.tu, clean = sg.clean, kv_tiles = (sg.nu + PER - 1) / PER;
                for (int u = 0; u < ntile && ok; ++u) {
                    // in a clean tile this row's head keeps a block whole or not at all (bit e)
                    const bool tree = u >= kv_tiles, dirty = u >= clean;
                    uint32_t kept = (1u << PER) - 1u;
                    if (!dirty && a.idx) {
                        uint32_t w[PER];
                        if constexpr (PER >= 4) {
#pragma unroll
                            for (int e = 0; e < PER; e += 4)
                                *reinterpret_cast<uint4 *>(w + e) = *reinterpret_cast<const uint4 *>(ulist + u * PER + e);
                        } else {
#pragma unroll
                            for (int e = 0; e < PER; ++e) w[e] = ulist[u * PER + e];
                        }
                        kept = 0;
#pragma unroll
                        for (int e = 0; e < PER; ++e) kept |= ((w[e] >> (16 + head)) & 1u) << e;
                        if (!live) kept = (1u << PER) - 1u;         // an unused row: anything
                    }
                    // (votes: a warp gives up as one)
                    ok = __all_sync(0xffffffffu, mbar_wait(&s_full, (tu + u) & 1, a.err));
                    if (!ok) break;
                    tc_fence_after();
                    // rows of V that no key of this sequence fills (behind the text, blocks
                    // that are not there, unused nodes) are made zero: their weight is
                    // zero, but 0 x NaN is not
                    if (dirty) {
                        bool fill;
                        if (tree) {
                            fill = (nmask[r][0] | nmask[r][1] | nmask[r][2] | nmask[r][3]) == 0u;
                        } else {
                            const int k = u * PER + r / BLK;
                            uint32_t hm;
                            fill = k >= sg.nu || block_at(k, hm) * BLK + r % BLK >= sg.P;
                        }
                        const int tt = tu + u, s = tt % ST;
                        ok = __all_sync(0xffffffffu, mbar_wait(&full_v[s], (tt / ST) & 1, a.err));
                        if (!ok) break;
                        if (fill) {
                            unsigned char *vr = smem + C::OFF_V + s * C::SLOT + r * 128;
#pragma unroll
                            for (int hf = 0; hf < C::HALVES; ++hf)
#pragma unroll
                                for (int c = 0; c < 8; ++c)
                                    *reinterpret_cast<uint4 *>(vr + hf * C::HALF + c * 16) = make_uint4(0, 0, 0, 0);
                        }
                        fence_async_shared();
                    }
                    if (warp_live) {
                        float x[kTile];
#pragma unroll
                        for (int c = 0; c < kTile / 32; ++c) tmem_ld32f(t_s + c * 32, x + c * 32);
                        tc_wait_ld();
                        if (dirty) {                     // single keys: by a mask of 128 bits
                            uint32_t see[4] = {0u, 0u, 0u, 0u};
                            if (tree) {
#pragma unroll
                                for (int c = 0; c < 4; ++c) see[c] = nmask[node][c];
                            } else {
#pragma unroll
                                for (int e = 0; e < PER; ++e) {
                                    if (u * PER + e >= sg.nu) continue;
                                    uint32_t hm;
                                    const int lim = sg.P - block_at(u * PER + e, hm) * BLK;
                                    if (!((hm >> head) & 1u)) continue;
                                    if constexpr (BLK == 16) {
                                        see[e / 2] |= (lim >= 16 ? 0xffffu : (1u << max(lim, 0)) - 1u) << (e % 2 * 16);
                                    } else {
#pragma unroll
                                        for (int c = 0; c < BLK / 32; ++c) {
                                            const int k = lim - c * 32;
                                            see[e * (BLK / 32) + c] = k >= 32 ? 0xffffffffu : (1u << max(k, 0)) - 1u;
                                        }
                                    }
                                }
                            }
#pragma unroll
                            for (int c = 0; c < kTile; ++c)
                                x[c] = (see[c >> 5] >> (c & 31)) & 1u ? x[c] : -INFINITY;
                        }
                        // maxima block by block, then of the kept ones
                        float mx = -INFINITY;
#pragma unroll
                        for (int e = 0; e < PER; ++e) {
                            constexpr int CH = BLK >= 64 ? 8 : BLK / 8;      // independent chains
                            float mp[CH];
#pragma unroll
                            for (int k = 0; k < CH; ++k) mp[k] = fmaxf(x[e * BLK + k], x[e * BLK + CH + k]);
#pragma unroll
                            for (int c = 2 * CH; c < BLK; c += 2 * CH)
#pragma unroll
                                for (int k = 0; k < CH; ++k)
                                    mp[k] = fmax3(mp[k], x[e * BLK + c + k], x[e * BLK + c + CH + k]);
#pragma unroll
                            for (int k = 1; k < CH; ++k) mp[0] = fmaxf(mp[0], mp[k]);
                            mx = fmaxf(mx, (kept >> e) & 1u ? mp[0] : -INFINITY);
                        }
                        mx *= a.scale_log2;
                        float alpha = 1.f;
                        bool rescale = false;
                        if (mx > m_used + kRescaleThreshold) {
                            alpha = fast_exp2(m_used - mx);
                            rescale = l > 0.f;
                            m_used = mx;
                        }
                        // the previous P V completed before S did: O is stable
                        if (__any_sync(0xffffffffu, rescale)) {
#pragma unroll 1
                            for (int c = 0; c < D / 16; ++c) {
                                float o0[16];
                                tmem_ld16f(t_o + c * 16, o0);
                                tc_wait_ld();
                                uint32_t o1[16];
#pragma unroll
                                for (int e = 0; e < 16; ++e) o1[e] = __float_as_uint(o0[e] * alpha);
                                tmem_st16(t_o + c * 16, o1);
                            }
                        }
                        const float base = m_used == -INFINITY ? 0.f : m_used;
                        uint64_t sp[4] = {0ull, 0ull, 0ull, 0ull};
                        const uint64_t scale2 = f32x2(a.scale_log2, a.scale_log2);
#pragma unroll
                        for (int c = 0; c < kTile / 32; ++c) {
                            uint32_t w[16];
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                // a block that is not kept: exponents of -inf
                                const bool k = (kept >> ((c * 32 + 2 * e) / BLK)) & 1u;
                                const float nb = k ? -base : -INFINITY;
                                float y0, y1;
                                f32x2_split(fma_f32x2(f32x2(x[c * 32 + 2 * e], x[c * 32 + 2 * e + 1]),
                                                      scale2, f32x2(nb, nb)), y0, y1);
                                const float p0 = fast_exp2(y0), p1 = fast_exp2(y1);
                                sp[e & 3] = add_f32x2(sp[e & 3], f32x2(p0, p1));
                                w[e] = pack_bf16x2(p0, p1);     // P to bf16 (see the head of the file)
                            }
                            tmem_st16(t_s + c * 16, w);
                        }
                        float rs0, rs1;
                        f32x2_split(add_f32x2(add_f32x2(sp[0], sp[1]), add_f32x2(sp[2], sp[3])), rs0, rs1);
                        l = l * alpha + (rs0 + rs1);
                        tc_wait_st();
                    }
                    tc_fence_before();
                    mbar_arrive(&p_ready);
                }
            }
            __syncthreads();
            if (tid == 0) {
                sg.tu += sg.ntile;
            }
            if (last) break;
            if (tid == 0) sg.s_lo += kRange;
            for (int x = tid; x < kRange / 2; x += kThreads) reinterpret_cast<uint32_t *>(mark)[x] = 0u;
            __syncthreads();
        }

        // ------------------------------------------------ the segment's state
        if (warp < 4) {
            const int r = tid - shift, row = row0 + max(r, 0), node = row % a.n;
            ok = __all_sync(0xffffffffu, ok && mbar_wait(&o_done, sg.segs & 1, a.err));
            tc_fence_after();
            const bool store = r >= 0 && row < a.G * a.n, whole = sg.whole;
            if (!store || (nmask[node][0] | nmask[node][1] | nmask[node][2] | nmask[node][3]) == 0u) {
                m_used = -INFINITY;                      // an unused row: no key
                l = 0.f;
            }
            // no key: l = 0, and O may never have been written. A NaN sum is not that: it goes out
            const bool use = ok && sg.had > 0 && l != 0.f;
            const float inv = use ? 1.f / l : 0.f;
            const uint32_t t_o = tmem_slot + 128 + ((uint32_t)(warp * 32) << 16);
            const size_t orow = (size_t)sg.unit * a.G * a.n + row;
            // the state of this run and unit, this row tile: [D][128], a warp's rows side by side
            const size_t slot = ((size_t)(blockIdx.x / a.nrt) + sg.unit) * a.nrt + blockIdx.x % a.nrt;
            if (__any_sync(0xffffffffu, store)) {
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    float o[32];
                    tmem_ld32f(t_o + c, o);
                    tc_wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = use ? o[e] : 0.f;
                    if (!store) continue;
                    if (whole) {
                        uint4 *dst = reinterpret_cast<uint4 *>(a.out + orow * D + c);
#pragma unroll
                        for (int e = 0; e < 32; e += 8)
                            dst[e / 8] = make_uint4(pack_bf16x2(o[e] * inv, o[e + 1] * inv),
                                                    pack_bf16x2(o[e + 2] * inv, o[e + 3] * inv),
                                                    pack_bf16x2(o[e + 4] * inv, o[e + 5] * inv),
                                                    pack_bf16x2(o[e + 6] * inv, o[e + 7] * inv));
                    } else {
                        float *dst = a.ws_o + (slot * D + c) * 128 + r;
#pragma unroll
                        for (int e = 0; e < 32; ++e) dst[e * 128] = o[e];
                    }
                }
            }
            if (store) {
                if (whole) {
                    if (a.lse) a.lse[orow] = use ? (m_used + log2f(l)) * kLn2 : -INFINITY;
                } else {
                    reinterpret_cast<float2 *>(a.ws_ml)[slot * 128 + r] = make_float2(m_used, l);
                }
            }
            tc_fence_before();
        }
        __syncthreads();
        tc_fence_after();
    }
    // copies still in flight on a failure path land before the CTA leaves
    if (warp == 4 && lane == 0) {
        if (sg.segs >= 0) mbar_drain(&bar_q, sg.segs & 1);
        if (!ok) {
            drain_ring<ST>(full_k, sg.tu);
            drain_ring<ST>(full_v, sg.tu);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 5) {
        tc_fence_after();
        tmem_dealloc(tmem_slot, 256);
    }
}

// Joins the states of the units that lie in several runs. A CTA has 32 rows of a unit, one
// per lane, and 32 features, four per warp.
constexpr int kJoinWarps = 8, kJoinCols = 4;
template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32) tree_join_kernel(const __grid_constant__ TreeArgs a) {
    const int lane = threadIdx.x & 31, c_lo = (blockIdx.y * kJoinWarps + (threadIdx.x >> 5)) * kJoinCols;
    const int unit = blockIdx.x / (a.nrt * 4), rt = blockIdx.x / 4 % a.nrt, srow = blockIdx.x % 4 * 32 + lane;
    const int b = unit / a.Hkv, row = rt * 128 + srow;
    grid_wait();
    const int chunk = run_chunk(a, run_total(a)), tb = tiles_of(a, b);
    int before = b * tb;
    if (a.lens) {
        before = 0;
        for (int x = lane; x < b; x += 32) before += tiles_of(a, x);
        before = __reduce_add_sync(0xffffffffu, before);
    }
    if (row >= a.G * a.n) return;
    const int p0 = before * a.Hkv + (unit - b * a.Hkv) * tb;
    const int c0 = p0 / chunk, ns = (p0 + tb - 1) / chunk - c0 + 1;
    if (ns == 1) return;                        // written by its run
    const size_t slot0 = ((size_t)c0 + unit) * a.nrt + rt, step = a.nrt;   // a run further: nrt slots
    const float2 *ml = reinterpret_cast<const float2 *>(a.ws_ml) + slot0 * 128 + srow;
    const float *src = a.ws_o + (slot0 * D + c_lo) * 128 + srow;
    // online over the runs, four at a time
    float M = -INFINITY, L = 0.f, o[kJoinCols] = {0.f, 0.f, 0.f, 0.f};
    for (int s0 = 0; s0 < ns; s0 += 4) {
        float2 st[4];
        float v[4][kJoinCols];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const bool in = s0 + k < ns;                 // no run there: an empty state
            const size_t at = in ? (s0 + k) * step : 0;
            st[k] = ml[at * 128];
#pragma unroll
            for (int e = 0; e < kJoinCols; ++e) v[k][e] = src[(at * D + e) * 128];
            if (in) continue;
            st[k] = make_float2(-INFINITY, 0.f);
#pragma unroll
            for (int e = 0; e < kJoinCols; ++e) v[k][e] = 0.f;
        }
        const float mn = fmaxf(fmaxf(M, fmaxf(st[0].x, st[1].x)), fmaxf(st[2].x, st[3].x));
        const float mb = mn == -INFINITY ? 0.f : mn, f = fast_exp2(M - mb);
        L *= f;
#pragma unroll
        for (int e = 0; e < kJoinCols; ++e) o[e] *= f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float g = fast_exp2(st[k].x - mb);
            L += st[k].y * g;
#pragma unroll
            for (int e = 0; e < kJoinCols; ++e) o[e] += v[k][e] * g;
        }
        M = mn;
    }
    const float inv = L != 0.f ? 1.f / L : 0.f;          // 0: a row without a key; NaN goes out
    const size_t orow = (size_t)unit * a.G * a.n + row;
    *reinterpret_cast<uint2 *>(a.out + orow * D + c_lo) =
        make_uint2(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv));
    if (a.lse && c_lo == 0) a.lse[orow] = L != 0.f ? (M + log2f(L)) * kLn2 : -INFINITY;
}

bool make_map(CUtensorMap *map, const void *base, uint64_t rows, int d, int box_rows) {
    EncodeTiledFn enc = encode_tiled_fn();
    if (!enc) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)d, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)d * 2};
    const cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
    const cuuint32_t estr[2] = {1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims, strides,
               box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int BLK>
cudaError_t launch_cfg(const TreeCall &c, TreeArgs a, cudaStream_t s) {
    using C = Cfg<D, BLK>;
    CUtensorMap mq, mk, mv, mk1, mv1;             // mk1, mv1: boxes of a whole tile
    const uint64_t kv_rows = (uint64_t)c.B * c.Hkv * c.T;
    if (!make_map(&mq, c.q, (uint64_t)c.B * c.Hq * c.n, D, 128) || !make_map(&mk, c.kc, kv_rows, D, BLK) ||
        !make_map(&mv, c.vc, kv_rows, D, BLK))
        return cudaErrorNotSupported;
    if (C::PER > 1 && (!make_map(&mk1, c.kc, kv_rows, D, kTile) || !make_map(&mv1, c.vc, kv_rows, D, kTile)))
        return cudaErrorNotSupported;
    cudaError_t e = allow_smem<tree_kernel<D, BLK>>(C::SMEM);
    if (e != cudaSuccess) return e;
    // no more runs than tiles (the most that the lengths allow)
    const long long most = (long long)c.B * c.Hkv * ((c.T - c.n + kTile - 1) / kTile + 1);
    void *args[] = {&mq, &mk, &mv, &mk1, &mv1, &a};
    e = launch_early(reinterpret_cast<const void *>(tree_kernel<D, BLK>),
                     dim3((unsigned)((most < a.runs ? most : a.runs) * a.nrt)), dim3(kThreads), C::SMEM, args, s);
    if (e != cudaSuccess) return e;
    void *jargs[] = {&a};
    return launch_early(reinterpret_cast<const void *>(tree_join_kernel<D>),
                        dim3((unsigned)(c.B * c.Hkv * a.nrt * 4), D / (kJoinWarps * kJoinCols)), dim3(kJoinWarps * 32),
                        0, jargs, s);
}

template <int D>
cudaError_t launch_d(const TreeCall &c, const TreeArgs &a, cudaStream_t s) {
    // without lists the keys are read 128 at a time, whatever the block
    switch (c.idx ? c.block : kTile) {
        case 16: return launch_cfg<D, 16>(c, a, s);
        case 32: return launch_cfg<D, 32>(c, a, s);
        case 64: return launch_cfg<D, 64>(c, a, s);
        default: return launch_cfg<D, 128>(c, a, s);
    }
}

// Row tiles per (b, kv-head), and the runs that leaves.
int row_tiles(int G, int n) { return (G * n + 127) / 128; }
int runs_of(int nrt) { return kCtas / nrt; }
size_t state_rows(int B, int Hq, int Hkv, int n) {
    const int nrt = row_tiles(Hq / Hkv, n);
    return ((size_t)runs_of(nrt) + (size_t)B * Hkv) * nrt * 128;
}

}  // namespace

// One state per run and unit it touches: (O, m, l) of its rows.
size_t tree_workspace_bytes(int B, int Hq, int Hkv, int n, int, int d, int) {
    return state_rows(B, Hq, Hkv, n) * (size_t)(d + 2) * sizeof(float);
}

cudaError_t launch_tree(const TreeCall &c, cudaStream_t s) {
    TreeArgs a;
    a.parents = c.parents; a.lens = c.lens; a.idx = c.idx; a.count = c.count;
    a.out = static_cast<__nv_bfloat16 *>(c.out);
    a.lse = c.lse;
    a.ws_o = static_cast<float *>(c.workspace);
    a.ws_ml = a.ws_o + state_rows(c.B, c.Hq, c.Hkv, c.n) * c.d;
    a.B = c.B; a.Hq = c.Hq; a.Hkv = c.Hkv; a.G = c.Hq / c.Hkv; a.n = c.n; a.T = c.T; a.cap = c.cap;
    a.nrt = row_tiles(a.G, a.n);
    a.runs = runs_of(a.nrt);
    a.scale_log2 = c.scale * kLog2e;
    a.err = c.err;
    return c.d == 64 ? launch_d<64>(c, a, s) : launch_d<128>(c, a, s);
}

}  // namespace spa
