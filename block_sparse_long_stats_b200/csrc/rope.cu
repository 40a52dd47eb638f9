// Rotary positions: q, k (and, appending to a cache, v) of one call in one launch.
//
//   y1 = m (x1 cos a - x2 sin a),  y2 = m (x2 cos a + x1 sin a),  a = pos * freq[c]
//
// Bound by HBM: every element is read and written once, with 3 flops per pair
// feature. What could cost more is the angles: pos * freq reaches 1e5 radians and
// more, where an fp32 product is off by a hundredth of a radian, so the turn number
// pos * freq / 2 pi is taken and reduced in fp64 and only the fraction goes to the fp32
// sincospi. A thread therefore owns V pairs of one token (two 16-byte accesses a head)
// and walks over up to 16 heads with one set of sines: the 8 fp64 reductions are spent
// once per token and group of heads, three times for 32 + 8 heads and once per head only
// where there are too few tokens to fill the GPU. Two heads' loads at a time in 64 registers (eight
// CTAs per SM) rotate a 32K prompt of 32 + 8 heads in 127 us (5.3 TB/s, 80 % of the measured
// copy bandwidth); four at a time in 128 registers took 178 us.
#include <math.h>

#include "serve.h"

namespace spa {
namespace {

constexpr int kThreads = 128;
constexpr int kBatch = 2;        // heads whose loads are in flight together

struct RopeArgs {
    const void *x[3];
    void *y[3];
    spa_strides xs[3], ys[3];
    int h_end[3];                // heads of q, q + k, q + k + v
    long long tokens;
    int L, d, rot, T, heads_per_thread, units_rot, units;
    int pos0;
    float mscale, sign;
    bool append;
    const int32_t *pos, *rows;
    int *err;
    double turns[kRopeMaxPairs]; // turns per position of each pair
};

template <typename T>
__device__ __forceinline__ float to_f(T x);
template <>
__device__ __forceinline__ float to_f<float>(float x) { return x; }
template <>
__device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ float from_f<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// V elements moved with one access (V * sizeof(T) is 16, 8 or one element's size).
template <typename T, int V>
struct alignas(V * sizeof(T)) Vec {
    T e[V];
};

// A unit is 2 V features of a head: V pairs (features c.. and c + rot/2.. of the half
// layout, 2 V consecutive ones of the interleaved), or 2 V consecutive features
// behind the rotated part, which are copied.
template <typename T, int V, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads, 8) rope_kernel(const __grid_constant__ RopeArgs a) {
    grid_wait();
    const long long id = (long long)blockIdx.x * kThreads + threadIdx.x;
    const long long tok = id / a.units;
    if (tok >= a.tokens) return;
    const int u = (int)(id - tok * a.units);
    const long long b = tok / a.L;
    const int t = (int)(tok - b * a.L);

    int row = t;                          // row of the k and v outputs
    bool store_kv = true;
    int p = a.pos0 + t;
    if (a.append) {
        const long long r = (a.rows ? (long long)a.rows[b] : (long long)a.pos0) + t;
        store_kv = r >= 0 && r < a.T;
        if (!store_kv && u == 0 && blockIdx.y == 0) set_error(a.err, SPA_DEVERR_BAD_INDEX);
        row = (int)r;
        p = (int)r;
    }
    if (a.pos) p = a.pos[b * a.L + t];

    const bool turn = u < a.units_rot;
    int o1, o2;                           // feature offsets of the unit's two vectors
    if (turn) {
        o1 = INTERLEAVED ? u * 2 * V : u * V;
        o2 = INTERLEAVED ? o1 + V : o1 + a.rot / 2;
    } else {
        o1 = a.rot + (u - a.units_rot) * 2 * V;
        o2 = o1 + V;
    }
    const bool has2 = o2 < a.d;           // the copied tail may end in half a unit
    float cs[V], sn[V];
    if (turn) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const double n = (double)p * a.turns[u * V + e];
            float s, c;
            sincospif(2.f * (float)(n - rint(n)), &s, &c);
            cs[e] = c * a.mscale;
            sn[e] = s * a.sign;           // mscale, negative for the gradient
        }
    }
    const int h_lo = blockIdx.y * a.heads_per_thread;
    const int h_hi = min(a.h_end[2], h_lo + a.heads_per_thread);
    for (int h0 = h_lo; h0 < h_hi; h0 += kBatch) {
        Vec<T, V> v1[kBatch], v2[kBatch];
        T *dst[kBatch];
        bool rot_h[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int h = h0 + k;
            dst[k] = nullptr;
            if (h >= h_hi) continue;
            const int w = h < a.h_end[0] ? 0 : (h < a.h_end[1] ? 1 : 2);
            const int hl = h - (w == 0 ? 0 : a.h_end[w - 1]);
            if (w > 0 && !store_kv) continue;
            const T *src = static_cast<const T *>(a.x[w]) + b * a.xs[w].b + hl * a.xs[w].h + t * a.xs[w].l;
            dst[k] = static_cast<T *>(a.y[w]) + b * a.ys[w].b + hl * a.ys[w].h +
                     (w == 0 ? t : row) * a.ys[w].l;
            rot_h[k] = turn && w < 2;
            v1[k] = *reinterpret_cast<const Vec<T, V> *>(src + o1);
            if (has2) v2[k] = *reinterpret_cast<const Vec<T, V> *>(src + o2);
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            if (!dst[k]) continue;
            if (rot_h[k]) {
                Vec<T, V> y1, y2;
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    if constexpr (INTERLEAVED && V > 1) {
                        // pair e is features 2e, 2e + 1 of the 2 V
                        const float x1 = to_f((2 * e < V ? v1[k] : v2[k]).e[(2 * e) % V]);
                        const float x2 = to_f((2 * e + 1 < V ? v1[k] : v2[k]).e[(2 * e + 1) % V]);
                        (2 * e < V ? y1 : y2).e[(2 * e) % V] = from_f<T>(x1 * cs[e] - x2 * sn[e]);
                        (2 * e + 1 < V ? y1 : y2).e[(2 * e + 1) % V] = from_f<T>(x2 * cs[e] + x1 * sn[e]);
                    } else {
                        const float x1 = to_f(v1[k].e[e]), x2 = to_f(v2[k].e[e]);
                        y1.e[e] = from_f<T>(x1 * cs[e] - x2 * sn[e]);
                        y2.e[e] = from_f<T>(x2 * cs[e] + x1 * sn[e]);
                    }
                }
                v1[k] = y1;
                v2[k] = y2;
            }
            *reinterpret_cast<Vec<T, V> *>(dst[k] + o1) = v1[k];
            if (has2) *reinterpret_cast<Vec<T, V> *>(dst[k] + o2) = v2[k];
        }
    }
}

// Whether accesses of V elements are aligned in every tensor, and the rotated part
// and the copied one are whole numbers of them.
bool takes(const RopeCall &c, int V) {
    const int size = c.bf16 ? 2 : 4;
    if ((c.interleaved ? c.rot % (2 * V) : (c.rot / 2) % V) || c.d % V) return false;
    for (const RopeTensor &t : c.t) {
        if (!t.H) continue;
        const uintptr_t base = reinterpret_cast<uintptr_t>(t.x) | reinterpret_cast<uintptr_t>(t.y);
        const int64_t str = t.xs.b | t.xs.h | t.xs.l | t.ys.b | t.ys.h | t.ys.l;   // low bits: divisibility
        if (base % (uintptr_t)(V * size) || str % V) return false;
    }
    return true;
}

template <typename T, int V>
cudaError_t launch_v(const RopeCall &c, RopeArgs &a, cudaStream_t s) {
    a.units_rot = c.rot / 2 / V;
    a.units = a.units_rot + (c.d - c.rot + 2 * V - 1) / (2 * V);
    const long long threads = a.tokens * a.units;
    // heads per thread: enough threads to fill the GPU (148 SMs x 2048) come before
    // sharing the sines between heads; at most 16, so that the loads of a token stay near one another in time
    const int heads = a.h_end[2];
    long long split = (148ll * 2048 + threads - 1) / threads;
    if (split > heads) split = heads;
    int per = (int)((heads + split - 1) / split);
    if (per > 16) per = 16;
    a.heads_per_thread = per;
    const dim3 grid((unsigned)((threads + kThreads - 1) / kThreads), (unsigned)((heads + per - 1) / per));
    void *args[] = {&a};
    return launch_early(c.interleaved ? reinterpret_cast<const void *>(rope_kernel<T, V, true>)
                                      : reinterpret_cast<const void *>(rope_kernel<T, V, false>),
                        grid, dim3(kThreads), 0, args, s);
}

}  // namespace

cudaError_t launch_rope(const RopeCall &c, cudaStream_t s) {
    RopeArgs a;
    int heads = 0;
    for (int w = 0; w < 3; ++w) {
        a.x[w] = c.t[w].x;
        a.y[w] = c.t[w].y;
        a.xs[w] = c.t[w].xs;
        a.ys[w] = c.t[w].ys;
        heads += c.t[w].H;
        a.h_end[w] = heads;
    }
    a.tokens = (long long)c.B * c.L;
    a.L = c.L; a.d = c.d; a.rot = c.rot; a.T = c.T;
    a.pos0 = c.pos0;
    a.mscale = c.mscale;
    a.sign = c.backward ? -c.mscale : c.mscale;
    a.append = c.append;
    a.pos = c.pos;
    a.rows = c.rows;
    a.err = c.err;
    constexpr double kTwoPi = 6.283185307179586476925286766559;
    for (int i = 0; i < c.rot / 2; ++i) a.turns[i] = c.freqs[i] / kTwoPi;
    if (c.bf16) {
        if (takes(c, 8)) return launch_v<__nv_bfloat16, 8>(c, a, s);
        if (takes(c, 4)) return launch_v<__nv_bfloat16, 4>(c, a, s);
        return launch_v<__nv_bfloat16, 1>(c, a, s);
    }
    if (takes(c, 4)) return launch_v<float, 4>(c, a, s);
    return launch_v<float, 1>(c, a, s);
}

}  // namespace spa
