// Attention weight that every cached key receives, summed over queries and the query
// heads of its kv-head. One thread per key.
#include <math.h>

#include "serve.h"

namespace spa {
namespace {

template <int D>
__global__ void __launch_bounds__(128) weight_kernel(WeightCall a) {
    const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(a.q);
    const __nv_bfloat16 *k = static_cast<const __nv_bfloat16 *>(a.k);
    const int t = blockIdx.x * 128 + threadIdx.x, bg = blockIdx.y;
    if (t >= a.T) return;
    const int b = bg / a.Hkv, g = bg % a.Hkv, G = a.Hq / a.Hkv;
    int len = a.lens ? a.lens[b] : a.T;
    if (len < a.Lq || len > a.T) {
        set_error(a.err, SPA_DEVERR_BAD_COUNT);
        len = len < a.Lq ? a.Lq : a.T;
    }
    const __nv_bfloat16 *kr = k + ((size_t)bg * a.T + t) * D;
    const int q0 = (len - a.Lq) / a.block, nq = (len - 1) / a.block - q0 + 1;
    float sum = 0.f;
    for (int h = g * G; h < g * G + G && t < len; ++h)
        for (int qb = 0; qb < nq; ++qb) {
            const size_t unit = ((size_t)b * a.Hq + h) * nq + qb;
            bool kept = true;
            if (a.idx) {
                int cnt = a.count[unit], last = -1;
                if (cnt < 0 || cnt > a.cap) {
                    set_error(a.err, SPA_DEVERR_BAD_COUNT);
                    cnt = cnt < 0 ? 0 : a.cap;
                }
                kept = false;
                for (int e = 0; e < cnt; ++e) {
                    const int j = a.idx[unit * a.cap + e];
                    if (j <= last || j > (a.T - 1) / a.block) {
                        set_error(a.err, SPA_DEVERR_BAD_INDEX);
                        continue;
                    }
                    last = j;
                    kept = kept || j == t / a.block;
                }
            }
            if (!kept) continue;
            const int i_lo = max(max((q0 + qb) * a.block, len - a.Lq), t) - (len - a.Lq);
            const int i_hi = min((q0 + qb + 1) * a.block, len) - (len - a.Lq);
            for (int i = i_lo; i < i_hi; ++i) {
                const size_t row = ((size_t)b * a.Hq + h) * a.Lq + i;
                const float ls = a.lse[row];
                float dot = 0.f;
                for (int c = 0; c < D; ++c)
                    dot = fmaf(__bfloat162float(q[row * D + c]), __bfloat162float(kr[c]), dot);
                if (ls != -INFINITY) sum += expf(dot * a.scale - ls);
            }
        }
    const size_t o = (size_t)bg * a.T + t;
    a.out[o] = a.prev ? fmaf(a.decay, a.prev[o], sum) : sum;
}

}  // namespace

size_t weight_workspace_bytes(int, int, int, int, int) { return 16; }

cudaError_t launch_weight(const WeightCall &c, cudaStream_t s) {
    const dim3 grid((unsigned)((c.T + 127) / 128), (unsigned)(c.B * c.Hkv));
    if (c.d == 64)
        weight_kernel<64><<<grid, 128, 0, s>>>(c);
    else
        weight_kernel<128><<<grid, 128, 0, s>>>(c);
    return cudaGetLastError();
}

}  // namespace spa
