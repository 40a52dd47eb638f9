// Attention of a tree of drafted tokens over the kept blocks of a KV cache (bf16).
// One CTA per (b, query head, node), 128 keys at a time with the online softmax.
#include <math.h>

#include "serve.h"

namespace spa {
namespace {

template <int D>
__global__ void __launch_bounds__(128) tree_kernel(TreeCall a) {
    const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(a.q);
    const __nv_bfloat16 *kc = static_cast<const __nv_bfloat16 *>(a.kc);
    const __nv_bfloat16 *vc = static_cast<const __nv_bfloat16 *>(a.vc);
    __shared__ float qs[D], ps[128], red[4];
    __shared__ int key_s[128];
    const int i = blockIdx.x, h = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
    const int g = h / (a.Hq / a.Hkv);
    const size_t row = ((size_t)b * a.Hq + h) * a.n + i;
    const int32_t *par = a.parents + (size_t)b * a.n;
    if (tid < D) qs[tid] = __bfloat162float(q[row * D + tid]);
    int P = a.lens ? a.lens[b] : a.T - a.n;
    if (P < 0 || P > a.T - a.n) {
        set_error(a.err, SPA_DEVERR_BAD_COUNT);
        P = P < 0 ? 0 : a.T - a.n;
    }
    bool used = true;
    for (int j = i; j >= 0 && used;) {
        const int p = par[j];
        if (p >= j) set_error(a.err, SPA_DEVERR_BAD_INDEX);
        if (p >= j || p < -1) used = false;
        j = p;
    }
    const size_t base = ((size_t)b * a.Hkv + g) * a.T;
    float m = -INFINITY, l = 0.f, o = 0.f;
    auto fold = [&](int key) {          // one key per thread, -1: none
        __syncthreads();
        key_s[tid] = key;
        float x = -INFINITY;
        if (key >= 0) {
            float dot = 0.f;
            for (int c = 0; c < D; ++c) dot = fmaf(qs[c], __bfloat162float(kc[(base + key) * D + c]), dot);
            x = dot * a.scale;
        }
        float mx = x;
        for (int k = 16; k; k >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, k));
        if (!(tid & 31)) red[tid >> 5] = mx;
        __syncthreads();
        mx = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
        const float mn = fmaxf(m, mx);
        const float f = mn == -INFINITY ? 1.f : expf(m - mn);
        ps[tid] = key >= 0 ? expf(x - mn) : 0.f;
        __syncthreads();
        l *= f;
        o *= f;
        for (int u = 0; u < 128; ++u)
            if (key_s[u] >= 0) {
                l += ps[u];
                if (tid < D) o = fmaf(ps[u], __bfloat162float(vc[(base + key_s[u]) * D + tid]), o);
            }
        m = mn;
    };
    if (used) {
        const int nb = (a.T + a.block - 1) / a.block;
        const int per = 128 / a.block;
        const size_t unit = (size_t)b * a.Hq + h;
        int cnt = a.idx ? a.count[unit] : nb;
        if (cnt < 0 || (a.idx && cnt > a.cap)) {
            set_error(a.err, SPA_DEVERR_BAD_COUNT);
            cnt = cnt < 0 ? 0 : a.cap;
        }
        for (int e0 = 0; e0 < cnt; e0 += per) {
            const int e = e0 + tid / a.block;
            int j = -1;
            if (e < cnt) {
                j = a.idx ? a.idx[unit * a.cap + e] : e;
                if (j < 0 || j >= nb || (a.idx && e > 0 && a.idx[unit * a.cap + e - 1] >= j)) {
                    set_error(a.err, SPA_DEVERR_BAD_INDEX);
                    j = -1;
                }
            }
            const int key = j * a.block + tid % a.block;
            fold(j >= 0 && key < P ? key : -1);
        }
        bool see = false;
        for (int j = i; j >= 0; j = par[j]) see = see || j == tid;
        fold(see ? P + tid : -1);
    }
    if (tid < D)
        static_cast<__nv_bfloat16 *>(a.out)[row * D + tid] = __float2bfloat16_rn(l > 0.f ? o / l : 0.f);
    if (a.lse && tid == 0) a.lse[row] = l > 0.f ? m + logf(l) : -INFINITY;
}

}  // namespace

size_t tree_workspace_bytes(int, int, int, int, int, int, int) { return 16; }

cudaError_t launch_tree(const TreeCall &c, cudaStream_t s) {
    const dim3 grid((unsigned)c.n, (unsigned)c.Hq, (unsigned)c.B);
    if (c.d == 64)
        tree_kernel<64><<<grid, 128, 0, s>>>(c);
    else
        tree_kernel<128><<<grid, 128, 0, s>>>(c);
    return cudaGetLastError();
}

}  // namespace spa
