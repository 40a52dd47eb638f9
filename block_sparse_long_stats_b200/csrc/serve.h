// Launchers of the serving kernels: rotary positions, tree attention, accumulated
// attention weight, eviction. Arguments are validated in serve_api.cu before any of
// these is called.
#pragma once

#include <atomic>

#include "kernels.h"

namespace spa {

// Programmatic dependent launch: a kernel launched by launch_early may start while the
// one before it on the stream still runs (its launch and set-up are hidden), and calls
// grid_wait before it touches global memory or takes tensor memory: from there on
// everything before it is done.
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

inline cudaError_t launch_early(const void *kern, dim3 grid, dim3 block, size_t smem, void **args, cudaStream_t s,
                                unsigned cluster = 1) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = cluster;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelExC(&cfg, kern, args);
}

// 16 consecutive TMEM columns of this thread's lane.
__device__ __forceinline__ void tmem_ld16f(uint32_t taddr, float *x) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]), "=f"(x[6]), "=f"(x[7]),
          "=f"(x[8]), "=f"(x[9]), "=f"(x[10]), "=f"(x[11]), "=f"(x[12]), "=f"(x[13]), "=f"(x[14]), "=f"(x[15])
        : "r"(taddr));
}

// Lets a kernel use `bytes` of dynamic shared memory: set once per kernel and device (one
// Kern per call site's template arguments keeps the devices that have it).
template <auto Kern>
cudaError_t allow_smem(size_t bytes) {
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 64 && (done.load(std::memory_order_relaxed) >> dev) & 1u) return cudaSuccess;
    e = cudaFuncSetAttribute(Kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess && dev < 64) done.fetch_or(1ull << dev, std::memory_order_relaxed);
    return e;
}

constexpr int kRopeMaxPairs = 128;

struct RopeTensor {
    const void *x = nullptr;
    void *y = nullptr;
    spa_strides xs{0, 0, 0}, ys{0, 0, 0};
    int H = 0;
};

// q, k and (append) v of one call; v's rows are copied, not rotated.
struct RopeCall {
    RopeTensor t[3];
    bool bf16 = true;
    int B = 0, L = 0, d = 0, rot = 0;
    bool interleaved = false, backward = false, append = false;
    int T = 0;                          // append: rows of the caches
    const double *freqs = nullptr;      // host
    float mscale = 1.f;
    const int32_t *pos = nullptr, *rows = nullptr;
    int pos0 = 0;                       // append without rows: the first cache row
    int *err = nullptr;
};
cudaError_t launch_rope(const RopeCall &c, cudaStream_t s);

struct TreeCall {
    const void *q, *kc, *vc;
    int B, Hq, Hkv, n, T, d, block, cap;
    const int32_t *parents, *lens, *idx, *count;
    float scale;
    void *workspace, *out;
    float *lse;
    int *err;
};
size_t tree_workspace_bytes(int B, int Hq, int Hkv, int n, int T, int d, int block);
cudaError_t launch_tree(const TreeCall &c, cudaStream_t s);

struct WeightCall {
    const void *q, *k;
    int B, Hq, Hkv, Lq, T, d, block, cap;
    const float *lse;
    const int32_t *lens, *idx, *count;
    float scale, decay;
    const float *prev;
    void *workspace;
    float *out;
    int *err;
};
// Blocks of a list: the grid of the kernel that marks them has a row per 512.
constexpr int kMaxMarkBlocks = 65534 * 512;
size_t weight_workspace_bytes(int B, int Hkv, int Lq, int T, int block);
cudaError_t launch_weight(const WeightCall &c, cudaStream_t s);

cudaError_t launch_evict_select(const float *score, const int32_t *lens, int B, int Hkv, int T,
                                int n_keep, int n_sink, int n_recent, int32_t *keep,
                                int32_t *count, int *err, cudaStream_t s);
cudaError_t launch_cache_gather(const void *kc, const void *vc, const float *score, int B, int Hkv,
                                int T, int row_bytes, const int32_t *keep, int n_keep,
                                const int32_t *count, int T_out, void *k_out, void *v_out,
                                float *score_out, int *err, cudaStream_t s);

}  // namespace spa
