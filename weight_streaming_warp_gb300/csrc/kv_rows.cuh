// kv_rows.cuh -- what the kernels over block tables share: pages of a length, a block's saturating
// scan, and launches of one cluster.
#pragma once

#include "cluster_choice.h"
#include "common.cuh"

namespace wsw {

// pages of `len` < 2^31 positions
__device__ __forceinline__ int pages_of(int len, int shift) {
    return static_cast<int>((static_cast<unsigned>(len) + (1u << shift) - 1) >> shift);
}

// a + b, at most cap < 2^31 (a, b <= cap)
__device__ __forceinline__ int add_sat(int a, int b, int cap) {
    const unsigned s = static_cast<unsigned>(a) + static_cast<unsigned>(b);
    return s < static_cast<unsigned>(cap) ? static_cast<int>(s) : cap;
}

// Exclusive saturating prefix of v <= cap over the block's threads, and the block's total.
// Every thread calls it; sm holds 33 values.
__device__ __forceinline__ int block_scan(int v, int cap, int *sm, int *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    int x = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(WSW_FULL_MASK, x, d);
        if (lane >= d) x = add_sat(x, y, cap);
    }
    if (lane == 31) sm[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int w = lane < warps ? sm[lane] : 0;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(WSW_FULL_MASK, w, d);
            if (lane >= d) w = add_sat(w, y, cap);
        }
        sm[lane + 1] = w;
        if (lane == 0) sm[0] = 0;
    }
    __syncthreads();
    *total = sm[32];
    const int x_before = __shfl_up_sync(WSW_FULL_MASK, x, 1);
    const int before = add_sat(sm[warp], lane ? x_before : 0, cap);
    __syncthreads();  // sm may be reused
    return before;
}

// The barrier of a cluster; within it, what a thread wrote to global memory before is seen after.
__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
}

// ------------------------------------------------------------------- host --

// Sets the options of a kernel that runs as one cluster on the current device, once, and says how
// many CTAs that cluster can have; `choice` is the kernel's own.
inline cudaError_t cluster_ctas(ClusterChoice &choice, const void *kernel, int threads, int max_smem, int device,
                                unsigned *ctas) {
    const cudaError_t e = ensure_smem(kernel, max_smem);
    if (e != cudaSuccess) return e;
    *ctas = choice.of(device, [kernel, threads, max_smem] {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess) {
            cudaGetLastError();
            return false;
        }
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = 16;
        attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        cfg.gridDim = dim3(16);
        cfg.blockDim = dim3(threads);
        cfg.dynamicSmemBytes = max_smem;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        int clusters = 0;
        if (cudaOccupancyMaxActiveClusters(&clusters, kernel, &cfg) != cudaSuccess) {
            cudaGetLastError();
            return false;
        }
        return clusters > 0;
    });
    return cudaSuccess;
}

// Launches `ctas` CTAs in clusters of `cluster`.
template <typename A>
cudaError_t launch_cluster(void (*kernel)(A), unsigned ctas, unsigned cluster, unsigned threads, size_t smem,
                           cudaStream_t stream, bool pdl, const A &a) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.numAttrs = 1;
    if (pdl) {
        attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[1].val.programmaticStreamSerializationAllowed = 1;
        cfg.numAttrs = 2;
    }
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

// Whether [a, a + an) and [b, b + bn) have a byte in common.
inline bool overlap(const void *a, int64_t an, const void *b, int64_t bn) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return an > 0 && bn > 0 && x < y + static_cast<uintptr_t>(bn) && y < x + static_cast<uintptr_t>(an);
}

}  // namespace wsw
