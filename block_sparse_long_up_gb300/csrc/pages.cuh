// pages.cuh -- what the kernels that keep the cache's books share: one cluster of blocks whose
// warps take equal runs of the work in order, and the scan over them.
#pragma once

#include "paged.cuh"

namespace up {

struct PagePool {
    int32_t *refs;  // sequences that hold each page
    int32_t *free;  // the free pages, a stack
    int32_t *num_free;
    int num_pages;
    unsigned int *err;
};

struct PageTable {
    int32_t *entries;  // [num_seqs][max_pages]
    int num_seqs, max_pages, page_size;
};

struct ForkArgs {
    PagePool pool;
    PageTable from;
    const int32_t *kv_lens, *parents;
    int children;
    int32_t *table, *lens, *copies;  // copies: [3][children]
};

struct KvCompactArgs {
    PagedKv kv;
    const int32_t *cu_seqlens, *cu_blocks;
    const uint8_t *keep;
    int32_t *lens_out;
    void *workspace;
    int64_t num_flags;
    int T, G;  // T: the most tokens that cu_seqlens may end at
    long long wait_limit;
};

cudaError_t launch_reserve(const PagePool &pool, const PageTable &t, const int32_t *have, const int32_t *want,
                           cudaStream_t st);
cudaError_t launch_release(const PagePool &pool, const PageTable &t, const int32_t *first, const int32_t *end,
                           cudaStream_t st);
cudaError_t launch_fork(const ForkArgs &a, cudaStream_t st);
int64_t copy_blocks(const PagedKv &kv, int n);  // 2^31 - 1 at most
cudaError_t launch_copy_pages(const PagedKv &kv, const int32_t *copies, int n, cudaStream_t st);
size_t kv_compact_workspace(int64_t T, int num_seqs, int Hk, int d);
cudaError_t launch_kv_compact(const KvCompactArgs &a, int num_sms, cudaStream_t st);

namespace books {

constexpr int kBlocks = 8;  // of the cluster
constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kAllWarps = kBlocks * kWarps;

__device__ __forceinline__ int cluster_warp() { return blockIdx.x * kWarps + (threadIdx.x >> 5); }

// All threads of the cluster meet; what each wrote before is there for all (released and acquired at
// the cluster's scope, and read through L2: __ldcg).
__device__ __forceinline__ void arrive() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void await_all() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void meet() {
    arrive();
    await_all();
}

// Shared memory of another block of the cluster.
__device__ __forceinline__ int read_other(const int *mine, int block) {
    uint32_t at = (uint32_t)__cvta_generic_to_shared(mine), there;
    int v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(at), "r"(block));
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(there) : "memory");
    return v;
}

__device__ __forceinline__ void write_other(int *mine, int block, int v) {
    uint32_t at = (uint32_t)__cvta_generic_to_shared(mine), there;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(at), "r"(block));
    asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(there), "r"(v) : "memory");
}

// Sum of `mine` (a warp's) over the warps before this one in the cluster; *total over all.  Every thread
// of the cluster comes here once, with its warp's value, and meets the others again before it
// leaves: nobody may while another block reads its sum.
__device__ __forceinline__ int before_warp(int mine, int *total) {
    __shared__ int s_warp[kWarps], s_block;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) s_warp[warp] = mine;
    __syncthreads();
    int inc = s_warp[lane];  // one value a lane: kWarps is 32
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, inc, k);
        if (lane >= k) inc += y;
    }
    const int own = warp ? __shfl_sync(0xffffffffu, inc, warp - 1) : 0;
    if (threadIdx.x == 31) s_block = inc;
    meet();
    int before = 0, all = 0;
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) {
        const int v = read_other(&s_block, b);
        if (b < (int)blockIdx.x) before += v;
        all += v;
    }
    *total = all;
    return before + own;
}
static_assert(kWarps == 32, "one warp's lanes scan the block");

}  // namespace books

}  // namespace up
