// What the kernels over packed rows and the paged cache share: a sequence's rows in cu_seqlens and the
// place of a slot.
#pragma once

#include "common.cuh"
#include "kernels.h"

namespace blk {

constexpr int kStatusInvalidArg = 1;  // == BLK_ERR_INVALID_ARG
constexpr int kStatusCacheFull = 4;   // == BLK_ERR_CACHE_FULL
constexpr int kMaxNodes = 64;         // rows of a sequence that parents can order into a tree

__device__ __forceinline__ void record(DevStatus* st, int code) {
  if (st) atomicCAS(&st->code, 0, code);
}

// Rows [lo, lo + n) of sequence b: cu[b] .. cu[b + 1], clamped to [0, rows]; cu null: row b alone.
struct SeqRows {
  int lo, n;
};
__device__ __forceinline__ SeqRows seq_rows(const int* cu, int b, int rows) {
  if (!cu) return {b, 1};
  const int lo = min(max(cu[b], 0), rows), hi = min(max(cu[b + 1], 0), rows);
  return {lo, max(0, hi - lo)};
}

// Whether cu falls or leaves [0, rows] at entry b.
__device__ __forceinline__ bool seq_bad(const int* cu, int b, int rows) {
  return cu && (cu[b + 1] < cu[b] || cu[b] < 0 || cu[b + 1] > rows);
}

// The first row of head 0 of the slot's page, counted in rows of head_dim over the whole cache, and the
// row within a page: row of head h = at(h). page < 0: the table names no page of the cache.
struct PagePlace {
  int page, row;
};
__device__ __forceinline__ PagePlace page_place(const PagedCache& c, int b, int slot) {
  const int page = c.pages[(size_t)b * c.max_pages + (slot >> c.page_shift)];
  return {page >= 0 && page < c.n_pages ? page : -1, slot & ((1 << c.page_shift) - 1)};
}
__device__ __forceinline__ long long place_row(const PagedCache& c, const PagePlace& at, int Hkv, int head) {
  return (((long long)at.page * Hkv + head) << c.page_shift) + at.row;
}

// cluster-wide barrier in two halves
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// Launch in clusters of `size` CTAs along x, with programmatic stream serialization.
template <typename... KArgs, typename... Args>
inline cudaError_t launch_clusters(void (*kern)(KArgs...), int grid, int block, int smem, int size, cudaStream_t s, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)block);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)size;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...);
}

}  // namespace blk
