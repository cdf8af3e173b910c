// attn_params.h -- parameters of the attention step between a decoder layer's
// q|k|v and o linears: page assignment (kv_assign.cu), head norms with rotary
// positions into the paged cache (rope_cache.cu) and decode attention over the
// cache (paged_attention.cu).
#pragma once
#include <cuda_runtime.h>

#include <atomic>
#include <cstddef>
#include <cstdint>

#include "attn_split.cuh"

namespace svq {

constexpr int kMaxOrdered = 65536;       // entries of an output row that is written in another order
constexpr int kMaxSeqs = 4096;           // requests of one call (their prefix sums stay in shared memory)

struct KvAssignParams {
  const int32_t* lens;
  const int32_t* n_new;
  int32_t* table;                        // [n_seqs][width]
  int32_t* free_pages;                   // [n_pages], a stack
  const int32_t* n_free;
  int32_t* lens_out;
  int32_t* n_free_out;
  int32_t* cu_rows;                      // [n_seqs + 1]
  int32_t* positions;                    // [max_rows]
  int32_t* slots;                        // [max_rows]
  int32_t* status;
  FastDiv by_page;
  int n_seqs, width, page_size, n_pages, max_rows;
};
cudaError_t launch_kv_assign(const KvAssignParams& p, cudaStream_t st);

// A paged cache: element (page, token, head, d) of K and of V at
// page * page_stride + token * token_stride + head * head_stride + d.
struct KvView {
  uint16_t* k;
  uint16_t* v;
  int64_t page_stride, token_stride, head_stride;
  int n_pages, page_size, n_heads;
};

struct RopeCacheParams {
  const void* q;
  const void* k;
  const void* v;
  int64_t ldq, ldk, ldv;                 // elements between rows
  const uint16_t* q_gamma;               // fp16 [D] or null (no norm)
  const uint16_t* k_gamma;
  const double* inv_freq;                // [rot / 2] radians per position
  const int32_t* positions;
  const int32_t* slots;
  uint16_t* q_out;                       // [M][n_q][D]
  int32_t* status;
  KvView kv;
  float eps, factor;
  int M, n_q, rot, interleaved;
  // set by the launcher: slices of a row, of its queries, of its keys; steps of a slice
  FastDiv by_slices;
  int q_slices, kv_slices, steps;
};
// x_dtype: 0 fp32, 1 fp16, 2 bf16; kv_bf16: type of q_out and the cache.
cudaError_t launch_rope_cache(const RopeCacheParams& p, int head_dim, int x_dtype, int kv_bf16, int num_sms,
                              cudaStream_t st);

struct PagedAttnParams {
  const uint16_t* q;                     // [n_rows][n_q][D]
  const int32_t* lens;
  const int32_t* cu_rows;                // [n_seqs + 1] or null (row b = request b)
  const int32_t* table;                  // [n_seqs][width]
  const int32_t* order;                  // [n_q * D] or null
  uint16_t* out;                         // [n_rows][n_q * D]
  float* lse;                            // [n_rows][n_q] or null
  int32_t* status;
  unsigned* counters;                    // [ctas], zero between calls
  float* cta_part;                       // [ctas][2][rows * D + 2 * rows]
  float* warp_part;                      // [ctas][warps][rows * D]
  KvView kv;
  float scale_log2;
  FastDiv by_heads, by_row_tiles, by_page;   // key heads * row tiles, row tiles, tokens per page
  int n_seqs, width, n_q, n_rows, group, row_tiles, out_bf16;
};

struct PagedAttnPlan {
  int ctas, warps, rows;                 // rows: query heads of one unit, padded to 8 or 16
  size_t smem, ws_total, cta_part, warp_part;
};
// Host plan for a head layout (the lengths are read on the device): false when
// no kernel handles it.
bool plan_paged_attn(int n_q, int n_kv, int head_dim, int n_seqs, int num_sms, PagedAttnPlan* plan);
cudaError_t launch_paged_attn(const PagedAttnParams& p, const PagedAttnPlan& plan, int head_dim, int kv_bf16,
                              cudaStream_t st);

// Lets a kernel use that much dynamic shared memory on the current device.  Set
// once per device (the call costs a fifth of a launch): `have` is the kernel's own
// table of what was set.
template <typename Kern>
cudaError_t allow_smem(Kern kern, size_t bytes, std::atomic<int> (&have)[64]) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && have[dev].load(std::memory_order_acquire) >= (int)bytes) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess && dev < 64) have[dev].store((int)bytes, std::memory_order_release);
  return e;
}

// Launch with programmatic stream serialization (the kernel waits with
// griddepcontrol.wait) and, for cluster > 1, as clusters of that many CTAs.
template <typename Kern, typename... P>
cudaError_t launch_dependent(Kern kern, dim3 grid, unsigned threads, size_t smem, unsigned cluster,
                             cudaStream_t st, const P&... p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kern, p...);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace svq
