// Shared by the kernels that write a step's rows into the cache: copy-on-write's second half.
#pragma once

#include "sv_internal.cuh"

namespace sv {

// Copy-on-write, second half (the first is kv_alloc_kernel's): the sequence's first new row lands
// in slot `slot` of `blk`, a private copy whose count holds -(source id + 1); brings over the
// source's rows before `slot` (every head, K and V) and sets the count to 1. Called by all
// threads of the CTA that writes the row; `row_bytes` is a row's size in the pool.
__device__ __forceinline__ void copy_shared_block(const KV &kv, int blk, int slot, int row_bytes, int32_t *status) {
  const int m = kv.ref_count[blk];
  if (m >= 0) return;
  const int src = -m - 1;
  const int per_head = slot * (row_bytes / 16);  // the rows before `slot` are contiguous in a (block, head)
  const size_t head_bytes = (size_t)kv.block_size * row_bytes;
  if (src >= 0 && src < kv.num_blocks) {
    for (int x = threadIdx.x; x < kv.num_kv_heads * per_head; x += blockDim.x) {
      const int h = x / per_head, v = x - h * per_head;
      const size_t so = ((size_t)src * kv.num_kv_heads + h) * head_bytes + (size_t)v * 16;
      const size_t d_o = ((size_t)blk * kv.num_kv_heads + h) * head_bytes + (size_t)v * 16;
      *reinterpret_cast<uint4 *>((uint8_t *)kv.k_pool + d_o) = *reinterpret_cast<const uint4 *>((const uint8_t *)kv.k_pool + so);
      *reinterpret_cast<uint4 *>((uint8_t *)kv.v_pool + d_o) = *reinterpret_cast<const uint4 *>((const uint8_t *)kv.v_pool + so);
    }
  } else if (threadIdx.x == 0) {
    record(status, SV_ERR_BAD_BLOCK_ID);
  }
  __syncthreads();  // every thread has read the marker
  if (threadIdx.x == 0) kv.ref_count[blk] = 1;
}

}  // namespace sv
