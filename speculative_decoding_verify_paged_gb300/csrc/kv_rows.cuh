// Shared by the kernels that write a step's rows into the cache: copy-on-write's second half.
#pragma once

#include "sv_internal.cuh"

namespace sv {

// The last b < n with cu[b] <= row (0 if none), by the whole warp: 32 probes at a time.
__device__ __forceinline__ int owner_of(const int32_t *cu, int n, int row) {
  const int lane = threadIdx.x & 31;
  int lo = 0, len = n;
  while (len > 1) {
    const int step = (len + 31) >> 5;
    const bool below = lane * step < len && cu[lo + lane * step] <= row;
    const int k = max(0, __popc(__ballot_sync(0xffffffffu, below)) - 1);
    lo += k * step;
    len = min(step, len - k * step);
  }
  return lo;
}

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
    if (kv.fp4) {
      const int sb = kv.head_dim / 16, words = slot * sb / 2;  // an even number of scales a row
      for (int x = threadIdx.x; x < kv.num_kv_heads * words; x += blockDim.x) {
        const int h = x / words, v = x - h * words;
        const size_t so = ((size_t)src * kv.num_kv_heads + h) * kv.block_size * sb + (size_t)v * 2;
        const size_t d_o = ((size_t)blk * kv.num_kv_heads + h) * kv.block_size * sb + (size_t)v * 2;
        *reinterpret_cast<uint16_t *>(kv.k_bs + d_o) = *reinterpret_cast<const uint16_t *>(kv.k_bs + so);
        *reinterpret_cast<uint16_t *>(kv.v_bs + d_o) = *reinterpret_cast<const uint16_t *>(kv.v_bs + so);
      }
    }
  } else if (threadIdx.x == 0) {
    record(status, SV_ERR_BAD_BLOCK_ID);
  }
  __syncthreads();  // every thread has read the marker
  if (threadIdx.x == 0) kv.ref_count[blk] = 1;
}

}  // namespace sv
