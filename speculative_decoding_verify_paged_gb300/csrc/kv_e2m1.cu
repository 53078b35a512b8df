// Rows into a 4-bit pool as they are (sv_kv_append, after kv_alloc_kernel has taken the blocks), and rows of
// a pool of any type as dense rows (sv_kv_gather). The format is in e2m1.cuh.
//
// Both are copies with a conversion on the way: a value is read once and written once (store: 2 bytes in and
// 9/16 out, gather the other way round), so memory bounds long calls and the chain launch -> owner of the row -> length ->
// block id -> rows short ones. A CTA takes a few consecutive rows: its first warp finds where they stand, then a thread
// takes 16 values of a row (a group of codes; 16 or 32 bytes of wider types) at a time.
//
// 8 heads of 128 values. Rows into the pool (two launches, the allocation's among them): 256 x 64 19.2 us (4.5 TB/s of what it
// cannot do without, 86 MB), 32 x 6 5.5 us. Rows out of it (one launch): those 256 x 64 18.4 us, 74K rows of 32 sequences
// 66 us (5.9 TB/s), from E4M3, bf16 and fp32 pools 74, 95 and 186 us (6.2, 6.4 and 6.5 TB/s); 4 short sequences' 4.8 us.
#include <algorithm>

#include "e2m1.cuh"
#include "kv_rows.cuh"

namespace sv {
namespace {

constexpr int kThreads = 256;
constexpr int kMostRows = 32;  // of a CTA: a lane of its first warp finds each

// 32 bytes that a thread reads or writes; W: aligned to 32 bytes, in one access
template <bool W> __device__ __forceinline__ void read32(const uint8_t *p, uint32_t (&w)[8]) {
  if (W) {
    asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(p));
  } else {
    const uint4 a = reinterpret_cast<const uint4 *>(p)[0], b = reinterpret_cast<const uint4 *>(p)[1];
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
  }
}
template <bool W> __device__ __forceinline__ void write32(uint8_t *p, const uint32_t (&w)[8]) {
  if (W) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
                 "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4 *>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4 *>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// Where the CTA's rows stand in the cache: the number of each among a head's rows of the pool, [block][head] apart
// (block * num_kv_heads * block_size + slot), or -1; none where `heed` and the status word holds an error. By the first
// warp, a lane a row.
template <typename First>
__device__ __forceinline__ void find_rows(const KV &kv, const int32_t *cu, int row0, int rows, long long *at, int32_t *status,
                                          bool heed, First first_of) {
  const int lane = threadIdx.x & 31;
  if (threadIdx.x >= 32) return;
  const bool failed = __any_sync(0xffffffffu, heed && status_set(status));
  int b = owner_of(cu, kv.batch, row0);
  if (lane >= rows) return;
  at[lane] = -1;
  if (failed) return;
  const int row = row0 + lane, bsh = __ffs(kv.block_size) - 1;
  while (b + 1 < kv.batch && cu[b + 1] <= row) ++b;
  const int lo = cu[b], i = row - lo, n = cu[b + 1] - lo;
  long long to = -1;
  if (i >= 0 && i < n) {  // else: past cu[batch]
    const long long first = first_of(b);
    if (first < 0 || first + n > (long long)kv.max_blocks * kv.block_size) {
      record(status, SV_ERR_BAD_LENGTH);
    } else {
      const int pos = (int)(first + i), blk = kv.block_table[(size_t)b * kv.max_blocks + (pos >> bsh)];
      if (blk < 0 || blk >= kv.num_blocks) record(status, SV_ERR_BAD_BLOCK_ID);
      else to = (long long)blk * kv.num_kv_heads * kv.block_size + (pos & (kv.block_size - 1));
    }
  }
  at[lane] = to;
}

// 16 bf16 values in w -> two words of codes and their scale
__device__ __forceinline__ uint2 encode16(const uint32_t (&w)[8], float scale, float inv6, uint8_t *s) {
  float x[2][8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    x[k >> 2][2 * (k & 3)] = __uint_as_float(w[k] << 16);
    x[k >> 2][2 * (k & 3) + 1] = __uint_as_float(w[k] & 0xffff0000u);
  }
  const uint32_t code = block_scale(max_nan(top_of(x[0]), top_of(x[1])), inv6);
  const float r = code_factor(code, scale);
  *s = (uint8_t)code;
  return make_uint2(codes8(x[0], r), codes8(x[1], r));
}

template <bool W>
__global__ void __launch_bounds__(kThreads) kv_store_kernel(KV kv, const uint8_t *new_k, const uint8_t *new_v, const int32_t *cu_q,
                                                            int total_q, int per_cta, float k_inv6, float v_inv6, int32_t *status) {
  __shared__ long long s_at[kMostRows];
  const int row0 = blockIdx.x * per_cta, rows = min(per_cta, total_q - row0);
  const int groups = kv.head_dim / 16, cols = kv.num_kv_heads * groups, items = rows * cols;
  uint32_t k[8], v[8];
  auto load = [&](int x) {  // (a row's groups are contiguous, and so are the CTA's rows)
    const size_t from = ((size_t)row0 * cols + x) * 32;
    read32<W>(new_k + from, k);
    read32<W>(new_v + from, v);
  };
  // the rows are the call's own inputs, read before the wait (the allocation, which lets this kernel start, has waited for the
  // kernels before it); what the allocation writes comes after it, and cu_q with it
  if ((int)threadIdx.x < items) load(threadIdx.x);
  grid_dependency_wait();
  grid_dependents_launch();
  find_rows(kv, cu_q, row0, rows, s_at, status, true, [&](int b) { return (long long)kv.seq_lens[b]; });
  __syncthreads();
  for (int x = threadIdx.x; x < items; x += kThreads) {
    if (x >= kThreads) load(x);
    const int r = x / cols, col = x - r * cols, h = col / groups, g = col - h * groups;
    const long long at = s_at[r];
    if (at < 0) continue;
    const size_t to = (size_t)(at + (long long)h * kv.block_size) * groups + g;
    reinterpret_cast<uint2 *>(kv.k_pool)[to] = encode16(k, kv.k_scale, k_inv6, kv.k_bs + to);
    reinterpret_cast<uint2 *>(kv.v_pool)[to] = encode16(v, kv.v_scale, v_inv6, kv.v_bs + to);
  }
}

enum { kBf16, kF32, kE4m3, kE2m1 };

// Values of one access: 32 bytes of the output
template <int T> constexpr int kVals = T == kF32 ? 8 : 16;

template <int T, bool W>
__device__ __forceinline__ void decode(const uint8_t *pool, const uint8_t *bs, size_t unit, float scale, uint8_t *out) {
  uint32_t w[8];
  if (T == kBf16 || T == kF32) {
    read32<W>(pool + unit * 32, w);
  } else if (T == kE4m3) {
    const uint4 c = reinterpret_cast<const uint4 *>(pool)[unit];
    const uint32_t in[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const __half2 h = __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(in[q >> 1] >> (16 * (q & 1))), __NV_E4M3));
      const float2 f = __half22float2(h);
      const __nv_bfloat162 o = __floats2bfloat162_rn(f.x * scale, f.y * scale);
      w[q] = *reinterpret_cast<const uint32_t *>(&o);
    }
  } else {
    const uint2 c = reinterpret_cast<const uint2 *>(pool)[unit];
    const float step = __fmul_rn(e4m3_value(bs[unit]), scale);
    uint32_t p[8];
    widen8(c.x, p[0], p[1], p[2], p[3]);
    widen8(c.y, p[4], p[5], p[6], p[7]);
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const float2 f = pair_of(p[q]);
      const __nv_bfloat162 o = __floats2bfloat162_rn(f.x * step, f.y * step);
      w[q] = *reinterpret_cast<const uint32_t *>(&o);
    }
  }
  write32<W>(out, w);
}

// (Nothing that follows on the stream starts before this kernel is complete: a later append may read its outputs ahead of
// its own dependency wait.)
template <int T, bool W>
__global__ void __launch_bounds__(kThreads) kv_gather_kernel(KV kv, uint8_t *out_k, uint8_t *out_v, const int32_t *cu, int total,
                                                             int per_cta, const int32_t *first, int32_t *status) {
  __shared__ long long s_at[kMostRows];
  grid_dependency_wait();  // the earlier kernel on the stream is complete and visible
  const int row0 = blockIdx.x * per_cta, rows = min(per_cta, total - row0);
  find_rows(kv, cu, row0, rows, s_at, status, false, [&](int b) { return (long long)(first != nullptr ? first[b] : kv.seq_lens[b]); });
  __syncthreads();
  const int units = kv.head_dim / kVals<T>, cols = kv.num_kv_heads * units, items = rows * cols;
#pragma unroll 2
  for (int x = threadIdx.x; x < items; x += kThreads) {
    const int r = x / cols, col = x - r * cols, h = col / units, g = col - h * units;
    const long long at = s_at[r];
    if (at < 0) continue;
    const size_t unit = (size_t)(at + (long long)h * kv.block_size) * units + g, to = ((size_t)row0 * cols + x) * 32;
    if (out_k != nullptr) decode<T, W>((const uint8_t *)kv.k_pool, kv.k_bs, unit, kv.k_scale, out_k + to);
    if (out_v != nullptr) decode<T, W>((const uint8_t *)kv.v_pool, kv.v_bs, unit, kv.v_scale, out_v + to);
  }
}
// Head sizes that are 8 more than a multiple of 16, in bf16: rows in units of 16 bytes
__global__ void __launch_bounds__(kThreads) kv_gather_narrow_kernel(KV kv, uint4 *out_k, uint4 *out_v, const int32_t *cu, int total,
                                                                    int per_cta, const int32_t *first, int32_t *status) {
  __shared__ long long s_at[kMostRows];
  grid_dependency_wait();  // the earlier kernel on the stream is complete and visible
  const int row0 = blockIdx.x * per_cta, rows = min(per_cta, total - row0);
  find_rows(kv, cu, row0, rows, s_at, status, false, [&](int b) { return (long long)(first != nullptr ? first[b] : kv.seq_lens[b]); });
  __syncthreads();
  const int units = kv.head_dim / 8, cols = kv.num_kv_heads * units, items = rows * cols;
  for (int x = threadIdx.x; x < items; x += kThreads) {
    const int r = x / cols, col = x - r * cols, h = col / units, g = col - h * units;
    const long long at = s_at[r];
    if (at < 0) continue;
    const size_t unit = (size_t)(at + (long long)h * kv.block_size) * units + g, to = (size_t)row0 * cols + x;
    if (out_k != nullptr) out_k[to] = reinterpret_cast<const uint4 *>(kv.k_pool)[unit];
    if (out_v != nullptr) out_v[to] = reinterpret_cast<const uint4 *>(kv.v_pool)[unit];
  }
}

// Rows of a CTA, with so many CTAs an SM: kMostRows at most.
int rows_per_cta(int total, int per_sm) { return std::max(1, std::min(kMostRows, ceil_div(total, num_sms() * per_sm))); }
// The store's registers let four CTAs stay on an SM: one wave while its CTAs have rows enough for that, else two, the second
// under the first one's tail. (us with 4, 8 and 12 CTAs an SM, 8 heads of 128: 1024 rows 6.2, 8.6, 8.6; 6144 10.8, 12.4,
// 13.0; 10240 14.5, 16.1, 17.2; 16384 19.2, 20.4, 22.8; 24000, where four are a wave and a quarter, 31.0, 26.1, 28.2; 32768
// 34.6, 33.6, 35.6; 65536 the same.)
int store_rows(int total) { return rows_per_cta(total, ceil_div(total, num_sms() * 4) <= kMostRows ? 4 : 8); }
// The gather's let eight. (The same sizes: 4.6, 4.6, 4.6; 10.4, 9.4, 9.5; 14.8, 12.7, 13.6; 21.5, 18.4, 19.1; 27.7, 24.3, 26.7;
// 33.4, 32.2, 34.7.)
int gather_rows(int total) { return rows_per_cta(total, 8); }
bool aligned32(const void *a, const void *b) { return (((uintptr_t)a | (uintptr_t)b) & 31u) == 0; }

}  // namespace

cudaError_t launch_kv_store_e2m1(const KV &kv, const void *new_k, const void *new_v, const int32_t *cu_q, int total_q,
                                 int32_t *status, cudaStream_t st) {
  if (kv.ref_count != nullptr) {
    const cudaError_t e = launch_private_copies(kv, cu_q, status, st);
    if (e != cudaSuccess) return e;
  }
  const int per = store_rows(total_q);
  auto kernel = aligned32(new_k, new_v) ? kv_store_kernel<true> : kv_store_kernel<false>;
  return launch_pdl(kernel, dim3((unsigned)ceil_div(total_q, per)), dim3(kThreads), 0, st, kv, (const uint8_t *)new_k,
                    (const uint8_t *)new_v, cu_q, total_q, per, 1.f / (6.f * kv.k_scale), 1.f / (6.f * kv.v_scale), status);
}

cudaError_t launch_kv_gather(const KV &kv, void *out_k, void *out_v, const int32_t *cu_rows, int total_rows,
                             const int32_t *first, int32_t *status, cudaStream_t st) {
  const int per = gather_rows(total_rows);
  const dim3 grid((unsigned)ceil_div(total_rows, per));
  if (kv.elem_bytes == 2 && kv.head_dim % 16 != 0)
    return launch_pdl(kv_gather_narrow_kernel, grid, dim3(kThreads), 0, st, kv, (uint4 *)out_k, (uint4 *)out_v, cu_rows, total_rows, per,
                      first, status);
  auto go = [&](auto wide, auto narrow) {
    const bool w = aligned32(out_k, out_v) && (kv.fp4 || kv.fp8 || aligned32(kv.k_pool, kv.v_pool));
    return launch_pdl(w ? wide : narrow, grid, dim3(kThreads), 0, st, kv, (uint8_t *)out_k, (uint8_t *)out_v, cu_rows, total_rows, per,
                      first, status);
  };
  if (kv.fp4) return go(kv_gather_kernel<kE2m1, true>, kv_gather_kernel<kE2m1, false>);
  if (kv.fp8) return go(kv_gather_kernel<kE4m3, true>, kv_gather_kernel<kE4m3, false>);
  return kv.elem_bytes == 2 ? go(kv_gather_kernel<kBf16, true>, kv_gather_kernel<kBf16, false>)
                            : go(kv_gather_kernel<kF32, true>, kv_gather_kernel<kF32, false>);
}

}  // namespace sv
