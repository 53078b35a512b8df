// Attention with modified scores (sv_spec_verify_attn_scored) on CUDA cores: fp32 caches and the
// head sizes and block sizes that the warp-matrix kernels (attn_scored.cuh) do not take.
//
// For sequence b, query row i at position p_i and query head h, over the visible keys t at
// positions p_t (p_t = t for the committed keys t < c, the new row's own position after that):
//   s_t = cap tanh(scale <q, k_t> / cap) - slope_h (p_i - p_t),   o = sum_t softmax_t(s) v_t,
// visible: t < c, or the new row t - c is (j <= i, or bit j of the row's tree mask); and
// p_i - p_t < window. A key that a row does not see never enters its sums, whatever it holds.
//
// A CTA owns (key split, KV head, sequence) and all G n_b query rows of the KV head, 16 at a time;
// keys go through shared memory 32 at a time; a warp keeps four rows' running maximum and sum and
// their accumulators, a lane per key for the scores and a lane per column for the weighted sum.
// Splits that the window leaves no key in write an empty partial (log-sum-exp -inf). A visible
// NaN makes its row's sum and log-sum-exp NaN, and the merge of the splits carries it on.
#include <cuda_fp8.h>

#include "sv_internal.cuh"

namespace sv {
namespace {

constexpr int kThreads = 128;
constexpr int kKeys = 32;         // keys per shared-memory tile
constexpr int kRowsPerPass = 16;  // query rows per pass (4 per warp)
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
__device__ __forceinline__ float pool_f32(__nv_bfloat16 x, float) { return __bfloat162float(x); }
__device__ __forceinline__ float pool_f32(float x, float) { return x; }
__device__ __forceinline__ float pool_f32(uint8_t x, float scale) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw(x, __NV_E4M3);
  return __half2float(__half(h)) * scale;
}

template <typename T, typename KT /* pool element */, int NK /* head_dim / 32 */>
__global__ void __launch_bounds__(kThreads) attn_scored_simt_kernel(ScoredArgs sa) {
  grid_dependency_wait();  // the earlier kernel on the stream is complete and visible
  grid_dependents_launch();
  constexpr int D = NK * 32;
  __shared__ float q_s[kRowsPerPass][D];
  __shared__ float k_s[kKeys][D + 1];
  __shared__ float v_s[kKeys][D];
  __shared__ int s_bad;

  const AttnArgs &a = sa.a;
  const int split = blockIdx.x, kvh = blockIdx.y, b = blockIdx.z;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const KV &kv = a.kv;
  const int c = kv.seq_lens[b];
  const int row0 = a.cu_q[b];
  const int n = a.cu_q[b + 1] - row0;
  const long long L64 = (long long)c + n;
  if (c < 0 || n < 0 || n > a.max_q || row0 < 0 || (long long)row0 + n > a.total_q || L64 > a.max_seq_len ||
      L64 > (long long)kv.max_blocks * kv.block_size) {
    if (split == 0 && kvh == 0 && tid == 0) record(a.status, SV_ERR_BAD_LENGTH);
    return;
  }
  const int L = (int)L64;
  const int nsplit = (L + a.chunk - 1) / a.chunk;
  if (split >= nsplit) return;
  // no row is before position c, so no row sees a key before c - window + 1
  const int first = sa.window > 0 ? max(0, c - sa.window + 1) : 0;
  const int kb = max(split * a.chunk, first / kKeys * kKeys), ke = min(L, (split + 1) * a.chunk);
  const int G = a.num_q_heads / kv.num_kv_heads;
  const int R = G * n;
  const T *qp = reinterpret_cast<const T *>(a.q);
  const KT *kp = reinterpret_cast<const KT *>(kv.k_pool);
  const KT *vp = reinterpret_cast<const KT *>(kv.v_pool);
  if (tid == 0) s_bad = 0;

  for (int rg = 0; rg < R; rg += kRowsPerPass) {
    __syncthreads();
    for (int x = tid; x < kRowsPerPass * D; x += kThreads) {
      const int rr = x / D, d = x % D, r = rg + rr;
      float val = 0.f;
      if (r < R) {
        const int i = r / G, g = r % G;
        val = to_f32(qp[((size_t)(row0 + i) * a.num_q_heads + kvh * G + g) * D + d]);
      }
      q_s[rr][d] = val;
    }
    float m[4], l[4], acc[4][NK], slope[4];
    int pos[4];
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      m[w] = -INFINITY;
      l[w] = 0.f;
#pragma unroll
      for (int k = 0; k < NK; ++k) acc[w][k] = 0.f;
      const int r = rg + warp * 4 + w, i = r < R ? r / G : 0, g = r < R ? r % G : 0;
      pos[w] = n > 0 && sa.positions != nullptr ? sa.positions[row0 + i] : c + i;
      if (n > 0 && pos[w] < c && lane == 0) record(a.status, SV_ERR_BAD_LENGTH);
      slope[w] = sa.slopes != nullptr ? sa.slopes[kvh * G + g] * kLog2e : 0.f;
    }
    for (int kt = kb; kt < ke; kt += kKeys) {
      __syncthreads();
      for (int x = tid; x < kKeys * D; x += kThreads) {
        const int j = x / D, d = x % D, t = kt + j;
        float kk = 0.f, vv = 0.f;
        if (t < ke) {
          const int blk = kv.block_table[(size_t)b * kv.max_blocks + t / kv.block_size];
          if (blk >= 0 && blk < kv.num_blocks) {
            const size_t off = (((size_t)blk * kv.num_kv_heads + kvh) * kv.block_size + t % kv.block_size) * D + d;
            kk = pool_f32(kp[off], kv.k_scale);
            vv = pool_f32(vp[off], kv.v_scale);
          } else {
            s_bad = 1;
          }
        }
        k_s[j][d] = kk;
        v_s[j][d] = vv;
      }
      __syncthreads();
      const int t = kt + lane, j = t - c;
      int pt = t;
      if (j >= 0 && j < n && sa.positions != nullptr) pt = sa.positions[row0 + j];
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const int rr = warp * 4 + w, r = rg + rr;
        if (r >= R) continue;
        const int i = r / G;
        bool vis = t < ke && (sa.window <= 0 || pos[w] - pt < sa.window);
        if (vis && j >= 0)
          vis = a.mask_kind == SV_MASK_CAUSAL ? j <= i : (j < 64 && ((a.tree_mask[row0 + i] >> j) & 1ull));
        float s = -INFINITY;
        if (vis) {
          float dot = 0.f;
#pragma unroll 8
          for (int d = 0; d < D; ++d) dot = fmaf(q_s[rr][d], k_s[lane][d], dot);
          s = dot * a.scale_log2;
          if (sa.cap > 0.f) s = sa.cap * tanhf(s / sa.cap);  // both in units of log2
          s -= slope[w] * (float)(pos[w] - pt);
        }
        const unsigned seen = __ballot_sync(0xffffffffu, vis);
        const float mn = fmaxf(m[w], warp_max(s));
        if (seen == 0u) continue;
        const float ref = mn == -INFINITY ? 0.f : mn;
        const float p = vis ? exp2f(s - ref) : 0.f;
        const float alpha = exp2f(m[w] - ref);
        l[w] = l[w] * alpha + warp_sum(p);
#pragma unroll
        for (int k = 0; k < NK; ++k) acc[w][k] *= alpha;
        for (unsigned left = seen; left != 0u; left &= left - 1u) {
          const int key = __ffs(left) - 1;
          const float pj = __shfl_sync(0xffffffffu, p, key);
#pragma unroll
          for (int k = 0; k < NK; ++k) acc[w][k] = fmaf(pj, v_s[key][lane + 32 * k], acc[w][k]);
        }
        m[w] = mn;
      }
    }
    // write this pass's rows
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const int r = rg + warp * 4 + w;
      if (r >= R) continue;
      const int i = r / G, g = r % G, h = kvh * G + g;
      const size_t qrow = (size_t)(row0 + i) * a.num_q_heads + h;
      const float inv = l[w] == 0.f ? 0.f : 1.f / l[w];  // a row that sees no key gets zeros
      if (nsplit == 1) {
        T *op = reinterpret_cast<T *>(a.out);
#pragma unroll
        for (int k = 0; k < NK; ++k) op[qrow * D + lane + 32 * k] = from_f32<T>(acc[w][k] * inv);
      } else {
        const size_t prow = (size_t)split * a.total_q * a.num_q_heads + qrow;
#pragma unroll
        for (int k = 0; k < NK; ++k) a.ws_o[prow * D + lane + 32 * k] = acc[w][k] * inv;
        if (lane == 0) a.ws_lse[prow] = l[w] == 0.f ? -INFINITY : m[w] + log2f(l[w]);
      }
    }
  }
  __syncthreads();
  if (tid == 0 && s_bad) record(a.status, SV_ERR_BAD_BLOCK_ID);
}

// One warp per (query row, query head): o = sum_s 2^(lse_s) o_s / sum_s 2^(lse_s) over the splits.
template <typename T>
__global__ void __launch_bounds__(kThreads) attn_scored_simt_combine(ScoredArgs sa) {
  grid_dependency_wait();  // the earlier kernel on the stream is complete and visible
  grid_dependents_launch();
  const AttnArgs &a = sa.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.y;
  const int c = a.kv.seq_lens[b], row0 = a.cu_q[b], n = a.cu_q[b + 1] - row0;
  const long long L = (long long)c + n;
  if (c < 0 || n < 0 || n > a.max_q || row0 < 0 || (long long)row0 + n > a.total_q || L > a.max_seq_len ||
      L > (long long)a.kv.max_blocks * a.kv.block_size)
    return;
  const int x = blockIdx.x * (kThreads / 32) + warp;  // (row, head) of the sequence
  const int nsplit = ((int)L + a.chunk - 1) / a.chunk;
  if (x >= n * a.num_q_heads || nsplit <= 1) return;
  const int D = a.kv.head_dim;
  const size_t idx = (size_t)row0 * a.num_q_heads + x, stride = (size_t)a.total_q * a.num_q_heads;
  float M = -INFINITY;
  for (int s = 0; s < nsplit; ++s) M = fmaxf(M, a.ws_lse[s * stride + idx]);
  const float ref = M == -INFINITY ? 0.f : M;
  T *op = reinterpret_cast<T *>(a.out);
  for (int d = lane; d < D; d += 32) {
    float num = 0.f, den = 0.f;
    for (int s = 0; s < nsplit; ++s) {
      const float w = exp2f(a.ws_lse[s * stride + idx] - ref);
      den += w;
      num = fmaf(w, a.ws_o[(s * stride + idx) * D + d], num);
    }
    op[idx * D + d] = from_f32<T>(den == 0.f ? 0.f : num / den);
  }
}

template <typename T, typename KT>
cudaError_t launch_t(const ScoredArgs &sa, cudaStream_t st) {
  const dim3 grid(sa.a.max_splits, sa.a.kv.num_kv_heads, sa.a.kv.batch);
  auto go = [&](auto kernel) { return launch_pdl(kernel, grid, dim3(kThreads), 0, st, sa); };
  switch (sa.a.kv.head_dim / 32) {
    case 1: return go(attn_scored_simt_kernel<T, KT, 1>);
    case 2: return go(attn_scored_simt_kernel<T, KT, 2>);
    case 3: return go(attn_scored_simt_kernel<T, KT, 3>);
    case 4: return go(attn_scored_simt_kernel<T, KT, 4>);
    case 5: return go(attn_scored_simt_kernel<T, KT, 5>);
    case 6: return go(attn_scored_simt_kernel<T, KT, 6>);
    case 7: return go(attn_scored_simt_kernel<T, KT, 7>);
    default: return go(attn_scored_simt_kernel<T, KT, 8>);
  }
}

}  // namespace

cudaError_t launch_attn_scored_simt(const ScoredArgs &sa, int dtype, cudaStream_t st) {
  cudaError_t e;
  if (dtype == SV_DTYPE_E4M3) e = launch_t<__nv_bfloat16, uint8_t>(sa, st);  // bf16 queries and outputs
  else e = dtype == SV_DTYPE_BF16 ? launch_t<__nv_bfloat16, __nv_bfloat16>(sa, st) : launch_t<float, float>(sa, st);
  if (e != cudaSuccess || sa.a.max_splits <= 1) return e;
  const dim3 grid((unsigned)ceil_div(sa.a.max_q * sa.a.num_q_heads, kThreads / 32), (unsigned)sa.a.kv.batch);
  return dtype == SV_DTYPE_F32 ? launch_pdl(attn_scored_simt_combine<float>, grid, dim3(kThreads), 0, st, sa)
                               : launch_pdl(attn_scored_simt_combine<__nv_bfloat16>, grid, dim3(kThreads), 0, st, sa);
}

}  // namespace sv
