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
// keys go through shared memory as fp32, 32 at a time, in 16-byte reads; a warp keeps four rows' running
// maximum and sum and their accumulators, a lane per key for the scores (four rows' products on
// each 16-byte read of its key) and a lane per column for the weighted sum (four keys' weights a read).
// Bound: latency for the short splits it is cut into (four CTAs an SM), the products for wide units.
// Splits that the window leaves no key in write an empty partial (log-sum-exp -inf). A visible
// NaN makes its row's sum and log-sum-exp NaN, and the merge of the splits carries it on.
#include <cuda_fp16.h>
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
// 16 bytes of a row as fp32 into shared memory
__device__ __forceinline__ void widen16(float *dst, uint4 w, float, const float *) {
  *reinterpret_cast<uint4 *>(dst) = w;
}
__device__ __forceinline__ void widen16(float *dst, uint4 w, float, const __nv_bfloat16 *) {
  reinterpret_cast<float4 *>(dst)[0] = make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u),
                                                   __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u));
  reinterpret_cast<float4 *>(dst)[1] = make_float4(__uint_as_float(w.z << 16), __uint_as_float(w.z & 0xffff0000u),
                                                   __uint_as_float(w.w << 16), __uint_as_float(w.w & 0xffff0000u));
}
__device__ __forceinline__ void widen16(float *dst, uint4 w, float scale, const uint8_t *) {
  const uint32_t word[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    float v[4];
#pragma unroll
    for (int h = 0; h < 4; ++h)
      v[h] = __half2float(__half(__nv_cvt_fp8_to_halfraw((uint8_t)(word[q] >> (8 * h)), __NV_E4M3))) * scale;
    reinterpret_cast<float4 *>(dst)[q] = make_float4(v[0], v[1], v[2], v[3]);
  }
}

template <typename T, typename KT /* pool element */, int NK /* head_dim / 32 */>
__global__ void __launch_bounds__(kThreads) attn_scored_simt_kernel(ScoredArgs sa) {
  grid_dependency_wait();  // the earlier kernel on the stream is complete and visible
  grid_dependents_launch();
  constexpr int D = NK * 32;
  constexpr int kVec = 16 / sizeof(KT), kChunks = D / kVec;  // values in 16 bytes of a pool row; reads of a row
  __shared__ __align__(16) float q_s[kRowsPerPass][D];
  __shared__ __align__(16) float k_s[kKeys][D + 4];
  __shared__ __align__(16) float v_s[kKeys][D];
  __shared__ __align__(16) float p_s[kRowsPerPass][kKeys];
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
    unsigned hide[4];  // keys of the tile that a row does not see
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
#pragma unroll 4
      for (int x = tid; x < kKeys * kChunks; x += kThreads) {
        const int j = x / kChunks, d = x % kChunks * kVec, t = kt + j;
        uint4 kk = make_uint4(0, 0, 0, 0), vv = kk;
        if (t < ke) {
          const int blk = kv.block_table[(size_t)b * kv.max_blocks + t / kv.block_size];
          if (blk >= 0 && blk < kv.num_blocks) {
            const size_t off = (((size_t)blk * kv.num_kv_heads + kvh) * kv.block_size + t % kv.block_size) * D + d;
            kk = *reinterpret_cast<const uint4 *>(kp + off);
            vv = *reinterpret_cast<const uint4 *>(vp + off);
          } else {
            s_bad = 1;
          }
        }
        widen16(&k_s[j][d], kk, kv.k_scale, (const KT *)nullptr);
        widen16(&v_s[j][d], vv, kv.v_scale, (const KT *)nullptr);
      }
      __syncthreads();
      const int t = kt + lane, j = t - c;
      int pt = t;
      if (j >= 0 && j < n && sa.positions != nullptr) pt = sa.positions[row0 + j];
      if (rg + warp * 4 >= R) continue;  // none of this warp's rows
      float dot[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
      for (int d = 0; d < D; d += 4) {
        const float4 kk = *reinterpret_cast<const float4 *>(&k_s[lane][d]);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const float4 qq = *reinterpret_cast<const float4 *>(&q_s[warp * 4 + w][d]);
          dot[w] = fmaf(qq.x, kk.x, fmaf(qq.y, kk.y, fmaf(qq.z, kk.z, fmaf(qq.w, kk.w, dot[w]))));
        }
      }
      unsigned any = 0u;  // keys that some row of the warp sees
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const int r = rg + warp * 4 + w, i = r < R ? r / G : 0;
        bool vis = r < R && t < ke && (sa.window <= 0 || pos[w] - pt < sa.window);
        if (vis && j >= 0)
          vis = a.mask_kind == SV_MASK_CAUSAL ? j <= i : (j < 64 && ((a.tree_mask[row0 + i] >> j) & 1ull));
        float s = -INFINITY;
        if (vis) {
          s = dot[w] * a.scale_log2;
          if (sa.cap > 0.f) s = sa.cap * tanhf(s / sa.cap);  // both in units of log2
          s -= slope[w] * (float)(pos[w] - pt);
        }
        const unsigned seen = __ballot_sync(0xffffffffu, vis);
        float p = 0.f;
        if (seen != 0u) {
          const float mn = fmaxf(m[w], warp_max(s)), ref = mn == -INFINITY ? 0.f : mn;
          p = vis ? exp2f(s - ref) : 0.f;
          const float alpha = exp2f(m[w] - ref);
          l[w] = l[w] * alpha + warp_sum(p);
#pragma unroll
          for (int k = 0; k < NK; ++k) acc[w][k] *= alpha;
          m[w] = mn;
        }
        p_s[warp * 4 + w][lane] = p;
        any |= seen;
        hide[w] = r < R ? ~seen : 0u;
      }
      __syncwarp();
      // a row takes nothing of a key that it does not see, whatever the key's values are
      bool odd = false;
      if ((any & hide[0]) | (any & hide[1]) | (any & hide[2]) | (any & hide[3]))
        for (int d = 0; d < D; d += 4) {
          const float4 v = *reinterpret_cast<const float4 *>(&v_s[lane][d]);
          odd |= !(fabsf(v.x) + fabsf(v.y) + fabsf(v.z) + fabsf(v.w) < INFINITY);
        }
      odd = __any_sync(0xffffffffu, odd && ((any >> lane) & 1u));
      for (int x = 0; x < kKeys; x += 4) {
        if (((any >> x) & 15u) == 0u) continue;
        float4 pw[4];
#pragma unroll
        for (int w = 0; w < 4; ++w) pw[w] = *reinterpret_cast<const float4 *>(&p_s[warp * 4 + w][x]);
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          if (!((any >> (x + y)) & 1u)) continue;
#pragma unroll
          for (int k = 0; k < NK; ++k) {
            const float v = v_s[x + y][lane + 32 * k];
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const float pj = y == 0 ? pw[w].x : y == 1 ? pw[w].y : y == 2 ? pw[w].z : pw[w].w;
              if (!odd || !((hide[w] >> (x + y)) & 1u)) acc[w][k] = fmaf(pj, v, acc[w][k]);
            }
          }
        }
      }
      __syncwarp();
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
  for (int s = lane; s < nsplit; s += 32) M = fmaxf(M, a.ws_lse[s * stride + idx]);
  M = warp_max(M);
  const float ref = M == -INFINITY ? 0.f : M;
  float num[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, den = 0.f;  // columns lane + 32 k
  for (int s0 = 0; s0 < nsplit; s0 += 32) {
    const float w = s0 + lane < nsplit ? exp2f(a.ws_lse[(s0 + lane) * stride + idx] - ref) : 0.f;
    den += w;
    const int n_s = min(32, nsplit - s0);
#pragma unroll 4
    for (int s = 0; s < n_s; ++s) {
      const float ws = __shfl_sync(0xffffffffu, w, s);
      const float *o = a.ws_o + ((s0 + s) * stride + idx) * D + lane;
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k * 32 < D) num[k] = fmaf(ws, o[32 * k], num[k]);
    }
  }
  den = warp_sum(den);
  T *op = reinterpret_cast<T *>(a.out);
#pragma unroll
  for (int k = 0; k < 8; ++k)
    if (k * 32 < D) op[idx * D + lane + 32 * k] = from_f32<T>(den == 0.f ? 0.f : num[k] / den);
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
