// Attention with modified scores (sv_spec_verify_attn_scored) on CUDA cores: fp32 caches and the
// head sizes and block sizes that the warp-matrix kernels (attn_scored.cuh) do not take.
//
// For sequence b, query row i at position p_i and query head h, over the visible keys t at
// positions p_t (p_t = t for the committed keys t < c, the new row's own position after that):
//   s_t = cap tanh(scale <q, k_t> / cap) - slope_h (p_i - p_t),   o = sum_t softmax_t(s) v_t,
// visible: t < c, or the new row t - c is (j <= i, or bit j of the row's tree mask); and
// p_i - p_t < window. A key that a row does not see never enters its sums, whatever it holds.
//
// A CTA owns (key split, KV head, sequence) and all G n_b query rows of the KV head, up to 32 at a time;
// keys go through shared memory as fp32, 32 at a time: K of the next tile loads under the softmax and the
// weighted sum, V under the scores (16-byte copies that no thread waits for; narrow caches are widened on
// the way, and loaded in turn). A lane keeps a key for the scores and a column for the weighted sum.
// Layouts, by the query rows a KV head can have:
//  * more than 16, fp32 caches: a warp keeps 8 rows (a 16-byte read of a key or a value meets 8 rows);
//  * 5 and more: a warp keeps 4;
//  * 4 and fewer: the four warps share the rows: each takes a quarter of the head's values in the scores
//    (summed through shared memory) and of the columns in the weighted sum. The softmax is computed four times.
// Up to eight splits of a sequence are one thread-block cluster, whose CTAs merge their rows through shared
// memory; more leave partials in the workspace for a second kernel.
//
// Bound: shared-memory reads (8 + 4 wavefronts to 32 FMAs of a warp in the scores), and latency for short
// splits. fp32, us: 4 sequences of 37 to 200 tokens, 5 rows, two heads of 64 values 12; 8 sequences of 1K to 2K
// tokens, eight heads of 128 values: 4, 16 and 64 rows a KV head 45, 63, 260 (without asynchronous copies, four
// rows a warp throughout: 91, 105, 357).
// Splits that the window leaves no key in write an empty partial (log-sum-exp -inf). A visible
// NaN makes its row's sum and log-sum-exp NaN, and the merge of the splits carries it on.
#include <type_traits>

#include <cooperative_groups.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "sv_internal.cuh"

namespace sv {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 128;
constexpr int kKeys = 32;         // keys per shared-memory tile
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
// 16 bytes into shared memory, zeros if !there: nobody waits until copies_landed
__device__ __forceinline__ void copy16(float *dst, const void *src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src),
               "r"(there ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LATER /* groups that may still be on their way */>
__device__ __forceinline__ void copies_landed() {
  asm volatile("cp.async.wait_group %0;" ::"n"(LATER) : "memory");
}
// 16 bytes of a narrow row as fp32 into shared memory
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

template <typename T, typename KT /* pool element */, int NK /* head_dim / 32 */, int RW /* rows a warp keeps */,
          bool SHARED /* the warps share RW rows */>
__global__ void __launch_bounds__(kThreads) attn_scored_simt_kernel(ScoredArgs sa) {
  grid_dependency_wait();  // the earlier kernel on the stream is complete and visible
  grid_dependents_launch();
  constexpr int D = NK * 32, kWarps = kThreads / 32;
  constexpr int kVec = 16 / sizeof(KT), kChunks = D / kVec;  // values in 16 bytes of a pool row; reads of a row
  constexpr int kRows = SHARED ? RW : RW * kWarps;           // of a pass
  constexpr int kCols = SHARED ? (NK + kWarps - 1) / kWarps : NK;  // columns a lane keeps
  __shared__ __align__(16) float q_s[kRows][D];
  __shared__ __align__(16) float k_s[kKeys][D + 4];
  __shared__ __align__(16) float v_s[kKeys][D];
  __shared__ __align__(16) float p_s[RW * kWarps][kKeys];
  __shared__ float lse_s[kRows];
  __shared__ float part_s[SHARED ? kWarps : 1][RW][kKeys];  // a quarter's part of the scores
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
  const bool merge_here = sa.cluster && nsplit > 1;  // the same for the whole cluster
  if (split >= nsplit && !merge_here) return;
  // no row is before position c, so no row sees a key before c - window + 1
  const int first = sa.window > 0 ? max(0, c - sa.window + 1) : 0;
  const int kb = max(split * a.chunk, first / kKeys * kKeys), ke = min(L, (split + 1) * a.chunk);
  const int G = a.num_q_heads / kv.num_kv_heads;
  const int R = G * n;
  const int bs_shift = __ffs(kv.block_size) - 1;
  const T *qp = reinterpret_cast<const T *>(a.q);
  const KT *kp = reinterpret_cast<const KT *>(kv.k_pool);
  const KT *vp = reinterpret_cast<const KT *>(kv.v_pool);
  if (tid == 0) s_bad = 0;

  // a lane's key of the tile at kt: its block id, or -1 (past the split; a bad id)
  auto block_of = [&](int kt) {
    const int t = kt + lane;
    if (t >= ke) return -1;
    const int id = kv.block_table[(size_t)b * kv.max_blocks + (t >> bs_shift)];
    if (id >= 0 && id < kv.num_blocks) return id;
    s_bad = 1;
    return -1;
  };
  // the tile at kt of a pool into shared memory; all lanes take part
  auto fetch = [&](float *dst, int pitch, const KT *pool, float scale, int kt, int ids) {
    for (int x = tid; x < kKeys * kChunks; x += kThreads) {  // kKeys * kChunks is a multiple of 32
      const int j = x / kChunks, d = x % kChunks * kVec, t = kt + j;
      const int id = __shfl_sync(0xffffffffu, ids, j);
      const size_t off = (((size_t)max(id, 0) * kv.num_kv_heads + kvh) * kv.block_size + (t & (kv.block_size - 1))) * D + d;
      if constexpr (sizeof(KT) == 4) {
        copy16(dst + j * pitch + d, pool + off, id >= 0);
      } else {
        const uint4 w = id >= 0 ? *reinterpret_cast<const uint4 *>(pool + off) : make_uint4(0, 0, 0, 0);
        widen16(dst + j * pitch + d, w, scale, (const KT *)nullptr);
      }
    }
    copies_end();
  };

  for (int rg = 0; rg < R; rg += kRows) {
    __syncthreads();
    int ids = kb < ke ? block_of(kb) : -1;
    if (kb < ke) fetch(&k_s[0][0], D + 4, kp, kv.k_scale, kb, ids);
    for (int x = tid; x < kRows * D; x += kThreads) {
      const int rr = x / D, d = x % D, r = rg + rr;
      float val = 0.f;
      if (r < R) {
        const int i = r / G, g = r % G;
        val = to_f32(qp[((size_t)(row0 + i) * a.num_q_heads + kvh * G + g) * D + d]);
      }
      q_s[rr][d] = val;
    }
    const int rw = SHARED ? 0 : warp * RW;  // the warp's first row of the pass
    float m[RW], l[RW], acc[RW][kCols], slope[RW];
    unsigned hide[RW];  // keys of the tile that a row does not see
    int pos[RW];
#pragma unroll
    for (int w = 0; w < RW; ++w) {
      m[w] = -INFINITY;
      l[w] = 0.f;
#pragma unroll
      for (int k = 0; k < kCols; ++k) acc[w][k] = 0.f;
      const int r = rg + rw + w, i = r < R ? r / G : 0, g = r < R ? r % G : 0;
      pos[w] = n > 0 && sa.positions != nullptr ? sa.positions[row0 + i] : c + i;
      if (n > 0 && pos[w] < c && lane == 0) record(a.status, SV_ERR_BAD_LENGTH);
      slope[w] = sa.slopes != nullptr ? sa.slopes[kvh * G + g] * kLog2e : 0.f;
    }
    for (int kt = kb; kt < ke; kt += kKeys) {
      copies_landed<0>();
      __syncthreads();  // K is there, and the last tile's V is done with
      fetch(&v_s[0][0], D, vp, kv.v_scale, kt, ids);
      if (kt + kKeys < ke) ids = block_of(kt + kKeys);
      const bool mine = rg + rw < R;  // some of the warp's rows exist
      const int t = kt + lane, j = t - c;
      int pt = t;
      if (j >= 0 && j < n && sa.positions != nullptr) pt = sa.positions[row0 + j];
      float dot[RW];
#pragma unroll
      for (int w = 0; w < RW; ++w) dot[w] = 0.f;
      if (mine) {
        constexpr int kSpan = SHARED ? D / kWarps : D;
        constexpr int kSum = kSpan % 32 == 0 ? 32 : kSpan;  // values of a partial sum: a sum in sums of 32 rounds less
        const int d0 = SHARED ? warp * kSpan : 0;
#pragma unroll 1
        for (int d1 = d0; d1 < d0 + kSpan; d1 += kSum) {
          float sum[RW];
#pragma unroll
          for (int w = 0; w < RW; ++w) sum[w] = 0.f;
#pragma unroll
          for (int d = 0; d < kSum; d += 4) {
            const float4 kk = *reinterpret_cast<const float4 *>(&k_s[lane][d1 + d]);
#pragma unroll
            for (int w = 0; w < RW; ++w) {
              const float4 qq = *reinterpret_cast<const float4 *>(&q_s[rw + w][d1 + d]);
              sum[w] = fmaf(qq.x, kk.x, fmaf(qq.y, kk.y, fmaf(qq.z, kk.z, fmaf(qq.w, kk.w, sum[w]))));
            }
          }
#pragma unroll
          for (int w = 0; w < RW; ++w) dot[w] += sum[w];
        }
      }
      if constexpr (SHARED)
#pragma unroll
        for (int w = 0; w < RW; ++w) part_s[warp][w][lane] = dot[w];
      __syncthreads();  // every warp is done with K
      if (kt + kKeys < ke) fetch(&k_s[0][0], D + 4, kp, kv.k_scale, kt + kKeys, ids);
      else copies_end();
      unsigned any = 0u, hidden = 0u;  // keys that some row of the warp sees, that some row does not
      if (mine) {
        if constexpr (SHARED)
#pragma unroll
          for (int w = 0; w < RW; ++w)
            dot[w] = (part_s[0][w][lane] + part_s[1][w][lane]) + (part_s[2][w][lane] + part_s[3][w][lane]);
#pragma unroll
        for (int w = 0; w < RW; ++w) {
          const int r = rg + rw + w, i = r < R ? r / G : 0;
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
            for (int k = 0; k < kCols; ++k) acc[w][k] *= alpha;
            m[w] = mn;
          }
          p_s[warp * RW + w][lane] = p;
          any |= seen;
          hide[w] = r < R ? ~seen : 0u;
          hidden |= hide[w];
        }
      }
      copies_landed<1>();
      __syncthreads();  // V is there
      if (!mine) continue;
      // a row takes nothing of a key that it does not see, whatever the key's values are
      bool odd = false;
      if (any & hidden)
        for (int d = 0; d < D; d += 4) {
          const float4 v = *reinterpret_cast<const float4 *>(&v_s[lane][d]);
          odd |= !(fabsf(v.x) + fabsf(v.y) + fabsf(v.z) + fabsf(v.w) < INFINITY);
        }
      odd = __any_sync(0xffffffffu, odd && ((any >> lane) & 1u));
      auto column = [&](int k) { return lane + 32 * (SHARED ? warp + kWarps * k : k); };
      auto add = [&](int x, auto checked) {  // four keys
        float4 pw[RW];
#pragma unroll
        for (int w = 0; w < RW; ++w) pw[w] = *reinterpret_cast<const float4 *>(&p_s[warp * RW + w][x]);
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          if (decltype(checked)::value && !((any >> (x + y)) & 1u)) continue;
#pragma unroll
          for (int k = 0; k < kCols; ++k) {
            if (SHARED && column(k) >= D) continue;
            const float v = v_s[x + y][column(k)];
#pragma unroll
            for (int w = 0; w < RW; ++w) {
              const float pj = y == 0 ? pw[w].x : y == 1 ? pw[w].y : y == 2 ? pw[w].z : pw[w].w;
              if (!decltype(checked)::value || !odd || !((hide[w] >> (x + y)) & 1u)) acc[w][k] = fmaf(pj, v, acc[w][k]);
            }
          }
        }
      };
      if (any == 0xffffffffu && hidden == 0u) {
#pragma unroll 2
        for (int x = 0; x < kKeys; x += 4) add(x, std::false_type{});
      } else {
#pragma unroll 1
        for (int x = 0; x < kKeys; x += 4)
          if (((any >> x) & 15u) != 0u) add(x, std::true_type{});
      }
    }
    copies_landed<0>();
    float(*o_s)[D] = v_s;  // this split's rows, when every warp is done with the values
    static_assert(kRows <= kKeys, "the rows take the values' place");
    if (merge_here) __syncthreads();
    // write this pass's rows
#pragma unroll
    for (int w = 0; w < RW; ++w) {
      const int r = rg + rw + w;
      if (r >= R) continue;
      const int i = r / G, g = r % G, h = kvh * G + g;
      const size_t qrow = (size_t)(row0 + i) * a.num_q_heads + h;
      const float inv = l[w] == 0.f ? 0.f : 1.f / l[w];  // a row that sees no key gets zeros
      const float lse = l[w] == 0.f ? -INFINITY : m[w] + log2f(l[w]);
      const size_t prow = (size_t)split * a.total_q * a.num_q_heads + qrow;
#pragma unroll
      for (int k = 0; k < kCols; ++k) {
        const int d = lane + 32 * (SHARED ? warp + kWarps * k : k);
        if (SHARED && d >= D) continue;
        if (nsplit == 1) reinterpret_cast<T *>(a.out)[qrow * D + d] = from_f32<T>(acc[w][k] * inv);
        else if (merge_here) o_s[rw + w][d] = acc[w][k] * inv;
        else a.ws_o[prow * D + d] = acc[w][k] * inv;
      }
      if (nsplit > 1 && lane == 0 && (!SHARED || warp == 0)) *(merge_here ? &lse_s[rw + w] : &a.ws_lse[prow]) = lse;
    }
    if (merge_here) {  // a row to a warp of the cluster, from every CTA's shared memory
      cg::cluster_group cluster = cg::this_cluster();
      cluster.sync();
      for (int x = split * kWarps + warp; x < min(kRows, R - rg); x += gridDim.x * kWarps) {
        const float lse = lane < nsplit ? *cluster.map_shared_rank(&lse_s[x], lane) : -INFINITY;
        const float M = warp_max(lse), wt = exp2f(lse - (M == -INFINITY ? 0.f : M)), den = warp_sum(wt);
        float num[NK];
#pragma unroll
        for (int k = 0; k < NK; ++k) num[k] = 0.f;
        for (int y = 0; y < nsplit; ++y) {
          const float *o = cluster.map_shared_rank(&o_s[x][0], y), wy = __shfl_sync(0xffffffffu, wt, y);
#pragma unroll
          for (int k = 0; k < NK; ++k) num[k] = fmaf(wy, o[lane + 32 * k], num[k]);
        }
        const int r = rg + x, i = r / G, h = kvh * G + r % G;
        T *op = reinterpret_cast<T *>(a.out) + ((size_t)(row0 + i) * a.num_q_heads + h) * D + lane;
#pragma unroll
        for (int k = 0; k < NK; ++k) op[32 * k] = from_f32<T>(den == 0.f ? 0.f : num[k] / den);
      }
      cluster.sync();  // the others' rows have been read
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

template <typename T, typename KT, int NK>
cudaError_t launch_n(const ScoredArgs &sa, cudaStream_t st) {
  const dim3 grid(sa.a.max_splits, sa.a.kv.num_kv_heads, sa.a.kv.batch);
  auto go = [&](auto kernel) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)sa.a.max_splits;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = sa.cluster ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, sa);
  };
  const long long rows = (long long)(sa.a.num_q_heads / sa.a.kv.num_kv_heads) * sa.a.max_q;
  if (rows <= 4) return go(attn_scored_simt_kernel<T, KT, NK, 4, true>);
  if constexpr (sizeof(KT) == 4)
    if (rows > 16) return go(attn_scored_simt_kernel<T, KT, NK, 8, false>);
  return go(attn_scored_simt_kernel<T, KT, NK, 4, false>);
}
template <typename T, typename KT>
cudaError_t launch_t(const ScoredArgs &sa, cudaStream_t st) {
  switch (sa.a.kv.head_dim / 32) {
    case 1: return launch_n<T, KT, 1>(sa, st);
    case 2: return launch_n<T, KT, 2>(sa, st);
    case 3: return launch_n<T, KT, 3>(sa, st);
    case 4: return launch_n<T, KT, 4>(sa, st);
    case 5: return launch_n<T, KT, 5>(sa, st);
    case 6: return launch_n<T, KT, 6>(sa, st);
    case 7: return launch_n<T, KT, 7>(sa, st);
    default: return launch_n<T, KT, 8>(sa, st);
  }
}

}  // namespace

cudaError_t launch_attn_scored_simt(const ScoredArgs &sa, int dtype, cudaStream_t st) {
  cudaError_t e;
  if (dtype == SV_DTYPE_E4M3) e = launch_t<__nv_bfloat16, uint8_t>(sa, st);  // bf16 queries and outputs
  else e = dtype == SV_DTYPE_BF16 ? launch_t<__nv_bfloat16, __nv_bfloat16>(sa, st) : launch_t<float, float>(sa, st);
  if (e != cudaSuccess || sa.a.max_splits <= 1 || sa.cluster) return e;
  const dim3 grid((unsigned)ceil_div(sa.a.max_q * sa.a.num_q_heads, kThreads / 32), (unsigned)sa.a.kv.batch);
  return dtype == SV_DTYPE_F32 ? launch_pdl(attn_scored_simt_combine<float>, grid, dim3(kThreads), 0, st, sa)
                               : launch_pdl(attn_scored_simt_combine<__nv_bfloat16>, grid, dim3(kThreads), 0, st, sa);
}

}  // namespace sv
