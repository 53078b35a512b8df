// Head norms and position rotation of query and key rows, alone (sv_qk_norm_rope) or on the
// way into the paged cache (sv_kv_append_rope, after kv_alloc_kernel has taken the blocks).
//
// For a head x of D values, its norm weight w (if given) and its row's position p:
//   y_e = x_e * rsqrt(mean_e x_e^2 + eps) * (w_e + offset)              (y = x without a weight)
//   (a, b) -> (a cos t - b sin t, b cos t + a sin t),  t = p * inv_freq[i],
// over the pairs i < rot / 2 of y: (y_i, y_{i + rot/2}), or (y_2i, y_2i+1) when interleaved. All
// of it in fp32 and one rounding at the end, to the output's type (for an E4M3 pool straight from
// fp32 to the code nearest to y / scale: rounding to bf16 on the way would round twice). The
// angle is the exact product of the position and the fp32 frequency up to one rounding in fp64,
// reduced to a fraction of a turn there: in fp32 the angle of position 10^5 would be off by 4e-3.
//
// A CTA takes one row. A lane holds 8 consecutive values of a head, a group of pow2ceil(D / 8)
// lanes a head, so a row's heads are slots of a group each, spread over the CTA's warps. A
// thread's place in its head is the same in all its slots, so its 8 weights (query and key) and
// its 8 (cos, sin) are loaded once. The sum of squares is a butterfly over the group; the
// rotation's partners are a shuffle away (rot a multiple of 16), in the same lane (interleaved),
// or exchanged through shared memory.
//
// The work is bound by memory: every value is read once and written once.
#include <cuda_fp8.h>

#include "kv_rows.cuh"

namespace sv {
namespace {

constexpr int kSlotsAhead = 4;  // slots of a thread whose loads are in flight together

template <typename T> struct Vec8;  // 8 values of a row as loaded
template <> struct Vec8<__nv_bfloat16> {
  uint4 r;
  __device__ __forceinline__ void load(const uint8_t *p) { r = *reinterpret_cast<const uint4 *>(p); }
  __device__ __forceinline__ void store(uint8_t *p) const { *reinterpret_cast<uint4 *>(p) = r; }
  __device__ __forceinline__ void zero() { r = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      x[2 * k] = __uint_as_float(w[k] << 16);
      x[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
    }
  }
  __device__ __forceinline__ void set(const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * k], x[2 * k + 1]);
      w[k] = *reinterpret_cast<const uint32_t *>(&v);
    }
    r = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <> struct Vec8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const uint8_t *p) {
    a = reinterpret_cast<const float4 *>(p)[0];
    b = reinterpret_cast<const float4 *>(p)[1];
  }
  __device__ __forceinline__ void store(uint8_t *p) const {
    reinterpret_cast<float4 *>(p)[0] = a;
    reinterpret_cast<float4 *>(p)[1] = b;
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
  __device__ __forceinline__ void set(const float (&x)[8]) {
    a = make_float4(x[0], x[1], x[2], x[3]);
    b = make_float4(x[4], x[5], x[6], x[7]);
  }
};

// 8 fp32 values -> E4M3 codes of x / scale (fp32 division; nearest, ties to even; saturating)
__device__ __forceinline__ uint2 quantize8(const float (&x)[8], float scale) {
  uint32_t w[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    w[q] = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float2 v = make_float2(__fdiv_rn(x[4 * q + 2 * h], scale), __fdiv_rn(x[4 * q + 2 * h + 1], scale));
      w[q] |= (uint32_t)__nv_cvt_float2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3) << (16 * h);
    }
  }
  return make_uint2(w[0], w[1]);
}

// cos and sin of position * freq
__device__ __forceinline__ float2 turn(int position, float freq) {
  const double turns = (double)position * (double)freq * 0.15915494309189535;  // radians / (2 pi)
  float s, c;
  sincospif((float)(2.0 * (turns - rint(turns))), &s, &c);
  return make_float2(c, s);
}

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

// APPEND: keys and values go to the cache (kv, cu_q, status); else keys go to k_out.
template <typename T, bool APPEND>
__global__ void __launch_bounds__(256) head_rows_kernel(const HeadArgs a) {
  __shared__ float2 s_turn[128];     // (cos, sin) of the row's angles
  __shared__ float s_swap[8][32 * 8];  // partners that neither a shuffle nor the lane itself holds
  if (!APPEND) {
    // what follows on the stream may read the rows before its own dependency wait: this kernel
    // lets it start only when it is complete (no grid_dependents_launch)
    grid_dependency_wait();
  }
  const int row = blockIdx.x;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per_head = a.head_dim >> 3;  // lanes that hold a head
  const int gsh = 31 - __clz(2 * per_head - 1), gl = 1 << gsh;  // lanes of a head's group
  const int place = lane & (gl - 1);     // this thread's 8 values of a head
  const bool holds = place < per_head;
  const int heads = a.hq + a.hkv * (APPEND ? 2 : 1);  // queries, keys, values
  const int groups = blockDim.x >> gsh;
  const int group = threadIdx.x >> gsh;
  const size_t esz = sizeof(T);
  const uint8_t *qrow = a.q + (size_t)row * a.q_stride;
  const uint8_t *krow = a.k + (size_t)row * a.k_stride;
  const uint8_t *vrow = a.v + (size_t)row * a.v_stride;
  auto src = [&](int h) -> const uint8_t * {
    const uint8_t *base = h < a.hq ? qrow + (size_t)h * a.head_dim * esz
                          : h < a.hq + a.hkv ? krow + (size_t)(h - a.hq) * a.head_dim * esz
                                             : vrow + (size_t)(h - a.hq - a.hkv) * a.head_dim * esz;
    return base + (size_t)place * 8 * esz;
  };
  // The rows, weights, frequencies, positions, cu_q and (append) lengths are complete before this
  // kernel starts: kv_alloc_kernel, the one ahead of it, writes none of them and let it launch
  // only after its own dependency wait. What that kernel writes is read after the wait below.
  Vec8<T> x[kSlotsAhead];
#pragma unroll
  for (int u = 0; u < kSlotsAhead; ++u) {
    const int h = group + u * groups;
    if (h < heads && holds) x[u].load(src(h));
    else x[u].zero();
  }
  int b = 0, i = 0, n = 1, c = 0, pos = 0;
  if (APPEND) {
    b = owner_of(a.cu_q, a.kv.batch, row);
    const int row0 = a.cu_q[b];
    i = row - row0;
    n = a.cu_q[b + 1] - row0;
    c = a.kv.seq_lens[b];
  }
  if (a.positions != nullptr) pos = a.positions[row];
  else pos = c + i;
  const int half = a.rot >> 1;
  for (int e = threadIdx.x; e < half; e += blockDim.x) s_turn[e] = turn(pos, a.inv_freq[e]);
  Vec8<T> qw, kw;
  qw.zero();
  kw.zero();
  if (holds && a.q_weight != nullptr) qw.load(a.q_weight + (size_t)place * 8 * esz);
  if (holds && a.k_weight != nullptr) kw.load(a.k_weight + (size_t)place * 8 * esz);
  __syncthreads();
  // this thread's values of a head: value j turns by (cs[j], sn[j]), sn with the sign its partner takes
  float cs[8], sn[8];
  uint32_t turns = 0;  // bit j: value j is rotated
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int e = place * 8 + j;
    cs[j] = 1.f;
    sn[j] = 0.f;
    if (e < a.rot) {
      const bool first = a.interleaved ? (e & 1) == 0 : e < half;
      const float2 t = s_turn[a.interleaved ? e >> 1 : (first ? e : e - half)];
      cs[j] = t.x;
      sn[j] = first ? -t.y : t.y;
      turns |= 1u << j;
    }
  }
  const bool by_shuffle = !a.interleaved && (half & 7) == 0;
  const int hl = half >> 3;
  const int partner = (lane & ~(gl - 1)) + (place < hl ? place + hl : place < 2 * hl ? place - hl : place);

  int blk = 0, slot = 0;
  bool write = true;
  if (APPEND) {
    grid_dependency_wait();
    grid_dependents_launch();
    if (status_set(a.status)) return;
    if (i < 0 || i >= n) return;  // rows past cu_q[batch]: nothing to write
    const int at = c + i;
    blk = a.kv.block_table[(size_t)b * a.kv.max_blocks + at / a.kv.block_size];
    if (blk < 0 || blk >= a.kv.num_blocks) {
      if (threadIdx.x == 0) record(a.status, SV_ERR_BAD_BLOCK_ID);
      return;
    }
    slot = at % a.kv.block_size;
    if (i == 0 && slot > 0 && a.kv.ref_count != nullptr)
      copy_shared_block(a.kv, blk, slot, a.kv.head_dim * a.kv.elem_bytes, a.status);
  }

  for (int base = 0; base < heads; base += kSlotsAhead * groups) {
    if (base > 0) {
#pragma unroll
      for (int u = 0; u < kSlotsAhead; ++u) {
        const int h = base + group + u * groups;
        if (h < heads && holds) x[u].load(src(h));
        else x[u].zero();
      }
    }
#pragma unroll
    for (int u = 0; u < kSlotsAhead; ++u) {
      const int h = base + group + u * groups;
      if (base + u * groups >= heads) break;  // uniform: no thread has this slot
      write = h < heads && holds;
      const bool is_q = h < a.hq, is_v = h >= a.hq + a.hkv;
      float y[8];
      x[u].get(y);
      // the norm
      const bool norm = is_q ? a.q_weight != nullptr : (!is_v && a.k_weight != nullptr);
      float ss = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(y[j], y[j], ss);
      for (int o = gl >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (norm) {
        const float r = rsqrtf(ss * a.inv_dim + a.eps);
        float w[8];
        if (is_q) qw.get(w);
        else kw.get(w);
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = y[j] * r * (w[j] + a.offset);
      }
      // the rotation
      float p[8];
      if (by_shuffle) {
#pragma unroll
        for (int j = 0; j < 8; ++j) p[j] = __shfl_sync(0xffffffffu, y[j], partner);
      } else if (a.interleaved) {
#pragma unroll
        for (int j = 0; j < 8; ++j) p[j] = y[j ^ 1];
      } else {
        float *sw = s_swap[warp];
#pragma unroll
        for (int j = 0; j < 8; ++j) sw[lane * 8 + j] = y[j];
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int e = place * 8 + j;
          const int q = e < half ? e + half : e < a.rot ? e - half : e;
          p[j] = sw[(lane & ~(gl - 1)) * 8 + q];
        }
        __syncwarp();
      }
      if (!is_v) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if ((turns >> j) & 1u) y[j] = fmaf(y[j], cs[j], p[j] * sn[j]);
      }
      if (!write) continue;
      // the output, rounded once
      if (is_q) {
        x[u].set(y);
        x[u].store(a.q_out + (size_t)row * a.q_out_stride + ((size_t)h * a.head_dim + place * 8) * esz);
      } else if (!APPEND) {
        x[u].set(y);
        x[u].store(a.k_out + (size_t)row * a.k_out_stride + ((size_t)(h - a.hq) * a.head_dim + place * 8) * esz);
      } else {
        const int kvh = is_v ? h - a.hq - a.hkv : h - a.hq;
        const size_t at =
            (((size_t)blk * a.hkv + kvh) * a.kv.block_size + slot) * a.head_dim + (size_t)place * 8;  // value in the pool
        uint8_t *pool = reinterpret_cast<uint8_t *>(is_v ? a.kv.v_pool : a.kv.k_pool);
        if (a.kv.fp8) {
          *reinterpret_cast<uint2 *>(pool + at) = quantize8(y, is_v ? a.kv.v_scale : a.kv.k_scale);
        } else {
          if (!is_v) x[u].set(y);  // values are copied as they are
          x[u].store(pool + at * esz);
        }
      }
    }
  }
}

template <typename T, bool APPEND>
cudaError_t launch_rows(const HeadArgs &a, int total_q, cudaStream_t st) {
  int gl = 1;
  while (gl < a.head_dim / 8) gl *= 2;
  const int lanes = (a.hq + a.hkv * (APPEND ? 2 : 1)) * gl;
  int threads = 64;
  while (threads < 256 && threads * (kSlotsAhead - 1) < lanes) threads *= 2;
  return launch_pdl(head_rows_kernel<T, APPEND>, dim3((unsigned)total_q), dim3(threads), 0, st, a);
}

}  // namespace

cudaError_t launch_head_rows(const HeadArgs &a, int dtype, int total_q, bool append, cudaStream_t st) {
  if (dtype == SV_DTYPE_F32) return append ? launch_rows<float, true>(a, total_q, st) : launch_rows<float, false>(a, total_q, st);
  return append ? launch_rows<__nv_bfloat16, true>(a, total_q, st) : launch_rows<__nv_bfloat16, false>(a, total_q, st);
}

}  // namespace sv
