// Head norms and position rotation of query and key rows, alone (sv_qk_norm_rope) or on the
// way into the paged cache (sv_kv_append_rope, after kv_alloc_kernel has taken the blocks).
//
// For a head x of D values, its norm weight w (if given) and its row's position p:
//   y_e = x_e * rsqrt(mean_e x_e^2 + eps) * (w_e + offset)              (y = x without a weight)
//   (a, b) -> (a cos t - b sin t, b cos t + a sin t),  t = p * inv_freq[i]  (p: on pair i's axis, if there are several),
// over the pairs i < rot / 2 of y: (y_i, y_{i + rot/2}), or (y_2i, y_2i+1) when interleaved. All
// of it in fp32 and one rounding at the end, to the output's type (for an E4M3 pool straight from
// fp32 to the code nearest to y / scale: rounding to bf16 on the way would round twice; into an E2M1 pool as in
// e2m1.cuh, two neighbouring lanes to a scale). The
// angle is the product of the position and the fp32 frequency as a 64-bit fraction of a turn, rounded
// once to fp32 (see turn): a product in fp32 would be off by 4e-3 at position 10^5.
//
// A lane holds 8 consecutive values of a head, a group of pow2ceil(D / 8) lanes a head, a warp
// 32 / group heads at a time (an iteration). A warp's item is a chunk of one row's iterations, queries,
// keys and values in turn, and needs no other warp: it makes a (cos, sin) table of the row and folds it
// with the norm's weights into two factors per value, once per kind of head, so that a head costs
//   out_j = r (x_j A_j + x'_j B_j),  A = cos * w,  B = +-sin * w',  r = rsqrt(mean x^2 + eps)
// with x' the pair's other value and w' its weight: a shuffle of the row's packed words away (rot a
// multiple of 16), in the same lane (interleaved, rot a multiple of 8), or exchanged through
// shared memory (the kernel for other sizes of heads and rotations).
//
// Bound: memory, every value read once and written once; next to it the issue of instructions (some
// 80 an iteration of 512 bytes), which is why the head size is a template parameter where it is 64,
// 128 or 256 and nothing but shuffles, products and conversions is left in the loop. Long
// batches take whole rows as items; short ones are cut, evenly, until every resident warp has a chunk.
// Short calls are latency: a launch, then the chain of reads that finds a row's place.
//
// bf16, 32 + 8 heads of 128 values: 16384 rows 60.1 us (5.6 TB/s of rows), 4 rows 3.5 us; 640 rows of 64 + 8
// heads 6.2 us. With the append: 256 x 64 rows 77.3 us (5.2 TB/s), 32 x 6 rows 6.2 us, 1.5K rows into an E4M3
// pool 15.1 us; 256 x 64 into E4M3 and E2M1 pools 77.8 and 79.3 us, 32 x 6 rows 6.2 and 6.4. With three axes 16384 rows take
// 60.3 us, 4 rows 4.4 us, 256 x 64 appended 78.8, 79.1 and 80.6 (bf16, E4M3, E2M1); in fp32 16384 rows 105 us (6.4 TB/s), 4 rows 3.0.
#include <cuda_fp8.h>

#include <algorithm>

#include "e2m1.cuh"
#include "kv_rows.cuh"

namespace sv {
namespace {

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

// 8 fp32 values -> E4M3 codes of x / scale (fp32 division; nearest, ties to even; saturating). inv: 1 / scale
// where that is exact (a power of two, the division's result bit for bit), else 0.
__device__ __forceinline__ uint2 quantize8(const float (&x)[8], float scale, float inv) {
  uint32_t w[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    w[q] = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float x0 = x[4 * q + 2 * h], x1 = x[4 * q + 2 * h + 1];
      const float2 v = inv != 0.f ? make_float2(x0 * inv, x1 * inv) : make_float2(__fdiv_rn(x0, scale), __fdiv_rn(x1, scale));
      w[q] |= (uint32_t)__nv_cvt_float2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3) << (16 * h);
    }
  }
  return make_uint2(w[0], w[1]);
}

// cos and sin of position * freq. A turn is 2^64: freq = M 2^E turns by M 2^E / (2 pi) per position, the
// product of M with the first 64 bits of 2^66 / (2 pi), shifted; times the position it wraps exactly.
// The cut digits of 1 / (2 pi) leave a position's turn off by |freq| / 4 units of 2^-64 and the shift by one more, so
// the whole by |position| (1 + |freq| / 4) 2^-64 turns (2^-33 at position 2^31); its upper 32 bits, which leave out 2^-32 of a
// turn, are rounded to fp32 and go to sincospif.
__device__ __forceinline__ float2 turn(int position, float freq) {
  const uint32_t bits = __float_as_uint(freq);
  const int e = (bits >> 23) & 255;
  const unsigned long long m = (bits & 0x7fffffu) | (e ? 0x800000u : 0u), k = 0xa2f9836e4e44152aull;
  const unsigned long long hi = __umul64hi(m, k), lo = m * k;
  const int s = 152 - (e ? e : 1);  // 2 - E
  unsigned long long per = s >= 64 ? (s < 128 ? hi >> (s - 64) : 0ull)
                                   : s > 0 ? (hi << (64 - s)) | (lo >> s) : (s > -64 ? lo << -s : 0ull);
  if (bits >> 31) per = 0ull - per;
  const unsigned long long f = (unsigned long long)(long long)position * per;
  if (e == 255) return make_float2(__int_as_float(0x7fffffff), __int_as_float(0x7fffffff));  // no angle: NaN
  float sn, cs;
  sincospif((float)(int)(f >> 32) * 4.656612873077393e-10f /* 2^-31 */, &sn, &cs);
  return make_float2(cs, sn);
}

constexpr int kThreads = 128;
// Warps in residence against loads in flight (16384 rows; 256 x 64 appended): 5 CTAs an SM with 5 iterations ahead
// 69 and 86 us, 6 with 4 63 and 78, 7 with 4 60 and 77, 7 with 3 65 and 83, 8 with 4 (spilling) 61 and 82.
constexpr int kCtasPerSm = 7;

// The pair's other values x' of a lane's 8.
template <typename T> __device__ __forceinline__ void from_lane(const Vec8<T> &x, int lane, float (&p)[8]);
template <> __device__ __forceinline__ void from_lane(const Vec8<__nv_bfloat16> &x, int lane, float (&p)[8]) {
  Vec8<__nv_bfloat16> y;
  y.r.x = __shfl_sync(0xffffffffu, x.r.x, lane);
  y.r.y = __shfl_sync(0xffffffffu, x.r.y, lane);
  y.r.z = __shfl_sync(0xffffffffu, x.r.z, lane);
  y.r.w = __shfl_sync(0xffffffffu, x.r.w, lane);
  y.get(p);
}
template <> __device__ __forceinline__ void from_lane(const Vec8<float> &x, int lane, float (&p)[8]) {
  float v[8];
  x.get(v);
#pragma unroll
  for (int j = 0; j < 8; ++j) p[j] = __shfl_sync(0xffffffffu, v[j], lane);
}

enum Pairs { kShuffle, kInLane, kExchange };  // where a value's pair is

// APPEND: keys and values go to the cache (kv, cu_q, status); else keys go to k_out. DIM: the head
// size, or 0: any (with PAIRS == kExchange). F4: an E2M1 pool. A warp takes chunk x % chunks of row x / chunks.
template <typename T, bool APPEND, int PAIRS, int DIM, bool F4>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) head_rows_kernel(const HeadArgs a, int chunks, int per_chunk,
                                                                         long long items) {
  constexpr int kAhead = sizeof(T) == 2 ? 4 : 2;  // iterations whose loads are in flight together
  constexpr int kEsz = sizeof(T);
  __shared__ float2 s_turn[kThreads / 32][128];
  __shared__ float s_swap[PAIRS == kExchange ? kThreads / 32 : 1][32 * 8];
  if (!APPEND) {
    // what follows on the stream may read the rows before its own dependency wait: this kernel
    // lets it start only when it is complete (no grid_dependents_launch)
    grid_dependency_wait();
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int dim = DIM ? DIM : a.head_dim, per_head = dim >> 3;  // lanes that hold a head
  const int gsh = DIM == 64 ? 3 : DIM == 128 ? 4 : DIM == 256 ? 5 : 31 - __clz(2 * per_head - 1);
  const int gl = 1 << gsh, hpw = 32 >> gsh;  // lanes of a head's group, heads of an iteration
  const int place = lane & (gl - 1), sub = lane >> gsh;
  const bool holds = DIM != 0 || place < per_head;
  const int nq = (a.hq + hpw - 1) / hpw, nk = (a.hkv + hpw - 1) / hpw;
  const int all = nq + nk + (APPEND ? nk : 0);  // iterations of a row
  const int half = a.rot >> 1, hl = half >> 3;
  const long long item = (long long)blockIdx.x * (kThreads / 32) + warp;
  const int row = (int)(item / chunks), i0 = (int)(item - (long long)row * chunks) * per_chunk, i1 = min(all, i0 + per_chunk);
  if (item >= items || i0 >= i1) {
    if (APPEND) grid_dependency_wait();  // completion stays transitive along the stream
    return;
  }
  // The rows, weights, frequencies, positions, cu_q and lengths are complete before this kernel
  // starts: the append's kernel ahead of it writes none of them and let it launch only after its own
  // dependency wait. What that kernel writes is read after the wait below.
  const size_t in_head = (size_t)sub * dim + place * 8;  // this lane's values of an iteration
  const uint8_t *in_q = a.q + (size_t)row * a.q_stride + in_head * kEsz;
  const uint8_t *in_k = a.k + (size_t)row * a.k_stride + in_head * kEsz;
  const uint8_t *in_v = APPEND ? a.v + (size_t)row * a.v_stride + in_head * kEsz : nullptr;
  const int step = hpw * dim;  // values of an iteration
  Vec8<T> x[kAhead];
  // iterations [it, it + kAhead) of a kind that begins at iteration `first` and ends before `end`
  auto load = [&](const uint8_t *in, int count, int it, int end, int first) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int k = it + u - first;
      if (it + u < end && holds && k * hpw + sub < count) x[u].load(in + (size_t)k * step * kEsz);
      else x[u].zero();
    }
  };
  const int kind0 = i0 < nq ? 0 : i0 < nq + nk ? 1 : 2;
  load(kind0 == 0 ? in_q : kind0 == 1 ? in_k : in_v, kind0 == 0 ? a.hq : a.hkv, i0,
       min(i1, kind0 == 0 ? nq : kind0 == 1 ? nq + nk : all), kind0 == 0 ? 0 : kind0 == 1 ? nq : nq + nk);
  int b = 0, i = 0, n = 1, c = 0;
  if (APPEND) {
    b = owner_of(a.cu_q, a.kv.batch, row);
    const int row0 = a.cu_q[b];
    i = row - row0;
    n = a.cu_q[b + 1] - row0;
    c = a.kv.seq_lens[b];
  }
  if (kind0 < 2 && half > 0) {
    if (a.axes > 1 && a.positions != nullptr) {
      for (int e = lane; e < half; e += 32) s_turn[warp][e] = turn(a.positions[(size_t)a.axis[e] * a.rows + row], a.inv_freq[e]);
    } else {
      const int pos = a.positions != nullptr ? a.positions[row] : c + i;
      for (int e = lane; e < half; e += 32) s_turn[warp][e] = turn(pos, a.inv_freq[e]);
    }
    __syncwarp();
  }
  uint8_t *out[3] = {a.q_out + (size_t)row * a.q_out_stride + in_head * kEsz,
                     APPEND ? nullptr : a.k_out + (size_t)row * a.k_out_stride + in_head * kEsz, nullptr};
  size_t out_step[2] = {(size_t)step * kEsz, (size_t)step * kEsz};  // of an iteration: queries; keys and values
  size_t scale_at = 0, scale_step = 0;                              // F4: of the lane's block scale
  if (APPEND) {
    grid_dependency_wait();
    grid_dependents_launch();
    if (status_set(a.status)) return;
    if (i < 0 || i >= n) return;  // rows past cu_q[batch]: nothing to write
    const int at = c + i, bsh = __ffs(a.kv.block_size) - 1;
    const int blk = a.kv.block_table[(size_t)b * a.kv.max_blocks + (at >> bsh)];
    if (blk < 0 || blk >= a.kv.num_blocks) {
      if (lane == 0) record(a.status, SV_ERR_BAD_BLOCK_ID);
      return;
    }
    const int eb = a.kv.elem_bytes;
    const size_t value = ((((size_t)blk * a.hkv + sub) << bsh) + (at & (a.kv.block_size - 1))) * dim + place * 8;
    const size_t off = F4 ? value / 2 : value * eb;
    out[1] = reinterpret_cast<uint8_t *>(a.kv.k_pool) + off;
    out[2] = reinterpret_cast<uint8_t *>(a.kv.v_pool) + off;
    out_step[1] = F4 ? ((size_t)hpw * dim << bsh) / 2 : ((size_t)hpw * dim << bsh) * eb;
    scale_at = value / 16;
    scale_step = ((size_t)hpw * dim << bsh) / 16;
  }

  const int other = place < hl ? place + hl : place < 2 * hl ? place - hl : place;  // the pair's place (kShuffle)
  const bool turned = PAIRS == kExchange || place * 8 < a.rot;                      // this lane's values are rotated
#pragma unroll
  for (int kind = 0; kind < (APPEND ? 3 : 2); ++kind) {
    const int first = kind == 0 ? 0 : kind == 1 ? nq : nq + nk;
    const int lo = max(i0, first), end = min(i1, kind == 0 ? nq : kind == 1 ? nq + nk : all);
    if (lo >= end) continue;  // uniform
    const int count = kind == 0 ? a.hq : a.hkv;
    const uint8_t *weight = kind == 0 ? a.q_weight : a.k_weight;
    float A[8], Bf[8];   // the kind's factors
    uint32_t turns = 0;  // kExchange: bit j: value j is rotated
    if (kind < 2) {
      float w[8], wo[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = wo[j] = 1.f;
      if (weight != nullptr && holds) {
        Vec8<T> v;
        v.load(weight + place * 8 * kEsz);
        v.get(w);
        if (PAIRS == kShuffle) {
          v.load(weight + other * 8 * kEsz);
          v.get(wo);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int e = place * 8 + j, o = a.interleaved ? e ^ 1 : e < half ? e + half : e - half;
            if (PAIRS == kInLane) wo[j] = w[j ^ 1];
            else if (e < a.rot) wo[j] = to_f32(reinterpret_cast<const T *>(weight)[o]);
          }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          w[j] += a.offset;
          wo[j] += a.offset;
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int e = place * 8 + j;
        A[j] = w[j];
        Bf[j] = 0.f;
        if (e < a.rot) {
          const bool lower = PAIRS == kInLane || (PAIRS == kExchange && a.interleaved) ? (j & 1) == 0 : e < half;
          const bool pairs2 = PAIRS == kInLane || (PAIRS == kExchange && a.interleaved);
          const float2 t = s_turn[warp][pairs2 ? e >> 1 : (lower ? e : e - half)];
          A[j] = t.x * w[j];
          Bf[j] = lower ? -t.y * wo[j] : t.y * wo[j];
          turns |= 1u << j;
        }
      }
    }
    for (int it = lo; it < end; it += kAhead) {
      // (the item's first loads are on their way since its start)
      if (it > i0) load(kind == 0 ? in_q : kind == 1 ? in_k : in_v, count, it, end, first);
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        if (it + u >= end) break;  // uniform
        const int k = it + u - first;
        float y[8];
        if (kind < 2 || a.kv.fp8 || F4) x[u].get(y);
        if (kind < 2) {
          float r = 1.f;
          if (weight != nullptr) {
            float ss = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = fmaf(y[j], y[j], ss);
            if (DIM) {
#pragma unroll
              for (int o = 1; o < DIM / 8; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            } else {
              for (int o = 1; o < gl; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            }
            r = rsqrtf(ss * a.inv_dim + a.eps);
          }
          float p[8];
          if (PAIRS == kShuffle) {
            from_lane(x[u], (lane & ~(gl - 1)) + other, p);
          } else if (PAIRS == kInLane) {
#pragma unroll
            for (int j = 0; j < 8; ++j) p[j] = y[j ^ 1];
          } else {
            float *sw = s_swap[warp];
#pragma unroll
            for (int j = 0; j < 8; ++j) sw[lane * 8 + j] = y[j];
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const int e = place * 8 + j, o = a.interleaved ? e ^ 1 : e < half ? e + half : e - half;
              p[j] = sw[(lane & ~(gl - 1)) * 8 + ((turns >> j) & 1u ? o : e)];
            }
            __syncwarp();
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const bool rotate = PAIRS == kExchange ? ((turns >> j) & 1u) != 0 : turned;
            y[j] = r * (rotate ? fmaf(p[j], Bf[j], y[j] * A[j]) : y[j] * A[j]);
          }
        }
        float top = 0.f;  // F4: the largest of the lane's and its neighbour's values
        if (F4 && kind > 0) {
          top = top_of(y);
          top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, 1));
        }
        if (!holds || k * hpw + sub >= count) continue;
        // the output, rounded once
        uint8_t *dst = out[kind] + (size_t)k * out_step[kind > 0];
        if (F4 && kind > 0) {
          const uint32_t s = block_scale(top, kind == 2 ? a.v_inv : a.k_inv);
          *reinterpret_cast<uint32_t *>(dst) = codes8(y, code_factor(s, kind == 2 ? a.kv.v_scale : a.kv.k_scale));
          if ((place & 1) == 0) (kind == 2 ? a.kv.v_bs : a.kv.k_bs)[scale_at + (size_t)k * scale_step] = (uint8_t)s;
        } else if (APPEND && kind > 0 && a.kv.fp8) {
          *reinterpret_cast<uint2 *>(dst) = quantize8(y, kind == 2 ? a.kv.v_scale : a.kv.k_scale, kind == 2 ? a.v_inv : a.k_inv);
        } else {
          if (kind < 2) x[u].set(y);  // values are copied as they are
          x[u].store(dst);
        }
      }
    }
  }
}

template <typename T, bool APPEND, bool F4 = false>
cudaError_t launch_rows(const HeadArgs &a, int total_q, cudaStream_t st) {
  int gl = 1;
  while (gl < a.head_dim / 8) gl *= 2;
  const int hpw = 32 / gl, nk = ceil_div(a.hkv, hpw);
  const int all = ceil_div(a.hq, hpw) + nk * (APPEND ? 2 : 1);
  // as many iterations an item as give every resident warp one, whole rows at most
  const long long warps = (long long)num_sms() * kCtasPerSm * (kThreads / 32);
  const int most = (int)std::min<long long>(all, ((long long)all * total_q + warps - 1) / warps);
  const int chunks = ceil_div(all, most), per_chunk = ceil_div(all, chunks);
  const long long items = (long long)total_q * chunks;
  const unsigned ctas = (unsigned)((items + kThreads / 32 - 1) / (kThreads / 32));
  auto go = [&](auto kernel) { return launch_pdl(kernel, dim3(ctas), dim3(kThreads), 0, st, a, chunks, per_chunk, items); };
  const int d = a.head_dim;
  if (d == 64 || d == 128 || d == 256) {
    if (!a.interleaved && a.rot % 16 == 0)
      return d == 64 ? go(head_rows_kernel<T, APPEND, kShuffle, 64, F4>) : d == 128 ? go(head_rows_kernel<T, APPEND, kShuffle, 128, F4>)
                                                                                   : go(head_rows_kernel<T, APPEND, kShuffle, 256, F4>);
    if (a.interleaved && a.rot % 8 == 0)
      return d == 64 ? go(head_rows_kernel<T, APPEND, kInLane, 64, F4>) : d == 128 ? go(head_rows_kernel<T, APPEND, kInLane, 128, F4>)
                                                                                  : go(head_rows_kernel<T, APPEND, kInLane, 256, F4>);
  }
  return go(head_rows_kernel<T, APPEND, kExchange, 0, F4>);
}

// One CTA per sequence whose first new row lands in a private copy of a shared block.
__global__ void __launch_bounds__(256) kv_private_copy_kernel(KV kv, const int32_t *cu_q, int32_t *status) {
  grid_dependency_wait();  // the allocation is complete and visible
  grid_dependents_launch();
  if (status_set(status)) return;
  const int b = blockIdx.x, c = kv.seq_lens[b], slot = c % kv.block_size;
  if (cu_q[b + 1] - cu_q[b] < 1 || slot == 0) return;
  const int blk = kv.block_table[(size_t)b * kv.max_blocks + c / kv.block_size];
  if (blk < 0 || blk >= kv.num_blocks) return;  // the rows' kernel reports it
  copy_shared_block(kv, blk, slot, kv.row_bytes, status);
}

}  // namespace

cudaError_t launch_private_copies(const KV &kv, const int32_t *cu_q, int32_t *status, cudaStream_t st) {
  return launch_pdl(kv_private_copy_kernel, dim3(kv.batch), dim3(256), 0, st, kv, cu_q, status);
}

cudaError_t launch_head_rows(const HeadArgs &a, int dtype, int total_q, bool append, cudaStream_t st) {
  if (append && a.kv.ref_count != nullptr) {
    const cudaError_t e = launch_private_copies(a.kv, a.cu_q, a.status, st);
    if (e != cudaSuccess) return e;
  }
  if (append && a.kv.fp4) return launch_rows<__nv_bfloat16, true, true>(a, total_q, st);
  if (dtype == SV_DTYPE_F32) return append ? launch_rows<float, true>(a, total_q, st) : launch_rows<float, false>(a, total_q, st);
  return append ? launch_rows<__nv_bfloat16, true>(a, total_q, st) : launch_rows<__nv_bfloat16, false>(a, total_q, st);
}

}  // namespace sv
