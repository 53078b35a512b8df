// Attention with modified scores (sv_spec_verify_attn_scored) over bf16 and E4M3 caches, with
// warp-level matrix instructions; instantiated per head size in attn_scored_d*.cu.
//
// The mathematics (base-2 exponents; p_t the position of key t, c the committed tokens):
//   s_t = cap tanh(scale <q, k_t> / cap) + slope (p_t - c),   o = sum_t 2^(s_t - m) v_t / sum_t 2^(s_t - m)
// with everything in units of log2. The distance bias -slope (p_i - p_t) differs from the term above
// by a constant of the row, which the softmax cancels: a key's term is the same for all rows of a head.
// tanh(y) = 1 - 2 / (1 + 2^(2 y log2 e)): two special-function instructions; its absolute error,
// about 2^-22, times the cap is what reaches a score (caps above kFastCap take tanhf).
//
// Bound: memory. A verify step's unit (one KV head of one sequence) has G n_b query rows, 1 to some
// 40: at 4 flops per row and value of K and V that is far below the card's ratio of flops to bytes,
// so the kernel is built to keep loads in flight; the matrix instructions of a warp, without tensor
// memory and its hand-offs, leave time to spare at these row counts. (128 query rows and more per
// unit are bound by the products.)
//
// Work: as many CTAs as fit the GPU stay for the whole launch. The key tiles of all units laid end
// to end (each unit preceded by `alpha` positions, what starting and finishing one costs) are cut
// into equal contiguous ranges, one per CTA. A unit that one CTA holds whole is written by it; a
// shared one leaves a normalised partial and its log-sum-exp in one of the CTA's two slots, and
// attn_scored_combine merges the partials in the order of the CTAs (so results repeat bit for bit).
// With a window a unit's tiles start at its first visible one: keys out of sight are not read.
//
// A CTA's four warps are WK key groups x WR row groups. Every tile of TK keys goes into a ring of
// kStages shared-memory stages by TMA, a box per block (or per tile, where blocks are larger), the pool
// seen as (128 bytes, 8 rows, 128-byte parts of a row, groups of 8 rows) and swizzled so that
// ldmatrix reads without bank conflicts. The warps take turns in issuing a tile, each a turn after it has
// read the block ids; a stage is refilled when all four have arrived on its barrier, so that no
// barrier of the whole CTA is left in the loop. A warp takes 16 keys at a time:
//   S^T (keys x rows) = K Q^T, A = K (ldmatrix), B = Q held in registers, accumulators fp32;
//   the running maximum of a row moves only when a score passes it by 2^8 (one vote per 16 keys), and
//   not at all where the cap bounds the scores well enough (kBoundedCap);
//   P^T = 2^(S^T - m) in bf16 (fp16 for E4M3 pools) turned into a B operand by movmatrix;
//   O^T (dims x rows) += V^T P^T, A = V^T (ldmatrix.trans), accumulators fp32 in registers.
// Query rows sit on the n dimension, so that 24 rows (4 heads x 6) cost 24 and not 32. At the end
// of a piece the WK key groups' (m, l, O) are merged through shared memory.
//
// A cap's constant term is dropped like the bias's: -2 cap / (1 + 2^(2 y log2 e)) is what is left.
// E4M3 codes become fp16 operands in registers (exactly). ldmatrix moves pairs of codes; which
// dimension lands at which place of the operand differs from the bf16 form, and Q's registers and O's
// columns follow it.
//
// All mbarrier waits are bounded: after one that gives up, a warp goes through the rest of its work
// without waiting (on whatever the stages hold) and the call records SV_ERR_TIMEOUT.
#pragma once

#include <cuda.h>
#include <cuda_fp16.h>

#include "sv_internal.cuh"

namespace sv {
namespace scored {

constexpr int kThreads = 128;
constexpr float kMoveAt = 8.f;     // the running maximum moves when a score passes it by this (log2)
constexpr float kFastCap = 200.f;  // caps up to this take the two-instruction tanh
// Capped scores lie within [-2 cap, 0] (the constant dropped): up to this cap (log2 units) weights of
// 2^-120 and more keep their precision in bf16 and fp32, and no maximum is needed.
constexpr float kBoundedCap = 60.f;
constexpr float kNone = -3.3e38f;  // a running maximum before the first visible key

struct Params {
  ScoredArgs s;
  float cap_in;  // what a product is multiplied with to give 2 y log2(e)
  int G;         // query heads per KV head
  int ctas, alpha, rows_cap, rb_max;
  int box;       // rows of a TMA box: min(block_size, TK)
  float *part_o;    // [ctas][2][rows_cap][D]
  float *part_lse;  // [ctas][2][rows_cap], log2
  int *prefix;      // [batch + 1]: first position of each sequence's units, then all positions
};

template <int D_, int NT_, int WR_, bool F8_>
struct Cfg {
  static constexpr int D = D_, NT = NT_, WR = WR_, WK = 4 / WR_, RB = WR_ * NT_ * 8;  // RB: rows of a unit
  static constexpr bool F8 = F8_;
  static constexpr int ROWB = D * (F8 ? 1 : 2);  // bytes of a key's row
  static constexpr int CH = ROWB / 16;           // 16-byte chunks of it
  // 32 KB of K and V per stage where that is 64 or 128 keys; three stages of it let two CTAs share
  // an SM (bf16 rows of 256 values: one CTA with three stages of 64 KB)
  static constexpr int TK = ROWB <= 128 ? 128 : 64;
  static constexpr int kStageBytes = 2 * TK * ROWB;
  static constexpr int kCtasPerSm = kStageBytes > 32768 ? 1 : 2;
  static constexpr int kStages = kStageBytes > 32768 ? 3 : 98304 / kStageBytes;
  static constexpr int kRing = kStages * kStageBytes;
  static constexpr int kPad = D + 4;  // floats of a row in the merge buffer
  static_assert(WK * RB * kPad * 4 <= kRing, "the merge buffer fits the ring");
  static_assert(TK % (16 * WK) == 0 && RB <= kThreads && 2 * (TK / 8) <= 32, "a row per thread, a box per lane");
  static constexpr size_t kSmem = kRing + 1024;  // the ring starts on a 1 KB boundary
};

struct Seq {
  int c, row0, n, L, rbs, t0, tiles;  // t0: first tile that a row may see; tiles: from there
};

__device__ __forceinline__ Seq load_seq(const Params &P, int b, int tk, int rb_rows, bool *bad) {
  const AttnArgs &a = P.s.a;
  Seq s;
  s.c = a.kv.seq_lens[b];
  s.row0 = a.cu_q[b];
  s.n = a.cu_q[b + 1] - s.row0;
  const long long L = (long long)s.c + s.n;
  const bool ok = s.c >= 0 && s.n >= 0 && s.n <= a.max_q && s.row0 >= 0 && (long long)s.row0 + s.n <= a.total_q &&
                  L <= a.max_seq_len && L <= (long long)a.kv.max_blocks * a.kv.block_size;
  *bad = !ok;
  s.L = ok ? (int)L : 0;
  s.rbs = ok ? (P.G * s.n + rb_rows - 1) / rb_rows : 0;
  const int lo = P.s.window > 0 ? max(0, s.c - P.s.window + 1) : 0;  // no row is before position c
  s.t0 = lo / tk;
  s.tiles = s.rbs > 0 ? (s.L + tk - 1) / tk - s.t0 : 0;
  return s;
}
__device__ __forceinline__ int seq_work(const Params &P, const Seq &s) {
  return s.tiles > 0 ? P.s.a.kv.num_kv_heads * s.rbs * (s.tiles + P.alpha) : 0;
}
__device__ __forceinline__ int range_start(int c, int W, int ctas) { return (int)(((long long)c * W) / ctas); }
__device__ __forceinline__ int range_owner(int x, int W, int ctas) {
  return (int)((((long long)x + 1) * ctas + W - 1) / W) - 1;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t smem_at(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
// A box of rows from row y (a multiple of 8) on: groups of [part 0: 8 rows x 128 B][part 1: ...]..., or
// (rows of 64 bytes) as they are.
template <int ROWB> __device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap *map, int y, uint32_t bar) {
  if (ROWB >= 128)
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %2, %2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(y >> 3), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(y), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void ldm4(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ void ldm4t(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ uint32_t turn8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
template <bool F16>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (F16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <bool F16> __device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if (F16) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
  }
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&v);
}
// The E4M3 codes in the lower half of a word as an fp16 pair (exact).
__device__ __forceinline__ uint32_t widen(uint32_t w) {
  uint32_t y;
  asm("{.reg .b16 l, h; mov.b32 {l, h}, %1; cvt.rn.f16x2.e4m3x2 %0, l;}" : "=r"(y) : "r"(w));
  return y;
}
__device__ __forceinline__ uint32_t without_nan(uint32_t x) {  // an fp16 pair, NaN halves set to zero
  if ((x & 0x7c00u) == 0x7c00u) x &= 0xffff0000u;
  if ((x & 0x7c000000u) == 0x7c000000u) x &= 0xffffu;
  return x;
}

__device__ __forceinline__ bool nonfinite2(uint32_t x) {  // a bf16 pair
  return (x & 0x7f80u) == 0x7f80u || (x & 0x7f800000u) == 0x7f800000u;
}

template <class C>
__global__ void __launch_bounds__(kThreads, C::kCtasPerSm)
    attn_scored_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v, const Params P) {
  grid_dependency_wait();  // the earlier kernel on the stream is complete and visible
  grid_dependents_launch();
  constexpr int D = C::D, NT = C::NT, TK = C::TK, CH = C::CH, RB = C::RB, WK = C::WK, ST = C::kStages;
  constexpr int KT = D / 16;  // 16-value steps of a head
  constexpr bool F8 = C::F8;
  extern __shared__ uint8_t smem[];
  __shared__ __align__(8) uint64_t s_full[ST], s_free[ST];  // a stage's copies have landed; all warps have read it
  __shared__ int s_dead;                                    // a wait gave up
  __shared__ uint64_t s_mask[RB];      // tree mask of a row
  __shared__ int s_pos[RB], s_row[RB];  // position, and row of the sequence (-1: padding)
  __shared__ float s_slope[RB];
  __shared__ int s_place[64];  // position of a new row minus c
  __shared__ float s_m[WK][RB], s_l[WK][RB];
  __shared__ int s_scan[4], s_first_b, s_first_base, s_top[4];

  const AttnArgs &a = P.s.a;
  const KV &kv = a.kv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int wk = warp % WK, wr = warp / WK;
  const int B = kv.batch;
  uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem) + 1023) & ~uintptr_t(1023));
  const uint32_t ring_at = smem_at(ring);
  if (tid == 0) {
    for (int k = 0; k < ST; ++k) {
      bar_init(smem_at(&s_full[k]), 1);
      bar_init(smem_at(&s_free[k]), 4);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    s_dead = 0;
  }

  // ---- this CTA's range [g0, g1) of the launch's W positions ----
  auto scan = [&](int v, int *total) {  // inclusive sum over the CTA's threads
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) s_scan[warp] = x;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      before += w < warp ? s_scan[w] : 0;
      all += s_scan[w];
    }
    __syncthreads();
    *total = all;
    return x + before;
  };
  int mine = 0, W, run = 0;
  if (tid == 0) s_first_b = s_first_base = 0;
  for (int b = tid; b < B; b += kThreads) {
    bool bad;
    const Seq s = load_seq(P, b, TK, RB, &bad);
    if (bad && blockIdx.x == 0) record(a.status, SV_ERR_BAD_LENGTH);
    mine += seq_work(P, s);
  }
  scan(mine, &W);
  int pos = range_start(blockIdx.x, W, P.ctas);
  const int end = range_start(blockIdx.x + 1, W, P.ctas);
  for (int b0 = 0; b0 < B; b0 += kThreads) {  // the sequence that holds the first position; CTA 0 stores the prefix
    const int b = b0 + tid;
    int v = 0, tot;
    bool bad;
    if (b < B) v = seq_work(P, load_seq(P, b, TK, RB, &bad));
    const int excl = run + scan(v, &tot) - v;
    if (blockIdx.x == 0 && b < B) P.prefix[b] = excl;
    if (v > 0 && excl <= pos && pos < excl + v) {
      s_first_b = b;
      s_first_base = excl;
    }
    run += tot;
    if (blockIdx.x != 0 && run > pos) break;  // uniform
  }
  if (blockIdx.x == 0 && tid == 0) P.prefix[B] = W;
  __syncthreads();
  int b = s_first_b, base = s_first_base;
  bool bad_seq;
  Seq s = load_seq(P, b, TK, RB, &bad_seq);

  const int bs_shift = __ffs(kv.block_size) - 1, box = P.box;
  const float sl2 = F8 ? a.scale_log2 * kv.k_scale : a.scale_log2;
  const float cap = P.s.cap, cap_in = F8 ? P.cap_in * kv.k_scale : P.cap_in;
  const bool fast_cap = cap <= kFastCap * 1.4426950408889634f;
  const int window = P.s.window;
  const bool biased = P.s.slopes != nullptr;
  const bool bounded = !F8 && cap > 0.f && cap <= kBoundedCap && !biased;
  bool first_piece = true;
  int issued[2] = {-1, -1};  // this warp's last tiles
  static_assert(ST <= 8, "a warp has two tiles in flight at most");
  uint32_t tile0 = 0;  // tiles of the CTA's earlier pieces: tile x of the launch goes to stage x % ST
  bool dead = false;
  auto wait = [&](uint64_t &bar, uint32_t parity) {
    if (dead) return;
    const bool landed = mbar_wait_bounded(smem_at(&bar), parity, a.wait_ns);
    dead = __any_sync(0xffffffffu, !landed || *(volatile int *)&s_dead != 0);
    if (dead) s_dead = 1;
  };
  // what ldmatrix adds to a row's place for 16-value step q (mod 4) of its head: chunk 2 q + (0 or 1), swizzled
  const int lr = lane & 7, lm = lane >> 3;
  const int k_row = lm & 1, k_hi = lm >> 1, v_row = F8 ? lm & 1 : lm >> 1, v_hi = F8 ? lm >> 1 : lm & 1;
  uint32_t k_off[4], v_off[4];
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    k_off[x] = CH >= 8 ? ((x * 2 + k_hi) ^ lr) << 4 : (((x * 2 + k_hi) & (CH - 1)) ^ ((lr >> 1) & 3)) << 4;
    v_off[x] = CH >= 8 ? ((x * 2 + v_hi) ^ lr) << 4 : (((x * 2 + v_hi) & (CH - 1)) ^ ((lr >> 1) & 3)) << 4;
  }
  constexpr int kRow = C::ROWB >= 128 ? 128 : 64;  // bytes between a group's rows
  const uint32_t k_lane = k_row * 8 * C::ROWB + lr * kRow, v_lane = v_row * 8 * C::ROWB + lr * kRow;

  // failure-path test: a wait that nothing ends (no tile has been read yet), as for copies that never come
  if (a.stall == SV_STALL_ATTENTION) wait(s_free[0], 0);

  while (pos < end) {
    // ---- the next piece: tiles [kt0, kt1) of a unit ----
    int work = seq_work(P, s);
    while (pos - base >= work && b + 1 < B) {
      base += work;
      s = load_seq(P, ++b, TK, RB, &bad_seq);
      work = seq_work(P, s);
    }
    if (pos - base >= work) break;  // cannot happen while the lengths stay put
    const int U = s.tiles + P.alpha;
    const int unit = (pos - base) / U, off = (pos - base) - unit * U;
    const int npos = min(U - off, end - pos);
    pos += npos;
    const int kt0 = s.t0 + max(0, off - P.alpha), kt1 = s.t0 + off + npos - P.alpha;
    if (kt1 <= kt0) continue;  // only the unit's lead-in lies in this range
    const int kvh = unit / s.rbs, rb = unit - kvh * s.rbs;
    const bool whole = kt0 == s.t0 && kt1 == s.t0 + s.tiles;
    const int c = s.c, ke = min(s.L, kt1 * TK);
    const int lo = window > 0 ? max(0, c - window + 1) : 0;
    const int rows = min(RB, P.G * s.n - rb * RB);  // live rows of the block

    __syncthreads();  // the previous piece's shared memory is free
    // ---- rows of the block, new keys' places, the first tiles' pool rows ----
    int top = c;
    if (tid < RB) {
      const bool live = tid < rows;
      const int r = rb * RB + tid, i = live ? r / P.G : 0, head = kvh * P.G + (live ? r - i * P.G : 0);
      const int p = P.s.positions != nullptr ? P.s.positions[s.row0 + i] : c + i;
      if (p < c) record(a.status, SV_ERR_BAD_LENGTH);
      s_pos[tid] = p;
      s_row[tid] = live ? i : -1;
      s_mask[tid] = live && a.mask_kind == SV_MASK_TREE ? a.tree_mask[s.row0 + i] : 0ull;
      s_slope[tid] = biased ? P.s.slopes[head] * 1.4426950408889634f : 0.f;
      top = live ? p : c;
    }
    if (tid < 64 && tid < s.n) s_place[tid] = P.s.positions != nullptr ? P.s.positions[s.row0 + tid] - c : tid;
    top = __reduce_max_sync(0xffffffffu, top);
    if (lane == 0) s_top[warp] = top;
    const int32_t *bt = kv.block_table + (size_t)b * kv.max_blocks;
    // This warp issues tiles k = turn, turn + 4, ... of the piece: lane 2 j (2 j + 1) the keys' (values') box
    // of rows j box ... of the tile, skipping boxes without a visible key.
    const int ntiles = kt1 - kt0;
    int turn = (int)((warp - tile0) & 3u);
    const int box_row = (lane >> 1) * box;
    auto block_of = [&](int k) -> int {  // physical block of this lane's box of tile k; -2: none
      const int tok = (kt0 + k) * TK + box_row;
      return k < ntiles && box_row < TK && tok < ke && tok + box > lo ? bt[tok >> bs_shift] : -2;
    };
    int id = block_of(turn);
    auto issue_until = [&](int limit) {  // this warp's tiles below limit
      while (turn < min(limit, ntiles)) {
        const uint32_t x = tile0 + turn, st = x % ST;
        if (turn >= ST) wait(s_free[st], (x / ST - 1) & 1u);
        if (dead) {  // nothing more is issued
          turn += 4;
          continue;
        }
        const bool want = id != -2, bad = want && (id < 0 || id >= kv.num_blocks), go = want && !bad;
        if (bad) record(a.status, SV_ERR_BAD_BLOCK_ID);
        const uint32_t bar = smem_at(&s_full[st]);
        const int boxes = __popc(__ballot_sync(0xffffffffu, go));
        if (lane == 0) bar_expect(bar, boxes * box * C::ROWB);
        __syncwarp();
        if (go) {
          const int tok = (kt0 + turn) * TK + box_row;
          const int y = ((id * kv.num_kv_heads + kvh) << bs_shift) + (tok & (kv.block_size - 1));
          const uint32_t dst = ring_at + st * C::kStageBytes + (lane & 1) * TK * C::ROWB + box_row * C::ROWB;
          load_box<C::ROWB>(dst, (lane & 1) ? &map_v : &map_k, y, bar);
        }
        __syncwarp();
        issued[1] = issued[0];
        issued[0] = (int)x;
        turn += 4;
        id = block_of(turn);
      }
    };
    issue_until(ST - 1);  // the stages are free: the previous piece is done with them
    __syncthreads();
    const int row_top = max(max(s_top[0], s_top[1]), max(s_top[2], s_top[3]));
    const int all_see = window > 0 ? row_top - window + 1 : 0;  // keys from here to c are visible to every row

    // ---- Q into registers ----
    uint32_t q[NT][KT][2];
    {
      const uint32_t *src = reinterpret_cast<const uint32_t *>(a.q);
      bool over = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int rl = (wr * NT + nt) * 8 + g, i = s_row[rl];
        const int r = rb * RB + rl;
        const size_t at = i < 0 ? 0 : ((size_t)(s.row0 + i) * a.num_q_heads + kvh * P.G + (r - i * P.G)) * (D / 2);
#pragma unroll
        for (int kk = 0; kk < KT; ++kk) {
          if (F8) {
            const uint2 x = i < 0 ? make_uint2(0, 0) : *reinterpret_cast<const uint2 *>(src + at + kk * 8 + 2 * t);
            q[nt][kk][0] = pack2<true>(__uint_as_float(x.x << 16), __uint_as_float(x.x & 0xffff0000u));
            q[nt][kk][1] = pack2<true>(__uint_as_float(x.y << 16), __uint_as_float(x.y & 0xffff0000u));
#pragma unroll
            for (int h = 0; h < 2; ++h)
              over |= (q[nt][kk][h] & 0x7c00u) == 0x7c00u || (q[nt][kk][h] & 0x7c000000u) == 0x7c000000u;
          } else {
            q[nt][kk][0] = i < 0 ? 0u : src[at + kk * 8 + t];
            q[nt][kk][1] = i < 0 ? 0u : src[at + kk * 8 + t + 4];
          }
        }
      }
      if (F8 && over) record(a.status, SV_ERR_NONFINITE);  // a query element beyond the fp16 range
    }

    float o[KT][NT][4], m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = bounded ? 0.f : kNone;
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int mt = 0; mt < KT; ++mt) o[mt][nt][0] = o[mt][nt][1] = o[mt][nt][2] = o[mt][nt][3] = 0.f;
    }

    for (int kt = kt0; kt < kt1; ++kt) {
      const uint32_t x = tile0 + (kt - kt0), st = x % ST;
      issue_until(kt - kt0 + ST);
      wait(s_full[st], (x / ST) & 1u);
      const uint32_t k_at = ring_at + st * C::kStageBytes + k_lane, v_at = ring_at + st * C::kStageBytes + TK * C::ROWB + v_lane;
#pragma unroll 1
      for (int k16 = wk * 16; k16 < TK; k16 += WK * 16) {
        const int key0 = kt * TK + k16;
        if (key0 >= ke || key0 + 16 <= lo) continue;  // warp-uniform: nothing to see here
        // ---- S^T = K Q^T ----
        float sc[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) sc[nt][0] = sc[nt][1] = sc[nt][2] = sc[nt][3] = 0.f;
        const uint32_t kaddr = k_at + k16 * C::ROWB;
        if (!F8) {
#pragma unroll
          for (int kk = 0; kk < KT; ++kk) {
            uint32_t f[4];
            ldm4(f, kaddr + k_off[kk & 3] + (kk >> 2) * 1024);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma<false>(sc[nt], f, q[nt][kk][0], q[nt][kk][1]);
          }
        } else {
#pragma unroll
          for (int k2 = 0; k2 < KT / 2; ++k2) {
            uint32_t f[4];
            ldm4(f, kaddr + k_off[k2 & 3] + (k2 >> 2) * 1024);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t e[4] = {widen(f[2 * h]), widen(f[2 * h + 1]), widen(f[2 * h] >> 16), widen(f[2 * h + 1] >> 16)};
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma<true>(sc[nt], e, q[nt][2 * k2 + h][0], q[nt][2 * k2 + h][1]);
            }
          }
        }
        // ---- scores ----
        if (cap == 0.f) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[nt][e] *= sl2;
        } else if (fast_cap) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[nt][e] = -2.f * cap * rcp(1.f + ex2(sc[nt][e] * cap_in));
        } else {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[nt][e] = cap * tanhf(sc[nt][e] * sl2 / cap) - cap;
        }
        const bool edge = key0 + 16 > min(c, ke) || key0 < all_see;  // warp-uniform: some row may not see some key
        if (biased && !edge) {
          const float d0 = (float)(key0 + g - c), d1 = d0 + 8.f;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const float2 sl = *reinterpret_cast<const float2 *>(&s_slope[(wr * NT + nt) * 8 + 2 * t]);
            sc[nt][0] = fmaf(sl.x, d0, sc[nt][0]);
            sc[nt][1] = fmaf(sl.y, d0, sc[nt][1]);
            sc[nt][2] = fmaf(sl.x, d1, sc[nt][2]);
            sc[nt][3] = fmaf(sl.y, d1, sc[nt][3]);
          }
        }
        if (edge) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int key = key0 + g + 8 * h, j = key - c;
            const int place = j >= 0 && key < ke ? s_place[j] : j;  // position of the key minus c
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int rl = (wr * NT + nt) * 8 + 2 * t + e, i = s_row[rl];
                bool vis = key < ke && i >= 0;
                if (vis && j >= 0) vis = a.mask_kind == SV_MASK_CAUSAL ? j <= i : ((s_mask[rl] >> j) & 1ull) != 0;
                if (vis && window > 0) vis = s_pos[rl] - c - place < window;
                sc[nt][2 * h + e] = vis ? fmaf(s_slope[rl], (float)place, sc[nt][2 * h + e]) : -INFINITY;
              }
          }
        }
        // ---- the running maximum ----
        if (!bounded) {
          bool move = false;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              move |= sc[nt][e] > m[nt][e & 1] + kMoveAt;
            }
          if (__any_sync(0xffffffffu, move)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float mx = fmaxf(sc[nt][e], sc[nt][e + 2]);
#pragma unroll
                for (int y = 4; y < 32; y <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, y));
                const float mn = fmaxf(m[nt][e], mx);
                const float f = mn == m[nt][e] ? 1.f : ex2(m[nt][e] - mn);
                m[nt][e] = mn;
                l[nt][e] *= f;
#pragma unroll
                for (int mt = 0; mt < KT; ++mt) {
                  o[mt][nt][e] *= f;
                  o[mt][nt][e + 2] *= f;
                }
              }
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[nt][e] -= m[nt][e & 1];
        }
        // ---- P^T ----
        uint32_t pb[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[nt][e] = ex2(sc[nt][e]);
          l[nt][0] += sc[nt][0] + sc[nt][2];
          l[nt][1] += sc[nt][1] + sc[nt][3];
          pb[nt][0] = turn8x8(pack2<F8>(sc[nt][0], sc[nt][1]));
          pb[nt][1] = turn8x8(pack2<F8>(sc[nt][2], sc[nt][3]));
        }
        // ---- O^T += V^T P^T ----
        if (!F8) {
          const uint32_t vaddr = v_at + k16 * C::ROWB;
          bool odd = false;  // an infinity or NaN among this step's values
#pragma unroll
          for (int mt = 0; mt < KT; ++mt) {
            uint32_t f[4];
            ldm4t(f, vaddr + v_off[mt & 3] + (mt >> 2) * 1024);
            if (edge) {  // 0 * infinity must not reach a row that does not see the key
#pragma unroll
              for (int x = 0; x < 4; ++x)
                if (nonfinite2(f[x])) {
                  odd = true;
                  if ((f[x] & 0x7f80u) == 0x7f80u) f[x] &= 0xffff0000u;
                  if ((f[x] & 0x7f800000u) == 0x7f800000u) f[x] &= 0xffffu;
                }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma<false>(o[mt][nt], f, pb[nt][0], pb[nt][1]);
          }
          if (edge && __any_sync(0xffffffffu, odd)) {
            // the values set to zero above, for the rows that see their keys
            const uint8_t *vs = ring + st * C::kStageBytes + TK * C::ROWB + k16 * C::ROWB;
#pragma unroll 1
            for (int key = 0; key < 16; ++key) {
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                const float e0 = key < 8 ? sc[nt][0] : sc[nt][2], e1 = key < 8 ? sc[nt][1] : sc[nt][3];
                const float p0 = __shfl_sync(0xffffffffu, e0, (key & 7) * 4 + t);
                const float p1 = __shfl_sync(0xffffffffu, e1, (key & 7) * 4 + t);
#pragma unroll
                for (int mt = 0; mt < KT; ++mt)
#pragma unroll
                  for (int h = 0; h < 2; ++h) {
                    const uint32_t x =
                        *reinterpret_cast<const uint16_t *>(vs + (key >> 3) * 8 * C::ROWB + (key & 7) * 128 + (mt >> 2) * 1024 +
                                                            ((((mt & 3) * 2 + h) ^ (key & 7)) << 4) + g * 2);
                    if ((x & 0x7f80u) != 0x7f80u) continue;
                    const float v = __uint_as_float(x << 16);
                    if (p0 > 0.f) o[mt][nt][2 * h] += p0 * v;
                    if (p1 > 0.f) o[mt][nt][2 * h + 1] += p1 * v;
                  }
              }
            }
          }
        } else {
          const uint32_t vaddr = v_at + k16 * C::ROWB;
#pragma unroll
          for (int m2 = 0; m2 < KT / 2; ++m2) {
            uint32_t f[4];
            ldm4t(f, vaddr + v_off[m2 & 3] + (m2 >> 2) * 1024);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              // a word: two dimensions of one key below, of the next key above; pairs of keys are wanted
              const uint32_t w0 = __byte_perm(f[2 * h], 0u, 0x3120), w1 = __byte_perm(f[2 * h + 1], 0u, 0x3120);
              uint32_t e[4] = {widen(w0), widen(w0 >> 16), widen(w1), widen(w1 >> 16)};
              if (edge) {  // slots that no row sees may hold anything
#pragma unroll
                for (int y = 0; y < 4; ++y) e[y] = without_nan(e[y]);
              }
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma<true>(o[m2 * 2 + h][nt], e, pb[nt][0], pb[nt][1]);
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) bar_arrive(smem_at(&s_free[st]));
    }
    // ---- the key groups' results, merged ----
    __syncthreads();  // every warp is done with the ring
    tile0 += ntiles;
    float *buf = reinterpret_cast<float *>(ring);  // [WK][RB][kPad]
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int rl = (wr * NT + nt) * 8 + 2 * t + e;
        float sum = l[nt][e];
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
        if (g == 0) {
          s_m[wk][rl] = m[nt][e];
          s_l[wk][rl] = sum;
        }
        float *dst = buf + (wk * RB + rl) * C::kPad;
#pragma unroll
        for (int mt = 0; mt < KT; ++mt) {
          dst[mt * 16 + (F8 ? 2 * g : g)] = o[mt][nt][e];
          dst[mt * 16 + (F8 ? 2 * g + 1 : g + 8)] = o[mt][nt][e + 2];
        }
      }
    __syncthreads();
    const size_t slot = ((size_t)blockIdx.x * 2 + (first_piece ? 0 : 1)) * P.rows_cap;
    if (tid < rows) {
      float M = s_m[0][tid], tot = 0.f;
#pragma unroll
      for (int w = 1; w < WK; ++w) M = fmaxf(M, s_m[w][tid]);
      const float ref = M;  // finite: kNone at the least
#pragma unroll
      for (int w = 0; w < WK; ++w) tot += s_l[w][tid] * ex2(s_m[w][tid] - ref);
      const float inv = tot == 0.f ? 0.f : (F8 ? kv.v_scale : 1.f) / tot;
      if (!whole) P.part_lse[slot + tid] = tot == 0.f ? -INFINITY : M + log2f(tot);
#pragma unroll
      for (int w = 0; w < WK; ++w) s_l[w][tid] = ex2(s_m[w][tid] - ref) * inv;
    }
    __syncthreads();
    for (int x = tid; x < rows * (D / 8); x += kThreads) {
      const int rl = x / (D / 8), d8 = (x % (D / 8)) * 8;
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = 0.f;
#pragma unroll
      for (int w = 0; w < WK; ++w) {
        const float f = s_l[w][rl];
        const float4 *src = reinterpret_cast<const float4 *>(buf + (w * RB + rl) * C::kPad + d8);
        const float4 x0 = src[0], x1 = src[1];
        v[0] = fmaf(f, x0.x, v[0]), v[1] = fmaf(f, x0.y, v[1]), v[2] = fmaf(f, x0.z, v[2]), v[3] = fmaf(f, x0.w, v[3]);
        v[4] = fmaf(f, x1.x, v[4]), v[5] = fmaf(f, x1.y, v[5]), v[6] = fmaf(f, x1.z, v[6]), v[7] = fmaf(f, x1.w, v[7]);
      }
      if (whole) {
        const int i = s_row[rl], head = kvh * P.G + (rb * RB + rl) - i * P.G;
        *reinterpret_cast<uint4 *>(reinterpret_cast<__nv_bfloat16 *>(a.out) +
                                   ((size_t)(s.row0 + i) * a.num_q_heads + head) * D + d8) =
            make_uint4(pack2<false>(v[0], v[1]), pack2<false>(v[2], v[3]), pack2<false>(v[4], v[5]), pack2<false>(v[6], v[7]));
      } else {
        float4 *dst = reinterpret_cast<float4 *>(P.part_o + (slot + rl) * D + d8);
        dst[0] = make_float4(v[0], v[1], v[2], v[3]);
        dst[1] = make_float4(v[4], v[5], v[6], v[7]);
      }
    }
    first_piece = false;
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the merge's accesses, before the next piece's copies
  }
  if (dead) {
    if (lane == 0) record(a.status, SV_ERR_TIMEOUT);
    // the copies this warp has in flight land before the CTA's shared memory is released
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (issued[k] >= 0) mbar_wait_bounded(smem_at(&s_full[issued[k] % ST]), (issued[k] / ST) & 1, kDrainBudgetNs);
  }
  __syncthreads();
}

// Merges the partials of every unit that two or more CTAs shared: o = sum_p 2^lse_p o_p / sum_p 2^lse_p,
// in the order of the CTAs. A thread takes 8 values of a row, four pieces' loads in flight.
template <class C>
__global__ void __launch_bounds__(128) attn_scored_combine(const Params P) {
  grid_dependents_launch();
  grid_dependency_wait();  // the earlier kernel on the stream is complete and visible
  constexpr int D = C::D;
  const AttnArgs &a = P.s.a;
  const int b = blockIdx.x, kvh = blockIdx.y / P.rb_max, rb = blockIdx.y % P.rb_max;
  const int W = P.prefix[a.kv.batch], base = P.prefix[b];
  bool bad;
  const Seq s = load_seq(P, b, C::TK, C::RB, &bad);
  if (s.tiles <= 0 || rb >= s.rbs) return;
  const int T0 = base + (kvh * s.rbs + rb) * (s.tiles + P.alpha) + P.alpha, T1 = T0 + s.tiles;
  const int c0 = range_owner(T0, W, P.ctas), c1 = range_owner(T1 - 1, W, P.ctas);
  if (c0 == c1) return;  // one CTA held the whole unit and wrote its rows
  // the unit is CTA c0's first piece only if its range starts within the unit's lead-in
  const int slot0 = range_start(c0, W, P.ctas) >= T0 - P.alpha ? 0 : 1;
  constexpr int kPc = 4;
  const int rows = min(C::RB, P.G * s.n - rb * C::RB);
  for (int x = threadIdx.x; x < rows * (D / 8); x += blockDim.x) {
    const int rl = x / (D / 8), d8 = (x % (D / 8)) * 8;
    float M = -INFINITY, den = 0.f, acc[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) acc[k] = 0.f;
    for (int cb = c0; cb <= c1; cb += kPc) {
      float lse[kPc];
      float4 v[kPc][2];
#pragma unroll
      for (int k = 0; k < kPc; ++k) {
        // a CTA whose range is empty (more CTAs than positions) holds nothing
        const bool in = cb + k <= c1 && range_start(cb + k, W, P.ctas) < range_start(cb + k + 1, W, P.ctas);
        const int cc = in ? cb + k : c0;
        const size_t at = ((size_t)cc * 2 + (cc == c0 ? slot0 : 0)) * P.rows_cap + rl;
        lse[k] = in ? __ldcg(P.part_lse + at) : -INFINITY;
        const float4 *src = reinterpret_cast<const float4 *>(P.part_o + at * D + d8);
        v[k][0] = in ? __ldcg(src) : make_float4(0.f, 0.f, 0.f, 0.f);
        v[k][1] = in ? __ldcg(src + 1) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      float mn = M;
#pragma unroll
      for (int k = 0; k < kPc; ++k) mn = fmaxf(mn, lse[k]);
      const float ref = mn == -INFINITY ? 0.f : mn;
      const float f = exp2f(M - ref);
      M = mn;
      den *= f;
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[k] *= f;
#pragma unroll
      for (int k = 0; k < kPc; ++k) {
        const float w = exp2f(lse[k] - ref);  // NaN for a row whose sum is NaN: it stays one
        den += w;
        acc[0] = fmaf(w, v[k][0].x, acc[0]), acc[1] = fmaf(w, v[k][0].y, acc[1]);
        acc[2] = fmaf(w, v[k][0].z, acc[2]), acc[3] = fmaf(w, v[k][0].w, acc[3]);
        acc[4] = fmaf(w, v[k][1].x, acc[4]), acc[5] = fmaf(w, v[k][1].y, acc[5]);
        acc[6] = fmaf(w, v[k][1].z, acc[6]), acc[7] = fmaf(w, v[k][1].w, acc[7]);
      }
    }
    const float inv = den == 0.f ? 0.f : 1.f / den;
    const int r = rb * C::RB + rl, i = r / P.G, head = kvh * P.G + r - i * P.G;
    *reinterpret_cast<uint4 *>(reinterpret_cast<__nv_bfloat16 *>(a.out) + ((size_t)(s.row0 + i) * a.num_q_heads + head) * D + d8) =
        make_uint4(pack2<false>(acc[0] * inv, acc[1] * inv), pack2<false>(acc[2] * inv, acc[3] * inv),
                   pack2<false>(acc[4] * inv, acc[5] * inv), pack2<false>(acc[6] * inv, acc[7] * inv));
  }
}

struct Layout {
  int ctas, rows_cap, rb_max;
  size_t lse_offset, prefix_offset, bytes;
};

template <class C>
Layout layout_of(const KV &kv, int G, int max_q, int max_seq_len) {
  Layout l;
  l.rb_max = (G * max_q + C::RB - 1) / C::RB;
  const long long tiles = (long long)kv.batch * kv.num_kv_heads * l.rb_max * ((max_seq_len + C::TK - 1) / C::TK);
  l.ctas = (int)std::max(1LL, std::min<long long>((long long)C::kCtasPerSm * num_sms(), tiles));
  l.rows_cap = std::min(C::RB, G * max_q);
  const size_t slots = (size_t)l.ctas * 2 * l.rows_cap;
  l.lse_offset = slots * C::D * sizeof(float);
  l.prefix_offset = (l.lse_offset + slots * sizeof(float) + 255) / 256 * 256;
  l.bytes = l.prefix_offset + ((size_t)kv.batch + 1) * sizeof(int);
  return l;
}

constexpr int kAlpha = 2;  // positions of a unit's lead-in

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                   const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn tensor_map_encoder();  // null without a driver that has it

template <class C> bool make_map(CUtensorMap *map, void *pool, const KV &kv, int box) {
  const cuuint64_t rows = (cuuint64_t)kv.num_blocks * kv.num_kv_heads * kv.block_size;
  const EncodeTiledFn fn = tensor_map_encoder();
  if (fn == nullptr) return false;
  const cuuint32_t one[4] = {1, 1, 1, 1};
  if (C::ROWB >= 128) {
    const cuuint64_t dim[4] = {128, 8, C::ROWB / 128, rows / 8}, stride[3] = {C::ROWB, 128, 8 * C::ROWB};
    const cuuint32_t b[4] = {128, 8, C::ROWB / 128, (cuuint32_t)box / 8};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, pool, dim, stride, b, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  }
  const cuuint64_t dim[2] = {64, rows}, stride[1] = {64};
  const cuuint32_t b[2] = {64, (cuuint32_t)box};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, pool, dim, stride, b, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Launches (st != null via `go`) or sizes one instance.
template <class C>
cudaError_t run(const ScoredArgs &sa, void *workspace, size_t *bytes, cudaStream_t st, bool go) {
  const KV &kv = sa.a.kv;
  Params p;
  p.s = sa;
  p.G = sa.a.num_q_heads / kv.num_kv_heads;
  const Layout l = layout_of<C>(kv, p.G, sa.a.max_q, sa.a.max_seq_len);
  *bytes = l.bytes;
  if (!go) return cudaSuccess;
  p.cap_in = sa.cap > 0.f ? sa.a.scale_log2 * 2.f * 1.4426950408889634f / sa.cap : 0.f;
  p.ctas = l.ctas;
  p.alpha = kAlpha;
  p.rows_cap = l.rows_cap;
  p.rb_max = l.rb_max;
  p.part_o = reinterpret_cast<float *>(workspace);
  p.part_lse = reinterpret_cast<float *>(reinterpret_cast<uint8_t *>(workspace) + l.lse_offset);
  p.prefix = reinterpret_cast<int *>(reinterpret_cast<uint8_t *>(workspace) + l.prefix_offset);
  p.box = std::min(kv.block_size, C::TK);
  CUtensorMap mk, mv;
  if (!make_map<C>(&mk, kv.k_pool, kv, p.box) || !make_map<C>(&mv, kv.v_pool, kv, p.box)) return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(attn_scored_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem);
  if (e != cudaSuccess) return e;
  e = launch_pdl(attn_scored_kernel<C>, dim3(p.ctas), dim3(kThreads), C::kSmem, st, mk, mv, p);
  if (e != cudaSuccess) return e;
  return launch_pdl(attn_scored_combine<C>, dim3(kv.batch, kv.num_kv_heads * p.rb_max), dim3(128), 0, st, p);
}

// The smallest block of query rows that holds a unit's, else blocks of the largest.
template <int D, bool F8>
cudaError_t pick(const ScoredArgs &sa, void *workspace, size_t *bytes, cudaStream_t st, bool go) {
  const int rows = sa.a.num_q_heads / sa.a.kv.num_kv_heads * sa.a.max_q;
  if (rows <= 8) return run<Cfg<D, 1, 1, F8>>(sa, workspace, bytes, st, go);
  if (rows <= 16) return run<Cfg<D, 2, 1, F8>>(sa, workspace, bytes, st, go);
  if constexpr (D <= 128) {
    if (rows <= 24) return run<Cfg<D, 3, 1, F8>>(sa, workspace, bytes, st, go);
    if (rows <= 32) return run<Cfg<D, 4, 1, F8>>(sa, workspace, bytes, st, go);
    if (rows <= 48) return run<Cfg<D, 3, 2, F8>>(sa, workspace, bytes, st, go);
    if (rows <= 64) return run<Cfg<D, 4, 2, F8>>(sa, workspace, bytes, st, go);
    return run<Cfg<D, 4, 4, F8>>(sa, workspace, bytes, st, go);
  } else {
    if (rows <= 32) return run<Cfg<D, 2, 2, F8>>(sa, workspace, bytes, st, go);
    return run<Cfg<D, 2, 4, F8>>(sa, workspace, bytes, st, go);
  }
}

}  // namespace scored
}  // namespace sv
