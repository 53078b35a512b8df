// Attention with modified scores (sv_spec_verify_attn_scored) over bf16 and E4M3 caches, with
// warp-level matrix instructions; instantiated per head size in attn_scored_d*.cu.
//
// The mathematics (base-2 exponents; p_t the position of key t, c the committed tokens):
//   s_t = cap tanh(scale <q, k_t> / cap) + slope (p_t - p_0),   o = sum_t 2^(s_t - m) v_t / sum_t 2^(s_t - m)
// with everything in units of log2 and p_0 the position of the sequence's first row. The distance bias
// -slope (p_i - p_t) differs from the term above by a constant of the row, which the softmax cancels: a key's
// term is the same for all rows of a head. (Counted from c instead, rows whose positions lie far past c would
// have terms so large that fp32 has no bits left for the scores.)
// tanh(y) = 1 - 2 / (1 + 2^(2 y log2 e)): two special-function instructions; its absolute error,
// about 2^-22, times the cap is what reaches a score (caps above kFastCap take tanhf).
//
// Fewer bits than fp32, and why: the weights are rounded to the type of V's operand, bf16 (off by 2^-8 of themselves at
// most) or, over E4M3 pools, fp16 (2^-11), since a matrix instruction takes operands of one type; the sum of the weights
// is of the unrounded ones. Over E4M3 pools the queries are fp16 for the same reason (2^-11; what lies below 2^-14
// is off by up to 2^-25, beyond 65504 the call records SV_ERR_NONFINITE). The cap's 2^x and reciprocal are the
// approximate ones: 2^-19 of the cap at most, far below what the rounded weights leave. Against 64 bits a bf16 row is off by
// 0.0023 of its size, where one rounding of the output alone leaves 0.0017.
//
// Bound: memory up to some 16 query rows a unit (one KV head of one sequence: G n_b rows), where 70 us for
// 32 sequences of 2K to 4K tokens are 83% of the measured copy rate; beyond, the chain of a warp's step, ldmatrix ->
// products -> scores -> movmatrix -> products, of which the two warps of a scheduler hide only a part: with 24 rows a warp a step of
// 16 keys is 48 products of 16 x 8 x 16 at 8 cycles of a quarter SM, and two warps' 768 cycles of products
// stand in the 1800 that their steps take (43%). Units of more than kWideRows rows go to
// attn_scored_wide.cu, whose blocks of 128 rows cost too much for fewer (40 rows: 93 us here, 97 there; in
// sequences of 600 tokens 94 and 121).
//
// Times (us, 8 KV heads of 128 values; share of the copy rate): 32 sequences of 2K to 4K tokens in bf16 with 4,
// 16, 32 and 48 rows a KV head 69 (85%), 75, 94 (66%), 96 (63%); 32 x 6 rows over 0.5K to 4K tokens, capped, 60.5
// (72%); four sequences of 32K tokens in E4M3 53 (74%); 128 sequences in a window of 1024, biased, 88 (46%: 4
// short units a CTA, each 7000 cycles of setting up and merging).
//
// Work: as many CTAs as fit the GPU stay for the whole launch. The key tiles of all units laid end
// to end (each unit preceded by `alpha` positions, what starting and finishing one costs) are cut
// into equal contiguous ranges, one per CTA. A unit that one CTA holds whole is written by it; a
// shared one leaves a normalised partial and its log-sum-exp in one of the CTA's two slots, and
// attn_scored_combine merges the partials in the order of the CTAs (so results repeat bit for bit).
// With a window a unit's tiles start at its first visible one: keys out of sight are not read.
//
// A CTA's warps are one producer and WK key groups x WR row groups of consumers, each with NT x 8 rows
// (Cfg; `pick` says which). The producer walks the CTA's pieces and brings tiles of TK keys (16 KB of K and
// V) into a ring of kStages stages by TMA, a box per block (or per tile, where blocks are larger), the
// pool seen as (128 bytes, 8 rows, 128-byte parts of a row, groups of 8 rows) and swizzled so that
// ldmatrix reads without bank conflicts; it runs on into the next piece while the consumers finish one. A
// consumer takes every WK-th 16 keys of a piece:
//   S^T (keys x rows) = K Q^T, A = K (ldmatrix), B = Q held in registers, accumulators fp32;
//   the running maximum of a row moves only when a score passes it by far (kMoveAt; one vote a step), and
//   not at all where the cap bounds the scores well enough (kBoundedCap);
//   P^T = 2^(S^T - m) in bf16 (fp16 for E4M3 pools) turned into a B operand by movmatrix;
//   O^T (dims x rows) += V^T P^T, A = V^T (ldmatrix.trans), accumulators fp32 in registers.
// Query rows sit on the n dimension, so that 24 rows (4 heads x 6) cost 24 and not 32. At the end
// of a piece the WK key groups' (m, l, O) are merged through shared memory, 8 rows of each warp at a time.
//
// A warp's step is a chain of products, special functions and products again, so it is made large (32 keys where
// registers allow, Cfg::M, else 16) and two CTAs of four consumers share an SM: their registers go by role (kConsumerRegs).
// (16 to 18 warps of 8 rows each, which read K and V from shared memory once a row group: 32 x 6 rows 62 us, but
// wide units 154 against 96. No split of registers, three consumers: 70.) Steps at the edges (new rows, the
// window's start) see keys as bits of a row and are kept out of the way of the others.
//
// A cap's constant term is dropped like the bias's: -2 cap / (1 + 2^(2 y log2 e)) is what is left (the tanhf form
// keeps it: next to a large cap the rest would lose its last bits).
// E4M3 codes become fp16 operands in registers (exactly). ldmatrix moves pairs of codes; which
// dimension lands at which place of the operand differs from the bf16 form, and Q's registers and O's
// columns follow it.
//
// All mbarrier waits are bounded: after one that gives up, a warp goes through the rest of its work
// without waiting (on whatever the stages hold) and the call records SV_ERR_TIMEOUT.
#pragma once

#include <cuda.h>
#include <cuda_fp16.h>

#include <climits>
#include <type_traits>

#include "sv_internal.cuh"

namespace sv {
namespace scored {

// The running maximum moves when a score passes it by this (log2): weights in bf16 and sums in fp32 have
// room for 2^60, weights in fp16 for 2^8 and their sums over the row group's products.
template <bool F16> constexpr float kMoveAt = F16 ? 8.f : 60.f;
constexpr float kFastCap = 200.f;  // caps up to this take the two-instruction tanh
// Capped scores lie within [-2 cap, 0] (the constant dropped): up to this cap (log2 units) weights of
// 2^-120 and more keep their precision in bf16 and fp32, and no maximum is needed.
constexpr float kBoundedCap = 60.f;
// Registers of a thread: as launched (256 threads, two CTAs an SM), and after the split.
constexpr int kLaunchRegs = 128, kProducerRegs = 40, kConsumerRegs = 216;
static_assert(kProducerRegs + kConsumerRegs == 2 * kLaunchRegs, "a split above the launch's share would wait forever");
constexpr float kNone = -3.3e38f;  // a running maximum before the first visible key

struct Params {
  ScoredArgs s;
  float cap_in;  // what a product is multiplied with to give 2 y log2(e)
  int G;         // query heads per KV head
  int ctas, alpha, rows_cap;
  int box;       // rows of a TMA box: min(block_size, TK)
  float *part_o;    // [ctas][2][rows_cap][D]
  float *part_lse;  // [ctas][2][rows_cap], log2
  int *prefix;      // [batch + 1]: first position of each sequence's units, then all positions
};

template <int D_, int NT_, int WR_, int WK_, bool F8_>
struct Cfg {
  static constexpr int D = D_, NT = NT_, WR = WR_, WK = WK_, RB = WR_ * NT_ * 8;  // RB: rows of a unit
  static constexpr bool F8 = F8_;
  // four consumer warps, then four of which the first produces: register shares go by four warps
  static constexpr int kConsumers = 4, kThreads = 256, kCtasPerSm = 2;
  static_assert(WK * WR == kConsumers, "a consumer on each quarter of the SM");
  static constexpr int ROWB = D * (F8 ? 1 : 2);  // bytes of a key's row
  // Infinities and NaN that an edge step takes out of its values come back to the rows that see their keys at the
  // end of the piece, from the pool, else in the step. One way or the other hardly ever runs; what it does to the loop's
  // code is what differs (us, 32 sequences of 0.5K to 4K tokens): heads of 64, one and six tokens 35.1 and 37.8 here, 41.9
  // and 40.5 in the step; heads of 128 60.7 and 59.5, 40 rows in short sequences 97 and 92; E4M3, four
  // sequences of 32K tokens 53 and 60.
  static constexpr bool kLate = F8 || D == 64;
  // Positions of a unit's lead-in. 24 rows a warp: 5 against 4 90 and 94 us (128 units a window), 60.4 and 61.6 (32 x 6
  // rows), 7 gains nothing more; fewer rows: one token of 32 sequences 69.4 and 68.5 us.
  static constexpr int kAlpha = NT >= 3 ? 5 : 4;
  static constexpr int TK = 8192 / ROWB;         // keys of a tile: 16 KB of K and V
  // a step: M x 16 keys; two where registers allow, so that a chain of products hides another
  static constexpr int M = TK >= 32 && D_ * NT_ <= (WR_ == 4 ? 384 : 256) && (WK_ < 4 || TK >= 64) ? 2 : 1;
  static constexpr int S = TK / (16 * M);        // steps of a tile
  static constexpr int kStageBytes = 2 * TK * ROWB;
  // Values of a row that are merged at a time: all, or 64 where the shared memory is better spent on
  // stages (four key groups of few rows hold two stages; 6 of them against 4: 70.7 and 74.5 us for one
  // token of 32 sequences of 2 to 4 K, 86 % and 81 % of the memory rate).
  static constexpr bool kNarrow = D == 128 && NT_ <= 2 && WK_ == 4;
  static constexpr int kChunk = D == 128 && !kNarrow ? 128 : 64, kStages = kNarrow ? 6 : 4;
  static constexpr int kRing = kStages * kStageBytes;
  static constexpr int kPad = kChunk + 4;                   // floats of a row in the merge buffer
  static constexpr int kMerge = kConsumers * 8 * kPad * 4;  // 8 rows of every consumer
  static constexpr size_t kSmem = 1024 + kRing + kMerge;  // the ring starts on a 1 KB boundary
  static_assert(kCtasPerSm * (kSmem + 4608) <= 228 * 1024, "shared memory of an SM");
  // A parity wait for a stage's phase n returns at once while phase n - 1 has not completed, so a consumer has
  // to have seen phase n - 1: it visits every tile, or every ST-th of the stages that it uses. (At the
  // start of a piece all phases of the earlier pieces' tiles have been seen by some consumer, and the
  // consumers have met at a barrier since.)
  static constexpr int gcd(int x, int y) { return y == 0 ? x : gcd(y, x % y); }
  static_assert(kStages % (WK / gcd(WK, S)) == 0, "a consumer sees each phase of its stages");
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
// a factor that has overflowed (tiny caps) as the largest finite one: zero times it stays zero
__host__ __device__ __forceinline__ float finite(float x) { return fminf(fmaxf(x, -3.4e38f), 3.4e38f); }
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
// The bytes of a word that are E4M3 NaN codes, the halves that are bf16 infinities or NaN, as masks
__device__ __forceinline__ uint32_t nan_codes(uint32_t x) {
  const uint32_t top = ((x & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
  return (top << 1) - (top >> 7);
}
__device__ __forceinline__ uint32_t nonfinite(uint32_t x) {
  return ((x & 0x7f80u) == 0x7f80u ? 0xffffu : 0u) | ((x & 0x7f800000u) == 0x7f800000u ? 0xffff0000u : 0u);
}
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// A CTA's position in the work order: the sequence that holds it and where that one's positions begin.
struct Place {
  int b, base, pos, end;
  Seq s;
};
// The part of a unit that comes next: tiles [kt0, kt1) (kt1 <= kt0: only lead-in positions).
struct Piece {
  int kt0, kt1, kvh, rb, lo, ke;
  bool whole;
};

template <class C> __device__ __forceinline__ bool next_piece(const Params &P, Place &at, Piece &p) {
  while (at.pos < at.end) {
    bool bad;
    int work = seq_work(P, at.s);
    while (at.pos - at.base >= work && at.b + 1 < P.s.a.kv.batch) {
      at.base += work;
      at.s = load_seq(P, ++at.b, C::TK, C::RB, &bad);
      work = seq_work(P, at.s);
    }
    if (at.pos - at.base >= work) break;  // cannot happen while the lengths stay put
    const Seq &s = at.s;
    const int U = s.tiles + P.alpha, unit = (at.pos - at.base) / U, off = (at.pos - at.base) - unit * U;
    const int npos = min(U - off, at.end - at.pos);
    at.pos += npos;
    p.kt0 = s.t0 + max(0, off - P.alpha);
    p.kt1 = s.t0 + off + npos - P.alpha;
    if (p.kt1 <= p.kt0) continue;  // only the unit's lead-in lies in this range
    p.kvh = unit / s.rbs;
    p.rb = unit - p.kvh * s.rbs;
    p.whole = p.kt0 == s.t0 && p.kt1 == s.t0 + s.tiles;
    p.ke = min(s.L, p.kt1 * C::TK);
    p.lo = P.s.window > 0 ? max(0, s.c - P.s.window + 1) : 0;
    return true;
  }
  at.pos = at.end;
  return false;
}

template <class C>
__global__ void __launch_bounds__(C::kThreads, C::kCtasPerSm)
    attn_scored_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v, const Params P) {
  grid_dependency_wait();  // the earlier kernel on the stream is complete and visible
  grid_dependents_launch();
  constexpr int D = C::D, NT = C::NT, TK = C::TK, RB = C::RB, WK = C::WK, WR = C::WR, ST = C::kStages, S = C::S, M = C::M;
  constexpr int KT = D / 16;  // 16-value steps of a head
  constexpr int kThreads = C::kThreads, kWarps = kThreads / 32, kC = C::kConsumers * 32;
  constexpr bool F8 = C::F8;
  extern __shared__ uint8_t smem[];
  __shared__ __align__(8) uint64_t s_full[ST], s_free[ST];  // a stage's copies have landed; its steps are done
  __shared__ int s_dead;                                    // a wait gave up
  __shared__ uint64_t s_mask[RB];         // new keys that a row sees
  __shared__ int s_reach[RB], s_row[RB];  // last place out of the window, and row of the sequence (-1: padding)
  __shared__ float s_slope[RB];
  __shared__ int s_place[64];  // position of a new row minus the first one's
  __shared__ float s_m[WK][RB], s_l[WK][RB];
  __shared__ int s_patch;  // a key of the piece's edge steps has an infinity or NaN among its values (kLate)
  __shared__ int s_scan[kWarps], s_first_b, s_first_base, s_top[kWarps];

  const AttnArgs &a = P.s.a;
  const KV &kv = a.kv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int B = kv.batch;
  uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem) + 1023) & ~uintptr_t(1023));
  const uint32_t ring_at = smem_at(ring);
  if (tid == 0) {
    for (int k = 0; k < ST; ++k) {
      bar_init(smem_at(&s_full[k]), 1);
      bar_init(smem_at(&s_free[k]), S * WR);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    s_dead = 0;
    s_first_b = s_first_base = 0;
  }

  // ---- this CTA's range [pos, end) of the launch's W positions ----
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
    for (int w = 0; w < kWarps; ++w) {
      before += w < warp ? s_scan[w] : 0;
      all += s_scan[w];
    }
    __syncthreads();
    *total = all;
    return x + before;
  };
  auto work_of = [&](int b, bool report) {
    bool bad = false;
    const int v = b < B ? seq_work(P, load_seq(P, b, TK, RB, &bad)) : 0;
    if (bad && report && blockIdx.x == 0) record(a.status, SV_ERR_BAD_LENGTH);
    return v;
  };
  int v = work_of(tid, true), W, incl = scan(v, &W), run = 0;  // the first kThreads sequences: most batches whole
  if (B > kThreads) {
    int more = 0, rest;
    for (int b = tid + kThreads; b < B; b += kThreads) more += work_of(b, true);
    run = W;
    scan(more, &rest);
    W += rest;
  }
  Place at;
  at.pos = range_start(blockIdx.x, W, P.ctas);
  at.end = range_start(blockIdx.x + 1, W, P.ctas);
  for (int b0 = 0; b0 < B; b0 += kThreads) {  // the sequence that holds the first position; CTA 0 stores the prefix
    const int b = b0 + tid;
    if (b0 > 0) {
      int tot;
      v = work_of(b, false);
      incl = run + scan(v, &tot);
      run += tot;
    }
    const int excl = incl - v;
    if (blockIdx.x == 0 && b < B) P.prefix[b] = excl;
    if (v > 0 && excl <= at.pos && at.pos < incl) {
      s_first_b = b;
      s_first_base = excl;
    }
    if (blockIdx.x != 0 && b0 > 0 && run > at.pos) break;  // uniform
  }
  if (blockIdx.x == 0 && tid == 0) P.prefix[B] = W;
  __syncthreads();
  at.b = s_first_b;
  at.base = s_first_base;
  {
    bool bad;
    at.s = load_seq(P, at.b, TK, RB, &bad);
  }
  Piece p;
  uint32_t tile0 = 0;  // tiles of the CTA's earlier pieces: tile x of the launch goes to stage x % ST
  bool dead = false;
  auto wait = [&](uint64_t &bar, uint32_t parity) {
    uint32_t done;
    asm volatile("{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
                 : "=r"(done)
                 : "r"(smem_at(&bar)), "r"(parity)
                 : "memory");
    if (__all_sync(0xffffffffu, done != 0) || dead) return;
    const bool landed = mbar_wait_bounded(smem_at(&bar), parity, a.wait_ns);
    dead = __any_sync(0xffffffffu, !landed || *(volatile int *)&s_dead != 0);
    if (dead) s_dead = 1;
  };
  const int bs_shift = __ffs(kv.block_size) - 1;

  // The registers that the launch gives every thread alike (kLaunchRegs) are shared out again. (Each
  // setmaxnreg stands in its own branch: the compiler then allocates each branch by its share.)
  if (warp >= C::kConsumers) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kProducerRegs));
    if (warp == C::kConsumers) {
      // ================= producer =================
      // Lane 2 j (2 j + 1) takes the keys' (values') box of rows j box ... of a tile. Block ids come from a
      // 64-block window of the block table, two entries per lane, loaded one window before they are used.
      const int box = P.box, box_row = (lane >> 1) * box;
      if (a.stall == SV_STALL_ATTENTION) wait(s_free[0], 0);  // failure-path test: a wait that nothing ends
      while (next_piece<C>(P, at, p)) {
        const int32_t *bt = kv.block_table + (size_t)at.b * kv.max_blocks;
        const int last = (p.ke - 1) >> bs_shift;
        auto load_id = [&](int blk) { return blk <= last ? bt[blk] : -1; };
        int wbase = max(p.kt0 * TK, p.lo) >> bs_shift;
        int cur = load_id(wbase + lane), nxt = load_id(wbase + 32 + lane);
        {  // the piece's query rows on their way to L2
          const int R = min(RB, P.G * at.s.n - p.rb * RB);
          for (int x = lane; x < R * (D / 64); x += 32) {
            const int r = p.rb * RB + x / (D / 64), i = r / P.G, head = p.kvh * P.G + r - i * P.G;
            const char *q = reinterpret_cast<const char *>(a.q) + (((size_t)(at.s.row0 + i) * a.num_q_heads + head) * D + x % (D / 64) * 64) * 2;
            asm volatile("prefetch.global.L2 [%0];" ::"l"(q));
          }
        }
        for (int kt = p.kt0; kt < p.kt1; ++kt, ++tile0) {
          const uint32_t st = tile0 % ST;
          const int tok = kt * TK + box_row, first = max(kt * TK, p.lo) >> bs_shift;
          while (first >= wbase + 32) {  // uniform
            wbase += 32;
            cur = nxt;
            nxt = load_id(wbase + 32 + lane);
          }
          // boxes without a key that some row may see are not read
          const bool want = box_row < TK && tok < p.ke && tok + box > p.lo;
          const int src = want ? (tok >> bs_shift) - wbase : 0;
          const int id0 = __shfl_sync(0xffffffffu, cur, src & 31), id1 = __shfl_sync(0xffffffffu, nxt, src & 31);
          const int id = src < 32 ? id0 : id1;
          const bool bad = want && (id < 0 || id >= kv.num_blocks), go = want && !bad;
          if (bad) record(a.status, SV_ERR_BAD_BLOCK_ID);
          if (tile0 >= ST) wait(s_free[st], (tile0 / ST - 1) & 1u);
          if (dead) break;  // nothing more is issued
          const uint32_t bar = smem_at(&s_full[st]);
          const int boxes = __popc(__ballot_sync(0xffffffffu, go));
          if (lane == 0) bar_expect(bar, boxes * box * C::ROWB);
          __syncwarp();
          if (go) {
            const int y = ((id * kv.num_kv_heads + p.kvh) << bs_shift) + (tok & (kv.block_size - 1));
            load_box<C::ROWB>(ring_at + st * C::kStageBytes + (lane & 1) * TK * C::ROWB + box_row * C::ROWB,
                              (lane & 1) ? &map_v : &map_k, y, bar);
          }
          __syncwarp();
        }
        if (dead) break;
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kConsumerRegs));
    // ================= consumers =================
    const int g = lane >> 2, t = lane & 3;
    const int wk = warp % WK, wr = warp / WK;
    float *merge = reinterpret_cast<float *>(ring + C::kRing);  // [consumer][8][kPad]
    auto together = [&] { asm volatile("bar.sync 1, %0;" ::"n"(kC) : "memory"); };
    const float sl2 = F8 ? a.scale_log2 * kv.k_scale : a.scale_log2;
    const float cap = P.s.cap, cap_in = F8 ? finite(P.cap_in * kv.k_scale) : P.cap_in;
    const bool fast_cap = cap <= kFastCap * 1.4426950408889634f;
    const int window = P.s.window;
    const bool biased = P.s.slopes != nullptr;
    const bool bounded = !F8 && cap > 0.f && cap <= kBoundedCap && !biased;
    bool first_piece = true;
    // what ldmatrix adds to a row's place for 16-value step q (mod 4) of its head: chunk 2 q + (0 or 1), swizzled
    const int lr = lane & 7, lm = lane >> 3;
    const int k_row = lm & 1, k_hi = lm >> 1, v_row = F8 ? lm & 1 : lm >> 1, v_hi = F8 ? lm >> 1 : lm & 1;
    constexpr int CH = C::ROWB / 16, kRow = C::ROWB >= 128 ? 128 : 64;  // chunks of a row; bytes between a group's rows
    uint32_t k_off[4], v_off[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      k_off[x] = k_row * 8 * C::ROWB + lr * kRow + (CH >= 8 ? ((x * 2 + k_hi) ^ lr) << 4 : (((x * 2 + k_hi) & 3) ^ ((lr >> 1) & 3)) << 4);
      v_off[x] = TK * C::ROWB + v_row * 8 * C::ROWB + lr * kRow +
                 (CH >= 8 ? ((x * 2 + v_hi) ^ lr) << 4 : (((x * 2 + v_hi) & 3) ^ ((lr >> 1) & 3)) << 4);
    }

    while (next_piece<C>(P, at, p)) {
      const Seq &s = at.s;
      const int c = s.c, ke = p.ke, lo = p.lo, kvh = p.kvh, rb = p.rb;
      const int rows = min(RB, P.G * s.n - rb * RB);  // live rows of the block
      // ---- rows of the block and the new keys' places (every consumer is done with the previous piece's) ----
      int top = c;
      for (int x = tid; x < RB; x += kC) {
        const bool live = x < rows;
        const int r = rb * RB + x, i = live ? r / P.G : 0, head = kvh * P.G + (live ? r - i * P.G : 0);
        const int pos = P.s.positions != nullptr ? P.s.positions[s.row0 + i] : c + i;
        if (pos < c) record(a.status, SV_ERR_BAD_LENGTH);
        s_row[x] = live ? i : -1;
        // places (positions minus c) from reach + 1 on are within the window; new keys are bits of the mask
        s_reach[x] = !live ? 1 << 30 : window > 0 ? pos - c - window : -(1 << 30);
        uint64_t mask = 0ull;
        if (live) {
          mask = a.mask_kind == SV_MASK_TREE ? a.tree_mask[s.row0 + i] : (2ull << i) - 1ull;
          if (s.n < 64) mask &= (1ull << s.n) - 1ull;
          if (window > 0 && pos - c >= window)
            for (int j = 0; j < s.n; ++j) {
              const int place = P.s.positions != nullptr ? P.s.positions[s.row0 + j] - c : j;
              if (place <= pos - c - window) mask &= ~(1ull << j);
            }
        }
        s_mask[x] = mask;
        s_slope[x] = biased ? P.s.slopes[head] * 1.4426950408889634f : 0.f;
        top = max(top, live ? pos : c);
      }
      const int origin = P.s.positions != nullptr ? P.s.positions[s.row0] : c;  // the bias counts from here
      for (int x = tid; x < s.n; x += kC) s_place[x] = P.s.positions != nullptr ? P.s.positions[s.row0 + x] - origin : x;
      top = __reduce_max_sync(0xffffffffu, top);
      if (lane == 0) s_top[warp] = top;
      if (C::kLate && tid == 0) s_patch = 0;

      // ---- Q into registers ----
      uint32_t q[NT][KT][2];
      {
        const uint32_t *src = reinterpret_cast<const uint32_t *>(a.q);
        bool over = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const int rl = (wr * NT + nt) * 8 + g, r = rb * RB + rl, i = r / P.G;
          const bool live = rl < rows;
          const size_t from = live ? ((size_t)(s.row0 + i) * a.num_q_heads + kvh * P.G + (r - i * P.G)) * (D / 2) : 0;
#pragma unroll
          for (int kk = 0; kk < KT; ++kk) {
            if (F8) {
              const uint2 x = live ? *reinterpret_cast<const uint2 *>(src + from + kk * 8 + 2 * t) : make_uint2(0, 0);
              q[nt][kk][0] = pack2<true>(__uint_as_float(x.x << 16), __uint_as_float(x.x & 0xffff0000u));
              q[nt][kk][1] = pack2<true>(__uint_as_float(x.y << 16), __uint_as_float(x.y & 0xffff0000u));
#pragma unroll
              for (int h = 0; h < 2; ++h)
                over |= (q[nt][kk][h] & 0x7c00u) == 0x7c00u || (q[nt][kk][h] & 0x7c000000u) == 0x7c000000u;
            } else {
              q[nt][kk][0] = live ? src[from + kk * 8 + t] : 0u;
              q[nt][kk][1] = live ? src[from + kk * 8 + t + 4] : 0u;
            }
          }
        }
        if (F8 && over) record(a.status, SV_ERR_NONFINITE);  // a query element beyond the fp16 range
      }
      together();
      int row_top = s_top[0];
#pragma unroll
      for (int w = 1; w < C::kConsumers; ++w) row_top = max(row_top, s_top[w]);
      const int all_see = window > 0 ? row_top - window + 1 : 0;  // keys from here to c are visible to every row

      float o[KT][NT][4], m[NT][2], l[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        m[nt][0] = m[nt][1] = bounded ? 0.f : kNone;
        l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
        for (int mt = 0; mt < KT; ++mt) o[mt][nt][0] = o[mt][nt][1] = o[mt][nt][2] = o[mt][nt][3] = 0.f;
      }

      const int steps = (p.kt1 - p.kt0) * S;
      for (int step = wk; step < steps; step += WK) {
        const uint32_t x = tile0 + step / S, st = x % ST;
        wait(s_full[st], (x / ST) & 1u);
        const int key0 = p.kt0 * TK + step * 16 * M;
        if (key0 < ke && key0 + 16 * M > lo) {  // warp-uniform: else nothing to see here
          const uint32_t tile = ring_at + st * C::kStageBytes + (step % S) * 16 * M * C::ROWB;
          // ---- S^T = K Q^T ----
          float sc[M][NT][4];
#pragma unroll
          for (int u = 0; u < M; ++u)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) sc[u][nt][0] = sc[u][nt][1] = sc[u][nt][2] = sc[u][nt][3] = 0.f;
          // ldmatrix results in flight: a read takes as long as five products, and one feeds this many
          constexpr int kFeedK = M * NT * (F8 ? 2 : 1), kFeedV = NT * (F8 ? 2 : 1);
          constexpr int PB = 1 + (4 + kFeedK) / kFeedK, PV = 1 + (4 + kFeedV) / kFeedV;
          constexpr int KL = F8 ? KT / 2 : KT, VL = KL;  // reads of 16 keys, K and V
          auto k_at = [&](int x, int u) { return tile + u * 16 * C::ROWB + k_off[x & 3] + (x >> 2) * 1024; };
          auto v_at = [&](int x) { return tile + x / VL * 16 * C::ROWB + v_off[x % VL & 3] + (x % VL >> 2) * 1024; };
          {
            uint32_t f[PB][M][4];
#pragma unroll
            for (int kk = 0; kk < PB - 1 && kk < KL; ++kk)
#pragma unroll
              for (int u = 0; u < M; ++u) ldm4(f[kk][u], k_at(kk, u));
#pragma unroll
            for (int kk = 0; kk < KL; ++kk) {
              if (kk + PB - 1 < KL) {
#pragma unroll
                for (int u = 0; u < M; ++u) ldm4(f[(kk + PB - 1) % PB][u], k_at(kk + PB - 1, u));
              }
              if (!F8) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                  for (int u = 0; u < M; ++u) mma<false>(sc[u][nt], f[kk % PB][u], q[nt][kk][0], q[nt][kk][1]);
              } else {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  uint32_t e[M][4];
#pragma unroll
                  for (int u = 0; u < M; ++u) {
                    const uint32_t c0 = f[kk % PB][u][2 * h], c1 = f[kk % PB][u][2 * h + 1];
                    e[u][0] = widen(c0), e[u][1] = widen(c1), e[u][2] = widen(c0 >> 16), e[u][3] = widen(c1 >> 16);
                  }
#pragma unroll
                  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int u = 0; u < M; ++u) mma<true>(sc[u][nt], e[u], q[nt][2 * kk + h][0], q[nt][2 * kk + h][1]);
                }
              }
            }
          }
          uint32_t vf[PV][4];  // the first values are on their way during the softmax
#pragma unroll
          for (int y = 0; y < PV - 1; ++y) ldm4t(vf[y], v_at(y));
          // ---- scores ----
          float *const sv = &sc[0][0][0];
          constexpr int kE = M * NT * 4;  // of them; element x: key half (x >> 1) & 1, row x & 1 of its n tile
          if (cap == 0.f) {
#pragma unroll
            for (int y = 0; y < kE; ++y) sv[y] *= sl2;
          } else if (fast_cap) {
#pragma unroll
            for (int y = 0; y < kE; ++y) sv[y] = -2.f * cap * rcp(1.f + ex2(sv[y] * cap_in));
          } else {
#pragma unroll
            for (int y = 0; y < kE; ++y) sv[y] = cap * tanhf(sv[y] * sl2 / cap);
          }
          const bool edge = key0 + 16 * M > min(c, ke) || key0 < all_see;  // warp-uniform: some row may not see some key
          if (biased && !edge) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const float2 sl = *reinterpret_cast<const float2 *>(&s_slope[(wr * NT + nt) * 8 + 2 * t]);
#pragma unroll
              for (int u = 0; u < M; ++u) {
                const float d0 = (float)(key0 + 16 * u + g - origin), d1 = (float)(key0 + 16 * u + g + 8 - origin);
                sc[u][nt][0] = fmaf(sl.x, d0, sc[u][nt][0]);
                sc[u][nt][1] = fmaf(sl.y, d0, sc[u][nt][1]);
                sc[u][nt][2] = fmaf(sl.x, d1, sc[u][nt][2]);
                sc[u][nt][3] = fmaf(sl.y, d1, sc[u][nt][3]);
              }
            }
          }
          bool odd = false;  // an edge step whose values hold an infinity or NaN
          if (edge) {
            const int base = key0 - c;  // place of the step's first key
            if (biased) {
#pragma unroll
              for (int h = 0; h < 2 * M; ++h) {
                const int j = base + g + 8 * h;
                const float place = (float)(j >= 0 && j < s.n ? s_place[j] : c + j - origin);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                  for (int e = 0; e < 2; ++e) {
                    float &v = sc[h >> 1][nt][2 * (h & 1) + e];
                    v = fmaf(s_slope[(wr * NT + nt) * 8 + 2 * t + e], place, v);
                  }
              }
            }
            // A row's view of the step's keys as bits: committed keys beyond its reach, and its mask of new ones.
            const uint32_t old = base >= 0 ? 0u : base <= -32 ? ~0u : (1u << -base) - 1u;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int rl = (wr * NT + nt) * 8 + 2 * t + e, first = s_reach[rl] + 1 - base;
                const uint64_t mask = s_mask[rl];
                const uint32_t near = first <= 0 ? ~0u : first >= 32 ? 0u : ~0u << first;
                const uint32_t fresh =
                    base >= 0 ? (base < 64 ? (uint32_t)(mask >> base) : 0u) : (base > -32 ? (uint32_t)mask << -base : 0u);
                const uint32_t seen = ((old & near) | fresh) >> g;
#pragma unroll
                for (int h = 0; h < 2 * M; ++h) {
                  float &v = sc[h >> 1][nt][2 * (h & 1) + e];
                  v = (seen >> (8 * h)) & 1u ? v : -INFINITY;
                }
              }
            // Do the step's values hold what must not meet a weight of zero? (E4M3: NaN codes of unused slots.)
            constexpr int kChunks = 16 * M * C::ROWB / 16;
            uint8_t *vs = ring + st * C::kStageBytes + (TK + (step % S) * 16 * M) * C::ROWB;
#pragma unroll 4
            for (int y = lane; y < kChunks; y += 32) {
              const uint4 w = *reinterpret_cast<const uint4 *>(vs + y * 16);
              odd |= (F8 ? nan_codes(w.x) | nan_codes(w.y) | nan_codes(w.z) | nan_codes(w.w)
                         : nonfinite(w.x) | nonfinite(w.y) | nonfinite(w.z) | nonfinite(w.w)) != 0u;
            }
            odd = __any_sync(0xffffffffu, odd);
            if constexpr (C::kLate) {  // the rows that see a key get them at the piece's end
              if (odd) {
#pragma unroll 1
                for (int y = lane; y < kChunks * 4; y += 32) {
                  uint32_t *w = reinterpret_cast<uint32_t *>(vs) + y;
                  const uint32_t out = F8 ? nan_codes(*w) : nonfinite(*w);
                  if (out == 0u) continue;
                  if (F8) *w &= ~out;  // (one product for all steps)
                  const int key = key0 + (C::ROWB >= 128 ? y / (2 * C::ROWB) * 8 + y / 32 % 8 : y / 16);
                  if (key >= lo && key < ke) s_patch = 1;
                }
                if (F8) fence_async();  // before the next copies into the stage
              }
              if (F8 && (odd || WR > 1)) {  // (another row group may have been here since the first values were read)
                __syncwarp();
#pragma unroll
                for (int y = 0; y < PV - 1; ++y) ldm4t(vf[y], v_at(y));
              }
            }
          }
          // ---- the running maximum ----
          if (!bounded) {
            bool move = false;
#pragma unroll
            for (int u = 0; u < M; ++u)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  move |= sc[u][nt][e] > m[nt][e & 1] + kMoveAt<F8>;
                }
            if (__any_sync(0xffffffffu, move)) {
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  float mx = fmaxf(sc[0][nt][e], sc[0][nt][e + 2]);
#pragma unroll
                  for (int u = 1; u < M; ++u) mx = fmaxf(mx, fmaxf(sc[u][nt][e], sc[u][nt][e + 2]));
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
            for (int u = 0; u < M; ++u)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) sc[u][nt][e] -= m[nt][e & 1];
          }
          // ---- P^T ----
          uint32_t pb[M][NT][2];
#pragma unroll
          for (int u = 0; u < M; ++u)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
              for (int e = 0; e < 4; ++e) sc[u][nt][e] = ex2(sc[u][nt][e]);
              l[nt][0] += sc[u][nt][0] + sc[u][nt][2];
              l[nt][1] += sc[u][nt][1] + sc[u][nt][3];
              pb[u][nt][0] = turn8x8(pack2<F8>(sc[u][nt][0], sc[u][nt][1]));
              pb[u][nt][1] = turn8x8(pack2<F8>(sc[u][nt][2], sc[u][nt][3]));
            }
          // ---- O^T += V^T P^T ----
          auto pv = [&](auto checked) {  // checked: without infinities and NaN
            constexpr bool kCheck = decltype(checked)::value;
#pragma unroll
            for (int x = 0; x < M * VL; ++x) {
              if (x + PV - 1 < M * VL) ldm4t(vf[(x + PV - 1) % PV], v_at(x + PV - 1));
              uint32_t(&w)[4] = vf[x % PV];
              const int u = x / VL, mt = x % VL;
              if (!F8) {
                if (kCheck) {  // 0 * infinity must not reach a row that does not see the key
#pragma unroll
                  for (int y = 0; y < 4; ++y) {
                    if ((w[y] & 0x7f80u) == 0x7f80u) w[y] &= 0xffff0000u;
                    if ((w[y] & 0x7f800000u) == 0x7f800000u) w[y] &= 0xffffu;
                  }
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) mma<false>(o[mt][nt], w, pb[u][nt][0], pb[u][nt][1]);
              } else {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  // a word: two dimensions of one key below, of the next key above; pairs of keys are wanted
                  const uint32_t w0 = __byte_perm(w[2 * h], 0u, 0x3120), w1 = __byte_perm(w[2 * h + 1], 0u, 0x3120);
                  const uint32_t e[4] = {widen(w0), widen(w0 >> 16), widen(w1), widen(w1 >> 16)};
#pragma unroll
                  for (int nt = 0; nt < NT; ++nt) mma<true>(o[mt * 2 + h][nt], e, pb[u][nt][0], pb[u][nt][1]);
                }
              }
            }
          };
          if (F8 || !odd) {
            pv(std::false_type());
          } else if (C::kLate) {
            pv(std::true_type());
          } else {
            pv(std::true_type());
            // The infinities and NaN set to zero above, for the rows that see their keys, whatever the weight: a weight that
            // is zero in fp32 is not zero.
            const uint8_t *vs = ring + st * C::kStageBytes + (TK + (step % S) * 16 * M) * C::ROWB;
#pragma unroll 1
            for (int key = 0; key < 16 * M; ++key) {
              const int place = key0 + key - c;
              bool sees[NT][2];
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const int rl = (wr * NT + nt) * 8 + 2 * t + e;
                  sees[nt][e] = place < 0 ? place > s_reach[rl] : place < 64 && ((s_mask[rl] >> place) & 1ull) != 0;
                }
#pragma unroll
              for (int mt = 0; mt < KT; ++mt)
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                  const uint32_t w = *reinterpret_cast<const uint16_t *>(vs + (key >> 3) * 8 * C::ROWB + (key & 7) * 128 + (mt >> 2) * 1024 +
                                                                         ((((mt & 3) * 2 + y) ^ (key & 7)) << 4) + g * 2);
                  if ((w & 0x7f80u) != 0x7f80u) continue;
#pragma unroll
                  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                      if (sees[nt][e]) o[mt][nt][2 * y + e] += __uint_as_float(w << 16);
                }
            }
          }
        }
        __syncwarp();
        if (lane == 0) bar_arrive(smem_at(&s_free[st]));
      }
      tile0 += p.kt1 - p.kt0;

      // ---- the key groups' results, merged, 8 rows of each row group at a time ----
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float sum = l[nt][e];
#pragma unroll
          for (int y = 4; y < 32; y <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, y);
          if (g == 0) {
            s_m[wk][(wr * NT + nt) * 8 + 2 * t + e] = m[nt][e];
            s_l[wk][(wr * NT + nt) * 8 + 2 * t + e] = sum;
          }
        }
      const size_t slot = ((size_t)blockIdx.x * 2 + (first_piece ? 0 : 1)) * P.rows_cap;
      bool patch = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int d0 = 0; d0 < D; d0 += C::kChunk) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float *dst = merge + ((wr * WK + wk) * 8 + 2 * t + e) * C::kPad;
#pragma unroll
            for (int mt = 0; mt < C::kChunk / 16; ++mt) {
              dst[mt * 16 + (F8 ? 2 * g : g)] = o[d0 / 16 + mt][nt][e];
              dst[mt * 16 + (F8 ? 2 * g + 1 : g + 8)] = o[d0 / 16 + mt][nt][e + 2];
            }
          }
          together();
          if (nt == 0 && d0 == 0) {  // every group's weight in a row, over the rows' total
            patch = C::kLate && s_patch != 0;
            for (int rl = tid; rl < rows; rl += kC) {
              float mx = s_m[0][rl], tot = 0.f;
#pragma unroll
              for (int w = 1; w < WK; ++w) mx = fmaxf(mx, s_m[w][rl]);  // finite: kNone at the least
#pragma unroll
              for (int w = 0; w < WK; ++w) tot += s_l[w][rl] * ex2(s_m[w][rl] - mx);
              const float inv = tot == 0.f ? 0.f : (F8 ? kv.v_scale : 1.f) / tot;
              if (!p.whole) P.part_lse[slot + rl] = tot == 0.f ? -INFINITY : mx + log2f(tot);
#pragma unroll
              for (int w = 0; w < WK; ++w) s_l[w][rl] = ex2(s_m[w][rl] - mx) * inv;
            }
            together();
          }
          for (int x = tid; x < WR * C::kChunk; x += kC) {  // 8 values of a row
            const int r8 = x / (C::kChunk / 8), d8 = x % (C::kChunk / 8) * 8, rl = ((r8 >> 3) * NT + nt) * 8 + (r8 & 7);
            if (rl >= rows) continue;
            float v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = 0.f;
#pragma unroll
            for (int w = 0; w < WK; ++w) {
              const float f = s_l[w][rl];
              const float4 *src = reinterpret_cast<const float4 *>(merge + (((r8 >> 3) * WK + w) * 8 + (r8 & 7)) * C::kPad + d8);
              const float4 x0 = src[0], x1 = src[1];
              v[0] = fmaf(f, x0.x, v[0]), v[1] = fmaf(f, x0.y, v[1]), v[2] = fmaf(f, x0.z, v[2]), v[3] = fmaf(f, x0.w, v[3]);
              v[4] = fmaf(f, x1.x, v[4]), v[5] = fmaf(f, x1.y, v[5]), v[6] = fmaf(f, x1.z, v[6]), v[7] = fmaf(f, x1.w, v[7]);
            }
            if (p.whole) {
              const int i = s_row[rl], head = kvh * P.G + (rb * RB + rl) - i * P.G;
              *reinterpret_cast<uint4 *>(reinterpret_cast<__nv_bfloat16 *>(a.out) +
                                         ((size_t)(s.row0 + i) * a.num_q_heads + head) * D + d0 + d8) =
                  make_uint4(pack2<false>(v[0], v[1]), pack2<false>(v[2], v[3]), pack2<false>(v[4], v[5]), pack2<false>(v[6], v[7]));
            } else {
              float4 *dst = reinterpret_cast<float4 *>(P.part_o + (slot + rl) * D + d0 + d8);
              dst[0] = make_float4(v[0], v[1], v[2], v[3]);
              dst[1] = make_float4(v[4], v[5], v[6], v[7]);
            }
          }
          together();
        }
      if (patch) {
        // The infinities and NaN that edge steps took out, for the rows that see their keys, whatever the weight: looked for in
        // the pool again and added to what has been written.
#pragma unroll 1
        for (int x = tid; x < rows * D; x += kC) {
          const int rl = x / D, d = x % D;
          float add = 0.f;
#pragma unroll 1
          for (int key = max(p.kt0 * TK, lo); key < ke; ++key) {
            const int key0 = key & ~(16 * M - 1), place = key - c;
            if (!(key0 + 16 * M > min(c, ke) || key0 < all_see)) {  // on to the next edge step
              key = (min(c, ke) & ~(16 * M - 1)) - 1;
              continue;
            }
            if (!(place < 0 ? place > s_reach[rl] : (s_mask[rl] >> place) & 1ull)) continue;
            const int id = kv.block_table[(size_t)at.b * kv.max_blocks + (key >> bs_shift)];
            if (id < 0 || id >= kv.num_blocks) continue;
            const size_t from = (((size_t)id * kv.num_kv_heads + kvh) * kv.block_size + (key & (kv.block_size - 1))) * D + d;
            const uint32_t w = F8 ? static_cast<const uint8_t *>(kv.v_pool)[from] : static_cast<const uint16_t *>(kv.v_pool)[from];
            if ((F8 ? nan_codes(w) : nonfinite(w)) != 0u) add += __uint_as_float(F8 ? 0x7fffffffu : w << 16);
          }
          if (add == 0.f) continue;
          if (p.whole) {
            const int i = s_row[rl], head = kvh * P.G + (rb * RB + rl) - i * P.G;
            __nv_bfloat16 *dst = reinterpret_cast<__nv_bfloat16 *>(a.out) + ((size_t)(s.row0 + i) * a.num_q_heads + head) * D + d;
            *dst = __float2bfloat16_rn(__bfloat162float(*dst) + add);
          } else {
            P.part_o[(slot + rl) * D + d] += add;
          }
        }
        together();
      }
      first_piece = false;
    }
  }
  if (dead && lane == 0) record(a.status, SV_ERR_TIMEOUT);
  __syncthreads();
  // after a wait that gave up: the copies in flight land before the CTA's shared memory is released
  if (s_dead && warp == C::kConsumers)
    for (uint32_t x = tile0 > ST ? tile0 - ST : 0; x < tile0; ++x)
      mbar_wait_bounded(smem_at(&s_full[x % ST]), (x / ST) & 1u, kDrainBudgetNs);
}

// Merges the partials of every unit that two or more CTAs shared: o = sum_p 2^lse_p o_p / sum_p 2^lse_p,
// in the order of the CTAs. A thread takes 8 values of a row, the loads of four pieces in flight, or of eight where
// a unit has 8 rows at most: those may be cut into many (one sequence of 32K tokens 41 -> 36 us), while wider
// ones mostly have two or three (32 x 6 rows 61 -> 63 us with eight).
// CTA (x, y) has kMergeThreads items of unit x, or (BORDERS) of the unit on the border between the ranges of CTAs x
// and x + 1, if that is its first. Launches with more units than CTAs go by borders, most units being whole
// (128 x 5 rows over 600 tokens 95.4 -> 93.8 us); for the others finding a border's unit costs more (32 x 6 rows
// 60.9 -> 62.7).
constexpr int kMergeThreads = 256;
template <class C, bool BORDERS>
__global__ void __launch_bounds__(kMergeThreads) attn_scored_combine(const Params P) {
  grid_dependents_launch();
  grid_dependency_wait();  // the earlier kernel on the stream is complete and visible
  constexpr int D = C::D;
  const AttnArgs &a = P.s.a;
  const int B = a.kv.batch, W = P.prefix[B];
  int b, of_seq = 0, border = 0;  // the unit's sequence, and its place in it or the border
  if (BORDERS) {
    if (W <= 0) return;
    border = range_start(blockIdx.x + 1, W, P.ctas);
    if (border >= W) return;
    const int lane = threadIdx.x & 31;
    b = 0;  // the last sequence that begins there or before
    for (int len = B; len > 1;) {
      const int step = (len + 31) >> 5;
      const bool below = lane * step < len && P.prefix[b + lane * step] <= border;
      const int k = max(0, __popc(__ballot_sync(0xffffffffu, below)) - 1);
      b += k * step;
      len = min(step, len - k * step);
    }
  } else {
    b = blockIdx.x % B;
    of_seq = blockIdx.x / B;
  }
  bool bad;
  const int base = P.prefix[b];
  const Seq s = load_seq(P, b, C::TK, C::RB, &bad);
  if (s.tiles <= 0) return;
  const int U = s.tiles + P.alpha, unit = BORDERS ? (border - base) / U : of_seq;
  if (!BORDERS && unit >= a.kv.num_kv_heads * s.rbs) return;
  const int kvh = unit / s.rbs, rb = unit - kvh * s.rbs;
  const int T0 = base + unit * U + P.alpha, T1 = T0 + s.tiles;
  const int c0 = range_owner(T0, W, P.ctas), c1 = range_owner(T1 - 1, W, P.ctas);
  // one CTA held the whole unit and wrote its rows, or another border of it comes first
  if (c0 == c1 || (BORDERS && c0 != (int)blockIdx.x)) return;
  // the unit is CTA c0's first piece only if its range starts within the unit's lead-in
  const int slot0 = range_start(c0, W, P.ctas) >= T0 - P.alpha ? 0 : 1;
  constexpr int kPc = C::RB <= 8 ? 8 : 4;
  const int rows = min(C::RB, P.G * s.n - rb * C::RB);
  const int x = blockIdx.y * kMergeThreads + threadIdx.x;
  if (x < rows * (D / 8)) {
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
        const bool in = cb + k <= c1 && (W >= P.ctas || range_start(cb + k, W, P.ctas) < range_start(cb + k + 1, W, P.ctas));
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
  int ctas, rows_cap;
  long long units;  // if every sequence has max_q rows
  size_t lse_offset, prefix_offset, bytes;  // bytes 0: the work order does not fit its 32-bit positions
};

template <class C>
Layout layout_of(const KV &kv, int G, int max_q, int max_seq_len) {
  Layout l;
  const int blocks = (G * max_q + C::RB - 1) / C::RB;
  l.units = (long long)kv.batch * kv.num_kv_heads * blocks;
  const int unit_tiles = (max_seq_len + C::TK - 1) / C::TK;
  const long long tiles = l.units * unit_tiles;
  l.ctas = (int)std::max(1LL, std::min<long long>((long long)C::kCtasPerSm * num_sms(), tiles));
  l.rows_cap = std::min(C::RB, G * max_q);
  const size_t slots = (size_t)l.ctas * 2 * l.rows_cap;
  l.lse_offset = slots * C::D * sizeof(float);
  l.prefix_offset = (l.lse_offset + slots * sizeof(float) + 255) / 256 * 256;
  // A unit has at most unit_tiles + kAlpha positions, with this instance's own tile and block of rows; positions,
  // their sums over the batch and the prefix are 32-bit.
  const bool fits = l.units <= INT_MAX / (unit_tiles + C::kAlpha);
  l.bytes = fits ? l.prefix_offset + ((size_t)kv.batch + 1) * sizeof(int) : 0;
  return l;
}

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

// A call's parameters and the size of its workspace (0: not a call for this instance).
template <class C>
Layout plan(const ScoredArgs &sa, void *workspace, size_t *bytes, Params *p) {
  const KV &kv = sa.a.kv;
  p->s = sa;
  p->G = sa.a.num_q_heads / kv.num_kv_heads;
  const Layout l = layout_of<C>(kv, p->G, sa.a.max_q, sa.a.max_seq_len);
  *bytes = l.bytes;
  p->cap_in = sa.cap > 0.f ? finite(sa.a.scale_log2 * 2.f * 1.4426950408889634f / sa.cap) : 0.f;
  p->ctas = l.ctas;
  p->alpha = C::kAlpha;
  p->rows_cap = l.rows_cap;
  p->box = std::min(kv.block_size, C::TK);
  p->part_o = reinterpret_cast<float *>(workspace);
  p->part_lse = reinterpret_cast<float *>(reinterpret_cast<uint8_t *>(workspace) + l.lse_offset);
  p->prefix = reinterpret_cast<int *>(reinterpret_cast<uint8_t *>(workspace) + l.prefix_offset);
  return l;
}

template <class C> cudaError_t launch_combine(const Params &p, const Layout &l, cudaStream_t st) {
  if (l.ctas <= 1) return cudaSuccess;  // no borders
  const unsigned y = (l.rows_cap * (C::D / 8) + kMergeThreads - 1) / kMergeThreads;
  if (l.units > l.ctas) return launch_pdl(attn_scored_combine<C, true>, dim3(l.ctas - 1, y), dim3(kMergeThreads), 0, st, p);
  return launch_pdl(attn_scored_combine<C, false>, dim3((unsigned)l.units, y), dim3(kMergeThreads), 0, st, p);
}

// Launches (`go`) or sizes one instance.
template <class C>
cudaError_t run(const ScoredArgs &sa, void *workspace, size_t *bytes, cudaStream_t st, bool go) {
  const KV &kv = sa.a.kv;
  Params p;
  const Layout l = plan<C>(sa, workspace, bytes, &p);
  if (!go || *bytes == 0) return cudaSuccess;
  static const bool split_fits = [] {  // the kernel was compiled for the registers that its split shares out
    cudaFuncAttributes fa;
    return cudaFuncGetAttributes(&fa, attn_scored_kernel<C>) == cudaSuccess && fa.numRegs == kLaunchRegs;
  }();
  if (!split_fits) return cudaErrorInvalidConfiguration;
  CUtensorMap mk, mv;
  if (!make_map<C>(&mk, kv.k_pool, kv, p.box) || !make_map<C>(&mv, kv.v_pool, kv, p.box)) return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(attn_scored_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem);
  if (e != cudaSuccess) return e;
  e = launch_pdl(attn_scored_kernel<C>, dim3(p.ctas), dim3(C::kThreads), C::kSmem, st, mk, mv, p);
  if (e != cudaSuccess) return e;
  return launch_combine<C>(p, l, st);
}

// Units of more query rows go to attn_scored_wide.cu, where it takes them: with 64 rows a KV head 32 sequences of 2K to
// 4K tokens take 106 us here and 97 there, 64 of 200 to 300 tokens 64 and 50; with 48 rows 96 and 100.
constexpr int kWideRows = 48;
bool wide_fits(const ScoredArgs &sa);
cudaError_t run_wide(const ScoredArgs &sa, void *workspace, size_t *bytes, cudaStream_t st, bool go);

// The smallest block of query rows that holds a unit's, else blocks of the largest.
template <int D, bool F8>
cudaError_t pick(const ScoredArgs &sa, void *workspace, size_t *bytes, cudaStream_t st, bool go) {
  const int rows = sa.a.num_q_heads / sa.a.kv.num_kv_heads * sa.a.max_q;
  auto on = [&](auto cfg) { return run<decltype(cfg)>(sa, workspace, bytes, st, go); };
  if constexpr (D == 64) {
    if (rows <= 8) return on(Cfg<D, 1, 1, 4, F8>());
    if (rows <= 16) return on(Cfg<D, 2, 1, 4, F8>());
    if (rows <= 32) return on(Cfg<D, 4, 1, 4, F8>());
    if (rows <= 48) return on(Cfg<D, 3, 2, 2, F8>());
    if (rows <= 64) return on(Cfg<D, 4, 2, 2, F8>());
    return on(Cfg<D, 4, 4, 1, F8>());
  } else if constexpr (D == 128) {
    if (rows <= 8) return on(Cfg<D, 1, 1, 4, F8>());
    if (rows <= 16) return on(Cfg<D, 2, 1, 4, F8>());
    if (rows <= 24) return on(Cfg<D, 3, 1, 4, F8>());
    if (rows <= 32) return on(Cfg<D, 2, 2, 2, F8>());
    if (rows <= 48) return on(Cfg<D, 3, 2, 2, F8>());
    auto here = [&] { return rows <= 64 ? on(Cfg<D, 2, 4, 1, F8>()) : on(Cfg<D, 3, 4, 1, F8>()); };
    if (!wide_fits(sa)) return here();
    // a cap past the two-instruction tanh stays here; the workspace suits both, and so do the positions
    size_t most = 0;
    run_wide(sa, nullptr, &most, st, false);
    if (go && sa.cap <= kFastCap * 1.4426950408889634f) return run_wide(sa, workspace, bytes, st, go);
    const cudaError_t e = here();
    *bytes = *bytes == 0 || most == 0 ? 0 : std::max(*bytes, most);
    return e;
  } else {
    if (rows <= 16) return on(Cfg<D, 1, 2, 2, F8>());
    return on(Cfg<D, 1, 4, 1, F8>());
  }
}

}  // namespace scored
}  // namespace sv
