// Attention with modified scores for wide units (more than kWideRows query rows per KV head and sequence:
// draft trees, long drafts, wide query groups) on the 5th-generation tensor cores: bf16 and E2M1 caches with
// heads of 128 values. The mathematics, the work order, the partials and their merge are those of
// attn_scored.cuh.
//
// Bound: the special functions and what surrounds them. 256 query rows a unit are 256 flops per byte of K
// and V, past what memory limits. Of 64 keys for 256 rows the two products take an estimated 1000 cycles of an SM
// (Q is read from shared memory again for each tile), the softmax 1300 with a cap (two 2^x and a quarter of a
// reciprocal a score) and 500 without. Measured is 3000 and 2800 a tile: a warp's read, cap, maximum, weights
// and write are a chain, and two warps a scheduler hide only part of it.
//
// Times (us, bf16, 8 KV heads of 128 values; in brackets the warp-matrix kernels of attn_scored.cuh):
//   16 trees of 61 rows x 4 heads over 8192 tokens, capped 192 [455], 690 TFLOP/s;
//   32 sequences over 2K to 4K tokens: 256 rows a KV head 177 capped, 147 without [407 capped],
//   128 rows 116, 108 [270], 100 rows 107 [271], 72 rows 106 [168], 64 rows 97 [106].
//
// A unit is one KV head of one sequence and up to 256 query rows, as two blocks of 128, one row per
// tensor-memory lane, so that K and V are read once for all of them. One CTA an SM, eleven warps:
//  * softmax a and b, four warps each: a thread keeps one row. It reads its 64 scores from tensor memory,
//    caps, biases and masks them, moves its running maximum if they pass it by far (then rescales its
//    row of O), and writes P = 2^(s - m) as bf16 over the scores;
//  * the producer: K and V tiles of 64 keys (2 x 16 KB) by TMA into the stages;
//  * two issuers, a block each (one lane): S = Q K^T (M 128, N 64, both operands in shared memory) into one
//    of the block's two S buffers, then O += P V (P in tensor memory, V with its dimensions major):
//      S(t + 1), P V(t), S(t + 2), P V(t + 1), ...
//    so the next scores are there when a row is done with its last ones. Products of one thread finish
//    in the order of their issue: S(t + 1) may overwrite P(t - 1), whose product was issued before it.
// Tensor memory: S_a, S_b (two buffers of 64 columns each, P over them), O_a, O_b (128 each): all 512 columns.
// Before a piece its rows zero O, so every P V accumulates.
//
// (128 keys a tile with one S buffer a block waited a third of its time for the next scores, one issuer for
// both blocks made each wait for the other: the trees took 278 and 274 us, against 247 with these in place of
// them.) Where a cap bounds the scores, 32 of them become weights while the other 32 are read, with no maximum.
//
// A unit of 128 rows or fewer is one block: a and b hold the same rows, take a tile each in turn, and merge
// their rows at the end. The values of both lie in the same lanes of tensor memory, so a row's two warps
// exchange m and l alone and write half of its values each. (100 rows, with b idle: 170 us; both at work with
// four stages 130, with Q once and six 116; 107 with pieces cut by what starting one costs.) Launches whose
// units may be larger leave b idle in smaller ones.
//
// Edge tiles (new rows, the window's start, the end) see keys as bits of a row. Values past the end of
// the sequence are set to zero in the stage; infinities and NaN of keys that some row does not see are
// taken out of it too, and added to the rows that see them by hand.
//
// Weights are bf16 for the product with V (2^-8 of themselves at most), and the cap's reciprocals and 2^x the approximate
// ones (2^-19 of the cap), as in attn_scored.cuh.
//
// E2M1 caches (CODES): four converters stand in the producer's place, one a scheduler, two of K and two of V. Each has a ring of
// its own, three tiles of asynchronous 16-byte copies that run on into the CTA's next piece, and writes the fp16 values (exact,
// e2m1.cuh) where the TMA would have put them. Q becomes fp16 next to a power of two of its row, as in attn_e2m1.cuh,
// and joins the row's factor; weights are fp16 (as there), so the running maximum stays for
// capped scores too. Trees as above, not capped: 169 us, 780 TFLOP/s (595 on warp-level instructions; 184 with the codes
// a tile ahead in registers). 32 sequences over 2K to 4K tokens: 256 rows a KV head 146, 128 rows 124, 64 rows 117.
// A tile takes 3000 cycles whether 128 rows meet it or 256: a converter is busy for 1700 of them (800 for the copies' addresses,
// 850 for its 64 conversions a lane), and a tile's way from there to the end of P V is long.
// Registers: four warps more, so fewer for each. The others' 80 is where nothing they use in a loop spills (64 took 40% longer for
// 64 rows and 8% for the trees); their places in the order are in shared memory for that. The softmax's 176 spill 286 and 434
// bytes (up to 128 rows): 0.7% of the trees' instructions.
//
// All waits are bounded, as in attn_scored.cuh.
#include <algorithm>

#include "attn_scored.cuh"
#include "e2m1.cuh"

namespace sv {
namespace scored {
namespace {

struct Wide {  // what the work order and the merge need
  static constexpr int D = 128, TK = 64, RB = 256, ROWB = 256, kCtasPerSm = 1;
  // (72, 128 and 256 rows a KV head over 2K to 4K tokens: 4 111, 123 and 186 us, 13 106, 115 and 177, 26 111, 118, 188)
  static constexpr int kAlpha = 12;
};
constexpr int kSoft = 8;                   // softmax warps
// Register shares go by four warps: the producer, two issuers and one that does nothing; with codes the two issuers, two
// that do nothing, and four converters.
template <bool CODES>
constexpr int kOthers = CODES ? 8 : 4;
template <bool CODES>
constexpr int kWideThreads = (kSoft + kOthers<CODES>) * 32;
// Registers of a thread as launched, of the softmax warps and of the others after the split
template <bool CODES>
constexpr int kWideRegs = CODES ? 128 : 168;
template <bool CODES>
constexpr int kSoftRegs = CODES ? 176 : 216;
template <bool CODES>
constexpr int kOtherRegs = CODES ? 80 : 72;
template <bool CODES>
constexpr bool kSplitFits = kSoft * kSoftRegs<CODES> + kOthers<CODES> * kOtherRegs<CODES> == (kSoft + kOthers<CODES>) * kWideRegs<CODES>;
static_assert(kSplitFits<false> && kSplitFits<true>, "a split above the launch's share would wait forever");
constexpr int kTile = Wide::TK;            // keys of a tile
constexpr int kBlock = 128;                // rows of a block
constexpr int kHalf = kTile * 256;         // bytes of a tile's K or V
constexpr int kStage = 2 * kHalf;
constexpr int kQBytes = kBlock * 256;      // of a block
// One block of rows: its Q once, and two stages more (the blocks hold two tiles each)
template <bool ONE, bool CODES>
constexpr int kStages = !ONE ? 4 : CODES ? 5 : 6;
constexpr int kRaw = 32 * 72, kAhead = 3;  // codes: bytes of a converter's 32 keys; so many tiles are on their way or there
template <bool ONE, bool CODES>
constexpr int kWideSmem = 1024 + kStages<ONE, CODES> * kStage + (ONE ? 1 : 2) * kQBytes + (CODES ? 4 * kAhead * kRaw : 0);
static_assert(kWideSmem<true, true> + 2048 <= 227 * 1024 && kWideSmem<false, true> + 2048 <= 227 * 1024, "shared memory of an SM");
constexpr int kColO = 256;                 // S_a 0 (and 64), S_b 128 (and 192), O_a 256, O_b 384

__device__ __forceinline__ uint64_t operand(uint32_t at, uint32_t lbo, uint32_t sbo) {  // 128-byte swizzle
  return (uint64_t)((at & 0x3FFFF) >> 4) | (uint64_t)((lbo >> 4) & 0x3FFF) << 16 | (uint64_t)((sbo >> 4) & 0x3FFF) << 32 |
         (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
// kind::f16, fp32 accumulate, bf16 operands (fp16 ones of codes), M 128; N 64 (keys), and N 128 (values) with B's N
// dimension major
template <bool CODES>
constexpr uint32_t kTypes = (1u << 4) | (CODES ? 0u : (1u << 7) | (1u << 10));
template <bool CODES>
constexpr uint32_t kIdescS = kTypes<CODES> | (8u << 17) | (8u << 24);
template <bool CODES>
constexpr uint32_t kIdescV = kTypes<CODES> | (1u << 16) | (16u << 17) | (8u << 24);

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, int accumulate) {
  asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
               "l"(a), "l"(b), "r"(idesc), "r"(accumulate));
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, int accumulate) {
  asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
               "r"(a), "l"(b), "r"(idesc), "r"(accumulate));
}
__device__ __forceinline__ void commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
// True in one lane of a full warp, the same one each time. (Under `lane == 0` a product took 84 to 144 cycles to
// issue: the compiler does not know that its operands are one thread's.)
__device__ __forceinline__ bool elected() {
  uint32_t yes;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(yes));
  return yes != 0;
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

#define SV_O8(x, o) "=r"(x[o]), "=r"(x[o + 1]), "=r"(x[o + 2]), "=r"(x[o + 3]), "=r"(x[o + 4]), "=r"(x[o + 5]), "=r"(x[o + 6]), "=r"(x[o + 7])
#define SV_I8(x, o) "r"(x[o]), "r"(x[o + 1]), "r"(x[o + 2]), "r"(x[o + 3]), "r"(x[o + 4]), "r"(x[o + 5]), "r"(x[o + 6]), "r"(x[o + 7])
// 32 columns of this thread's lane
__device__ __forceinline__ void tmem_get(uint32_t at, uint32_t *x) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,"
      "%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : SV_O8(x, 0), SV_O8(x, 8), SV_O8(x, 16), SV_O8(x, 24)
      : "r"(at));
}
__device__ __forceinline__ void tmem_put(uint32_t at, const uint32_t *x) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,"
      "%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(at),
      SV_I8(x, 0), SV_I8(x, 8), SV_I8(x, 16), SV_I8(x, 24)
      : "memory");
}
// What this thread has asked for has arrived; x passes through, so that nothing is made of it before
#define SV_P8(x, o) "+r"(x[o]), "+r"(x[o + 1]), "+r"(x[o + 2]), "+r"(x[o + 3]), "+r"(x[o + 4]), "+r"(x[o + 5]), "+r"(x[o + 6]), "+r"(x[o + 7])
__device__ __forceinline__ void tmem_landed(uint32_t *x) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" : SV_P8(x, 0), SV_P8(x, 8), SV_P8(x, 16), SV_P8(x, 24)::"memory");
}
__device__ __forceinline__ void tmem_put_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// the smaller of two, a NaN if one is
__device__ __forceinline__ float min_nan(float x, float y) {
  float z;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(z) : "f"(x), "f"(y));
  return z;
}
// cap (tanh(x / cap') - 1) = -2 cap / (1 + 2^(x in)) of four scores with one reciprocal: 1/a = bcd / (abcd) and so
// on. Past 2^30 tanh is 1 in fp32, and the product stays finite. A NaN in one is a NaN in all.
// (16 trees of 61 rows over 8192 tokens: a reciprocal each 278 us, for two 218, for four 206. The kernels of
// attn_scored.cuh gain nothing by it: other instructions bound them.)
__device__ __forceinline__ void cap_four(float (&x)[4], float in, float cap) {
  float e[4];
#pragma unroll
  for (int y = 0; y < 4; ++y) e[y] = 1.f + ex2(min_nan(x[y] * in, 30.f));
  const float ab = e[0] * e[1], cd = e[2] * e[3], all = -2.f * cap * rcp(ab * cd), of_ab = all * cd, of_cd = all * ab;
  x[0] = of_ab * e[1];
  x[1] = of_ab * e[0];
  x[2] = of_cd * e[3];
  x[3] = of_cd * e[2];
}

// byte of (row, 16-byte chunk of its 16) in 128 rows as the TMA lays them
__device__ __forceinline__ uint32_t chunk_at(int row, int chunk) {
  return (row >> 3) * 2048 + (chunk >> 3) * 1024 + (row & 7) * 128 + (((chunk & 7) ^ (row & 7)) << 4);
}

// The halves of a word that are fp16 infinities or NaN, as a mask
__device__ __forceinline__ uint32_t nonfinite16(uint32_t x) {
  return ((x & 0x7c00u) == 0x7c00u ? 0xffffu : 0u) | ((x & 0x7c000000u) == 0x7c000000u ? 0xffff0000u : 0u);
}

template <bool ONE, bool CODES>
__global__ void __launch_bounds__(kWideThreads<CODES>, 1)
    attn_scored_wide_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v, const Params P) {
  grid_dependency_wait();  // the earlier kernel on the stream is complete and visible
  grid_dependents_launch();
  constexpr int kThreads = kWideThreads<CODES>, kWarps = kThreads / 32, kWideStages = kStages<ONE, CODES>;
  extern __shared__ uint8_t smem[];
  __shared__ __align__(8) uint64_t s_full[kWideStages], s_free[kWideStages];  // stages
  __shared__ __align__(8) uint64_t s_q[2], s_s[2][2], s_p[2][2], s_o[2][2];  // blocks: Q written; by buffer S there, P written, P V done
  __shared__ __align__(8) uint64_t s_seen;                // one block of rows: the second issuer is past a piece without work
  __shared__ __align__(8) uint64_t s_done;                // every product issued has finished
  __shared__ Place s_at[CODES ? kOthers<CODES> : 1];  // of the warps with few registers: where they are in the order
  __shared__ int s_dead, s_scan[kWarps], s_first_b, s_first_base;
  __shared__ uint32_t s_tmem;
  __shared__ int s_place[64], s_top[kSoft];
  __shared__ float2 s_ml[ONE ? kBlock : 1];  // a block's m and l, on their way to the other

  const AttnArgs &a = P.s.a;
  const KV &kv = a.kv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int B = kv.batch;
  uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem) + 1023) & ~uintptr_t(1023));
  uint8_t *qs = ring + kWideStages * kStage;  // Q of block a, of block b (one block of rows: of both)
  if (tid == 0) {
    for (int k = 0; k < kWideStages; ++k) {
      bar_init(smem_at(&s_full[k]), CODES ? 4 : 1);
      bar_init(smem_at(&s_free[k]), 2);
    }
    for (int k = 0; k < 2; ++k) {
      bar_init(smem_at(&s_q[k]), ONE ? 8 : 4);
      bar_init(smem_at(&s_s[k][0]), 1);
      bar_init(smem_at(&s_s[k][1]), 1);
      bar_init(smem_at(&s_p[k][0]), 4);
      bar_init(smem_at(&s_p[k][1]), 4);
      bar_init(smem_at(&s_o[k][0]), 1);
      bar_init(smem_at(&s_o[k][1]), 1);
    }
    bar_init(smem_at(&s_seen), 1);
    bar_init(smem_at(&s_done), 2);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    s_dead = 0;
    s_first_b = s_first_base = 0;
  }
  if (warp == kSoft + 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_at(&s_tmem)), "r"(512) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
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
    const int v = b < B ? seq_work(P, load_seq(P, b, Wide::TK, Wide::RB, &bad)) : 0;
    if (bad && report && blockIdx.x == 0) record(a.status, SV_ERR_BAD_LENGTH);
    return v;
  };
  int v0 = work_of(tid, true), W, incl = scan(v0, &W), run = 0;
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
  for (int b0 = 0; b0 < B; b0 += kThreads) {
    const int b = b0 + tid;
    if (b0 > 0) {
      int tot;
      v0 = work_of(b, false);
      incl = run + scan(v0, &tot);
      run += tot;
    }
    const int excl = incl - v0;
    if (blockIdx.x == 0 && b < B) P.prefix[b] = excl;
    if (v0 > 0 && excl <= at.pos && at.pos < incl) {
      s_first_b = b;
      s_first_base = excl;
    }
    if (blockIdx.x != 0 && b0 > 0 && run > at.pos) break;  // uniform
  }
  if (blockIdx.x == 0 && tid == 0) P.prefix[B] = W;
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = s_tmem;
  at.b = s_first_b;
  at.base = s_first_base;
  {
    bool bad;
    at.s = load_seq(P, at.b, Wide::TK, Wide::RB, &bad);
  }
  Piece p = {};
  bool dead = false;
  auto wait = [&](uint64_t &bar, uint32_t parity) {
    if (dead) return;
    const bool landed = mbar_wait_bounded(smem_at(&bar), parity, a.wait_ns);
    dead = __any_sync(0xffffffffu, !landed || *(volatile int *)&s_dead != 0);
    if (dead) s_dead = 1;
  };
  uint32_t tile0 = 0;  // tiles of the CTA's earlier pieces: tile x of the launch goes to stage x % kWideStages
  auto two_blocks = [&] { return !ONE && P.G * at.s.n - p.rb * Wide::RB > kBlock; };
  auto active = [&](int blk) { return blk == 0 || (ONE ? p.kt1 - p.kt0 > 1 : two_blocks()); };  // has a part in the piece

  if (warp >= kSoft) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs<CODES>));
    if (CODES && lane == 0) s_at[warp - kSoft] = at;
    __syncwarp();
    auto advance = [&] {
      if constexpr (!CODES) return next_piece<Wide>(P, at, p);
      at = s_at[warp - kSoft];
      __syncwarp();
      const bool has = next_piece<Wide>(P, at, p);
      if (lane == 0) s_at[warp - kSoft] = at;
      __syncwarp();
      return has;
    };
    if (CODES && warp >= kSoft + 4) {
      // ================= converters: two of K, two of V, half of a tile's keys each =================
      const int half = (warp & 1) * 4, bs_shift = __ffs(kv.block_size) - 1;  // the first of its 4 runs of 8 keys
      const bool val = warp >= kSoft + 6;
      const uint8_t *codes = (const uint8_t *)(val ? kv.v_pool : kv.k_pool), *scales = val ? kv.v_bs : kv.k_bs;
      const uint32_t raw = smem_at(qs) + (ONE ? 1 : 2) * kQBytes + (warp & 3) * kAhead * kRaw;
      if (a.stall == SV_STALL_ATTENTION) wait(s_free[0], 0);  // failure-path test: a wait that nothing ends
      int kt = 0, id = 0, ahead = 0;  // next tile to be asked for; lane y & 3: the block of its y-th run; tiles asked for and not yet written
      uint32_t put = 0, get = 0;
      bool more = advance();
      auto look = [&] {  // which blocks the next tile's keys lie in; the numbers arrive while the last tile is converted
        const int key = kt * Wide::TK + 8 * (half + (lane & 3));
        if (key < p.ke && key + 8 > p.lo) id = kv.block_table[(size_t)at.b * kv.max_blocks + (key >> bs_shift)];
      };
      auto bring = [&] {
        const int k0 = kt * Wide::TK + 8 * half;
        const int first = k0 + 8 * (lane & 3);
        const bool want = first < p.ke && first + 8 > p.lo, bad = want && (id < 0 || id >= kv.num_blocks);
        if (bad) record(a.status, SV_ERR_BAD_BLOCK_ID);
        const int mine = !want || bad ? -1 : ((id * kv.num_kv_heads + p.kvh) << bs_shift) + (first & (kv.block_size - 1));
        const uint32_t dst = raw + put * kRaw;
        put = put + 1 == kAhead ? 0 : put + 1;
        const int r8 = lane >> 2, c = lane & 3;
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const int row = __shfl_sync(0xffffffffu, mine, y), key = k0 + 8 * y + r8;
          copy_some(dst + (8 * y + r8) * 64 + ((c ^ ((r8 >> 1) & 3)) << 4), codes + (size_t)(max(row, 0) + r8) * 64 + c * 16,
                    row >= 0 && key >= p.lo && key < p.ke ? 16 : 0);  // a place that is no key's is zeros
        }
        const int row = __shfl_sync(0xffffffffu, mine, (lane >> 2) & 3), key = k0 + 2 * lane;  // scales: 16 bytes are two keys'
        if (lane < 16) copy_some(dst + 32 * 64 + lane * 16, scales + (size_t)(max(row, 0) + 2 * c) * 8, row >= 0 ? max(0, min(16, (p.ke - key) * 8)) : 0);
        asm volatile("cp.async.commit_group;" ::: "memory");
        ++ahead;
        if (++kt == p.kt1) {
          more = advance();
          kt = p.kt0;
        }
        if (more) look();
      };
      kt = p.kt0;
      if (more) look();
      const int r8 = lane & 7, ch = lane >> 3;  // a lane's row of 8, its 32 values
      while (true) {
        while (more && ahead < kAhead) bring();
        if (ahead == 0) break;
        if (ahead == kAhead) copies_wait<kAhead - 1>();
        else copies_wait<0>();
        __syncwarp();
        const uint32_t st = tile0 % kWideStages;
        if (tile0 >= kWideStages) wait(s_free[st], (tile0 / kWideStages - 1) & 1u);
        if (dead) break;
        const uint32_t src = raw + get * kRaw;
        uint8_t *dst = ring + st * kStage + (val ? kHalf : 0) + half * 2048 + r8 * 128 + (ch >> 1) * 1024;
        get = get + 1 == kAhead ? 0 : get + 1;
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          uint32_t w[4];
          read_words<16>(src + (8 * y + r8) * 64 + ((ch ^ ((r8 >> 1) & 3)) << 4), w);
          const uint32_t two = widen(read_half(src + 32 * 64 + (8 * y + r8) * 8 + ch * 2));
#pragma unroll
          for (int j = 0; j < 4; ++j) {  // (a word's 8 values have one scale; a write's 8 lanes are 8 rows: no bank twice)
            uint4 f;
            widen8(w[j], f.x, f.y, f.z, f.w);
            const uint32_t scale = __byte_perm(two, 0u, j < 2 ? 0x1010 : 0x3232);
            f = make_uint4(mul2(f.x, scale), mul2(f.y, scale), mul2(f.z, scale), mul2(f.w, scale));
            *reinterpret_cast<uint4 *>(dst + y * 2048 + ((((ch & 1) * 4 + j) ^ r8) << 4)) = f;
          }
        }
        fence_async();
        __syncwarp();
        if (lane == 0) bar_arrive(smem_at(&s_full[st]));
        ++tile0;
        --ahead;
      }
      copies_wait<0>();
    } else if (!CODES && warp == kSoft) {
      // ================= producer =================
      const int bs_shift = __ffs(kv.block_size) - 1, box = P.box, box_row = (lane >> 1) * box;
      if (a.stall == SV_STALL_ATTENTION) wait(s_free[0], 0);  // failure-path test: a wait that nothing ends
      while (next_piece<Wide>(P, at, p)) {
        const int32_t *bt = kv.block_table + (size_t)at.b * kv.max_blocks;
        const int last = (p.ke - 1) >> bs_shift;
        auto load_id = [&](int blk) { return blk <= last ? bt[blk] : -1; };
        int wbase = max(p.kt0 * Wide::TK, p.lo) >> bs_shift;
        int cur = load_id(wbase + lane), nxt = load_id(wbase + 32 + lane);
        for (int kt = p.kt0; kt < p.kt1; ++kt, ++tile0) {
          const uint32_t st = tile0 % kWideStages;
          const int tok = kt * Wide::TK + box_row, first = max(kt * Wide::TK, p.lo) >> bs_shift;
          while (first >= wbase + 32) {  // uniform
            wbase += 32;
            cur = nxt;
            nxt = load_id(wbase + 32 + lane);
          }
          const bool want = box_row < Wide::TK && tok < p.ke && tok + box > p.lo;
          const int src = want ? (tok >> bs_shift) - wbase : 0;
          const int id0 = __shfl_sync(0xffffffffu, cur, src & 31), id1 = __shfl_sync(0xffffffffu, nxt, src & 31);
          const int id = src < 32 ? id0 : id1;
          const bool bad = want && (id < 0 || id >= kv.num_blocks), go = want && !bad;
          if (bad) record(a.status, SV_ERR_BAD_BLOCK_ID);
          if (tile0 >= kWideStages) wait(s_free[st], (tile0 / kWideStages - 1) & 1u);
          if (dead) break;  // nothing more is issued
          const uint32_t bar = smem_at(&s_full[st]);
          const int boxes = __popc(__ballot_sync(0xffffffffu, go));
          if (lane == 0) bar_expect(bar, boxes * box * Wide::ROWB);
          __syncwarp();
          if (go) {
            const int y = ((id * kv.num_kv_heads + p.kvh) << bs_shift) + (tok & (kv.block_size - 1));
            load_box<Wide::ROWB>(smem_at(ring) + st * kStage + (lane & 1) * kHalf + box_row * Wide::ROWB,
                                 (lane & 1) ? &map_v : &map_k, y, bar);
          }
          __syncwarp();
        }
        if (dead) break;
      }
    } else if (warp == kSoft + 1 || warp == kSoft + 2) {
      // ================= issuers =================
      const int blk = warp - kSoft - 1;
      const uint32_t at_s = tmem + blk * 128, at_o = tmem + kColO + blk * 128, at_q = smem_at(qs) + (ONE ? 0 : blk * kQBytes);
      uint32_t cq = 0, cs = 0, cp = 0;  // pieces, scores and weights of the block so far
      auto issue_s = [&](uint32_t x) {
        fence_after();
        const uint32_t buf = cs++ & 1u, k = smem_at(ring) + x % kWideStages * kStage;
        if (elected()) {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            const uint32_t off = (kk >> 2) * 1024 + (kk & 3) * 32;
            mma_ss(at_s + buf * 64, operand(at_q + off, 16, 2048), operand(k + off, 16, 2048), kIdescS<CODES>, kk > 0);
          }
          commit(smem_at(&s_s[blk][buf]));
        }
        __syncwarp();
      };
      auto issue_pv = [&](uint32_t x) {  // when P is there
        const uint32_t buf = cp & 1u, v = smem_at(ring) + x % kWideStages * kStage + kHalf;
        wait(s_p[blk][buf], (cp++ >> 1) & 1u);
        if (dead) return;
        fence_after();
        if (elected()) {
#pragma unroll
          for (int kk = 0; kk < kTile / 16; ++kk)
            mma_ts(at_o, at_s + buf * 64 + kk * 8, operand(v + kk * 4096, 1024, 2048), kIdescV<CODES>, 1);
          commit(smem_at(&s_o[blk][buf]));
          commit(smem_at(&s_free[x % kWideStages]));
        }
        __syncwarp();
      };
      auto landed = [&](uint32_t x) { wait(s_full[x % kWideStages], (x / kWideStages) & 1u); };
      while (!dead && advance()) {
        const int n = p.kt1 - p.kt0;
        auto pass = [&](int t) {  // the other block's tile
          landed(tile0 + t);
          if (!dead && lane == 0) bar_arrive(smem_at(&s_free[(tile0 + t) % kWideStages]));
        };
        const bool work = active(blk);
        if (ONE || work) wait(s_q[ONE ? 0 : blk], cq++ & 1u);
        if constexpr (ONE) {  // each sees every tile land, in turn
          if (!work && !dead && lane == 0) bar_arrive(smem_at(&s_seen));
          if (blk == 1) pass(0);
          for (int t = blk - 2; t < n && !dead; t += 2) {
            if (t >= 0 && t + 1 < n) pass(t + 1);
            if (t + 2 < n) {
              landed(tile0 + t + 2);
              if (dead) break;
              issue_s(tile0 + t + 2);
            }
            if (t >= 0) issue_pv(tile0 + t);
          }
        } else if (work) {
          for (int t = -1; t < n && !dead; ++t) {
            if (t + 1 < n) {
              landed(tile0 + t + 1);
              if (dead) break;
              issue_s(tile0 + t + 1);
            }
            if (t >= 0) issue_pv(tile0 + t);
          }
        } else {
          for (int t = 0; t < n && !dead; ++t) pass(t);
        }
        tile0 += n;
      }
      // every product issued finishes before tensor memory is released
      if (elected()) commit(smem_at(&s_done));
      __syncwarp();
      if (!__all_sync(0xffffffffu, mbar_wait_bounded(smem_at(&s_done), 0, kDrainBudgetNs))) dead = true;
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs<CODES>));
    // ================= softmax: one row per thread =================
    const int blk = warp >> 2, row = (warp & 3) * 32 + lane;  // row of the block
    const uint32_t lane_at = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t to = lane_at + kColO + blk * 128;
    // what scores are multiplied with (codes: times the keys' pool scale, and of each row's power of two, piece by piece)
    const float sl2_all = CODES ? a.scale_log2 * kv.k_scale : a.scale_log2, cap_in_all = CODES ? P.cap_in * kv.k_scale : P.cap_in;
    const float cap = P.s.cap;
    const bool biased = P.s.slopes != nullptr;
    const bool bounded = !CODES && cap > 0.f && cap <= kBoundedCap && !biased;  // (fp16 weights reach less far)
    const bool plain = cap == 0.f && !biased && sl2_all >= 0.f;
    const int window = P.s.window;
    auto together = [&] { asm volatile("bar.sync 1, 256;" ::: "memory"); };  // both blocks
    auto of_tile = [&](bool two) {                                            // the threads at a tile
      if (two) asm volatile("bar.sync 2, 256;" ::: "memory");
      else if (!ONE || blk == 0) asm volatile("bar.sync 2, 128;" ::: "memory");
      else asm volatile("bar.sync 3, 128;" ::: "memory");
    };
    // ... and whether any of them has one. (The barrier itself carries the vote: a flag in shared memory could be set for the
    // next tile by a warp that is ahead before a slow one has read it, and the barriers would no longer pair up.)
    auto any_of_tile = [&](bool two, bool one) {
      uint32_t any;
      auto vote = [&](auto id, auto threads) {
        asm volatile("{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.or.pred q, %2, %3, p;\n selp.u32 %0, 1, 0, q;\n}\n"
                     : "=r"(any)
                     : "r"((uint32_t)one), "n"(decltype(id)::value), "n"(decltype(threads)::value)
                     : "memory");
      };
      using std::integral_constant;
      if (two) vote(integral_constant<int, 2>(), integral_constant<int, 256>());
      else if (!ONE || blk == 0) vote(integral_constant<int, 2>(), integral_constant<int, 128>());
      else vote(integral_constant<int, 3>(), integral_constant<int, 128>());
      return any != 0u;
    };
    bool first_piece = true;
    uint32_t cs = 0;  // tiles of the block so far: S in buffer cs & 1, the same buffer's s_o when its P V is done
    auto zero_o = [&] {
      uint32_t z[32];
#pragma unroll
      for (int k = 0; k < 32; ++k) z[k] = 0u;
#pragma unroll
      for (int k = 0; k < 4; ++k) tmem_put(to + k * 32, z);
      tmem_put_wait();
    };
    // A piece's Q into shared memory: this row, or half of it where both blocks have it
    constexpr int kParts = ONE ? 8 : 16;
    uint4 part[kParts];
    float down = 1.f;  // codes: the power of two that a row's Q has been divided by
    auto get_q = [&](const Place &pl, const Piece &pc) {
      const int r = pc.rb * Wide::RB + (ONE ? 0 : blk * kBlock) + row, i = r / P.G;
      const bool live = r < P.G * pl.s.n;
      const uint4 *src = reinterpret_cast<const uint4 *>(
          reinterpret_cast<const __nv_bfloat16 *>(a.q) +
          (live ? ((size_t)(pl.s.row0 + i) * a.num_q_heads + pc.kvh * P.G + (r - i * P.G)) * 128 : 0));
#pragma unroll
      for (int c = 0; c < kParts; ++c) part[c] = live ? src[(ONE ? 8 * blk : 0) + c] : make_uint4(0, 0, 0, 0);
      if constexpr (CODES) {  // fp16 next to a power of two that brings the row's largest value to 2^14 .. 2^15
        uint32_t most = 0u;  // the largest magnitude's bits, in each half
        auto look = [&](const uint4 &x) {
          most = __vmaxu2(most, __vmaxu2(__vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu), __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu)));
        };
#pragma unroll
        for (int c = 0; c < kParts; ++c) look(part[c]);
        if constexpr (ONE)
          for (int c = 0; c < 8; ++c) look(live ? src[8 * (blk ^ 1) + c] : make_uint4(0, 0, 0, 0));
        const int e = max(most & 0xffffu, most >> 16) >> 7, field = min(268 - e, 253);  // (as in attn_e2m1.cuh)
        const float up = __int_as_float(field << 23);
        down = __int_as_float((254 - field) << 23);
        auto half2_of = [&](uint32_t x) { return pack2<true>(__uint_as_float(x << 16) * up, __uint_as_float(x & 0xffff0000u) * up); };
#pragma unroll
        for (int c = 0; c < kParts; ++c) part[c] = make_uint4(half2_of(part[c].x), half2_of(part[c].y), half2_of(part[c].z), half2_of(part[c].w));
      }
    };
    auto put_q = [&] {
      uint8_t *dst = qs + (ONE ? 0 : blk * kQBytes);
#pragma unroll
      for (int c = 0; c < kParts; ++c) *reinterpret_cast<uint4 *>(dst + chunk_at(row, (ONE ? 8 * blk : 0) + c)) = part[c];
      fence_async();
      __syncwarp();
      if (lane == 0) bar_arrive(smem_at(&s_q[ONE ? 0 : blk]));
    };
    uint32_t without = 0;  // pieces in which this block had no part
    bool has = next_piece<Wide>(P, at, p);
    if (has && (ONE || active(blk))) {
      get_q(at, p);
      put_q();
    }
    while (has) {
      const Seq s = at.s;
      const Piece pc = p;
      const float sl2 = CODES ? finite(sl2_all * down) : sl2_all, cap_in = CODES ? finite(cap_in_all * down) : cap_in_all;
      const bool two = two_blocks(), mine = ONE || blk == 0 || two;  // a and b have rows; this block has
      has = next_piece<Wide>(P, at, p);                          // at and p: the next piece from here on
      const int c = s.c, ke = pc.ke, rl = (ONE ? 0 : blk * kBlock) + row, r = pc.rb * Wide::RB + rl;
      const int n_tiles = pc.kt1 - pc.kt0, t0 = ONE ? blk : 0, tx = ONE ? tid & 127 : tid;
      const bool live = r < P.G * s.n;
      const int i = live ? r / P.G : 0, head = pc.kvh * P.G + (live ? r - i * P.G : 0);
      // ---- this row: position, new keys that it sees, reach (the last place out of its window) ----
      const int where = P.s.positions != nullptr ? P.s.positions[s.row0 + i] : c + i;
      if (where < c) record(a.status, SV_ERR_BAD_LENGTH);
      const int reach = !live ? 1 << 30 : window > 0 ? where - c - window : -(1 << 30);
      const float slope = biased ? P.s.slopes[head] * 1.4426950408889634f : 0.f;
      uint64_t mask = 0ull;
      if (live) {
        mask = a.mask_kind == SV_MASK_TREE ? a.tree_mask[s.row0 + i] : (2ull << i) - 1ull;
        if (s.n < 64) mask &= (1ull << s.n) - 1ull;
        if (window > 0 && where - c >= window)
          for (int j = 0; j < s.n; ++j) {
            const int place = P.s.positions != nullptr ? P.s.positions[s.row0 + j] - c : j;
            if (place <= reach) mask &= ~(1ull << j);
          }
      }
      together();  // both blocks are done with the previous piece's places
      const int origin = P.s.positions != nullptr ? P.s.positions[s.row0] : c;  // the bias counts from here
      if (tid < s.n) s_place[tid] = P.s.positions != nullptr ? P.s.positions[s.row0 + tid] - origin : tid;
      const int warp_top = __reduce_max_sync(0xffffffffu, live ? where : c);
      if (lane == 0) s_top[warp] = warp_top;
      together();
      int row_top = s_top[0];
#pragma unroll
      for (int w = 1; w < kSoft; ++w) row_top = max(row_top, s_top[w]);
      const int all_see = window > 0 ? row_top - window + 1 : 0;  // keys from here to c are visible to every row
      if (!mine) {
        tile0 += n_tiles;
        first_piece = false;
        if (has && active(blk)) {
          get_q(at, p);
          put_q();
        }
        continue;
      }
      const bool warp_live = __any_sync(0xffffffffu, live);
      zero_o();
      fence_before();
      float m = bounded ? 0.f : kNone, l = 0.f;
      for (int t = t0; t < n_tiles; t += ONE ? 2 : 1, ++cs) {
        const int key0 = (pc.kt0 + t) * kTile, base = key0 - c;
        const uint32_t x = tile0 + t, ts = lane_at + blk * 128 + (cs & 1u) * 64;
        wait(s_s[blk][cs & 1u], (cs >> 1) & 1u);
        fence_after();
        // O may be touched once P V of the tile before is done (a barrier a buffer: its phase before that ended two tiles ago)
        auto o_free = [&] {
          if (t > t0) wait(s_o[blk][(cs - 1) & 1u], ((cs - 1) >> 1) & 1u);
          fence_after();
        };
        auto raise = [&](float mx) {  // the running maximum, if this one passes it by far
          // (fp16 weights end soon: what passes is the exact difference, not one to a rounded sum)
          const bool move = CODES ? mx - m > kMoveAt<CODES> : mx > m + kMoveAt<CODES>;
          if (!__any_sync(0xffffffffu, move)) return;
          const float below = mx - kBelow<CODES>, f = move ? ex2(m - below) : 1.f;
          if (move) m = below;
          l *= f;
          uint32_t o[32];
          o_free();
#pragma unroll 1
          for (int k = 0; k < 4; ++k) {
            tmem_get(to + k * 32, o);
            tmem_landed(o);
#pragma unroll
            for (int y = 0; y < 32; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * f);
            tmem_put(to + k * 32, o);
          }
          tmem_put_wait();
        };
        const bool edge = key0 + kTile > min(c, ke) || key0 < all_see;  // the same for the whole CTA
        uint8_t *vs = ring + x % kWideStages * kStage + kHalf;
        bool odd = false;
        if (edge) {
          // Values that no weight of zero may meet: slots past the end or before the first visible key hold
          // anything and become zeros; infinities and NaN among the others are looked for.
          wait(s_full[x % kWideStages], (x / kWideStages) & 1u);  // (landed: this makes the copies visible here)
          for (int y = tx; y < kTile * 16; y += two ? 256 : 128) {
            const int key = y >> 4;
            uint4 *w = reinterpret_cast<uint4 *>(vs + chunk_at(key, y & 15));
            if (key0 + key >= ke || key0 + key < pc.lo) *w = make_uint4(0, 0, 0, 0);
            else if (CODES) odd |= (nonfinite16(w->x) | nonfinite16(w->y) | nonfinite16(w->z) | nonfinite16(w->w)) != 0u;
            else odd |= (nonfinite(w->x) | nonfinite(w->y) | nonfinite(w->z) | nonfinite(w->w)) != 0u;
          }
          fence_async();
          odd = any_of_tile(two, odd);
        }
        if (warp_live || odd) {
          uint32_t w[kTile];
          tmem_get(ts, w);
          float part[4] = {0.f, 0.f, 0.f, 0.f};
          if (bounded && !edge) {
            // no maximum, no bias, every key is seen: 32 keys' weights while the other 32 scores are on their way
            tmem_landed(w);
            tmem_get(ts + 32, w + 32);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              if (h == 1) tmem_landed(w + 32);
#pragma unroll
              for (int k = 32 * h; k < 32 * h + 32; k += 4) {
                float x[4];
#pragma unroll
                for (int y = 0; y < 4; ++y) x[y] = __uint_as_float(w[k + y]);
                cap_four(x, cap_in, cap);
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                  x[y] = ex2(x[y]);
                  part[y] += x[y];
                }
                w[k / 2] = pack2<CODES>(x[0], x[1]);
                w[k / 2 + 1] = pack2<CODES>(x[2], x[3]);
              }
            }
            l += (part[0] + part[1]) + (part[2] + part[3]);
          } else if (plain && !edge) {  // scores as they are, times a factor that keeps their order
            tmem_get(ts + 32, w + 32);
            tmem_landed(w);
            tmem_landed(w + 32);
            float mx = kNone;
#pragma unroll
            for (int k = 0; k < kTile; ++k) mx = fmaxf(mx, __uint_as_float(w[k]));
            raise(mx * sl2);
            float mul = sl2;
            if (CODES && __any_sync(0xffffffffu, !(fabsf(mx * sl2) < 0x1p22f))) {
              // the maximum is a rounded product, and fp16 has no room for what an exact one may have more
              mul = 1.f;
#pragma unroll
              for (int k = 0; k < kTile; ++k) w[k] = __float_as_uint(__uint_as_float(w[k]) * sl2);
            }
#pragma unroll
            for (int k = 0; k < kTile; k += 2) {
              const float x = ex2(fmaf(__uint_as_float(w[k]), mul, -m)), y = ex2(fmaf(__uint_as_float(w[k + 1]), mul, -m));
              part[k & 2] += x;
              part[(k & 2) + 1] += y;
              w[k / 2] = pack2<CODES>(x, y);
            }
            l += (part[0] + part[1]) + (part[2] + part[3]);
          } else {
            tmem_get(ts + 32, w + 32);
            tmem_landed(w);
            tmem_landed(w + 32);
            uint32_t seen[kTile / 32];  // at an edge: the row's view of the tile's keys as bits
            // ---- scores ----
            if (cap == 0.f) {
#pragma unroll
              for (int k = 0; k < kTile; ++k) w[k] = __float_as_uint(__uint_as_float(w[k]) * sl2);
            } else if (!edge) {
#pragma unroll
              for (int k = 0; k < kTile; k += 4) {
                float x[4];
#pragma unroll
                for (int y = 0; y < 4; ++y) x[y] = __uint_as_float(w[k + y]);
                cap_four(x, cap_in, cap);
#pragma unroll
                for (int y = 0; y < 4; ++y) w[k + y] = __float_as_uint(x[y]);
              }
            } else {  // a key that the row does not see may be a NaN: each by itself
#pragma unroll
              for (int k = 0; k < kTile; ++k)
                w[k] = __float_as_uint(-2.f * cap * rcp(1.f + ex2(__uint_as_float(w[k]) * cap_in)));
            }
            if (biased) {
              if (!edge) {
                const float f0 = (float)(key0 - origin);
#pragma unroll
                for (int k = 0; k < kTile; ++k)
                  w[k] = __float_as_uint(fmaf(slope, f0 + (float)k, __uint_as_float(w[k])));
              } else {
#pragma unroll
                for (int k = 0; k < kTile; ++k) {
                  const int j = base + k;
                  const float place = (float)(j >= 0 && j < s.n ? s_place[j] : c + j - origin);
                  w[k] = __float_as_uint(fmaf(slope, place, __uint_as_float(w[k])));
                }
              }
            }
            if (edge) {
#pragma unroll
              for (int q = 0; q < kTile / 32; ++q) {
                const int b0 = base + 32 * q, first = reach + 1 - b0;
                const uint32_t old = b0 >= 0 ? 0u : b0 <= -32 ? ~0u : (1u << -b0) - 1u;
                const uint32_t near = first <= 0 ? ~0u : first >= 32 ? 0u : ~0u << first;
                const uint32_t fresh = b0 >= 0 ? (b0 < 64 ? (uint32_t)(mask >> b0) : 0u) : (b0 > -32 ? (uint32_t)mask << -b0 : 0u);
                seen[q] = (old & near) | fresh;
#pragma unroll
                for (int k = 0; k < 32; ++k)
                  if (!((seen[q] >> k) & 1u)) w[q * 32 + k] = 0xff800000u;  // -inf
              }
            }
            // ---- the running maximum ----
            if (!bounded) {
              float mx = kNone;
#pragma unroll
              for (int k = 0; k < kTile; ++k) mx = fmaxf(mx, __uint_as_float(w[k]));
              raise(mx);
            }
            // ---- P ----
#pragma unroll
            for (int k = 0; k < kTile; ++k) {
              const float e = ex2(__uint_as_float(w[k]) - m);
              part[k & 3] += e;
              w[k] = __float_as_uint(e);
            }
            l += (part[0] + part[1]) + (part[2] + part[3]);
            if (odd) {
              // infinities and NaN, for the rows that see their keys, whatever the weight (one that is zero in fp32 is not
              // zero); then out of the tile
              o_free();
#pragma unroll 1
              for (int k = 0; k < 4; ++k) {
                uint32_t o[32];
                tmem_get(to + k * 32, o);
                tmem_landed(o);
#pragma unroll 1
                for (int key = 0; key < kTile; ++key) {
                  if (!(((key < 32 ? seen[0] : seen[1]) >> (key & 31)) & 1u)) continue;
#pragma unroll
                  for (int y = 0; y < 4; ++y) {
                    const uint4 u = *reinterpret_cast<const uint4 *>(vs + chunk_at(key, k * 4 + y));
                    const uint32_t word[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                    for (int z = 0; z < 8; ++z) {
                      const uint32_t v = (word[z >> 1] >> (16 * (z & 1))) & 0xffffu;
                      if (CODES ? (v & 0x7c00u) == 0x7c00u : (v & 0x7f80u) == 0x7f80u)  // (codes: a NaN, in bf16's bits one too)
                        o[y * 8 + z] = __float_as_uint(__uint_as_float(o[y * 8 + z]) + __uint_as_float(v << 16));
                    }
                  }
                }
                tmem_put(to + k * 32, o);
              }
              tmem_put_wait();
            }
#pragma unroll
            for (int k = 0; k < kTile / 2; ++k) w[k] = pack2<CODES>(__uint_as_float(w[2 * k]), __uint_as_float(w[2 * k + 1]));
          }
          tmem_put(ts, w);
          tmem_put_wait();
        }
        if (odd) {
          of_tile(two);  // every row has taken its share
          for (int y = tx; y < kTile * 16; y += two ? 256 : 128) {
            uint32_t *w = reinterpret_cast<uint32_t *>(vs + chunk_at(y >> 4, y & 15));
#pragma unroll
            for (int z = 0; z < 4; ++z) {
              w[z] &= ~(CODES ? nonfinite16(w[z]) : nonfinite(w[z]));
            }
          }
          fence_async();
          of_tile(two);
        }
        fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(smem_at(&s_p[blk][cs & 1u]));  // (a warp may be a tile ahead of its block's slowest)
      }
      tile0 += n_tiles;
      // the piece's last S is done with Q: the next piece's rows take its place
      if (has && (ONE || active(blk))) {
        get_q(at, p);
        if (!ONE) put_q();
      }
      // ---- the piece's rows ----
      if (!ONE || t0 < n_tiles) wait(s_o[blk][(cs - 1) & 1u], ((cs - 1) >> 1) & 1u);
      else wait(s_seen, without++ & 1u);  // (Q's barrier runs one piece ahead of its issuers at most)
      fence_after();
      float f_own = 1.f, f_other = 0.f;  // one block of rows: both warps of a row merge, each 64 of its values
      if constexpr (ONE) {
        float2 other;
        if (blk == 1) s_ml[row] = make_float2(m, l);
        fence_before();
        together();
        if (has) put_q();  // both blocks are done with Q
        if (blk == 0) {
          other = s_ml[row];
          s_ml[row] = make_float2(m, l);
        }
        together();
        if (blk == 1) other = s_ml[row];
        const float top = fmaxf(m, other.x);
        f_own = ex2(m - top);
        f_other = ex2(other.x - top);
        l = l * f_own + other.y * f_other;
        m = top;
        fence_after();
      }
      if (warp_live) {
        const float inv = l == 0.f ? 0.f : (CODES ? kv.v_scale : 1.f) / l;
        const size_t slot = ((size_t)blockIdx.x * 2 + (first_piece ? 0 : 1)) * P.rows_cap + rl;
        if (live && !pc.whole && (!ONE || blk == 0)) P.part_lse[slot] = l == 0.f ? -INFINITY : m + log2f(l);
        auto write = [&](int k, const uint32_t (&o)[32], float f) {  // values 32 k and on, times f
          if (!live) return;
          if (pc.whole) {
            uint4 *dst = reinterpret_cast<uint4 *>(reinterpret_cast<__nv_bfloat16 *>(a.out) +
                                                   ((size_t)(s.row0 + i) * a.num_q_heads + head) * 128 + k * 32);
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              uint32_t q[4];
#pragma unroll
              for (int z = 0; z < 4; ++z)
                q[z] = pack2<false>(__uint_as_float(o[8 * y + 2 * z]) * f, __uint_as_float(o[8 * y + 2 * z + 1]) * f);
              dst[y] = make_uint4(q[0], q[1], q[2], q[3]);
            }
          } else {
            float4 *dst = reinterpret_cast<float4 *>(P.part_o + slot * 128 + k * 32);
#pragma unroll
            for (int y = 0; y < 8; ++y)
              dst[y] = make_float4(__uint_as_float(o[4 * y]) * f, __uint_as_float(o[4 * y + 1]) * f,
                                   __uint_as_float(o[4 * y + 2]) * f, __uint_as_float(o[4 * y + 3]) * f);
          }
        };
#pragma unroll 1
        for (int k = ONE ? 2 * blk : 0, end = ONE ? k + 2 : 4; k < end; ++k) {
          uint32_t o[32];
          tmem_get(to + k * 32, o);
          if constexpr (ONE) {
            uint32_t u[32];
            tmem_get(lane_at + kColO + (blk ^ 1) * 128 + k * 32, u);
            tmem_landed(o);
            tmem_landed(u);
#pragma unroll
            for (int y = 0; y < 32; ++y)
              o[y] = __float_as_uint(__uint_as_float(o[y]) * f_own + __uint_as_float(u[y]) * f_other);
          } else {
            tmem_landed(o);
          }
          write(k, o, inv);
        }
      }
      first_piece = false;
    }
  }
  if (dead && lane == 0) record(a.status, SV_ERR_TIMEOUT);
  fence_before();
  __syncthreads();
  fence_after();
  // after a wait that gave up: the copies in flight land before the CTA's shared memory is released
  if (!CODES && s_dead && warp == kSoft)
    for (uint32_t x = tile0 > kWideStages ? tile0 - kWideStages : 0; x < tile0; ++x)
      mbar_wait_bounded(smem_at(&s_full[x % kWideStages]), (x / kWideStages) & 1u, kDrainBudgetNs);
  if (warp == kSoft + 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
}

template <bool ONE, bool CODES>
cudaError_t launch_wide(const CUtensorMap &mk, const CUtensorMap &mv, const Params &p, cudaStream_t st) {
  auto kernel = attn_scored_wide_kernel<ONE, CODES>;
  static const bool split_fits = [&] {  // the kernel was compiled for the registers that its split shares out
    cudaFuncAttributes fa;
    return cudaFuncGetAttributes(&fa, kernel) == cudaSuccess && fa.numRegs == kWideRegs<CODES>;
  }();
  if (!split_fits) return cudaErrorInvalidConfiguration;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kWideSmem<ONE, CODES>);
  return e != cudaSuccess ? e : launch_pdl(kernel, dim3(p.ctas), dim3(kWideThreads<CODES>), (size_t)kWideSmem<ONE, CODES>, st, mk, mv, p);
}

}  // namespace

bool wide_fits(const ScoredArgs &sa) {
  const KV &kv = sa.a.kv;
  return (kv.fp4 || (!kv.fp8 && kv.elem_bytes == 2)) && kv.head_dim == 128 &&
         sa.a.num_q_heads / kv.num_kv_heads * sa.a.max_q > kWideRows;
}

cudaError_t run_wide(const ScoredArgs &sa, void *workspace, size_t *bytes, cudaStream_t st, bool go) {
  const KV &kv = sa.a.kv;
  Params p;
  const Layout l = plan<Wide>(sa, workspace, bytes, &p);
  if (!go || *bytes == 0) return cudaSuccess;
  CUtensorMap mk = {}, mv = {};  // (codes are read without)
  if (!kv.fp4 && (!make_map<Wide>(&mk, kv.k_pool, kv, p.box) || !make_map<Wide>(&mv, kv.v_pool, kv, p.box))) return cudaErrorInvalidValue;
  // One block of rows for all: 32 x 25 rows a head group of 4 over 2K to 4K tokens 170 -> 131 us with both blocks at work
  const bool one = sa.a.num_q_heads / kv.num_kv_heads * sa.a.max_q <= kBlock;
  const cudaError_t e = kv.fp4 ? (one ? launch_wide<true, true>(mk, mv, p, st) : launch_wide<false, true>(mk, mv, p, st))
                               : (one ? launch_wide<true, false>(mk, mv, p, st) : launch_wide<false, false>(mk, mv, p, st));
  if (e != cudaSuccess) return e;
  return launch_combine<Wide>(p, l, st);
}

}  // namespace scored
}  // namespace sv
