// Attention with modified scores over 4-bit caches (E2M1 codes with a scale for 16 values, e2m1.cuh), with
// warp-level matrix instructions; instantiated per head size in attn_e2m1_d*.cu. The mathematics, the work order (CTAs
// that stay, ranges of tiles, partials and their merge) and what an edge step is are those of attn_scored.cuh.
//
// A code times its block scale has 6 significant bits and lies between 2^-10 and 2688: exact in fp16, so K and V are fp16
// operands without a rounding, and the pool scales join the scores' factor and the outputs' normalisation in fp32.
// Queries become fp16 next to a power of two of their row that brings its largest value to 2^14 .. 2^15: bf16's 8
// bits stay, and what lies 2^-28 below that value is off by 2^-39 of it at most. No query is too large. Weights are rounded to fp16
// (2^-11 of themselves, 2^-32 of the row's largest where that is more), their sum is of the unrounded ones.
//
// A CTA is four warps, and each works by itself until the end of a piece: it takes M x 16 of a tile's keys, for all RB = 8
// NT rows of the unit, through a ring of stages of its own (16 keys' codes and scales: 18 D bytes), filled with 16-byte
// asynchronous copies that run on into the CTA's next piece. Nothing waits for another warp, so no barrier can run out. In
// a step
//   S^T (keys x rows) = K Q^T: a lane's share of a key is a run of D / 4 codes, which one or two reads bring: the order of
//     the values along the contraction is free, and Q's registers follow it;
//   weights as in attn_scored.cuh;
//   O^T (values x rows) += V^T P^T: a lane's share of a key is a run of D / 8 codes. Two keys' words become one of
//     pairs by two shifts and two selects, and O's rows follow the order in which they come.
// A pair of codes becomes an operand's word by one conversion and one product with its scale. The keys' and values' places in
// a stage are such that neither kind of read meets a bank twice.
//
// Bound: the issue of instructions, at the rate that few warps of long chains reach. 16 keys of 128 values are 64 conversions and as
// many products with scales whatever the rows, 48 matrix instructions and some 72 of softmax for 24 rows, 75 for copies and
// their addresses: about 500 with a piece's share of its set-up and merge. What a warp waits for is latency more than slots:
// an issue slot takes an instruction 40% of the time for 24 rows (two warps a scheduler at 244 registers) and 59% for 8 rows (four warps),
// fixed latencies first, then instruction fetch and the matrix pipe. Times, 8 KV heads of 128:
//   32 sequences of 0.5K to 4K tokens, 24 rows a KV head: 47 us (1.8 TB/s of the cache; 885 on CUDA cores);
//   4 sequences of 32K tokens, 8 rows: 48 us (3.1 TB/s); 128 of 16 to 8192 tokens, 12 to 36 rows, capped: 158 us.
// (Looking at a block's number as soon as it is asked for cost 5% of each.)
// Two steps' worth of keys (M = 2) give the chains something to hide behind; see pick4 for both. Two warps to a step, half of the
// values each, took 72 us for 24 rows, 75 for 8 and 108 for 40 (121 here, two blocks of 24): the second warp costs scores, copies and
// weights what it saves in products.
//
// More than 48 rows over heads of 128 values go to attn_scored_wide.cu.
#pragma once

#include "attn_scored.cuh"
#include "e2m1.cuh"

namespace sv {
namespace scored {

template <int D_, int NT_, int M_, int CTAS_, int STAGES_>
struct Cfg4 {
  static constexpr int D = D_, NT = NT_, RB = NT_ * 8, kCtasPerSm = CTAS_, kStages = STAGES_;
  static constexpr int M = M_, kKeys = 16 * M;  // keys of a step
  static constexpr int kWarps = 4, kThreads = 128, TK = kWarps * kKeys;
  // Positions of a unit's lead-in. (us with half, with these and with twice as many, the cases of pick4: heads of 128, 24 rows 45.3,
  // 43.4, 44.4; 32 rows 55.4, 52.8, 56.4; 40 rows of 600 tokens 121, 120, 119. Heads of 256, 24 rows 61.3, 59.3, 64.2; heads
  // of 64 67.5, 63.0, 59.5.)
  static constexpr int kAlpha = M == 1 ? 4 : 2;
  static constexpr int KT = D / 16;
  static constexpr int kCodes = 8 * D * M, kScales = D * M;  // bytes of a step's keys (or values): codes, block scales
  static constexpr int kStage = 2 * (kCodes + kScales);
  static constexpr int kRing = kWarps * kStages * kStage;
  static constexpr int kTiles = KT < 8 ? KT : 8;     // 16-value tiles of O that are merged at a time
  static constexpr int kPad = kTiles * 16 + 4;       // floats of a row in the merge buffer
  static constexpr int kMerge = kWarps * 8 * kPad * 4;
  static constexpr bool kQs = NT * KT > 16;  // Q in shared memory: registers are better spent on two chains of products
  static constexpr int kSmem = kRing + kMerge + (kQs ? NT * KT * 256 : 0);
  static_assert(kCtasPerSm * (kSmem + 3840) <= 227 * 1024, "shared memory of an SM");
};

// A piece and its sequence. Each warp keeps its place and its turns in shared memory: registers are short, and a piece is long.
struct Turn {
  Piece p;
  Seq s;
  int b;
};

template <class C>
__global__ void __launch_bounds__(C::kThreads, C::kCtasPerSm) attn_e2m1_kernel(const Params P) {
  grid_dependency_wait();  // the earlier kernel on the stream is complete and visible
  grid_dependents_launch();
  constexpr int D = C::D, NT = C::NT, TK = C::TK, RB = C::RB, KT = C::KT, ST = C::kStages, M = C::M, kKeys = C::kKeys;
  constexpr int kThreads = C::kThreads, kWarps = C::kWarps;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ uint64_t s_mask[RB];         // new keys that a row sees
  __shared__ int s_reach[RB], s_row[RB];  // last place out of the window, and row of the sequence (-1: padding)
  __shared__ float s_slope[RB];
  __shared__ int s_place[64];  // position of a new row minus the first one's
  __shared__ float s_m[kWarps][RB], s_l[kWarps][RB];
  __shared__ float s_in[RB];  // what a row's products are multiplied with
  __shared__ Place s_at[kWarps];
  __shared__ Turn s_turn[kWarps][2];  // the piece at hand and the next one
  __shared__ int s_patch;     // a key of the piece's edge steps has a NaN among its values
  __shared__ int s_scan[kWarps], s_first_b, s_first_base, s_top[kWarps];

  const AttnArgs &a = P.s.a;
  const KV &kv = a.kv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const int B = kv.batch;

  // ---- this CTA's range [pos, end) of the launch's W positions ----
  if (tid == 0) s_first_b = s_first_base = 0;
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
  {
    int v = work_of(tid, true), W, incl = scan(v, &W), run = 0;  // the first kThreads sequences: most batches whole
    if (B > kThreads) {
      int more = 0, rest;
      for (int b = tid + kThreads; b < B; b += kThreads) more += work_of(b, true);
      run = W;
      scan(more, &rest);
      W += rest;
    }
    const int pos = range_start(blockIdx.x, W, P.ctas);
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
      if (v > 0 && excl <= pos && pos < incl) {
        s_first_b = b;
        s_first_base = excl;
      }
      if (blockIdx.x != 0 && b0 > 0 && run > pos) break;  // uniform
    }
    if (blockIdx.x == 0 && tid == 0) P.prefix[B] = W;
    __syncthreads();
    Place at;
    bool bad;
    at.b = s_first_b;
    at.base = s_first_base;
    at.pos = pos;
    at.end = range_start(blockIdx.x + 1, W, P.ctas);
    at.s = load_seq(P, at.b, TK, RB, &bad);
    if (lane == 0) s_at[warp] = at;
    __syncwarp();
  }

  // ---- the ring: this warp's stages, and its way ahead of what is being used ----
  const uint32_t ring = smem_at(smem) + warp * ST * C::kStage;
  const int bs = kv.block_size, bs_shift = __ffs(bs) - 1;
  // What a lane copies of a stage: kPer times 16 bytes of the keys' codes and as many of the values'; then 16 bytes of scales.
  // Key r of the step stands in row r; of each 16 value rows row p holds key vkey(p), so that the four keys of one read
  // (p = 4 j + t) are 2 t + (j & 1) + 8 (j >> 1), as a B operand has them.
  constexpr int kChunks = D / 32, kPer = M * D / 64;  // 16-byte chunks of a row; of a stage to a lane
  auto vkey = [](int p) { return (p & 16) + 2 * (p & 3) + ((p >> 2) & 1) + 8 * ((p >> 3) & 1); };
  // (chunk c of row r stands in place c ^ these)
  auto k_turn = [](int r) { return D == 256 ? 4 * (r & 1) : 0; };
  auto v_turn = [](int p) { return D == 256 ? 2 * (p & 3) : D == 128 ? 2 * ((p >> 1) & 1) : 0; };
  // where the warp's copies are: the piece that they belong to, its tiles left, and the next one's first key
  int ahead_left = 0, ahead_key = 0, id = 0;
  uint32_t ahead_turn = 0;
  // Lane 2 M k + j: the block with the j-th 8 of the next tile's keys, if there are some to be read. (Asked for a tile before
  // the number is looked at: its way here would stand in every step.)
  auto load_ids = [&] {
    const Turn &y = s_turn[warp][ahead_turn];
    const int key = ahead_key + 8 * (lane & (2 * M - 1));
    if (key < y.p.ke && key + 8 > y.p.lo) id = kv.block_table[(size_t)y.b * kv.max_blocks + (key >> bs_shift)];
  };
  auto bring = [&](uint32_t stage) {
    const Turn &y8 = s_turn[warp][ahead_turn];
    const int key0 = ahead_key, ke = y8.p.ke, lo = y8.p.lo;
    const int mine8 = lane & (2 * M - 1), key8 = key0 + 8 * mine8;  // this lane's 8 keys
    const bool want = key8 < ke && key8 + 8 > lo, known = (uint32_t)id < (uint32_t)kv.num_blocks;
    if (want && !known) record(a.status, SV_ERR_BAD_BLOCK_ID);
    // the pool's row (32 bits: the host sees to it) of the first, less its place in the step
    const uint32_t mine = ((uint32_t)((known ? id : 0) * kv.num_kv_heads + y8.p.kvh) << bs_shift) + (key8 & (bs - 1)) - 8 * mine8;
    const uint32_t have = __ballot_sync(0xffffffffu, want && known);
    const bool all = have == 0xffffffffu && key0 >= lo && key0 + kKeys <= ke;  // every key is there
#pragma unroll
    for (int y = 0; y < kPer; ++y) {
      const int q = lane + 32 * y, r = q / kChunks, c = q % kChunks, rv = vkey(r), i8 = r >> 3;
      const uint32_t row = __shfl_sync(0xffffffffu, mine, i8);
      const uint32_t kd = stage + r * (D / 2) + ((c ^ k_turn(r)) << 4), vd = stage + C::kCodes + r * (D / 2) + ((c ^ v_turn(r)) << 4);
      const uint8_t *ks = (const uint8_t *)kv.k_pool + (uint64_t)(row + r) * (D / 2) + c * 16, *vs = (const uint8_t *)kv.v_pool + (uint64_t)(row + rv) * (D / 2) + c * 16;
      if (__builtin_expect(all, 1)) {
        copy_all(kd, ks);
        copy_all(vd, vs);
      } else {
        const bool there = (have >> i8) & 1u;
        const int kk = key0 + r, vk = key0 + rv;
        copy_some(kd, ks, there && kk < ke && kk >= lo ? 16 : 0);
        copy_some(vd, vs, there && vk < ke && vk >= lo ? 16 : 0);
      }
    }
#pragma unroll
    for (int y = 0; y < (M * D / 16 + 15) / 16; ++y) {  // scales: lanes 0 .. 15 the keys', the others the values'
      const int l = (lane & 15) + 16 * y, r = l * (256 / D), i8 = (r >> 3) & (2 * M - 1);
      const uint32_t row = __shfl_sync(0xffffffffu, mine, i8);
      const bool there = (have >> i8) & 1u;
      // those of keys past the end are zeros: what they scale is of no one
      if (l < M * D / 16)
        copy_some(stage + 2 * C::kCodes + (lane >> 4) * C::kScales + l * 16, (lane < 16 ? kv.k_bs : kv.v_bs) + (uint64_t)(row + r) * (D / 16),
                  all ? 16 : there ? max(0, min(16, (ke - key0 - r) * (D / 16))) : 0);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };

  // ---- constants of the launch ----
  float *merge = reinterpret_cast<float *>(smem + C::kRing);  // [warp][8][kPad]
  const uint32_t q_at = smem_at(smem) + C::kRing + C::kMerge + lane * 8;  // Q's operands, [n tile][16 values][lane]
  const float cap = P.s.cap;
  const bool fast_cap = cap <= kFastCap * 1.4426950408889634f;
  const int window = P.s.window;
  const bool biased = P.s.slopes != nullptr;
  // what a product is multiplied with, less the row's own factor
  const float factor = (cap > 0.f && fast_cap ? P.cap_in : a.scale_log2) * kv.k_scale;

  bool first_piece = true;
  int filled = 0;             // tiles on their way or there
  uint32_t get = 0, put = 0;  // stages
  auto next = [&](Turn &turn) {
    Place at = s_at[warp];
    Turn x = {};
    __syncwarp();
    const bool has = next_piece<C>(P, at, x.p);
    x.s = at.s;
    x.b = at.b;
    if (lane == 0) {
      s_at[warp] = at;
      turn = x;
    }
    __syncwarp();
    return has;
  };
  bool has = next(s_turn[warp][0]), ahead_is_next = true;  // the copies have gone on (or go first) to the next piece
  uint32_t turns = 0;
  auto start_copies = [&](const Turn &y, uint32_t turn) {
    ahead_left = y.p.kt1 - y.p.kt0;
    ahead_key = y.p.kt0 * TK + warp * kKeys;
    ahead_turn = turn & 1u;
    load_ids();
  };
  if (has) start_copies(s_turn[warp][0], 0);
  while (has) {
    const Turn &now = s_turn[warp][turns & 1u], &then = s_turn[warp][(turns + 1) & 1u];
    ++turns;
    const Piece &p = now.p;
    const Seq &s = now.s;
    const int &b = now.b;
    has = next(s_turn[warp][turns & 1u]);
    if (ahead_is_next && ahead_left == 0 && has) start_copies(then, turns);  // the copies had come to the end of what was known
    else ahead_is_next = false;
    const int n_tiles = p.kt1 - p.kt0;
    const int c = s.c, ke = p.ke, lo = p.lo, kvh = p.kvh, rb = p.rb;
    auto top_up = [&] {
      while (filled < ST && ahead_left > 0) {
        bring(ring + put * C::kStage);
        put = put + 1 == ST ? 0 : put + 1;
        ++filled;
        ahead_key += TK;
        if (--ahead_left > 0) {
          load_ids();
        } else if (!ahead_is_next && has) {
          ahead_is_next = true;
          start_copies(then, turns);
        }
      }
    };
    top_up();
    const int rows = min(RB, P.G * s.n - rb * RB);  // live rows of the block

    // ---- rows of the block and the new keys' places (every warp is done with the previous piece's) ----
    int top = c;
    for (int x = tid; x < RB; x += kThreads) {
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
    for (int x = tid; x < s.n; x += kThreads) s_place[x] = P.s.positions != nullptr ? P.s.positions[s.row0 + x] - origin : x;
    top = __reduce_max_sync(0xffffffffu, top);
    if (lane == 0) s_top[warp] = top;
    if (tid == 0) s_patch = 0;

    // ---- Q: fp16, each row next to a power of two; its operands in registers, or in shared memory for all warps ----
    uint32_t q[C::kQs ? 1 : NT][KT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      uint32_t(&w)[KT][2] = q[C::kQs ? 0 : nt];
      if (C::kQs && nt % kWarps != warp) continue;
      const int rl = nt * 8 + g, r = rb * RB + rl, i = r / P.G;
      const bool live = rl < rows;
      const uint2 *src = reinterpret_cast<const uint2 *>(a.q) +
                         (live ? ((size_t)(s.row0 + i) * a.num_q_heads + kvh * P.G + (r - i * P.G)) * (D / 4) : 0);
      uint32_t most = 0u;  // the largest magnitude's bits
#pragma unroll
      for (int kk = 0; kk < KT; ++kk) {  // four values from a lane's run (256: two runs) of the head
        const uint2 x = live ? src[(D == 256 ? 32 * (kk >> 3) + 8 * t + (kk & 7) : KT * t + kk)] : make_uint2(0, 0);
        w[kk][0] = x.x;
        w[kk][1] = x.y;
        most = max(most, max(max(x.x & 0x7fffu, (x.x >> 16) & 0x7fffu), max(x.y & 0x7fffu, (x.y >> 16) & 0x7fffu)));
      }
      most = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
      most = max(most, __shfl_xor_sync(0xffffffffu, most, 2));
      const int e = most >> 7, field = min(268 - e, 253);  // (infinities and NaN stay what they are, finite values beside them finite)
      const float up = __int_as_float(field << 23), down = __int_as_float((254 - field) << 23);
#pragma unroll
      for (int kk = 0; kk < KT; ++kk)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          w[kk][h] = pack2<true>(__uint_as_float(w[kk][h] << 16) * up, __uint_as_float(w[kk][h] & 0xffff0000u) * up);
      if (t == 0 && (C::kQs || warp == 0)) s_in[rl] = finite(factor * down);
      if constexpr (C::kQs)
#pragma unroll
        for (int kk = 0; kk < KT; ++kk)
          asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(q_at + (nt * KT + kk) * 256), "r"(w[kk][0]), "r"(w[kk][1]) : "memory");
    }
    __syncthreads();
    int row_top = s_top[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) row_top = max(row_top, s_top[w]);
    const int all_see = window > 0 ? row_top - window + 1 : 0;  // keys from here to c are visible to every row

    float in[NT][2];  // of rows 2 t and 2 t + 1 of each n tile
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const float2 x = *reinterpret_cast<const float2 *>(&s_in[nt * 8 + 2 * t]);
      in[nt][0] = x.x;
      in[nt][1] = x.y;
    }
    float o[KT][NT][4], m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = kNone;
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int mt = 0; mt < KT; ++mt) o[mt][nt][0] = o[mt][nt][1] = o[mt][nt][2] = o[mt][nt][3] = 0.f;
    }

    for (int tile = 0; tile < n_tiles; ++tile) {
      __syncwarp();  // every lane is done with the stage that is filled next
      top_up();
      if (filled == ST) copies_wait<ST - 1>();
      else copies_wait<0>();
      __syncwarp();
      const int key0 = (p.kt0 + tile) * TK + warp * kKeys;
      const uint32_t stage = ring + get * C::kStage;
      get = get + 1 == ST ? 0 : get + 1;
      --filled;
      if (__builtin_expect(key0 >= ke || key0 + kKeys <= lo, 0)) continue;  // warp-uniform: nothing to see here
      // ---- S^T = K Q^T ----
      constexpr int kWords = D / 32;  // a lane's words of a key's codes; of a value's half as many
      constexpr int kVw = kWords / 2, kVs = D == 256 ? 2 : 1;
      uint32_t kw[M][2][kWords], ks[M][2][(kWords + 1) / 2];
#pragma unroll
      for (int u = 0; u < M; ++u)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = 16 * u + g + 8 * h;
          const uint32_t row = stage + r * (D / 2), sc = stage + 2 * C::kCodes + r * (D / 16);
          if constexpr (D == 64) {
            read_words<8>(row + t * 8, kw[u][h]);
            ks[u][h][0] = read_byte(sc + t);
          } else if constexpr (D == 128) {
            read_words<16>(row + t * 16, kw[u][h]);
            ks[u][h][0] = read_half(sc + 2 * t);
          } else {
            read_words<16>(row + ((t ^ k_turn(r)) << 4), kw[u][h]);
            read_words<16>(row + (((t + 4) ^ k_turn(r)) << 4), kw[u][h] + 4);
            ks[u][h][0] = read_half(sc + 2 * t);
            ks[u][h][1] = read_half(sc + 8 + 2 * t);
          }
        }
      float sc[M][NT][4];
      {
        constexpr int kSplit = NT * M == 1 ? 2 : 1;  // chains of products
        float part[kSplit][M][NT][4];
#pragma unroll
        for (int y = 0; y < kSplit * M * NT * 4; ++y) (&part[0][0][0][0])[y] = 0.f;
        uint32_t scale[M][2];
#pragma unroll
        for (int w = 0; w < kWords; ++w) {
          uint32_t f[M][2][4];
#pragma unroll
          for (int u = 0; u < M; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              if (w % 2 == 0) {  // two words of 8 codes to a scale
                const uint32_t two = widen(ks[u][h][w >> 2]);
                scale[u][h] = __byte_perm(two, 0u, D > 64 && (w & 2) ? 0x3232 : 0x1010);
              }
              widen8(kw[u][h][w], f[u][h][0], f[u][h][1], f[u][h][2], f[u][h][3]);
#pragma unroll
              for (int y = 0; y < 4; ++y) f[u][h][y] = mul2(f[u][h][y], scale[u][h]);
            }
#pragma unroll
          for (int y = 0; y < 2; ++y)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              uint32_t b[2];
              if constexpr (C::kQs) read_words<8>(q_at + (nt * KT + 2 * w + y) * 256, b);
              else b[0] = q[nt][2 * w + y][0], b[1] = q[nt][2 * w + y][1];
#pragma unroll
              for (int u = 0; u < M; ++u) {
                const uint32_t e[4] = {f[u][0][2 * y], f[u][1][2 * y], f[u][0][2 * y + 1], f[u][1][2 * y + 1]};
                mma<true>(part[y % kSplit][u][nt], e, b[0], b[1]);
              }
            }
        }
#pragma unroll
        for (int u = 0; u < M; ++u)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int y = 0; y < 4; ++y)
              sc[u][nt][y] = (kSplit == 2 ? part[0][u][nt][y] + part[kSplit - 1][u][nt][y] : part[0][u][nt][y]) * in[nt][y & 1];
      }
      // the values' words and scales, on their way during the softmax: keys 2 t, 2 t + 1, 2 t + 8, 2 t + 9
      uint32_t vw[M][4][kVw], vs[M][2][kVs];  // vs: two keys' scales, a byte each
#pragma unroll
      for (int u = 0; u < M; ++u) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int pr = 16 * u + 4 * j + t;
          const uint32_t row = stage + C::kCodes + pr * (D / 2);
          if constexpr (D == 64) read_words<4>(row + g * 4, vw[u][j]);
          else if constexpr (D == 128) read_words<8>(row + (((g >> 1) ^ v_turn(pr)) << 4) + (g & 1) * 8, vw[u][j]);
          else read_words<16>(row + ((g ^ v_turn(pr)) << 4), vw[u][j]);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t at = stage + 2 * C::kCodes + C::kScales + (16 * u + 2 * t + 8 * j) * (D / 16);
          if constexpr (D == 256) {
            const uint32_t x = read_half(at + 2 * g), y = read_half(at + 16 + 2 * g);
            vs[u][j][0] = __byte_perm(x, y, 0x3340);
            vs[u][j][1] = __byte_perm(x, y, 0x3351);
          } else {
            const int gr = D == 64 ? g >> 1 : g;
            vs[u][j][0] = read_byte(at + gr) | read_byte(at + D / 16 + gr) << 8;
          }
        }
      }
      // ---- scores ---- (element e of an n tile: key half e >> 1, row 2 t + (e & 1))
      float *const sv = &sc[0][0][0];
      constexpr int kE = M * NT * 4;
      if (cap > 0.f) {
        if (fast_cap) {
#pragma unroll
          for (int y = 0; y < kE; ++y) sv[y] = -2.f * cap * rcp(1.f + ex2(sv[y]));
        } else {
#pragma unroll
          for (int y = 0; y < kE; ++y) sv[y] = cap * tanhf(sv[y] / cap);
        }
      }
      const bool edge = key0 + kKeys > min(c, ke) || key0 < all_see;  // warp-uniform: some row may not see some key
      if (__builtin_expect(biased, 0)) {
#pragma unroll
        for (int h = 0; h < 2 * M; ++h) {
          const int key = key0 + g + 8 * h, j = key - c;
          const float place = (float)(edge && j >= 0 && j < s.n ? s_place[j] : key - origin);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const float2 sl = *reinterpret_cast<const float2 *>(&s_slope[nt * 8 + 2 * t]);
            float *x = &sc[h >> 1][nt][2 * (h & 1)];
            x[0] = fmaf(sl.x, place, x[0]);
            x[1] = fmaf(sl.y, place, x[1]);
          }
        }
      }
      if (__builtin_expect(edge, 0)) {
        const int base = key0 - c;  // place of the step's first key
        // A row's view of the step's keys as bits: committed keys beyond its reach, and its mask of new ones.
        const uint32_t old = base >= 0 ? 0u : base <= -32 ? ~0u : (1u << -base) - 1u;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int rl = nt * 8 + 2 * t + e, first = s_reach[rl] + 1 - base;
            const uint64_t mask = s_mask[rl];
            const uint32_t near = first <= 0 ? ~0u : first >= 32 ? 0u : ~0u << first;
            const uint32_t fresh = base >= 0 ? (base < 64 ? (uint32_t)(mask >> base) : 0u) : (base > -32 ? (uint32_t)mask << -base : 0u);
            const uint32_t seen = ((old & near) | fresh) >> g;
#pragma unroll
            for (int h = 0; h < 2 * M; ++h)
              if (!((seen >> (8 * h)) & 1u)) sc[h >> 1][nt][2 * (h & 1) + e] = -INFINITY;
          }
        // Values that are NaN must not meet a weight of zero: their scales become zero, and the rows that see their keys
        // get them at the piece's end.
#pragma unroll
        for (int u = 0; u < M; ++u)
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int w = 0; w < kVs; ++w) {
              const uint32_t nan = nan_codes(vs[u][j][w]) & 0xffffu;
              if (nan != 0u) {
                vs[u][j][w] &= ~nan;
                const int key = key0 + 16 * u + 2 * t + 8 * j;
                if (((nan & 0xffu) && key >= lo && key < ke) || ((nan >> 8) && key + 1 >= lo && key + 1 < ke)) s_patch = 1;
              }
            }
      }
      // ---- the running maximum ----
      bool move = false;
#pragma unroll
      for (int u = 0; u < M; ++u)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) move |= sc[u][nt][e] - m[nt][e & 1] > kMoveAt<true>;
      if (__builtin_expect(__any_sync(0xffffffffu, move), 0)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float mx = fmaxf(sc[0][nt][e], sc[0][nt][e + 2]);
#pragma unroll
            for (int u = 1; u < M; ++u) mx = fmaxf(mx, fmaxf(sc[u][nt][e], sc[u][nt][e + 2]));
#pragma unroll
            for (int y = 4; y < 32; y <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, y));
            const float mn = fmaxf(m[nt][e], mx - kBelow<true>);
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
      // ---- P^T ----
      uint32_t pb[M][NT][2];
#pragma unroll
      for (int u = 0; u < M; ++u)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[u][nt][e] = ex2(sc[u][nt][e] - m[nt][e & 1]);
          l[nt][0] += sc[u][nt][0] + sc[u][nt][2];
          l[nt][1] += sc[u][nt][1] + sc[u][nt][3];
          pb[u][nt][0] = turn8x8(pack2<true>(sc[u][nt][0], sc[u][nt][1]));
          pb[u][nt][1] = turn8x8(pack2<true>(sc[u][nt][2], sc[u][nt][3]));
        }
      // ---- O^T += V^T P^T: tile mt has values (D / 8) g + 2 mt and the next one, in rows g and g + 8 ----
#pragma unroll
      for (int w = 0; w < kVw; ++w)
#pragma unroll
        for (int u = 0; u < M; ++u) {
          uint32_t f[2][8];  // pairs of keys; of the even values, of the odd ones
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint32_t x = vw[u][2 * j][w], y = vw[u][2 * j + 1][w], scale = widen(vs[u][j][D == 256 ? w >> 1 : 0]);
            constexpr uint32_t kLow = 0x0f0f0f0fu;
            widen8((x & kLow) | ((y << 4) & ~kLow), f[j][0], f[j][2], f[j][4], f[j][6]);
            widen8(((x >> 4) & kLow) | (y & ~kLow), f[j][1], f[j][3], f[j][5], f[j][7]);
#pragma unroll
            for (int y2 = 0; y2 < 8; ++y2) f[j][y2] = mul2(f[j][y2], scale);
          }
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const uint32_t e[4] = {f[0][2 * y], f[0][2 * y + 1], f[1][2 * y], f[1][2 * y + 1]};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma<true>(o[4 * w + y][nt], e, pb[u][nt][0], pb[u][nt][1]);
          }
        }
    }

    // ---- the warps' results, merged, 8 rows at a time ----
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float sum = l[nt][e];
#pragma unroll
        for (int y = 4; y < 32; y <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, y);
        if (g == 0) {
          s_m[warp][nt * 8 + 2 * t + e] = m[nt][e];
          s_l[warp][nt * 8 + 2 * t + e] = sum;
        }
      }
    const size_t slot = ((size_t)blockIdx.x * 2 + (first_piece ? 0 : 1)) * P.rows_cap;
    constexpr int MT = C::kTiles, kItems = 2 * MT;  // 8 values of a row each
    bool patch = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int m0 = 0; m0 < KT; m0 += MT) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float *dst = merge + (warp * 8 + 2 * t + e) * C::kPad + 2 * g;
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
            *reinterpret_cast<float2 *>(dst + mt * 16) = make_float2(o[m0 + mt][nt][e], o[m0 + mt][nt][e + 2]);
        }
        __syncthreads();
        if (nt == 0 && m0 == 0) {  // every warp's weight in a row, over the rows' total
          patch = s_patch != 0;
          for (int rl = tid; rl < rows; rl += kThreads) {
            float mx = s_m[0][rl], tot = 0.f;
#pragma unroll
            for (int w = 1; w < kWarps; ++w) mx = fmaxf(mx, s_m[w][rl]);  // finite: kNone at the least
#pragma unroll
            for (int w = 0; w < kWarps; ++w) tot += s_l[w][rl] * ex2(s_m[w][rl] - mx);
            const float inv = tot == 0.f ? 0.f : kv.v_scale / tot;
            if (!p.whole) P.part_lse[slot + rl] = tot == 0.f ? -INFINITY : mx + log2f(tot);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) s_l[w][rl] = ex2(s_m[w][rl] - mx) * inv;
          }
          __syncthreads();
        }
        for (int x = tid; x < 8 * kItems; x += kThreads) {
          const int r8 = x / kItems, u = x % kItems, vg = u / (MT / 4), mt0 = u % (MT / 4) * 4, rl = nt * 8 + r8;
          if (rl >= rows) continue;
          const int d = vg * (D / 8) + 2 * (m0 + mt0);
          float v[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] = 0.f;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            const float f = s_l[w][rl];
            const float *src = merge + (w * 8 + r8) * C::kPad + mt0 * 16 + 2 * vg;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 y = *reinterpret_cast<const float2 *>(src + k * 16);
              v[2 * k] = fmaf(f, y.x, v[2 * k]);
              v[2 * k + 1] = fmaf(f, y.y, v[2 * k + 1]);
            }
          }
          if (p.whole) {
            const int i = s_row[rl], head = kvh * P.G + (rb * RB + rl) - i * P.G;
            *reinterpret_cast<uint4 *>(reinterpret_cast<__nv_bfloat16 *>(a.out) + ((size_t)(s.row0 + i) * a.num_q_heads + head) * D + d) =
                make_uint4(pack2<false>(v[0], v[1]), pack2<false>(v[2], v[3]), pack2<false>(v[4], v[5]), pack2<false>(v[6], v[7]));
          } else {
            float4 *dst = reinterpret_cast<float4 *>(P.part_o + (slot + rl) * D + d);
            dst[0] = make_float4(v[0], v[1], v[2], v[3]);
            dst[1] = make_float4(v[4], v[5], v[6], v[7]);
          }
        }
        __syncthreads();
      }
    if (patch) {
      // The NaN that edge steps took out, for the rows that see their keys, whatever the weight: looked for in the pool again
      // and added to what has been written.
#pragma unroll 1
      for (int x = tid; x < rows * (D / 16); x += kThreads) {
        const int rl = x / (D / 16), gr = x % (D / 16);
        bool nan = false;
#pragma unroll 1
        for (int key = max(p.kt0 * TK, lo); key < ke && !nan; ++key) {
          const int key0 = key & ~(kKeys - 1), place = key - c;
          if (!(key0 + kKeys > min(c, ke) || key0 < all_see)) {  // on to the next edge step
            key = (min(c, ke) & ~(kKeys - 1)) - 1;
            continue;
          }
          if (!(place < 0 ? place > s_reach[rl] : (s_mask[rl] >> place) & 1ull)) continue;
          const int id = kv.block_table[(size_t)b * kv.max_blocks + (key >> bs_shift)];
          if (id < 0 || id >= kv.num_blocks) continue;
          nan = (kv.v_bs[((((size_t)id * kv.num_kv_heads + kvh) << bs_shift) + (key & (bs - 1))) * (D / 16) + gr] & 127u) == 127u;
        }
        if (!nan) continue;
        const int i = s_row[rl], head = kvh * P.G + (rb * RB + rl) - i * P.G;
        for (int d = gr * 16; d < gr * 16 + 16; ++d)
          if (p.whole)
            reinterpret_cast<uint16_t *>(a.out)[((size_t)(s.row0 + i) * a.num_q_heads + head) * D + d] = 0x7fffu;
          else
            P.part_o[(slot + rl) * D + d] = __int_as_float(0x7fffffff);
      }
    }
    __syncthreads();  // the rows' places are done with
    first_piece = false;
  }
}

// Launches (`go`) or sizes one instance.
template <class C>
cudaError_t run4(const ScoredArgs &sa, void *workspace, size_t *bytes, cudaStream_t st, bool go) {
  Params p;
  const Layout l = plan<C>(sa, workspace, bytes, &p);
  if (!go || *bytes == 0) return cudaSuccess;
  cudaError_t e = cudaFuncSetAttribute(attn_e2m1_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  e = launch_pdl(attn_e2m1_kernel<C>, dim3(p.ctas), dim3(C::kThreads), (size_t)C::kSmem, st, p);
  if (e != cudaSuccess) return e;
  return launch_combine<C>(p, l, st);
}

// The smallest block of query rows that holds a unit's, else blocks of the largest.
template <int D>
cudaError_t pick4(const ScoredArgs &sa, void *workspace, size_t *bytes, cudaStream_t st, bool go) {
  // CTAs an SM and stages: what registers and shared memory leave. Times in us: of 4 sequences of 32K tokens ("long"), 32 of 0.5K to
  // 4K, 128 of 512 to 640 ("short"); 16, 8 and 4 KV heads of 64, 128 and 256 values, so that the caches are of one size.
  const int rows = sa.a.num_q_heads / sa.a.kv.num_kv_heads * sa.a.max_q;
  auto on = [&](auto cfg) { return run4<decltype(cfg)>(sa, workspace, bytes, st, go); };
  if constexpr (D == 64) {
    // 8 rows, long: 53; three CTAs with five stages 63; 16 keys a step, eight stages 67
    if (rows <= 8) return on(Cfg4<D, 1, 2, 4, 4>());
    // 16 rows: 45 to 54 from run to run; two CTAs with six stages 49; 16 keys a step, eight stages 49 to 55; in a block of 32 63
    if (rows <= 16) return on(Cfg4<D, 2, 2, 3, 5>());
    // 32 rows: 67; in two blocks of 24 95; 16 keys a step 75. (24 and 40 rows would gain by blocks of 24: 63 and 57, 109 and 98.)
    return on(Cfg4<D, 4, 2, 2, 6>());
  } else if constexpr (D == 128) {
    // 8 rows, long: 48, and 32 sequences 32.5; three CTAs with three stages 53 and 36.6; 16 keys a step, four CTAs with four stages
    // 55 and 33.7. (256 sequences of 100 to 600 tokens: 57, 55 and 55.)
    if (rows <= 8) return on(Cfg4<D, 1, 2, 4, 2>());
    // 16 rows: 39.7; 16 keys a step, eight stages 43.2, three CTAs with five stages 55
    if (rows <= 16) return on(Cfg4<D, 2, 2, 2, 4>());
    // 25 to 32 rows in one block of 16 keys a step: 32 sequences of 2K to 4K tokens with 28 rows 69, in two blocks of 24 rows 93; 64 of
    // 200 to 300 36 and 48. (Blocks of 40 rows spill, took as long for 36 and 40 rows, and batches of 12 to 36 lost a fifth by them.)
    // Else blocks of 24: 24 rows 43.4; 16 keys a step, eight stages 47.5, three CTAs with five stages 53.
    if (rows > 24 && rows <= 32) return on(Cfg4<D, 4, 1, 2, 8>());
    if (!wide_fits(sa)) return on(Cfg4<D, 3, 2, 2, 4>());
    // a cap past the two-instruction tanh stays here; the workspace suits both, and so do the positions
    size_t most = 0;
    run_wide(sa, nullptr, &most, st, false);
    if (go && sa.cap <= kFastCap * 1.4426950408889634f) return run_wide(sa, workspace, bytes, st, go);
    const cudaError_t e = on(Cfg4<D, 3, 2, 2, 4>());
    *bytes = *bytes == 0 || most == 0 ? 0 : std::max(*bytes, most);
    return e;
  } else {
    // 8 rows, long: 49.9, and 128 of 200 to 640 tokens 35.9; three CTAs with two stages 50.9 and 36.6; 32 keys a step, two stages 46.3
    // and 39.0
    if (rows <= 8) return on(Cfg4<D, 1, 1, 2, 4>());
    // 16 rows: 39.3; three stages 38.1; in two blocks of 8 49.1
    return on(Cfg4<D, 2, 1, 2, 4>());
  }
}

}  // namespace scored
}  // namespace sv
