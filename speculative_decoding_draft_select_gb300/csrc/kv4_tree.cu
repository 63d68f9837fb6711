// Attention of many rows (trees) over the 4-bit cache on the fifth-generation
// tensor cores.  The mathematics and the division of the work are those of
// kv4_attention.cu; here a row tile is one or two accumulators of 128 rows
// (MT) and a tile 128 positions, and per tile
//   S = Q K^T   128 x 128 x D, Q and K in shared memory
//   P = 2^(S c - max + 7) in fp16, written over S in tensor memory
//   O += P V    128 x D x 128, P from tensor memory, V in shared memory
// all operands fp16 with fp32 accumulation.  Roles of a CTA:
//   warps 0 .. 4 MT - 1   softmax: a thread owns one row of an accumulator, so
//       maximum and sum need no exchange; it also writes the results.  The
//       first warp of an accumulator issues its matrix instructions: its next
//       step waits for them in any case.
//   the next 4 MT warps   unpack the cache: codes go from memory through
//       registers (one tile ahead, whichever segment it belongs to) to swizzled
//       fp16 slabs; Q likewise.
// 16 warps an SM leave each thread 128 registers: with a warp more for the
// issue (96 registers) the codes read ahead spilled, and a spill waits for
// its load.  The softmax goes over a row 32 columns at a time for the same
// reason (64-node trees, B=128, 32 heads over 8 of 128, contexts 16..2048:
// 323 us with the issuing warp, 281 without, 266 with 32 columns, 259 with K
// read ahead sooner).  Bound by the softmax passes (without them 182 of 266) and by the hand-overs
// between the roles (155 cycles each); the tensor pipe works 23% of the time.
// Unpacking with twice the threads took 286 us, weights in shared memory
// instead of tensor memory 326, no search for a maximum (weights watched for
// their size instead) 267.
// With MT = 2 the exponentials of one accumulator run under the products of
// the other, on one CTA per SM with two stages of K and V; with MT = 1 two
// CTAs share an SM to the same end.
//
// Rescaling.  O is only rescaled when a row's maximum has grown by more than
// 2^8 (weights are held times 2^7, so they stay below fp16's 2^15); the result
// divides by the sum of the same weights, so a maximum that lags is exact.
//
// Ordering.  Every hand-over is an mbarrier with a bounded wait; a wait that
// runs out is counted in SPEC_STAT_WAIT_TIMEOUT, the CTA's roles stop, its
// matrix operations are drained, its tensor memory is freed and it returns
// (results void).  A wait names a phase by its parity, so nobody may be two
// phases behind: K's barriers (which the softmax also waits for, to read the
// tile's present positions) go round four buffers, since K of tile j + 2 may
// be unpacked while tile j is in the softmax; Q's and V's alternate between
// two; freed stages have a barrier each.
//
// With a sliding window and sinks (WIN, see kv4_attention.cu) only the bits of
// what a row sees change.  64-node trees, B=128, contexts 16..8192, window 1024:
// 253 us, as far from the products' floor as over whole contexts: by the number of
// tiles 22 us each (3.3 a tile of a CTA's 6.7 segments, of which the tensor pipe
// works a quarter) and 57 for all segments' beginnings, ends and the merge.  16-node
// trees of 48 rows, D = 64, B=64, window 509: 33 us; where no segment is cut (B=76)
// 2.8 us for each of five tiles and 13 for the launches, Q and the ends.
#include "kv4_attn.cuh"
#include "tcgen05.cuh"

namespace specdec {
namespace {

constexpr int kTT = 128;             // positions of a tile
constexpr int kEnds = 2;             // tiles that a segment's beginning and end cost
constexpr float kHeldExp = 7.0f;     // weights are held times 2^7
constexpr float kLagExp = 8.0f;      // a row's maximum may lag by 2^8

template <int D, int MT>
struct TreeCfg {
  static constexpr int kStages = MT == 2 ? 2 : 1;
  static constexpr int kSoftThreads = 128 * MT;
  static constexpr int kUnpackThreads = 128 * MT;
  static constexpr int kThreads = kSoftThreads + kUnpackThreads;
  static constexpr int kSlabs = D / 64;
  static constexpr int kSlab = kTT * 128;          // bytes: 128 rows of 64 elements
  static constexpr int kOperand = kSlabs * kSlab;  // K, V or one accumulator's Q
  // a warp's 32 rows of 64 bytes of results, 16 bytes of padding each
  static constexpr int kStageRow = 80, kStageWarp = 32 * kStageRow;
  static constexpr size_t kSmem = static_cast<size_t>(kOperand) * (MT + 2 * kStages) + 4 * MT * kStageWarp + 1024;
  // columns: S of each accumulator, then O of each
  static constexpr uint32_t kCols = MT * 256;
};

// Stores 8 fp16 channels, unit `u` of row r, to a slab.
__device__ __forceinline__ void put_unit(uint8_t* slab, int r, int u, const uint32_t* v) {
  *reinterpret_cast<uint4*>(slab + r * 128 + ((u ^ (r & 7)) << 4)) = make_uint4(v[0], v[1], v[2], v[3]);
}

// A warp's wait: all lanes get the same answer, so none is left behind in a
// warp-wide operation when a wait runs out.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, int* abort) {
  return __all_sync(0xffffffffu, tc::bar_wait(bar, parity, abort));
}

__device__ __forceinline__ uint32_t word_of4(const uint4& v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// A group of 32 channels: codes and their (step, lo).
struct Chunk {
  uint4 c;
  uint32_t m;
};

// Which of the nodes [first, first + 128) this thread's node sees, a bit each
// (nodes below 0 are context: set; nodes past the request's: clear).  A lane
// loads the mask bytes of its place in each word for four of the warp's nodes
// at a time, ballots give the words.  All loads come first and none is behind
// a condition of its own (a load that is tested where it was issued is a wait
// each).
template <bool WIN>
__device__ __forceinline__ void node_words(const AttnArgs& a, const Part& p, int node, int first, uint32_t* words) {
  const int lane = threadIdx.x & 31;
  const int n_lo = __shfl_sync(0xffffffffu, node, 0), n_hi = __shfl_sync(0xffffffffu, node, 31);
  const uint8_t* mask = a.mask + static_cast<int64_t>(p.b) * a.N * a.N;
  int nd[4], at[4];
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    nd[w] = first + 32 * w + lane;
    at[w] = min(max(nd[w], 0), p.nodes - 1);
  }
  int depth[4] = {0, 0, 0, 0};
  if (WIN && a.window < p.nodes) {
#pragma unroll
    for (int w = 0; w < 4; ++w) depth[w] = attn_depth(a, p, at[w]);
  }
#pragma unroll 1
  for (int nb = n_lo; nb <= n_hi; nb += 4) {
    uint8_t on[4][4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int n = min(nb + q, n_hi);
      const uint8_t* row = mask + (spec_in(n, a.N, a.stats) ? n : 0) * a.N;
#pragma unroll
      for (int w = 0; w < 4; ++w) on[q][w] = a.mask ? __ldg(row + at[w]) : static_cast<uint8_t>(at[w] <= n);
      if (WIN && a.window < p.nodes) {
        const int dn = attn_depth(a, p, n);
#pragma unroll
        for (int w = 0; w < 4; ++w)
          if (!attn_near_depths(a, p, dn, depth[w])) on[q][w] = 0;
      }
    }
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint32_t bits = __ballot_sync(0xffffffffu, nd[w] < 0 || (nd[w] < p.nodes && on[q][w] != 0));
        if (nb + q == node) words[w] = bits;
      }
  }
}

// A thread's row of S, 32 columns (a word of `see`) at a time: the largest
// element that `see` shows, and the weights 2^(S c - base) as fp16 over S's
// first columns (column i of P holds positions 2 i and 2 i + 1; it never
// reaches columns that are still to be read), with their fp32 sum.  Words that
// every lane sees whole skip the mask.  A word an iteration and none ahead: a
// load from tensor memory takes some 30 cycles, and the code of all roles has
// to stay small, since instruction fetches are what a tile waits for.
__device__ __forceinline__ uint32_t pick(const uint32_t* v, int i) {
  return i < 2 ? (i == 0 ? v[0] : v[1]) : (i == 2 ? v[2] : v[3]);
}
__device__ __forceinline__ float row_max(uint32_t col, const uint32_t* see) {
  uint32_t x[32];
  float m[4] = {neg_inf(), neg_inf(), neg_inf(), neg_inf()};
#pragma unroll 1
  for (int w = 0; w < kTT / 32; ++w) {
    const uint32_t sw = pick(see, w);
    tc::ld32(col + 32 * w, x);
    tc::wait_ld32(x);
    if (__any_sync(0xffffffffu, sw != ~0u)) {
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (!((sw >> i) & 1u)) x[i] = 0xff800000u;
    }
#pragma unroll
    for (int i = 0; i < 32; ++i) m[i & 3] = fmaxf(m[i & 3], __uint_as_float(x[i]));
  }
  return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}
// far: the maximum is so far from zero that the rounding of S c in it would
// show in 2^(S c - base), where S c is not rounded: the weights then start from
// the rounded products too.
constexpr float kFar = 0x1p20f;  // S c is rounded by 2^-4 at most up to here
__device__ __forceinline__ float row_weights(uint32_t col, const uint32_t* see, float c, float base, bool far) {
  uint32_t x[32], y[16];
  const bool any_far = __any_sync(0xffffffffu, far);
  const float before = far ? c : 1.0f;
  if (far) c = 1.0f;
  const float2 c2 = splat(c), nb2 = splat(-base);
  float2 acc[2] = {splat(0.0f), splat(0.0f)};
#pragma unroll 1
  for (int w = 0; w < kTT / 32; ++w) {
    const uint32_t sw = pick(see, w);
    tc::ld32(col + 32 * w, x);
    tc::wait_ld32(x);
    if (any_far) {
#pragma unroll
      for (int i = 0; i < 32; ++i) x[i] = __float_as_uint(__fmul_rn(__uint_as_float(x[i]), before));
    }
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
      const float2 e = exp2_2(fma2(make_float2(__uint_as_float(x[i]), __uint_as_float(x[i + 1])), c2, nb2));
      x[i] = __float_as_uint(e.x);
      x[i + 1] = __float_as_uint(e.y);
    }
    if (__any_sync(0xffffffffu, sw != ~0u)) {
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (!((sw >> i) & 1u)) x[i] = 0;
    }
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
      const float2 e = make_float2(__uint_as_float(x[i]), __uint_as_float(x[i + 1]));
      acc[(i >> 1) & 1] = add2(acc[(i >> 1) & 1], e);
      y[i / 2] = h2_u32(__floats2half2_rn(e.x, e.y));
    }
    tc::st16(col + 16 * w, y);
  }
  const float2 t = add2(acc[0], acc[1]);
  return t.x + t.y;
}

template <int D, int MT, bool WIN>
__global__ void __launch_bounds__(TreeCfg<D, MT>::kThreads, MT == 2 ? 1 : 2) kv4_tree_kernel(const AttnArgs a) {
  pdl_enter();
  using C = TreeCfg<D, MT>;
  constexpr int R = kTreeRows * MT, S = C::kStages, CH = D / 32;  // CH: groups of a head row
  extern __shared__ uint8_t tree_sm[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(tree_sm) + 1023) & ~uintptr_t(1023));
  if (!spec_smem_ok((smem - tree_sm) + C::kSmem - 1024, a.stats)) return;
  uint8_t* sm_q = smem;                       // [MT] operands
  uint8_t* sm_k = sm_q + MT * C::kOperand;    // [S]
  uint8_t* sm_v = sm_k + S * C::kOperand;     // [S]
  uint8_t* sm_o = sm_v + S * C::kOperand;     // [4 MT] warps' staging
  __shared__ __align__(8) uint64_t q_full[2], k_full[4], v_full[2], k_empty[2], v_empty[2], s_full[MT], p_full[MT],
      o_full[MT], turn[MT], drain;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ uint32_t s_there[4][4];      // positions of the tile that have a slot
  __shared__ float s_c[2][R];             // factor of a row's scores
  __shared__ uint32_t s_seen[4 * MT][6][32];  // nodes that a thread's node sees
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int kUnpackWarp = C::kSoftThreads / 32;

  CutSegment* cut = reinterpret_cast<CutSegment*>(a.ws) + blockIdx.x;
  if (tid == 0) *cut = CutSegment{0, 0, 0, 0};
  Line line;
  Walk<kTT, kEnds, R, WIN> walk;
  if (!attn_stretch<C::kThreads>(a, line, walk)) return;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      tc::bar_init(&q_full[i], C::kUnpackThreads / 32);
      tc::bar_init(&v_full[i], C::kUnpackThreads / 32);
      tc::bar_init(&k_empty[i], MT);
      tc::bar_init(&v_empty[i], MT);
    }
    for (int i = 0; i < 4; ++i) tc::bar_init(&k_full[i], C::kUnpackThreads / 32);
    for (int i = 0; i < MT; ++i) {
      tc::bar_init(&s_full[i], 1);
      tc::bar_init(&p_full[i], 4);
      tc::bar_init(&o_full[i], 1);
      tc::bar_init(&turn[i], 4);
    }
    tc::bar_init(&drain, MT);
    s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0) tc::alloc<C::kCols>(&s_tmem);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = s_tmem;

  if (warp >= kUnpackWarp) {
    // ------------------------------------------------------------- unpack
    const int ut = tid - C::kSoftThreads, uw = warp - kUnpackWarp;
    constexpr int UT = C::kUnpackThreads, kStep = UT / CH, kPer = kTT / kStep;  // positions of a thread: kStep apart
    const int g = ut % CH, p_of = ut / CH;  // group, first position
    // with two slabs, groups 2 and 3 store their units in the order 2, 3, 0, 1:
    // the eight lanes of a store phase then hit eight different units
    const bool swap = CH == 4 && g >= 2;
    // the cursor that reads ahead: slots two tiles before their use, codes one:
    // with two accumulators K's as soon as the tile before has left its
    // registers (B=128, 256 rows: 266 us behind V's instead, 259 so), with one
    // behind V's, since registers spill otherwise (64 rows: 162 us, 168)
    auto ahead = walk;
    Part ap;
    int at = -1;  // tile of the slots below, -1: the line is at its end
    int32_t slot[kPer];
    const uint8_t* head = nullptr;
    bool count = false;
    bool more = ahead.next(a, ap);
    int next_tile = more ? ap.t0 : 0;
    auto load_slots = [&]() {
      at = -1;
      if (!more) return;
      at = next_tile;
      head = a.pool + static_cast<int64_t>(ap.h) * kv4_head_bytes(D);
      count = ap.h == 0 && ap.rt == 0 && g == 0;
      const int32_t* row = a.table + static_cast<int64_t>(ap.b) * a.max_ctx;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int pos = at * kTT + p_of + i * kStep;
        // -2: no position, -1 or out of range: a bad slot
        slot[i] = pos < ap.end ? __ldg(row + pos + (WIN && pos >= ap.cut ? ap.gap : 0)) : -2;
      }
      if (++next_tile == ap.t1) {
        more = ahead.next(a, ap);
        next_tile = ap.t0;
      }
    };
    Chunk k[kPer], v[kPer];
    uint32_t have = 0;  // bit i: position i of this thread has a slot
    auto load_chunks = [&](bool of_k, bool of_v) {
      if (of_k) have = 0;
      if (at < 0) return;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        if (of_k) k[i] = Chunk{make_uint4(0, 0, 0, 0), 0};
        if (of_v) v[i] = Chunk{make_uint4(0, 0, 0, 0), 0};
        if (slot[i] >= 0 && slot[i] < a.num_slots) {
          const uint8_t* s = head + slot[i] * a.slot_stride;
          if (of_k) k[i].c = __ldg(reinterpret_cast<const uint4*>(s) + g);
          if (of_v) v[i].c = __ldg(reinterpret_cast<const uint4*>(s + D / 2) + g);
          if (of_k) k[i].m = __ldg(reinterpret_cast<const uint32_t*>(s + D) + g);
          if (of_v) v[i].m = __ldg(reinterpret_cast<const uint32_t*>(s + D + D / 8) + g);
          if (of_k) have |= 1u << i;
        } else if (of_k && count && slot[i] != -2) {
          bump(a.stats, SPEC_STAT_BAD_REQUEST);
        }
      }
    };
    // nodes: V of a tile with nodes, whose bytes may never have been written
    auto unpack_to = [&](uint8_t* dst, const Chunk& c, int pos, bool nodes) {
      uint8_t* slab = dst + (g >> 1) * C::kSlab;
      uint32_t st = __byte_perm(c.m, 0, 0x1010), lo = __byte_perm(c.m, 0, 0x3232);
      if (nodes) {
        const uint32_t keep = finite_values(st, lo);
        st &= keep;
        lo &= keep;
      }
      const uint32_t w[4] = {swap ? c.c.z : c.c.x, swap ? c.c.w : c.c.y, swap ? c.c.x : c.c.z, swap ? c.c.y : c.c.w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint32_t x[4];
        dequant4(w[q], st, lo, x);
        put_unit(slab, pos, (g & 1) * 4 + (swap ? q ^ 2 : q), x);
      }
    };
    load_slots();
    load_chunks(true, true);
    load_slots();
    Part p;
    bool ok = true;
    int64_t j = 0;
    int seg = 0;
#pragma unroll 1
    while (ok && walk.next(a, p)) {
      if (p.bad && p.h == 0 && p.rt == 0 && ut == 0) bump(a.stats, SPEC_STAT_BAD_REQUEST);
      // Q of the segment, behind its first K and once the S of the segment
      // before are done: all rows are copied as they are to where they belong,
      // then each lane turns its own bytes into fp16 in place (eight lanes a
      // row, D / 8 channels a lane).  The rows are on their way to the L2 cache
      // before
      const int r0 = p.rt * R, rows = min(R, p.nodes * a.G - r0);
      constexpr int per = D / 8;
      const int sub = lane & 7, q_row = uw * 4 + (lane >> 3);
      if ((sub & 3) == 0)
#pragma unroll 1
        for (int r = q_row; r < rows; r += UT / 8)
          asm volatile("prefetch.global.L2 [%0];" ::"l"(a.q + attn_q(a, p.b, p.h, r0 + r, D) + sub * per));
      auto q_unit = [&](int r, int i) {
        const int ch = sub * per + 8 * i, rr = r % kTreeRows;
        return reinterpret_cast<uint4*>(sm_q + (r / kTreeRows) * C::kOperand + (ch / 64) * C::kSlab + rr * 128 +
                                        (((ch % 64 / 8) ^ (rr & 7)) << 4));
      };
      auto store_q = [&]() {
#pragma unroll 1
        for (int r = q_row; r < R; r += UT / 8) {
          const uint16_t* src = a.q + attn_q(a, p.b, p.h, r0 + min(r, rows - 1), D) + sub * per;
#pragma unroll
          for (int i = 0; i < per / 8; ++i) cp_async16(q_unit(r, i), src + 8 * i, r < rows ? 16 : 0);
        }
        cp_async_commit();
        cp_async_wait<0>();
#pragma unroll 1
        for (int r = q_row; r < R; r += UT / 8) {
          // the largest magnitude: bf16 bits without the sign compare as integers
          uint32_t big = 0;
          uint4 raw[per / 8];
#pragma unroll
          for (int i = 0; i < per / 8; ++i) {
            raw[i] = *q_unit(r, i);
#pragma unroll
            for (int z = 0; z < 4; ++z) big = __vmaxu2(big, word_of4(raw[i], z) & 0x7fff7fffu);
          }
#pragma unroll
          for (int o = 1; o < 8; o <<= 1) big = __vmaxu2(big, __shfl_xor_sync(0xffffffffu, big, o));
          const int bits = static_cast<int>(max(big & 0xffffu, big >> 16));
          // 2^e <= max < 2^(e + 1), but 126 at most (2^-127 is no normal number;
          // the largest is then below 4); zeros, and rows with an infinity or NaN,
          // are taken as they are
          const int e = bits == 0 || bits >= 0x7f80 ? 0 : min(max((bits >> 7) - 127, -126), 126);
          const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
          if (sub == 0) s_c[seg & 1][r] = a.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
#pragma unroll
          for (int i = 0; i < per / 8; ++i) {
            uint32_t y[4];
#pragma unroll
            for (int z = 0; z < 4; ++z) {
              const uint32_t w = word_of4(raw[i], z);
              y[z] = h2_u32(__floats2half2_rn(bf16_lo(w) * down, bf16_hi(w) * down));
            }
            *q_unit(r, i) = make_uint4(y[0], y[1], y[2], y[3]);
          }
        }
        tc::fence_smem();
        __syncwarp();
        if (lane == 0) tc::bar_arrive(&q_full[seg & 1]);
      };

#pragma unroll 1
      for (int tile = p.t0; tile < p.t1; ++tile, ++j) {
        const int st = static_cast<int>(j % S);
        // K: the stage is free once S of tile j - S has been computed
        if (j >= S) ok = wait_warp(&k_empty[st], static_cast<uint32_t>(j / S - 1) & 1u, &s_abort);
        if (!ok) break;
#pragma unroll
        for (int i = 0; i < kPer; ++i) unpack_to(sm_k + st * C::kOperand, k[i], p_of + i * kStep, false);
        // which of this warp's positions have a slot: 32 / CH in a row from
        // uw 32 / CH + i kStep on, CH lanes each
        const bool all = __all_sync(0xffffffffu, have == (1u << kPer) - 1u);
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          uint32_t bits = (1u << (32 / CH)) - 1u;
          if (!all) {
            const unsigned bal = __ballot_sync(0xffffffffu, (have >> i) & 1u);
            bits = 0;
#pragma unroll 1
            for (int q = 0; q < 32 / CH; ++q) bits |= ((bal >> (q * CH)) & 1u) << q;
          }
          if (lane == 0) {
            uint8_t* to = reinterpret_cast<uint8_t*>(s_there[j & 3]) + (uw * (32 / CH) + i * kStep) / 8;
            if (CH == 4) *to = static_cast<uint8_t>(bits);
            else *reinterpret_cast<uint16_t*>(to) = static_cast<uint16_t>(bits);
          }
        }
        tc::fence_smem();
        __syncwarp();
        if (lane == 0) tc::bar_arrive(&k_full[j & 3]);
        if (MT == 2) load_chunks(true, false);
        if (tile == p.t0) {
          if (j > 0)
            for (int m = 0; m < MT && ok; ++m) ok = wait_warp(&s_full[m], (j - 1) & 1, &s_abort);
          if (!ok) break;
          store_q();
        }
        // V: free once O of tile j - S has been computed
        if (j >= S) ok = wait_warp(&v_empty[st], static_cast<uint32_t>(j / S - 1) & 1u, &s_abort);
        if (!ok) break;
#pragma unroll
        for (int i = 0; i < kPer; ++i)
          unpack_to(sm_v + st * C::kOperand, v[i], p_of + i * kStep, (tile + 1) * kTT > p.start);
        tc::fence_smem();
        __syncwarp();
        if (lane == 0) tc::bar_arrive(&v_full[j & 1]);
        load_chunks(MT == 1, true);
        load_slots();
      }
      ++seg;
    }
  } else {
    // ------------------------------------------------------------ softmax
    const int m = warp >> 2;                                     // accumulator
    const int r = m * kTreeRows + (warp & 3) * 32 + lane;        // row of the row tile
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const bool issuer = (warp & 3) == 0;
    constexpr uint32_t kIdS = tc::idesc_f16(kTT, false), kIdO = tc::idesc_f16(D, true);
    const uint32_t s_col = tmem + lanes + m * kTT, o_col = tmem + lanes + MT * kTT + m * D;
    int seen_b = -1, seen_rt = -1;  // whose words s_seen holds (a thread reads its own only)
    Part p;
    bool ok = true;
    int64_t j = 0;
    int seg = 0;
#pragma unroll 1
    while (ok && walk.next(a, p)) {
      const int r0 = p.rt * R, rows = min(R, p.nodes * a.G - r0);
      const bool active = r - lane < rows;  // the warp has a row
      const int node = attn_node(a, r0 + min(r, rows - 1));
      if (p.t0 == 0 && p.t1 < p.tiles && tid == 0)
        *cut = CutSegment{p.b, p.h, p.rt, line.pieces(static_cast<int>(blockIdx.x), p.tiles, p.t1)};
      ok = wait_warp(&q_full[seg & 1], (seg >> 1) & 1, &s_abort);
      if (!ok) break;
      const float c = s_c[seg & 1][r];
      float top = neg_inf(), sum = 0.0f;  // maximum in use (units of log2), sum of weights
#pragma unroll 1
      for (int tile = p.t0; tile < p.t1; ++tile, ++j) {
        ok = wait_warp(&k_full[j & 3], (j >> 2) & 1, &s_abort);
        if (issuer) {
          // S, once K is there and O of the tile before is done: P lies over S
          if (j > 0) ok = ok && wait_warp(&o_full[m], static_cast<uint32_t>(j - 1) & 1u, &s_abort);
          if (ok && lane == 0) {
            tc::fence_after();
            const uint64_t qd = tc::desc(tc::smem_addr(sm_q + m * C::kOperand), 0);
            const uint64_t kd = tc::desc(tc::smem_addr(sm_k + static_cast<int>(j % S) * C::kOperand), 0);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t off = ((kk / 4) * C::kSlab + (kk % 4) * 32) >> 4;  // addresses stay below 2^18
              tc::mma_ss(tmem + m * kTT, qd + off, kd + off, kIdS, kk != 0 ? 1u : 0u);
            }
            tc::commit(&s_full[m]);
            tc::commit(&k_empty[j % S]);
          }
          __syncwarp();
        }
        if (!ok) break;
        const int p0 = tile * kTT;
        uint32_t see[4] = {~0u, ~0u, ~0u, ~0u};
        if (active && p0 + kTT > p.start) {
          const int shift = p0 - p.start;  // node of the tile's first position
          const bool keep = a.N <= kTT;    // then the words of all nodes serve every head of the request
          if (!keep || p.b != seen_b || p.rt != seen_rt) {
            node_words<WIN>(a, p, node, keep ? 0 : shift, see);
            seen_b = p.b;
            seen_rt = p.rt;
            if (keep) {
              // a word of context before the nodes' four, one of nothing behind
#pragma unroll
              for (int w = 0; w < 4; ++w) s_seen[warp][w + 1][lane] = see[w];
              s_seen[warp][0][lane] = ~0u;
              s_seen[warp][5][lane] = 0u;
            }
          }
          if (keep) {
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const int i = (shift >> 5) + w + 1;
              see[w] = __funnelshift_r(s_seen[warp][min(max(i, 0), 5)][lane], s_seen[warp][min(max(i + 1, 0), 5)][lane],
                                       shift & 31);
            }
          }
        }
        if (WIN && active && p0 + kTT > p.cut && attn_all_see(a, p) > max(p0, p.cut)) {
          // the context before the window of this thread's node: places [cut, to)
          const int to = min(p.start + attn_depth(a, p, node) - a.window + 1, p.start);
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const int lo = min(max(p.cut - p0 - 32 * w, 0), 32), hi = min(max(to - p0 - 32 * w, lo), 32);
            see[w] &= ~(__funnelshift_lc(~0u, 0u, hi) & ~__funnelshift_lc(~0u, 0u, lo));
          }
        }
        ok = wait_warp(&s_full[m], j & 1, &s_abort);
        // the accumulators take turns: in step with one another both would
        // wait for the exponentials and then both for the products
        if (MT == 2 && (m == 1 || j > 0))
          ok = ok && wait_warp(&turn[m], static_cast<uint32_t>(m == 1 ? j : j - 1) & 1u, &s_abort);
        if (!ok) break;
        tc::fence_after();
        if (active) {
#pragma unroll
          for (int i = 0; i < 4; ++i) see[i] &= s_there[j & 3][i];
          float mx = row_max(s_col, see);
          mx = mx == neg_inf() ? mx : mx * c;
          // the difference, since far from zero top + 8 may round up by more than
          // the weights have room for
          const bool grow = mx - top > kLagExp;  // from -inf too; never to it
          if (__any_sync(0xffffffffu, grow)) {
            const float f = grow ? (top == neg_inf() ? 0.0f : fast_exp2(top - mx)) : 1.0f;
            if (grow) top = mx;
            if (tile > p.t0) {  // O of the segment's earlier tiles
              sum *= f;
#pragma unroll 1
              for (int w = 0; w < D / 16; ++w) {
                uint32_t x[16];
                tc::ld16(o_col + 16 * w, x);
                tc::wait_ld(x);
#pragma unroll
                for (int i = 0; i < 16; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) * f);
                tc::st16(o_col + 16 * w, x);
              }
            }
          }
          const float from = top == neg_inf() ? 0.0f : top;
          sum += row_weights(s_col, see, c, weight_base(from, kHeldExp), fabsf(from) > kFar);
          tc::wait_st();
        }
        tc::fence_before();
        __syncwarp();
        if (lane == 0) {
          tc::bar_arrive(&p_full[m]);
          if (MT == 2) tc::bar_arrive(&turn[(m + 1) % MT]);
        }
        if (issuer) {
          ok = wait_warp(&p_full[m], j & 1, &s_abort) && wait_warp(&v_full[j & 1], (j >> 1) & 1, &s_abort);
          if (!ok) break;
          if (lane == 0) {
            tc::fence_after();
            const uint64_t vd = tc::desc(tc::smem_addr(sm_v + static_cast<int>(j % S) * C::kOperand), C::kSlab);
#pragma unroll
            for (int kk = 0; kk < kTT / 16; ++kk)  // a part's first tile starts O afresh
              tc::mma_ts(tmem + MT * kTT + m * D, tmem + m * kTT + kk * 8, vd + (kk * 16 * 128 >> 4), kIdO,
                         (tile == p.t0 && kk == 0) ? 0u : 1u);
            tc::commit(&o_full[m]);
            tc::commit(&v_empty[j % S]);
          }
          __syncwarp();
        }
      }
      if (!ok) break;
      // the segment's part is done: its last O
      ok = wait_warp(&o_full[m], static_cast<uint32_t>(j - 1) & 1u, &s_abort);
      if (!ok) break;
      tc::fence_after();
      if (active) {
        float* part = attn_part(a, blockIdx.x, p.t0 > 0 ? 0 : 1, R, D);
        const float inv = attn_inv(sum);
        // 64 bytes of every row at a time through shared memory, so that four
        // lanes store them together: a lane that stores its own row touches 32
        // lines an instruction (8.5k cycles a segment instead of 2k)
        uint8_t* stage = sm_o + warp * C::kStageWarp;
        const int cols = p.complete() ? 32 : 16;
        char* base = reinterpret_cast<char*>(p.complete() ? static_cast<void*>(a.out) : static_cast<void*>(part));
        int64_t to[4];  // where this lane's 16 bytes of the rows 8 i + lane / 4 go
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int rr = r - lane + 8 * i + (lane >> 2);
          to[i] = p.complete() ? attn_row(a, p.b, p.h, r0 + rr) * (D * 2) : static_cast<int64_t>(rr) * (D * 4);
          to[i] += 16 * (lane & 3);
        }
#pragma unroll 1
        for (int w = 0; w < D / cols; ++w) {
          uint32_t x[16];
          if (p.complete()) {
            uint32_t y[32];
            tc::ld32(o_col + 32 * w, y);
            tc::wait_ld32(y);
#pragma unroll
            for (int i = 0; i < 16; ++i)
              x[i] = f_bf16(__uint_as_float(y[2 * i]) * inv) |
                     static_cast<uint32_t>(f_bf16(__uint_as_float(y[2 * i + 1]) * inv)) << 16;
          } else {
            tc::ld16(o_col + 16 * w, x);
            tc::wait_ld(x);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *reinterpret_cast<uint4*>(stage + lane * C::kStageRow + 16 * i) =
                make_uint4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int lr = 8 * i + (lane >> 2);  // row of the warp
            if (r - lane + lr < rows) {
              const uint4 v = *reinterpret_cast<const uint4*>(stage + lr * C::kStageRow + 16 * (lane & 3));
              *reinterpret_cast<uint4*>(base + (i == 0 ? to[0] : i == 1 ? to[1] : i == 2 ? to[2] : to[3]) + 64 * w) = v;
            }
          }
          __syncwarp();
        }
        if (r < rows) {
          if (!p.complete()) {
            part[R * D + 2 * r] = top;
            part[R * D + 2 * r + 1] = sum;
          } else if (a.lse) {
            a.lse[attn_row(a, p.b, p.h, r0 + r)] = attn_lse(top, sum, kHeldExp);
          }
        }
      }
      ++seg;
    }
    if (issuer && lane == 0) {
      // nothing in flight when tensor memory is freed
      tc::commit(&drain);
      const long long t0 = clock64();
      while (!tc::bar_test(&drain, 0) && clock64() - t0 < tc::kWaitCycles) {
      }
    }
    __syncwarp();
  }
  tc::fence_before();
  __syncthreads();
  if (warp == 0) {
    tc::fence_after();
    tc::dealloc<C::kCols>(tmem);
  }
  if (tid == 0 && s_abort) bump(a.stats, SPEC_STAT_WAIT_TIMEOUT);
}

template <int D, int MT, bool WIN>
int launch_tree(AttnArgs a, int sms, cudaStream_t s) {
  using C = TreeCfg<D, MT>;
  constexpr int R = kTreeRows * MT;
  constexpr auto kernel = kv4_tree_kernel<D, MT, WIN>;
  if (!allow_smem<kernel>(C::kSmem)) return SPEC_ERR_CUDA;
  a.ctas = sms * (MT == 2 ? 1 : 2);
  a.ctas = a.ctas < kTreeMaxCtas / MT ? a.ctas : kTreeMaxCtas / MT;
  launch_k(kernel, static_cast<unsigned>(a.ctas), C::kThreads, C::kSmem, s, a);
  launch_merge<D>(a, R, kHeldExp, s);
  return launch_status();
}

template <bool WIN>
int launch_tree(const AttnArgs& a, int D, int sms, cudaStream_t s) {
  // two accumulators where there are rows for them (8 KV heads, contexts
  // 16..2048, in us with one / with two: D=128, B=128: 96 rows 160 / 223, 128
  // rows 161 / 226, 160 rows 291 / 246; B=8: 128 rows 31.1 / 31.6, 160 rows 36.8
  // / 34.8; D=64, B=128: 128 rows 118 / 190, 160 rows 208 / 213; B=8: 128 rows
  // 27.5 / 27.7, 160 rows 31.8 / 31.2)
  const bool two = static_cast<int64_t>(a.N) * a.G > kTreeRows;
  if (D == 128) return two ? launch_tree<128, 2, WIN>(a, sms, s) : launch_tree<128, 1, WIN>(a, sms, s);
  return two ? launch_tree<64, 2, WIN>(a, sms, s) : launch_tree<64, 1, WIN>(a, sms, s);
}

}  // namespace

int launch_tree_attention(AttnArgs a, int D, int sms, cudaStream_t s) {
  return a.window != 0 ? launch_tree<true>(a, D, sms, s) : launch_tree<false>(a, D, sms, s);
}

}  // namespace specdec
