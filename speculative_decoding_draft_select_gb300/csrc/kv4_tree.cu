// Attention of many rows (trees) over the 4-bit cache on the fifth-generation
// tensor cores.  The mathematics and the division of the work are those of
// kv4_attention.cu; here a row tile is one or two accumulators of 128 rows
// (MT) and a tile 128 positions, and per tile
//   S = Q K^T   128 x 128 x D, Q and K in shared memory
//   P = 2^(S c - max + 7) in fp16, written over S in tensor memory
//   O += P V    128 x D x 128, P from tensor memory, V in shared memory
// all operands fp16 with fp32 accumulation.  Roles of a CTA:
//   warps 0 .. 4 MT - 1   softmax: a thread owns one row of an accumulator, so
//       maximum and sum need no exchange; it also writes the results.
//   the next 4 MT warps   unpack the cache: codes go from memory through
//       registers (one tile ahead, whichever segment it belongs to) to swizzled
//       fp16 slabs; Q likewise.
//   the last warp         one thread issues the matrix instructions.
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
  static constexpr int kThreads = kSoftThreads + kUnpackThreads + 32;
  static constexpr int kSlabs = D / 64;
  static constexpr int kSlab = kTT * 128;          // bytes: 128 rows of 64 elements
  static constexpr int kOperand = kSlabs * kSlab;  // K, V or one accumulator's Q
  static constexpr size_t kSmem = static_cast<size_t>(kOperand) * (MT + 2 * kStages) + 1024;
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

// A group of 32 channels: codes and their (step, lo).
struct Chunk {
  uint4 c;
  uint32_t m;
};

// A thread's row of S, 16 columns at a time with the next 16 on their way:
// the largest element that `see` shows, and the weights 2^(S c - base) as fp16
// over S's first columns (column i of P holds positions 2 i and 2 i + 1; it
// never reaches columns that are still to be read), with their fp32 sum.
// Rolled to a word of `see` an iteration: unrolled further, the roles' code
// together falls out of the instruction cache.
__device__ __forceinline__ uint32_t pick(const uint32_t* v, int i) {
  return i < 2 ? (i == 0 ? v[0] : v[1]) : (i == 2 ? v[2] : v[3]);
}
template <bool MASKED>
__device__ __forceinline__ float row_max(uint32_t col, const uint32_t* see) {
  uint32_t x[2][16];
  float m[4] = {neg_inf(), neg_inf(), neg_inf(), neg_inf()};
  tc::ld16(col, x[0]);
#pragma unroll 1
  for (int w = 0; w < kTT / 32; ++w) {
    const uint32_t sw = MASKED ? pick(see, w) : 0;
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      tc::wait_ld(x[hf]);
      // the load behind the last one rereads S's first columns
      tc::ld16(col + ((32 * w + 16 * (hf + 1)) & (kTT - 1)), x[hf ^ 1]);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float y = __uint_as_float(x[hf][i]);
        if (MASKED) y = (sw >> (16 * hf + i)) & 1u ? y : neg_inf();
        m[i & 3] = fmaxf(m[i & 3], y);
      }
    }
  }
  tc::wait_ld(x[0]);
  return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}
template <bool MASKED>
__device__ __forceinline__ float row_weights(uint32_t col, const uint32_t* see, float c, float base) {
  uint32_t x[2][16], y[8];
  const float2 c2 = splat(c), nb2 = splat(-base);
  float2 acc[2] = {splat(0.0f), splat(0.0f)};
  tc::ld16(col, x[0]);
#pragma unroll 1
  for (int w = 0; w < kTT / 32; ++w) {
    const uint32_t sw = MASKED ? pick(see, w) : 0;
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      tc::wait_ld(x[hf]);
      // behind the last: columns that no P of this loop reaches (16 w + 8 .. < 64)
      tc::ld16(col + (w == kTT / 32 - 1 && hf == 1 ? kTT - 16 : 32 * w + 16 * (hf + 1)), x[hf ^ 1]);
#pragma unroll
      for (int i = 0; i < 16; i += 2) {
        float2 e = exp2_2(fma2(make_float2(__uint_as_float(x[hf][i]), __uint_as_float(x[hf][i + 1])), c2, nb2));
        if (MASKED) {
          e.x = (sw >> (16 * hf + i)) & 1u ? e.x : 0.0f;
          e.y = (sw >> (16 * hf + i + 1)) & 1u ? e.y : 0.0f;
        }
        acc[(i >> 1) & 1] = add2(acc[(i >> 1) & 1], e);
        y[i / 2] = h2_u32(__floats2half2_rn(e.x, e.y));
      }
      tc::st8(col + 16 * w + 8 * hf, y);
    }
  }
  tc::wait_ld(x[0]);
  const float2 t = add2(acc[0], acc[1]);
  return t.x + t.y;
}

template <int D, int MT>
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
  __shared__ __align__(8) uint64_t q_full[2], k_full[4], v_full[2], k_empty[2], v_empty[2], s_full[MT], p_full[MT],
      o_full[MT], drain;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ uint32_t s_there[4][4];      // positions of the tile that have a slot
  __shared__ float s_c[2][R];             // factor of a row's scores
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int kMmaWarp = C::kThreads / 32 - 1, kUnpackWarp = C::kSoftThreads / 32;

  CutSegment* cut = reinterpret_cast<CutSegment*>(a.ws) + blockIdx.x;
  if (tid == 0) *cut = CutSegment{0, 0, 0, 0};
  Line line;
  Walk<kTT, kEnds, R> walk;
  if (!attn_stretch<kTT, kEnds, R, C::kThreads>(a, line, walk)) return;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      tc::bar_init(&q_full[i], C::kUnpackThreads / 32);
      tc::bar_init(&v_full[i], C::kUnpackThreads / 32);
      tc::bar_init(&k_empty[i], 1);
      tc::bar_init(&v_empty[i], 1);
    }
    for (int i = 0; i < 4; ++i) tc::bar_init(&k_full[i], C::kUnpackThreads / 32);
    for (int i = 0; i < MT; ++i) {
      tc::bar_init(&s_full[i], 1);
      tc::bar_init(&p_full[i], 4);
      tc::bar_init(&o_full[i], 1);
    }
    tc::bar_init(&drain, 1);
    s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kMmaWarp) tc::alloc<C::kCols>(&s_tmem);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = s_tmem;

  if (warp == kMmaWarp) {
    if (lane == 0) {
      // the line of tiles: S of tile j + 1 is issued behind O of tile j
      constexpr uint32_t kIdS = tc::idesc_f16(kTT, false), kIdO = tc::idesc_f16(D, true);
      Part p;
      // S of tile j, accumulator m; `fresh`: the tile begins segment `seg`
      auto issue_s = [&](int64_t j, int m, bool fresh, int seg) {
        const int st = static_cast<int>(j % S);
        if (m == 0 && !tc::bar_wait(&k_full[j & 3], (j >> 2) & 1, &s_abort)) return false;
        if (m == 0 && fresh && !tc::bar_wait(&q_full[seg & 1], (seg >> 1) & 1, &s_abort)) return false;
        tc::fence_after();
        const uint32_t qa = tc::smem_addr(sm_q + m * C::kOperand), ka = tc::smem_addr(sm_k + st * C::kOperand);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk / 4) * C::kSlab + (kk % 4) * 32;
          tc::mma_ss(tmem + m * kTT, tc::desc(qa + off, 0), tc::desc(ka + off, 0), kIdS, kk != 0 ? 1u : 0u);
        }
        tc::commit(&s_full[m]);
        if (m == MT - 1) tc::commit(&k_empty[st]);
        return true;
      };
      bool ok = walk.next(a, p), begins = true;
      int seg = 0, tiles = p.t1 - p.t0;
      for (int m = 0; m < MT && ok; ++m) ok = issue_s(0, m, true, 0);
      for (int64_t j = 0; ok; ++j) {
        // tile j + 1, if there is one, is of this segment or begins the next
        const bool last = --tiles == 0, next = !last || walk.next(a, p);
        if (last && next) {
          tiles = p.t1 - p.t0;
          ++seg;
        }
        const int st = static_cast<int>(j % S);
        for (int m = 0; m < MT && ok; ++m) {
          ok = tc::bar_wait(&p_full[m], j & 1, &s_abort);
          if (m == 0) ok = ok && tc::bar_wait(&v_full[j & 1], (j >> 1) & 1, &s_abort);
          if (!ok) break;
          tc::fence_after();
          const uint32_t va = tc::smem_addr(sm_v + st * C::kOperand);
#pragma unroll
          for (int kk = 0; kk < kTT / 16; ++kk)  // a segment's first tile starts O afresh
            tc::mma_ts(tmem + MT * kTT + m * D, tmem + m * kTT + kk * 8, tc::desc(va + kk * 16 * 128, C::kSlab), kIdO,
                       (begins && kk == 0) ? 0u : 1u);
          tc::commit(&o_full[m]);
          if (m == MT - 1) tc::commit(&v_empty[st]);
          if (next) {
            // P lies over S: O has to be done before S is written again
            ok = tc::bar_wait(&o_full[m], j & 1, &s_abort) && issue_s(j + 1, m, last, seg);
          }
        }
        if (!next) break;
        begins = last;
      }
      // nothing in flight when tensor memory is freed
      tc::commit(&drain);
      const long long t0 = clock64();
      while (!tc::bar_test(&drain, 0) && clock64() - t0 < tc::kWaitCycles) {
      }
    }
    __syncwarp();
  } else if (warp >= kUnpackWarp) {
    // ------------------------------------------------------------- unpack
    const int ut = tid - C::kSoftThreads, uw = warp - kUnpackWarp;
    constexpr int UT = C::kUnpackThreads, kStep = UT / CH, kPer = kTT / kStep;  // positions of a thread: kStep apart
    const int g = ut % CH, p_of = ut / CH;  // group, first position
    // with two slabs, groups 2 and 3 store their units in the order 2, 3, 0, 1:
    // the eight lanes of a store phase then hit eight different units
    const bool swap = CH == 4 && g >= 2;
    // the cursor that reads ahead: slots two tiles before their use, codes one
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
        slot[i] = pos < ap.end ? __ldg(row + pos) : -2;  // -2: no position, -1 or out of range: a bad slot
      }
      if (++next_tile == ap.t1) {
        more = ahead.next(a, ap);
        next_tile = ap.t0;
      }
    };
    Chunk k[kPer], v[kPer];
    uint32_t have = 0;  // bit i: position i of this thread has a slot
    auto load_chunks = [&]() {
      have = 0;
      if (at < 0) return;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        k[i].c = v[i].c = make_uint4(0, 0, 0, 0);
        k[i].m = v[i].m = 0;
        if (slot[i] >= 0 && slot[i] < a.num_slots) {
          const uint8_t* s = head + slot[i] * a.slot_stride;
          k[i].c = __ldg(reinterpret_cast<const uint4*>(s) + g);
          v[i].c = __ldg(reinterpret_cast<const uint4*>(s + D / 2) + g);
          k[i].m = __ldg(reinterpret_cast<const uint32_t*>(s + D) + g);
          v[i].m = __ldg(reinterpret_cast<const uint32_t*>(s + D + D / 8) + g);
          have |= 1u << i;
        } else if (count && slot[i] != -2) {
          bump(a.stats, SPEC_STAT_BAD_REQUEST);
        }
      }
    };
    auto unpack_to = [&](uint8_t* dst, const Chunk& c, int pos) {
      uint8_t* slab = dst + (g >> 1) * C::kSlab;
      const uint32_t st = __byte_perm(c.m, 0, 0x1010), lo = __byte_perm(c.m, 0, 0x3232);
      const uint32_t w[4] = {swap ? c.c.z : c.c.x, swap ? c.c.w : c.c.y, swap ? c.c.x : c.c.z, swap ? c.c.y : c.c.w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint32_t x[4];
        dequant4(w[q], st, lo, x);
        put_unit(slab, pos, (g & 1) * 4 + (swap ? q ^ 2 : q), x);
      }
    };
    load_slots();
    load_chunks();
    load_slots();
    Part p;
    bool ok = true;
    int64_t j = 0;
    int seg = 0;
    while (ok && walk.next(a, p)) {
      if (p.bad && p.h == 0 && p.rt == 0 && ut == 0) bump(a.stats, SPEC_STAT_BAD_REQUEST);
      // Q of the segment: read, then stored once the S of the segment before
      // are done (the wait for a K stage below covers one stage only).  Eight
      // lanes a row, D / 8 channels a lane, four rows of a lane in flight
      const int r0 = p.rt * R, rows = min(R, p.nodes * a.G - r0);
      constexpr int per = D / 8, kBatch = 2 * MT;
      const int sub = lane & 7;
#pragma unroll 1
      for (int rb = uw * 4 + (lane >> 3); rb < R; rb += UT / 8 * kBatch) {
        uint4 raw[kBatch][per / 8];
#pragma unroll
        for (int q = 0; q < kBatch; ++q) {
          const int r = rb + q * (UT / 8);
#pragma unroll
          for (int i = 0; i < per / 8; ++i) raw[q][i] = make_uint4(0, 0, 0, 0);
          if (r < rows) {
            const int rw = r0 + r, n = rw / a.G;
            const uint16_t* src = a.q + (static_cast<int64_t>(p.b) * a.N + n) * a.q_stride +
                                  static_cast<int64_t>(p.h * a.G + rw - n * a.G) * D + sub * per;
#pragma unroll
            for (int i = 0; i < per / 8; ++i) raw[q][i] = __ldg(reinterpret_cast<const uint4*>(src) + i);
          }
        }
        if (rb < UT / 8 && j > 0)
          for (int m = 0; m < MT && ok; ++m) ok = wait_warp(&s_full[m], (j - 1) & 1, &s_abort);
        if (!ok) break;
#pragma unroll
        for (int q = 0; q < kBatch; ++q) {
          const int r = rb + q * (UT / 8);
          float x[per], mx = 0.0f;
#pragma unroll
          for (int i = 0; i < per / 8; ++i) unpack<SPEC_BF16>(raw[q][i], x + 8 * i);
#pragma unroll
          for (int i = 0; i < per; ++i) mx = fmaxf(mx, fabsf(x[i]));
#pragma unroll
          for (int o = 1; o < 8; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
          const int e = max(mx > 0.0f && isfinite(mx) ? static_cast<int>(__float_as_uint(mx) >> 23) - 127 : 0, -126);
          // the sign of the scale goes into q, so that a larger S is a larger score
          const float down = copysignf(__uint_as_float(static_cast<uint32_t>(127 - e) << 23), a.scale_log2);
          if (sub == 0) s_c[seg & 1][r] = fabsf(a.scale_log2) * __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
          uint8_t* op = sm_q + (r / kTreeRows) * C::kOperand;
#pragma unroll
          for (int i = 0; i < per; i += 8) {
            const int ch = sub * per + i;
            uint32_t y[4];
#pragma unroll
            for (int z = 0; z < 4; ++z) y[z] = h2_u32(__floats2half2_rn(x[i + 2 * z] * down, x[i + 2 * z + 1] * down));
            put_unit(op + (ch / 64) * C::kSlab, r % kTreeRows, (ch % 64) / 8, y);
          }
        }
      }
      if (!ok) break;
      tc::fence_smem();
      __syncwarp();
      if (lane == 0) tc::bar_arrive(&q_full[seg & 1]);

      for (int tile = p.t0; tile < p.t1; ++tile, ++j) {
        const int st = static_cast<int>(j % S);
        // K: the stage is free once S of tile j - S has been computed
        if (j >= S) ok = wait_warp(&k_empty[st], static_cast<uint32_t>(j / S - 1) & 1u, &s_abort);
        if (!ok) break;
#pragma unroll
        for (int i = 0; i < kPer; ++i) unpack_to(sm_k + st * C::kOperand, k[i], p_of + i * kStep);
        // which of this warp's positions have a slot: 32 / CH in a row from
        // uw 32 / CH + i kStep on, CH lanes each
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const unsigned bal = __ballot_sync(0xffffffffu, (have >> i) & 1u);
          if (lane == 0) {
            uint32_t bits = 0;
#pragma unroll
            for (int q = 0; q < 32 / CH; ++q) bits |= ((bal >> (q * CH)) & 1u) << q;
            uint8_t* to = reinterpret_cast<uint8_t*>(s_there[j & 3]) + (uw * (32 / CH) + i * kStep) / 8;
            to[0] = static_cast<uint8_t>(bits);
            if (CH == 2) to[1] = static_cast<uint8_t>(bits >> 8);
          }
        }
        tc::fence_smem();
        __syncwarp();
        if (lane == 0) tc::bar_arrive(&k_full[j & 3]);
        // V: free once O of tile j - S has been computed
        if (j >= S) ok = wait_warp(&v_empty[st], static_cast<uint32_t>(j / S - 1) & 1u, &s_abort);
        if (!ok) break;
#pragma unroll
        for (int i = 0; i < kPer; ++i) unpack_to(sm_v + st * C::kOperand, v[i], p_of + i * kStep);
        tc::fence_smem();
        __syncwarp();
        if (lane == 0) tc::bar_arrive(&v_full[j & 1]);
        load_chunks();
        load_slots();
      }
      ++seg;
    }
  } else {
    // ------------------------------------------------------------ softmax
    const int m = warp >> 2;                                     // accumulator
    const int r = m * kTreeRows + (warp & 3) * 32 + lane;        // row of the row tile
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_col = tmem + lanes + m * kTT, o_col = tmem + lanes + MT * kTT + m * D;
    Part p;
    bool ok = true;
    int64_t j = 0;
    int seg = 0;
    while (ok && walk.next(a, p)) {
      const int r0 = p.rt * R, rows = min(R, p.nodes * a.G - r0);
      const bool active = r - lane < rows;  // the warp has a row
      const int node = (r0 + min(r, rows - 1)) / a.G;
      if (p.t0 == 0 && p.t1 < p.tiles && tid == 0)
        *cut = CutSegment{p.b, p.h, p.rt, line.pieces(static_cast<int>(blockIdx.x), p.tiles, p.t1)};
      ok = wait_warp(&q_full[seg & 1], (seg >> 1) & 1, &s_abort);
      if (!ok) break;
      const float c = s_c[seg & 1][r];
      float top = neg_inf(), sum = 0.0f;  // maximum in use (units of log2), sum of weights
      for (int tile = p.t0; tile < p.t1; ++tile, ++j) {
        const int p0 = tile * kTT;
        uint32_t see[4] = {~0u, ~0u, ~0u, ~0u};
        bool masked = false;
        if (active && p0 + kTT > p.start) {
          // positions of nodes: bit i of word w is position p0 + 32 w + i, the
          // node that less start.  A lane loads the mask byte of its position
          // for four of the warp's nodes at a time, ballots give their words
          masked = true;
          const int n_lo = __shfl_sync(0xffffffffu, node, 0), n_hi = __shfl_sync(0xffffffffu, node, 31);
          for (int nb = n_lo; nb <= n_hi; nb += 4) {
            bool on[4][4];
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
              for (int w = 0; w < 4; ++w) {
                const int nd = p0 + 32 * w + lane - p.start, n = min(nb + q, n_hi);
                on[q][w] = nd < 0;
                if (nd >= 0 && nd < p.nodes)
                  on[q][w] = a.mask ? __ldg(a.mask + (static_cast<int64_t>(p.b) * a.N + n) * a.N + nd) != 0 : nd <= n;
              }
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
              for (int w = 0; w < 4; ++w) {
                const uint32_t bits = __ballot_sync(0xffffffffu, on[q][w]);
                if (nb + q == node) see[w] = bits;
              }
          }
        }
        ok = wait_warp(&k_full[j & 3], (j >> 2) & 1, &s_abort) && wait_warp(&s_full[m], j & 1, &s_abort);
        if (!ok) break;
        tc::fence_after();
        if (active) {
#pragma unroll
          for (int i = 0; i < 4; ++i) see[i] &= s_there[j & 3][i];
          masked = masked || (see[0] & see[1] & see[2] & see[3]) != ~0u;  // missing slots are the same in every lane
          float mx = masked ? row_max<true>(s_col, see) : row_max<false>(s_col, see);
          mx = mx == neg_inf() ? mx : mx * c;
          const bool grow = mx > top + kLagExp || (top == neg_inf() && mx > top);
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
          const float base = (top == neg_inf() ? 0.0f : top) - kHeldExp;
          sum += masked ? row_weights<true>(s_col, see, c, base) : row_weights<false>(s_col, see, c, base);
          tc::wait_st();
        }
        tc::fence_before();
        __syncwarp();
        if (lane == 0) tc::bar_arrive(&p_full[m]);
      }
      if (!ok) break;
      // the segment's part is done: its last O
      ok = wait_warp(&o_full[m], static_cast<uint32_t>(j - 1) & 1u, &s_abort);
      if (!ok) break;
      tc::fence_after();
      if (active) {
        const int rw = r0 + r, n = rw / a.G;
        const int64_t at = (static_cast<int64_t>(p.b) * a.N + n) * a.Hq + p.h * a.G + rw - n * a.G;
        float* part = attn_part(a, blockIdx.x, p.t0 > 0 ? 0 : 1, R, D);
        const float inv = attn_inv(sum);
#pragma unroll 1
        for (int w = 0; w < D / 16; ++w) {
          uint32_t x[16];
          tc::ld16(o_col + 16 * w, x);
          tc::wait_ld(x);
          if (r < rows && p.complete()) {
            uint4* dst = reinterpret_cast<uint4*>(a.out + at * D + 16 * w);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              uint32_t y[4];
#pragma unroll
              for (int q = 0; q < 4; ++q)
                y[q] = f_bf16(__uint_as_float(x[8 * i + 2 * q]) * inv) |
                       static_cast<uint32_t>(f_bf16(__uint_as_float(x[8 * i + 2 * q + 1]) * inv)) << 16;
              dst[i] = make_uint4(y[0], y[1], y[2], y[3]);
            }
          } else if (r < rows) {
            uint4* dst = reinterpret_cast<uint4*>(part + r * D + 16 * w);
#pragma unroll
            for (int i = 0; i < 4; ++i) dst[i] = make_uint4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
          }
          __syncwarp();  // the next load is warp-wide
        }
        if (r < rows) {
          if (!p.complete()) {
            part[R * D + 2 * r] = top;
            part[R * D + 2 * r + 1] = sum;
          } else if (a.lse) {
            a.lse[at] = attn_lse(top, sum, kHeldExp);
          }
        }
      }
      ++seg;
    }
  }
  tc::fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc::fence_after();
    tc::dealloc<C::kCols>(tmem);
  }
  if (tid == 0 && s_abort) bump(a.stats, SPEC_STAT_WAIT_TIMEOUT);
}

template <int D, int MT>
int launch_tree(AttnArgs a, int sms, cudaStream_t s) {
  using C = TreeCfg<D, MT>;
  constexpr int R = kTreeRows * MT;
  auto kernel = kv4_tree_kernel<D, MT>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(C::kSmem)) !=
      cudaSuccess) {
    cudaGetLastError();
    return SPEC_ERR_CUDA;
  }
  a.ctas = sms * (MT == 2 ? 1 : 2);
  a.ctas = a.ctas < kTreeMaxCtas / MT ? a.ctas : kTreeMaxCtas / MT;
  launch_k(kernel, static_cast<unsigned>(a.ctas), C::kThreads, C::kSmem, s, a);
  launch_merge<D>(a, R, kHeldExp, s);
  return launch_status();
}

}  // namespace

int launch_tree_attention(AttnArgs a, int D, int sms, cudaStream_t s) {
  const bool two = static_cast<int64_t>(a.N) * a.G > kTreeRows;
  if (D == 128) return two ? launch_tree<128, 2>(a, sms, s) : launch_tree<128, 1>(a, sms, s);
  return two ? launch_tree<64, 2>(a, sms, s) : launch_tree<64, 1>(a, sms, s);
}

}  // namespace specdec
