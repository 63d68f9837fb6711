// Attention of the tree's nodes over the 4-bit paged KV cache.
//
// "EAGLE speculative decoding in four parts" (ai-infra-handbooks),
// "Drafting, verification and slots": the target verifies all nodes of a tree
// in one forward under the tree attention mask.  Node n of request b attends
// to every position of the context and, at position seq_len + m, to node m
// where tree_mask[b][n][m] is set (itself and its ancestors):
//   out = sum_p w_p v_p / sum_p w_p,  w_p = 2^(x_p - max x),
//   x_p = (q . k_p) scale log2(e).
// One pass over the cache with a running maximum and sum (fp32).  The codes
// become fp16 values lo + code * step in registers (one rounding, relative
// 2^-11) and feed the tensor cores with fp32 sums; q is scaled by a power of
// two per row so that its largest element lies in [1, 2), which makes its
// fp16 form exact but for elements 2^-14 smaller.  Weights are scaled by 2^15
// before they are rounded to fp16 (relative 2^-12), so that a weight keeps
// its bits down to 2^-29 of the largest; the sum that divides uses the
// unrounded weights.
//
// The rows of a KV head (N nodes times G query heads) are cut into row tiles.
// Three kernels, by the rows: here up to 8 (positions in tiles of 128) and up
// to 16 (tiles of 64) with matrix instructions from registers, each warp with
// its own positions and a ring of asynchronous copies; more rows in
// kv4_tree.cu.  Work is dealt out evenly whatever the
// lengths are: the tiles of all (request, KV head, row tile) segments form
// one line, each CTA takes an equal stretch of it, and a segment that is cut
// between CTAs leaves partial (max, sum, weighted values) in the workspace,
// which a second kernel merges in a fixed order.  The host knows no lengths.
//
// Bound by latency at three warps a scheduler (164 registers hold O and the
// codes at hand), neither by the issue slots (46% in use) nor by the memory: per
// issue 0.9 warps each wait for memory, for shared memory and for the
// instruction before, and 0.6 for the CTA's other warps, which meet five times
// a segment of nine tiles on average.  960 instructions a warp and 32 positions
// of 8 rows, 536 of them unpacking.  Measured at D = 128, 8 KV heads: B=128, 32
// heads, contexts 16..2048: 80 us for 172 MB (227 MB from DRAM: the 160 bytes
// of a head touch three 64-byte pieces, and other CTAs read the neighbours at
// other times); B=4, 64 heads, contexts 60001..131001: 153 us for 491 MB.
//
// With a sliding window and sinks (WIN) the same kernels walk places instead of
// positions: the sinks and, behind a gap, what the root's window shows, so work
// and reads follow the window and not the context, and slots in the gap are not
// looked up.  Rows of deeper nodes hide the window's first positions, in the one
// or two tiles where that happens.  Measured at D = 128, 8 KV heads, 32 heads,
// B=128, contexts 16..8192, window 2048 and 4 sinks: 109 us for 297 MB (471 MB
// from DRAM, 4.4 TB/s; issue slots 48% in use): as above.
#include "kv4_attn.cuh"

namespace specdec {
namespace {

constexpr int kTile = 64;        // positions of a tile: 16 per warp
constexpr int kEnds = 2;         // tiles that a segment's beginning and end cost
// Of four times 32 positions.  With a window the segments are short and alike,
// and nearly all CTAs cut one (8 KV heads, B=128, window 2048: 116 us with 1,
// 109 with 2, 111 with 4).
template <bool WIN>
constexpr int kEnds8 = WIN ? 2 : 1;
constexpr int kAttThreads = 128;
constexpr int kAttWarps = kAttThreads / 32;
constexpr float kWeightExp = 15.0f;  // weights are held times 2^15

template <int BYTES>
struct Vec;
template <>
struct Vec<16> {
  using type = uint4;
};
template <>
struct Vec<8> {
  using type = uint2;
};
template <>
struct Vec<4> {
  using type = uint32_t;
};

__device__ __forceinline__ uint32_t word_of(const uint4& v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}
__device__ __forceinline__ uint32_t word_of(const uint2& v, int i) { return i == 0 ? v.x : v.y; }
__device__ __forceinline__ uint32_t word_of(uint32_t v, int) { return v; }

// A warp's P positions of a tile in shared memory: a stage of a ring that
// only this warp fills (asynchronous copies of 16 bytes, a position's bytes by
// neighbouring lanes) and reads.  With t = lane % 4 and g = lane / 4 a lane
// reads, of positions g and g + 8, the D/4 channels of K from t D/4 on (its
// share of the B fragments of q k^T, whose order of channels is free), and of
// positions 2t, 2t + 1, 2t + 8, 2t + 9 the D/8 channels of V from g D/8 on (its
// share of the B fragments of w v: channel g D/8 + i is column g of block i).
// K's codes lie 16 words a position apart and V's with their (step, lo) 20
// (D = 64: 8 and 12), which makes every read free of bank conflicts.
template <int D, int P>
struct Stage {
  static constexpr int kVRow = D == 128 ? 80 : 48;              // D = 64: with K's (step, lo) too
  static constexpr int kKMeta = P * 64;                         // D = 128 only
  static constexpr int kV = D == 128 ? P * 80 : P * 32;         // V's first byte
  static constexpr int kBytes = P * kv4_head_bytes(D);
  // A lane's share of one position: K's codes and (step, lo), V's.
  __device__ __forceinline__ static void k(const uint8_t* s, int pos, int t, typename Vec<D / 8>::type& c,
                                           uint32_t& m) {
    c = *reinterpret_cast<const typename Vec<D / 8>::type*>(s + pos * (D / 2) + t * (D / 8));
    m = *reinterpret_cast<const uint32_t*>(
        s + (D == 128 ? kKMeta + pos * 16 + t * 4 : kV + pos * kVRow + D / 2 + (t >> 1) * 4));
  }
  __device__ __forceinline__ static void v(const uint8_t* s, int pos, int g, typename Vec<D / 16>::type& c,
                                           uint32_t& m) {
    const uint8_t* row = s + kV + pos * kVRow;
    c = *reinterpret_cast<const typename Vec<D / 16>::type*>(row + g * (D / 16));
    m = *reinterpret_cast<const uint32_t*>(row + (D == 128 ? 64 + (g >> 1) * 4 : 40 + (g >> 2) * 4));
  }
};

// A warp's ring of RING stages and the cursor that fills it, across segments:
// slots RING + 1 tiles before their use, codes RING.  A tile is 4 P positions,
// P for each of four warps.  A pair of lanes copies a position's 32-byte
// sectors (one instruction: 16 positions), so the addresses are two shuffles a
// 16 positions and constants.
template <int D, int P, int RING, int E, int R, bool WIN>
struct Filler {
  using St = Stage<D, P>;
  static constexpr int kTile = 4 * P;
  Walk<kTile, E, R, WIN> ahead;
  Part ap;
  bool more, loaded;
  int next_tile;
  int32_t slot;  // of position lane % P of the warp's; -2: no position
  const uint8_t* head;
  const int32_t* row;  // the request's slots from this lane's place of tile 0 on
  unsigned ring;
  unsigned* there;  // [RING]: positions of a stage that have a slot

  __device__ __forceinline__ void segment(const AttnArgs& a) {
    next_tile = ap.t0;
    head = a.pool + ap.h * kv4_head_bytes(D);
    row = a.table + static_cast<int64_t>(ap.b) * a.max_ctx + (threadIdx.x >> 5) * P + (threadIdx.x & (P - 1));
  }
  __device__ __forceinline__ void begin(const AttnArgs& a, const Walk<kTile, E, R, WIN>& walk, uint8_t* stages,
                                        unsigned* t) {
    ahead = walk;
    more = ahead.next(a, ap);
    segment(a);
    ring = static_cast<unsigned>(__cvta_generic_to_shared(stages));
    there = t;
    load_slot();
#pragma unroll 1
    for (int i = 0; i < RING - 1; ++i) {
      copy(a, i);
      load_slot();
    }
  }
  __device__ __forceinline__ void load_slot() {
    loaded = more;
    if (!more) return;
    const int pos = next_tile * kTile + static_cast<int>((threadIdx.x >> 5) * P + (threadIdx.x & (P - 1)));
    slot = pos < ap.end && spec_in(pos, ap.end, nullptr)
               ? __ldg(row + next_tile * kTile + (WIN && pos >= ap.cut ? ap.gap : 0))
               : -2;
    ++next_tile;
  }
  // Copies the tile whose slots were loaded last; one commit group, empty
  // behind the line's end.
  __device__ __forceinline__ void copy(const AttnArgs& a, int st) {
    if (loaded) {
      const int lane = threadIdx.x & 31, b = lane & 1;
      const bool ok = slot >= 0 && slot < a.num_slots;
      if (!ok && slot != -2 && ap.h == 0 && ap.rt == 0 && lane < P) bump(a.stats, SPEC_STAT_BAD_REQUEST);
      const unsigned have = __ballot_sync(0xffffffffu, ok) & (0xffffffffu >> (32 - P));
      if (lane == 0) there[st] = have;
      const uint64_t mine = reinterpret_cast<uint64_t>(head) +
                            static_cast<uint64_t>(ok ? slot : 0) * static_cast<uint32_t>(a.slot_stride);
#pragma unroll
      for (int u = 0; u < P / 16; ++u) {
        const int pos = u * 16 + (lane >> 1);
        const uint64_t src = __shfl_sync(0xffffffffu, mine, pos) + b * 16;
        // a position without a slot is zeroed: its weights are zero, its values must not be NaN
        const unsigned size = (have >> pos) & 1u ? 16u : 0u;
        const unsigned k = ring + st * St::kBytes + pos * (D / 2) + b * 16;
        const unsigned v = ring + st * St::kBytes + St::kV + pos * St::kVRow + b * 16;
        constexpr int kk = D / 64;  // sectors of K's codes, and of V's
#pragma unroll
        for (int i = 0; i < kk; ++i) {
          put(k + 32 * i, src + 32 * i, size);
          put(v + 32 * i, src + D / 2 + 32 * i, size);
        }
        if (D == 128) put(b ? v - 16 + 64 : ring + st * St::kBytes + St::kKMeta + pos * 16, src + 128, size);
        else if (b == 0) put(v + 32, src + 64, size);
      }
    }
    if (more && next_tile == ap.t1) {
      more = ahead.next(a, ap);
      segment(a);
    }
    cp_async_commit();
  }
  __device__ __forceinline__ static void put(unsigned dst, uint64_t src, unsigned size) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(size) : "memory");
  }
  // The next tile into the stage that was read last, then the wait for stage
  // `st`; returns its positions.
  __device__ __forceinline__ unsigned turn(const AttnArgs& a, int st) {
    __syncwarp();  // every lane has read the stage before
    copy(a, (st + RING - 1) % RING);
    load_slot();
    cp_async_wait<RING - 1>();
    __syncwarp();  // every lane's copies of this tile have landed
    return there[st];
  }
};

constexpr int kRing = 4;     // stages of a warp, of 16 positions
constexpr int kRing8 = 3;    // and of 32, with up to eight rows

// Shared memory of a CTA: the warps' rings, q in the order of the A fragments,
// the warps' row statistics, and the weighted values of two warps' 16 rows at
// a time (rows 16 floats longer than D and 4 floats of padding per 32
// channels, so the fragment's stores spread over the banks).
template <int D>
struct AttShared {
  static constexpr int kRow = D + 16;
  uint8_t ring[kAttWarps][kRing][Stage<D, 16>::kBytes];
  uint4 q[D / 16][32];
  float c[16];  // factor of a row's scores
  float m[kAttWarps][16], l[kAttWarps][16];
  unsigned there[kAttWarps][kRing];  // positions of a stage that have a slot
  float o[2][16][kRow];
};

__device__ __forceinline__ int padded(int ch) { return ch + (ch >> 5) * 4; }

// Row r of (b, h) of q (zeros when !in), D / 32 channels a lane from lane D/32
// on, and its largest magnitude.
template <int D>
__device__ __forceinline__ void q_row(const AttnArgs& a, int b, int h, int r, bool in, float* x, float& mx) {
  constexpr int per = D / 32;
  const int lane = threadIdx.x & 31;
  uint32_t w[per / 2];
#pragma unroll
  for (int j = 0; j < per / 2; ++j) w[j] = 0;
  if (in) {
    const uint16_t* src = a.q + attn_q(a, b, h, r, D) + lane * per;
    if (per == 4) {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(src));
      w[0] = v.x;
      w[per / 2 - 1] = v.y;
    } else {
      w[0] = __ldg(reinterpret_cast<const uint32_t*>(src));
    }
  }
  mx = 0.0f;
#pragma unroll
  for (int j = 0; j < per; ++j) {
    x[j] = j & 1 ? bf16_hi(w[j / 2]) : bf16_lo(w[j / 2]);
    mx = fmaxf(mx, fabsf(x[j]));
  }
  mx = warp_max(mx);
}
// The power of two that brings mx into [1, 2) (1 for zeros, infinities and NaN;
// 2^126 at most and 2^-126 at least, which leaves the largest mx below 4); the
// row's scores are multiplied by *factor.
__device__ __forceinline__ float q_scale(float mx, float scale_log2, float* factor) {
  const int bits = static_cast<int>(__float_as_uint(mx) >> 23);
  const int e = mx > 0.0f && isfinite(mx) ? min(max(bits - 127, -126), 126) : 0;
  if ((threadIdx.x & 31) == 0) *factor = scale_log2 * __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
  return __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
}

// Query rows [r0, r0 + 16) of (b, h) into shared memory: a warp per row.
template <int D>
__device__ void load_q(const AttnArgs& a, AttShared<D>& sh, int b, int h, int r0, int rows) {
  constexpr int per = D / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll 4
  for (int r = warp; r < 16; r += kAttWarps) {
    float x[per], mx;
    q_row<D>(a, b, h, r0 + r, r < rows, x, mx);
    const float down = q_scale(mx, a.scale_log2, sh.c + r);
    // channel ch = t D/4 + 4 kk + 2 i + odd: A register 2 i + (row half) of
    // lane 4 (row % 8) + t at step kk
#pragma unroll
    for (int j = 0; j < per; j += 2) {
      const int ch = lane * per + j, t = ch / (D / 4), kk = ch % (D / 4) / 4, i = ch % 4 / 2;
      reinterpret_cast<uint32_t*>(&sh.q[kk][(r % 8) * 4 + t])[2 * i + (r % 16) / 8] =
          h2_u32(__floats2half2_rn(x[j] * down, x[j + 1] * down));
    }
  }
}

// In a tile with nodes: (step, lo) of four positions of V, zero where no append
// can have written them.
__device__ __forceinline__ void drop_unwritten(uint32_t& st0, uint32_t& lo0, uint32_t& st1, uint32_t& lo1) {
  const uint32_t k0 = finite_values(st0, lo0), k1 = finite_values(st1, lo1);
  st0 &= k0, lo0 &= k0;
  st1 &= k1, lo1 &= k1;
}

// Row r's maximum and sum of weights over the warps.  A warp without a maximum
// has a sum of zero, or NaN where q has one (its scores have no maximum): it
// counts as it is.
template <int R>
__device__ __forceinline__ void warps_sum(const float (&m)[kAttWarps][R], const float (&l)[kAttWarps][R], int r,
                                          float& top, float& sum) {
  top = m[0][r];
#pragma unroll
  for (int w = 1; w < kAttWarps; ++w) top = fmaxf(top, m[w][r]);
  sum = 0.0f;
#pragma unroll
  for (int w = 0; w < kAttWarps; ++w) sum += l[w][r] * (m[w][r] == neg_inf() ? 1.0f : fast_exp2(m[w][r] - top));
}

// Four channels of a row's weighted values: the result, or this CTA's partial.
template <int D>
__device__ __forceinline__ void attn_store(const AttnArgs& a, const Part& p, int r, int R, int ch, const float4& acc,
                                           float top, float sum, float* part) {
  if (!p.complete()) {
    const int rr = r - p.rt * R;
    *reinterpret_cast<float4*>(part + rr * D + ch) = acc;
    if (ch == 0) {
      part[R * D + 2 * rr] = top;
      part[R * D + 2 * rr + 1] = sum;
    }
    return;
  }
  const float inv = attn_inv(sum);
  const int64_t at = attn_row(a, p.b, p.h, r);
  uint2 v;
  v.x = f_bf16(acc.x * inv) | static_cast<uint32_t>(f_bf16(acc.y * inv)) << 16;
  v.y = f_bf16(acc.z * inv) | static_cast<uint32_t>(f_bf16(acc.w * inv)) << 16;
  *reinterpret_cast<uint2*>(a.out + at * D + ch) = v;
  if (a.lse && ch == 0) a.lse[at] = attn_lse(top, sum, kWeightExp);
}

template <int D, bool WIN>
__global__ void __launch_bounds__(kAttThreads, 3) kv4_attention_kernel(const AttnArgs a) {
  pdl_enter();
  constexpr int R = 16, H = 2;  // halves of a fragment's rows
  using St = Stage<D, 16>;
  extern __shared__ __align__(16) unsigned char att_sm[];
  AttShared<D>& sh = *reinterpret_cast<AttShared<D>*>(att_sm);
  if (!spec_smem_ok(sizeof(sh), a.stats)) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, t = lane & 3, g = lane >> 2;
  CutSegment* cut = reinterpret_cast<CutSegment*>(a.ws) + blockIdx.x;
  if (threadIdx.x == 0) *cut = CutSegment{0, 0, 0, 0};
  Line line;
  Walk<kTile, kEnds, R, WIN> walk;
  if (!attn_stretch<kAttThreads>(a, line, walk)) return;

  Filler<D, 16, kRing, kEnds, R, WIN> fill;
  fill.begin(a, walk, sh.ring[warp][0], sh.there[warp]);
  int st = 0;  // stage of the tile at hand

  Part rq;
#pragma unroll 1
  while (walk.next(a, rq)) {
    const int b = rq.b, h = rq.h, rt = rq.rt, t0 = rq.t0, t1 = rq.t1;
    const int r0 = rt * R, rows = min(R, rq.nodes * a.G - r0);
    if (rq.bad && h == 0 && rt == 0 && threadIdx.x == 0) bump(a.stats, SPEC_STAT_BAD_REQUEST);

    load_q<D>(a, sh, b, h, r0, rows);
    __syncthreads();
    float cr[H], m[H], l[H], o[D / 8][4];
#pragma unroll
    for (int i = 0; i < H; ++i) {
      cr[i] = sh.c[g + 8 * i];
      m[i] = neg_inf();
      l[i] = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[i][j] = 0.0f;

#pragma unroll 1
    for (int tile = t0; tile < t1; ++tile) {
      const unsigned there = fill.turn(a, st);
      const uint8_t* s8 = sh.ring[warp][st];
      st = (st + 1) % kRing;
      if (there == 0) continue;
      float s[2][4];
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[j][i] = 0.0f;
      typename Vec<D / 8>::type kc[2];
      uint32_t km[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) St::k(s8, g + 8 * j, t, kc[j], km[j]);
#pragma unroll
      for (int wd = 0; wd < D / 32; ++wd) {  // words of 8 channels: two steps of 16 (4 channels a lane)
        uint32_t kv[2][4];
#pragma unroll
        for (int j = 0; j < 2; ++j)
          dequant4(word_of(kc[j], wd), __byte_perm(km[j], 0, 0x1010), __byte_perm(km[j], 0, 0x3232), kv[j]);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const uint4 qa = sh.q[wd * 2 + half][lane];
#pragma unroll
          for (int j = 0; j < 2; ++j) mma16816(s[j], qa, kv[j][2 * half], kv[j][2 * half + 1]);
        }
      }
      // scores in units of log2, masked; s[j][i]: row g + 8 (i / 2),
      // position 8 j + 2 t + i % 2
      const int p0 = tile * kTile + warp * 16;
      const bool whole = there == 0xffffu && attn_context<WIN>(a, rq, p0, p0 + 16);
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < 2 * H; ++i) s[j][i] *= cr[i >> 1];
      if (!whole) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int i = 0; i < 2 * H; ++i) {
            const int at = 8 * j + 2 * t + (i & 1), r = g + 8 * (i >> 1);
            bool see = (there >> at) & 1u;
            if (see && (WIN || p0 + at >= rq.start))
              see = r < rows && attn_sees<WIN>(a, rq, attn_node(a, r0 + r), p0 + at);
            if (!see) s[j][i] = neg_inf();
          }
      }
      float mn[H], al[H];
      bool up = false;
#pragma unroll
      for (int i = 0; i < H; ++i) {
        float x = fmaxf(fmaxf(s[0][2 * i], s[0][2 * i + 1]), fmaxf(s[1][2 * i], s[1][2 * i + 1]));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
        mn[i] = fmaxf(m[i], x);
        up = up || mn[i] != m[i];
        const float base_m = mn[i] == neg_inf() ? 0.0f : mn[i];
        al[i] = fast_exp2(m[i] - base_m);
        m[i] = mn[i];
        mn[i] = weight_base(base_m, kWeightExp);
      }
      if (__any_sync(0xffffffffu, up)) {
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
#pragma unroll
          for (int e = 0; e < 2 * H; ++e) o[i][e] *= al[e >> 1];
#pragma unroll
        for (int i = 0; i < H; ++i) l[i] *= al[i];
      }
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < 2 * H; ++i) {
          s[j][i] = fast_exp2(s[j][i] - mn[i >> 1]);
          l[i >> 1] += s[j][i];
        }
      const uint4 pa =
          make_uint4(h2_u32(__floats2half2_rn(s[0][0], s[0][1])), h2_u32(__floats2half2_rn(s[0][2], s[0][3])),
                     h2_u32(__floats2half2_rn(s[1][0], s[1][1])), h2_u32(__floats2half2_rn(s[1][2], s[1][3])));
      typename Vec<D / 16>::type vc[4];
      uint32_t vm[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) St::v(s8, 2 * t + (j & 1) + 8 * (j >> 1), g, vc[j], vm[j]);
      uint32_t st0 = __byte_perm(vm[0], vm[1], 0x5410), lo0 = __byte_perm(vm[0], vm[1], 0x7632);
      uint32_t st1 = __byte_perm(vm[2], vm[3], 0x5410), lo1 = __byte_perm(vm[2], vm[3], 0x7632);
      if (!whole) drop_unwritten(st0, lo0, st1, lo1);
#pragma unroll
      for (int wd = 0; wd < D / 64; ++wd) {
        // even channels of a word lie in its low half, odd ones in its high
        // half: the pair of positions of a channel is a byte permutation away
#pragma unroll
        for (int odd = 0; odd < 2; ++odd) {
          const uint32_t sel = odd ? 0x7632u : 0x5410u;
          uint32_t v0[4], v1[4];
          dequant4(__byte_perm(word_of(vc[0], wd), word_of(vc[1], wd), sel), st0, lo0, v0);
          dequant4(__byte_perm(word_of(vc[2], wd), word_of(vc[3], wd), sel), st1, lo1, v1);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            mma16816(o[wd * 8 + 2 * j + odd], pa, v0[j], v1[j]);
        }
      }
    }

    // merge the warps: 2 and 3 hand their values to 0 and 1, then 1 to 0's place
    float* part = attn_part(a, blockIdx.x, t0 > 0 ? 0 : 1, R, D);
    if (t0 == 0 && t1 < rq.tiles && threadIdx.x == 0)
      *cut = CutSegment{b, h, rt, line.pieces(static_cast<int>(blockIdx.x), rq.tiles, t1)};
#pragma unroll
    for (int i = 0; i < H; ++i) {
      float x = l[i];
      x += __shfl_xor_sync(0xffffffffu, x, 1);
      x += __shfl_xor_sync(0xffffffffu, x, 2);
      if (t == 0) {
        sh.m[warp][g + 8 * i] = m[i];
        sh.l[warp][g + 8 * i] = x;
      }
    }
    __syncthreads();
    float f[H];
#pragma unroll
    for (int i = 0; i < H; ++i) {
      const int r = g + 8 * i;
      float top = sh.m[0][r];
#pragma unroll
      for (int w = 1; w < kAttWarps; ++w) top = fmaxf(top, sh.m[w][r]);
      f[i] = m[i] == neg_inf() ? 0.0f : fast_exp2(m[i] - top);
    }
#pragma unroll
    for (int stage = 0; stage < 2; ++stage) {
      // stage 0: warps 2 and 3 store; stage 1: warps 0 and 1 add
      if ((stage == 0) == (warp >= 2)) {
#pragma unroll
        for (int i = 0; i < H; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int c = 0; c < D / 8; c += 4) {
              const int ch = (2 * t + e) * (D / 8) + c;
              float4* at = reinterpret_cast<float4*>(&sh.o[warp & 1][g + 8 * i][padded(ch)]);
              float4 x = make_float4(o[c][2 * i + e] * f[i], o[c + 1][2 * i + e] * f[i],
                                     o[c + 2][2 * i + e] * f[i], o[c + 3][2 * i + e] * f[i]);
              if (stage == 1) {
                const float4 y = *at;
                x = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
              }
              *at = x;
            }
      }
      __syncthreads();
    }
    for (int i = threadIdx.x; i < 8 * H * (D / 4); i += kAttThreads) {
      const int r = i / (D / 4), ch = (i - r * (D / 4)) * 4;
      if (r >= rows) continue;
      const float4 x = *reinterpret_cast<const float4*>(&sh.o[0][r][padded(ch)]);
      const float4 y = *reinterpret_cast<const float4*>(&sh.o[1][r][padded(ch)]);
      const float4 acc = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
      float top, sum;
      warps_sum(sh.m, sh.l, r, top, sum);
      attn_store<D>(a, rq, r0 + r, R, ch, acc, top, sum, part);
    }
    __syncthreads();
  }
  cp_async_wait<0>();
}

// Up to eight rows (single tokens of up to eight query heads a KV head).  The
// products are taken transposed: S^T = K Q^T and O^T = V^T P^T with positions
// and channels as the 16 rows of a fragment and the eight query rows as its
// columns, half the matrix instructions and half the registers of O.  The same
// lanes' registers serve: K's B fragments of two position blocks are the A
// fragment of 16 positions, V's of two channel blocks that of 16 channels.  The
// weights (position g, rows 2t, 2t + 1) become the B fragment (positions 2t,
// 2t + 1, row g) by one 8 x 8 transposition a block (movmatrix).  A warp takes
// 32 positions at a time: what a tile costs beside the unpacking (the slots,
// the copies' addresses, the maximum) is shared by more positions.  The most of
// its instructions unpack the codes: 26 a position and lane of 128 channels.
template <int D>
struct AttShared8 {
  static constexpr int kRow = D + 4;
  uint8_t ring[kAttWarps][kRing8][Stage<D, 32>::kBytes];
  uint2 q[D / 16][32];
  float c[8];
  float m[kAttWarps][8], l[kAttWarps][8];
  unsigned there[kAttWarps][kRing8];
  float o[2][8][kRow];
};

__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

template <int D, bool WIN>
__global__ void __launch_bounds__(kAttThreads, 3) kv4_attention8_kernel(const AttnArgs a) {
  pdl_enter();
  constexpr int R = 8, T = 4 * 32;
  using St = Stage<D, 32>;
  extern __shared__ __align__(16) unsigned char att_sm[];
  AttShared8<D>& sh = *reinterpret_cast<AttShared8<D>*>(att_sm);
  if (!spec_smem_ok(sizeof(sh), a.stats)) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, t = lane & 3, g = lane >> 2;
  CutSegment* cut = reinterpret_cast<CutSegment*>(a.ws) + blockIdx.x;
  if (threadIdx.x == 0) *cut = CutSegment{0, 0, 0, 0};
  Line line;
  Walk<T, kEnds8<WIN>, R, WIN> walk;
  if (!attn_stretch<kAttThreads>(a, line, walk)) return;
  Filler<D, 32, kRing8, kEnds8<WIN>, R, WIN> fill;
  fill.begin(a, walk, sh.ring[warp][0], sh.there[warp]);
  int st = 0;  // stage of the tile at hand

  Part rq;
#pragma unroll 1
  while (walk.next(a, rq)) {
    const int b = rq.b, h = rq.h, t0 = rq.t0, t1 = rq.t1;
    const int rows = min(R, rq.nodes * a.G);
    if (rq.bad && h == 0 && threadIdx.x == 0) bump(a.stats, SPEC_STAT_BAD_REQUEST);
    // a warp's two rows of q: channel ch = t D/4 + 4 kk + 2 i + odd is B
    // register i of lane 4 row + t at step kk
#pragma unroll
    for (int rr = 0; rr < 2; ++rr) {
      const int r = warp * 2 + rr;
      float mx;
      constexpr int per = D / 32;
      float x[per];
      q_row<D>(a, b, h, r, r < rows, x, mx);
      const float down = q_scale(mx, a.scale_log2, sh.c + r);
#pragma unroll
      for (int j = 0; j < per; j += 2) {
        const int ch = lane * per + j, tt = ch / (D / 4), kk = ch % (D / 4) / 4, i = ch % 4 / 2;
        reinterpret_cast<uint32_t*>(&sh.q[kk][r * 4 + tt])[i] = h2_u32(__floats2half2_rn(x[j] * down, x[j + 1] * down));
      }
    }
    __syncthreads();
    float cr[2], m[2], l[2], o[D / 16][4];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      cr[e] = sh.c[2 * t + e];
      m[e] = neg_inf();
      l[e] = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[i][j] = 0.0f;

#pragma unroll 1
    for (int tile = t0; tile < t1; ++tile) {
      const unsigned there = fill.turn(a, st);
      const uint8_t* s8 = sh.ring[warp][st];
      st = (st + 1) % kRing8;
      if (there == 0) continue;
      // s[u][2 i + e]: position 16 u + g + 8 i, row 2 t + e
      float s[2][4];
      typename Vec<D / 8>::type kc[2][2];
      uint32_t km[2][2];
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          St::k(s8, 16 * u + g + 8 * j, t, kc[u][j], km[u][j]);
          s[u][2 * j] = s[u][2 * j + 1] = 0.0f;
        }
#pragma unroll
      for (int wd = 0; wd < D / 32; ++wd) {
        const uint2 q0 = sh.q[wd * 2][lane], q1 = sh.q[wd * 2 + 1][lane];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          uint32_t kv[2][4];
#pragma unroll
          for (int j = 0; j < 2; ++j)
            dequant4(word_of(kc[u][j], wd), __byte_perm(km[u][j], 0, 0x1010), __byte_perm(km[u][j], 0, 0x3232), kv[j]);
          mma16816(s[u], make_uint4(kv[0][0], kv[1][0], kv[0][1], kv[1][1]), q0.x, q0.y);
          mma16816(s[u], make_uint4(kv[0][2], kv[1][2], kv[0][3], kv[1][3]), q1.x, q1.y);
        }
      }
      const int p0 = tile * T + warp * 32;
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[u][i] *= cr[i & 1];
      const bool whole = there == 0xffffffffu && attn_context<WIN>(a, rq, p0, p0 + 32);
      if (!whole) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int at = 16 * u + g + 8 * (i >> 1), r = 2 * t + (i & 1);
            bool see = (there >> at) & 1u;
            if (see && (WIN || p0 + at >= rq.start)) see = r < rows && attn_sees<WIN>(a, rq, attn_node(a, r), p0 + at);
            if (!see) s[u][i] = neg_inf();
          }
      }
      float mn[2], al[2];
      bool up = false;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x = fmaxf(fmaxf(s[0][e], s[0][2 + e]), fmaxf(s[1][e], s[1][2 + e]));
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, off));
        mn[e] = fmaxf(m[e], x);
        up = up || mn[e] != m[e];
        const float base_m = mn[e] == neg_inf() ? 0.0f : mn[e];
        al[e] = fast_exp2(m[e] - base_m);
        m[e] = mn[e];
        mn[e] = weight_base(base_m, kWeightExp);
      }
      if (__any_sync(0xffffffffu, up)) {
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) o[i][j] *= al[j & 1];
        l[0] *= al[0];
        l[1] *= al[1];
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s[u][i] = fast_exp2(s[u][i] - mn[i & 1]);
          l[i & 1] += s[u][i];
        }
        const uint32_t p_lo = transpose8(h2_u32(__floats2half2_rn(s[u][0], s[u][1])));
        const uint32_t p_hi = transpose8(h2_u32(__floats2half2_rn(s[u][2], s[u][3])));
        typename Vec<D / 16>::type vc[4];
        uint32_t vm[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) St::v(s8, 16 * u + 2 * t + (j & 1) + 8 * (j >> 1), g, vc[j], vm[j]);
        uint32_t st0 = __byte_perm(vm[0], vm[1], 0x5410), lo0 = __byte_perm(vm[0], vm[1], 0x7632);
        uint32_t st1 = __byte_perm(vm[2], vm[3], 0x5410), lo1 = __byte_perm(vm[2], vm[3], 0x7632);
        if (!whole) drop_unwritten(st0, lo0, st1, lo1);
#pragma unroll
        for (int wd = 0; wd < D / 64; ++wd) {
          uint32_t v[2][2][4];  // odd channel, upper positions, pair of channels
#pragma unroll
          for (int odd = 0; odd < 2; ++odd) {
            const uint32_t sel = odd ? 0x7632u : 0x5410u;
            dequant4(__byte_perm(word_of(vc[0], wd), word_of(vc[1], wd), sel), st0, lo0, v[odd][0]);
            dequant4(__byte_perm(word_of(vc[2], wd), word_of(vc[3], wd), sel), st1, lo1, v[odd][1]);
          }
#pragma unroll
          for (int j = 0; j < 4; ++j)  // channels g D/8 + 8 wd + 2 j (o[..][0, 1]) and the next (o[..][2, 3])
            mma16816(o[wd * 4 + j], make_uint4(v[0][0][j], v[1][0][j], v[0][1][j], v[1][1][j]), p_lo, p_hi);
        }
      }
    }

    // merge the warps: 2 and 3 store, 0 and 1 add, then all sum the two
    float* part = attn_part(a, blockIdx.x, t0 > 0 ? 0 : 1, R, D);
    if (t0 == 0 && t1 < rq.tiles && threadIdx.x == 0)
      *cut = CutSegment{b, h, 0, line.pieces(static_cast<int>(blockIdx.x), rq.tiles, t1)};
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float x = l[e];
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
      if (g == 0) {
        sh.m[warp][2 * t + e] = m[e];
        sh.l[warp][2 * t + e] = x;
      }
    }
    __syncthreads();
    float f[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float top = sh.m[0][2 * t + e];
#pragma unroll
      for (int w = 1; w < kAttWarps; ++w) top = fmaxf(top, sh.m[w][2 * t + e]);
      f[e] = m[e] == neg_inf() ? 0.0f : fast_exp2(m[e] - top);
    }
#pragma unroll
    for (int stage = 0; stage < 2; ++stage) {
      if ((stage == 0) == (warp >= 2)) {
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int i = 0; i < D / 16; i += 2) {
            float4* at = reinterpret_cast<float4*>(&sh.o[warp & 1][2 * t + e][g * (D / 8) + 2 * i]);
            float4 x = make_float4(o[i][e] * f[e], o[i][2 + e] * f[e], o[i + 1][e] * f[e], o[i + 1][2 + e] * f[e]);
            if (stage == 1) {
              const float4 y = *at;
              x = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
            }
            *at = x;
          }
      }
      __syncthreads();
    }
    for (int i = threadIdx.x; i < rows * (D / 4); i += kAttThreads) {
      const int r = i / (D / 4), ch = (i - r * (D / 4)) * 4;
      const float4 x = *reinterpret_cast<const float4*>(&sh.o[0][r][ch]);
      const float4 y = *reinterpret_cast<const float4*>(&sh.o[1][r][ch]);
      const float4 acc = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
      float top, sum;
      warps_sum(sh.m, sh.l, r, top, sum);
      attn_store<D>(a, rq, r, R, ch, acc, top, sum, part);
    }
    __syncthreads();
  }
  cp_async_wait<0>();
}

template <auto KERNEL, int D, int R>
int launch_rows(AttnArgs& a, size_t smem, int ctas, cudaStream_t s) {
  if (!allow_smem<KERNEL>(smem)) return SPEC_ERR_CUDA;
  a.ctas = ctas < kMaxCtas ? ctas : kMaxCtas;
  launch_k(KERNEL, static_cast<unsigned>(a.ctas), kAttThreads, smem, s, a);
  launch_merge<D>(a, R, kWeightExp, s);
  return launch_status();
}

template <int D, bool WIN>
int launch_few(AttnArgs& a, int R, int sms, cudaStream_t s) {
  if (R == 8) return launch_rows<kv4_attention8_kernel<D, WIN>, D, 8>(a, sizeof(AttShared8<D>), sms * 3, s);
  return launch_rows<kv4_attention_kernel<D, WIN>, D, 16>(a, sizeof(AttShared<D>), sms * 3, s);
}

// Rows of a row tile here: 8 or 16 where they suffice; 0: more rows than that
// go to the tensor-memory kernel (kv4_tree.cu), whose time hardly depends on
// them.  8 KV heads, contexts 16..2048 (B=1: 777), in us, as row tiles of 8 /
// of 16 / in kv4_tree.cu:
//            D=128                                    D=64
//            B=1            B=8            B=128      B=1            B=8            B=128
//   1 row    8.4/9.7/15.0   14.2/14.8/22.9 73/128/137 7.2/8.6/13.1   10.8/11.6/19.7 60/59/99
//   4 rows   8.8/10.5/15.6  15.0/15.8/23.4 77/127/138 7.9/9.9/13.8   12.2/12.9/20.8 63/60/99
//   8 rows   9.6/11.5/16.3  16.3/17.1/23.9 79/127/139 8.6/11.2/14.7  13.8/14.7/21.8 64/66/99
//   12 rows    -/11.8/16.4    -/17.3/24.1   -/136/140   -/11.9/14.8    -/15.1/22.0   -/76/100
//   16 rows    -/12.3/16.4    -/17.8/24.2   -/138/141   -/12.1/14.8    -/15.3/22.1   -/82/100
//   24 rows    -/12.8/16.9    -/24.6/25.0   -/258/143   -/12.4/15.3    -/17.4/22.7   -/140/101
//   32 rows    -/13.0/17.1    -/25.7/25.4   -/261/144   -/12.7/15.4    -/18.3/22.9   -/153/101
// Few requests of 17 to 48 rows would do better with several row tiles of 16
// (the first row tile's codes are then in the L2 cache for the next); the host
// knows B but not the lengths that decide it, so the rule looks at rows alone.
int rows_of(int64_t rows) { return rows <= 8 ? 8 : (rows <= 16 ? 16 : 0); }

// With a window the host knows how many places a row sees at most: calls of more
// than 16 rows whose row tiles of 16 fit in few tiles go to the kernel of 16, whose
// segments cost less to begin and end (a window that shows the whole table takes
// the kernel that the call without one takes).  In us, in kv4_tree.cu / here, by
// tiles:
//   D=128  552: 23.3/18.1   1081: 22.5/17.4   2073: 24.6/25.1   4416: 65/88
//   D=64   811: 19.8/13.5   4264: 30.3/27.5   6490: 33.4/38.2
// One limit for both, where D=128 turns: D=64 would gain a tenth up to some 5000.
constexpr int64_t kFewTiles = 2000;
bool few_tiles(int B, int N, int Hkv, int64_t rows, int64_t max_ctx, int sinks, int window) {
  const int64_t places = static_cast<int64_t>(sinks) + window + N;
  const int64_t tiles = (places + kTile - 1) / kTile;
  return places < max_ctx && static_cast<int64_t>(B) * Hkv * ((rows + 15) / 16) * tiles <= kFewTiles;
}

// The upper limits of a call's sizes.
bool attn_sizes(int B, int N, int Hq, int Hkv, int D) {
  return spec_kv4_slot_bytes(Hkv, D) >= 0 && N <= SPEC_MAX_NODES && Hq <= SPEC_KV4_MAX_HEADS * 16 && B <= 65535;
}

// Both entry points; window 0: none.
int attention(int B, int N, int Hq, int Hkv, int D, const void* q, int64_t q_stride, const void* pool,
              int64_t num_slots, int64_t slot_stride, const int32_t* num_nodes, const int32_t* seq_lens,
              const int32_t* positions, const int32_t* req_to_token, int64_t max_ctx, const uint8_t* tree_mask,
              int sinks, int window, float scale, void* out, float* lse, int32_t* stats, void* ws, size_t ws_bytes,
              spec_stream_t stream) {
  if (B < 0 || N < 0 || Hkv < 1 || Hq < 1 || Hq % Hkv != 0 || max_ctx < 1 || num_slots < 1 || !(scale > 0.0f) ||
      !isfinite(scale))
    return SPEC_ERR_INVALID_ARG;
  const int64_t row_bytes = spec_kv4_slot_bytes(Hkv, D);
  if (!attn_sizes(B, N, Hq, Hkv, D)) return SPEC_ERR_UNSUPPORTED;
  // a row's factor, scale log2(e) times a power of two down to 2^-126, must not vanish
  if (scale < 0x1p-20f || scale > 0x1p20f) return SPEC_ERR_UNSUPPORTED;
  if (slot_stride < row_bytes || q_stride < static_cast<int64_t>(Hq) * D) return SPEC_ERR_INVALID_ARG;
  if (slot_stride % 16 != 0 || q_stride % 8 != 0 || num_slots > INT32_MAX || max_ctx > INT32_MAX - 2 * kTile ||
      slot_stride > INT32_MAX)
    return SPEC_ERR_UNSUPPORTED;
  if (B == 0 || N == 0) return SPEC_OK;
  if (!q || !pool || !seq_lens || !req_to_token || !out || !ws) return SPEC_ERR_INVALID_ARG;
  for (const void* p : {q, pool, static_cast<const void*>(out)})
    if ((reinterpret_cast<uintptr_t>(p) & 15) != 0) return SPEC_ERR_UNSUPPORTED;
  if ((reinterpret_cast<uintptr_t>(ws) & 15) != 0) return SPEC_ERR_INVALID_ARG;
  if (ws_bytes < spec_kv4_attention_ws_size(B, N, Hq, Hkv, D)) return SPEC_ERR_WORKSPACE;
  // results are written while other CTAs still read q
  const uintptr_t q0 = reinterpret_cast<uintptr_t>(q), o0 = reinterpret_cast<uintptr_t>(out);
  const int64_t tokens = static_cast<int64_t>(B) * N, wide = static_cast<int64_t>(Hq) * D;
  if (q0 < o0 + 2 * tokens * wide && o0 < q0 + 2 * ((tokens - 1) * q_stride + wide)) return SPEC_ERR_INVALID_ARG;
  const int sms = attn_sms();
  if (sms == 0) {
    cudaGetLastError();
    return SPEC_ERR_CUDA;
  }
  AttnArgs a{static_cast<const uint16_t*>(q), q_stride, B, N, Hq, Hkv, Hq / Hkv,
             ((1ull << 40) + Hq / Hkv - 1) / (Hq / Hkv), static_cast<const uint8_t*>(pool),
             num_slots, slot_stride, req_to_token, max_ctx, seq_lens, num_nodes, tree_mask, positions, sinks, window,
             scale * kLog2e, static_cast<uint16_t*>(out), lse, static_cast<float*>(ws), 0, stats};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int64_t rows = static_cast<int64_t>(N) * a.G;
  int R = rows_of(rows);
  if (R == 0 && window != 0 && few_tiles(B, N, Hkv, rows, max_ctx, sinks, window)) R = 16;
  if (R == 0) return launch_tree_attention(a, D, sms, s);
  if (window != 0) return D == 128 ? launch_few<128, true>(a, R, sms, s) : launch_few<64, true>(a, R, sms, s);
  return D == 128 ? launch_few<128, false>(a, R, sms, s) : launch_few<64, false>(a, R, sms, s);
}

}  // namespace
}  // namespace specdec

using namespace specdec;

extern "C" size_t spec_kv4_attention_ws_size(int B, int N, int Hq, int Hkv, int D) {
  if (B < 1 || N < 1 || Hkv < 1 || Hq < Hkv || Hq % Hkv != 0 || !attn_sizes(B, N, Hq, Hkv, D)) return 0;
  const int64_t rows = static_cast<int64_t>(N) * (Hq / Hkv);
  const int R = rows_of(rows);
  // more than 16 rows may go to the kernel of 16 (few_tiles), which needs less
  static_assert(kMaxCtas * 16 <= kTreeMaxCtas * kTreeRows, "either kernel's partials");
  return align256(R == 0 ? attn_ws_bytes(kTreeMaxCtas, kTreeRows, D) : attn_ws_bytes(kMaxCtas, R, D));
}

extern "C" int spec_kv4_attention(int B, int N, int Hq, int Hkv, int D, const void* q, int64_t q_stride,
                                  const void* pool, int64_t num_slots, int64_t slot_stride,
                                  const int32_t* num_nodes_or_null, const int32_t* seq_lens,
                                  const int32_t* req_to_token, int64_t max_ctx, const uint8_t* tree_mask_or_null,
                                  float scale, void* out, float* lse_or_null, int32_t* stats_or_null, void* ws,
                                  size_t ws_bytes, spec_stream_t stream) {
  return attention(B, N, Hq, Hkv, D, q, q_stride, pool, num_slots, slot_stride, num_nodes_or_null, seq_lens, nullptr,
                   req_to_token, max_ctx, tree_mask_or_null, 0, 0, scale, out, lse_or_null, stats_or_null, ws, ws_bytes,
                   stream);
}

extern "C" int spec_kv4_attention_window(int B, int N, int Hq, int Hkv, int D, const void* q, int64_t q_stride,
                                         const void* pool, int64_t num_slots, int64_t slot_stride,
                                         const int32_t* num_nodes_or_null, const int32_t* seq_lens,
                                         const int32_t* positions_or_null, const int32_t* req_to_token,
                                         int64_t max_ctx, const uint8_t* tree_mask_or_null, int32_t sinks,
                                         int32_t window, float scale, void* out, float* lse_or_null,
                                         int32_t* stats_or_null, void* ws, size_t ws_bytes, spec_stream_t stream) {
  if (sinks < 0 || window < 1) return SPEC_ERR_INVALID_ARG;
  return attention(B, N, Hq, Hkv, D, q, q_stride, pool, num_slots, slot_stride, num_nodes_or_null, seq_lens,
                   positions_or_null, req_to_token, max_ctx, tree_mask_or_null, sinks, window, scale, out, lse_or_null,
                   stats_or_null, ws, ws_bytes, stream);
}
