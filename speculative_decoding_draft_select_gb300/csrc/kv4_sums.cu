// The attention that every cached position has received, summed over the
// committed rows and all query heads:
//   out[p] = prev[p] + sum over rows i and heads h of exp(scale q_ih . k_p - lse_ih)
// for the positions p that row i sees, p <= seq_len + i.  Rows are the nodes of
// the accepted path, whose K compaction has put in order, and lse what their
// attention returned ("EAGLE speculative decoding in four parts",
// ai-infra-handbooks, "Drafting, verification and slots": only the accepted
// path is kept, so only its rows count).  No softmax is left to do: with lse at
// hand every position stands alone, and one pass over K's half of the cache
// rows gives the sums.
//
// K is lo + c step per group of 32 channels, so
//   q . k = sum over groups (step (q . c) + lo sum q).
// The codes c enter the tensor cores as they are: a nibble in an fp16 register's
// lowest bits is the subnormal c 2^-24, four bits higher c 2^-20, both exact, so
// unpacking is a mask (and a shift for every second pair).  q is scaled by a
// power of two per row (and by 2^-4 more where its code lies higher), exact but
// for elements 2^-24 of the row's largest.  Products, sums and the steps are
// fp32; lo times the group's sum of q is one matrix step more, with the sum as
// three fp16 terms (2^-33).  The scores are then as good as fp32 sums.
//
// Positions are the 16 rows of a fragment, query rows its eight columns, so a
// lane sums its positions' weights over columns, row tiles and heads in
// registers.  A CTA takes a stretch of 32-position chunks, cut by their cost; its
// items are (chunk, head) pairs, a chunk's heads one after another (a cache row
// is read from end to end, and its address found once), dealt evenly to the
// warps.  The rows of q are turned into fragments in shared memory once a request,
// every warp fills its own ring of asynchronous copies, and the warps' sums meet
// in shared memory and are added in the warps' order: no atomics.
//
// More than 32 rows a KV head go to kv4_sums_rows.cu, request by request; this
// launch then lays their rows out for it.
//
// Bound by the memory: DRAM delivers whole 128-byte lines, and K's codes and
// (step, lo) of two heads touch all lines of a row, V's half included (180 MB read
// for 87 MB asked at B=128, 32 heads over 8 of 128, contexts 16..2048).  Measured
// there: one token 37 us, of which about 6 are the launch, the lengths' scan and
// the first loads, and the slope over the length is 6.1 TB/s of whole lines;
// accepted paths of 1 to 7 tokens 58 us (63 with the second launch, which finds
// nothing to do), where the second pass over the codes of longer paths shows.
// Before: heads outermost with fragments in registers 48 us (twice the lines,
// since other warps read a row's other heads at other times); chunks dealt out
// evenly instead of by cost 72 us for the paths; four row tiles a pass instead of
// two 63 to 90 (registers: one CTA an SM, or spills).
#include "kv4_sums.cuh"

namespace specdec {
namespace {

constexpr int kChunk = 32;      // positions of an item
constexpr int kMaxChunks = 32;  // chunks of a CTA's segment at most
constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMine = kMaxChunks / kWarps + 2;  // chunks that a warp has a part of
constexpr int kStages = 2;
// Tiles of eight query rows in shared memory: all of a request's where they
// fit; more heads or rows take several passes, the latter over the same codes.
// Up to eight rows take the kernel with one tile a pass (one token, B=128: 37 us
// with it, 41 with two tiles; its 80 registers leave room for three CTAs).
template <int RT>
struct SumCfg {
  static constexpr int kTiles = 8 * RT;
  static constexpr int kCtas = RT == 1 ? 3 : 2;  // of an SM
};

// mma16816 without sums before: D = A B.
__device__ __forceinline__ void mma16816_zero(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}

__device__ __forceinline__ int sum_chunks(const SumReq& r) { return (r.end + kChunk - 1) / kChunk; }
__device__ __forceinline__ int sum_tiles(const SumArgs& a, const SumReq& r) { return (r.rows * a.G + 7) / 8; }
// What a chunk costs: copying and unpacking its codes about what a row tile does.
__device__ __forceinline__ int sum_cost(const SumArgs& a, const SumReq& r) { return sum_tiles(a, r) + 1; }
__device__ __forceinline__ int64_t sum_units(const SumArgs& a, const SumReq& r) {
  return static_cast<int64_t>(sum_chunks(r)) * sum_cost(a, r);
}
// Chunks of this cost that begin before `units` of their request's.
__device__ __forceinline__ int chunks_before(int64_t units, int cost) {
  const int64_t x = units + cost - 1;
  return static_cast<int>(x <= 0xffffffffll ? static_cast<uint32_t>(x) / static_cast<uint32_t>(cost) : x / cost);
}

// A tile of eight query rows of a KV head as B fragments: lane by lane, per
// group of 32 channels two steps of 16; the groups' sums; and of its columns
// the factor that turns products into units of log2, lse in these (rows that
// do not count: 0 and +infinity), and the row of the path.
template <int D>
struct QTile {
  uint2 b[D / 16][32];
  uint2 lo[32];
  float c[8], l[8];
  int row[8];
};

template <int D, int TILES>
struct SumShared {
  uint8_t ring[kWarps][kStages][kChunk * Pos<D>::kBytes];
  QTile<D> q[TILES];
  float sum[kWarps][kMine][kChunk];
  unsigned there[kWarps][kStages];
};

// Rows [r0, r0 + 8) of KV head h as a tile: a warp's work.
template <int D>
__device__ __forceinline__ void load_tile(const SumArgs& a, int b, int h, int r0, const SumReq& rq, bool count,
                                          QTile<D>& x) {
  const int lane = threadIdx.x & 31, t = lane & 3, g = lane >> 2;
  const int r = r0 + g, i = static_cast<int>(static_cast<uint64_t>(r) * a.g_inv >> 40);
  bool in = i < rq.rows;
  int n = in ? i : 0;
  if (in && a.path) {
    n = __ldg(a.path + static_cast<int64_t>(b) * a.N + i);
    in = n >= 0 && n < a.N;
    if (!in && count && t == 0 && r == i * a.G) bump(a.stats, SPEC_STAT_BAD_REQUEST);
    if (!in) n = 0;
  }
  const int64_t at = static_cast<int64_t>(b) * a.N + n;
  const int head = h * a.G + r - i * a.G;
  const float lse = in ? __ldg(a.lse + at * a.Hq + head) : neg_inf();
  uint4 v[D / 32];
#pragma unroll
  for (int k = 0; k < D / 32; ++k) {
    v[k] = make_uint4(0, 0, 0, 0);
    if (in)
      v[k] = __ldg(
          reinterpret_cast<const uint4*>(a.q + at * a.q_stride + static_cast<int64_t>(head) * D + k * 32 + t * 8));
  }
  in = in && isfinite(lse);
  // the largest magnitude: bf16 bits without the sign compare as integers
  uint32_t big = 0;
#pragma unroll
  for (int k = 0; k < D / 32; ++k) {
    if (!in) v[k] = make_uint4(0, 0, 0, 0);
    big = __vmaxu2(big, __vmaxu2(__vmaxu2(v[k].x & 0x7fff7fffu, v[k].y & 0x7fff7fffu),
                                 __vmaxu2(v[k].z & 0x7fff7fffu, v[k].w & 0x7fff7fffu)));
  }
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) big = __vmaxu2(big, __shfl_xor_sync(0xffffffffu, big, o));
  const int bits = static_cast<int>(max(big & 0xffffu, big >> 16));
  // 2^e <= max < 2^(e + 1): the largest becomes [2^14, 2^15)
  const int e = bits == 0 || bits >= 0x7f80 ? 0 : max((bits >> 7) - 127, -113);
  const float up = __uint_as_float(static_cast<uint32_t>(127 + 14 - e) << 23), half_up = up * 0.0625f;
  float sums[D / 32];
#pragma unroll
  for (int k = 0; k < D / 32; ++k) {
    const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
    uint32_t y[4];
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float f = j & 1 ? half_up : up, y0 = bf16_lo(w[j]) * f, y1 = bf16_hi(w[j]) * f;
      y[j] = h2_u32(__floats2half2_rn(y0, y1));
      s += j & 1 ? (y0 + y1) * 16.0f : y0 + y1;
    }
    x.b[2 * k][lane] = make_uint2(y[0], y[1]);
    x.b[2 * k + 1][lane] = make_uint2(y[2], y[3]);
    // 32 channels of at most 2^15 each, times 2^-5: fp16's range
    s *= 0.03125f;
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    sums[k] = s;
  }
  // groups' sums as three terms: A's columns hold lo of the groups three times.
  // Lane t has rows 2t, 2t + 1 of B (first register) and 2t + 8, 2t + 9 (second)
  uint32_t term[3][2];
#pragma unroll
  for (int z = 0; z < 3; ++z)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int k0 = 2 * k, k1 = 2 * k + 1;
      const float s0 = k0 < D / 32 ? sums[k0 % (D / 32)] : 0.0f, s1 = k1 < D / 32 ? sums[k1 % (D / 32)] : 0.0f;
      const __half2 y = __floats2half2_rn(s0, s1);
      term[z][k] = h2_u32(y);
      if (k0 < D / 32) sums[k0 % (D / 32)] -= __low2float(y);
      if (k1 < D / 32) sums[k1 % (D / 32)] -= __high2float(y);
    }
  x.lo[lane] = make_uint2(t == 0 ? term[0][0] : t == 1 ? term[0][1] : t == 2 ? term[1][0] : term[1][1],
                          t == 0 ? term[2][0] : t == 1 ? term[2][1] : 0u);
  if (t == 0) {
    // products come times 2^(14 - e - 24): finite while scale log2(e) 2^e is below 2^118
    x.c[g] = in ? a.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 + e) << 23) * 0x1p10f : 0.0f;
    x.l[g] = in ? lse * kLog2e : __uint_as_float(0x7f800000u);
    x.row[g] = i;
  }
}

// A warp's items, the cursor that fills its ring: (chunk, head) pairs, the
// chunk's heads one after another, so that a chunk's slots and addresses are
// found once and a cache row is read from end to end.
template <int D>
struct Ring {
  int left;         // items to be copied
  int chunk, head;  // of the next one
  int32_t slot;     // of position lane of the chunk behind the one at hand; -2: none
  uint64_t src[D / 32], meta;  // where this lane's copies of the chunk's head 0 come from
  unsigned size, have;         // bit u: the copy's position has a slot; positions that have one
  unsigned base;

  __device__ __forceinline__ void load(const int32_t* row, int at, int end) {
    const int pos = at * kChunk + static_cast<int>(threadIdx.x & 31);
    slot = pos < end ? __ldg(row + pos) : -2;
  }
  // Takes over the chunk whose slots were loaded last, and loads the next one's.
  __device__ __forceinline__ void enter(const SumArgs& a, const int32_t* row, int at, int end, int h, bool count) {
    constexpr int per = D / 32;
    const int lane = threadIdx.x & 31;
    const bool ok = slot >= 0 && slot < a.num_slots;
    if (!ok && slot != -2 && count && h == 0) bump(a.stats, SPEC_STAT_BAD_REQUEST);
    have = __ballot_sync(0xffffffffu, ok);
    const uint64_t mine = reinterpret_cast<uint64_t>(a.pool) +
                          static_cast<uint64_t>(ok ? slot : 0) * static_cast<uint64_t>(a.slot_stride);
    size = 0;
#pragma unroll
    for (int u = 0; u < per; ++u) {
      const int pos = u * (32 / per) + lane / per;
      src[u] = __shfl_sync(0xffffffffu, mine, pos) + (lane % per) * 16;
      size |= ((have >> pos) & 1u) << u;
    }
    meta = mine + D;
    load(row, at + 1, end);
  }
  __device__ __forceinline__ void copy(const SumArgs& a, const int32_t* row, int first, int end, int h0, int heads,
                                       int st, unsigned* there, bool count) {
    using P = Pos<D>;
    if (left > 0) {
      constexpr int per = D / 32;
      const int lane = threadIdx.x & 31;
      const unsigned to = base + st * (kChunk * P::kBytes);
      const unsigned off = static_cast<unsigned>(h0 + head) * kv4_head_bytes(D);
      if (lane == 0) there[st] = have;
#pragma unroll
      for (int u = 0; u < per; ++u)
        put_async(to + (u * (32 / per) + lane / per) * P::kBytes + (lane % per) * 16, src[u] + off,
                  ((size >> u) & 1u) * 16u);
      put_async(to + lane * P::kBytes + P::kCodes, meta + off, ((have >> lane) & 1u) * 16u);
      --left;
      if (++head == heads) {
        head = 0;
        ++chunk;
        if (left > 0) enter(a, row, first + chunk, end, 0, count);
      }
    }
    cp_async_commit();
  }
};

// A row of q that a lane holds D / 8 channels of, eight lanes a row.
template <int D>
struct RowPart {
  static constexpr int kVecs = D / 64;
  uint4 v[kVecs];
  __device__ __forceinline__ void load(const SumArgs& a, int64_t at, int head, bool in) {
    const uint16_t* src = a.q + at * a.q_stride + static_cast<int64_t>(head) * D + (threadIdx.x & 7) * (D / 8);
#pragma unroll
    for (int z = 0; z < kVecs; ++z) v[z] = in ? __ldg(reinterpret_cast<const uint4*>(src) + z) : make_uint4(0, 0, 0, 0);
  }
  // Exponent of the row's largest element: 2^e <= it < 2^(e + 1), at least
  // -117 (zeros, and rows with an infinity or NaN: 0).
  __device__ __forceinline__ int exponent() const {
    uint32_t big = 0;
#pragma unroll
    for (int z = 0; z < kVecs; ++z)
      big = __vmaxu2(big, __vmaxu2(__vmaxu2(v[z].x & 0x7fff7fffu, v[z].y & 0x7fff7fffu),
                                   __vmaxu2(v[z].z & 0x7fff7fffu, v[z].w & 0x7fff7fffu)));
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) big = __vmaxu2(big, __shfl_xor_sync(0xffffffffu, big, o));
    const int bits = static_cast<int>(max(big & 0xffffu, big >> 16));
    return bits == 0 || bits >= 0x7f80 ? 0 : max((bits >> 7) - 127, -117);
  }
};
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }

// Rows [r0, r0 + 128) of KV head h as a block in the workspace: a CTA's work,
// four rows a warp at a time.
template <int D>
__device__ __forceinline__ void write_block(const SumArgs& a, int b, int h, int r0, const SumReq& rq,
                                            RowsBlock<D>& out) {
  constexpr int kTurns = kRowsBlock / (4 * kWarps);
  __shared__ int s_top[kWarps], s_fold[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane & 7, c0 = warp * 4 + (lane >> 3);
  RowPart<D> x[kTurns];
  int row[kTurns], e[kTurns];
  float nl[kTurns];
  int top = -127;
#pragma unroll
  for (int z = 0; z < kTurns; ++z) {
    const int r = r0 + c0 + z * 4 * kWarps;
    row[z] = static_cast<int>(static_cast<uint64_t>(r) * a.g_inv >> 40);
    int node = row[z] < rq.rows ? row[z] : -1;
    if (a.path && node >= 0) {
      node = __ldg(a.path + static_cast<int64_t>(b) * a.N + row[z]);
      if (node < 0 || node >= a.N) {
        if (h == 0 && sub == 0 && r == row[z] * a.G) bump(a.stats, SPEC_STAT_BAD_REQUEST);
        node = -1;
      }
    }
    const int64_t at = static_cast<int64_t>(b) * a.N + max(node, 0);
    const int head = h * a.G + r - row[z] * a.G;
    const float lse = node >= 0 ? __ldg(a.lse + at * a.Hq + head) : neg_inf();
    nl[z] = isfinite(lse) ? -lse * kLog2e : neg_inf();
    x[z].load(a, at, head, isfinite(lse));
  }
#pragma unroll
  for (int z = 0; z < kTurns; ++z) {
    e[z] = x[z].exponent();
    if (nl[z] != neg_inf()) top = max(top, e[z]);
  }
#pragma unroll
  for (int o = 8; o < 32; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (lane == 0) s_top[warp] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) top = max(top, s_top[w]);
  // products come times 2^(9 - e).  Rows 2^-8 of the largest still lose nothing
  // above 2^-25 of their own largest element; one is large enough for a row that
  // does not count to come out as 2^-512, and for lse's terms to fit
  const float one = a.scale_log2 * pow2(max(top, -117)) * 0x1p-9f;
  bool fold = one >= 0x1p-17f && one <= 0x1p100f;
#pragma unroll
  for (int z = 0; z < kTurns; ++z)
    if (nl[z] != neg_inf()) fold = fold && e[z] >= top - 8 && fabsf(nl[z]) < one * 0x1p25f;
  fold = __all_sync(0xffffffffu, fold);
  if (lane == 0) s_fold[warp] = fold;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) fold = fold && s_fold[w] != 0;
#pragma unroll
  for (int z = 0; z < kTurns; ++z) {
    const int c = c0 + z * 4 * kWarps;
    const bool in = nl[z] != neg_inf();
    // the largest becomes at most [2^9, 2^10), a group's sum at most 2^15
    const float up = pow2(9 - (fold ? top : e[z]));
    float s = 0.0f;
#pragma unroll
    for (int v = 0; v < RowPart<D>::kVecs; ++v) {
      const uint32_t w[4] = {x[z].v[v].x, x[z].v[v].y, x[z].v[v].z, x[z].v[v].w};
      uint32_t y[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float y0 = bf16_lo(w[j]) * up, y1 = bf16_hi(w[j]) * up;
        y[j] = h2_u32(__floats2half2_rn(y0, y1));
        s += y0 + y1;
      }
      const int ch = sub * (D / 8) + 8 * v;
      *reinterpret_cast<uint4*>(out.q + ch / 64 * RowsBlock<D>::kSlab + c * 128 + ((ch % 64 / 8 ^ (c & 7)) << 4)) =
          make_uint4(y[0], y[1], y[2], y[3]);
    }
#pragma unroll
    for (int o = 1; o < 256 / D; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    // a lane writes three terms: a group's first lane the group's, lane 1 lse's;
    // the columns between are zeros where D = 64 has two groups, 15 always
    const bool of_lse = sub == 1;
    float t = of_lse ? (!fold ? 0.0f : in ? nl[z] / one * 0x1p-10f : -65504.0f) : s;
    if (of_lse || sub % (256 / D) == 0) {
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        const __half y = __float2half_rn(t);
        t -= __half2float(y);
        const int col = of_lse ? 12 + k : 4 * k + sub / (256 / D);
        *reinterpret_cast<__half*>(out.sums + col / 8 * (kRowsBlock * 16) + c * 16 + col % 8 * 2) = y;
      }
    } else if (D == 64 && (sub == 2 || sub == 3)) {
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        const int col = 4 * k + sub;
        *reinterpret_cast<uint16_t*>(out.sums + col / 8 * (kRowsBlock * 16) + c * 16 + col % 8 * 2) = 0;
      }
    }
    if (sub == 7) *reinterpret_cast<uint16_t*>(out.sums + kRowsBlock * 16 + c * 16 + 14) = 0;
    if (sub == 0) {
      out.c[c] = fold ? one : in ? a.scale_log2 * pow2(e[z]) * 0x1p-9f : 0.0f;
      out.nl[c] = nl[z];
      out.row[c] = row[z];
    }
  }
  if (threadIdx.x == 0) out.fold = fold;
  __syncthreads();
}

// The blocks of the requests that go to the tensor-memory kernel.
template <int D>
__device__ __noinline__ void write_blocks(const SumArgs& a) {
  const int blocks = (a.N * a.G + kRowsBlock - 1) / kRowsBlock, each = a.Hkv * blocks;
  const int64_t all = static_cast<int64_t>(a.B) * each;
#pragma unroll 1
  for (int64_t i = blockIdx.x; i < all; i += gridDim.x) {
    const int b = static_cast<int>(i / each), k = static_cast<int>(i - static_cast<int64_t>(b) * each);
    const int h = k / blocks, block = k - h * blocks;
    const SumReq rq = any_req(a, b);
    if (rq.rows * a.G > a.upto && block * kRowsBlock < rq.rows * a.G)
      write_block<D>(a, b, h, block * kRowsBlock, rq, static_cast<RowsBlock<D>*>(a.ws)[i]);
  }
}

// RT: row tiles of eight that a pass over the codes takes at most.
template <int D, int RT>
__global__ void __launch_bounds__(kThreads, SumCfg<RT>::kCtas) kv4_sums_kernel(const SumArgs a, int ctas) {
  pdl_enter();
  constexpr int TILES = SumCfg<RT>::kTiles;
  extern __shared__ __align__(16) unsigned char sums_sm[];
  using Shared = SumShared<D, TILES>;
  Shared& sh = *reinterpret_cast<Shared*>(sums_sm);
  if (!spec_smem_ok(sizeof(sh), a.stats)) return;
  __shared__ int64_t s_warp[kWarps], s_pre;
  __shared__ int s_b;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, t = lane & 3, g = lane >> 2;

  // this CTA's stretch [lo, hi) of the line of all requests' chunks, by their
  // cost: the chunks that begin in it.  pre: where request b begins
  int64_t lo, hi, pre;
  int b;
  {
    const int per = (a.B + kThreads - 1) / kThreads;
    const int b0 = min(a.B, static_cast<int>(threadIdx.x) * per), b1 = min(a.B, b0 + per);
    int64_t mine = 0;
    bool others = false;  // requests for the tensor-memory kernel
#pragma unroll 1
    for (int i = b0; i < b1; ++i) {
      const SumReq r = any_req(a, i);
      if (r.rows * a.G <= a.upto) mine += sum_units(a, r);
      else others = true;
      if (r.bad && blockIdx.x == 0) bump(a.stats, SPEC_STAT_BAD_REQUEST);
    }
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) s_warp[warp] = incl;
    others = __syncthreads_or(others) != 0;
    if (RT > 1 && others) write_blocks<D>(a);
    int64_t total = 0;
    pre = incl - mine;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      if (i < warp) pre += s_warp[i];
      total += s_warp[i];
    }
    const int64_t n = min(static_cast<int64_t>(ctas), total), cta = blockIdx.x;
    if (cta >= n) return;
    lo = cta * total / n;
    hi = (cta + 1) * total / n;
    if (lo >= pre && lo < pre + mine) {
      int i = b0;
#pragma unroll 1
      for (;; ++i) {
        const int64_t u = sum_units(a, sum_req(a, i));
        if (lo < pre + u) break;
        pre += u;
      }
      s_pre = pre;
      s_b = i;
    }
    __syncthreads();
    b = s_b;
    pre = s_pre;
  }

#pragma unroll 1
  for (; pre < hi; ++b) {
    const SumReq rq = sum_req(a, b);
    const int32_t* row = a.table + static_cast<int64_t>(b) * a.max_ctx;
    const int tiles = sum_tiles(a, rq), cost = sum_cost(a, rq);
    const int64_t units = sum_units(a, rq);
    int chunk = pre < lo ? chunks_before(lo - pre, cost) : 0;
    const int all = pre + units <= hi ? sum_chunks(rq) : chunks_before(hi - pre, cost);
    pre += units;
    // a pass: `heads` heads, `rts` tiles of rows of each
    const int rts = min(tiles, RT), heads = min(a.Hkv, TILES / max(rts, 1));
    const bool once = rts == tiles && heads == a.Hkv;  // then the tiles stay for the whole request
    bool loaded = false;
#pragma unroll 1
    while (chunk < all) {
      const int chunks = min(all - chunk, kMaxChunks);
      // this warp's items and their first chunk: the same in all passes but for a last one of fewer heads
#pragma unroll
      for (int i = 0; i < kMine; ++i) sh.sum[warp][i][lane] = 0.0f;
      const int from0 = chunks * warp / kWarps;  // the first chunk of any pass
#pragma unroll 1
      for (int h0 = 0; h0 < a.Hkv; h0 += heads)
#pragma unroll 1
        for (int rt0 = 0; rt0 < tiles; rt0 += RT) {
          const int hs = min(heads, a.Hkv - h0), mine = min(rts, tiles - rt0), items = chunks * hs;
          const int from = items * warp / kWarps, to = items * (warp + 1) / kWarps;
          Ring<D> ring;
          ring.left = to - from;
          ring.chunk = from / hs, ring.head = from - ring.chunk * hs;
          ring.base = static_cast<unsigned>(__cvta_generic_to_shared(sh.ring[warp][0]));
          const bool count = rt0 == 0 && h0 == 0;
          int ch = ring.chunk, h = ring.head;
          if (ring.left > 0) {
            ring.load(row, chunk + ch, rq.end);
            ring.enter(a, row, chunk + ch, rq.end, h, count);
          }
#pragma unroll 1
          for (int i = 0; i < kStages - 1; ++i) ring.copy(a, row, chunk, rq.end, h0, hs, i, sh.there[warp], count);
          if (!loaded) {
            if (!once) __syncthreads();  // every warp is done with the pass before
#pragma unroll 1
            for (int i = warp; i < hs * mine; i += kWarps) {
              const int hh = i / mine, x = i - hh * mine;
              load_tile<D>(a, b, h0 + hh, (rt0 + x) * 8, rq, h0 + hh == 0 && chunk == 0, sh.q[hh * rts + x]);
            }
            __syncthreads();
            loaded = once;
          }
          int st = 0;
          float w[4] = {0.0f, 0.0f, 0.0f, 0.0f};  // of positions 8 j + g of the chunk
          auto flush = [&](int c) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              w[j] += __shfl_xor_sync(0xffffffffu, w[j], 1);
              w[j] += __shfl_xor_sync(0xffffffffu, w[j], 2);
            }
            const float x = t == 0 ? w[0] : t == 1 ? w[1] : t == 2 ? w[2] : w[3];
            if (spec_in(c - from0, kMine, a.stats)) sh.sum[warp][c - from0][8 * t + g] += x;
            w[0] = w[1] = w[2] = w[3] = 0.0f;
          };
#pragma unroll 1
          for (int item = from; item < to; ++item) {
            __syncwarp();  // every lane has read the stage before
            ring.copy(a, row, chunk, rq.end, h0, hs, (st + kStages - 1) % kStages, sh.there[warp], count);
            cp_async_wait<kStages - 1>();
            __syncwarp();  // every lane's copies of this item have landed
            const unsigned there = sh.there[warp][st];
            const uint8_t* s8 = sh.ring[warp][st];
            st = (st + 1) % kStages;
            const QTile<D>* q = sh.q + h * rts;

            // s[x][u][2 i + e]: position 16 u + 8 i + g, column 2 t + e of tile x
            float s[RT][2][4];
#pragma unroll
            for (int k = 0; k < D / 32; ++k) {
              uint32_t c[2][2][4];  // step of 16 channels, block of 16 positions, register
              float step[4];        // of positions 8 j + g
#pragma unroll
              for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  const uint8_t* p8 = s8 + (16 * u + 8 * i + g) * Pos<D>::kBytes;
                  const uint32_t v = *reinterpret_cast<const uint32_t*>(p8 + k * 16 + t * 4);
                  step[2 * u + i] = __half2float(*reinterpret_cast<const __half*>(p8 + Pos<D>::kCodes + k * 4));
                  c[0][u][i] = v & 0x000f000fu;
                  c[0][u][2 + i] = v & 0x00f000f0u;
                  c[1][u][i] = (v >> 8) & 0x000f000fu;
                  c[1][u][2 + i] = (v >> 8) & 0x00f000f0u;
                }
#pragma unroll
              for (int x = 0; x < RT; ++x)
                if (x == 0 || x < mine) {
                  const uint2 b0 = q[x].b[2 * k][lane], b1 = q[x].b[2 * k + 1][lane];
#pragma unroll
                  for (int u = 0; u < 2; ++u) {
                    float p[4];
                    mma16816_zero(p, c[0][u], b0.x, b0.y);
                    mma16816(p, make_uint4(c[1][u][0], c[1][u][1], c[1][u][2], c[1][u][3]), b1.x, b1.y);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                      s[x][u][j] = k == 0 ? step[2 * u + (j >> 1)] * p[j]
                                          : fmaf(step[2 * u + (j >> 1)], p[j], s[x][u][j]);
                  }
                }
            }
            // lo of two groups: those of this lane's columns of A
            uint32_t lo_a[2][4];
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const uint8_t* m8 = s8 + (16 * u + 8 * i + g) * Pos<D>::kBytes + Pos<D>::kCodes;
                uint2 m = make_uint2(0, 0);
                if (D == 128 || (t & 1) == 0) m = *reinterpret_cast<const uint2*>(m8 + 8 * (t & 1));
                lo_a[u][i] = lo_a[u][2 + i] = __byte_perm(m.x, m.y, 0x7632);
              }
            const int at0 = (chunk + ch) * kChunk;
            const bool whole = there == 0xffffffffu && at0 + kChunk <= rq.start + 1;
#pragma unroll
            for (int x = 0; x < RT; ++x)
              if (x == 0 || x < mine) {
                const uint2 lo = q[x].lo[lane];
                const float2 c = *reinterpret_cast<const float2*>(q[x].c + 2 * t);
                const float2 l = *reinterpret_cast<const float2*>(q[x].l + 2 * t);
                // the groups' sums were held times 2^(14 - e - 5), the products 2^(14 - e - 24)
                const float2 c_lo = make_float2(c.x * 0x1p-19f, c.y * 0x1p-19f);
                const int2 i_of = *reinterpret_cast<const int2*>(q[x].row + 2 * t);
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                  float p[4];
                  mma16816_zero(p, lo_a[u], lo.x, lo.y);
#pragma unroll
                  for (int j = 0; j < 4; ++j) {
                    const float y = fast_exp2(fmaf(p[j], j & 1 ? c_lo.y : c_lo.x,
                                                   fmaf(s[x][u][j], j & 1 ? c.y : c.x, j & 1 ? -l.y : -l.x)));
                    if (whole) {
                      w[2 * u + (j >> 1)] += y;
                    } else {
                      const int at = 16 * u + 8 * (j >> 1) + g;
                      if (((there >> at) & 1u) != 0 && at0 + at <= rq.start + (j & 1 ? i_of.y : i_of.x))
                        w[2 * u + (j >> 1)] += y;
                    }
                  }
                }
              }
            if (++h == hs) {
              h = 0;
              flush(ch);
              ++ch;
            }
          }
          if (h != 0) flush(ch);
          cp_async_wait<0>();
          __syncwarp();
        }
      __syncthreads();
      const int64_t at = static_cast<int64_t>(b) * a.max_ctx + static_cast<int64_t>(chunk) * kChunk;
      for (int i = threadIdx.x; i < min(chunks * kChunk, rq.end - chunk * kChunk); i += kThreads) {
        const int c = i / kChunk;
        float x = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const int k = c - chunks * w / kWarps;  // chunks of a warp: from its first on, in all passes
          if (k >= 0 && k < kMine) x += sh.sum[w][k][i % kChunk];
        }
        a.out[at + i] = a.prev ? a.prev[at + i] + x : x;
      }
      __syncthreads();
      chunk += chunks;
    }
  }
}

// Rows of a KV head above which the tensor-memory kernel takes a request, whose
// time hardly depends on them up to 128.  8 KV heads of 128, in us, here / there
// (two launches):
//              B=1, 4000     B=4, 60000     B=128, 1000
//   16 rows     8.8 / 14.6    59 /  99       44 / 88
//   24 rows    12.4 / 14.8   105 /  99       72 / 88
//   32 rows    14.1 / 14.8   112 /  99       80 / 89
//   36 rows    17.6 / 14.9   154 / 101         -
//   64 rows    24.5 / 15.0   215 / 102         -
constexpr int kManyRows = 32;

// The upper limits of a call's sizes.
bool sum_sizes(int B, int N, int Hq, int Hkv, int D) {
  return spec_kv4_slot_bytes(Hkv, D) >= 0 && N <= SPEC_MAX_NODES && Hq <= SPEC_KV4_MAX_HEADS * 16 && B <= 65535;
}

template <int D, int RT>
int launch_sums(const SumArgs& a, int sms, cudaStream_t s) {
  constexpr auto kernel = kv4_sums_kernel<D, RT>;
  constexpr size_t smem = sizeof(SumShared<D, SumCfg<RT>::kTiles>);
  if (!allow_smem<kernel>(smem)) return SPEC_ERR_CUDA;
  const int ctas = sms * SumCfg<RT>::kCtas;
  launch_k(kernel, static_cast<unsigned>(ctas), kThreads, smem, s, a, ctas);
  return launch_status();
}

}  // namespace
}  // namespace specdec

using namespace specdec;

extern "C" size_t spec_kv4_weight_sums_ws_size(int B, int N, int Hq, int Hkv, int D) {
  if (B < 1 || N < 1 || Hkv < 1 || Hq < Hkv || Hq % Hkv != 0 || !sum_sizes(B, N, Hq, Hkv, D)) return 0;
  const int64_t rows = static_cast<int64_t>(N) * (Hq / Hkv);
  if (rows <= kManyRows) return 0;
  return static_cast<size_t>(B) * Hkv * ((rows + kRowsBlock - 1) / kRowsBlock) *
         (D == 128 ? sizeof(RowsBlock<128>) : sizeof(RowsBlock<64>));
}

extern "C" int spec_kv4_weight_sums(int B, int N, int Hq, int Hkv, int D, const void* q, int64_t q_stride,
                                    const float* lse, const int32_t* accept_path_or_null,
                                    const int32_t* accept_length_or_null, const void* pool, int64_t num_slots,
                                    int64_t slot_stride, const int32_t* seq_lens, const int32_t* req_to_token,
                                    int64_t max_ctx, float scale, const float* prev_or_null, float* out,
                                    int32_t* stats_or_null, void* ws, size_t ws_bytes, spec_stream_t stream) {
  if (B < 0 || N < 0 || Hkv < 1 || Hq < 1 || Hq % Hkv != 0 || max_ctx < 1 || num_slots < 1 || !(scale > 0.0f) ||
      !isfinite(scale))
    return SPEC_ERR_INVALID_ARG;
  const int64_t row = spec_kv4_slot_bytes(Hkv, D);
  if (!sum_sizes(B, N, Hq, Hkv, D)) return SPEC_ERR_UNSUPPORTED;
  if (scale < 0x1p-20f || scale > 0x1p20f) return SPEC_ERR_UNSUPPORTED;
  if (slot_stride < row || q_stride < static_cast<int64_t>(Hq) * D) return SPEC_ERR_INVALID_ARG;
  if (slot_stride % 16 != 0 || q_stride % 8 != 0 || num_slots > INT32_MAX || max_ctx > INT32_MAX - 2 * kRowsBlock ||
      slot_stride > INT32_MAX)
    return SPEC_ERR_UNSUPPORTED;
  if (B == 0 || N == 0) return SPEC_OK;
  if (!q || !lse || !pool || !seq_lens || !req_to_token || !out) return SPEC_ERR_INVALID_ARG;
  for (const void* p : {q, pool})
    if ((reinterpret_cast<uintptr_t>(p) & 15) != 0) return SPEC_ERR_UNSUPPORTED;
  // the old sums are read while others' new ones are written, unless they are the same
  const uintptr_t p0 = reinterpret_cast<uintptr_t>(prev_or_null), o0 = reinterpret_cast<uintptr_t>(out);
  const uintptr_t wide = static_cast<uintptr_t>(B) * max_ctx * 4;
  if (prev_or_null && p0 != o0 && p0 < o0 + wide && o0 < p0 + wide) return SPEC_ERR_INVALID_ARG;
  const size_t need = spec_kv4_weight_sums_ws_size(B, N, Hq, Hkv, D);
  if (need > 0 && (!ws || (reinterpret_cast<uintptr_t>(ws) & 15) != 0)) return SPEC_ERR_INVALID_ARG;
  if (ws_bytes < need) return SPEC_ERR_WORKSPACE;
  const int sms = attn_sms();
  if (sms == 0) {
    cudaGetLastError();
    return SPEC_ERR_CUDA;
  }
  const int G = Hq / Hkv;
  SumArgs a{static_cast<const uint16_t*>(q), q_stride, lse, accept_path_or_null, accept_length_or_null, B, N, Hq,
            Hkv, G, ((1ull << 40) + G - 1) / G, static_cast<const uint8_t*>(pool), num_slots, slot_stride,
            seq_lens, req_to_token, max_ctx, scale * kLog2e, prev_or_null, out, stats_or_null, nullptr, 0, INT32_MAX};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int64_t rows = static_cast<int64_t>(N) * G;
  // the host knows how many rows there may be, the device how many there are:
  // each request goes to the kernel that suits it
  const bool many = rows > kManyRows;
  a.upto = many ? kManyRows : INT32_MAX;
  a.ws = many ? ws : nullptr;
  const bool one = rows <= 8;
  const int e = D == 128 ? (one ? launch_sums<128, 1>(a, sms, s) : launch_sums<128, 2>(a, sms, s))
                         : (one ? launch_sums<64, 1>(a, sms, s) : launch_sums<64, 2>(a, sms, s));
  if (e != SPEC_OK || !many) return e;
  a.above = kManyRows;
  a.upto = INT32_MAX;
  return launch_sums_rows(a, D, sms, s);
}
