// What the two attention kernels over the 4-bit cache share: the arguments,
// the division of the work, the unpacking of codes and the merge of partials.
#pragma once

#include <atomic>

#include "kv4.cuh"

namespace specdec {

struct AttnArgs {
  const uint16_t* q;
  int64_t q_stride;
  int B, N, Hq, Hkv, G;
  uint64_t g_inv;  // ceil(2^40 / G)
  const uint8_t* pool;
  int64_t num_slots, slot_stride;
  const int32_t* table;
  int64_t max_ctx;
  const int32_t* seq_lens;
  const int32_t* num_nodes;
  const uint8_t* mask;
  float scale_log2;
  uint16_t* out;
  float* lse;
  float* ws;
  int ctas;  // of the attention launch
  int32_t* stats;
};

// Row r of a KV head is query head r % G of node r / G.  With r < 2^23 and G <=
// 2^12 (both checked by the host), r g_inv is r 2^40 / G and an excess of r
// (g_inv G - 2^40) / G < r <= 2^23, which is less than the 2^40 / G >= 2^28 that
// the next quotient is away: the shift is exact.
__device__ __forceinline__ int attn_node(const AttnArgs& a, int r) {
  return static_cast<int>(static_cast<uint64_t>(r) * a.g_inv >> 40);
}
// Index of row r of (b, h) in [B, N, Hq].
__device__ __forceinline__ int64_t attn_row(const AttnArgs& a, int b, int h, int r) {
  const int n = attn_node(a, r);
  return (static_cast<int64_t>(b) * a.N + n) * a.Hq + h * a.G + r - n * a.G;
}

// Element of q where row r of (b, h) begins.
__device__ __forceinline__ int64_t attn_q(const AttnArgs& a, int b, int h, int r, int D) {
  const int n = attn_node(a, r);
  return (static_cast<int64_t>(b) * a.N + n) * a.q_stride + static_cast<int64_t>(h * a.G + r - n * a.G) * D;
}

// Request b: nodes, positions [0, end) of which [start, end) are nodes, tiles
// of T positions and row tiles of R rows.  A request whose positions do not
// fit the table has no positions (its rows get zeros) and one empty tile.
struct Req {
  int nodes, start, end, tiles, row_tiles;
  bool bad;
};

template <int T>
__device__ __forceinline__ Req attn_req(const AttnArgs& a, int b, int R) {
  Req r;
  r.nodes = kv4_nodes(a.num_nodes, b, a.N);
  r.start = __ldg(a.seq_lens + b);
  r.bad = r.start < 0 || static_cast<int64_t>(r.start) + r.nodes > a.max_ctx;
  r.end = r.bad ? 0 : r.start + r.nodes;
  if (r.bad) r.start = 0;
  r.tiles = r.nodes == 0 ? 0 : (r.bad ? 1 : (r.end + T - 1) / T);
  r.row_tiles = (r.nodes * a.G + R - 1) / R;
  return r;
}

// The line.  Each (request, KV head, row tile) with a row is a segment: E
// units for its beginning and end (reading q, writing the result: about what
// E tiles cost), then one per tile.  CTA i of the launch's n takes units
// [i total / n, (i + 1) total / n).
template <int E>
__device__ __forceinline__ int64_t attn_units(const Req& r, int Hkv) {
  return r.tiles == 0 ? 0 : static_cast<int64_t>(r.tiles + E) * r.row_tiles * Hkv;
}

// A part of a segment: tiles [t0, t1) of its `tiles`.
struct Part {
  int b, h, rt, t0, t1;
  int nodes, start, end, tiles;
  bool bad;
  __device__ __forceinline__ bool complete() const { return t0 == 0 && t1 == tiles; }
};

// A CTA's stretch of the line, walked segment by segment.
template <int T, int E, int R>
struct Walk {
  int64_t left;  // units
  int skip;      // units of the segment (b, h, rt) that an earlier CTA has
  int b, h, rt, row_tiles;
  int nodes, start, end, tiles;
  bool bad;
  __device__ __forceinline__ void request(const AttnArgs& a) {
    const Req r = attn_req<T>(a, b, R);
    nodes = r.nodes, start = r.start, end = r.end, tiles = r.tiles, row_tiles = r.row_tiles, bad = r.bad;
  }
  __device__ __forceinline__ bool next(const AttnArgs& a, Part& p) {
#pragma unroll 1
    while (left > 0) {
      if (h == a.Hkv) {
        h = 0;
#pragma unroll 1
        do {
          ++b;
          request(a);
        } while (tiles == 0);
      }
      const int len = tiles + E - skip, take = left < len ? static_cast<int>(left) : len;
      p.t0 = max(skip - E, 0);
      p.t1 = skip + take - E;
      p.b = b, p.h = h, p.rt = rt, p.nodes = nodes, p.start = start, p.end = end, p.tiles = tiles, p.bad = bad;
      left -= take;
      skip = 0;
      if (++rt == row_tiles) rt = 0, ++h;
      if (p.t1 > p.t0) return true;
    }
    return false;
  }
};

// What a CTA needs to know of the whole line.
struct Line {
  int64_t total, ctas;  // units, CTAs that share them (no more than there are units)
  // CTAs from this one on that hold a part of the segment whose tiles [0, t1)
  // end this CTA's stretch
  __device__ __forceinline__ int pieces(int cta, int tiles, int t1) const {
    const int64_t end = (cta + 1) * total / ctas + tiles - t1;  // unit behind the segment's last
    return static_cast<int>((end * ctas - 1) / total) - cta + 1;
  }
};

// Finds this CTA's stretch (block-wide, every thread gets the result); false
// when it has none.
template <int T, int E, int R, int THREADS>
__device__ __forceinline__ bool attn_stretch(const AttnArgs& a, Line& line, Walk<T, E, R>& w) {
  __shared__ int64_t s_warp[THREADS / 32];
  __shared__ int64_t s_off;
  __shared__ int s_b;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per = (a.B + THREADS - 1) / THREADS;
  const int b0 = min(a.B, static_cast<int>(threadIdx.x) * per), b1 = min(a.B, b0 + per);
  int64_t mine = 0;
#pragma unroll 1
  for (int b = b0; b < b1; ++b) mine += attn_units<E>(attn_req<T>(a, b, R), a.Hkv);
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) s_warp[warp] = incl;
  __syncthreads();
  int64_t pre = incl - mine;
  line.total = 0;
#pragma unroll
  for (int i = 0; i < THREADS / 32; ++i) {
    if (i < warp) pre += s_warp[i];
    line.total += s_warp[i];
  }
  line.ctas = min(static_cast<int64_t>(a.ctas), line.total);
  const int64_t cta = blockIdx.x;
  if (cta >= line.ctas) return false;
  const int64_t lo = cta * line.total / line.ctas;
  if (lo >= pre && lo < pre + mine) {
    int b = b0;
#pragma unroll 1
    for (;; ++b) {
      const int64_t u = attn_units<E>(attn_req<T>(a, b, R), a.Hkv);
      if (lo < pre + u) break;
      pre += u;
    }
    s_off = lo - pre;
    s_b = b;
  }
  __syncthreads();
  w.left = (cta + 1) * line.total / line.ctas - lo;
  w.b = s_b;
  w.request(a);
  const int64_t seg = s_off / (w.tiles + E);
  w.skip = static_cast<int>(s_off - seg * (w.tiles + E));
  w.h = static_cast<int>(seg / w.row_tiles);
  w.rt = static_cast<int>(seg - static_cast<int64_t>(w.h) * w.row_tiles);
  return true;
}

__device__ __forceinline__ uint32_t h2_u32(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ __half2 u32_h2(uint32_t u) { return *reinterpret_cast<__half2*>(&u); }

// Code pairs of one register to fp16 values: the four nibbles j = 0..3 of
// both halves, out[j] = (lo + c * step) of nibble j.  A nibble ORed into the
// fraction of 1024 (or, 4 bits higher, 16 c) is exact, and so is the
// subtraction; the multiply-add rounds once.
__device__ __forceinline__ void dequant4(uint32_t x, uint32_t step2, uint32_t lo2, uint32_t* out) {
  const __half2 st = u32_h2(step2), lo = u32_h2(lo2);
  const __half2 k1024 = u32_h2(0xe400e400u), k16 = u32_h2(0x2c002c00u), k64 = u32_h2(0xd400d400u);
#pragma unroll
  for (int j = 0; j < 4; j += 2) {
    const uint32_t y = j ? x >> 8 : x;
    const __half2 a = __hadd2(u32_h2((y & 0x000f000fu) | 0x64006400u), k1024);        // - 1024
    const __half2 b = __hfma2(u32_h2((y & 0x00f000f0u) | 0x64006400u), k16, k64);     // / 16 - 64
    out[j] = h2_u32(__hfma2(a, st, lo));
    out[j + 1] = h2_u32(__hfma2(b, st, lo));
  }
}

// Which halves of a (step, lo) pair of registers decode to finite values alone,
// as a mask: every lo + c * step lies between lo and lo + 15 * step, and the sum
// is an infinity or NaN where one of its terms is.  Appended rows pass.  A node
// that every row's mask hides may never have been appended; its weights are
// zero, and its values, taken as zeros where they do not pass, add nothing to
// any row (0 times an infinity or NaN would).
__device__ __forceinline__ uint32_t finite_values(uint32_t step2, uint32_t lo2) {
  const __half2 last = __hfma2(u32_h2(step2), u32_h2(0x4b804b80u), u32_h2(lo2));  // 15
  return __hle2_mask(__habs2(last), u32_h2(0x7bff7bffu));                          // the largest finite
}

__device__ __forceinline__ uint16_t f_bf16(float x) {
  uint16_t r;
  asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(r) : "f"(x));
  return r;
}

// Weights are 2^(x - base) with base = max - held, rounded up: beyond 2^24 the
// difference is no fp32 number, and rounded down it would let weights pass
// 2^held and fp16's largest.  (Weights then lose held's powers of two; scores
// that far from zero differ by more than that or not at all.)
__device__ __forceinline__ float weight_base(float top, float held) { return __fadd_ru(top, -held); }

// The result of a row from its weighted values, weights' sum and maximum: no
// position gives zeros, NaN stays.
__device__ __forceinline__ float attn_inv(float sum) { return sum > 0.0f ? 1.0f / sum : (sum == 0.0f ? 0.0f : sum); }
// held: the power of two that the weights were held times.
__device__ __forceinline__ float attn_lse(float top, float sum, float held) {
  return sum == 0.0f ? neg_inf() : (top + log2f(sum) - held) * 0.6931471805599453f;
}

// The workspace: a header per CTA, then two partials per CTA of R rows, each
// R D weighted values and R pairs (maximum, sum of weights).  A CTA's stretch
// may begin within a segment (partial 0) and end within one that it began
// (partial 1); the header names the latter, with the number of CTAs that hold
// parts of it (0: none), this CTA's partial 1 and the next ones' partial 0.
struct __align__(16) CutSegment {
  int b, h, rt, pieces;
};
constexpr int kMaxCtas = 608;  // CTAs of a launch at most: 4 on each of 152 SMs
constexpr size_t kHeaderBytes = (kMaxCtas * sizeof(CutSegment) + 255) / 256 * 256;

__host__ __device__ __forceinline__ size_t attn_ws_bytes(int ctas, int R, int D) {
  return kHeaderBytes + static_cast<size_t>(ctas) * 2 * R * (D + 2) * sizeof(float);
}
__device__ __forceinline__ float* attn_part(const AttnArgs& a, int64_t cta, int which, int R, int D) {
  return reinterpret_cast<float*>(reinterpret_cast<char*>(a.ws) + kHeaderBytes) + (cta * 2 + which) * (R * (D + 2));
}

// Merges a cut segment's partials in the order of the positions: block (CTA
// that began the segment, eight rows).  A warp takes a row; with fewer than
// eight rows, several warps split the row's partials.
constexpr int kMergeThreads = 256, kMergeWarps = kMergeThreads / 32;

template <int D>
__global__ void __launch_bounds__(kMergeThreads) kv4_merge_kernel(const AttnArgs a, int R, float held) {
  pdl_enter();
  constexpr int per = D / 32;
  const int4 hdr = __ldg(reinterpret_cast<const int4*>(a.ws) + blockIdx.x);
  const int b = hdr.x, h = hdr.y, rt = hdr.z, pieces = hdr.w;
  if (pieces == 0) return;
  const int first = blockIdx.y * kMergeWarps;
  const int rows = min(min(R, kv4_nodes(a.num_nodes, b, a.N) * a.G - rt * R) - first, kMergeWarps);
  if (rows <= 0) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int split = kMergeWarps;  // warps of a row
  while (split * rows > kMergeWarps) split /= 2;
  const int mine = warp / split, share = warp % split, r = first + mine;
  __shared__ float s_o[kMergeWarps][D], s_l[kMergeWarps];
  float top = neg_inf(), l = 0.0f, acc[per];
#pragma unroll
  for (int j = 0; j < per; ++j) acc[j] = 0.0f;
  auto part = [&](int i) { return attn_part(a, blockIdx.x + i, i == 0 ? 1 : 0, R, D); };
  if (mine < rows) {
    for (int i = lane; i < pieces; i += 32) top = fmaxf(top, __ldg(part(i) + R * D + 2 * r));
    top = warp_max(top);
#pragma unroll 4
    for (int i = share; i < pieces; i += split) {
      const float* p = part(i);
      const float2 ml = __ldg(reinterpret_cast<const float2*>(p + R * D) + r);
      float x[per];
      if (per == 4) {
        const float4 v = __ldg(reinterpret_cast<const float4*>(p + r * D) + lane);
        x[0] = v.x, x[1] = v.y, x[per - 2] = v.z, x[per - 1] = v.w;
      } else {
        const float2 v = __ldg(reinterpret_cast<const float2*>(p + r * D) + lane);
        x[0] = v.x, x[1] = v.y;
      }
      const float f = ml.x == neg_inf() ? 0.0f : fast_exp2(ml.x - top);
      l += ml.y * f;
#pragma unroll
      for (int j = 0; j < per; ++j) acc[j] += x[j] * f;
    }
  }
  if (split > 1) {
#pragma unroll
    for (int j = 0; j < per; ++j) s_o[warp][lane * per + j] = acc[j];
    if (lane == 0) s_l[warp] = l;
    __syncthreads();
    if (share != 0) return;
    for (int w = 1; w < split; ++w) {
      l += s_l[warp + w];
#pragma unroll
      for (int j = 0; j < per; ++j) acc[j] += s_o[warp + w][lane * per + j];
    }
  }
  if (mine >= rows) return;
  const float inv = attn_inv(l);
  const int64_t at = attn_row(a, b, h, rt * R + r);
  if (!spec_in(at, static_cast<int64_t>(a.B) * a.N * a.Hq, a.stats) || !spec_in(blockIdx.x + pieces - 1, a.ctas, a.stats))
    return;
  uint32_t v[per / 2];
#pragma unroll
  for (int j = 0; j < per; j += 2)
    v[j / 2] = f_bf16(acc[j] * inv) | static_cast<uint32_t>(f_bf16(acc[j + 1] * inv)) << 16;
#pragma unroll
  for (int j = 0; j < per / 2; ++j) reinterpret_cast<uint32_t*>(a.out + at * D + lane * per)[j] = v[j];
  if (a.lse && lane == 0) a.lse[at] = attn_lse(top, l, held);
}

template <int D>
void launch_merge(const AttnArgs& a, int R, float held, cudaStream_t s) {
  const int64_t rows = static_cast<int64_t>(a.N) * a.G < R ? static_cast<int64_t>(a.N) * a.G : R;
  const dim3 grid(static_cast<unsigned>(a.ctas), static_cast<unsigned>((rows + kMergeWarps - 1) / kMergeWarps));
  launch_k(kv4_merge_kernel<D>, grid, kMergeThreads, 0, s, a, R, held);
}

// The number of SMs of the current device (0: no answer), asked once a device:
// a query is a noticeable part of a call of a few microseconds.
inline int attn_sms() {
  static std::atomic<int> known[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  std::atomic<int>& k = known[dev & 63];
  int sms = dev < 64 ? k.load(std::memory_order_relaxed) : 0;
  if (sms == 0) {
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    if (dev < 64) k.store(sms, std::memory_order_relaxed);
  }
  return sms;
}
// Limits of the tensor-memory kernel's launches (kv4_tree.cu) and its entry.
constexpr int kTreeRows = 128;     // rows of an accumulator
constexpr int kTreeMaxCtas = 304;  // two on each of 152 SMs (one with two accumulators)
int launch_tree_attention(AttnArgs a, int D, int sms, cudaStream_t s);

}  // namespace specdec
