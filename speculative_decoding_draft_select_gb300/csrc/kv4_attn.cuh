// What the two attention kernels over the 4-bit cache share: the arguments,
// the division of the work, the unpacking of codes and the merge of partials.
#pragma once

#include "kv4.cuh"

namespace specdec {

struct AttnArgs {
  const uint16_t* q;
  int64_t q_stride;
  int B, N, Hq, Hkv, G;
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

// Request b's share of the line: nodes, positions, tiles along the positions
// and row tiles.  A request whose positions do not fit the table has no
// positions (its rows get zeros) and one empty tile.
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
__device__ __forceinline__ int64_t attn_units(const Req& r, int Hkv) {
  return static_cast<int64_t>(r.tiles) * r.row_tiles * Hkv;
}

// The line's length and, for CTA `cta` of `ctas` (or for request `want` when
// want >= 0), where it begins: block-wide, every thread gets the result.
struct Where {
  int64_t total;   // units of all requests
  int64_t ctas;    // CTAs that share them: no more than there are units
  int64_t before;  // units of the requests before b
  int b;
};

template <int T, int THREADS>
__device__ __forceinline__ Where attn_where(const AttnArgs& a, int R, int cta, int want) {
  __shared__ int64_t s_warp[THREADS / 32];
  __shared__ int64_t s_before;
  __shared__ int s_b;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per = (a.B + THREADS - 1) / THREADS;
  const int b0 = min(a.B, static_cast<int>(threadIdx.x) * per), b1 = min(a.B, b0 + per);
  int64_t mine = 0;
  for (int b = b0; b < b1; ++b) mine += attn_units(attn_req<T>(a, b, R), a.Hkv);
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (threadIdx.x == 0) s_b = a.B;
  if (lane == 31) s_warp[warp] = incl;
  __syncthreads();
  int64_t pre = incl - mine, total = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) pre += s_warp[w];
    total += s_warp[w];
  }
  const int64_t ctas = min(static_cast<int64_t>(a.ctas), total);
  const int64_t x = want >= 0 ? 0 : (cta < ctas ? cta * total / ctas : total);
  if (want >= 0 ? (want >= b0 && want < b1) : (x >= pre && x < pre + mine)) {
    int b = b0;
    for (;; ++b) {
      if (b == want) break;
      const int64_t u = attn_units(attn_req<T>(a, b, R), a.Hkv);
      if (want < 0 && x < pre + u) break;
      pre += u;
    }
    s_before = pre;
    s_b = b;
  }
  __syncthreads();
  const Where w{total, ctas, s_before, s_b};
  __syncthreads();
  return w;
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

__device__ __forceinline__ uint16_t f_bf16(float x) {
  uint16_t r;
  asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(r) : "f"(x));
  return r;
}

// The result of a row from its weighted values, weights' sum and maximum: no
// position gives zeros, NaN stays.
__device__ __forceinline__ float attn_inv(float sum) { return sum > 0.0f ? 1.0f / sum : (sum == 0.0f ? 0.0f : sum); }
// held: the power of two that the weights were held times.
__device__ __forceinline__ float attn_lse(float top, float sum, float held) {
  return sum == 0.0f ? neg_inf() : (top + log2f(sum) - held) * 0.6931471805599453f;
}

// Merges the partials of the segments that were cut between CTAs: block
// (row tile, KV head, request).  A warp takes a row; where there are fewer
// rows than warps, the warps split the row's partials.
constexpr int kMergeThreads = 128, kMergeWarps = kMergeThreads / 32;

template <int D, int T>
__global__ void __launch_bounds__(kMergeThreads) kv4_merge_kernel(const AttnArgs a, int R, float held) {
  pdl_enter();
  constexpr int per = D / 32;
  const int b = blockIdx.z, h = blockIdx.y, rt = blockIdx.x;
  const Req rq = attn_req<T>(a, b, R);
  if (rt >= rq.row_tiles) return;
  const Where w0 = attn_where<T, kMergeThreads>(a, R, 0, b);
  const int64_t s0 = w0.before + (static_cast<int64_t>(h) * rq.row_tiles + rt) * rq.tiles, s1 = s0 + rq.tiles;
  const int64_t i0 = ((s0 + 1) * w0.ctas - 1) / w0.total, i1 = (s1 * w0.ctas - 1) / w0.total;
  if (i0 == i1) return;  // one CTA had the whole segment
  const int pieces = static_cast<int>(i1 - i0) + 1;
  auto part = [&](int i) {
    return a.ws + ((i0 + i) * 2 + (i == 0 ? 1 : 0)) * static_cast<int64_t>(R * (D + 2));
  };
  const int rows = min(R, rq.nodes * a.G - rt * R);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool split = rows < kMergeWarps;  // all warps on one row
  __shared__ float s_o[kMergeWarps][D], s_l[kMergeWarps];
  for (int r = split ? 0 : warp; r < rows; r += split ? 1 : kMergeWarps) {
    float top = neg_inf();
    for (int i = lane; i < pieces; i += 32) top = fmaxf(top, part(i)[R * D + 2 * r]);
    top = warp_max(top);
    float l = 0.0f, acc[per];
#pragma unroll
    for (int j = 0; j < per; ++j) acc[j] = 0.0f;
    const int first = split ? warp : 0, step = split ? kMergeWarps : 1;
#pragma unroll 4
    for (int i = first; i < pieces; i += step) {
      const float* p = part(i);
      const float pm = p[R * D + 2 * r], pl = p[R * D + 2 * r + 1];
      const float f = pm == neg_inf() ? 0.0f : fast_exp2(pm - top);
      l += pl * f;
#pragma unroll
      for (int j = 0; j < per; ++j) acc[j] += p[r * D + lane * per + j] * f;
    }
    if (split) {
#pragma unroll
      for (int j = 0; j < per; ++j) s_o[warp][lane * per + j] = acc[j];
      if (lane == 0) s_l[warp] = l;
      __syncthreads();
      l = 0.0f;
#pragma unroll
      for (int j = 0; j < per; ++j) acc[j] = 0.0f;
#pragma unroll
      for (int w = 0; w < kMergeWarps; ++w) {
        l += s_l[w];
#pragma unroll
        for (int j = 0; j < per; ++j) acc[j] += s_o[w][lane * per + j];
      }
      __syncthreads();
      if (warp != 0) continue;
    }
    const float inv = attn_inv(l);
    const int rw = rt * R + r, n = rw / a.G;
    const int64_t at = (static_cast<int64_t>(b) * a.N + n) * a.Hq + h * a.G + rw - n * a.G;
    uint32_t v[per / 2];
#pragma unroll
    for (int j = 0; j < per; j += 2)
      v[j / 2] = f_bf16(acc[j] * inv) | static_cast<uint32_t>(f_bf16(acc[j + 1] * inv)) << 16;
#pragma unroll
    for (int j = 0; j < per / 2; ++j) reinterpret_cast<uint32_t*>(a.out + at * D + lane * per)[j] = v[j];
    if (a.lse && lane == 0) a.lse[at] = attn_lse(top, l, held);
  }
}

// Limits of the tensor-memory kernel's launches (kv4_tree.cu) and its entry.
constexpr int kTreeRows = 128;     // rows of an accumulator
constexpr int kTreeMaxCtas = 304;  // two on each of 152 SMs
int launch_tree_attention(AttnArgs a, int D, int sms, cudaStream_t s);
size_t tree_attention_ws(int64_t rows, int D);

}  // namespace specdec
