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
// The rows of a KV head (N nodes times G query heads) are cut into row tiles
// and the positions into tiles of 64.  Work is dealt out evenly whatever the
// lengths are: the tiles of all (request, KV head, row tile) segments form
// one line, each CTA takes an equal stretch of it, and a segment that is cut
// between CTAs leaves partial (max, sum, weighted values) in the workspace,
// which a second kernel merges in a fixed order.  The host knows no lengths.
#include "kv4_attn.cuh"

namespace specdec {
namespace {

constexpr int kTile = 64;        // positions of a tile: 16 per warp
constexpr int kEnds = 2;         // tiles that a segment's beginning and end cost
constexpr int kAttThreads = 128;
constexpr int kAttWarps = kAttThreads / 32;
constexpr float kWeightExp = 15.0f;  // weights are held times 2^15

// D += A B, 16 x 8 x 16, fp16 operands and fp32 sums.
__device__ __forceinline__ void mma16816(float* d, const uint4& a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}

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

template <class T>
__device__ __forceinline__ T ld_code(const uint8_t* p) {
  return __ldg(reinterpret_cast<const T*>(p));
}
__device__ __forceinline__ uint32_t word_of(const uint4& v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}
__device__ __forceinline__ uint32_t word_of(const uint2& v, int i) { return i == 0 ? v.x : v.y; }
__device__ __forceinline__ uint32_t word_of(uint32_t v, int) { return v; }
__device__ __forceinline__ void zero(uint4& v) { v = make_uint4(0, 0, 0, 0); }
__device__ __forceinline__ void zero(uint2& v) { v = make_uint2(0, 0); }
__device__ __forceinline__ void zero(uint32_t& v) { v = 0; }

// The codes a lane holds of its warp's 16 positions.  With t = lane % 4 and
// g = lane / 4: of positions g and g + 8 the D/4 channels of K from t D/4 on
// (the lane's share of the B fragments of q k^T, whose order of channels is
// free); of positions 2t, 2t + 1, 2t + 8, 2t + 9 the D/8 channels of V from
// g D/8 on (its share of the B fragments of w v: channel g D/8 + i is column
// g of block i).  So every code goes from memory to its lane's registers
// and no shared memory is needed; quads (K) and octets (V) of lanes read the
// 64 contiguous bytes of a head row.
template <int D>
struct Raw {
  typename Vec<D / 8>::type k[2];
  typename Vec<D / 16>::type v[4];
  uint32_t km[2], vm[4];
};

// The slot of position p (lanes 0..15 of a warp), -1 when there is none.
__device__ __forceinline__ int attn_slot(const AttnArgs& a, const int32_t* row, int p, int end, bool count) {
  if (p >= end) return -1;
  const int32_t s = __ldg(row + p);
  if (s >= 0 && s < a.num_slots) return s;
  if (count) bump(a.stats, SPEC_STAT_BAD_REQUEST);
  return -1;
}

template <int D>
__device__ __forceinline__ void load_raw(Raw<D>& r, const uint8_t* head, int64_t slot_stride, int slot, int lane) {
  const int t = lane & 3, g = lane >> 2;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int s = __shfl_sync(0xffffffffu, slot, g + 8 * j);
    zero(r.k[j]);
    r.km[j] = 0;
    if (s >= 0) {
      const uint8_t* p = head + s * slot_stride;
      r.k[j] = ld_code<typename Vec<D / 8>::type>(p + t * (D / 8));
      r.km[j] = __ldg(reinterpret_cast<const uint32_t*>(p + D + (t * (D / 4) / kKv4Group) * 4));
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int s = __shfl_sync(0xffffffffu, slot, 2 * t + (j & 1) + 8 * (j >> 1));
    zero(r.v[j]);
    r.vm[j] = 0;
    if (s >= 0) {
      const uint8_t* p = head + s * slot_stride;
      r.v[j] = ld_code<typename Vec<D / 16>::type>(p + D / 2 + g * (D / 16));
      r.vm[j] = __ldg(reinterpret_cast<const uint32_t*>(p + D + D / 8 + (g * (D / 8) / kKv4Group) * 4));
    }
  }
}

// Shared memory of a CTA: q in the order of the A fragments, the warps' row
// statistics, and the warps' weighted values of 16 rows at a time (rows 16
// floats longer than D and 4 floats of padding per 32 channels, so the
// fragment's stores spread over the banks).
template <int D, int MT>
struct AttShared {
  static constexpr int kRow = D + 16;
  uint4 q[MT][D / 16][32];
  float c[16 * MT];  // factor of a row's scores
  float m[kAttWarps][16 * MT], l[kAttWarps][16 * MT];
  float o[kAttWarps][16][kRow];
};

__device__ __forceinline__ int padded(int ch) { return ch + (ch >> 5) * 4; }

// Query rows [r0, r0 + 16 MT) of (b, h) into shared memory: a warp per row.
template <int D, int MT>
__device__ void load_q(const AttnArgs& a, AttShared<D, MT>& sh, int b, int h, int r0, int rows) {
  constexpr int per = D / 32;  // channels of a lane: [lane per, + per)
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int r = warp; r < 16 * MT; r += kAttWarps) {
    float x[per];
#pragma unroll
    for (int j = 0; j < per; ++j) x[j] = 0.0f;
    if (r < rows) {
      const int row = r0 + r, n = attn_node(a, row);
      const uint16_t* src = a.q + (static_cast<int64_t>(b) * a.N + n) * a.q_stride +
                            static_cast<int64_t>(h * a.G + row - n * a.G) * D + lane * per;
      if (per == 4) {
        const uint2 w = __ldg(reinterpret_cast<const uint2*>(src));
        x[0] = bf16_lo(w.x);
        x[1] = bf16_hi(w.x);
        x[per - 2] = bf16_lo(w.y);
        x[per - 1] = bf16_hi(w.y);
      } else {
        const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(src));
        x[0] = bf16_lo(w);
        x[1] = bf16_hi(w);
      }
    }
    float mx = 0.0f;
#pragma unroll
    for (int j = 0; j < per; ++j) mx = fmaxf(mx, fabsf(x[j]));
    mx = warp_max(mx);
    // 2^e <= mx < 2^(e+1) for a normal mx; rows of zeros or subnormals are
    // taken times 2^126
    const int e = mx > 0.0f && isfinite(mx) ? static_cast<int>(__float_as_uint(mx) >> 23) - 127 : 0;
    const float down = __uint_as_float(static_cast<uint32_t>(127 - max(e, -126)) << 23);
    if (lane == 0) sh.c[r] = a.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 + max(e, -126)) << 23);
    // channel ch = t D/4 + 4 kk + 2 i + odd: A register 2 i + (row half) of
    // lane 4 (row % 8) + t at step kk
#pragma unroll
    for (int j = 0; j < per; j += 2) {
      const int ch = lane * per + j, t = ch / (D / 4), kk = ch % (D / 4) / 4, i = ch % 4 / 2;
      const __half2 v = __floats2half2_rn(x[j] * down, x[j + 1] * down);
      reinterpret_cast<uint32_t*>(&sh.q[r / 16][kk][(r % 8) * 4 + t])[2 * i + (r % 16) / 8] = h2_u32(v);
    }
  }
}

template <int D, int MT>
__global__ void __launch_bounds__(kAttThreads, MT == 1 ? 3 : 2) kv4_attention_kernel(const AttnArgs a) {
  pdl_enter();
  constexpr int R = 16 * MT;
  extern __shared__ __align__(16) unsigned char att_sm[];
  AttShared<D, MT>& sh = *reinterpret_cast<AttShared<D, MT>*>(att_sm);
  if (!spec_smem_ok(sizeof(sh), a.stats)) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, t = lane & 3, g = lane >> 2;
  CutSegment* cut = reinterpret_cast<CutSegment*>(a.ws) + blockIdx.x;
  if (threadIdx.x == 0) *cut = CutSegment{0, 0, 0, 0};
  Line line;
  Walk<kTile, kEnds, R> walk;
  if (!attn_stretch<kTile, kEnds, R, kAttThreads>(a, line, walk)) return;
  Part rq;
  while (walk.next(a, rq)) {
    const int b = rq.b, h = rq.h, rt = rq.rt, t0 = rq.t0, t1 = rq.t1;
    const int r0 = rt * R, rows = min(R, rq.nodes * a.G - r0);
    if (rq.bad && h == 0 && rt == 0 && threadIdx.x == 0) bump(a.stats, SPEC_STAT_BAD_REQUEST);

    load_q<D, MT>(a, sh, b, h, r0, rows);
    __syncthreads();
    float cr[MT][2], m[MT][2], l[MT][2], o[MT][D / 8][4];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        cr[mt][i] = sh.c[mt * 16 + g + 8 * i];
        m[mt][i] = neg_inf();
        l[mt][i] = 0.0f;
      }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[mt][i][j] = 0.0f;

    const int32_t* row = a.table + static_cast<int64_t>(b) * a.max_ctx;
    const uint8_t* head = a.pool + static_cast<int64_t>(h) * kv4_head_bytes(D);
    const bool count = h == 0 && rt == 0 && lane < 16;
    // positions of this warp: [tile * 64 + warp * 16, + 16); slots are read
    // two tiles ahead of their use, codes one tile ahead
    auto slot_at = [&](int tile) {
      return tile < t1 ? attn_slot(a, row, tile * kTile + warp * 16 + (lane & 15), rq.end, count) : -1;
    };
    int slot = slot_at(t0), slot_next = slot_at(t0 + 1);
    Raw<D> raw;
    load_raw<D>(raw, head, a.slot_stride, slot, lane);
    for (int tile = t0; tile < t1; ++tile) {
      const unsigned there = __ballot_sync(0xffffffffu, slot >= 0);  // bit i: position i of the 16
      const Raw<D> cur = raw;
      load_raw<D>(raw, head, a.slot_stride, slot_next, lane);
      slot = slot_next;
      slot_next = slot_at(tile + 2);
      if ((there & 0xffffu) == 0) continue;
      float s[MT][2][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[mt][j][i] = 0.0f;
#pragma unroll
      for (int wd = 0; wd < D / 32; ++wd) {  // words of 8 channels: two steps of 16 (4 channels a lane)
        uint32_t kv[2][4];
#pragma unroll
        for (int j = 0; j < 2; ++j)
          dequant4(word_of(cur.k[j], wd), __byte_perm(cur.km[j], 0, 0x1010), __byte_perm(cur.km[j], 0, 0x3232), kv[j]);
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            const uint4 qa = sh.q[mt][wd * 2 + half][lane];
#pragma unroll
            for (int j = 0; j < 2; ++j) mma16816(s[mt][j], qa, kv[j][2 * half], kv[j][2 * half + 1]);
          }
      }
      // scores in units of log2, masked; s[..][j][i]: row g + 8 (i / 2),
      // position 8 j + 2 t + i % 2
      const int p0 = tile * kTile + warp * 16;
      const bool whole = (there & 0xffffu) == 0xffffu && p0 + 16 <= rq.start;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            s[mt][j][i] *= cr[mt][i >> 1];
            if (!whole) {
              const int at = 8 * j + 2 * t + (i & 1), node = p0 + at - rq.start;
              bool see = (there >> at) & 1u;
              if (see && node >= 0) {
                const int r = mt * 16 + g + 8 * (i >> 1), n = attn_node(a, r0 + r);
                see = r < rows && (a.mask ? __ldg(a.mask + (static_cast<int64_t>(b) * a.N + n) * a.N + node) != 0
                                          : node <= n);
              }
              if (!see) s[mt][j][i] = neg_inf();
            }
          }
      uint4 pa[MT];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        float mn[2], al[2];
        bool up = false;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float x = fmaxf(fmaxf(s[mt][0][2 * i], s[mt][0][2 * i + 1]), fmaxf(s[mt][1][2 * i], s[mt][1][2 * i + 1]));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
          mn[i] = fmaxf(m[mt][i], x);
          up = up || mn[i] != m[mt][i];
          const float base_m = mn[i] == neg_inf() ? 0.0f : mn[i];
          al[i] = fast_exp2(m[mt][i] - base_m);
          m[mt][i] = mn[i];
          mn[i] = base_m - kWeightExp;
        }
        if (__any_sync(0xffffffffu, up)) {
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {
            o[mt][i][0] *= al[0];
            o[mt][i][1] *= al[0];
            o[mt][i][2] *= al[1];
            o[mt][i][3] *= al[1];
          }
          l[mt][0] *= al[0];
          l[mt][1] *= al[1];
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            s[mt][j][i] = fast_exp2(s[mt][j][i] - mn[i >> 1]);
            l[mt][i >> 1] += s[mt][j][i];
          }
        pa[mt] = make_uint4(h2_u32(__floats2half2_rn(s[mt][0][0], s[mt][0][1])),
                            h2_u32(__floats2half2_rn(s[mt][0][2], s[mt][0][3])),
                            h2_u32(__floats2half2_rn(s[mt][1][0], s[mt][1][1])),
                            h2_u32(__floats2half2_rn(s[mt][1][2], s[mt][1][3])));
      }
      const uint32_t st0 = __byte_perm(cur.vm[0], cur.vm[1], 0x5410), lo0 = __byte_perm(cur.vm[0], cur.vm[1], 0x7632);
      const uint32_t st1 = __byte_perm(cur.vm[2], cur.vm[3], 0x5410), lo1 = __byte_perm(cur.vm[2], cur.vm[3], 0x7632);
#pragma unroll
      for (int wd = 0; wd < D / 64; ++wd) {
        // even channels of a word lie in its low half, odd ones in its high
        // half: the pair of positions of a channel is a byte permutation away
#pragma unroll
        for (int odd = 0; odd < 2; ++odd) {
          const uint32_t sel = odd ? 0x7632u : 0x5410u;
          uint32_t v0[4], v1[4];
          dequant4(__byte_perm(word_of(cur.v[0], wd), word_of(cur.v[1], wd), sel), st0, lo0, v0);
          dequant4(__byte_perm(word_of(cur.v[2], wd), word_of(cur.v[3], wd), sel), st1, lo1, v1);
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) mma16816(o[mt][wd * 8 + 2 * j + odd], pa[mt], v0[j], v1[j]);
        }
      }
    }

    // merge the warps
    const bool complete = rq.complete();
    float* part = attn_part(a, blockIdx.x, t0 > 0 ? 0 : 1, R, D);
    if (t0 == 0 && t1 < rq.tiles && threadIdx.x == 0)
      *cut = CutSegment{b, h, rt, line.pieces(static_cast<int>(blockIdx.x), rq.tiles, t1)};
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float x = l[mt][i];
        x += __shfl_xor_sync(0xffffffffu, x, 1);
        x += __shfl_xor_sync(0xffffffffu, x, 2);
        if (t == 0) {
          sh.m[warp][mt * 16 + g + 8 * i] = m[mt][i];
          sh.l[warp][mt * 16 + g + 8 * i] = x;
        }
      }
    __syncthreads();
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      if (mt > 0) __syncthreads();
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = mt * 16 + g + 8 * i;
        float top = sh.m[0][r];
#pragma unroll
        for (int w = 1; w < kAttWarps; ++w) top = fmaxf(top, sh.m[w][r]);
        const float f = m[mt][i] == neg_inf() ? 0.0f : fast_exp2(m[mt][i] - top);
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int c = 0; c < D / 8; c += 4) {
            const int ch = (2 * t + e) * (D / 8) + c;
            *reinterpret_cast<float4*>(&sh.o[warp][g + 8 * i][padded(ch)]) =
                make_float4(o[mt][c][2 * i + e] * f, o[mt][c + 1][2 * i + e] * f, o[mt][c + 2][2 * i + e] * f,
                            o[mt][c + 3][2 * i + e] * f);
          }
      }
      __syncthreads();
      for (int i = threadIdx.x; i < 16 * (D / 4); i += kAttThreads) {
        const int rr = i / (D / 4), ch = (i - rr * (D / 4)) * 4, r = mt * 16 + rr;
        if (r >= rows) continue;
        float top = sh.m[0][r], sum = 0.0f;
#pragma unroll
        for (int w = 1; w < kAttWarps; ++w) top = fmaxf(top, sh.m[w][r]);
        float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < kAttWarps; ++w) {
          const float4 x = *reinterpret_cast<const float4*>(&sh.o[w][rr][padded(ch)]);
          acc.x += x.x;
          acc.y += x.y;
          acc.z += x.z;
          acc.w += x.w;
          if (sh.m[w][r] != neg_inf()) sum += sh.l[w][r] * fast_exp2(sh.m[w][r] - top);
        }
        if (!complete) {
          *reinterpret_cast<float4*>(part + r * D + ch) = acc;
          if (ch == 0) {
            part[R * D + 2 * r] = top;
            part[R * D + 2 * r + 1] = sum;
          }
          continue;
        }
        const float inv = attn_inv(sum);
        const int64_t at = attn_row(a, b, h, r0 + r);
        uint2 v;
        v.x = f_bf16(acc.x * inv) | static_cast<uint32_t>(f_bf16(acc.y * inv)) << 16;
        v.y = f_bf16(acc.z * inv) | static_cast<uint32_t>(f_bf16(acc.w * inv)) << 16;
        *reinterpret_cast<uint2*>(a.out + at * D + ch) = v;
        if (a.lse && ch == 0) a.lse[at] = attn_lse(top, sum, kWeightExp);
      }
    }
    __syncthreads();
  }
}

template <int D, int MT>
int launch_attention(AttnArgs a, int sms, cudaStream_t s) {
  constexpr int R = 16 * MT;
  const size_t smem = sizeof(AttShared<D, MT>);
  auto kernel = kv4_attention_kernel<D, MT>;
  if (smem > 48 * 1024 && cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(smem)) != cudaSuccess) {
    cudaGetLastError();
    return SPEC_ERR_CUDA;
  }
  a.ctas = sms * (MT == 1 ? 3 : 2);
  a.ctas = a.ctas < kMaxCtas ? a.ctas : kMaxCtas;
  launch_k(kernel, static_cast<unsigned>(a.ctas), kAttThreads, smem, s, a);
  launch_merge<D>(a, R, kWeightExp, s);
  return launch_status();
}

// Rows of a row tile here: 16 where they suffice, else 32; 0: more rows than
// that go to the tensor-memory kernel (kv4_tree.cu).
int rows_of(int64_t rows) { return rows <= 16 ? 16 : (rows <= 32 ? 32 : 0); }

}  // namespace
}  // namespace specdec

using namespace specdec;

extern "C" size_t spec_kv4_attention_ws_size(int B, int N, int Hq, int Hkv, int D) {
  if (B < 1 || N < 1 || Hkv < 1 || Hq < Hkv || Hq % Hkv != 0 || spec_kv4_slot_bytes(Hkv, D) < 0) return 0;
  const int64_t rows = static_cast<int64_t>(N) * (Hq / Hkv);
  const int R = rows_of(rows);
  return align256(R == 0 ? attn_ws_bytes(kTreeMaxCtas, kTreeRows, D) : attn_ws_bytes(kMaxCtas, R, D));
}

extern "C" int spec_kv4_attention(int B, int N, int Hq, int Hkv, int D, const void* q, int64_t q_stride,
                                  const void* pool, int64_t num_slots, int64_t slot_stride,
                                  const int32_t* num_nodes_or_null, const int32_t* seq_lens,
                                  const int32_t* req_to_token, int64_t max_ctx, const uint8_t* tree_mask_or_null,
                                  float scale, void* out, float* lse_or_null, int32_t* stats_or_null, void* ws,
                                  size_t ws_bytes, spec_stream_t stream) {
  if (B < 0 || N < 0 || Hkv < 1 || Hq < 1 || Hq % Hkv != 0 || max_ctx < 1 || num_slots < 1 || !isfinite(scale))
    return SPEC_ERR_INVALID_ARG;
  const int64_t row = spec_kv4_slot_bytes(Hkv, D);
  if (row < 0 || N > SPEC_MAX_NODES || Hq > SPEC_KV4_MAX_HEADS * 16 || B > 65535) return SPEC_ERR_UNSUPPORTED;
  if (slot_stride < row || q_stride < static_cast<int64_t>(Hq) * D) return SPEC_ERR_INVALID_ARG;
  if (slot_stride % 16 != 0 || q_stride % 8 != 0 || num_slots > INT32_MAX || max_ctx > INT32_MAX - 2 * kTile)
    return SPEC_ERR_UNSUPPORTED;
  if (B == 0 || N == 0) return SPEC_OK;
  if (!q || !pool || !seq_lens || !req_to_token || !out || !ws) return SPEC_ERR_INVALID_ARG;
  for (const void* p : {q, pool, static_cast<const void*>(out)})
    if ((reinterpret_cast<uintptr_t>(p) & 15) != 0) return SPEC_ERR_UNSUPPORTED;
  if ((reinterpret_cast<uintptr_t>(ws) & 15) != 0) return SPEC_ERR_INVALID_ARG;
  if (ws_bytes < spec_kv4_attention_ws_size(B, N, Hq, Hkv, D)) return SPEC_ERR_WORKSPACE;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return SPEC_ERR_CUDA;
  }
  AttnArgs a{static_cast<const uint16_t*>(q), q_stride, B, N, Hq, Hkv, Hq / Hkv,
             ((1ull << 40) + Hq / Hkv - 1) / (Hq / Hkv), static_cast<const uint8_t*>(pool),
             num_slots, slot_stride, req_to_token, max_ctx, seq_lens, num_nodes_or_null, tree_mask_or_null,
             scale * kLog2e, static_cast<uint16_t*>(out), lse_or_null, static_cast<float*>(ws), 0, stats_or_null};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int R = rows_of(static_cast<int64_t>(N) * a.G);
  if (R == 0) return launch_tree_attention(a, D, sms, s);
  const bool small = R == 16;
  if (D == 128) return small ? launch_attention<128, 1>(a, sms, s) : launch_attention<128, 2>(a, sms, s);
  return small ? launch_attention<64, 1>(a, sms, s) : launch_attention<64, 2>(a, sms, s);
}
