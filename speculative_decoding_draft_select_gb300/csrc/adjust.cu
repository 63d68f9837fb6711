// Adjustment of the target logits of every tree node: penalties for repeated
// tokens, biases and grammar masks.
//
// zero-to-sglang ch.10 "Speculative decoding (code walk-through)", 5.1:
// verification uses the processed target probabilities.  This is the part of
// the processing that precedes temperature, top-k and top-p.  For row (b, n)
// and token v, with the request's history (prompt, then answer) and the
// tokens on the path from the root to n as the text so far:
//   x1 = seen ? (x > 0 ? x / rep : x * rep) : x     seen: in the text
//   x2 = x1 - count * freq, less pres if count > 0  count: in the answer part
//   x3 = x2 + bias
//   out = allowed ? x3 : -inf
// in fp32, each operation rounded once (no contraction), rounded to the
// logits' type at the end.
//
// One pass over the logits, bound by their bandwidth.  A CTA owns a chunk of
// the vocabulary of one request and all of its rows, so the history is
// scanned once per chunk and its counts serve N rows from shared memory:
//   info[t]  count (low 29 bits), kSeen, kBias; a token that some node of
//            the tree carries holds kPath and the number of its slot instead
//   bits     one bit per token with a non-zero info
// Most tokens have none: a 16-byte vector of logits whose bits are clear is
// copied (or masked), 8 table entries are never looked at.  Tokens on paths
// differ by row: the pass leaves them as they are and the same warp then
// fixes the row's few path tokens from the slot's list of nodes, so each
// element is computed once even in place.
#include <climits>

#include "common.cuh"

namespace specdec {
namespace {

constexpr int kAdjThreads = 256;
constexpr int kAdjWarps = kAdjThreads / 32;
constexpr int kAdjMaxChunk = 4096;  // tokens of a chunk: 16 KB of info, 16 KB of biases
constexpr int kAdjMinChunk = 512;
constexpr int kAdjUnroll = 4;       // 16-byte vectors in flight per lane

constexpr uint32_t kPath = 1u << 31, kSeen = 1u << 30, kBias = 1u << 29, kCount = kBias - 1;

struct AdjArgs {
  const void* in;
  void* out;
  int N;
  int64_t V;
  const int32_t* num_nodes;
  const int32_t* history;  // [B, max_hist]
  int64_t max_hist;
  const int32_t* hist_len;
  const int32_t* prompt_len;
  const float* rep;
  const float* freq;
  const float* pres;
  const int32_t* draft_token;  // [B, N]
  const uint8_t* tree_mask;    // [B, N, N]
  const int32_t* bias_ids;     // [B, M]
  const float* bias_vals;
  int M;
  const int32_t* allowed;  // [mask_rows, words]
  int64_t mask_rows;
  const int32_t* allowed_row;  // [B, N]
  int32_t* stats;
};

// Reads that the same kernel may write in place (not the read-only path).
__device__ __forceinline__ uint4 ld_plain(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}
__device__ __forceinline__ void st_vec(void* p, const uint4& v) {
  asm volatile("st.global.cs.v4.u32 [%0], {%1,%2,%3,%4};" ::"l"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

template <int DT>
__device__ __forceinline__ float adj_load(const void* p, int64_t i) {
  if (DT == SPEC_BF16)
    return __uint_as_float(static_cast<uint32_t>(static_cast<const volatile uint16_t*>(p)[i]) << 16);
  return static_cast<const volatile float*>(p)[i];
}
__device__ __forceinline__ uint16_t to_bf16(float x) {
  uint16_t r;
  asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(r) : "f"(x));
  return r;
}
template <int DT>
__device__ __forceinline__ void adj_store(void* p, int64_t i, float x) {
  if (DT == SPEC_BF16) static_cast<uint16_t*>(p)[i] = to_bf16(x);
  else static_cast<float*>(p)[i] = x;
}

struct Penalty {
  float rep, freq, pres;
};

__device__ __forceinline__ float adj_value(float x, uint32_t info, float bias, const Penalty& p) {
  if (info & kSeen) x = x > 0.0f ? __fdiv_rn(x, p.rep) : __fmul_rn(x, p.rep);
  const uint32_t c = info & kCount;
  if (c) x = __fsub_rn(__fsub_rn(x, __fmul_rn(static_cast<float>(c), p.freq)), p.pres);
  if (info & kBias) x = __fadd_rn(x, bias);
  return x;
}

// The n (<= 8) bits [t, t + n) of a bit array; words past the last that these
// bits touch are not read.
__device__ __forceinline__ uint32_t bits_at(const uint32_t* w, int t, int n) {
  const int i = t >> 5, s = t & 31;
  uint32_t v = w[i] >> s;
  if (s + n > 32) v |= w[i + 1] << (32 - s);
  return v & ((1u << n) - 1u);
}

template <int DT>
__global__ void __launch_bounds__(kAdjThreads, 4) adjust_kernel(const AdjArgs a, int chunk) {
  pdl_enter();
  constexpr int esz = DT == SPEC_BF16 ? 2 : 4, kv = Logit<DT>::kVec;
  extern __shared__ __align__(16) uint32_t adj_sm[];
  const int b = blockIdx.y, N = a.N;
  uint32_t* info = adj_sm;                                          // [chunk]
  float* bias = reinterpret_cast<float*>(info + chunk);             // [chunk]
  uint32_t* bits = reinterpret_cast<uint32_t*>(bias + (a.M > 0 ? chunk : 0));  // [chunk / 32]
  int32_t* slot_tok = reinterpret_cast<int32_t*>(bits + chunk / 32);  // [N] token of a slot, from the chunk's start
  int32_t* slot_head = slot_tok + N;                                // [N] last node that carries it
  uint32_t* slot_info = reinterpret_cast<uint32_t*>(slot_head + N); // [N] its info without the path
  int32_t* next = reinterpret_cast<int32_t*>(slot_info + N);        // [N] node before it in the slot's list
  if (!spec_smem_ok(reinterpret_cast<char*>(next + (a.draft_token ? N : 0)) - reinterpret_cast<char*>(adj_sm), a.stats))
    return;
  __shared__ int s_slots;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int nodes = N;
  if (a.num_nodes) nodes = min(max(__ldg(a.num_nodes + b), 0), N);
  if (nodes == 0) return;
  const int64_t c0 = static_cast<int64_t>(blockIdx.x) * chunk;
  const int len = static_cast<int>(min(static_cast<int64_t>(chunk), a.V - c0));  // tokens [c0, c0 + len)

  // the chunk's table
  for (int i = tid; i < chunk / 4; i += kAdjThreads) reinterpret_cast<uint4*>(info)[i] = make_uint4(0, 0, 0, 0);
  for (int i = tid; i < chunk / 32; i += kAdjThreads) bits[i] = 0;
  if (tid == 0) s_slots = 0;
  Penalty pen{1.0f, 0.0f, 0.0f};
  if (a.rep) {
    const float r = __ldg(a.rep + b);
    if (r > 0.0f) pen.rep = r;
    else if (blockIdx.x == 0 && tid == 0) bump(a.stats, SPEC_STAT_BAD_REQUEST);
  }
  if (a.freq) pen.freq = __ldg(a.freq + b);
  if (a.pres) pen.pres = __ldg(a.pres + b);
  __syncthreads();
  auto mark = [&](int t) { atomicOr(bits + (t >> 5), 1u << (t & 31)); };
  if (a.history) {
    int64_t hl = a.hist_len ? __ldg(a.hist_len + b) : a.max_hist;
    if (hl < 0 || hl > a.max_hist) {
      if (blockIdx.x == 0 && tid == 0) bump(a.stats, SPEC_STAT_BAD_REQUEST);
      hl = hl < 0 ? 0 : a.max_hist;
    }
    const int64_t pl = a.prompt_len ? __ldg(a.prompt_len + b) : 0;
    const int32_t* h = a.history + b * a.max_hist;
    for (int64_t i = tid; i < hl; i += kAdjThreads) {
      const int64_t t = __ldg(h + i) - c0;
      if (t >= 0 && t < len) {
        if (i >= pl) atomicAdd(info + t, 1u);
        atomicOr(info + t, kSeen);
        mark(static_cast<int>(t));
      }
    }
  }
  if (a.M > 0) {
    const int32_t* ids = a.bias_ids + static_cast<int64_t>(b) * a.M;
    const float* vals = a.bias_vals + static_cast<int64_t>(b) * a.M;
    for (int i = tid; i < a.M; i += kAdjThreads) {
      const int32_t id = __ldg(ids + i);
      const int64_t t = id - c0;
      if (t < 0 || t >= len) continue;
      // an id listed more than once: its first entry adds them in list order
      bool first = true;
      for (int j = 0; j < i && first; ++j) first = __ldg(ids + j) != id;
      if (!first) continue;
      float s = __ldg(vals + i);
      for (int j = i + 1; j < a.M; ++j)
        if (__ldg(ids + j) == id) s = __fadd_rn(s, __ldg(vals + j));
      bias[t] = s;
      atomicOr(info + t, kBias);
      mark(static_cast<int>(t));
    }
  }
  __syncthreads();
  if (a.draft_token) {
    // nodes 1.. (the root is in the history): a slot per distinct token in
    // the chunk, with the list of the nodes that carry it
    const int32_t* tok = a.draft_token + static_cast<int64_t>(b) * N;
    for (int m = 1 + tid; m < nodes; m += kAdjThreads) {
      const int64_t t = __ldg(tok + m) - c0;
      if (t < 0 || t >= len) continue;
      const uint32_t old = atomicOr(info + t, kPath);
      if (!(old & kPath)) {
        const int j = atomicAdd(&s_slots, 1);
        if (spec_in(j, N, a.stats)) {
          slot_tok[j] = static_cast<int32_t>(t);
          slot_info[j] = old;
          slot_head[j] = -1;
        }
        mark(static_cast<int>(t));
      }
    }
    __syncthreads();
    for (int j = tid; j < s_slots; j += kAdjThreads) info[slot_tok[j]] = kPath | static_cast<uint32_t>(j);
    __syncthreads();
    for (int m = 1 + tid; m < nodes; m += kAdjThreads) {
      const int64_t t = __ldg(tok + m) - c0;
      if (t < 0 || t >= len) continue;
      const int j = static_cast<int>(info[t] & ~kPath);
      if (spec_in(j, N, a.stats)) next[m] = atomicExch(slot_head + j, m);
    }
    __syncthreads();
  }
  const int slots = a.draft_token ? s_slots : 0;

  // rows: a warp takes a part of a row at a time (a whole chunk when there
  // are rows enough for the warps)
  int parts = 1;
  while (parts * nodes < kAdjWarps && chunk / (parts * 2) >= 32 * kv) parts *= 2;
  const int psize = chunk / parts;
  const uint32_t words = static_cast<uint32_t>((a.V + 31) / 32);
  for (int u = warp; u < nodes * parts; u += kAdjWarps) {
    const int n = u / parts, p0 = (u - n * parts) * psize, p1 = min(len, p0 + psize);
    if (p0 >= p1) continue;
    const int64_t row = static_cast<int64_t>(b) * N + n;
    const char* in = static_cast<const char*>(a.in) + (row * a.V + c0) * esz;
    char* out = static_cast<char*>(a.out) + (row * a.V + c0) * esz;
    const uint32_t* ok = nullptr;  // this row's allowed ids, from the chunk's start (a multiple of 32)
    if (a.allowed) {
      const int64_t r = a.allowed_row ? __ldg(a.allowed_row + row) : row;
      if (r >= a.mask_rows) {
        if (blockIdx.x == 0 && p0 == 0 && lane == 0) bump(a.stats, SPEC_STAT_BAD_REQUEST);
      } else if (r >= 0) {
        ok = reinterpret_cast<const uint32_t*>(a.allowed) + r * words + c0 / 32;
      }
    }
    auto one = [&](int t) {  // element t of the chunk, unless it is a path token
      const uint32_t e = info[t];
      float x = adj_load<DT>(in, t);
      if (!(e & kPath)) {
        x = adj_value(x, e, (e & kBias) ? bias[t] : 0.0f, pen);
        if (ok && !((__ldg(ok + (t >> 5)) >> (t & 31)) & 1u)) x = neg_inf();
      }
      adj_store<DT>(out, t, x);
    };
    // aligned span of the part; rows whose input and output are aligned
    // differently go element by element
    const int ha = static_cast<int>(((16 - ((reinterpret_cast<uintptr_t>(in) + p0 * esz) & 15)) & 15) / esz);
    const bool same = ((reinterpret_cast<uintptr_t>(in) ^ reinterpret_cast<uintptr_t>(out)) & 15) == 0;
    const int head = same ? min(ha, p1 - p0) : p1 - p0;
    const int nvec = (p1 - p0 - head) / kv;
    const int v0 = p0 + head;
    for (int t = p0 + lane; t < v0; t += 32) one(t);
    for (int i0 = 0; i0 < nvec; i0 += 32 * kAdjUnroll) {
      uint4 raw[kAdjUnroll];
      uint32_t al[kAdjUnroll];
#pragma unroll
      for (int q = 0; q < kAdjUnroll; ++q) {
        const int i = i0 + q * 32 + lane;
        if (i < nvec) raw[q] = ld_plain(in + (v0 + i * kv) * esz);
      }
#pragma unroll
      for (int q = 0; q < kAdjUnroll; ++q) {
        const int i = i0 + q * 32 + lane;
        al[q] = ok && i < nvec ? bits_at(ok, v0 + i * kv, kv) : (1u << kv) - 1u;
      }
#pragma unroll
      for (int q = 0; q < kAdjUnroll; ++q) {
        const int i = i0 + q * 32 + lane;
        if (i >= nvec) continue;
        const int t = v0 + i * kv;
        const uint32_t special = bits_at(bits, t, kv);
        uint32_t keep = al[q];
        uint32_t* w = reinterpret_cast<uint32_t*>(&raw[q]);
        if (special) {
          for (uint32_t left = special; left; left &= left - 1) {
            const int j = __ffs(left) - 1;
            const uint32_t e = info[t + j];
            if (e & kPath) {
              keep |= 1u << j;  // as it is: fixed below
              continue;
            }
            const float bv = (e & kBias) ? bias[t + j] : 0.0f;
            if (DT == SPEC_BF16) {
              const uint32_t word = j < 4 ? (j < 2 ? raw[q].x : raw[q].y) : (j < 6 ? raw[q].z : raw[q].w);
              const float y = adj_value((j & 1) ? bf16_hi(word) : bf16_lo(word), e, bv, pen);
              const uint32_t h = to_bf16(y);
              const uint32_t nw = (j & 1) ? (word & 0xffffu) | (h << 16) : (word & 0xffff0000u) | h;
              if (j < 2) raw[q].x = nw;
              else if (j < 4) raw[q].y = nw;
              else if (j < 6) raw[q].z = nw;
              else raw[q].w = nw;
            } else {
              const uint32_t word = j < 2 ? (j < 1 ? raw[q].x : raw[q].y) : (j < 3 ? raw[q].z : raw[q].w);
              const uint32_t nw = __float_as_uint(adj_value(__uint_as_float(word), e, bv, pen));
              if (j == 0) raw[q].x = nw;
              else if (j == 1) raw[q].y = nw;
              else if (j == 2) raw[q].z = nw;
              else raw[q].w = nw;
            }
          }
        }
        if (keep != (1u << kv) - 1u) {
          if (DT == SPEC_BF16) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              if (!(keep & (1u << (2 * j)))) w[j] = (w[j] & 0xffff0000u) | 0xff80u;
              if (!(keep & (2u << (2 * j)))) w[j] = (w[j] & 0xffffu) | 0xff800000u;
            }
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (!(keep & (1u << j))) w[j] = 0xff800000u;
          }
        }
        st_vec(out + static_cast<int64_t>(t) * esz, raw[q]);
      }
    }
    for (int t = v0 + nvec * kv + lane; t < p1; t += 32) one(t);
    // the row's path tokens; in place, the value read is the one that the
    // pass above wrote back unchanged
    __syncwarp();
    for (int j = lane; j < slots; j += 32) {
      const int t = slot_tok[j];
      if (t < p0 || t >= p1) continue;
      uint32_t e = slot_info[j];
      uint32_t extra = 0;
      for (int m = slot_head[j]; m >= 0; m = next[m]) {
        if (!spec_in(m, N, a.stats)) break;
        extra += a.tree_mask ? (__ldg(a.tree_mask + row * N + m) != 0 ? 1u : 0u) : (m <= n ? 1u : 0u);
      }
      if (extra) e = (e | kSeen) + extra;
      float x = adj_value(adj_load<DT>(in, t), e, (e & kBias) ? bias[t] : 0.0f, pen);
      if (ok && !((__ldg(ok + (t >> 5)) >> (t & 31)) & 1u)) x = neg_inf();
      adj_store<DT>(out, t, x);
    }
    __syncwarp();
  }
}

}  // namespace
}  // namespace specdec

using namespace specdec;

extern "C" int spec_adjust_logits(int B, int N, int64_t V, int dtype, const void* logits, void* out,
                                  const int32_t* num_nodes_or_null, const int32_t* history_or_null, int64_t max_history,
                                  const int32_t* history_lens_or_null, const int32_t* prompt_lens_or_null,
                                  const float* rep_penalty_or_null, const float* freq_penalty_or_null,
                                  const float* pres_penalty_or_null, const int32_t* draft_token_or_null,
                                  const uint8_t* tree_mask_or_null, const int32_t* bias_ids_or_null,
                                  const float* bias_vals_or_null, int max_bias, const int32_t* allowed_or_null,
                                  int64_t mask_rows, const int32_t* allowed_row_or_null, int32_t* stats_or_null,
                                  spec_stream_t stream) {
  if (B < 0 || N < 1 || V < 1 || max_history < 0 || max_bias < 0) return SPEC_ERR_INVALID_ARG;
  if (dtype != SPEC_F32 && dtype != SPEC_BF16) return SPEC_ERR_UNSUPPORTED;
  if (V > SPEC_MAX_VOCAB || N > SPEC_MAX_NODES || B > 65535 || max_history > (1 << 28)) return SPEC_ERR_UNSUPPORTED;
  if (allowed_or_null && (mask_rows < 1 || (!allowed_row_or_null && mask_rows < static_cast<int64_t>(B) * N)))
    return SPEC_ERR_INVALID_ARG;
  if (max_bias > 0 && (!bias_ids_or_null || !bias_vals_or_null)) return SPEC_ERR_INVALID_ARG;
  if (B == 0) return SPEC_OK;
  if (!logits || !out) return SPEC_ERR_INVALID_ARG;
  const unsigned esz = dtype == SPEC_BF16 ? 2 : 4;
  if (reinterpret_cast<uintptr_t>(logits) % esz || reinterpret_cast<uintptr_t>(out) % esz) return SPEC_ERR_INVALID_ARG;
  if (out != logits) {  // in place, or memory of its own
    const uintptr_t i = reinterpret_cast<uintptr_t>(logits), o = reinterpret_cast<uintptr_t>(out);
    const uint64_t size = static_cast<uint64_t>(B) * N * V * esz;
    if ((i < o ? o - i : i - o) < size) return SPEC_ERR_INVALID_ARG;
  }
  AdjArgs a{logits, out, N, V, num_nodes_or_null, max_history > 0 ? history_or_null : nullptr, max_history,
            history_lens_or_null, prompt_lens_or_null, rep_penalty_or_null, freq_penalty_or_null,
            pres_penalty_or_null, draft_token_or_null, tree_mask_or_null, bias_ids_or_null, bias_vals_or_null,
            max_bias, allowed_or_null, mask_rows, allowed_row_or_null, stats_or_null};
  int chunk = kAdjMaxChunk;
  while (chunk > kAdjMinChunk && static_cast<int64_t>(B) * ((V + chunk - 1) / chunk) < 2 * 152) chunk /= 2;
  const size_t smem = sizeof(uint32_t) * (static_cast<size_t>(chunk) * (max_bias > 0 ? 2 : 1) + chunk / 32 +
                                          (draft_token_or_null ? 4 * static_cast<size_t>(N) : 0));
  auto kernel = dtype == SPEC_BF16 ? adjust_kernel<SPEC_BF16> : adjust_kernel<SPEC_F32>;
  if (smem > 48 * 1024 && cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(smem)) != cudaSuccess) {
    cudaGetLastError();
    return SPEC_ERR_CUDA;
  }
  const dim3 grid(static_cast<unsigned>((V + chunk - 1) / chunk), static_cast<unsigned>(B));
  launch_k(kernel, grid, kAdjThreads, smem, reinterpret_cast<cudaStream_t>(stream), a, chunk);
  return launch_status();
}
