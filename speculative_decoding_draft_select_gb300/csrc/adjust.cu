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
//   list     the tokens of the chunk that have any of these (few)
// The pass itself copies vectors of 16 bytes and writes -inf where the mask
// says so (vectors without an allowed token are not read); the same warp then
// computes the row's listed tokens from the values at hand.  A masked token is
// -inf whatever else holds of it, so the pass leaves every value that is still
// needed, in place too; in place without a mask only the listed tokens are
// touched at all.  (Looking the bits of every vector up in the pass instead
// took 128 instructions a vector where histories crowd: 64-node trees, B=128,
// V=128256, bf16: 890 us.)  Measured there: 750 us for 4.27 GB, 5.7 TB/s; the
// listed tokens take 40 of them, the masks' bits 64, histories 30.
#include <climits>

#include "common.cuh"

namespace specdec {
namespace {

constexpr int kAdjThreads = 256;
constexpr int kAdjWarps = kAdjThreads / 32;
constexpr int kAdjMaxChunk = 4096;  // tokens of a chunk: 16 KB of info, 16 KB of biases
constexpr int kAdjMinChunk = 512;
constexpr int kAdjUnroll = 4;       // 16-byte vectors in flight per lane
constexpr int kAdjFirst = 1;        // listed tokens in flight per lane beside the pass
constexpr int kAdjBatch = 4;        // and behind it
constexpr int kAdjSort = 128;       // more listed tokens than this are put in order

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
  asm volatile("st.global.v4.u32 [%0], {%1,%2,%3,%4};" ::"l"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
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

// Listed tokens of a lane: from the chunk's start (-1: none), their mask words,
// their values.
template <int Q>
struct Listed {
  static constexpr int size = Q;
  int tok[Q];
  uint32_t word[Q];
  float val[Q];
};

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

// The kv (4 or 8) bits of a mask from token t on.  whole: t is a multiple of
// kv, so they lie in one byte; otherwise words past the last that the bits
// touch are not read.
__device__ __forceinline__ uint32_t bits_at(const uint32_t* w, int t, int kv, bool whole) {
  if (whole) {
    const uint32_t b = __ldg(reinterpret_cast<const uint8_t*>(w) + (t >> 3));
    return kv == 8 ? b : (b >> (t & 4)) & 15u;
  }
  const int i = t >> 5, s = t & 31;
  uint32_t v = __ldg(w + i) >> s;
  if (s + kv > 32) v |= __ldg(w + i + 1) << (32 - s);
  return v & ((1u << kv) - 1u);
}

template <int DT>
__global__ void __launch_bounds__(kAdjThreads, 4) adjust_kernel(const AdjArgs a, int chunk) {
  pdl_enter();
  constexpr int esz = DT == SPEC_BF16 ? 2 : 4, kv = Logit<DT>::kVec;
  constexpr uint32_t kAll = (1u << kv) - 1u;
  extern __shared__ __align__(16) uint32_t adj_sm[];
  const int b = blockIdx.x, N = a.N;
  uint32_t* info = adj_sm;                                          // [chunk]
  float* bias = reinterpret_cast<float*>(info + chunk);             // [chunk]
  uint16_t* list = reinterpret_cast<uint16_t*>(bias + (a.M > 0 ? chunk : 0));  // [chunk] tokens with info, from the chunk's start
  int32_t* slot_tok = reinterpret_cast<int32_t*>(list + chunk);     // [N] token of a slot, likewise
  int32_t* slot_head = slot_tok + N;                                // [N] last node that carries it
  uint32_t* slot_info = reinterpret_cast<uint32_t*>(slot_head + N); // [N] its info without the path
  int32_t* next = reinterpret_cast<int32_t*>(slot_info + N);        // [N] node before it in the slot's list
  if (!spec_smem_ok(reinterpret_cast<char*>(a.draft_token ? next + N : slot_tok) - reinterpret_cast<char*>(adj_sm),
                    a.stats))
    return;
  __shared__ int s_slots, s_list, s_sorted, s_twice;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int nodes = N;
  if (a.num_nodes) nodes = min(max(__ldg(a.num_nodes + b), 0), N);
  if (nodes == 0) return;
  const int64_t c0 = static_cast<int64_t>(blockIdx.y) * chunk;
  const int len = static_cast<int>(min(static_cast<int64_t>(chunk), a.V - c0));  // tokens [c0, c0 + len)

  // the chunk's table
  for (int i = tid; i < chunk / 4; i += kAdjThreads) reinterpret_cast<uint4*>(info)[i] = make_uint4(0, 0, 0, 0);
  if (tid == 0) s_slots = s_list = s_sorted = s_twice = 0;
  Penalty pen{1.0f, 0.0f, 0.0f};
  if (a.rep) {
    const float r = __ldg(a.rep + b);
    if (r > 0.0f) pen.rep = r;
    else if (blockIdx.y == 0 && tid == 0) bump(a.stats, SPEC_STAT_BAD_REQUEST);
  }
  if (a.freq) pen.freq = __ldg(a.freq + b);
  if (a.pres) pen.pres = __ldg(a.pres + b);
  __syncthreads();
  // adds `bits` to token t's info; the first to do so lists it
  auto mark = [&](int t, uint32_t bits) {
    const uint32_t old = atomicOr(info + t, bits);
    if ((old & ~kCount) == 0) list[atomicAdd(&s_list, 1)] = static_cast<uint16_t>(t);
    return old;
  };
  if (a.history) {
    int64_t hl = a.hist_len ? __ldg(a.hist_len + b) : a.max_hist;
    if (hl < 0 || hl > a.max_hist) {
      if (blockIdx.y == 0 && tid == 0) bump(a.stats, SPEC_STAT_BAD_REQUEST);
      hl = hl < 0 ? 0 : a.max_hist;
    }
    const int64_t pl = a.prompt_len ? __ldg(a.prompt_len + b) : 0;
    const int32_t* h = a.history + b * a.max_hist;
    auto entry = [&](int32_t id, int64_t i) {
      const int64_t t = id - c0;
      if (t >= 0 && t < len) {
        mark(static_cast<int>(t), kSeen);
        if (i >= pl) atomicAdd(info + t, 1u);
      }
    };
    const int64_t quads = (reinterpret_cast<uintptr_t>(h) & 15) == 0 ? hl / 4 : 0;
#pragma unroll 2
    for (int64_t i = tid; i < quads; i += kAdjThreads) {
      const int4 v = __ldg(reinterpret_cast<const int4*>(h) + i);
      entry(v.x, 4 * i);
      entry(v.y, 4 * i + 1);
      entry(v.z, 4 * i + 2);
      entry(v.w, 4 * i + 3);
    }
    for (int64_t i = 4 * quads + tid; i < hl; i += kAdjThreads) entry(__ldg(h + i), i);
  }
  if (a.M > 0) {
    const int32_t* ids = a.bias_ids + static_cast<int64_t>(b) * a.M;
    const float* vals = a.bias_vals + static_cast<int64_t>(b) * a.M;
    for (int i = tid; i < a.M; i += kAdjThreads) {
      const int64_t t = __ldg(ids + i) - c0;
      if (t < 0 || t >= len) continue;
      if (mark(static_cast<int>(t), kBias) & kBias) s_twice = 1;
      bias[t] = __ldg(vals + i);
    }
    __syncthreads();
    // an id listed more than once: its first entry adds them in list order
    for (int i = s_twice ? tid : a.M; i < a.M; i += kAdjThreads) {
      const int32_t id = __ldg(ids + i);
      const int64_t t = id - c0;
      if (t < 0 || t >= len) continue;
      bool first = true;
      for (int j = 0; j < i && first; ++j) first = __ldg(ids + j) != id;
      if (!first) continue;
      float s = __ldg(vals + i);
      for (int j = i + 1; j < a.M; ++j)
        if (__ldg(ids + j) == id) s = __fadd_rn(s, __ldg(vals + j));
      bias[t] = s;
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
      const uint32_t old = mark(static_cast<int>(t), kPath);
      if (!(old & kPath)) {
        const int j = atomicAdd(&s_slots, 1);
        if (spec_in(j, N, a.stats)) {
          slot_tok[j] = static_cast<int32_t>(t);
          slot_info[j] = old;
          slot_head[j] = -1;
        }
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
  const int listed = s_list;
  if (listed > kAdjSort) {
    // where histories crowd, the list in the order of the tokens (by 32): its
    // accesses then share sectors (V=32000, 16 rows, 8000 ids of history: 69 us
    // without, 62 with)
    for (int t = tid; t < chunk; t += kAdjThreads) {
      const bool has = info[t] != 0;
      const uint32_t votes = __ballot_sync(0xffffffffu, has);
      int at = 0;
      if (lane == 0) at = atomicAdd(&s_sorted, __popc(votes));
      at = __shfl_sync(0xffffffffu, at, 0) + __popc(votes & ((1u << lane) - 1u));
      if (has && spec_in(at, chunk, a.stats)) list[at] = static_cast<uint16_t>(t);
    }
    __syncthreads();
  }
  const bool in_place = a.in == a.out;

  // rows: a warp takes a part of a row at a time (a whole chunk when there are
  // rows enough for the warps; smaller parts to even five rows out over eight
  // warps cost more than they gave: 63 us against 59)
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
        if (blockIdx.y == 0 && p0 == 0 && lane == 0) bump(a.stats, SPEC_STAT_BAD_REQUEST);
      } else if (r >= 0) {
        ok = reinterpret_cast<const uint32_t*>(a.allowed) + r * words + c0 / 32;
      }
    }
    // The row's listed tokens, several a lane at a time: begin loads their
    // values and mask words, finish computes and stores them.  The first ones
    // are loaded before the pass, whose stores leave these values as they are
    auto begin = [&](auto& x, int first) {
#pragma unroll
      for (int q = 0; q < x.size; ++q) {
        const int i = first + 32 * q;
        x.tok[q] = i < listed ? list[i] : -1;
        if (x.tok[q] < p0 || x.tok[q] >= p1) x.tok[q] = -1;
        const int at = x.tok[q] < 0 ? p0 : x.tok[q];
        x.word[q] = ok ? __ldg(ok + (at >> 5)) : ~0u;
        if (x.tok[q] >= 0) x.val[q] = adj_load<DT>(in, at);
      }
    };
    auto finish = [&](auto& x) {
#pragma unroll
      for (int q = 0; q < x.size; ++q) {
        const int t = x.tok[q];
        if (t < 0 || !((x.word[q] >> (t & 31)) & 1u)) continue;  // masked: -inf already
        uint32_t e = info[t];
        if (e & kPath) {
          const int j = static_cast<int>(e & ~kPath);
          if (!spec_in(j, N, a.stats)) continue;
          e = slot_info[j];
          uint32_t extra = 0;
          for (int m = slot_head[j]; m >= 0; m = next[m]) {
            if (!spec_in(m, N, a.stats)) break;
            extra += a.tree_mask ? (__ldg(a.tree_mask + row * N + m) != 0 ? 1u : 0u) : (m <= n ? 1u : 0u);
          }
          if (extra) e = (e | kSeen) + extra;
        }
        adj_store<DT>(out, t, adj_value(x.val[q], e, (e & kBias) ? bias[t] : 0.0f, pen));
      }
    };
    Listed<kAdjFirst> early;
    begin(early, lane);
    auto masked = [&](int t) { return ok && !((__ldg(ok + (t >> 5)) >> (t & 31)) & 1u); };
    if (!in_place || ok) {
      auto one = [&](int t) {
        if (masked(t)) adj_store<DT>(out, t, neg_inf());
        else if (DT == SPEC_BF16) reinterpret_cast<uint16_t*>(out)[t] = reinterpret_cast<const uint16_t*>(in)[t];
        else reinterpret_cast<uint32_t*>(out)[t] = reinterpret_cast<const uint32_t*>(in)[t];
      };
      // aligned span of the part; rows whose input and output are aligned
      // differently go element by element
      const int ha = static_cast<int>(((16 - ((reinterpret_cast<uintptr_t>(in) + p0 * esz) & 15)) & 15) / esz);
      const bool same = ((reinterpret_cast<uintptr_t>(in) ^ reinterpret_cast<uintptr_t>(out)) & 15) == 0;
      const int head = same ? min(ha, p1 - p0) : p1 - p0;
      const int nvec = (p1 - p0 - head) / kv;
      const int v0 = p0 + head;
      const bool whole = (v0 & (kv - 1)) == 0;
      // elements before and behind the vectors: fewer than kv each, loaded
      // ahead of the pass (after it, each of the two cost its own latencies)
      int edge = -1;
      uint32_t edge_word = ~0u, edge_bits = 0;
      if (same) {
        if (lane < 8) edge = p0 + lane < v0 ? p0 + lane : -1;
        else if (lane < 16) edge = v0 + nvec * kv + lane - 8 < p1 ? v0 + nvec * kv + lane - 8 : -1;
        if (edge >= 0) {
          if (ok) edge_word = __ldg(ok + (edge >> 5));
          edge_bits = DT == SPEC_BF16 ? reinterpret_cast<const volatile uint16_t*>(in)[edge]
                                      : reinterpret_cast<const volatile uint32_t*>(in)[edge];
        }
      } else {
        for (int t = p0 + lane; t < p1; t += 32) one(t);
      }
      uint32_t keep[kAdjUnroll], later[kAdjUnroll];  // mask bits of these vectors, of the next ones
      auto load_bits = [&](int i0, uint32_t* k) {
#pragma unroll
        for (int q = 0; q < kAdjUnroll; ++q) {
          const int i = i0 + q * 32;
          k[q] = ok && i < nvec ? bits_at(ok, v0 + i * kv, kv, whole) : kAll;
        }
      };
      load_bits(lane, later);
      for (int i0 = lane; i0 < nvec; i0 += 32 * kAdjUnroll) {
        uint4 raw[kAdjUnroll];
#pragma unroll
        for (int q = 0; q < kAdjUnroll; ++q) {
          const int i = i0 + q * 32;
          keep[q] = later[q];
          if (i < nvec && keep[q] != 0) raw[q] = ld_plain(in + (v0 + i * kv) * esz);
        }
        load_bits(i0 + 32 * kAdjUnroll, later);
#pragma unroll
        for (int q = 0; q < kAdjUnroll; ++q) {
          const int i = i0 + q * 32;
          if (i >= nvec || (in_place && keep[q] == kAll)) continue;
          uint4 v = raw[q];
          if (keep[q] != kAll) {
            if (keep[q] == 0) v = neg_inf_vec<DT>();
            uint32_t w[4] = {v.x, v.y, v.z, v.w};
            if (DT == SPEC_BF16) {
#pragma unroll
              for (int j = 0; j < 4; ++j) {  // bytes of the value, or of two -inf
                const uint32_t k2 = keep[q] >> (2 * j);
                w[j] = __byte_perm(w[j], 0xff80ff80u, 0x7654u - (k2 & 1u) * 0x44u - ((k2 >> 1) & 1u) * 0x4400u);
              }
            } else {
#pragma unroll
              for (int j = 0; j < 4; ++j)
                if (!(keep[q] & (1u << j))) w[j] = 0xff800000u;
            }
            v = make_uint4(w[0], w[1], w[2], w[3]);
          }
          st_vec(out + static_cast<int64_t>(v0 + i * kv) * esz, v);
        }
      }
      if (edge >= 0) {
        const bool drop = !((edge_word >> (edge & 31)) & 1u);
        if (DT == SPEC_BF16) reinterpret_cast<uint16_t*>(out)[edge] = drop ? 0xff80u : edge_bits;
        else reinterpret_cast<uint32_t*>(out)[edge] = drop ? 0xff800000u : edge_bits;
      }
      __syncwarp();
    }
    finish(early);
    for (int first = lane + 32 * kAdjFirst; first < listed; first += 32 * kAdjBatch) {
      Listed<kAdjBatch> more;
      begin(more, first);
      finish(more);
    }
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
  if (B == 0) return SPEC_OK;
  if (allowed_or_null && (mask_rows < 1 || (!allowed_row_or_null && mask_rows < static_cast<int64_t>(B) * N)))
    return SPEC_ERR_INVALID_ARG;
  if (max_bias > 0 && (!bias_ids_or_null || !bias_vals_or_null)) return SPEC_ERR_INVALID_ARG;
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
  // the largest chunk that gives 1000 CTAs (608 are resident): a chunk scans
  // the history once, but the one that holds the frequent ids has to be short
  // beside the whole (B=64, V=32000, 16 rows: 62 us at 2048 tokens, 87 at 4096
  // and 73 at 1024; B=128, V=128256, 64 rows: 757 at 4096, 795 at 2048)
  int chunk = kAdjMaxChunk;
  while (chunk > kAdjMinChunk && static_cast<int64_t>(B) * ((V + chunk - 1) / chunk) < 1000) chunk /= 2;
  const size_t smem = sizeof(uint32_t) * (static_cast<size_t>(chunk) * (max_bias > 0 ? 2 : 1) + chunk / 2 +
                                          (draft_token_or_null ? 4 * static_cast<size_t>(N) : 0));
  if (!(dtype == SPEC_BF16 ? allow_smem<adjust_kernel<SPEC_BF16>>(smem) : allow_smem<adjust_kernel<SPEC_F32>>(smem)))
    return SPEC_ERR_CUDA;
  auto kernel = dtype == SPEC_BF16 ? adjust_kernel<SPEC_BF16> : adjust_kernel<SPEC_F32>;
  // chunks in order, each for all requests: frequent ids crowd at the front of a
  // vocabulary, and the CTAs with the most to do should not come last
  const dim3 grid(static_cast<unsigned>(B), static_cast<unsigned>((V + chunk - 1) / chunk));
  launch_k(kernel, grid, kAdjThreads, smem, reinterpret_cast<cudaStream_t>(stream), a, chunk);
  return launch_status();
}
