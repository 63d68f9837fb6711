// The 4-bit KV cache: append (quantise and store) and gather (read back).
//
// zero-to-sglang ch.10 "Speculative decoding (code walk-through)" 5.2: the
// verify step writes the K and V of every tree node into the cache slots that
// were allocated before drafting.  Token (b, n) lies at logical position
// seq_lens[b] + n, physical slot req_to_token[b][position], the addressing of
// spec_compact_slots, which moves these rows as opaque bytes.
//
// A group of 32 channels x_0..x_31 of one K or V head row becomes
//   lo = fp16(min x), step = fp16((max x - min x) * fp32(1/15)),
//   code = clamp(rint((x - lo) * fp32(1 / step)), 0, 15)  (0 if step is 0),
// all in fp32 with each operation rounded once: asymmetric codes, since K has
// channels with a large mean; one (step, lo) per 32 channels costs 1 bit a
// channel and makes a group's codes one 16-byte vector.
//
// Both directions are one pass over their bytes: a quad of lanes per group, 8
// channels a lane, so the loads of a warp are 512 contiguous bytes (bf16)
// and the minimum and maximum are two shuffles.  Bound by bandwidth (and by
// launch latency at one token a request).
#include "kv4.cuh"

namespace specdec {
namespace {

constexpr int kKvThreads = 256;

// Where item `it` (a quad) works: the token's slot and its group.
struct Kv4Item {
  int b, n, kv, h, g;  // request, node, 0 = K / 1 = V, head, group of the head row
};

__device__ __forceinline__ Kv4Item kv4_item(uint32_t it, uint32_t N, uint32_t Hkv, uint32_t G) {
  Kv4Item r;
  const uint32_t per_kv = Hkv * G;
  const uint32_t tok = it / (2 * per_kv);
  uint32_t rest = it - tok * 2 * per_kv;
  r.kv = rest >= per_kv;
  rest -= r.kv ? per_kv : 0;
  r.h = static_cast<int>(rest / G);
  r.g = static_cast<int>(rest - r.h * G);
  r.b = static_cast<int>(tok / N);
  r.n = static_cast<int>(tok - r.b * N);
  return r;
}

// The slot of token (b, n), or -1 when its position or slot is out of range.
__device__ __forceinline__ int kv4_slot(int b, int n, const int32_t* __restrict__ seq_lens,
                                        const int32_t* __restrict__ req_to_token, int64_t max_ctx, int64_t num_slots) {
  const int64_t sl = __ldg(seq_lens + b);
  if (sl < 0 || sl + n >= max_ctx) return -1;
  const int32_t slot = __ldg(req_to_token + b * max_ctx + sl + n);
  return slot >= 0 && slot < num_slots ? slot : -1;
}

template <int DT>
__global__ void __launch_bounds__(kKvThreads)
    kv4_append_kernel(uint32_t items, int N, int Hkv, int G, const void* __restrict__ k, const void* __restrict__ v,
                      int64_t k_stride, int64_t v_stride, const int32_t* __restrict__ num_nodes,
                      const int32_t* __restrict__ seq_lens, const int32_t* __restrict__ req_to_token, int64_t max_ctx,
                      uint8_t* __restrict__ pool, int64_t num_slots, int64_t slot_stride,
                      int32_t* __restrict__ stats) {
  pdl_enter();
  constexpr int esz = DT == SPEC_BF16 ? 2 : 4;
  const uint32_t it = blockIdx.x * (kKvThreads / 4) + (threadIdx.x >> 2);
  const int sub = threadIdx.x & 3;
  const bool in = it < items;  // a quad is in or out as a whole
  const Kv4Item w = kv4_item(in ? it : 0, N, Hkv, G);
  const int64_t tok = static_cast<int64_t>(w.b) * N + w.n;
  const char* src = static_cast<const char*>(w.kv ? v : k) +
                    (tok * (w.kv ? v_stride : k_stride) + (static_cast<int64_t>(w.h) * G + w.g) * kKv4Group + sub * 8) * esz;
  float x[8];
  if (DT == SPEC_BF16) {
    unpack<SPEC_BF16>(ld_stream(src), x);
  } else {
    unpack<SPEC_F32>(ld_stream(src), x);
    unpack<SPEC_F32>(ld_stream(src + 16), x + 4);
  }
  const bool live = in && w.n < kv4_nodes(num_nodes, w.b, N);
  const int slot = live ? kv4_slot(w.b, w.n, seq_lens, req_to_token, max_ctx, num_slots) : -1;
  float mn = kKv4Limit, mx = -kKv4Limit;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    x[j] = isnan(x[j]) ? 0.0f : fminf(fmaxf(x[j], -kKv4Limit), kKv4Limit);
    mn = fminf(mn, x[j]);
    mx = fmaxf(mx, x[j]);
  }
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  }
  const __half lo = __float2half_rn(mn);
  const __half step = __float2half_rn(__fmul_rn(__fsub_rn(mx, mn), 1.0f / 15.0f));
  const float lof = __half2float(lo), stf = __half2float(step);
  const float inv = stf > 0.0f ? __frcp_rn(stf) : 0.0f;
  uint32_t word = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float c = fminf(fmaxf(rintf(__fmul_rn(__fsub_rn(x[j], lof), inv)), 0.0f), 15.0f);
    word |= static_cast<uint32_t>(c) << (4 * (j >> 1) + 16 * (j & 1));
  }
  if (slot < 0) {
    // one count per token: its first quad's first lane
    if (live && w.kv == 0 && w.h == 0 && w.g == 0 && sub == 0) bump(stats, SPEC_STAT_BAD_REQUEST);
    return;
  }
  const int D = G * kKv4Group;
  uint8_t* row = pool + slot * slot_stride + static_cast<int64_t>(w.h) * kv4_head_bytes(D);
  *reinterpret_cast<uint32_t*>(row + w.kv * (D / 2) + w.g * 16 + sub * 4) = word;
  if (sub == 0)
    *reinterpret_cast<uint32_t*>(row + D + w.kv * (D / 8) + w.g * 4) =
        static_cast<uint32_t>(__half_as_ushort(step)) | (static_cast<uint32_t>(__half_as_ushort(lo)) << 16);
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {  // a in the low half
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}

template <int DT>
__global__ void __launch_bounds__(kKvThreads)
    kv4_gather_kernel(uint32_t items, int N, int Hkv, int G, const uint8_t* __restrict__ pool, int64_t num_slots,
                      int64_t slot_stride, const int32_t* __restrict__ num_nodes,
                      const int32_t* __restrict__ seq_lens, const int32_t* __restrict__ req_to_token, int64_t max_ctx,
                      void* __restrict__ k, void* __restrict__ v, int32_t* __restrict__ stats) {
  pdl_enter();
  constexpr int esz = DT == SPEC_BF16 ? 2 : 4;
  const uint32_t it = blockIdx.x * (kKvThreads / 4) + (threadIdx.x >> 2);
  const int sub = threadIdx.x & 3;
  if (it >= items) return;
  const Kv4Item w = kv4_item(it, N, Hkv, G);
  if (w.n >= kv4_nodes(num_nodes, w.b, N)) return;
  const int slot = kv4_slot(w.b, w.n, seq_lens, req_to_token, max_ctx, num_slots);
  const int D = G * kKv4Group;
  float x[8];
  if (slot < 0) {
    if (w.kv == 0 && w.h == 0 && w.g == 0 && sub == 0) bump(stats, SPEC_STAT_BAD_REQUEST);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = 0.0f;
  } else {
    const uint8_t* row = pool + slot * slot_stride + static_cast<int64_t>(w.h) * kv4_head_bytes(D);
    const uint32_t word = __ldg(reinterpret_cast<const uint32_t*>(row + w.kv * (D / 2) + w.g * 16 + sub * 4));
    const uint32_t meta = __ldg(reinterpret_cast<const uint32_t*>(row + D + w.kv * (D / 8) + w.g * 4));
    const float st = __half2float(__ushort_as_half(static_cast<unsigned short>(meta & 0xffffu)));
    const float lo = __half2float(__ushort_as_half(static_cast<unsigned short>(meta >> 16)));
#pragma unroll
    for (int j = 0; j < 8; ++j)  // code * step is exact (15 bits), so the sum is the one rounding
      x[j] = __fmaf_rn(static_cast<float>((word >> (4 * (j >> 1) + 16 * (j & 1))) & 15u), st, lo);
  }
  const int64_t tok = static_cast<int64_t>(w.b) * N + w.n;
  char* dst = static_cast<char*>(w.kv ? v : k) +
              ((tok * Hkv + w.h) * static_cast<int64_t>(G) + w.g) * kKv4Group * esz + sub * 8 * esz;
  if (DT == SPEC_BF16) {
    *reinterpret_cast<uint4*>(dst) = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                                                pack_bf16(x[6], x[7]));
  } else {
    *reinterpret_cast<float4*>(dst) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4*>(dst + 16) = make_float4(x[4], x[5], x[6], x[7]);
  }
}

bool misaligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) != 0; }

// The checks that append and gather share; SPEC_OK with *items = 0 means
// there is nothing to do.
int kv4_check(int B, int64_t N, int Hkv, int D, int dtype, int64_t max_ctx, int64_t num_slots, int64_t slot_stride,
              int64_t* items) {
  *items = 0;
  if (B < 0 || N < 0 || Hkv < 1 || max_ctx < 1 || num_slots < 1) return SPEC_ERR_INVALID_ARG;
  if (dtype != SPEC_F32 && dtype != SPEC_BF16) return SPEC_ERR_UNSUPPORTED;
  const int64_t row = spec_kv4_slot_bytes(Hkv, D);
  if (row < 0) return SPEC_ERR_UNSUPPORTED;
  if (slot_stride < row) return SPEC_ERR_INVALID_ARG;
  if (slot_stride % 16 != 0 || num_slots > INT32_MAX || max_ctx > INT32_MAX || N > INT32_MAX)
    return SPEC_ERR_UNSUPPORTED;
  const int64_t per = 2 * static_cast<int64_t>(Hkv) * (D / kKv4Group);
  const int64_t tokens = static_cast<int64_t>(B) * N;
  if (tokens > INT32_MAX / per) return SPEC_ERR_UNSUPPORTED;
  *items = tokens * per;
  return SPEC_OK;
}

}  // namespace
}  // namespace specdec

using namespace specdec;

extern "C" int64_t spec_kv4_slot_bytes(int Hkv, int D) {
  if (Hkv < 1 || Hkv > SPEC_KV4_MAX_HEADS || (D != 64 && D != 128)) return -1;
  return static_cast<int64_t>(Hkv) * kv4_head_bytes(D);
}

extern "C" int spec_kv4_append(int B, int64_t N, int Hkv, int D, int dtype, const void* k, int64_t k_stride,
                               const void* v, int64_t v_stride, const int32_t* num_nodes_or_null,
                               const int32_t* seq_lens, const int32_t* req_to_token, int64_t max_ctx, void* pool,
                               int64_t num_slots, int64_t slot_stride, int32_t* stats_or_null, spec_stream_t stream) {
  int64_t items = 0;
  const int e = kv4_check(B, N, Hkv, D, dtype, max_ctx, num_slots, slot_stride, &items);
  if (e != SPEC_OK) return e;
  const int64_t row = static_cast<int64_t>(Hkv) * D;
  if (k_stride < row || v_stride < row) return SPEC_ERR_INVALID_ARG;
  if (items == 0) return SPEC_OK;
  if (!k || !v || !seq_lens || !req_to_token || !pool) return SPEC_ERR_INVALID_ARG;
  const int per16 = dtype == SPEC_BF16 ? 8 : 4;
  if (misaligned16(k) || misaligned16(v) || misaligned16(pool) || k_stride % per16 != 0 || v_stride % per16 != 0)
    return SPEC_ERR_UNSUPPORTED;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const unsigned grid = static_cast<unsigned>((items * 4 + kKvThreads - 1) / kKvThreads);
  auto kernel = dtype == SPEC_BF16 ? kv4_append_kernel<SPEC_BF16> : kv4_append_kernel<SPEC_F32>;
  launch_k(kernel, grid, kKvThreads, 0, s, static_cast<uint32_t>(items), static_cast<int>(N), Hkv, D / kKv4Group, k, v,
           k_stride, v_stride, num_nodes_or_null, seq_lens, req_to_token, max_ctx, static_cast<uint8_t*>(pool),
           num_slots, slot_stride, stats_or_null);
  return launch_status();
}

extern "C" int spec_kv4_gather(int B, int64_t N, int Hkv, int D, int dtype, const void* pool, int64_t num_slots,
                               int64_t slot_stride, const int32_t* num_nodes_or_null, const int32_t* seq_lens,
                               const int32_t* req_to_token, int64_t max_ctx, void* k, void* v, int32_t* stats_or_null,
                               spec_stream_t stream) {
  int64_t items = 0;
  const int e = kv4_check(B, N, Hkv, D, dtype, max_ctx, num_slots, slot_stride, &items);
  if (e != SPEC_OK) return e;
  if (items == 0) return SPEC_OK;
  if (!k || !v || !seq_lens || !req_to_token || !pool) return SPEC_ERR_INVALID_ARG;
  if (misaligned16(k) || misaligned16(v) || misaligned16(pool)) return SPEC_ERR_UNSUPPORTED;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const unsigned grid = static_cast<unsigned>((items * 4 + kKvThreads - 1) / kKvThreads);
  auto kernel = dtype == SPEC_BF16 ? kv4_gather_kernel<SPEC_BF16> : kv4_gather_kernel<SPEC_F32>;
  launch_k(kernel, grid, kKvThreads, 0, s, static_cast<uint32_t>(items), static_cast<int>(N), Hkv, D / kKv4Group,
           static_cast<const uint8_t*>(pool), num_slots, slot_stride, num_nodes_or_null, seq_lens, req_to_token,
           max_ctx, k, v, stats_or_null);
  return launch_status();
}
