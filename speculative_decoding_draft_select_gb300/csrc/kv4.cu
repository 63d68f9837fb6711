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
// Both directions are one pass over their bytes.  A warp takes up to 32 groups
// of one token, so the token's slot is looked up once; a quad of lanes takes a
// group, 8 channels a lane, so the loads of a warp are 512 contiguous bytes
// (bf16), four of them in flight, and the minimum and maximum are two
// shuffles.  Bound by bandwidth (and by launch latency at one token a
// request): 7 prompts of 8191 tokens, 4 heads of 64, fp32, written and read
// back 55 us for 272 MB; 128 trees of 64 nodes, 8 heads of 128, bf16 27 us
// for 88 MB.
#include "kv4.cuh"

namespace specdec {
namespace {

constexpr int kKvThreads = 256;

// A warp's part of a token: which one, its slot, and its first group of the
// token's (K's heads' groups, then V's).
struct Kv4Unit {
  int b, n, slot, first;
  bool live;  // a node of the request
};

// The slot of token (b, n), or -1 when its position or slot is out of range.
__device__ __forceinline__ int kv4_slot(int b, int n, const int32_t* __restrict__ seq_lens,
                                        const int32_t* __restrict__ req_to_token, int64_t max_ctx, int64_t num_slots) {
  const int64_t sl = __ldg(seq_lens + b);
  if (sl < 0 || sl + n >= max_ctx) return -1;
  const int32_t slot = __ldg(req_to_token + b * max_ctx + sl + n);
  return slot >= 0 && slot < num_slots ? slot : -1;
}

__device__ __forceinline__ Kv4Unit kv4_unit(uint32_t unit, uint32_t per_token, uint32_t N, const int32_t* num_nodes,
                                            const int32_t* seq_lens, const int32_t* req_to_token, int64_t max_ctx,
                                            int64_t num_slots, int steps) {
  Kv4Unit u;
  const uint32_t tok = unit / per_token;
  u.first = static_cast<int>(unit - tok * per_token) * (8 * steps);
  u.b = static_cast<int>(tok / N);
  u.n = static_cast<int>(tok - u.b * N);
  u.live = u.n < kv4_nodes(num_nodes, u.b, static_cast<int>(N));
  u.slot = u.live ? kv4_slot(u.b, u.n, seq_lens, req_to_token, max_ctx, num_slots) : -1;
  return u;
}

// Group q of a token (of 2 Hkv D / 32): K or V, head, group of the head row.
template <int D>
struct Kv4Group {
  int kv, h, g;
  __device__ __forceinline__ Kv4Group(int q, int Hkv) {
    constexpr int G = D / kKv4Group;
    kv = q >= Hkv * G;
    const int r = q - (kv ? Hkv * G : 0);
    h = r / G;
    g = r % G;
  }
  __device__ __forceinline__ int channel() const { return h * D + g * kKv4Group; }
  __device__ __forceinline__ int codes() const { return h * kv4_head_bytes(D) + kv * (D / 2) + g * 16; }
  __device__ __forceinline__ int meta() const { return h * kv4_head_bytes(D) + D + kv * (D / 8) + g * 4; }
};

template <int DT, int D, int STEPS>
__global__ void __launch_bounds__(kKvThreads)
    kv4_append_kernel(uint32_t units, uint32_t per_token, int N, int Hkv, const void* __restrict__ k,
                      const void* __restrict__ v, int64_t k_stride, int64_t v_stride,
                      const int32_t* __restrict__ num_nodes, const int32_t* __restrict__ seq_lens,
                      const int32_t* __restrict__ req_to_token, int64_t max_ctx, uint8_t* __restrict__ pool,
                      int64_t num_slots, int64_t slot_stride, int32_t* __restrict__ stats) {
  pdl_enter();
  constexpr int esz = DT == SPEC_BF16 ? 2 : 4;
  const uint32_t unit = blockIdx.x * (kKvThreads / 32) + (threadIdx.x >> 5);
  if (unit >= units) return;
  const int sub = threadIdx.x & 3, quad = (threadIdx.x & 31) >> 2;
  const int groups = 2 * Hkv * (D / kKv4Group);
  const Kv4Unit u = kv4_unit(unit, per_token, N, num_nodes, seq_lens, req_to_token, max_ctx, num_slots, STEPS);
  const int64_t tok = static_cast<int64_t>(u.b) * N + u.n;
  uint4 raw[STEPS][esz / 2];
#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
    const Kv4Group<D> q(min(u.first + i * 8 + quad, groups - 1), Hkv);  // behind the token's last: the last again
    const char* src = static_cast<const char*>(q.kv ? v : k) + (tok * (q.kv ? v_stride : k_stride) + q.channel() + sub * 8) * esz;
    raw[i][0] = ld_stream(src);
    if (DT == SPEC_F32) raw[i][esz / 2 - 1] = ld_stream(src + 16);
  }
  if (u.slot < 0) {
    if (u.live && u.first == 0 && (threadIdx.x & 31) == 0) bump(stats, SPEC_STAT_BAD_REQUEST);  // once per token
    return;
  }
  uint8_t* row = pool + u.slot * slot_stride;
#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
    const int id = u.first + i * 8 + quad;
    const Kv4Group<D> q(min(id, groups - 1), Hkv);
    float x[8];
    if (DT == SPEC_BF16) {
      unpack<SPEC_BF16>(raw[i][0], x);
    } else {
      unpack<SPEC_F32>(raw[i][0], x);
      unpack<SPEC_F32>(raw[i][esz / 2 - 1], x + 4);
    }
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
    if (id < groups) {
      *reinterpret_cast<uint32_t*>(row + q.codes() + sub * 4) = word;
      if (sub == 0)
        *reinterpret_cast<uint32_t*>(row + q.meta()) =
            static_cast<uint32_t>(__half_as_ushort(step)) | (static_cast<uint32_t>(__half_as_ushort(lo)) << 16);
    }
  }
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {  // a in the low half
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}

template <int DT, int D, int STEPS>
__global__ void __launch_bounds__(kKvThreads)
    kv4_gather_kernel(uint32_t units, uint32_t per_token, int N, int Hkv, const uint8_t* __restrict__ pool,
                      int64_t num_slots, int64_t slot_stride, const int32_t* __restrict__ num_nodes,
                      const int32_t* __restrict__ seq_lens, const int32_t* __restrict__ req_to_token, int64_t max_ctx,
                      void* __restrict__ k, void* __restrict__ v, int32_t* __restrict__ stats) {
  pdl_enter();
  constexpr int esz = DT == SPEC_BF16 ? 2 : 4;
  const uint32_t unit = blockIdx.x * (kKvThreads / 32) + (threadIdx.x >> 5);
  if (unit >= units) return;
  const int sub = threadIdx.x & 3, quad = (threadIdx.x & 31) >> 2;
  const int groups = 2 * Hkv * (D / kKv4Group);
  const Kv4Unit u = kv4_unit(unit, per_token, N, num_nodes, seq_lens, req_to_token, max_ctx, num_slots, STEPS);
  if (!u.live) return;
  if (u.slot < 0 && u.first == 0 && (threadIdx.x & 31) == 0) bump(stats, SPEC_STAT_BAD_REQUEST);
  const uint8_t* row = pool + (u.slot < 0 ? 0 : u.slot) * slot_stride;
  const int64_t tok = static_cast<int64_t>(u.b) * N + u.n;
  uint32_t word[STEPS], meta[STEPS];
#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
    const Kv4Group<D> q(min(u.first + i * 8 + quad, groups - 1), Hkv);
    word[i] = meta[i] = 0;  // a token out of range: zeros
    if (u.slot >= 0) {
      word[i] = __ldg(reinterpret_cast<const uint32_t*>(row + q.codes() + sub * 4));
      meta[i] = __ldg(reinterpret_cast<const uint32_t*>(row + q.meta()));
    }
  }
#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
    const int id = u.first + i * 8 + quad;
    if (id >= groups) break;
    const Kv4Group<D> q(id, Hkv);
    const float st = __half2float(__ushort_as_half(static_cast<unsigned short>(meta[i] & 0xffffu)));
    const float lo = __half2float(__ushort_as_half(static_cast<unsigned short>(meta[i] >> 16)));
    float x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)  // code * step is exact (15 bits), so the sum is the one rounding
      x[j] = __fmaf_rn(static_cast<float>((word[i] >> (4 * (j >> 1) + 16 * (j & 1))) & 15u), st, lo);
    char* dst = static_cast<char*>(q.kv ? v : k) + (tok * Hkv * D + q.channel() + sub * 8) * esz;
    if (DT == SPEC_BF16) {
      *reinterpret_cast<uint4*>(dst) = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                                                  pack_bf16(x[6], x[7]));
    } else {
      *reinterpret_cast<float4*>(dst) = make_float4(x[0], x[1], x[2], x[3]);
      *reinterpret_cast<float4*>(dst + 16) = make_float4(x[4], x[5], x[6], x[7]);
    }
  }
}

bool misaligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) != 0; }

// The checks that append and gather share; SPEC_OK with *units = 0 (warps'
// parts of tokens) means there is nothing to do.
int kv4_check(int B, int64_t N, int Hkv, int D, int dtype, int64_t max_ctx, int64_t num_slots, int64_t slot_stride,
              int64_t* units, int64_t* per_token,
              int* steps) {
  *units = 0;
  if (B < 0 || N < 0 || Hkv < 1 || max_ctx < 1 || num_slots < 1) return SPEC_ERR_INVALID_ARG;
  if (dtype != SPEC_F32 && dtype != SPEC_BF16) return SPEC_ERR_UNSUPPORTED;
  const int64_t row = spec_kv4_slot_bytes(Hkv, D);
  if (row < 0) return SPEC_ERR_UNSUPPORTED;
  if (slot_stride < row) return SPEC_ERR_INVALID_ARG;
  if (slot_stride % 16 != 0 || num_slots > INT32_MAX || max_ctx > INT32_MAX || N > INT32_MAX)
    return SPEC_ERR_UNSUPPORTED;
  const int64_t groups = 2 * static_cast<int64_t>(Hkv) * (D / kKv4Group);
  const int64_t tokens = static_cast<int64_t>(B) * N;
  if (tokens > INT32_MAX / groups) return SPEC_ERR_UNSUPPORTED;
  // groups of a warp, 8 a step: as many as the token has, up to four steps; one
  // step where the warps are few and latency is all there is.  8 heads of 128,
  // bf16, append / gather in us with one, two and four steps:
  //   128 tokens   1.8 2.2 3.0 / 1.7 1.9 2.2     2048    6.1  5.5  5.8 /  4.8  4.1  3.7
  //   512          2.6 2.7 3.1 / 2.3 2.2 2.2     8192   20.0 17.5 17.0 / 14.9 11.0  9.3
  //   1024         4.0 4.6 3.9 / 3.3 2.8 2.6     32768  76.6 65.5 60.6 / 64.8 43.6 33.9
  // and of 32768 tokens of 8 groups (2 heads of 64) 10.7 16.4 28.9 / 8.1 8.8
  // 10.1, of 16 groups (4 heads of 64, fp32) 20.3 18.2 29.5 / 16.0 14.7 13.7
  *steps = groups <= 8 || tokens * groups <= 8 * 8192 ? 1 : (groups <= 16 ? 2 : 4);
  *per_token = (groups + 8 * *steps - 1) / (8 * *steps);
  *units = tokens * *per_token;
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
  int64_t units = 0, per_token = 0;
  int steps = 0;
  const int e = kv4_check(B, N, Hkv, D, dtype, max_ctx, num_slots, slot_stride, &units, &per_token, &steps);
  if (e != SPEC_OK) return e;
  const int64_t row = static_cast<int64_t>(Hkv) * D;
  if (k_stride < row || v_stride < row) return SPEC_ERR_INVALID_ARG;
  if (units == 0) return SPEC_OK;
  if (!k || !v || !seq_lens || !req_to_token || !pool) return SPEC_ERR_INVALID_ARG;
  const int per16 = dtype == SPEC_BF16 ? 8 : 4;
  if (misaligned16(k) || misaligned16(v) || misaligned16(pool) || k_stride % per16 != 0 || v_stride % per16 != 0)
    return SPEC_ERR_UNSUPPORTED;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const unsigned grid = static_cast<unsigned>((units + kKvThreads / 32 - 1) / (kKvThreads / 32));
  auto pick = [&](auto one, auto two, auto four) { return steps == 1 ? one : (steps == 2 ? two : four); };
  constexpr int B16 = SPEC_BF16, F32 = SPEC_F32;
  auto kernel =
      dtype == B16
          ? (D == 128 ? pick(kv4_append_kernel<B16, 128, 1>, kv4_append_kernel<B16, 128, 2>, kv4_append_kernel<B16, 128, 4>)
                      : pick(kv4_append_kernel<B16, 64, 1>, kv4_append_kernel<B16, 64, 2>, kv4_append_kernel<B16, 64, 4>))
          : (D == 128 ? pick(kv4_append_kernel<F32, 128, 1>, kv4_append_kernel<F32, 128, 2>, kv4_append_kernel<F32, 128, 4>)
                      : pick(kv4_append_kernel<F32, 64, 1>, kv4_append_kernel<F32, 64, 2>, kv4_append_kernel<F32, 64, 4>));
  launch_k(kernel, grid, kKvThreads, 0, s, static_cast<uint32_t>(units), static_cast<uint32_t>(per_token),
           static_cast<int>(N), Hkv, k, v,
           k_stride, v_stride, num_nodes_or_null, seq_lens, req_to_token, max_ctx, static_cast<uint8_t*>(pool),
           num_slots, slot_stride, stats_or_null);
  return launch_status();
}

extern "C" int spec_kv4_gather(int B, int64_t N, int Hkv, int D, int dtype, const void* pool, int64_t num_slots,
                               int64_t slot_stride, const int32_t* num_nodes_or_null, const int32_t* seq_lens,
                               const int32_t* req_to_token, int64_t max_ctx, void* k, void* v, int32_t* stats_or_null,
                               spec_stream_t stream) {
  int64_t units = 0, per_token = 0;
  int steps = 0;
  const int e = kv4_check(B, N, Hkv, D, dtype, max_ctx, num_slots, slot_stride, &units, &per_token, &steps);
  if (e != SPEC_OK) return e;
  if (units == 0) return SPEC_OK;
  if (!k || !v || !seq_lens || !req_to_token || !pool) return SPEC_ERR_INVALID_ARG;
  if (misaligned16(k) || misaligned16(v) || misaligned16(pool)) return SPEC_ERR_UNSUPPORTED;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const unsigned grid = static_cast<unsigned>((units + kKvThreads / 32 - 1) / (kKvThreads / 32));
  auto pick = [&](auto one, auto two, auto four) { return steps == 1 ? one : (steps == 2 ? two : four); };
  constexpr int B16 = SPEC_BF16, F32 = SPEC_F32;
  auto kernel =
      dtype == B16
          ? (D == 128 ? pick(kv4_gather_kernel<B16, 128, 1>, kv4_gather_kernel<B16, 128, 2>, kv4_gather_kernel<B16, 128, 4>)
                      : pick(kv4_gather_kernel<B16, 64, 1>, kv4_gather_kernel<B16, 64, 2>, kv4_gather_kernel<B16, 64, 4>))
          : (D == 128 ? pick(kv4_gather_kernel<F32, 128, 1>, kv4_gather_kernel<F32, 128, 2>, kv4_gather_kernel<F32, 128, 4>)
                      : pick(kv4_gather_kernel<F32, 64, 1>, kv4_gather_kernel<F32, 64, 2>, kv4_gather_kernel<F32, 64, 4>));
  launch_k(kernel, grid, kKvThreads, 0, s, static_cast<uint32_t>(units), static_cast<uint32_t>(per_token),
           static_cast<int>(N), Hkv, static_cast<const uint8_t*>(pool), num_slots, slot_stride, num_nodes_or_null, seq_lens, req_to_token,
           max_ctx, k, v, stats_or_null);
  return launch_status();
}
