// What the two kernels that sum attention weights share: the arguments and a
// request's rows and positions.
#pragma once

#include "kv4_attn.cuh"

namespace specdec {

struct SumArgs {
  const uint16_t* q;
  int64_t q_stride;
  const float* lse;
  const int32_t* path;
  const int32_t* accepted;
  int B, N, Hq, Hkv, G;
  uint64_t g_inv;  // ceil(2^40 / G)
  const uint8_t* pool;
  int64_t num_slots, slot_stride;
  const int32_t* seq_lens;
  const int32_t* table;
  int64_t max_ctx;
  float scale_log2;
  const float* prev;
  float* out;
  int32_t* stats;
  void* ws;         // blocks of rows (RowsBlock) [B, Hkv, blocks of all N G rows]
  int above, upto;  // a launch takes the requests with above < rows a KV head <= upto
};

struct SumReq {
  int start, rows, end;  // row i sees positions p <= start + i; end = start + rows
  bool bad;
};
__device__ __forceinline__ SumReq any_req(const SumArgs& a, int b) {
  SumReq r;
  r.start = __ldg(a.seq_lens + b);
  r.rows = a.accepted ? __ldg(a.accepted + b) + 1 : a.N;
  r.bad = r.rows < 1 || r.rows > a.N || r.start < 0 || static_cast<int64_t>(r.start) + r.rows > a.max_ctx;
  if (r.bad) r.start = r.rows = 0;
  r.end = r.start + r.rows;
  return r;
}
// As the launch takes it: nothing where it goes to the other kernel.
__device__ __forceinline__ SumReq sum_req(const SumArgs& a, int b) {
  SumReq r = any_req(a, b);
  if (r.rows * a.G <= a.above || r.rows * a.G > a.upto) r.start = r.rows = r.end = 0;
  return r;
}

// Up to 128 query rows of a KV head as the tensor-memory kernel reads them: fp16
// rows (slabs of 64 channels, 128-byte swizzle) and 16 columns more (no swizzle:
// 8 rows of 16 bytes are a block of 128 bytes, the second 8 columns behind all
// rows): term z of group g's sum in column 4 z + g, and -lse in units of the
// products, 2^-10 of it, as three terms in columns 12 to 14.  Rows of similar
// size (the common case, fold) are scaled by one power of two: a weight is then
// 2^(S c) with one factor c, and nothing is read per column.  Else every row has
// its own power of two, factor and lse.
constexpr int kRowsBlock = 128;
template <int D>
struct RowsBlock {
  static constexpr int kSlab = kRowsBlock * 128;
  uint8_t q[D / 64 * kSlab];
  uint8_t sums[kRowsBlock * 32];
  float c[kRowsBlock], nl[kRowsBlock];  // factor of a row's products; -lse in units of log2 (-infinity: does not count)
  int row[kRowsBlock];                  // row of the path
  int fold, pad[127];                   // to a multiple of 1024 bytes
};
static_assert(sizeof(RowsBlock<128>) % 1024 == 0 && sizeof(RowsBlock<64>) % 1024 == 0, "blocks lie one after another");

// A position of a stage in shared memory: K's codes, then K's (step, lo); 20
// words (D = 64: 12) apart, which makes all reads free of bank conflicts.
template <int D>
struct Pos {
  static constexpr int kCodes = D / 2, kBytes = D == 128 ? 80 : 48;
};
__device__ __forceinline__ void put_async(unsigned dst, uint64_t src, unsigned size) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(size) : "memory");
}

// The tensor-memory kernel's entry (kv4_sums_rows.cu).
int launch_sums_rows(const SumArgs& a, int D, int sms, cudaStream_t s);

}  // namespace specdec
