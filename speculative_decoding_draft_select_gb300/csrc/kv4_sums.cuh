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
  int above, upto;  // a launch takes the requests with above < rows a KV head <= upto
  bool count_bad;
};

struct SumReq {
  int start, rows, end;  // row i sees positions p <= start + i; end = start + rows
  bool bad;
};
__device__ __forceinline__ SumReq sum_req(const SumArgs& a, int b) {
  SumReq r;
  r.start = __ldg(a.seq_lens + b);
  r.rows = a.accepted ? __ldg(a.accepted + b) + 1 : a.N;
  r.bad = r.rows < 1 || r.rows > a.N || r.start < 0 || static_cast<int64_t>(r.start) + r.rows > a.max_ctx;
  if (r.bad || r.rows * a.G <= a.above || r.rows * a.G > a.upto) r.start = r.rows = 0;
  r.end = r.start + r.rows;
  return r;
}

// The tensor-memory kernel's entry (kv4_sums_rows.cu).
int launch_sums_rows(const SumArgs& a, int D, int sms, cudaStream_t s);

}  // namespace specdec
