// Eviction of cached positions: requests that have grown past a limit are cut
// to a budget of positions, which keeps the first tokens (sinks), the latest
// ones, and of the rest those whose summed attention is largest.
//
// The cache's rows lie in the slots that req_to_token names, so with pages of
// one token the cut is a relabelling ("EAGLE speculative decoding in four
// parts", ai-infra-handbooks, "Drafting, verification and slots": slots are
// allocated, and freed, by their table); with larger pages the kept rows move
// up, in order, and whole pages are freed.  Sums follow their positions.
//
// Two launches:
//   select   a cluster per request.  Ranks are by a 32-bit key in which floats
//            compare as unsigned integers (NaN as -inf, -0 as 0) and positions
//            that stay in any case lie above every number.  Three counting
//            passes (11, 11 and 10 bits) find the key of the budget's last
//            position; the kept ones are those above it and, of equal ones, the
//            first.  One scan in the positions' order then gives each its place; the slots
//            and sums of the kept are put aside, and once the cluster has read
//            all of the old ones they take the first places.
//   payload  (pages of several tokens) a CTA, or a cluster where there are few,
//            takes a request's rows, a slice of their bytes: it reads kept rows
//            in order, two chunks ahead, and writes them up.  A row only ever
//            moves towards the front: what a chunk overwrites has been read by it
//            or a chunk before, so a barrier between a chunk's reads and its
//            writes is enough.  Slices are independent.
//
// Latency: a chain of counting passes with barriers between.  One request of 1500
// positions takes 13.7k cycles: 3.1k for lengths and keys, 1.9k a pass, 2 x 1.7k for
// the scan, 1k for the copies; the third pass, told by the second that it has all
// keys of its digits, is then left out (7.2 to 6.6 us).  Measured (us): that
// request 6.6; 4 of 60001..131001 to 32768 20 (with clusters of 8 26, and 33 with
// every CTA reading all others' counts); 128 of 16..2048 to 768 with rows of 4096
// bytes in pages of 16 78, of them 69 for 346 MB of payload (0.76 of the copy rate
// for all of the call's bytes).  Without the slots read a chunk ahead the payload
// took twice as long; with a search by halves for the first row that moves 3 more.
#include <climits>

#include "common.cuh"

namespace specdec {
namespace {

constexpr int kSelThreads = 512, kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kMaxCtas = 16;   // of a cluster
constexpr int kSlice = 131072 / kMaxCtas;  // keys of a CTA that stay in shared memory

struct EvictArgs {
  int B, page, budget, limit, sinks, recent;
  const int32_t* seq_lens;
  const float* sums;
  float* sums_out;
  int32_t* table;
  int64_t max_ctx;
  int32_t* kept;
  int32_t* freed;
  int64_t freed_cap;
  int32_t* num_freed;
  int32_t* new_len;
  int32_t* ws_table;  // [B, budget]: slots of the kept positions
  float* ws_sums;     // [B, budget]
  uint8_t* kv;
  int64_t num_slots, bps;
  int32_t* stats;
};

// Length of request b (-1: out of range), and whether it is cut.
__device__ __forceinline__ int evict_len(const EvictArgs& a, int b) {
  const int n = __ldg(a.seq_lens + b);
  return n < 0 || n > a.max_ctx ? -1 : n;
}
__device__ __forceinline__ int pages_of(int n, int page) { return n / page + (n % page != 0); }
// Entries of the freed list that a request of length n adds.
__device__ __forceinline__ int evict_freed(const EvictArgs& a, int n) {
  if (n <= a.limit) return 0;
  return a.page == 1 ? n - a.budget : pages_of(n, a.page) - pages_of(a.budget, a.page);
}

__device__ __forceinline__ uint32_t sum_key(float x) {
  const uint32_t u = __float_as_uint(order_key(x) + 0.0f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
// Whether position p of a request of length n stays in any case.
__device__ __forceinline__ bool evict_stays(const EvictArgs& a, int p, int n) {
  return p < a.sinks || p >= n - a.recent;
}
__device__ __forceinline__ uint32_t evict_key(const EvictArgs& a, const float* sums, int p, int n) {
  return evict_stays(a, p, n) ? ~0u : sum_key(__ldg(sums + p));
}

__device__ __forceinline__ uint4 ld_cluster4(const unsigned* local, unsigned rank) {
  const unsigned s = static_cast<unsigned>(__cvta_generic_to_shared(local));
  unsigned r;
  uint4 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(s), "r"(rank));
  asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(r)
               : "memory");
  return v;
}

__device__ __forceinline__ void st_cluster4(unsigned* local, unsigned rank, const uint4& v) {
  const unsigned s = static_cast<unsigned>(__cvta_generic_to_shared(local));
  unsigned r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(s), "r"(rank));
  asm volatile("st.shared::cluster.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(r), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}

// The sum over the threads before this one.
__device__ __forceinline__ int block_before(int v, int2* sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sh[warp].x = x;
  __syncthreads();
  int before = x - v;
#pragma unroll
  for (int w = 0; w < kSelWarps; ++w)
    if (w < warp) before += sh[w].x;
  return before;
}

struct SelectShared {
  unsigned hist[kBins], total[kBins];  // this CTA's, the cluster's
  int2 scan[kSelWarps];
  int64_t freed[kSelWarps];
  unsigned digit, above;
  int whole;
  int counts[2];  // this CTA's kept above the last key, and equal to it
  uint32_t key[kSlice];
};

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictArgs a, int ctas) {
  pdl_enter();
  extern __shared__ __align__(16) unsigned char evict_sm[];
  SelectShared& sh = *reinterpret_cast<SelectShared*>(evict_sm);
  if (!spec_smem_ok(sizeof(sh), a.stats)) return;
  const int b = blockIdx.x / ctas, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const unsigned rank = ctas > 1 ? cluster_rank() : 0u;

  // entries of the freed list before this request's, and of all requests
  int64_t before = 0, all = 0;
  for (int i = tid; i < a.B; i += kSelThreads) {
    const int f = evict_freed(a, evict_len(a, i));
    all += f;
    if (i < b) before += f;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    before += __shfl_xor_sync(0xffffffffu, before, o);
    all += __shfl_xor_sync(0xffffffffu, all, o);
  }
  if (lane == 0) sh.freed[warp] = before;
  __syncthreads();
  before = 0;
#pragma unroll
  for (int w = 0; w < kSelWarps; ++w) before += sh.freed[w];
  if (blockIdx.x == 0) {
    __syncthreads();
    if (lane == 0) sh.freed[warp] = all;
    __syncthreads();
    if (tid == 0) {
      for (int w = 1; w < kSelWarps; ++w) all += sh.freed[w];
      *a.num_freed = static_cast<int32_t>(all);
    }
  }
  if (b >= a.B) return;  // no request at all: the launch has one cluster for num_freed

  const int n = evict_len(a, b);
  const bool cut = n > a.limit;
  int32_t* kept = a.kept + static_cast<int64_t>(b) * a.budget;
  if (rank == 0 && tid == 0) {
    a.new_len[b] = cut ? a.budget : n;
    if (n < 0) bump(a.stats, SPEC_STAT_BAD_REQUEST);
  }
  const float* sums = a.sums + static_cast<int64_t>(b) * a.max_ctx;
  float* sums_out = a.sums_out + static_cast<int64_t>(b) * a.max_ctx;
  const int step = ctas * kSelThreads, t0 = static_cast<int>(rank) * kSelThreads + tid;  // of the cluster's threads
  if (!cut) {  // the whole cluster leaves
    for (int i = t0; i < a.budget; i += step) kept[i] = -1;
    if (sums_out != sums)
      for (int i = t0; i < n; i += step) sums_out[i] = __ldg(sums + i);
    return;
  }
  int32_t* table = a.table + static_cast<int64_t>(b) * a.max_ctx;
  // this CTA's positions [p0, p0 + mine), a run of each thread's; keys beyond
  // what shared memory holds are computed again in each pass
  const int each = (n + ctas - 1) / ctas;
  const int p0 = min(n, static_cast<int>(rank) * each), mine = min(each, n - p0);
  const int held = min(mine, kSlice);
  constexpr int kAhead = 8;  // loads of a thread in flight
  for (int i = tid; i < held; i += kAhead * kSelThreads) {
    float x[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) x[u] = i + u * kSelThreads < held ? __ldg(sums + p0 + i + u * kSelThreads) : 0.0f;
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int j = i + u * kSelThreads;
      if (j < held) sh.key[j] = evict_stays(a, p0 + j, n) ? ~0u : sum_key(x[u]);
    }
  }
  auto key_at = [&](int i) { return i < held ? sh.key[i] : evict_key(a, sums, p0 + i, n); };
  // visit(key, i) for i = from, from + every, ... below to; kAhead keys at a time
  // where shared memory holds them all
  auto for_keys = [&](int from, int to, int every, auto&& visit) {
    int i = from;
    if (held == mine) {
      for (; i + (kAhead - 1) * every < to; i += kAhead * every) {
        uint32_t k[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) k[u] = sh.key[i + u * every];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) visit(k[u], i + u * every);
      }
    }
    for (; i < to; i += every) visit(key_at(i), i);
  };

  uint32_t prefix = 0;
  int need = a.budget;  // positions still to be taken among those with this prefix
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
    for (int i = tid; i < kBins; i += kSelThreads) sh.hist[i] = 0;
    __syncthreads();
    for_keys(tid, mine, kSelThreads, [&](uint32_t k, int) {
      if (pass == 0 || (k >> (shift + bits)) == prefix) atomicAdd(&sh.hist[(k >> shift) & ((1u << bits) - 1)], 1u);
    });
    if (ctas > 1) cluster_barrier();
    else __syncthreads();
    // each CTA adds its share of the bins up and tells the others
    const unsigned* bins = sh.hist;
    if (ctas > 1) {
      const int quads = kBins / 4 / ctas;
      if (tid < quads) {
        const int at = (static_cast<int>(rank) * quads + tid) * 4;
        uint4 h = make_uint4(0, 0, 0, 0), other[kMaxCtas];  // all loads in flight at once
#pragma unroll
        for (int c = 0; c < kMaxCtas; ++c)
          if (c < ctas) other[c] = ld_cluster4(sh.hist + at, c);
#pragma unroll
        for (int c = 0; c < kMaxCtas; ++c)
          if (c < ctas) h.x += other[c].x, h.y += other[c].y, h.z += other[c].z, h.w += other[c].w;
#pragma unroll
        for (int c = 0; c < kMaxCtas; ++c)
          if (c < ctas) st_cluster4(sh.total + at, c, h);
      }
      bins = sh.total;
      cluster_barrier();
    }
    // bins from the top: a thread's run of four
    constexpr int per = 4;
    static_assert(per * kSelThreads == kBins, "a run of four bins each");
    const uint4 h = *reinterpret_cast<const uint4*>(bins + kBins - per * (tid + 1));
    const unsigned cnt[per] = {h.w, h.z, h.y, h.x};
    const int mine_sum = static_cast<int>(h.x + h.y + h.z + h.w);
    int run = block_before(mine_sum, sh.scan);
#pragma unroll
    for (int j = 0; j < per; ++j) {
      if (run < need && need <= run + static_cast<int>(cnt[j])) {
        sh.digit = static_cast<unsigned>(kBins - 1 - (tid * per + j));
        sh.above = static_cast<unsigned>(run);
        sh.whole = need - run == static_cast<int>(cnt[j]);
      }
      run += static_cast<int>(cnt[j]);
    }
    __syncthreads();
    prefix = prefix << bits | sh.digit;
    need -= static_cast<int>(sh.above);
    const bool whole = sh.whole != 0;
    __syncthreads();
    if (whole) {  // all keys with these digits are kept: the rest need not be told apart
      prefix = (prefix << shift) - 1;  // no key has digits of zeros alone
      need = 0;
      break;
    }
  }
  // keys above prefix are kept, and `need` of those equal to it

  // a run of whole words of 32 positions per warp
  const int run = ((mine + 31) / 32 + kSelWarps - 1) / kSelWarps * 32;
  const int i0 = min(mine, warp * run), i1 = min(mine, i0 + run);
  int2 found = make_int2(0, 0);
  for_keys(i0 + lane, i1, 32, [&](uint32_t k, int) {
    found.x += k > prefix;
    found.y += k == prefix;
  });
  found.x = warp_sum_int(found.x);
  found.y = warp_sum_int(found.y);
  if (lane == 0) sh.scan[warp] = found;
  __syncthreads();
  int2 at = make_int2(0, 0), total = make_int2(0, 0);
  for (int w = 0; w < kSelWarps; ++w) {
    const int2 y = sh.scan[w];
    if (w < warp) at.x += y.x, at.y += y.y;
    total.x += y.x, total.y += y.y;
  }
  if (ctas > 1) {  // no CTA leaves before its counts are read: a barrier follows
    if (tid == 0) sh.counts[0] = total.x, sh.counts[1] = total.y;
    cluster_barrier();
    int x[kMaxCtas], y[kMaxCtas];
#pragma unroll
    for (unsigned c = 0; c < kMaxCtas; ++c)
      if (c < rank) x[c] = ld_cluster(&sh.counts[0], c), y[c] = ld_cluster(&sh.counts[1], c);
#pragma unroll
    for (unsigned c = 0; c < kMaxCtas; ++c)
      if (c < rank) at.x += x[c], at.y += y[c];
  }
  int32_t* ws_table = a.ws_table + static_cast<int64_t>(b) * a.budget;
  float* ws_sums = a.ws_sums + static_cast<int64_t>(b) * a.budget;
  const unsigned below = (1u << lane) - 1u;
  constexpr int kWords = 4;  // words of 32 positions: loads in flight for the next ones while these find their places
  float x[kWords], x2[kWords];
  int32_t slot[kWords], slot2[kWords];
  auto fetch = [&](int w0) {
#pragma unroll
    for (int u = 0; u < kWords; ++u) {
      const int p = p0 + min(w0 + 32 * u + lane, i1 - 1);
      x2[u] = __ldg(sums + p);
      slot2[u] = table[p];
    }
  };
  if (i0 < i1) fetch(i0);
  for (int w0 = i0; w0 < i1; w0 += 32 * kWords) {
#pragma unroll
    for (int u = 0; u < kWords; ++u) x[u] = x2[u], slot[u] = slot2[u];
    if (w0 + 32 * kWords < i1) fetch(w0 + 32 * kWords);
#pragma unroll
    for (int u = 0; u < kWords; ++u) {
      const int i = w0 + 32 * u + lane, p = p0 + i;
      const bool in = i < i1;
      const uint32_t k = in ? key_at(i) : 0u;
      const unsigned above = __ballot_sync(0xffffffffu, in && k > prefix);
      const unsigned same = __ballot_sync(0xffffffffu, in && k == prefix);
      const int nth = at.y + __popc(same & below);                   // among the equal ones
      const int to = at.x + __popc(above & below) + min(nth, need);  // kept positions before this one
      at.x += __popc(above);
      at.y += __popc(same);
      if (!in) continue;
      if (k > prefix || (k == prefix && nth < need)) {
        if (!spec_in(to, a.budget, a.stats)) continue;
        kept[to] = p;
        ws_sums[to] = x[u];
        ws_table[to] = slot[u];
      } else if (a.page == 1) {
        if (spec_in(before + p - to, a.freed_cap, a.stats)) a.freed[before + p - to] = slot[u];
      }
    }
  }
  if (a.page > 1 && rank == 0) {
    const int first = pages_of(a.budget, a.page), count = pages_of(n, a.page) - first;
    for (int i = tid; i < count; i += kSelThreads) {
      const int32_t slot = table[static_cast<int64_t>(first + i) * a.page];
      if (spec_in(before + i, a.freed_cap, a.stats)) a.freed[before + i] = slot < 0 ? -1 : slot / a.page;
    }
  }
  // nobody reads the old slots and sums any more
  if (ctas > 1) cluster_barrier();
  else __syncthreads();
  for (int i = t0; i < a.budget; i += kWords * step) {
#pragma unroll
    for (int u = 0; u < kWords; ++u)
      if (i + u * step < a.budget) x[u] = ws_sums[i + u * step], slot[u] = ws_table[i + u * step];
#pragma unroll
    for (int u = 0; u < kWords; ++u)
      if (i + u * step < a.budget) {
        sums_out[i + u * step] = x[u];
        if (a.page == 1) table[i + u * step] = slot[u];
      }
  }
  for (int i = a.budget + t0; i < n; i += step) sums_out[i] = 0.0f;
}

constexpr int kMoveThreads = 256, kMoveStages = 3;

constexpr int kSliceVecs = 8;  // 16-byte vectors of a slice: a line of memory
constexpr int kRowsAt = kMoveThreads / kSliceVecs, kRows = 4 * kRowsAt;  // rows of a CTA's chunk: four vectors a thread

__global__ void __launch_bounds__(kMoveThreads) evict_payload_kernel(const EvictArgs a, int ctas) {
  pdl_enter();
  __shared__ __align__(16) uint4 sm[kMoveStages][4 * kMoveThreads];
  const int b = blockIdx.y;
  if (evict_len(a, b) <= a.limit) return;
  const int32_t* kept = a.kept + static_cast<int64_t>(b) * a.budget;
  // kept[i] - i never falls: the rows before the first that moves lie in place.
  // The block looks at 256 places at a time, since a search by halves is a chain of
  // ten loads and more
  int lo = 0, hi = a.budget;
#pragma unroll 1
  while (lo < hi) {
    const int step = (hi - lo + kMoveThreads - 1) / kMoveThreads, at = lo + static_cast<int>(threadIdx.x) * step;
    const int still = __syncthreads_count(at < hi && __ldg(kept + at) == at);  // places before the first that moves
    if (still == 0) break;
    hi = min(hi, lo + still * step);
    lo += (still - 1) * step + 1;
  }
  const int rows = kRows * ctas;  // of the cluster's chunk
  const int chunks = (a.budget - lo + rows - 1) / rows;
  const int rank = ctas > 1 ? static_cast<int>(cluster_rank()) : 0, slice = blockIdx.x / ctas;
  const int vec = threadIdx.x % kSliceVecs, first = lo + rank * kRows + threadIdx.x / kSliceVecs;
  const int64_t col = (static_cast<int64_t>(slice) * kSliceVecs + vec) * 16;
  const bool in = col < a.bps;
  const int32_t* from = a.ws_table + static_cast<int64_t>(b) * a.budget;
  const int32_t* to = a.table + static_cast<int64_t>(b) * a.max_ctx;
  // slots of this thread's four rows of a chunk: -1 behind the last
  auto slots = [&](const int32_t* list, int c, int32_t* s) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = first + c * rows + j * kRowsAt;
      s[j] = in && i < a.budget ? __ldg(list + i) : -1;
    }
  };
  auto slot_ok = [&](int32_t s) { return s >= 0 && s < a.num_slots; };
  int32_t src[4], dst[4];
  unsigned read[kMoveStages];  // bit j: row j of the stage's chunk has been read
  slots(from, 0, src);
  auto fetch = [&](int c, int st) {
    unsigned have = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (slot_ok(src[j])) {
        cp_async16(&sm[st][j * kMoveThreads + threadIdx.x], a.kv + src[j] * a.bps + col, 16);
        have |= 1u << j;
      }
    cp_async_commit();
    slots(from, c + 1, src);
    return have;
  };
#pragma unroll
  for (int c = 0; c < kMoveStages - 1; ++c) read[c] = fetch(c, c);
  slots(to, 0, dst);
#pragma unroll 1
  for (int c0 = 0; c0 < chunks; c0 += kMoveStages) {
#pragma unroll
    for (int s = 0; s < kMoveStages; ++s) {
      const int c = c0 + s;
      if (c >= chunks) break;  // the same in every thread
      read[(s + kMoveStages - 1) % kMoveStages] = fetch(c + kMoveStages - 1, (s + kMoveStages - 1) % kMoveStages);
      cp_async_wait<kMoveStages - 1>();
      // the chunk has been read whole (it lies in shared memory): its rows may be
      // overwritten.  Nothing written before has to be seen, so the cluster's
      // barrier does not wait for the stores of the chunk before
      if (ctas > 1)
        asm volatile("barrier.cluster.arrive.relaxed.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
      else
        __syncthreads();
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = first + c * rows + j * kRowsAt;
        if (((read[s] >> j) & 1u) != 0 && slot_ok(dst[j]))
          *reinterpret_cast<uint4*>(a.kv + dst[j] * a.bps + col) = sm[s][j * kMoveThreads + threadIdx.x];
        else if (in && i < a.budget && slice == 0 && vec == 0)
          bump(a.stats, SPEC_STAT_BAD_REQUEST);
      }
      slots(to, c + 1, dst);
    }
  }
  cp_async_wait<0>();
}

// Clusters of 16 are not portable and have to be allowed.
template <auto KERNEL>
bool allow_wide_clusters() {
  if (cudaFuncSetAttribute(KERNEL, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess) return true;
  cudaGetLastError();
  return false;
}

// CTAs of a request's cluster, by the longest request there can be: a CTA's
// keys then fit its shared memory up to 131072 positions.  Counts of a cluster
// cost two of its barriers a pass, so short requests have one CTA (37 requests of
// up to 4093 positions: 18.4 us with one, 21.4 with two; 131001: 26.1 with 8, 21.2
// with 16).  In a large batch most are shorter than that, and its requests fill
// the SMs by themselves (128 requests of 2000 positions in a table of 131072: 220 us
// with clusters of 16, 23 with two CTAs); keys that do not fit are then computed
// again in each pass.
int cluster_of(int B, int64_t max_ctx) {
  int ctas = max_ctx <= 4096 ? 1 : max_ctx <= 8192 ? 2 : max_ctx <= 16384 ? 4 : max_ctx <= 32768 ? 8 : kMaxCtas;
  while (ctas > 1 && static_cast<int64_t>(B) * ctas > 2 * 152) ctas /= 2;
  return ctas;
}

size_t evict_list(int B, int budget) { return align256(static_cast<size_t>(B) * budget * 4); }

}  // namespace
}  // namespace specdec

using namespace specdec;

extern "C" int64_t spec_evict_freed_capacity(int B, int64_t max_ctx, int page_size, int budget) {
  if (B < 0 || max_ctx < 1 || max_ctx > INT_MAX || page_size < 1 || budget < 1) return -1;
  const int64_t most = (max_ctx + page_size - 1) / page_size;
  const int64_t stay = (static_cast<int64_t>(budget) + page_size - 1) / page_size;
  return most > stay ? B * (most - stay) : 0;
}

extern "C" size_t spec_evict_ws_size(int B, int page_size, int budget) {
  if (B < 1 || B > 65535 || page_size < 1 || budget < 1) return 0;
  return evict_list(B, budget) * 2;
}

extern "C" int spec_evict_slots(int B, int page_size, int budget, int limit, int sinks, int recent,
                                const int32_t* seq_lens, const float* sums, float* sums_out, int32_t* req_to_token,
                                int64_t max_ctx, int32_t* kept, int32_t* freed, int64_t freed_capacity,
                                int32_t* num_freed, int32_t* new_kv_len, void* kv_pool_or_null, int64_t num_slots,
                                int64_t bytes_per_slot, int32_t* stats_or_null, void* ws, size_t ws_bytes,
                                spec_stream_t stream) {
  if (B < 0 || page_size < 1 || budget < 1 || limit < budget || sinks < 0 || recent < 0 || max_ctx < 1 ||
      static_cast<int64_t>(sinks) + recent > budget)
    return SPEC_ERR_INVALID_ARG;
  if (max_ctx > INT_MAX / 2 || budget > INT_MAX / 2 || B > 65535) return SPEC_ERR_UNSUPPORTED;
  if (!num_freed || freed_capacity < spec_evict_freed_capacity(B, max_ctx, page_size, budget))
    return SPEC_ERR_INVALID_ARG;
  if (B > 0 && (!seq_lens || !sums || !sums_out || !req_to_token || !kept || !new_kv_len || !ws ||
                (!freed && freed_capacity > 0)))
    return SPEC_ERR_INVALID_ARG;
  if (kv_pool_or_null) {
    if (num_slots < 1 || bytes_per_slot < 1) return SPEC_ERR_INVALID_ARG;
    if (bytes_per_slot % 16 != 0 || (reinterpret_cast<uintptr_t>(kv_pool_or_null) & 15) != 0 || num_slots > INT_MAX ||
        bytes_per_slot > INT_MAX)
      return SPEC_ERR_UNSUPPORTED;
  }
  if (B > 0 && (reinterpret_cast<uintptr_t>(ws) & 15) != 0) return SPEC_ERR_INVALID_ARG;
  if (B > 0 && ws_bytes < spec_evict_ws_size(B, page_size, budget)) return SPEC_ERR_WORKSPACE;
  auto overlap = [](const void* x, uint64_t n, const void* y, uint64_t m) {  // of n and m 32-bit values
    const uintptr_t x0 = reinterpret_cast<uintptr_t>(x), y0 = reinterpret_cast<uintptr_t>(y);
    return n > 0 && m > 0 && x0 < y0 + 4 * m && y0 < x0 + 4 * n;
  };
  // every CTA, and the payload's launch, reads the lengths while others write results
  const uint64_t requests = static_cast<uint64_t>(B);
  if (overlap(seq_lens, requests, new_kv_len, requests) || overlap(seq_lens, requests, kept, requests * budget) ||
      overlap(seq_lens, requests, freed, static_cast<uint64_t>(freed_capacity)) ||
      overlap(seq_lens, requests, num_freed, requests > 0 ? 1 : 0))
    return SPEC_ERR_INVALID_ARG;
  // the sums are read while their new ones are written, unless they are the same
  if (sums != sums_out && overlap(sums, requests * max_ctx, sums_out, requests * max_ctx)) return SPEC_ERR_INVALID_ARG;
  char* w = static_cast<char*>(ws);
  EvictArgs a{B, page_size, budget, limit, sinks, recent, seq_lens, sums, sums_out, req_to_token, max_ctx, kept, freed,
              freed_capacity, num_freed, new_kv_len,
              reinterpret_cast<int32_t*>(w + (B > 0 ? evict_list(B, budget) : 0)),
              reinterpret_cast<float*>(w), static_cast<uint8_t*>(kv_pool_or_null), num_slots, bytes_per_slot,
              stats_or_null};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (!allow_smem<evict_select_kernel>(sizeof(SelectShared))) return SPEC_ERR_CUDA;
  if (!allow_wide_clusters<evict_select_kernel>()) return SPEC_ERR_CUDA;
  const int ctas = cluster_of(B, max_ctx);
  launch_kc(evict_select_kernel, static_cast<unsigned>(B == 0 ? ctas : B * ctas), kSelThreads, sizeof(SelectShared), s,
            ctas, a, ctas);
  int e = launch_status();
  if (e != SPEC_OK || B == 0) return e;
  if (page_size == 1 || !kv_pool_or_null) return SPEC_OK;
  // CTAs of a slice's cluster: more until the launch fills the SMs twice or a
  // chunk takes all rows.  In us with one CTA / this rule: 1 request of 100000 to
  // 50000 positions, rows of 1280 bytes 311 / 53; 4 of 30000 to 20000 166 / 56; 16
  // of 4000 to 3000, 640 bytes 30 / 19; 128 of 2000 to 1000, 1280 bytes 73 / 70
  const int64_t slices = (bytes_per_slot / 16 + kSliceVecs - 1) / kSliceVecs;
  int c = 1;
  while (c < kMaxCtas && B * slices * c < 2 * 152 && c * kRows < budget) c *= 2;
  if (!allow_wide_clusters<evict_payload_kernel>()) return SPEC_ERR_CUDA;
  const dim3 grid(static_cast<unsigned>(slices * c), static_cast<unsigned>(B));
  launch_kc(evict_payload_kernel, grid, kMoveThreads, 0, s, c, a, c);
  return launch_status();
}
