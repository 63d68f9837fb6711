// Attention weights summed per cached position for many query rows (the last
// tokens of prompts), on the fifth-generation tensor cores.  The mathematics is
// that of kv4_sums.cu; here a step is 128 positions of one KV head and up to 128
// of its query rows, and S^T = K Q^T lies in tensor memory with a position per
// lane, so that a thread sums its position's weights over the columns in a
// register.
//
// K = lo + c step as exact fp16 operands: c step = hi + rem, the product rounded
// to fp16 and what it lost (a multiple of 2^-24 like step itself, so exact), and
// one step of 16 more columns that multiply the groups' lo with the groups' sums
// of q, three fp16 terms of each (2^-33).  All products of a step accumulate in
// fp32 in the same columns: 2 D + 16 instead of D products an element, with
// scores as good as fp32 sums.
//
// c step is the distance from the group's least value, up to 15 steps, which
// passes fp16's largest where a group spans more than that (steps above 4366;
// append's are below 7650).  Groups with steps from 4096 on are taken about their
// middle, K = lo + 8 step + (c - 8) step: |c - 8| step stays below 61200 and
// splits exactly as before, and 8 step, exact too, multiplies the groups' sums of
// q in 16 columns more.  Only products of tiles with such a group have them.
//
// Roles of a CTA:
//   warps 0 .. 7    weights: a thread's position is its lane; two groups of four
//       warps share a step's columns, since the next products but one wait for it.
//   warps 8 .. 15   unpack the cache, a position a thread: two groups take turns,
//       each warp with a ring of asynchronous copies of its 32 positions.
//   warp 16         issues the matrix instructions.
//   warp 17         copies the next KV head's rows, which kv4_sums_kernel has laid
//       out in the workspace.
// Steps go head by head over a segment of up to kSegTiles tiles of a request, so
// that a head's rows are copied once a segment; the segment's sums stay in shared
// memory until its last head.  The CTAs of a cluster share a segment's steps and
// add their sums through distributed shared memory, in rank order.  Every wait is
// bounded; a wait that runs out is counted in SPEC_STAT_WAIT_TIMEOUT and the CTA
// goes on without working (results void).
//
// Measured at 32 heads over 8 of 128, 32 rows each, B=4, contexts 60001..131001
// (100 GFLOP of scores, 391 M exponentials): 184 us with the launch that lays the
// rows out (180 without the look for wide groups).  A step took 1830 cycles
// without that look, of which the tensor pipe works 1090.  All products of a step
// go through one accumulator, one after the other, and two steps' S and operands
// fill the tensor memory.  The weights take 1350 cycles, the unpacking 2000 for
// two groups.  786 MB come from DRAM for 489 MB of rows, since the heads of a
// tile are some twenty steps apart; shorter segments read less and take longer (8
// tiles: 204 us). Steps on the way here: K's operands in shared memory 319 us
// (the matrix instructions then share its bandwidth), factor and lse read per
// column and rows converted by every CTA 289, groups of weights on alternate
// steps 206, one lane of a diverged warp issuing 204 instead of 182.
#include "kv4_sums.cuh"
#include "tcgen05.cuh"

namespace specdec {
namespace {

constexpr int kTile = 128;         // positions of a step
constexpr int kCols = kRowsBlock;  // query rows of a step at most
constexpr int kSegTiles = 48;      // tiles of a segment at most
constexpr int kUnpackWarp = 8, kIssueWarp = 16, kRowWarp = 17;
constexpr int kThreads = 18 * 32;
constexpr int kRing = 3;           // stages of an unpacking warp

template <int D>
struct RowsShared {
  RowsBlock<D> q[2];                // 1024-byte aligned
  uint8_t k_lo[2][kTile * 32];      // 128 rows of 16 elements, no swizzle
  float sum[2][kSegTiles * kTile];  // of the two groups of weights
  uint8_t ring[8][kRing][32 * Pos<D>::kBytes];  // of the unpacking warps
  uint8_t k_mid[2][kTile * 32];     // as k_lo: 8 step of wide groups, zeros of the others
};
// Tensor memory: S of both buffers, then hi and rem of both stages.
constexpr uint32_t kTmemCols = 512, kTmemA = 2 * kCols;

constexpr uint32_t kWideStep = 0x6c00u;  // 4096 in fp16: steps from here on make a group wide

__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }

// Descriptor of an operand without swizzle, K-major: 8 rows of 16 bytes are a
// block of 128 bytes; `leading` bytes between blocks along K, 128 along rows.
__device__ __forceinline__ uint64_t desc_plain(uint32_t addr, uint32_t leading) {
  return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) | static_cast<uint64_t>((leading & 0x3FFFFu) >> 4) << 16 |
         static_cast<uint64_t>(128 >> 4) << 32 | static_cast<uint64_t>(1) << 46;
}

// A cluster's stretch of the line of all requests' tiles, segment by segment,
// and this CTA's share of a segment's steps: every role walks it by itself.
struct Segments {
  int64_t lo, hi, pre;  // tiles; where request b begins
  int b, tile;          // next
  int t0, tiles, items, from, to;  // of the segment: steps [from, to) of items x tiles
  SumReq rq;
  int blocks;                      // of a head's rows

  __device__ __forceinline__ static int tiles_of(const SumReq& r) { return (r.end + kTile - 1) / kTile; }
  __device__ __forceinline__ bool next(const SumArgs& a, int rank, int ranks) {
#pragma unroll 1
    for (; pre + tile < hi; ++b, tile = 0) {
      rq = sum_req(a, b);
      const int all = tiles_of(rq);
      if (tile < all) {
        t0 = tile;
        tiles = static_cast<int>(min(static_cast<int64_t>(min(all - tile, kSegTiles)), hi - pre - tile));
        tile += tiles;
        blocks = (rq.rows * a.G + kCols - 1) / kCols;
        items = a.Hkv * blocks;
        const int64_t steps = static_cast<int64_t>(items) * tiles;
        from = static_cast<int>(steps * rank / ranks);
        to = static_cast<int>(steps * (rank + 1) / ranks);
        return true;
      }
      pre += all;
    }
    return false;
  }
};

// A wait, bounded like tc::bar_wait.  A lane that waits sleeps in the hardware
// for up to a microsecond at a time: some fifteen warps that poll take shared
// memory's bandwidth from the matrix instructions.
__device__ __forceinline__ bool wait_lane(uint64_t* bar, uint32_t parity, int* abort) {
  if (tc::bar_test(bar, parity)) return true;
  const uint32_t at = tc::smem_addr(bar);
  const long long t0 = clock64();
  for (;;) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.b32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(at), "r"(parity), "r"(1000u)
        : "memory");
    if (done != 0) return true;
    if (*reinterpret_cast<volatile int*>(abort) != 0) return false;
    if (clock64() - t0 > tc::kWaitCycles) {
      atomicExch(abort, 1);
      return false;
    }
  }
}
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, int* abort) {
  return __all_sync(0xffffffffu, wait_lane(bar, parity, abort));
}
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.b32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }

template <int D>
__global__ void __launch_bounds__(kThreads, 1) kv4_sums_rows_kernel(const SumArgs a, int clusters, int ranks) {
  pdl_enter();
  using Shared = RowsShared<D>;
  extern __shared__ uint8_t rows_sm[];
  Shared& sh = *reinterpret_cast<Shared*>((reinterpret_cast<uintptr_t>(rows_sm) + 1023) & ~uintptr_t(1023));
  if (!spec_smem_ok((reinterpret_cast<uint8_t*>(&sh) - rows_sm) + sizeof(Shared), a.stats)) return;
  __shared__ __align__(8) uint64_t q_full[2], q_empty[2], k_full[2], s_full[2], s_empty[2], drain;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort, s_b;
  __shared__ uint32_t s_wide[2];  // a byte per unpacking warp: its rows of the stage's k_mid are not all zeros
  __shared__ int64_t s_warp[kThreads / 32], s_pre;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = static_cast<int>(cluster_rank()), cluster = blockIdx.x / ranks;

  // the cluster's stretch of the line
  Segments seg;
  {
    const int per = (a.B + kThreads - 1) / kThreads;
    const int b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
    int64_t mine = 0;
#pragma unroll 1
    for (int i = b0; i < b1; ++i) {
      const SumReq r = sum_req(a, i);
      mine += Segments::tiles_of(r);
    }
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    int64_t total = 0, pre = incl - mine;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) {
      if (i < warp) pre += s_warp[i];
      total += s_warp[i];
    }
    const int64_t n = min(static_cast<int64_t>(clusters), total);
    if (cluster >= n) return;  // the whole cluster
    seg.lo = cluster * total / n;
    seg.hi = (cluster + 1) * total / n;
    if (seg.lo >= pre && seg.lo < pre + mine) {
      int i = b0;
#pragma unroll 1
      for (;; ++i) {
        const int u = Segments::tiles_of(sum_req(a, i));
        if (seg.lo < pre + u) break;
        pre += u;
      }
      s_pre = pre;
      s_b = i;
    }
    if (tid == 0) {
      for (int i = 0; i < 2; ++i) {
        tc::bar_init(&q_full[i], 1);
        tc::bar_init(&q_empty[i], 1 + kUnpackWarp);
        tc::bar_init(&k_full[i], 4);
        tc::bar_init(&s_full[i], 1);
        tc::bar_init(&s_empty[i], kUnpackWarp);
      }
      tc::bar_init(&drain, 1);
      s_abort = 0;
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0) tc::alloc<kTmemCols>(&s_tmem);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    seg.b = s_b;
    seg.pre = s_pre;
    seg.tile = static_cast<int>(seg.lo - seg.pre);
  }
  const uint32_t tmem = s_tmem;
  bool ok = true;
  unsigned j = 0, item_no = 0;  // steps and items so far: which buffer, which phase

  if (warp >= kRowWarp) {
    // --------------------------------------------------------------- rows
#pragma unroll 1
    while (seg.next(a, rank, ranks)) {
      if (lane == 0) {
        const int blocks = (a.N * a.G + kCols - 1) / kCols;  // of the workspace's heads
#pragma unroll 1
        for (int s = seg.from; ok && s < seg.to; ++item_no) {
          const int item = s / seg.tiles, h = item / seg.blocks, qb = item_no & 1;
          if (item_no >= 2) ok = wait_lane(&q_empty[qb], ((item_no >> 1) - 1) & 1, &s_abort);
          if (!ok) break;
          const RowsBlock<D>* src = static_cast<const RowsBlock<D>*>(a.ws) +
                                    (static_cast<int64_t>(seg.b) * a.Hkv + h) * blocks + item - h * seg.blocks;
          const uint32_t bar = tc::smem_addr(&q_full[qb]);
          asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar),
                       "r"(static_cast<uint32_t>(sizeof(RowsBlock<D>)))
                       : "memory");
          asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                           tc::smem_addr(&sh.q[qb])),
                       "l"(src), "r"(static_cast<uint32_t>(sizeof(RowsBlock<D>))), "r"(bar)
                       : "memory");
          s = (item + 1) * seg.tiles;  // the next item's first step
        }
      }
      __syncwarp();
      cluster_barrier();
      cluster_barrier();
    }
    if (lane == 0) {
      // no copy in flight when the CTA ends, although a wait has run out: the last
      // two items' are all that can be
      const long long t0 = clock64();
      for (unsigned i = item_no < 2 ? 0 : item_no - 2; i < item_no; ++i)
        while (!tc::bar_test(&q_full[i & 1], (i >> 1) & 1) && clock64() - t0 < tc::kWaitCycles) {
        }
    }
    __syncwarp();
  } else if (warp >= kUnpackWarp && warp < kIssueWarp) {
    // ------------------------------------------------------------- unpack
    const int u = (warp - kUnpackWarp) >> 2, uw = warp & 3, p = uw * 32 + lane;
    constexpr int vecs = D / 32;
    const unsigned ring = static_cast<unsigned>(__cvta_generic_to_shared(sh.ring[warp - kUnpackWarp][0]));
    int32_t slot;  // of this lane's position in the group's step to be copied next
    // a group's 32 channels, hi and rem, to tensor memory; less1024, less64: -1024 and
    // -64 as half2, or 8 less for codes less 8
    auto unpack = [](const uint4& code, uint32_t meta, uint32_t less1024, uint32_t less64, uint32_t to) {
      const uint32_t w[4] = {code.x, code.y, code.z, code.w};
      const __half2 step = u32_h2(__byte_perm(meta, 0, 0x1010)), sixteenth = u32_h2(0x2c002c00u);
      uint32_t hi[16], rem[16];
#pragma unroll
      for (int x = 0; x < 16; ++x) {
        const uint32_t y = x & 2 ? w[x >> 2] >> 8 : w[x >> 2];
        const __half2 c = x & 1 ? __hfma2(u32_h2((y & 0x00f000f0u) | 0x64006400u), sixteenth, u32_h2(less64))
                                : __hadd2(u32_h2((y & 0x000f000fu) | 0x64006400u), u32_h2(less1024));
        const __half2 v = __hmul2_rn(c, step);
        hi[x] = h2_u32(v);
        rem[x] = h2_u32(__hfma2(c, step, __hneg2(v)));
      }
      tc::st16(to, hi);
      tc::st16(to + D / 2, rem);
    };
    // this thread's row of k_mid, in the one stage that its group fills
    auto put_mid = [&](uint32_t a01, uint32_t a23) {  // three times, as lo
      uint8_t* row = sh.k_mid[u] + p * 16;
      *reinterpret_cast<uint4*>(row) = make_uint4(a01, a23, a01, a23);
      *reinterpret_cast<uint4*>(row + kTile * 16) = make_uint4(a01, a23, 0u, 0u);
    };
    put_mid(0u, 0u);
    if (lane == 0) reinterpret_cast<uint8_t*>(&s_wide[u])[uw] = 0;
    bool mid_set = false;  // the warp's rows of k_mid are not all zeros
#pragma unroll 1
    while (seg.next(a, rank, ranks)) {
      const int32_t* row = a.table + static_cast<int64_t>(seg.b) * a.max_ctx;
      // where a step is: KV head and tile of the segment
      struct At {
        int s, tile, block, h;
        __device__ __forceinline__ At(const Segments& seg, int step) : s(step) {
          const int item = step / seg.tiles;
          tile = step - item * seg.tiles, h = item / seg.blocks, block = item - h * seg.blocks;
        }
        __device__ __forceinline__ void next(const Segments& seg) {  // the group's next step
          s += 2;
          tile += 2;
          while (tile >= seg.tiles) {
            tile -= seg.tiles;
            if (++block == seg.blocks) block = 0, ++h;
          }
        }
      };
      const int mine = seg.from + static_cast<int>((j ^ u) & 1);  // the group's first step
      At of_slot(seg, mine), of_code(seg, mine);
      auto load_slot = [&]() {  // -2: no position
        slot = -2;
        const int pos = (seg.t0 + of_slot.tile) * kTile + p;
        if (of_slot.s < seg.to && pos < seg.rq.end) slot = __ldg(row + pos);
        of_slot.next(seg);
      };
      auto copy = [&](int to) {  // the positions' codes and (step, lo) to a stage; one commit group
        if (of_code.s < seg.to) {
          using P = Pos<D>;
          constexpr int per = D / 32;  // lanes of a position's codes
          const bool here = slot >= 0 && slot < a.num_slots;
          if (!here && slot != -2 && of_code.h == 0 && of_code.block == 0) bump(a.stats, SPEC_STAT_BAD_REQUEST);
          const unsigned have = __ballot_sync(0xffffffffu, here);
          const uint64_t mine = reinterpret_cast<uint64_t>(a.pool) +
                                static_cast<uint64_t>(here ? slot : 0) * static_cast<uint64_t>(a.slot_stride) +
                                static_cast<uint32_t>(of_code.h) * kv4_head_bytes(D);
          const unsigned at = ring + to * (32 * P::kBytes);
#pragma unroll
          for (int z = 0; z < per; ++z) {
            const int pos = z * (32 / per) + lane / per;
            const uint64_t src = __shfl_sync(0xffffffffu, mine, pos) + lane % per * 16;
            put_async(at + pos * P::kBytes + lane % per * 16, src, ((have >> pos) & 1u) * 16u);
          }
          put_async(at + lane * P::kBytes + P::kCodes, mine + D, here ? 16u : 0u);
        }
        cp_async_commit();
        of_code.next(seg);
      };
      load_slot();
#pragma unroll 1
      for (int i = 0; i < kRing - 1; ++i) {
        copy(i);
        load_slot();
      }
      int stage = 0;
#pragma unroll 1
      for (int s = seg.from; s < seg.to; ++s, ++j) {
        const int st = j & 1;
        if (st != u) continue;
        __syncwarp();  // every lane has read the stage before
        copy(stage == 0 ? kRing - 1 : stage - 1);
        load_slot();
        cp_async_wait<kRing - 1>();
        __syncwarp();  // every lane's copies of this step have landed
        uint4 code[vecs];
        uint32_t meta[vecs];
        const uint8_t* from = sh.ring[warp - kUnpackWarp][stage] + lane * Pos<D>::kBytes;
#pragma unroll
        for (int z = 0; z < vecs; ++z) {
          code[z] = *reinterpret_cast<const uint4*>(from + 16 * z);
          meta[z] = *reinterpret_cast<const uint32_t*>(from + Pos<D>::kCodes + 4 * z);
        }
        stage = stage + 1 == kRing ? 0 : stage + 1;
        // the stage is free once the products of two steps before are there
        if (ok && j >= 2) ok = wait_warp(&s_full[st], ((j >> 1) - 1) & 1, &s_abort);
        if (!ok) continue;
        tc::fence_after();
        const uint32_t to = tmem + (static_cast<uint32_t>(uw * 32) << 16) + kTmemA + st * D;
#pragma unroll
        for (int z = 0; z < vecs; ++z) unpack(code[z], meta[z], 0xe400e400u, 0xd400d400u, to + z * 16);
        uint32_t most = meta[0];  // its lower half: the largest step
#pragma unroll
        for (int z = 1; z < vecs; ++z) most = __vmaxu2(most, meta[z]);
        const bool wide = (most & 0xffffu) >= kWideStep;
        if (__any_sync(0xffffffffu, wide || mid_set)) {
          // wide groups again, from the stage and in a loop: few positions need it, and
          // code that every step fetches costs more than it computes
          uint32_t mid[2] = {0u, 0u};
          tc::wait_st();
#pragma unroll 1
          for (int z = 0; z < vecs; ++z) {
            const uint32_t m = *reinterpret_cast<const uint32_t*>(from + Pos<D>::kCodes + 4 * z);
            const bool about = (m & 0xffffu) >= kWideStep;
            unpack(*reinterpret_cast<const uint4*>(from + 16 * z), m, about ? 0xe408e408u : 0xe400e400u,
                   about ? 0xd480d480u : 0xd400d400u, to + z * 16);
            const uint32_t eight = about ? h2_u32(__hmul2_rn(u32_h2(m & 0xffffu), u32_h2(0x4800u))) : 0u;  // steps
            if (z < 2) mid[0] |= eight << (16 * z);
            else mid[1] |= eight << (16 * (z - 2));
          }
          put_mid(mid[0], mid[1]);
          mid_set = __any_sync(0xffffffffu, wide);
          if (lane == 0) reinterpret_cast<uint8_t*>(&s_wide[u])[uw] = mid_set;
        }
        // lo of the groups, three times: columns 0..3, 4..7, 8..11
        uint32_t lo[2];
        lo[0] = __byte_perm(meta[0], meta[1], 0x7632);
        lo[1] = vecs == 4 ? __byte_perm(meta[vecs - 2], meta[vecs - 1], 0x7632) : 0u;
        *reinterpret_cast<uint4*>(sh.k_lo[st] + p * 16) = make_uint4(lo[0], lo[1], lo[0], lo[1]);
        *reinterpret_cast<uint4*>(sh.k_lo[st] + kTile * 16 + p * 16) =
            make_uint4(lo[0], lo[1], 0x64006400u, 0x00006400u);  // 1024 beside lse's terms
        tc::wait_st();
        tc::fence_before();
        tc::fence_smem();
        __syncwarp();
        if (lane == 0) tc::bar_arrive(&k_full[st]);
      }
      __syncwarp();
      cluster_barrier();
      cluster_barrier();
    }
  } else if (warp == kIssueWarp) {
    // -------------------------------------------------------------- issue
    // the whole warp walks the steps, so that the operands' addresses are known to
    // be the same in all lanes (uniform registers); one lane issues
    const bool leader = elect_one();
    const uint32_t base = uniform(tmem);
#pragma unroll 1
    while (seg.next(a, rank, ranks)) {
      int left = min((seg.from / seg.tiles + 1) * seg.tiles, seg.to) - seg.from;  // steps of the item
      int block = seg.from / seg.tiles % seg.blocks;
#pragma unroll 1
      for (int s = seg.from; ok && s < seg.to;) {
        const int qb = uniform(item_no & 1);
        const int n = min(kCols, (seg.rq.rows * a.G - block * kCols + 31) / 32 * 32);
        const uint32_t id = uniform(tc::idesc_f16(n, false));
        const uint64_t qd = tc::desc(tc::smem_addr(sh.q[0].q) + qb * static_cast<uint32_t>(sizeof(sh.q[0])), 0);
        const uint64_t sums =
            desc_plain(tc::smem_addr(sh.q[0].sums) + qb * static_cast<uint32_t>(sizeof(sh.q[0])), kCols * 16);
        ok = wait_warp(&q_full[qb], (item_no >> 1) & 1, &s_abort);
        const unsigned steps = uniform(static_cast<uint32_t>(left));
        j = uniform(j);
#pragma unroll 1
        for (unsigned i = 0; i < steps; ++i, ++j) {
          const int st = j & 1;
          const uint32_t d = base + st * kCols, k_at = base + kTmemA + st * D;
          const uint64_t lo =
              desc_plain(tc::smem_addr(sh.k_lo[0]) + st * static_cast<uint32_t>(sizeof(sh.k_lo[0])), kTile * 16);
          if (!wait_warp(&k_full[st], (j >> 1) & 1, &s_abort) ||
              (j >= 2 && !wait_warp(&s_empty[st], ((j >> 1) - 1) & 1, &s_abort))) {
            ok = false;
            break;
          }
          tc::fence_after();
          const uint32_t wide = *reinterpret_cast<volatile uint32_t*>(&s_wide[st]);
          if (leader) {
#pragma unroll
            for (int part = 0; part < 2; ++part)
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk)
                tc::mma_ts(d, k_at + part * (D / 2) + kk * 8,
                           qd + (((kk / 4) * RowsBlock<D>::kSlab + (kk % 4) * 32) >> 4), id, part + kk != 0 ? 1u : 0u);
            tc::mma_ss(d, lo, sums, id, 1u);
            if (wide != 0) tc::mma_ss(d, lo + ((offsetof(Shared, k_mid) - offsetof(Shared, k_lo)) >> 4), sums, id, 1u);
            tc::commit(&s_full[st]);
          }
          __syncwarp();
        }
        if (ok && leader) tc::commit(&q_empty[qb]);
        __syncwarp();
        s += left;
        left = min(seg.tiles, seg.to - s);
        ++item_no;
        if (++block == seg.blocks) block = 0;
      }
      __syncwarp();
      cluster_barrier();
      cluster_barrier();
    }
    __syncwarp();
    if (leader) {
      // nothing in flight when tensor memory is freed
      tc::commit(&drain);
      const long long t0 = clock64();
      while (!tc::bar_test(&drain, 0) && clock64() - t0 < tc::kWaitCycles) {
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ weights
    const int e = warp >> 2, p = (warp & 3) * 32 + lane;
    const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
#pragma unroll 1
    while (seg.next(a, rank, ranks)) {
      const int32_t* row = a.table + static_cast<int64_t>(seg.b) * a.max_ctx;
      for (int i = p; i < seg.tiles * kTile; i += kTile) sh.sum[e][i] = 0.0f;
      int tile = seg.from % seg.tiles, block = seg.from / seg.tiles % seg.blocks;
#pragma unroll 1
      for (int s = seg.from; ok && s < seg.to; ++item_no) {
        const int qb = item_no & 1, count = min(seg.tiles - tile, seg.to - s);  // tiles of this head's rows
        ok = wait_warp(&q_full[qb], (item_no >> 1) & 1, &s_abort);
        if (!ok) break;
        const RowsBlock<D>& q = sh.q[qb];
        const int n = min(kCols, (seg.rq.rows * a.G - block * kCols + 31) / 32 * 32);
        const bool fold = q.fold != 0;
        const float2 one = splat(q.c[0]);
        float* sum = sh.sum[e] + tile * kTile + p;
        int d = (seg.t0 + tile) * kTile + p - seg.rq.start;  // rows from this one on see the position
#pragma unroll 1
        for (int i = 0; i < count; ++i, ++j, d += kTile, sum += kTile) {
          const int st = j & 1;
          ok = wait_warp(&s_full[st], (j >> 1) & 1, &s_abort);
          if (!ok) break;
          tc::fence_after();
          const bool whole = d - p + kTile <= 1;
          float2 acc[2] = {splat(0.0f), splat(0.0f)};
#pragma unroll 1
          for (int w = 32 * e; w < n; w += 64) {  // a group's columns
            uint32_t x[32];
            tc::ld32(lanes + st * kCols + w, x);
            tc::wait_ld32(x);
            if (fold) {
#pragma unroll
              for (int k = 0; k < 32; k += 2) {
                const float2 y = mul2(make_float2(__uint_as_float(x[k]), __uint_as_float(x[k + 1])), one);
                x[k] = __float_as_uint(y.x);
                x[k + 1] = __float_as_uint(y.y);
              }
            } else {
              const float4* c4 = reinterpret_cast<const float4*>(q.c + w);
              const float4* l4 = reinterpret_cast<const float4*>(q.nl + w);
#pragma unroll
              for (int k = 0; k < 32; k += 4) {
                const float4 c = c4[k / 4], l = l4[k / 4];
                x[k] = __float_as_uint(fmaf(__uint_as_float(x[k]), c.x, l.x));
                x[k + 1] = __float_as_uint(fmaf(__uint_as_float(x[k + 1]), c.y, l.y));
                x[k + 2] = __float_as_uint(fmaf(__uint_as_float(x[k + 2]), c.z, l.z));
                x[k + 3] = __float_as_uint(fmaf(__uint_as_float(x[k + 3]), c.w, l.w));
              }
            }
            if (!whole) {
#pragma unroll
              for (int k = 0; k < 32; ++k)
                if (d > q.row[w + k]) x[k] = 0xff800000u;
            }
#pragma unroll
            for (int k = 0; k < 32; k += 2)
              acc[(k >> 1) & 1] =
                  add2(acc[(k >> 1) & 1], exp2_2(make_float2(__uint_as_float(x[k]), __uint_as_float(x[k + 1]))));
          }
          tc::fence_before();
          __syncwarp();
          if (lane == 0) tc::bar_arrive(&s_empty[st]);
          const float2 t = add2(acc[0], acc[1]);
          *sum += t.x + t.y;
        }
        __syncwarp();
        if (ok && lane == 0) tc::bar_arrive(&q_empty[qb]);
        s += count;
        tile = 0;
        if (++block == seg.blocks) block = 0;
      }
      // the segment's sums of both groups, and of all CTAs of the cluster
      __syncwarp();
      cluster_barrier();
      const int64_t at = static_cast<int64_t>(seg.b) * a.max_ctx + static_cast<int64_t>(seg.t0) * kTile;
      const int count = min(seg.tiles * kTile, seg.rq.end - seg.t0 * kTile);
      for (int i = rank * 256 + tid; i < count; i += ranks * 256) {
        float x = 0.0f;
        for (int z = 0; z < ranks; ++z) x += ld_cluster(&sh.sum[0][i], z) + ld_cluster(&sh.sum[1][i], z);
        // a position without a slot has been a row of zeros so far
        const int32_t slot = __ldg(row + seg.t0 * kTile + i);
        if (slot < 0 || slot >= a.num_slots) x = 0.0f;
        a.out[at + i] = a.prev ? a.prev[at + i] + x : x;
      }
      __syncwarp();
      cluster_barrier();
    }
  }
  tc::fence_before();
  __syncthreads();
  if (warp == 0) {
    tc::fence_after();
    tc::dealloc<kTmemCols>(tmem);
  }
  if (tid == 0 && s_abort) bump(a.stats, SPEC_STAT_WAIT_TIMEOUT);
}

template <int D>
int launch_rows(const SumArgs& a, int ranks, int sms, cudaStream_t s) {
  constexpr auto kernel = kv4_sums_rows_kernel<D>;
  constexpr size_t smem = sizeof(RowsShared<D>) + 1024;
  static_assert(smem + 1024 <= 227 * 1024, "a CTA's shared memory");
  // a CTA holds all tensor memory of its SM while it waits for its cluster: two of
  // two clusters on one SM could wait for each other
  static_assert(2 * smem > 228 * 1024, "one CTA an SM");
  if (!allow_smem<kernel>(smem)) return SPEC_ERR_CUDA;
  const int clusters = sms / ranks;
  launch_kc(kernel, static_cast<unsigned>(clusters * ranks), kThreads, smem, s, ranks, a, clusters, ranks);
  return launch_status();
}

}  // namespace

int launch_sums_rows(const SumArgs& a, int D, int sms, cudaStream_t s) {
  // wider clusters where even the longest requests there can be give each no more
  // than a tile (128 rows, 8 KV heads; in us with 1, 2, 4, 8 CTAs: B=1, 4000
  // positions 26, 21, 17, 24; B=1, 16000: 27, 25, 36, 35; B=8, 2000: 28, 26, 37, 41;
  // B=4, 60000, 96 rows: 130, 127, 241, 253: clusters of four and more leave SMs
  // without one)
  const int ranks = a.B * ((a.max_ctx + kTile - 1) / kTile) <= sms / 4 ? 4 : 2;
  return D == 128 ? launch_rows<128>(a, ranks, sms, s) : launch_rows<64>(a, ranks, sms, s);
}

}  // namespace specdec
