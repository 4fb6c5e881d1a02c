// Causal attention of packed sequences with a sliding window and sinks, on the
// 5th-generation tensor cores (head dims 64 and 128).
//
// Per visible (query head, key) pair 4 d operations and one exponential: with
// d = 128 the tensor cores and the exponentials take about the same time per
// SM (a 128 x 128 tile: 2 x 512 cycles of MMA, 16384 exponentials at 16 a
// cycle), with d = 64 the exponentials are the bound.  Everything else is
// arranged to keep both units busy:
//
// A work item is a kv head and two tiles of 128 rows.  A tile's rows are
// tq = 128 / group consecutive packed tokens times the group of query heads
// that share the kv head (row = token * group + head): grouped heads read each
// key once, and short sequences still fill a tile.  Tiles do not care for
// sequence borders: a row admits the keys of its own sequence and window, and
// the item's keys are one range of packed rows, plus the first sequence's
// sinks when its window has left them behind.  One block runs per SM and,
// as it gets to them, takes over the items of the blocks that are not launched
// yet (cluster launch control), the last tokens (which see most) first:
//   warp 19 : plans items ahead of the others: key range, chunks and the start of
//             each row's sequence (searches in the offsets) into shared memory;
//   warp 18 : TMA -- the two Q tiles of an item and, per 128-key chunk, K and V
//             through a ring of slots (128-byte swizzle, rows past the batch
//             read as zeros);
//   warps 16, 17 : tcgen05.mma, a warp a tile, per chunk: O_X += P_X V of the
//             previous chunk, then S_X = Q_X K^T into the columns that P_X just
//             left (a warp's MMAs run in order).  While one tile's softmax
//             runs, the other tile's MMAs do: the warps take turns at the
//             tensor pipe, a chunk's MMAs of one tile at a time (interleaved,
//             both tiles' scores would be ready at the same time, and the
//             softmax and the MMAs would wait for each other).  One warp for
//             both tiles spent longer on its waits and descriptors than the
//             MMAs take.  K chunks of fewer keys
//             take fewer columns; chunks that a tile does not see are skipped;
//   warps 0..15 : softmax, eight warps a tile: a row belongs to two threads, one
//             for each 64 keys of a chunk (twice the warps for the latencies of
//             tensor memory and of the special-function unit to hide behind,
//             and half the code in each).  They read their scores, take the
//             exponentials with the scale folded into one packed FMA, and write
//             P as bf16 back to tensor memory.  The reference of the
//             exponentials is the row's maximum over its first chunk and moves
//             only after a chunk that was 2^8 ahead of it: then the row's
//             threads meet over the new maximum and rescale O (in tensor
//             memory, each half the dims) before the next chunk.  So no
//             exponential waits for a maximum, nor P for another thread.
//             32-key groups that every row of a
//             warp admits take no masks, those that none admits are skipped.
//             After the last chunk each thread reads half the dims of its row
//             of O, divides and stores.
// Tensor memory: S_0, S_1 (P over them), O_0, O_1: 512 columns for d = 128.
//
// A masked key has P = 0, but 0 times an infinity or NaN in its V row would
// still reach the tile's other rows: a row whose output is not finite, in a
// tile whose chunks hold such a V row that not every row sees, is computed
// again from the keys it sees alone (attend_row.cuh).
//
// Every wait is bounded; one that gives up counts into the error word that
// rm_op_timeouts reads, and its role stops.
//
// Measured on B200, among calls on other inputs (in brackets: replayed on the
// same ones): five documents of up to 32761 tokens, 32 heads on 8 of 128 dims,
// window 4096: 2.10 ms (2.03), 1.0 PFLOP/s of seen pairs (bound by a chunk's
// chain of scores, softmax and products with two tiles in flight, and by the
// power cap); 64 prompts of 256 to 560 tokens, 16 heads of 128: 155 us (140; an
// item is 1 to 5 chunks long, so its first maximum and its end weigh); 64
// texts of 2 to 100 tokens, 12 heads of 64: 16 us (latency).  Where every row
// is computed again (one document of 4096 tokens, 16 heads of 128, scores that
// climb): 59 ms instead of 97 us.
#include <cuda.h>

#include <algorithm>

#include "attend_row.cuh"
#include "kernels.h"
#include "sm100.cuh"

namespace rmk {
namespace {

RMK_BOUNDS_UNIT(attention_window)

__device__ int32_t g_window_err[ERR_WORDS];

constexpr int kTile = 128;              // rows of a tile, keys of a chunk
constexpr int kSoftmaxWarps = 16;
constexpr int kThreads = 32 * (kSoftmaxWarps + 4);     // two MMA warps, TMA, planner
constexpr float kLate = 40.f;           // log2; see the softmax
constexpr int kPlans = 2;               // items planned ahead
// Limit of a wait: 10 s, and 50 us for each packed token of the call.  A tile's
// roles wait while its softmax warps compute rows again (below): 32 rows a warp
// at most, each over at most every token, 0.5 us a key measured.
constexpr unsigned long long kLimitNs = 10000000000ull, kLimitNsPerToken = 50000ull;

// A work item: kv head; first token and token counts of its tiles; start of
// the sequence of a tile's first token, and that token's first key inside its
// window.
struct Plan {
  int h;                                // -1: no more items
  int t0, count[2];
  int start[2], lo[2];
  uint8_t begins[2 * kTile];            // per token: its sequence's start - t0, 0 = at or before t0
};

template <int D> struct Smem {
  static constexpr int kBox = kTile * 128;                 // 64 dims of 128 rows
  static constexpr int kBuf = kBox * (D / 64);             // a Q tile, K chunk or V chunk
  static constexpr int kSlots = D == 128 ? 4 : 8;          // two chunks, or four
  static constexpr int kQ = 0;
  static constexpr int kKv = 2 * kBuf;
  static constexpr int kOut = kKv + kSlots * kBuf;         // [2][2] boxes of 32 dims of a tile's output rows
  static constexpr int kBar = kOut + 2 * kBox;
  // q_full[2] q_empty[2] s_full[2] o_full[2] p_full[2][2] plan_full[]
  // plan_empty[] kv_full[] kv_empty[] pipe[2] claimed
  static constexpr int kBars = 15 + 2 * kPlans + 2 * kSlots;
  static constexpr int kClaim = (kBar + kBars * 8 + 15) / 16 * 16;
  static constexpr int kTmemSlot = kClaim + 16;
  static constexpr int kPlan = kTmemSlot + 16;
  static constexpr int kMeet = kPlan + kPlans * static_cast<int>(sizeof(Plan));   // 128 bytes for each two softmax warps
  static constexpr int kBytes = kMeet + kSoftmaxWarps / 2 * 128 + 1024;           // + alignment slack
  static_assert(kBytes <= 232448, "fits one CTA's shared memory");
};

struct WindowArgs {
  const bf16 *q, *k, *v;
  int64_t q_stride, k_stride, v_stride, out_stride;
  const int32_t* offsets;
  int n, hq, hkv, group, tq, tmax, window, sinks, items;
  bf16* out;
  float scale_log2;
  unsigned long long limit_ns;
};

// The issuing roles run as whole warps, whose control flow and operands stay
// uniform (a branch on the lane would cost moves to uniform registers around
// every instruction: 85 to 140 cycles an MMA instead of its 64); the one lane
// that issues is a predicate of the instruction.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}\n" : "=r"(r));
  return r;
}
__device__ __forceinline__ int uni(int x) { return __reduce_max_sync(0xffffffffu, x); }
__device__ __forceinline__ void mma_ss(uint32_t lead, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc ? 1u : 0u), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t lead, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc ? 1u : 0u), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void commit(uint32_t lead, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}\n" ::"r"(bar),
      "r"(lead)
      : "memory");
}
// MN-major operand (V as it lies: rows of keys, 64 dims of 128 bytes, 128-byte
// swizzle): 1024 bytes from 8 keys to the next 8 (stride offset), a box of 128
// rows from 64 dims to the next 64 (leading offset).
__device__ __forceinline__ uint64_t smem_desc_v(uint32_t saddr) {
  return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (1024ull << 16) | (64ull << 32) |
         (1ull << 46) | (2ull << 61);
}
// the larger of three, in one instruction
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ uint32_t low_bits(int x) {
  return x <= 0 ? 0u : (x >= 32 ? 0xffffffffu : ((1u << x) - 1u));
}
// Largest i in [0, n) with a[i] <= key, for a non-decreasing a with a[0] <= key,
// found by a warp: 32 places are read at a time (a search over 64 offsets for
// each token, a lane each, took 2.5 us of a short call's 14).
__device__ __forceinline__ int warp_upper_index(const int32_t* a, int n, int key, int lane) {
  int lo = 0;
  for (unsigned left = n; left > 1;) {
    const unsigned step = (left + 31) / 32, at = lane * step;
    const uint32_t le = __ballot_sync(0xffffffffu, at < left && a[lo + at] <= key) | 1u;
    const unsigned skip = (31 - __clz(le)) * step;
    lo += skip;
    left = min(step, left - skip);
  }
  return lo;
}

__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, unsigned long long limit_ns) {
  if (mbar_wait_for(bar, parity, limit_ns)) return true;
  atomicAdd(&g_window_err[ERR_TIMEOUT], 1);
  return false;
}

// Named barriers of the softmax: the 64 threads that share 32 rows of a tile
// (1..8), the 256 of a tile (9, 10) and the 128 of a tile's half of the dims
// (11..14).  The first two also AND a flag, so that a wait that gave up in one
// warp ends the others that meet it: none is left at a barrier.
__device__ __forceinline__ bool bar_all(int id, int threads, bool flag) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.and.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}\n"
      : "=r"(r)
      : "r"(flag ? 1u : 0u), "r"(id), "r"(threads)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void bar_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// An item's key chunks.  Chunks 0..nsc-1 cover the sinks [start, start +
// nsink) of the first token's sequence that lie before the window of every
// row; the others [lo, hi).
struct Chunks {
  int start, nsink, nsc, lo, hi, nc;
  __device__ __forceinline__ Chunks(const WindowArgs& a, const Plan& p)
      : start(uni(p.start[0])), lo(uni(p.lo[0])), hi(uni(p.t0 + p.count[0] + p.count[1])) {
    nsink = min(a.sinks, lo - start);
    nsc = (nsink + kTile - 1) / kTile;
    nc = nsc + (hi - lo + kTile - 1) / kTile;
  }
  __device__ __forceinline__ int base(int c) const {
    return c < nsc ? start + c * kTile : lo + (c - nsc) * kTile;
  }
  __device__ __forceinline__ int keys(int c) const {
    return min(kTile, c < nsc ? nsink - c * kTile : hi - base(c));
  }
};
// A tile's tokens [t0, t1) and what of the chunks it may see: its later rows
// see no earlier keys than its first, but for the sinks of sequences that
// begin in the tile, which are later still.
struct Tile {
  int t0, t1, start, lo;
  __device__ __forceinline__ Tile(const Plan& p, int x)
      : t0(uni(p.t0 + (x == 0 ? 0 : p.count[0]))), t1(uni(p.t0 + p.count[0] + (x == 0 ? 0 : p.count[1]))),
        start(uni(p.start[x])), lo(uni(p.lo[x])) {}
  __device__ __forceinline__ bool sees(const WindowArgs& a, int b, int keys) const {
    return t1 > t0 && keys > 0 && (b + keys > lo || (b - start < a.sinks && b + keys > start));
  }
  // of a chunk's keys from b on, those up to the tile's last token
  __device__ __forceinline__ int keys(const Chunks& c, int i, int b) const { return min(c.keys(i), t1 - b); }
  __device__ __forceinline__ int last(const Chunks& c) const { return c.nsc + (t1 - 1 - c.lo) / kTile; }
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    attn_window_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                       const __grid_constant__ CUtensorMap tmv, const __grid_constant__ CUtensorMap tmo,
                       const WindowArgs a) {
  using SL = Smem<D>;
  constexpr int NS = SL::kSlots;
  extern __shared__ uint8_t raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) &
                                           ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(sm);
  const uint32_t bar0 = sbase + SL::kBar;
  auto q_full = [&](int x) { return bar0 + 8u * x; };
  auto q_empty = [&](int x) { return bar0 + 8u * (2 + x); };
  auto s_full = [&](int x) { return bar0 + 8u * (4 + x); };
  auto o_full = [&](int x) { return bar0 + 8u * (6 + x); };
  auto p_full = [&](int x, int half) { return bar0 + 8u * (8 + 2 * x + half); };
  auto plan_full = [&](int e) { return bar0 + 8u * (12 + e); };
  auto plan_empty = [&](int e) { return bar0 + 8u * (12 + kPlans + e); };
  auto kv_full = [&](int s) { return bar0 + 8u * (12 + 2 * kPlans + s); };
  auto kv_empty = [&](int s) { return bar0 + 8u * (12 + 2 * kPlans + NS + s); };
  auto pipe = [&](int x) { return bar0 + 8u * (12 + 2 * kPlans + 2 * NS + x); };
  Plan* plans = reinterpret_cast<Plan*>(sm + SL::kPlan);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + SL::kTmemSlot);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int x = 0; x < 2; ++x) {
      mbar_init(q_full(x), 1);
      mbar_init(q_empty(x), 1);
      mbar_init(s_full(x), 1);
      mbar_init(p_full(x, 0), 4);        // the tile's four warps
      mbar_init(p_full(x, 1), 4);
      mbar_init(pipe(x), 1);
      mbar_init(o_full(x), 1);
    }
    mbar_init(pipe(2), 1);               // the planner's claims
    for (int e = 0; e < kPlans; ++e) {
      mbar_init(plan_full(e), 1);
      mbar_init(plan_empty(e), kSoftmaxWarps + 3);      // the warps that go by plans
    }
    for (int s = 0; s < NS; ++s) {
      mbar_init(kv_full(s), 1);
      mbar_init(kv_empty(s), 2);           // both tiles' products
    }
    mbar_init_fence();
  }
  if (warp == kSoftmaxWarps) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     smem_u32(tmem_slot))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_wait();
  // a wait of a whole warp: all lanes leave with one answer
  auto wait_warp = [&](uint32_t bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(bar, parity, a.limit_ns)) != 0; };
  const uint32_t tmem = *tmem_slot;
  auto s_at = [&](int x) { return tmem + static_cast<uint32_t>(x * kTile); };
  auto o_at = [&](int x) { return tmem + static_cast<uint32_t>(2 * kTile + x * kTile); };
  // the next plan, once it is made; the caller releases it when it has read it
  int plan = 0;
  uint32_t plan_turn = 0;
  auto next_plan = [&](const Plan*& p) {
    if (!wait_warp(plan_full(plan), plan_turn)) return false;
    p = plans + plan;
    return uni(p->h) >= 0;
  };
  auto release_plan = [&]() {
    __syncwarp();
    if (lane == 0) mbar_arrive(plan_empty(plan));
    if (++plan == kPlans) {
      plan = 0;
      plan_turn ^= 1;
    }
  };

  if (warp >= kSoftmaxWarps) {
    if (warp == kSoftmaxWarps + 2) {
      // ---- TMA producer ----
      const bool lead = elect_one() != 0;
      int slot = 0;                        // of the ring
      uint32_t turn = 1, loaded = 0;       // parity of an empty slot's wait; slots ever filled
      uint32_t q_turn = 0, q_loaded = 0;   // bit x
      bool ok = true;
      auto put = [&](const CUtensorMap* map, int h, int row) {
        if (((loaded >> slot) & 1) && !wait_warp(kv_empty(slot), turn)) return ok = false;
        loaded |= 1u << slot;
        const uint32_t dst = sbase + SL::kKv + slot * SL::kBuf;
        if (lead) {
          mbar_arrive_expect_tx(kv_full(slot), SL::kBuf);
#pragma unroll
          for (int c = 0; c < D / 64; ++c) tma_load_3d(dst + c * SL::kBox, map, c * 64, h, row, kv_full(slot));
        }
        if (++slot == NS) {
          slot = 0;
          turn ^= 1;
        }
        return true;
      };
      const Plan* p;
#pragma unroll 1
      while (ok && next_plan(p)) {
        const int h = uni(p->h);
        const Chunks ch(a, *p);
        const int q0[2] = {uni(p->t0), uni(p->t0 + p->count[0])};
        const bool any1 = uni(p->count[1]) > 0;
        release_plan();
#pragma unroll 1
        for (int c = 0; c < ch.nc && ok; ++c) {
          const int row = ch.base(c);
          if (!put(&tmk, h, row)) break;
          if (c == 0) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              if (!ok || (x == 1 && !any1)) continue;
              if (((q_loaded >> x) & 1) && !(ok = wait_warp(q_empty(x), ((q_turn >> x) & 1) ^ 1))) continue;
              if (lead) {
                mbar_arrive_expect_tx(q_full(x), a.tq * a.group * 128 * (D / 64));
#pragma unroll
                for (int k = 0; k < D / 64; ++k)
                  tma_load_3d(sbase + SL::kQ + x * SL::kBuf + k * SL::kBox, &tmq, k * 64, h * a.group, q0[x], q_full(x));
              }
              q_loaded |= 1u << x;
              q_turn ^= 1u << x;
            }
            if (!ok) break;
          }
          if (!put(&tmv, h, row)) break;
        }
      }
      // no copy into this CTA's shared memory may be in flight when it exits
      bool drained = true;
#pragma unroll 1
      for (int k = 0; k < NS && drained; ++k) {
        if (--slot < 0) {
          slot = NS - 1;
          turn ^= 1;
        }
        if ((loaded >> slot) & 1) drained = wait_warp(kv_full(slot), turn ^ 1);
      }
#pragma unroll 1
      for (int x = 0; x < 2 && drained; ++x)
        if ((q_loaded >> x) & 1) drained = wait_warp(q_full(x), ((q_turn >> x) & 1) ^ 1);
    }
    if (warp == kSoftmaxWarps + 3) {
      // ---- planner ----
      const int end = min(a.offsets[a.n], a.tmax), pairs = a.items / a.hkv;
      bool again = false, ok = true;       // a plan was in this place before
      uint32_t turn = 1;
      auto begin = [&]() { return !again || wait_warp(plan_empty(plan), turn); };
      auto publish = [&]() {
        __syncwarp();
        if (lane == 0) mbar_arrive(plan_full(plan));
        if (++plan == kPlans) {
          plan = 0;
          turn ^= 1;
          again = true;
        }
      };
      const uint32_t claim = sbase + SL::kClaim, claimed = pipe(2);
      uint32_t claim_turn = 0;
      int item = blockIdx.x;
#pragma unroll 1
      while (ok) {
        const int t0 = (pairs - 1 - item / a.hkv) * 2 * a.tq;
        const int count = min(2 * a.tq, end - t0);
        if (count > 0) {
          if (!(ok = begin())) break;
          Plan& p = plans[plan];
          // the sequence of the first token; then every later one that begins
          // here leaves its start at its first token, and the largest start up
          // to a token is that of its sequence
          const int s0 = warp_upper_index(a.offsets, a.n, t0, lane);
          int o = a.offsets[s0], s = s0 + 1 + lane;
          const int start0 = max(0, min(t0, o));
          if (lane == 0) in_bounds(o >= 0 && o <= t0);      // (offsets that begin behind 0 are cut to it)
          uint2* mine = reinterpret_cast<uint2*>(p.begins) + lane;     // eight tokens' bytes
          *mine = make_uint2(0u, 0u);
          __syncwarp();
          for (bool more = true; more; s += 32) {
            o = s > 0 && s < a.n ? a.offsets[s] : 0x7fffffff;
            if (o > t0 && o < t0 + count) p.begins[o - t0] = static_cast<uint8_t>(o - t0);
            more = __all_sync(0xffffffffu, o < t0 + count);
          }
          __syncwarp();
          uint2 b = *mine;
          uint32_t top = 0;
          auto upto = [&](uint32_t x) {
            uint32_t y = 0;
#pragma unroll
            for (int i = 0; i < 32; i += 8) {
              top = max(top, (x >> i) & 255u);
              y |= top << i;
            }
            return y;
          };
          upto(b.x);
          upto(b.y);
#pragma unroll
          for (int i = 1; i < 32; i <<= 1) {
            const uint32_t x = __shfl_up_sync(0xffffffffu, top, i);
            if (lane >= i) top = max(top, x);
          }
          top = __shfl_up_sync(0xffffffffu, top, 1);
          if (lane == 0) top = 0;
          b.x = upto(b.x);
          b.y = upto(b.y);
          *mine = b;
          __syncwarp();
          if (lane == 0) {
            p.h = item % a.hkv;
            p.t0 = t0;
            p.count[0] = min(count, a.tq);
            p.count[1] = count - p.count[0];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const int t = t0 + x * a.tq, at = p.begins[x * a.tq];
              p.start[x] = at == 0 ? start0 : t0 + at;
              p.lo[x] = a.window > 0 ? max(p.start[x], t - a.window + 1) : p.start[x];
            }
          }
          publish();
        }
        // the next item: the block of this grid that would have been launched
        // next is taken over instead (none left: this one is the last)
        if (lane == 0) {
          mbar_arrive_expect_tx(claimed, 16);
          asm volatile(
              "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(claim),
              "r"(claimed)
              : "memory");
        }
        if (!(ok = wait_warp(claimed, claim_turn))) break;
        claim_turn ^= 1;
        uint32_t taken, block;
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .b128 r;\n\t"
            "ld.shared.b128 r, [%2];\n\t"
            "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t"
            "mov.u32 %1, 0;\n\t"
            "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n\t}\n"
            : "=r"(taken), "=r"(block)
            : "r"(claim)
            : "memory");
        fence_proxy_async_smem();
        __syncwarp();
        if (!__any_sync(0xffffffffu, taken != 0)) break;
        item = static_cast<int>(block);
      }
      if (ok && begin()) {
        if (lane == 0) plans[plan].h = -1;
        publish();
      }
    }
    if (warp < kSoftmaxWarps + 2) {
      // ---- MMA issuers, one a tile ----
      const int x = warp - kSoftmaxWarps;
      const uint32_t lead = elect_one();
      constexpr uint32_t idesc_o = idesc_bf16_f32(kTile, D) | (1u << 16);     // B MN-major
      const uint32_t d_s = s_at(x), d_o = o_at(x);
      const uint64_t qd = smem_desc_k_sw128(sbase + SL::kQ + x * SL::kBuf);
      int slot = 0;                        // of the chunk's K; its V lies in the next one
      uint32_t turn = 0;                   // parity of that slot's full barrier
      uint32_t q_turn = 0, p_turn = 0, s_turn = 0, o_turn = 0;
      uint32_t pipe_turn = x ^ 1;          // tile 0 begins
      // the previous chunk's P V, if there is one still to be issued, and its V
      bool todo = false, opens = false, closes = false, ok = true;
      int v_slot = -1, v_steps = 0;
      uint32_t v_turn = 0;
      auto product = [&]() {
        const uint64_t v = smem_desc_v(sbase + SL::kKv + v_slot * SL::kBuf);
#pragma unroll
        for (int half = 0; half < 2; ++half) {                     // P comes 64 keys at a time
          // (for a half without keys too: its warps have then seen this
          // chunk's S, whose barrier may go on to the next)
          if (!(ok = wait_warp(p_full(x, half), p_turn))) return;
          tc_fence_after();
          if (v_steps >= half * 4 + 4) {
#pragma unroll
            for (int k = half * 4; k < half * 4 + 4; ++k)          // 16 keys: 2048 bytes of V
              mma_ts(lead, d_o, d_s + half * 64 + (k & 3) * 8, v + 128ull * k, idesc_o, !opens || k > 0);
          } else {
#pragma unroll 1
            for (int k = half * 4; k < v_steps; ++k)
              mma_ts(lead, d_o, d_s + half * 64 + (k & 3) * 8, v + 128ull * k, idesc_o, !opens || k > 0);
          }
        }
        p_turn ^= 1;
        if (closes) {
          commit(lead, o_full(x));
          o_turn ^= 1;
        }
      };
      const Plan* p;
#pragma unroll 1
      while (ok && next_plan(p)) {
        const Chunks ch(a, *p);
        const Tile tile(*p, x);
        release_plan();
        const int last = tile.last(ch);
        bool fresh = true;
#pragma unroll 1
        for (int c = 0; c < ch.nc && ok; ++c) {
          const int kb = ch.base(c), kn = tile.keys(ch, c, kb);
          const int n16 = (kn + 15) / 16;
          const bool sees = tile.sees(a, kb, kn);
          const uint32_t idesc_s = idesc_bf16_f32(kTile, n16 * 16);
          const uint64_t kd = smem_desc_k_sw128(sbase + SL::kKv + slot * SL::kBuf);
          // (A slot is released by both warps once it has been filled, used or
          // not: a warp that ran ahead would release it for the other.)
          if (v_slot >= 0 && !(ok = wait_warp(kv_full(v_slot), v_turn))) break;
          if (!(ok = wait_warp(kv_full(slot), turn))) break;
          if (!(ok = wait_warp(pipe(x), pipe_turn))) break;
          pipe_turn ^= 1;
          if (todo) product();
          if (!ok) break;
          if (sees) {
            if (fresh && !(ok = wait_warp(q_full(x), q_turn))) break;
            tc_fence_after();
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {                   // 16 dims: 32 bytes of a box's rows
              const uint64_t off = (ks / 4) * (SL::kBox / 16) + 2ull * (ks % 4);
              mma_ss(lead, d_s, qd + off, kd + off, idesc_s, ks > 0);
            }
            commit(lead, s_full(x));
            s_turn ^= 1;
            if (c == last) {
              commit(lead, q_empty(x));
              q_turn ^= 1;
            }
          }
          if (lead) mbar_arrive(pipe(x ^ 1));
          if (v_slot >= 0) commit(lead, kv_empty(v_slot));
          commit(lead, kv_empty(slot));
          todo = sees;
          opens = fresh;
          closes = c == last;
          if (sees) fresh = false;
          v_steps = n16;
          v_turn = turn;
          if ((v_slot = slot + 1) == NS) {
            v_slot = 0;
            v_turn ^= 1;
          }
          turn = v_turn;
          if ((slot = v_slot + 1) == NS) {
            slot = 0;
            turn ^= 1;
          }
        }
      }
      if (ok && todo && wait_warp(kv_full(v_slot), v_turn)) product();
      // tensor memory is freed after the last MMAs have completed (a barrier
      // never used is in phase 0: the wait for parity 1 returns at once)
      if (wait_warp(s_full(x), s_turn ^ 1)) wait_warp(o_full(x), o_turn ^ 1);
    }
  } else {
    // ---- softmax: half a row per thread ----
    const int x = warp >> 3, half = (warp >> 2) & 1, quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t ts = s_at(x) + lanes + half * 64;         // this half's scores, and P over them
    const uint32_t to = o_at(x) + lanes + half * (D / 2);    // and its dims of O
    const int pair_bar = 1 + x * 4 + quarter, tile_bar = 9 + x, dims_bar = 11 + 2 * x + half;
    // where a row's two threads meet, over a maximum or a sum: the second half's
    // part goes to the first, and the whole back, each between two barriers
    float* meet = reinterpret_cast<float*>(sm + SL::kMeet + (x * 4 + quarter) * 128) + lane;
    const int tok = row / a.group;
    const uint64_t sc2 = f32x2_splat(a.scale_log2);
    uint32_t s_turn = 0, o_turn = 0;
    bool ok = true;
    const Plan* p;
#pragma unroll 1
    while (bar_all(tile_bar, 256, next_plan(p))) {
      const int h = uni(p->h);
      const Chunks ch(a, *p);
      const Tile tile(*p, x);
      const int t = tile.t0 + tok;
      const bool mine = tok < a.tq && t < tile.t1;
      int start = 0, lo = 0, sink_end = 0;    // of the row's keys
      if (mine) {
        const int b = p->begins[t - p->t0];
        start = b == 0 ? ch.start : p->t0 + b;
        lo = a.window > 0 ? max(start, t - a.window + 1) : start;
        sink_end = start + min(a.sinks, lo - start);
      }
      release_plan();
      if (tile.t1 == tile.t0) continue;
      // keys that every row of the warp admits: [all_lo, all_hi]
      const int all_lo = __reduce_max_sync(0xffffffffu, lo);
      const int all_hi = __reduce_min_sync(0xffffffffu, mine ? t : 0x7fffffff);
      const bool any = __any_sync(0xffffffffu, mine);
      float ref = -INFINITY;             // base-2 reference of the row's exponentials
      float l = 0.f;                     // this half's sum
      bool begun = false, behind = false, set = false, late = false;
      float last_top = -INFINITY;
#pragma unroll 1
      for (int c = 0; c < ch.nc; ++c) {
        const int kb = ch.base(c), kn = tile.keys(ch, c, kb);
        if (!tile.sees(a, kb, kn)) continue;
        // columns of the half's two 32-key groups that the row admits, and the
        // groups that some and that every row of the warp admits
        uint32_t in[2] = {0xffffffffu, 0xffffffffu};
        bool some[2] = {true, true}, every[2] = {true, true};
        if (!(kn == kTile && kb >= all_lo && kb + kTile - 1 <= all_hi && any)) {
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const int q = 64 * half + 32 * y, b = kb + q;
            in[y] = !mine ? 0u
                : low_bits(kn - q) & ((low_bits(t + 1 - b) & ~low_bits(lo - b)) |
                                      (low_bits(sink_end - b) & ~low_bits(start - b)));
            some[y] = __any_sync(0xffffffffu, in[y] != 0u);
            every[y] = __all_sync(0xffffffffu, in[y] == 0xffffffffu || !mine);
          }
        }
        // Rows without a reference that see a key here, and after a chunk whose
        // maxima left some reference behind: the row's threads meet over its
        // maximum, and what is summed so far is rescaled.
        const bool sees = mine && ((lo < kb + kn && t >= kb) || (start < kb + kn && sink_end > kb));
        const bool look = behind || (!set && __any_sync(0xffffffffu, sees && ref == -INFINITY));
        ok = wait_warp(s_full(x), s_turn);
        s_turn ^= 1;
        tc_fence_after();
        // the scores of 32 keys; masked ones become -inf
        auto load = [&](int y, uint32_t (&s)[32]) {
          tmem_ld_32cols(ts + y * 32, s);
          tmem_wait_ld();
          if (!every[y]) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (!(in[y] & (1u << i))) s[i] = 0xff800000u;
          }
        };
        if (look) {
          float top = -INFINITY;
#pragma unroll 1
          for (int y = 0; y < 2; ++y) {
            if (!(y == 0 ? some[0] : some[1])) continue;
            uint32_t s[32];
            load(y, s);
            float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int i = 0; i < 32; i += 2)
              m4[(i / 2) & 3] = max3(m4[(i / 2) & 3], __uint_as_float(s[i]), __uint_as_float(s[i + 1]));
            top = fmaxf(top, fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * a.scale_log2);
          }
          top = fmaxf(top, last_top);
          if (half == 1) *meet = top;
          if (!bar_all(pair_bar, 64, ok)) {
            ok = false;
            break;
          }
          if (half == 0) *meet = fmaxf(top, *meet);
          bar_sync(pair_bar, 64);
          top = *meet;
          const float now = mine ? fmaxf(ref, top) : ref;
          const float keep = now == ref ? 1.f : (ref == -INFINITY ? 0.f : ex2_approx_ftz(ref - now));
          ref = now;
          l *= keep;
          if (begun) {
            // the earlier chunks' products are complete: S of this chunk was
            // issued behind them
#pragma unroll 1
            for (int q = 0; q < D / 32; ++q) {
              uint32_t o[16];
              tmem_ld_16cols(to + q * 16, o);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * keep);
              tmem_st_16cols(to + q * 16, o);
            }
            tmem_wait_st();
            tc_fence_before();
          }
          set = __all_sync(0xffffffffu, !mine || ref > -INFINITY);
          bar_sync(pair_bar, 64);        // O is rescaled, and the maxima are read
        }
        begun = true;
        // P against the reference, and the maximum beside it
        const uint64_t neg = f32x2_splat(ref == -INFINITY ? 0.f : -ref);
        float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        float sum4[4] = {0.f, 0.f, 0.f, 0.f};
        if (kn > 64 * half) {
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            uint32_t pk[16];
            if (some[y]) {
              uint32_t s[32];
              load(y, s);
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const float s0 = __uint_as_float(s[2 * i]), s1 = __uint_as_float(s[2 * i + 1]);
                m4[i & 3] = max3(m4[i & 3], s0, s1);
                float x0, x1;
                f32x2_unpack(f32x2_fma(f32x2_pack(s0, s1), sc2, neg), x0, x1);
                const float p0 = ex2_approx_ftz(x0), p1 = ex2_approx_ftz(x1);
                sum4[(i & 1) * 2] += p0;
                sum4[(i & 1) * 2 + 1] += p1;
                pk[i] = pack_bf16x2(p0, p1);
              }
            } else {
#pragma unroll
              for (int i = 0; i < 16; ++i) pk[i] = 0u;
            }
            tmem_st_16cols(ts + y * 16, pk);     // over scores that are read
          }
          tmem_wait_st();
        }
        // Without keys as well: S's barrier is waited for by parity, so it must
        // not complete again before every warp of the tile has passed it.
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full(x, half));
        l += (sum4[0] + sum4[1]) + (sum4[2] + sum4[3]);
        // Has a maximum left its reference behind?  By up to 2^kLate the sums
        // take it (P and O have the exponents of fp32), and the next chunk moves
        // the reference; by more, the row is computed again at the end.
        last_top = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * a.scale_log2;
        late = late || (mine && last_top > ref + kLate);
        const bool high = mine && last_top > ref + 8.f;
        behind = !bar_all(pair_bar, 64, ok && !high);
        if (behind && !bar_all(pair_bar, 64, ok)) {
          ok = false;
          break;
        }
      }
      if (ok) ok = wait_warp(o_full(x), o_turn);
      o_turn ^= 1;
      tc_fence_after();
      // the row's sum: the second half's part to the first, and back (not in a
      // column of S: the next item's scores may be on their way there)
      if (half == 1) *meet = l;
      bar_sync(pair_bar, 64);
      if (half == 0) *meet = l + *meet;
      if (!bar_all(tile_bar, 256, ok)) break;
      const float inv = 1.f / *meet;
      const int head = h * a.group + row % a.group;
      uint32_t w[D / 4];
      float worst = 0.f;
#pragma unroll
      for (int q = 0; q < D / 64; ++q) {
        uint32_t o[32];
        tmem_ld_32cols(to + q * 32, o);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float y0 = __uint_as_float(o[2 * i]) * inv, y1 = __uint_as_float(o[2 * i + 1]) * inv;
          worst = fmaf(y0, 0.f, fmaf(y1, 0.f, worst));      // NaN once one is not finite
          w[q * 16 + i] = pack_bf16x2(y0, y1);
        }
      }
      tc_fence_before();
      const uint32_t odd = __ballot_sync(0xffffffffu, mine && (worst != 0.f || late));
      // A whole tile of finite rows leaves through shared memory, 32 dims at a
      // time, as one box (row by row, a warp's store would touch 32 lines);
      // other tiles row by row.  (Behind this barrier S and O are read.)
      const bool box = bar_all(tile_bar, 256, odd == 0) && tile.t1 - tile.t0 == a.tq;
      if (box) {
        const uint32_t out = sbase + SL::kOut + (2 * x + half) * (SL::kBox / 2);
#pragma unroll
        for (int q = 0; q < D / 64; ++q) {
          // the previous box has been read out of shared memory
          if (row == 0) bulk_wait_group_read<0>();
          bar_sync(dims_bar, 128);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(out + row * 64 + ((i ^ ((row >> 1) & 3)) << 4)),
                         "r"(w[q * 16 + 4 * i]), "r"(w[q * 16 + 4 * i + 1]), "r"(w[q * 16 + 4 * i + 2]),
                         "r"(w[q * 16 + 4 * i + 3])
                         : "memory");
          fence_proxy_async_smem();
          bar_sync(dims_bar, 128);
          if (row == 0) {
            tma_store_3d(&tmo, out, half * (D / 2) + q * 32, h * a.group, tile.t0);
            bulk_commit_group();
          }
        }
      } else {
        if (mine) {
          bf16* dst = a.out + t * a.out_stride + static_cast<int64_t>(head) * D + half * (D / 2);
#pragma unroll
          for (int i = 0; i < D / 16; ++i)
            reinterpret_cast<uint4*>(dst)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        }
        bar_sync(tile_bar, 256);                // the rows are written before any is written again
      }
      if (odd != 0) {
        // does a V row that some row of the tile does not see hold the cause?
        bool cause = false;
        for (int c = 0; c < ch.nc; ++c) {
          const int kb = ch.base(c), kn = tile.keys(ch, c, kb);
          const int rows = min(((kn + 15) / 16) * 16, a.tmax - kb);      // what the products read
          if (!tile.sees(a, kb, kn) || (kb >= all_lo && kb + rows - 1 <= all_hi)) continue;
          for (int j = lane; j < rows; j += 32) {
            const bf16* vr = a.v + (kb + j) * a.v_stride + h * D;
            for (int e = 0; e < D / 8; ++e) {
              float f[8];
              Chunk8<bf16>::load(vr + 8 * e, f);
#pragma unroll
              for (int i = 0; i < 8; ++i) cause = cause || !(fabsf(f[i]) < INFINITY);
            }
          }
        }
        const uint32_t again = __any_sync(0xffffffffu, cause) ? odd : odd & __ballot_sync(0xffffffffu, late);
        {
          for (uint32_t left = again; left != 0; left &= left - 1) {
            const int src = __ffs(left) - 1;
            const int64_t tt = __shfl_sync(0xffffffffu, t, src);
            const int64_t hh = __shfl_sync(0xffffffffu, head, src);
            const int st = __shfl_sync(0xffffffffu, start, src), from = __shfl_sync(0xffffffffu, lo, src);
            const int se = __shfl_sync(0xffffffffu, sink_end, src);
            auto ptr = [&](int64_t j, const bf16*& kp, const bf16*& vp) {
              if (!in_bounds(j >= 0 && j <= tt && tt < a.tmax)) return;
              kp = a.k + j * a.k_stride + h * D;
              vp = a.v + j * a.v_stride + h * D;
            };
            const bf16* q = a.q + tt * a.q_stride + hh * D;
            RowState<D> state;
            attend_keys<D>(q, a.scale_log2, st, se, ptr, state);
            attend_keys<D>(q, a.scale_log2, from, tt + 1, ptr, state);
            const float il = 1.f / state.l;
#pragma unroll
            for (int i = 0; i < D / 32; ++i)
              a.out[tt * a.out_stride + hh * D + lane + 32 * i] = __float2bfloat16_rn(state.o[i] * il);
          }
        }
      }
    }
  }
  if (warp < kSoftmaxWarps) bulk_wait_group<0>();      // the boxes are written before shared memory goes
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kSoftmaxWarps) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

// One thread waits, through this file's wait, on an mbarrier that nothing completes.
__global__ void window_wait_selftest_kernel(unsigned long long limit_ns) {
  __shared__ __align__(8) uint64_t bar;
  if (threadIdx.x != 0) return;
  mbar_init(smem_u32(&bar), 1);
  mbar_init_fence();
  wait(smem_u32(&bar), 0, limit_ns);
}

template <int D>
cudaError_t launch(const WindowArgs& a, int T, int grid, cudaStream_t st) {
  CUtensorMap tq, tk, tv, to;
  const char* why = "";
  if (!make_tmap_heads(&tq, a.q, T, a.hq, D, a.q_stride, 64, a.group, a.tq, &why) ||
      !make_tmap_heads(&tk, a.k, T, a.hkv, D, a.k_stride, 64, 1, kTile, &why) ||
      !make_tmap_heads(&tv, a.v, T, a.hkv, D, a.v_stride, 64, 1, kTile, &why) ||
      !make_tmap_heads(&to, a.out, T, a.hq, D, a.out_stride, 32, a.group, a.tq, &why))
    return cudaErrorInvalidValue;
  auto kernel = attn_window_kernel<D>;
  static std::atomic<unsigned long long> allowed{0};
  const cudaError_t e = allow_smem(kernel, Smem<D>::kBytes, allowed);
  if (e != cudaSuccess) return e;
  PdlScope pdl(true);
  return launch_k(kernel, dim3(grid), dim3(kThreads), Smem<D>::kBytes, st, tq, tk, tv, to, a);
}

}  // namespace

cudaError_t bounds_errors_attention_window(int32_t* out, bool reset) {
  cudaError_t e = cudaMemcpyFromSymbol(out, g_bounds_attention_window, sizeof(int32_t));
  if (e == cudaSuccess && reset) {
    const int32_t zero = 0;
    e = cudaMemcpyToSymbol(g_bounds_attention_window, &zero, sizeof(int32_t));
  }
  return e;
}

cudaError_t window_wait_selftest(unsigned long long limit_ns, cudaStream_t st) {
  window_wait_selftest_kernel<<<1, 32, 0, st>>>(limit_ns);
  return cudaGetLastError();
}

cudaError_t window_timeouts(int32_t* out) {
  int32_t words[ERR_WORDS];
  const int32_t zero[ERR_WORDS] = {};
  cudaError_t e = cudaMemcpyFromSymbol(words, g_window_err, sizeof words);
  if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_window_err, zero, sizeof zero);
  if (e == cudaSuccess) *out = words[ERR_TIMEOUT];
  return e;
}

cudaError_t attn_window_launch(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                               const void* v, int64_t v_stride, const int32_t* offsets, int n,
                               int T, int hq, int hkv, int d, int window, int sinks, void* out,
                               int64_t out_stride, cudaStream_t st) {
  if (T < 1) return cudaSuccess;
  WindowArgs a;
  a.q = static_cast<const bf16*>(q);
  a.k = static_cast<const bf16*>(k);
  a.v = static_cast<const bf16*>(v);
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.out_stride = out_stride;
  a.offsets = offsets;
  a.n = n;
  a.hq = hq;
  a.hkv = hkv;
  a.group = hq / hkv;
  a.tq = kTile / a.group;
  a.tmax = T;
  a.window = window;
  a.sinks = sinks;
  a.out = static_cast<bf16*>(out);
  a.scale_log2 = 1.4426950408889634f / sqrtf(static_cast<float>(d));
  a.limit_ns = kLimitNs + kLimitNsPerToken * static_cast<unsigned long long>(T);
  const int64_t items = (static_cast<int64_t>(T) + 2 * a.tq - 1) / (2 * a.tq) * hkv;
  if (items > 0x7fffffff) return cudaErrorInvalidValue;
  a.items = static_cast<int>(items);
  // a block an item: those that run take the others over (planner)
  return d == 64 ? launch<64>(a, T, a.items, st) : launch<128>(a, T, a.items, st);
}

}  // namespace rmk
