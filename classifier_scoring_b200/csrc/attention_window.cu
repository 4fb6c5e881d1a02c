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
// sinks when its window has left them behind.  Items are dealt to one
// persistent CTA per SM, the last tokens (which see most) first:
//   warp 9, one lane : TMA -- the two Q tiles of an item and, per 128-key
//                      chunk, K and V through a ring of slots (128-byte
//                      swizzle, rows past the batch read as zeros);
//   warp 8, one lane : tcgen05.mma, per chunk and tile X: O_X += P_X V of the
//                      previous chunk, then S_X = Q_X K^T into the columns
//                      that P_X just left (the tensor pipe runs its MMAs in
//                      order).  While one tile's softmax runs, the other
//                      tile's MMAs do.  K chunks of fewer keys take fewer
//                      columns; chunks that a tile does not see are skipped;
//   warps 0..7       : softmax, four warps a tile, one row per thread: the row
//                      of S in registers, its maximum, the exponentials with
//                      the scale folded into one packed FMA, P as bf16 back to
//                      tensor memory.  The reference of the exponentials
//                      follows the maximum only when it falls 2^8 behind, and
//                      only then is O rescaled (in tensor memory, by the same
//                      thread); chunks that a warp's rows admit in full take no
//                      masks.  After the last chunk the thread reads its row
//                      of O, divides and stores it.
// Tensor memory: S_0, S_1 (P over them), O_0, O_1: 512 columns for d = 128.
//
// A masked key has P = 0, but 0 times an infinity or NaN in its V row would
// still reach the tile's other rows: a row whose output is not finite, in a
// tile whose chunks hold such a V row that not every row sees, is computed
// again from the keys it sees alone (attend_row.cuh).
//
// Every wait is bounded; one that gives up counts into the error word, and its
// role stops.
#include <cuda.h>

#include <algorithm>

#include "attend_row.cuh"
#include "kernels.h"
#include "sm100.cuh"

namespace rmk {
namespace {

__device__ int32_t g_window_err[ERR_WORDS];

constexpr int kTile = 128;              // rows of a tile, keys of a chunk
constexpr int kThreads = 320;           // 8 softmax warps, MMA, TMA
constexpr unsigned long long kLimitNs = 10000000000ull;

template <int D> struct Smem {
  static constexpr int kBox = kTile * 128;                 // 64 dims of 128 rows
  static constexpr int kBuf = kBox * (D / 64);             // a Q tile, K chunk or V chunk
  static constexpr int kSlots = D == 128 ? 5 : 10;
  static constexpr int kQ = 0;
  static constexpr int kKv = 2 * kBuf;
  static constexpr int kBar = kKv + kSlots * kBuf;
  // q_full[2] q_empty[2] s_full[2] p_full[2] o_full[2] kv_full[] kv_empty[]
  static constexpr int kBars = 10 + 2 * kSlots;
  static constexpr int kTmemSlot = kBar + kBars * 8;
  static constexpr int kBytes = kTmemSlot + 16 + 1024;     // + 1024-byte alignment slack
  static_assert(kBytes <= 232448, "fits one CTA's shared memory");
};

struct WindowArgs {
  const bf16 *q, *k, *v;
  int64_t q_stride, k_stride, v_stride, out_stride;
  const int32_t* offsets;
  int n, hq, hkv, group, tq, tmax, window, sinks, items;
  bf16* out;
  float scale_log2;
};

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc ? 1u : 0u)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc ? 1u : 0u)
      : "memory");
}
// MN-major operand (V as it lies: rows of keys, 64 dims of 128 bytes, 128-byte
// swizzle): 1024 bytes from 8 keys to the next 8 (stride offset), a box of 128
// rows from 64 dims to the next 64 (leading offset).
__device__ __forceinline__ uint64_t smem_desc_v(uint32_t saddr) {
  return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (1024ull << 16) | (64ull << 32) |
         (1ull << 46) | (2ull << 61);
}
__device__ __forceinline__ uint32_t low_bits(int x) {
  return x <= 0 ? 0u : (x >= 32 ? 0xffffffffu : ((1u << x) - 1u));
}
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity) {
  if (mbar_wait_for(bar, parity, kLimitNs)) return true;
  atomicAdd(&g_window_err[ERR_TIMEOUT], 1);
  return false;
}

// Where a token's keys begin: its sequence and its window.
struct Row {
  int start, lo;
};
__device__ __forceinline__ Row row_of(const WindowArgs& a, int t) {
  Row r;
  r.start = a.offsets[upper_index(a.offsets, a.n, t)];
  r.lo = a.window > 0 ? max(r.start, t - a.window + 1) : r.start;
  return r;
}

// A work item's tiles and key chunks.  Chunks 0..nsink_chunks-1 cover the
// sinks [start, start + nsink) of the first row's sequence that lie before
// the window of every row; the others [lo, hi).
struct Item {
  int h, t0[2], t1[2];            // kv head; tokens of the tiles (t1 = t0: none)
  int start, sinks, nsink, lo, hi, nsc, nc;
  Row first[2];                   // the tiles' first rows
  __device__ __forceinline__ bool load(const WindowArgs& a, int item, int end) {
    const int pairs = a.items / a.hkv;
    h = item % a.hkv;
    t0[0] = (pairs - 1 - item / a.hkv) * 2 * a.tq;
    if (t0[0] >= end) return false;
    t1[0] = t0[1] = min(t0[0] + a.tq, end);
    t1[1] = min(t0[1] + a.tq, end);
    first[0] = first[1] = row_of(a, t0[0]);
    if (t1[1] > t0[1]) first[1] = row_of(a, t0[1]);
    start = first[0].start;
    lo = first[0].lo;
    hi = t1[1];
    sinks = a.sinks;
    nsink = min(sinks, lo - start);
    nsc = (nsink + kTile - 1) / kTile;
    nc = nsc + (hi - lo + kTile - 1) / kTile;
    return true;
  }
  __device__ __forceinline__ int base(int c) const {
    return c < nsc ? start + c * kTile : lo + (c - nsc) * kTile;
  }
  __device__ __forceinline__ int keys(int c) const {
    return min(kTile, c < nsc ? nsink - c * kTile : hi - base(c));
  }
  // whether some row of tile x may see chunk c (its later rows see no earlier
  // keys than its first, but for the sinks of sequences that begin in the
  // tile, which are later still), and the tile's last chunk
  __device__ __forceinline__ bool sees(int x, int c) const {
    const int b = base(c), e = b + keys(c);
    return t1[x] > t0[x] && b < t1[x] && (e > first[x].lo || (b - first[x].start < sinks && e > first[x].start));
  }
  __device__ __forceinline__ int last(int x) const { return nsc + (t1[x] - 1 - lo) / kTile; }
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    attn_window_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                       const __grid_constant__ CUtensorMap tmv, const WindowArgs a) {
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
  auto p_full = [&](int x) { return bar0 + 8u * (6 + x); };
  auto o_full = [&](int x) { return bar0 + 8u * (8 + x); };
  auto kv_full = [&](int s) { return bar0 + 8u * (10 + s); };
  auto kv_empty = [&](int s) { return bar0 + 8u * (10 + NS + s); };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + SL::kTmemSlot);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int x = 0; x < 2; ++x) {
      mbar_init(q_full(x), 1);
      mbar_init(q_empty(x), 1);
      mbar_init(s_full(x), 1);
      mbar_init(p_full(x), 4);           // the tile's four warps
      mbar_init(o_full(x), 1);
    }
    for (int s = 0; s < NS; ++s) {
      mbar_init(kv_full(s), 1);
      mbar_init(kv_empty(s), 1);
    }
    mbar_init_fence();
  }
  if (warp == 8) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     smem_u32(tmem_slot))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  auto s_at = [&](int x) { return tmem + static_cast<uint32_t>(x * kTile); };
  auto o_at = [&](int x) { return tmem + static_cast<uint32_t>(2 * kTile + x * kTile); };
  const int end = a.offsets[a.n];
  Item it;

  if (warp == 9) {
    // ---- TMA producer ----
    if (lane == 0) {
      int g = 0, nq[2] = {0, 0};
      bool ok = true;
      auto put = [&](const CUtensorMap* map, int row) {
        const int s = g % NS;
        if (g >= NS && !wait(kv_empty(s), ((g / NS) - 1) & 1)) return ok = false;
        mbar_arrive_expect_tx(kv_full(s), SL::kBuf);
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
          tma_load_3d(sbase + SL::kKv + s * SL::kBuf + c * SL::kBox, map, c * 64, it.h, row, kv_full(s));
        ++g;
        return true;
      };
      for (int item = blockIdx.x; item < a.items && ok; item += gridDim.x) {
        if (!it.load(a, item, end)) continue;
        for (int c = 0; c < it.nc && ok; ++c) {
          const int row = it.base(c);
          if (!put(&tmk, row)) break;
          if (c == 0) {
            for (int x = 0; x < 2 && ok; ++x) {
              if (it.t1[x] == it.t0[x]) continue;
              if (nq[x] > 0 && !wait(q_empty(x), (nq[x] - 1) & 1)) {
                ok = false;
                break;
              }
              mbar_arrive_expect_tx(q_full(x), a.tq * a.group * 128 * (D / 64));
#pragma unroll
              for (int k = 0; k < D / 64; ++k)
                tma_load_3d(sbase + SL::kQ + x * SL::kBuf + k * SL::kBox, &tmq, k * 64, it.h * a.group,
                            it.t0[x], q_full(x));
              ++nq[x];
            }
            if (!ok) break;
          }
          if (!put(&tmv, row)) break;
        }
      }
      // no copy into this CTA's shared memory may be in flight when it exits
      bool drained = true;
      for (int k = g - 1; drained && k >= 0 && k >= g - NS; --k) drained = wait(kv_full(k % NS), (k / NS) & 1);
      for (int x = 0; x < 2 && drained; ++x)
        if (nq[x] > 0) drained = wait(q_full(x), (nq[x] - 1) & 1);
    }
  } else if (warp == 8) {
    // ---- MMA issuer ----
    if (lane == 0) {
      constexpr uint32_t idesc_o = idesc_bf16_f32(kTile, D) | (1u << 16);     // B MN-major
      int g = 0, nq[2] = {0, 0}, np[2] = {0, 0}, ns[2] = {0, 0}, no[2] = {0, 0};
      // the previous chunk's P V still to be issued
      bool todo[2] = {false, false}, opens[2] = {}, closes[2] = {};
      int v_use = 0, v_steps = 0;
      bool v_ready = false, ok = true;
      auto product = [&](int x) {
        if (!v_ready && !(ok = wait(kv_full(v_use % NS), (v_use / NS) & 1))) return;
        v_ready = true;
        if (!(ok = wait(p_full(x), np[x] & 1))) return;
        ++np[x];
        tc_fence_after();
        const uint32_t v = sbase + SL::kKv + (v_use % NS) * SL::kBuf;
        for (int k = 0; k < v_steps; ++k)
          mma_ts(o_at(x), s_at(x) + k * 8, smem_desc_v(v + k * 16 * 128), idesc_o, !opens[x] || k > 0);
        if (closes[x]) {
          tc_commit<1>(o_full(x));
          ++no[x];
        }
        todo[x] = false;
      };
      for (int item = blockIdx.x; item < a.items && ok; item += gridDim.x) {
        if (!it.load(a, item, end)) continue;
        bool fresh[2] = {true, true};
        const int last[2] = {it.last(0), it.last(1)};
        for (int c = 0; c < it.nc && ok; ++c) {
          const int n16 = (it.keys(c) + 15) / 16;
          const bool v_pending = todo[0] || todo[1];
          const int v_slot = v_use % NS;
          const bool sees[2] = {it.sees(0, c), it.sees(1, c)};
          bool k_ready = false;
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            if (todo[x]) product(x);
            if (!ok) break;
            if (x == 1 && v_pending) tc_commit<1>(kv_empty(v_slot));
            if (!sees[x]) continue;
            if (fresh[x] && !(ok = wait(q_full(x), nq[x] & 1))) break;
            if (!k_ready && !(ok = wait(kv_full(g % NS), (g / NS) & 1))) break;
            k_ready = true;
            tc_fence_after();
            const uint32_t idesc_s = idesc_bf16_f32(kTile, n16 * 16);
            const uint32_t q = sbase + SL::kQ + x * SL::kBuf, k = sbase + SL::kKv + (g % NS) * SL::kBuf;
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks)
              mma_ss(s_at(x), smem_desc_k_sw128(q + (ks / 4) * SL::kBox) + 2ull * (ks % 4),
                     smem_desc_k_sw128(k + (ks / 4) * SL::kBox) + 2ull * (ks % 4), idesc_s, ks > 0);
            tc_commit<1>(s_full(x));
            ++ns[x];
            if (c == last[x]) {
              tc_commit<1>(q_empty(x));
              ++nq[x];
            }
          }
          if (!ok) break;
          tc_commit<1>(kv_empty(g % NS));
          for (int x = 0; x < 2; ++x) {
            todo[x] = sees[x];
            opens[x] = fresh[x];
            closes[x] = c == last[x];
            if (sees[x]) fresh[x] = false;
          }
          v_use = g + 1;
          v_steps = n16;
          v_ready = false;
          g += 2;
        }
      }
      for (int x = 0; x < 2 && ok; ++x)
        if (todo[x]) product(x);
      // tensor memory is freed after the last MMAs have completed
      bool drained = true;
      for (int x = 0; x < 2 && drained; ++x) {
        if (ns[x] > 0) drained = wait(s_full(x), (ns[x] - 1) & 1);
        if (no[x] > 0 && drained) drained = wait(o_full(x), (no[x] - 1) & 1);
      }
    }
  } else {
    // ---- softmax: one row per thread ----
    const int x = warp >> 2;
    const int row = (warp & 3) * 32 + lane;
    const uint32_t quarter = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t ts = s_at(x) + quarter, to = o_at(x) + quarter;
    const int tok = row / a.group, head = row % a.group;
    const uint64_t sc2 = f32x2_splat(a.scale_log2);
    int ns = 0, no = 0;
    bool ok = true;
    for (int item = blockIdx.x; item < a.items && ok; item += gridDim.x) {
      if (!it.load(a, item, end)) continue;
      if (it.t1[x] == it.t0[x]) continue;
      const int t = it.t0[x] + tok;
      const bool mine = tok < a.tq && t < it.t1[x];
      Row r = {0, 0};
      if (mine) r = row_of(a, t);
      const int sink_end = mine ? min(r.start + min(a.sinks, r.lo - r.start), r.lo) : 0;
      // keys that every row of the warp admits: [all_lo, all_hi]
      const int all_lo = __reduce_max_sync(0xffffffffu, mine ? r.lo : 0);
      const int all_hi = __reduce_min_sync(0xffffffffu, mine ? t : 0x7fffffff);
      const bool any = __any_sync(0xffffffffu, mine);
      float ref = -INFINITY;             // base-2 reference of the row's exponentials
      uint64_t l2 = 0ull;
      bool begun = false;
      for (int c = 0; c < it.nc; ++c) {
        if (!it.sees(x, c)) continue;
        const int kb = it.base(c), kn = it.keys(c);
        if (!wait(s_full(x), ns & 1)) {
          ok = false;
          break;
        }
        ++ns;
        tc_fence_after();
        const bool full = kn == kTile && kb >= all_lo && kb + kTile - 1 <= all_hi && any;
        uint32_t s[4][32];
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (q * 32 < kn) tmem_ld_32cols(ts + q * 32, s[q]);
        tmem_wait_ld();
        if (!full) {
          // masked scores become -inf
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int b = kb + q * 32;
            const uint32_t in = !mine ? 0u
                : low_bits(kn - q * 32) & ((low_bits(t + 1 - b) & ~low_bits(r.lo - b)) |
                                           (low_bits(sink_end - b) & ~low_bits(r.start - b)));
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (!(in & (1u << i))) s[q][i] = 0xff800000u;
          }
        }
        float top = -INFINITY;
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int i = 0; i < 32; i += 2)
            top = fmaxf(top, fmaxf(__uint_as_float(s[q][i]), __uint_as_float(s[q][i + 1])));
        top *= a.scale_log2;
        const bool move = mine && top > ref + 8.f;
        if (__any_sync(0xffffffffu, move)) {
          const float now = move ? top : ref;
          const float keep = ref == -INFINITY ? 0.f : ex2_approx_ftz(ref - now);
          const float keep1 = move ? keep : 1.f;
          ref = now;
          const uint64_t k2 = f32x2_splat(keep1);
          l2 = f32x2_mul(l2, k2);
          if (begun) {
            // the earlier chunks' products are complete: S of this chunk was
            // issued behind them
#pragma unroll
            for (int q = 0; q < D / 16; ++q) {
              uint32_t o[16];
              tmem_ld_16cols(to + q * 16, o);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * keep1);
              tmem_st_16cols(to + q * 16, o);
            }
          }
        }
        begun = true;
        const uint64_t neg = f32x2_splat(ref == -INFINITY ? 0.f : -ref);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if (q * 32 >= kn) continue;
          uint32_t pk[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float x0, x1;
            f32x2_unpack(f32x2_fma(f32x2_pack(__uint_as_float(s[q][2 * i]), __uint_as_float(s[q][2 * i + 1])), sc2, neg),
                         x0, x1);
            const float p0 = ex2_approx_ftz(x0), p1 = ex2_approx_ftz(x1);
            l2 = f32x2_add(l2, f32x2_pack(p0, p1));
            pk[i] = pack_bf16x2(p0, p1);
          }
          tmem_st_16cols(ts + q * 16, pk);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full(x));
      }
      if (!ok || !wait(o_full(x), no & 1)) {
        ok = false;
        break;
      }
      ++no;
      tc_fence_after();
      float l0, l1;
      f32x2_unpack(l2, l0, l1);
      const float inv = 1.f / (l0 + l1);
      bf16* dst = a.out + t * a.out_stride + static_cast<int64_t>(it.h * a.group + head) * D;
      bool fine = true;
#pragma unroll
      for (int q = 0; q < D / 32; ++q) {
        uint32_t o[32];
        tmem_ld_32cols(to + q * 32, o);
        tmem_wait_ld();
        float worst = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const float y = __uint_as_float(o[i]) * inv;
          worst = fmaf(y, 0.f, worst);               // NaN once y is not finite
          o[i] = __float_as_uint(y);
        }
        fine = fine && worst == 0.f;
        if (mine) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              w[e] = pack_bf16x2(__uint_as_float(o[8 * i + 2 * e]), __uint_as_float(o[8 * i + 2 * e + 1]));
            reinterpret_cast<uint4*>(dst)[q * 4 + i] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
      tc_fence_before();
      const uint32_t odd = __ballot_sync(0xffffffffu, mine && !fine);
      if (odd != 0) {
        // does a V row that some row of the tile does not see hold the cause?
        bool cause = false;
        for (int c = 0; c < it.nc; ++c) {
          const int kb = it.base(c), kn = it.keys(c);
          if (!it.sees(x, c) || (kb >= all_lo && kb + kn - 1 <= all_hi)) continue;
          const int rows = min(kTile, ((kn + 15) / 16) * 16);
          for (int j = lane; j < rows; j += 32) {
            if (kb + j >= a.tmax) continue;
            const bf16* vr = a.v + (kb + j) * a.v_stride + it.h * D;
            for (int e = 0; e < D / 8; ++e) {
              float f[8];
              Chunk8<bf16>::load(vr + 8 * e, f);
#pragma unroll
              for (int i = 0; i < 8; ++i) cause = cause || !(fabsf(f[i]) < INFINITY);
            }
          }
        }
        if (__any_sync(0xffffffffu, cause)) {
          for (uint32_t left = odd; left != 0; left &= left - 1) {
            const int src = __ffs(left) - 1;
            const int64_t tt = __shfl_sync(0xffffffffu, t, src);
            const int hh = it.h * a.group + __shfl_sync(0xffffffffu, head, src);
            const int st = __shfl_sync(0xffffffffu, r.start, src), lo = __shfl_sync(0xffffffffu, r.lo, src);
            const int se = __shfl_sync(0xffffffffu, sink_end, src);
            auto ptr = [&](int64_t j, const bf16*& kp, const bf16*& vp) {
              kp = a.k + j * a.k_stride + it.h * D;
              vp = a.v + j * a.v_stride + it.h * D;
            };
            const bf16* q = a.q + tt * a.q_stride + static_cast<int64_t>(hh) * D;
            RowState<D> state;
            attend_keys<D>(q, a.scale_log2, st, se, ptr, state);
            attend_keys<D>(q, a.scale_log2, lo, tt + 1, ptr, state);
            const float il = 1.f / state.l;
#pragma unroll
            for (int i = 0; i < D / 32; ++i)
              a.out[tt * a.out_stride + static_cast<int64_t>(hh) * D + lane + 32 * i] =
                  __float2bfloat16_rn(state.o[i] * il);
          }
        }
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

template <int D>
cudaError_t launch(const WindowArgs& a, int T, int grid, cudaStream_t st) {
  CUtensorMap tq, tk, tv;
  const char* why = "";
  if (!make_tmap_heads(&tq, a.q, T, a.hq, D, a.q_stride, a.group, a.tq, &why) ||
      !make_tmap_heads(&tk, a.k, T, a.hkv, D, a.k_stride, 1, kTile, &why) ||
      !make_tmap_heads(&tv, a.v, T, a.hkv, D, a.v_stride, 1, kTile, &why))
    return cudaErrorInvalidValue;
  auto kernel = attn_window_kernel<D>;
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<D>::kBytes);
  if (e != cudaSuccess) return e;
  kernel<<<grid, kThreads, Smem<D>::kBytes, st>>>(tq, tk, tv, a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t attn_window_launch(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                               const void* v, int64_t v_stride, const int32_t* offsets, int n,
                               int T, int hq, int hkv, int d, int window, int sinks, void* out,
                               int64_t out_stride, int num_sms, cudaStream_t st) {
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
  const int64_t items = (static_cast<int64_t>(T) + 2 * a.tq - 1) / (2 * a.tq) * hkv;
  if (items > 0x7fffffff) return cudaErrorInvalidValue;
  a.items = static_cast<int>(items);
  const int grid = std::min(a.items, num_sms);
  return d == 64 ? launch<64>(a, T, grid, st) : launch<128>(a, T, grid, st);
}

}  // namespace rmk
