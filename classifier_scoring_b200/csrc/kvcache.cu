// Slot maps of a paged cache, and the norm, rotation and cache write of a
// step's queries and keys.
#include <cooperative_groups.h>
#include <cuda_fp8.h>

#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "paging.cuh"

namespace rmk {
namespace {

RMK_BOUNDS_UNIT(kvcache)

// ---------------------------------------------------------------------------
// Slot maps.  Bound by latency: a few dependent reads, a scan and the writes
// (on the device 2.9 us for a step of 64 requests, 5.9 us for 251k tokens of
// 1000, 3 MB; a call among others 8 us, the host's time).
// Every CTA scans the n requests for itself (n is small beside the tokens, and
// a scan costs less than handing its result on through memory), then the
// tokens and new pages are shared out over all threads.  len_after and
// used_after may be len_before and used_before: then all CTAs form one cluster
// whose barrier separates the reads from the writes (24 us for the 251k tokens).
// ---------------------------------------------------------------------------
// Tokens a thread takes in a row: eight share a search, a page lookup and wide
// stores (251k tokens of 1000 requests: 5.9 us); one where every thread has at
// most one, whose lookups then do not wait for one another.
constexpr int kSlotRun = 8;
constexpr int kSlotSingles = 148 * 256;
constexpr int kSlotStaged = 1024;       // requests
constexpr int kMaxSlotSeqs = 16384;

template <int kRun>
__global__ void __launch_bounds__(1024, 1)
    kv_slots_kernel(const int32_t* len_before, const int32_t* n_new, int n, PageDiv div,
                    const int32_t* __restrict__ free_pages, int n_free, const int32_t* used_before,
                    int32_t* block_table, int stride, int T, int32_t* __restrict__ offsets,
                    int32_t* __restrict__ positions, int64_t* __restrict__ slots,
                    int32_t* len_after, int32_t* used_after, int32_t* __restrict__ unserved,
                    bool wide, bool cluster) {
  extern __shared__ int32_t sh[];
  int32_t* off = sh;               // [n+1] first new token of request i
  int32_t* pg = off + n + 1;       // [n+1] first new page of request i
  int32_t* before = pg + n + 1;    // [n]
  __shared__ long long wsum_t[32], wsum_p[32];
  __shared__ int first_bad;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int threads = blockDim.x, P = div.P;
  if (tid == 0) first_bad = n;
  pdl_wait();
  const int used = *used_before;

  // each thread sums a stretch of requests, then the stretches are scanned.
  // What can never be served counts nothing: it ends the served ones below.
  // Long stretches are read by all threads in order first, and have odd lengths
  // so that the threads read them from different banks (16384 requests: 14 us,
  // 39 straight from memory; for 1000 the extra barrier costs 0.8 us of 3.6).
  const bool staged = n > kSlotStaged;
  if (staged) {
#pragma unroll 4
    for (int i = tid; i < n; i += threads) {
      before[i] = len_before[i];
      off[i] = n_new[i];
    }
    __syncthreads();
  }
  const int per = ((n + threads - 1) / threads) | (staged ? 1 : 0);
  const int i0 = min(n, tid * per), i1 = min(n, i0 + per);
  auto never = [&](int b, int m) { return b < 0 || m < 0 || m > 0x7fffffff - b; };
  long long st = 0, sp = 0;
  for (int i = i0; i < i1; ++i) {
    const int b = staged ? before[i] : len_before[i], m = staged ? off[i] : n_new[i];
    if (!staged) {
      before[i] = b;
      off[i] = m;
    }
    if (never(b, m)) continue;
    st += m;
    sp += div.ceil(b + m) - div.ceil(b);
  }
  long long ct = st, cp = sp;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, ct, o), y = __shfl_up_sync(0xffffffffu, cp, o);
    if (lane >= o) {
      ct += x;
      cp += y;
    }
  }
  if (lane == 31) {
    wsum_t[warp] = ct;
    wsum_p[warp] = cp;
  }
  __syncthreads();
  long long bt = ct - st, bp = cp - sp;
  {
    long long x = lane < warp ? wsum_t[lane] : 0, y = lane < warp ? wsum_p[lane] : 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      x += __shfl_xor_sync(0xffffffffu, x, o);
      y += __shfl_xor_sync(0xffffffffu, y, o);
    }
    bt += x;
    bp += y;
  }
  // the first request that does not fit ends the served ones; the sums of
  // later ones are not used
  for (int i = i0; i < i1; ++i) {
    const int b = before[i], m = off[i];
    const bool no = never(b, m);
    const int need = no ? 0 : div.ceil(b + m), have = no ? 0 : div.ceil(b);
    off[i] = static_cast<int32_t>(bt);
    pg[i] = static_cast<int32_t>(bp);
    bt += no ? 0 : m;
    bp += need - have;
    if (no || need > stride || bt > T || used < 0 || bp > static_cast<long long>(n_free) - used)
      atomicMin(&first_bad, i);
    if (i + 1 == n) {
      off[n] = static_cast<int32_t>(bt);
      pg[n] = static_cast<int32_t>(bp);
    }
  }
  __syncthreads();
  const int m = first_bad;
  const int tokens = off[m], pages = pg[m];
  if (cluster)                     // every CTA has read what the writes below may replace
    cooperative_groups::this_cluster().sync();

  const int at = static_cast<int>(blockIdx.x) * threads + tid;
  const int all = static_cast<int>(gridDim.x) * threads;
  for (int i = at; i <= n; i += all) {
    offsets[i] = i < m ? off[i] : tokens;
    if (i < n) len_after[i] = before[i] + (i < m ? off[i + 1] - off[i] : 0);
  }
  if (at == 0) {
    *used_after = used + pages;
    *unserved = n - m;
  }
  for (int g = at; g < pages; g += all) {
    const int i = upper_index(pg, m, g), b = div.ceil(before[i]) + (g - pg[i]);
    if (!in_bounds(b >= 0 && b < stride && used + g < n_free)) continue;
    block_table[static_cast<int64_t>(i) * stride + b] = free_pages[used + g];
  }
  // kRun consecutive tokens a thread: one search for their request, one
  // page lookup per page, wide stores
  for (int64_t t = static_cast<int64_t>(at) * kRun; t < T; t += static_cast<int64_t>(all) * kRun) {
    int64_t slot[kRun];
    int pos[kRun];
    int i = 0, p = 0, b = 0, rem = 0, page = 0, left = 0;      // left: tokens up to the request's end
    if (t < tokens) i = upper_index(off, m, t) - 1;
#pragma unroll
    for (int k = 0; k < kRun; ++k) {
      if (t + k >= tokens) {
        slot[k] = -1;
        pos[k] = 0;
        continue;
      }
      bool look = false;
      if (left == 0) {                                          // the next request that has tokens here
        do ++i; while (off[i + 1] <= t + k);
        p = before[i] + static_cast<int>(t + k - off[i]);
        left = static_cast<int>(off[i + 1] - (t + k));
        b = div.floor(p);
        rem = p - b * P;
        look = true;
      } else if (rem == P) {
        ++b;
        rem = 0;
        look = true;
      }
      if (look) {
        const int have = div.ceil(before[i]);
        if (in_bounds(i < m && b >= 0 && (b < have ? b < stride : used + pg[i] + b - have < n_free)))
          page = b < have ? block_table[static_cast<int64_t>(i) * stride + b]
                          : free_pages[used + pg[i] + b - have];
      }
      slot[k] = static_cast<int64_t>(page) * P + rem;
      pos[k] = p;
      ++p;
      ++rem;
      --left;
    }
    if (kRun % 4 == 0 && wide && t + kRun <= T) {
#pragma unroll
      for (int k = 0; k < kRun / 4; ++k)
        reinterpret_cast<int4*>(positions + t)[k] = make_int4(pos[4 * k], pos[4 * k + 1], pos[4 * k + 2], pos[4 * k + 3]);
#pragma unroll
      for (int k = 0; k < kRun / 2; ++k)
        reinterpret_cast<longlong2*>(slots + t)[k] = make_longlong2(slot[2 * k], slot[2 * k + 1]);
    } else {
#pragma unroll
      for (int k = 0; k < kRun; ++k)
        if (t + k < T) {
          slots[t + k] = slot[k];
          positions[t + k] = pos[k];
        }
    }
  }
}

// ---------------------------------------------------------------------------
// Norm, rotation and cache write.  Bound by memory: a token's heads are read
// and written once (72 bytes a 16-byte chunk of instructions leave the issue
// slots half idle at full bandwidth).  A warp takes one token, or a run of its
// heads when there are few tokens: the token's cosines and sines are computed
// once per warp and stay in registers for all its heads, as do the gains.
// LP lanes (a power of two from head_dim / 8 on) hold a head, eight dims each;
// a rotation's partner dims come by a shuffle where they lie a power of two of
// lanes away, else through shared memory, which takes any rot_dim.  No two
// warps meet, and a head is read whole before it is written, so the outputs
// may lie over the input.
// Measured on B200, 25k tokens of 16 + 16 + 16 heads of 128, normed and
// rotated into a bf16 cache: 142-144 us among calls on other inputs, 5.1 TB/s,
// 78% of a copy's rate (138-141 replayed on the same ones; partners through
// shared memory: 3 us more).
// ---------------------------------------------------------------------------
constexpr int kRopeWarps = 4;
constexpr int kRopeMaxDim = 256;
// Loads a lane has in flight, and blocks per SM that the registers allow: long
// heads take more loads, short ones (whose warps are soon done) more warps.
template <int LP> struct RopeShape {
  static constexpr int kBatch = LP >= 16 ? 4 : 2;
  static constexpr int kBlocks = LP >= 16 ? 4 : 5;
  static constexpr bool kSlotFirst = LP < 16;           // the slot's load over the trigonometry: long heads have no registers for it
};

struct RopeArgs {
  const bf16* qkv;
  int64_t qkv_stride;
  bf16* q_out;
  int64_t q_stride;
  bf16* k_out;
  int64_t k_stride;
  int T, hq, hkv, d, heads;                   // heads: those the call has to look at
  const float *q_gain, *k_gain;
  bool wide_gains;                            // both 16-byte aligned
  float eps, inv_d;
  const double* freqs;
  int rot, interleaved;
  int swap_lanes;                             // rot / 16 where that is a power of two, else 0
  float mscale;
  const int32_t* positions;
  void *kc, *vc;
  int64_t page_stride, n_slots;
  PageDiv div;
  const float *k_scale, *v_scale;
  const int64_t* slots;
  int parts, per_part;                        // warps per token, heads per warp
};

__device__ __forceinline__ void store_cache8(bf16* p, const float* f, float) { Chunk8<bf16>::store(p, f); }
__device__ __forceinline__ void store_cache8(__nv_fp8_e4m3* p, const float* f, float inv) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(f[4 * i] * inv, f[4 * i + 1] * inv), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(f[4 * i + 2] * inv, f[4 * i + 3] * inv), __NV_SATFINITE, __NV_E4M3);
    w[i] = lo | (hi << 16);
  }
  *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
}

template <typename E, int LP>
__global__ void __launch_bounds__(kRopeWarps * 32, RopeShape<LP>::kBlocks) qk_norm_rope_kernel(const RopeArgs a) {
  constexpr int kRopeBatch = RopeShape<LP>::kBatch;
  __shared__ __align__(16) float trig[kRopeWarps][2][kRopeMaxDim / 2];
  __shared__ __align__(16) float swap[kRopeWarps][32 * 8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  // a CTA's warps take tokens, or runs of one token's heads
  const int t = a.parts == 1 ? static_cast<int>(blockIdx.x) * kRopeWarps + warp : static_cast<int>(blockIdx.x);
  const int part = a.parts == 1 ? 0 : static_cast<int>(blockIdx.y) * kRopeWarps + warp;
  if (t >= a.T || part >= a.parts) return;
  const int position = a.rot > 0 ? a.positions[t] : 0;
  const int64_t early = RopeShape<LP>::kSlotFirst && a.kc != nullptr ? a.slots[t] : -1;
  constexpr int kPer = 32 / LP;               // heads a warp holds at once
  const int c = lane % LP, sub = lane / LP;   // this lane's dims 8c..8c+7 of its head
  const bool live = 8 * c < a.d;
  const int h0 = part * a.per_part, h1 = min(a.heads, h0 + a.per_part);
  // the row's heads by kind, this warp's share of each: [from[k], from[k+1]) of
  // queries, keys, values
  const int qk = a.hq + a.hkv;
  const int from[4] = {h0, min(max(h0, a.hq), h1), min(max(h0, qk), h1), h1};
  const bf16* src = a.qkv + t * a.qkv_stride + 8 * c + static_cast<int64_t>(sub) * a.d;
  const int step = kPer * a.d;
  // A batch of heads is loaded while the one before it is worked on, the first
  // one under the trigonometry.
  uint4 raw[kRopeBatch];
  auto load = [&](int h, int hb) {
#pragma unroll
    for (int b = 0; b < kRopeBatch; ++b)
      if (live && h + sub + b * kPer < hb) raw[b] = *reinterpret_cast<const uint4*>(src + static_cast<int64_t>(h) * a.d + b * step);
  };
  {
    const int k = from[1] > from[0] ? 0 : (from[2] > from[1] ? 1 : 2);
    load(from[k], from[k + 1]);
  }
  const int half = a.rot / 2;
  uint64_t cs[4], sn[4];                      // of the lane's dims: y = x cs + partner sn
  if (half > 0) {
    const double pos = position;
    for (int i = lane; i < half; i += 32) {
      // whole turns leave the angle in 64 bits, before it is rounded to fp32
      const double turns = pos * a.freqs[i] * 0.15915494309189535;
      float s, co;
      sincospif(2.f * static_cast<float>(turns - rint(turns)), &s, &co);
      trig[warp][0][i] = co * a.mscale;
      trig[warp][1][i] = s * a.mscale;
    }
    __syncwarp();
    float f[16];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int dim = 8 * c + e;
      f[e] = 1.f;
      f[8 + e] = 0.f;
      if (dim < a.rot) {
        const bool second = a.interleaved ? (e & 1) : dim >= half;
        const int i = a.interleaved ? dim >> 1 : (second ? dim - half : dim);
        f[e] = trig[warp][0][i];
        f[8 + e] = second ? trig[warp][1][i] : -trig[warp][1][i];
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      cs[e] = f32x2_pack(f[2 * e], f[2 * e + 1]);
      sn[e] = f32x2_pack(f[8 + 2 * e], f[8 + 2 * e + 1]);
    }
  }
  int64_t cache_row = -1;
  if (a.kc != nullptr) {
    const int64_t slot = RopeShape<LP>::kSlotFirst ? early : a.slots[t];
    if (slot >= 0 && slot < a.n_slots) {
      const int64_t page = slot <= 0x7fffffff ? a.div.floor(static_cast<int>(slot)) : slot / a.div.P;
      if (in_bounds(slot - page * a.div.P >= 0 && slot - page * a.div.P < a.div.P))
        cache_row = page * a.page_stride + (slot - page * a.div.P) * a.d;
    }
  }
  // the partner dims of an 8-dim chunk under RM_ROPE_HALF
  float* mine = swap[warp] + lane * 8;
  const float* head = swap[warp] + sub * LP * 8;
  const bool whole = half % 8 == 0;           // chunks pair with chunks
  const int partner = 8 * c < half ? 8 * c + half : 8 * c - half;
  const bool turns = 8 * c < a.rot;

  // heads [ha, hb) of one kind; head h of the row is head h - first of its
  // kind, written to out (row of this token, or null) and to the cache
  auto section = [&](auto kind, const int k, int first, const float* gain_at, bf16* out, E* cache,
                     const float* scale) {
    constexpr bool kValue = decltype(kind)::value;
    const int ha = from[k], hb = from[k + 1];
    if (ha >= hb) return;
    const bool norm = !kValue && gain_at != nullptr;
    uint64_t gain[4];
    if (norm && live) {
      if (a.wide_gains) {
        const float4 g0 = reinterpret_cast<const float4*>(gain_at + 8 * c)[0];
        const float4 g1 = reinterpret_cast<const float4*>(gain_at + 8 * c)[1];
        gain[0] = f32x2_pack(g0.x, g0.y);
        gain[1] = f32x2_pack(g0.z, g0.w);
        gain[2] = f32x2_pack(g1.x, g1.y);
        gain[3] = f32x2_pack(g1.z, g1.w);
      } else {                                // a slice of a packed parameter buffer
#pragma unroll
        for (int e = 0; e < 4; ++e) gain[e] = f32x2_pack(gain_at[8 * c + 2 * e], gain_at[8 * c + 2 * e + 1]);
      }
    }
    const int cache_head = a.div.P * a.d;
    int own = ha + sub - first;               // this lane's head among its kind
    bf16* dst = out == nullptr ? nullptr : out + static_cast<int64_t>(own) * a.d + 8 * c;
    E* cdst = cache == nullptr ? nullptr : cache + cache_row + static_cast<int64_t>(own) * cache_head + 8 * c;
    for (int h = ha + sub; h - sub < hb; h += kRopeBatch * kPer) {
      uint4 now[kRopeBatch];
#pragma unroll
      for (int b = 0; b < kRopeBatch; ++b) now[b] = live && h + b * kPer < hb ? raw[b] : make_uint4(0u, 0u, 0u, 0u);
      if (h - sub + kRopeBatch * kPer < hb) load(h - sub + kRopeBatch * kPer, hb);
      else if (k < 2 && from[k + 2] > hb) load(hb, from[k + 2]);
      else if (k < 1) load(from[2], from[3]);
#pragma unroll
      for (int b = 0; b < kRopeBatch; ++b) {
        if (h - sub + b * kPer >= hb) break;
        uint64_t x[4] = {f32x2_pack(bf16_lo(now[b].x), bf16_hi(now[b].x)), f32x2_pack(bf16_lo(now[b].y), bf16_hi(now[b].y)),
                         f32x2_pack(bf16_lo(now[b].z), bf16_hi(now[b].z)), f32x2_pack(bf16_lo(now[b].w), bf16_hi(now[b].w))};
        if (norm) {
          uint64_t ss2 = f32x2_mul(x[0], x[0]);
#pragma unroll
          for (int e = 1; e < 4; ++e) ss2 = f32x2_fma(x[e], x[e], ss2);
          float s0, s1;
          f32x2_unpack(ss2, s0, s1);
          const float ss = group_sum<LP>(s0 + s1);
          const uint64_t inv = f32x2_splat(rsqrtf(fmaf(ss, a.inv_d, a.eps)));
#pragma unroll
          for (int e = 0; e < 4; ++e) x[e] = f32x2_mul(f32x2_mul(x[e], inv), gain[e]);
        }
        if (!kValue && half > 0) {
          uint64_t y[4];
          if (a.interleaved) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float lo, hi;
              f32x2_unpack(x[e], lo, hi);
              y[e] = f32x2_pack(hi, lo);
            }
          } else if (a.swap_lanes != 0) {     // the partner chunk is a fixed lane away
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] = __shfl_xor_sync(0xffffffffu, x[e], a.swap_lanes);
          } else {
            __syncwarp();
            reinterpret_cast<ulonglong2*>(mine)[0] = make_ulonglong2(x[0], x[1]);
            reinterpret_cast<ulonglong2*>(mine)[1] = make_ulonglong2(x[2], x[3]);
            __syncwarp();
            if (turns) {
              if (whole) {
                const ulonglong2 y0 = reinterpret_cast<const ulonglong2*>(head + partner)[0];
                const ulonglong2 y1 = reinterpret_cast<const ulonglong2*>(head + partner)[1];
                y[0] = y0.x; y[1] = y0.y; y[2] = y1.x; y[3] = y1.y;
              } else {
                float f[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  const int dim = 8 * c + e;
                  f[e] = dim < a.rot ? head[dim < half ? dim + half : dim - half] : 0.f;
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) y[e] = f32x2_pack(f[2 * e], f[2 * e + 1]);
              }
            }
          }
          if (turns) {
            if (8 * c + 8 <= a.rot) {
#pragma unroll
              for (int e = 0; e < 4; ++e) x[e] = f32x2_fma(x[e], cs[e], f32x2_mul(y[e], sn[e]));
            } else {                          // dims behind rot_dim stay, whatever their neighbours hold
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (8 * c + 2 * e < a.rot) x[e] = f32x2_fma(x[e], cs[e], f32x2_mul(y[e], sn[e]));
            }
          }
        }
        if (live && h + b * kPer < hb) {
          float f[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) f32x2_unpack(x[e], f[2 * e], f[2 * e + 1]);
          if (dst != nullptr) Chunk8<bf16>::store(dst + b * step, f);
          if (cdst != nullptr)
            store_cache8(cdst + static_cast<int64_t>(b * kPer) * cache_head, f,
                         scale != nullptr ? 1.f / scale[own + b * kPer] : 1.f);
        }
      }
      own += kRopeBatch * kPer;
      if (dst != nullptr) dst += kRopeBatch * step;
      if (cdst != nullptr) cdst += static_cast<int64_t>(kRopeBatch * kPer) * cache_head;
    }
  };
  using Turned = std::integral_constant<bool, false>;
  using Value = std::integral_constant<bool, true>;
  E* kc = cache_row < 0 ? nullptr : static_cast<E*>(a.kc);
  E* vc = cache_row < 0 ? nullptr : static_cast<E*>(a.vc);
  section(Turned{}, 0, 0, a.q_gain, a.q_out + t * a.q_stride, static_cast<E*>(nullptr), nullptr);
  section(Turned{}, 1, a.hq, a.k_gain, a.k_out == nullptr ? nullptr : a.k_out + t * a.k_stride, kc, a.k_scale);
  section(Value{}, 2, qk, nullptr, static_cast<bf16*>(nullptr), vc, a.v_scale);
}

template <typename E, int LP> cudaError_t rope_go(RopeArgs a, int num_sms, cudaStream_t st) {
  // one warp per token once that fills the GPU (sixteen warps an SM); fewer
  // tokens are cut into runs of heads
  constexpr int kPer = 32 / LP;
  const int steps = (a.heads + kPer - 1) / kPer;
  const int want = std::max(1, std::min(steps, 16 * num_sms / std::max(1, a.T)));
  const int per = (steps + want - 1) / want;
  a.per_part = per * kPer;
  a.parts = (steps + per - 1) / per;
  const dim3 grid = a.parts == 1 ? dim3((static_cast<unsigned>(a.T) + kRopeWarps - 1) / kRopeWarps)
                                 : dim3(static_cast<unsigned>(a.T), (a.parts + kRopeWarps - 1) / kRopeWarps);
  PdlScope pdl(true);
  return launch_k(qk_norm_rope_kernel<E, LP>, grid, dim3(kRopeWarps * 32), 0, st, a);
}

template <int kRun>
cudaError_t slots_go(const int32_t* len_before, const int32_t* n_new, int n, int page_size,
                     const int32_t* free_pages, int n_free, const int32_t* used_before,
                     int32_t* block_table, int stride, int T, int32_t* offsets,
                     int32_t* positions, int64_t* slots, int32_t* len_after,
                     int32_t* used_after, int32_t* unserved, cudaStream_t st) {
  const size_t smem = (3 * static_cast<size_t>(n) + 2) * 4;
  if (smem > 48 * 1024) {
    static std::atomic<unsigned long long> allowed{0};
    const cudaError_t e = allow_smem(kv_slots_kernel<kRun>, (3 * kMaxSlotSeqs + 2) * 4, allowed);
    if (e != cudaSuccess) return e;
  }
  const PageDiv div = page_div(page_size);
  // One CTA for a step's few tokens; a run of tokens per thread over many CTAs
  // for prompts (251k tokens of 1000 requests: 24 us on one cluster of eight
  // CTAs, 5.9 us on 123); one cluster when the lengths advance in place.
  const int64_t runs = (static_cast<int64_t>(T) + kRun - 1) / kRun;
  const bool in_place = len_after == len_before || used_after == used_before;
  const int threads = n > kSlotStaged ? 1024 : 256;
  int ctas = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(148, (runs + threads - 1) / threads)));
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  const bool cluster = in_place && ctas > 1;
  if (cluster) attr[1].val.clusterDim.x = ctas = 8;
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(cluster ? 1024 : threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = cluster ? 2 : 1;
  const bool wide = ((reinterpret_cast<uintptr_t>(positions) | reinterpret_cast<uintptr_t>(slots)) & 15) == 0;
  return cudaLaunchKernelEx(&cfg, kv_slots_kernel<kRun>, len_before, n_new, n, div, free_pages, n_free,
                            used_before, block_table, stride, T, offsets, positions, slots,
                            len_after, used_after, unserved, wide, cluster);
}

}  // namespace

cudaError_t bounds_errors_kvcache(int32_t* out, bool reset) {
  cudaError_t e = cudaMemcpyFromSymbol(out, g_bounds_kvcache, sizeof(int32_t));
  if (e == cudaSuccess && reset) {
    const int32_t zero = 0;
    e = cudaMemcpyToSymbol(g_bounds_kvcache, &zero, sizeof(int32_t));
  }
  return e;
}

cudaError_t kv_slots_launch(const int32_t* len_before, const int32_t* n_new, int n, int page_size,
                            const int32_t* free_pages, int n_free, const int32_t* used_before,
                            int32_t* block_table, int stride, int T, int32_t* offsets,
                            int32_t* positions, int64_t* slots, int32_t* len_after,
                            int32_t* used_after, int32_t* unserved, cudaStream_t st) {
  auto go = T <= kSlotSingles ? slots_go<1> : slots_go<kSlotRun>;
  return go(len_before, n_new, n, page_size, free_pages, n_free, used_before, block_table, stride, T, offsets,
            positions, slots, len_after, used_after, unserved, st);
}

cudaError_t qk_norm_rope_launch(const void* qkv, int64_t qkv_stride, void* q_out, int64_t q_stride,
                                void* k_out, int64_t k_stride, int T, int hq, int hkv, int d,
                                const float* q_gain, const float* k_gain, float eps,
                                const rm_rope& rope, const int32_t* positions,
                                const rm_kv_cache& cache, const int64_t* slots, int num_sms,
                                cudaStream_t st) {
  if (T < 1) return cudaSuccess;
  RopeArgs a;
  a.qkv = static_cast<const bf16*>(qkv);
  a.qkv_stride = qkv_stride;
  a.q_out = static_cast<bf16*>(q_out);
  a.q_stride = q_stride;
  a.k_out = static_cast<bf16*>(k_out);
  a.k_stride = k_stride;
  a.T = T;
  a.hq = hq;
  a.hkv = hkv;
  a.d = d;
  a.heads = cache.k != nullptr ? hq + 2 * hkv : (k_out != nullptr ? hq + hkv : hq);
  a.q_gain = q_gain;
  a.k_gain = k_gain;
  a.wide_gains = ((reinterpret_cast<uintptr_t>(q_gain) | reinterpret_cast<uintptr_t>(k_gain)) & 15) == 0;
  a.eps = eps;
  a.inv_d = 1.f / static_cast<float>(d);
  a.freqs = rope.freqs;
  a.rot = rope.rot_dim;
  a.interleaved = rope.layout;
  const int apart = rope.rot_dim % 16 == 0 ? rope.rot_dim / 16 : 0;
  a.swap_lanes = (apart & (apart - 1)) == 0 ? apart : 0;
  a.mscale = rope.mscale;
  a.positions = positions;
  a.kc = cache.k;
  a.vc = cache.v;
  a.page_stride = cache.page_stride;
  a.n_slots = static_cast<int64_t>(cache.n_pages) * cache.page_size;
  a.div = page_div(std::max(1, cache.page_size));
  a.k_scale = cache.k_scale;
  a.v_scale = cache.v_scale;
  a.slots = slots;
  auto go = [&](auto elem) {
    using E = decltype(elem);
    if (d <= 8) return rope_go<E, 1>(a, num_sms, st);
    if (d <= 16) return rope_go<E, 2>(a, num_sms, st);
    if (d <= 32) return rope_go<E, 4>(a, num_sms, st);
    if (d <= 64) return rope_go<E, 8>(a, num_sms, st);
    if (d <= 128) return rope_go<E, 16>(a, num_sms, st);
    return rope_go<E, 32>(a, num_sms, st);
  };
  return cache.dtype == RM_E4M3 ? go(__nv_fp8_e4m3{}) : go(bf16{});
}

}  // namespace rmk
