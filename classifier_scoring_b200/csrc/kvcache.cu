// Slot maps of a paged cache, and the norm, rotation and cache write of a
// step's queries and keys.
#include <cooperative_groups.h>
#include <cuda_fp8.h>

#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace rmk {
namespace {

// ---------------------------------------------------------------------------
// Slot maps.  One cluster of CTAs: every CTA scans the n requests for itself
// (n is small beside the tokens; a scan costs less than handing its result
// on), the cluster's barrier separates the reads of len_before and
// used_before from the writes of len_after and used_after, which may be the
// same memory, and the tokens and new pages are shared out over all threads.
// ---------------------------------------------------------------------------
constexpr int kSlotThreads = 1024;
constexpr int kSlotRun = 8;

__global__ void __launch_bounds__(kSlotThreads, 1)
    kv_slots_kernel(const int32_t* len_before, const int32_t* n_new, int n, int P,
                    const int32_t* __restrict__ free_pages, int n_free, const int32_t* used_before,
                    int32_t* block_table, int stride, int T, int32_t* __restrict__ offsets,
                    int32_t* __restrict__ positions, int64_t* __restrict__ slots,
                    int32_t* len_after, int32_t* used_after, int32_t* __restrict__ unserved, bool wide) {
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  extern __shared__ int32_t sh[];
  int32_t* off = sh;               // [n+1] first new token of request i
  int32_t* pg = off + n + 1;       // [n+1] first new page of request i
  int32_t* before = pg + n + 1;    // [n]
  __shared__ long long wsum_t[32], wsum_p[32];
  __shared__ int first_bad;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) first_bad = n;
  const int used = *used_before;

  // each thread sums a stretch of requests, then the stretches are scanned
  const int per = (n + kSlotThreads - 1) / kSlotThreads;
  const int i0 = min(n, tid * per), i1 = min(n, i0 + per);
  long long st = 0, sp = 0;
  for (int i = i0; i < i1; ++i) {
    const int b = len_before[i];
    const long long e = static_cast<long long>(b) + n_new[i];
    before[i] = b;
    st += n_new[i];
    sp += (e + P - 1) / P - (static_cast<long long>(b) + P - 1) / P;
  }
  long long ct = st, cp = sp;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long a = __shfl_up_sync(0xffffffffu, ct, o), b = __shfl_up_sync(0xffffffffu, cp, o);
    if (lane >= o) {
      ct += a;
      cp += b;
    }
  }
  if (lane == 31) {
    wsum_t[warp] = ct;
    wsum_p[warp] = cp;
  }
  __syncthreads();
  long long bt = ct - st, bp = cp - sp;
  for (int w = 0; w < warp; ++w) {
    bt += wsum_t[w];
    bp += wsum_p[w];
  }
  // the first request that does not fit ends the served ones; the sums of
  // later ones may be anything and are not used
  for (int i = i0; i < i1; ++i) {
    const long long b = before[i], nn = n_new[i];
    const long long have = (b + P - 1) / P, need = (b + nn + P - 1) / P;
    off[i] = static_cast<int32_t>(bt);
    pg[i] = static_cast<int32_t>(bp);
    bt += nn;
    bp += need - have;
    if (b < 0 || nn < 0 || need > stride || bt > T || used < 0 ||
        bp > static_cast<long long>(n_free) - used)
      atomicMin(&first_bad, i);
    if (i + 1 == n) {
      off[n] = static_cast<int32_t>(bt);
      pg[n] = static_cast<int32_t>(bp);
    }
  }
  __syncthreads();
  const int m = first_bad;
  const int tokens = off[m], pages = pg[m];
  cluster.sync();                  // every CTA has read what the writes below may replace

  const int at = static_cast<int>(cluster.block_rank()) * kSlotThreads + tid;
  const int all = static_cast<int>(cluster.num_blocks()) * kSlotThreads;
  for (int i = at; i <= n; i += all) {
    offsets[i] = i < m ? off[i] : tokens;
    if (i < n) len_after[i] = before[i] + (i < m ? off[i + 1] - off[i] : 0);
  }
  if (at == 0) {
    *used_after = used + pages;
    *unserved = n - m;
  }
  for (int g = at; g < pages; g += all) {
    const int i = upper_index(pg, m, g);
    const int have = (before[i] + P - 1) / P;
    block_table[static_cast<int64_t>(i) * stride + have + (g - pg[i])] = free_pages[used + g];
  }
  // kSlotRun consecutive tokens a thread: one search for their request, one
  // page lookup per page, wide stores
  for (int64_t t = static_cast<int64_t>(at) * kSlotRun; t < T; t += static_cast<int64_t>(all) * kSlotRun) {
    int64_t slot[kSlotRun];
    int pos[kSlotRun];
    int i = 0, p = 0, b = 0, rem = 0, page = 0, left = 0;      // left: tokens up to the request's end
    if (t < tokens) i = upper_index(off, m, t) - 1;
#pragma unroll
    for (int k = 0; k < kSlotRun; ++k) {
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
        b = p / P;
        rem = p - b * P;
        look = true;
      } else if (rem == P) {
        ++b;
        rem = 0;
        look = true;
      }
      if (look) {
        const int have = (before[i] + P - 1) / P;
        page = b < have ? block_table[static_cast<int64_t>(i) * stride + b]
                        : free_pages[used + pg[i] + b - have];
      }
      slot[k] = static_cast<int64_t>(page) * P + rem;
      pos[k] = p;
      ++p;
      ++rem;
      --left;
    }
    if (wide && t + kSlotRun <= T) {
#pragma unroll
      for (int k = 0; k < kSlotRun / 4; ++k)
        reinterpret_cast<int4*>(positions + t)[k] = make_int4(pos[4 * k], pos[4 * k + 1], pos[4 * k + 2], pos[4 * k + 3]);
#pragma unroll
      for (int k = 0; k < kSlotRun / 2; ++k)
        reinterpret_cast<longlong2*>(slots + t)[k] = make_longlong2(slot[2 * k], slot[2 * k + 1]);
    } else {
#pragma unroll
      for (int k = 0; k < kSlotRun; ++k)
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
// a rotation's partner dims are exchanged through shared memory, which takes
// any rot_dim.  No two warps meet, and a head is read whole before it is
// written, so the outputs may lie over the input.
// ---------------------------------------------------------------------------
constexpr int kRopeWarps = 4;
constexpr int kRopeMaxDim = 256;
constexpr int kRopeBatch = 4;                 // loads a lane has in flight

struct RopeArgs {
  const bf16* qkv;
  int64_t qkv_stride;
  bf16* q_out;
  int64_t q_stride;
  bf16* k_out;
  int64_t k_stride;
  int T, hq, hkv, d, heads;                   // heads: those the call has to look at
  const float *q_gain, *k_gain;
  float eps;
  const double* freqs;
  int rot, interleaved;
  float mscale;
  const int32_t* positions;
  void *kc, *vc;
  int64_t page_stride, n_slots;
  int page_size;
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
__global__ void __launch_bounds__(kRopeWarps * 32) qk_norm_rope_kernel(const RopeArgs a) {
  __shared__ __align__(16) float trig[kRopeWarps][2][kRopeMaxDim / 2];
  __shared__ __align__(16) float swap[kRopeWarps][32 * 8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kRopeWarps + warp;
  const int t = static_cast<int>(item / a.parts), part = static_cast<int>(item % a.parts);
  if (t >= a.T) return;
  constexpr int kPer = 32 / LP;               // heads a warp holds at once
  const int c = lane % LP, sub = lane / LP;   // this lane's dims 8c..8c+7 of its head
  const bool live = 8 * c < a.d;
  const int h0 = part * a.per_part, h1 = min(a.heads, h0 + a.per_part);
  const bf16* src = a.qkv + t * a.qkv_stride + 8 * c;
  uint4 raw[kRopeBatch];
  auto load = [&](int h) {
#pragma unroll
    for (int b = 0; b < kRopeBatch; ++b) {
      const int hh = h + b * kPer + sub;
      if (live && hh < h1) raw[b] = *reinterpret_cast<const uint4*>(src + static_cast<int64_t>(hh) * a.d);
    }
  };
  load(h0);

  const int half = a.rot / 2;
  float cs[8], sn[8];                         // of the lane's dims: y = x cs + partner sn
  if (half > 0) {
    const double pos = a.positions[t];
    for (int i = lane; i < half; i += 32) {
      // whole turns leave the angle in 64 bits, before it is rounded to fp32
      const double turns = pos * a.freqs[i] * 0.15915494309189535;
      float s, co;
      sincospif(2.f * static_cast<float>(turns - rint(turns)), &s, &co);
      trig[warp][0][i] = co * a.mscale;
      trig[warp][1][i] = s * a.mscale;
    }
    __syncwarp();
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int dim = 8 * c + e;
      cs[e] = 1.f;
      sn[e] = 0.f;
      if (dim < a.rot) {
        const bool second = a.interleaved ? (e & 1) : dim >= half;
        const int i = a.interleaved ? dim >> 1 : (second ? dim - half : dim);
        cs[e] = trig[warp][0][i];
        sn[e] = second ? trig[warp][1][i] : -trig[warp][1][i];
      }
    }
  }
  float gq[8], gk[8];
  if (a.q_gain != nullptr && live) {
    load_f32x8(a.q_gain + 8 * c, gq);
    load_f32x8(a.k_gain + 8 * c, gk);
  }
  int64_t cache_row = -1;
  if (a.kc != nullptr) {
    const int64_t slot = a.slots[t];
    if (slot >= 0 && slot < a.n_slots) {
      const int64_t page = slot / a.page_size;
      cache_row = page * a.page_stride + (slot - page * a.page_size) * a.d;
    }
  }
  // the partner dims of an 8-dim chunk under RM_ROPE_HALF
  float* mine = swap[warp] + lane * 8;
  const float* head = swap[warp] + sub * LP * 8;
  const bool whole = half % 8 == 0;           // chunks pair with chunks
  const int partner = 8 * c < half ? 8 * c + half : 8 * c - half;

  for (int h = h0; h < h1; h += kRopeBatch * kPer) {
    uint4 now[kRopeBatch];
#pragma unroll
    for (int b = 0; b < kRopeBatch; ++b) now[b] = raw[b];
    if (h + kRopeBatch * kPer < h1) load(h + kRopeBatch * kPer);
#pragma unroll
    for (int b = 0; b < kRopeBatch; ++b) {
      if (h + b * kPer >= h1) break;
      const int hh = h + b * kPer + sub;
      const bool on = live && hh < h1;
      const bool is_v = hh >= a.hq + a.hkv, is_q = hh < a.hq;
      float x[8] = {};
      if (on) {
        const uint4 v = now[b];
        x[0] = bf16_lo(v.x); x[1] = bf16_hi(v.x); x[2] = bf16_lo(v.y); x[3] = bf16_hi(v.y);
        x[4] = bf16_lo(v.z); x[5] = bf16_hi(v.z); x[6] = bf16_lo(v.w); x[7] = bf16_hi(v.w);
      }
      if (a.q_gain != nullptr) {
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
        ss = group_sum<LP>(ss);
        if (!is_v) {
          const float inv = 1.f / sqrtf(ss / static_cast<float>(a.d) + a.eps);
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] *= inv * (is_q ? gq[e] : gk[e]);
        }
      }
      if (half > 0) {
        float y[8];
        if (a.interleaved) {
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = x[e ^ 1];
        } else {
          __syncwarp();
          *reinterpret_cast<float4*>(mine) = make_float4(x[0], x[1], x[2], x[3]);
          *reinterpret_cast<float4*>(mine + 4) = make_float4(x[4], x[5], x[6], x[7]);
          __syncwarp();
          if (8 * c < a.rot) {
            if (whole) {
              load_f32x8(head + partner, y);
            } else {
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const int dim = 8 * c + e;
                y[e] = dim < a.rot ? head[dim < half ? dim + half : dim - half] : 0.f;
              }
            }
          }
        }
        if (!is_v && 8 * c < a.rot) {
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = fmaf(x[e], cs[e], 8 * c + e < a.rot ? y[e] * sn[e] : 0.f);
        }
      }
      if (!on) continue;
      if (is_q) {
        Chunk8<bf16>::store(a.q_out + t * a.q_stride + static_cast<int64_t>(hh) * a.d + 8 * c, x);
        continue;
      }
      const int kvh = hh - a.hq - (is_v ? a.hkv : 0);
      if (!is_v && a.k_out != nullptr)
        Chunk8<bf16>::store(a.k_out + t * a.k_stride + static_cast<int64_t>(kvh) * a.d + 8 * c, x);
      if (cache_row >= 0) {
        const float* scale = is_v ? a.v_scale : a.k_scale;
        store_cache8(static_cast<E*>(is_v ? a.vc : a.kc) + cache_row + static_cast<int64_t>(kvh) * a.page_size * a.d + 8 * c,
                     x, scale != nullptr ? 1.f / scale[kvh] : 1.f);
      }
    }
  }
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
  const int64_t ctas = (static_cast<int64_t>(a.T) * a.parts + kRopeWarps - 1) / kRopeWarps;
  if (ctas > 0x7fffffff) return cudaErrorInvalidValue;
  qk_norm_rope_kernel<E, LP><<<static_cast<unsigned>(ctas), kRopeWarps * 32, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t kv_slots_launch(const int32_t* len_before, const int32_t* n_new, int n, int page_size,
                            const int32_t* free_pages, int n_free, const int32_t* used_before,
                            int32_t* block_table, int stride, int T, int32_t* offsets,
                            int32_t* positions, int64_t* slots, int32_t* len_after,
                            int32_t* used_after, int32_t* unserved, cudaStream_t st) {
  const size_t smem = (3 * static_cast<size_t>(n) + 2) * 4;
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(
        kv_slots_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  // one CTA until its threads have more than one run of tokens each
  const int ctas = T > kSlotRun * kSlotThreads ? 8 : 1;
  const bool wide = ((reinterpret_cast<uintptr_t>(positions) | reinterpret_cast<uintptr_t>(slots)) & 15) == 0;
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kSlotThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv_slots_kernel, len_before, n_new, n, page_size, free_pages,
                            n_free, used_before, block_table, stride, T, offsets, positions, slots,
                            len_after, used_after, unserved, wide);
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
  a.eps = eps;
  a.freqs = rope.freqs;
  a.rot = rope.rot_dim;
  a.interleaved = rope.layout;
  a.mscale = rope.mscale;
  a.positions = positions;
  a.kc = cache.k;
  a.vc = cache.v;
  a.page_stride = cache.page_stride;
  a.n_slots = static_cast<int64_t>(cache.n_pages) * cache.page_size;
  a.page_size = cache.page_size;
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
