// Slot maps of a paged cache, and the norm, rotation and cache write of a
// step's queries and keys.
#include <cooperative_groups.h>
#include <cuda_fp8.h>

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

__global__ void __launch_bounds__(kSlotThreads, 1)
    kv_slots_kernel(const int32_t* len_before, const int32_t* n_new, int n, int P,
                    const int32_t* __restrict__ free_pages, int n_free, const int32_t* used_before,
                    int32_t* block_table, int stride, int T, int32_t* __restrict__ offsets,
                    int32_t* __restrict__ positions, int64_t* __restrict__ slots,
                    int32_t* len_after, int32_t* used_after, int32_t* __restrict__ unserved) {
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
  for (int t = at; t < T; t += all) {
    int64_t slot = -1;
    int pos = 0;
    if (t < tokens) {
      const int i = upper_index(off, m, t);
      pos = before[i] + (t - off[i]);
      const int have = (before[i] + P - 1) / P, b = pos / P;
      const int page = b < have ? block_table[static_cast<int64_t>(i) * stride + b]
                                : free_pages[used + pg[i] + b - have];
      slot = static_cast<int64_t>(page) * P + (pos - b * P);
    }
    slots[t] = slot;
    positions[t] = pos;
  }
}

// ---------------------------------------------------------------------------
// Norm, rotation and cache write: one CTA per token, a warp per head.
// ---------------------------------------------------------------------------
constexpr int kRopeThreads = 256;
constexpr int kRopeMaxDim = 256;

template <typename E> struct CacheElem;
template <> struct CacheElem<bf16> {
  static __device__ __forceinline__ bf16 from(float v, float) { return __float2bfloat16_rn(v); }
};
template <> struct CacheElem<__nv_fp8_e4m3> {
  static __device__ __forceinline__ __nv_fp8_e4m3 from(float v, float inv) {
    __nv_fp8_e4m3 r;
    r.__x = __nv_cvt_float_to_fp8(v * inv, __NV_SATFINITE, __NV_E4M3);
    return r;
  }
};

template <typename E>
__global__ void __launch_bounds__(kRopeThreads)
    qk_norm_rope_kernel(const bf16* qkv, int64_t qkv_stride, bf16* q_out, int64_t q_stride,
                        bf16* k_out, int64_t k_stride, int hq, int hkv, int d,
                        const float* __restrict__ q_gain, const float* __restrict__ k_gain,
                        float eps, const double* __restrict__ freqs, int rot, int interleaved,
                        float mscale, const int32_t* __restrict__ positions, E* kc, E* vc,
                        int64_t page_stride, int64_t n_slots, int page_size,
                        const float* __restrict__ k_scale, const float* __restrict__ v_scale,
                        const int64_t* __restrict__ slots) {
  __shared__ float cs[kRopeMaxDim / 2], sn[kRopeMaxDim / 2];
  __shared__ float row[kRopeThreads / 32][kRopeMaxDim];
  const int t = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int half = rot / 2;
  for (int i = threadIdx.x; i < half; i += kRopeThreads) {
    // whole turns leave the angle before it is rounded to fp32
    const double turns = positions[t] * freqs[i] * 0.15915494309189535;
    float s, c;
    sincospif(2.f * static_cast<float>(turns - rint(turns)), &s, &c);
    cs[i] = c * mscale;
    sn[i] = s * mscale;
  }
  __syncthreads();
  int64_t cache_row = -1;
  if (kc != nullptr) {
    const int64_t slot = slots[t];
    if (slot >= 0 && slot < n_slots)
      cache_row = (slot / page_size) * page_stride + (slot % page_size) * d;
  }
  const bf16* src = qkv + t * qkv_stride;
  for (int h = warp; h < hq + 2 * hkv; h += kRopeThreads / 32) {
    const bool is_v = h >= hq + hkv;
    if (is_v && cache_row < 0) continue;
    float* r = row[warp];
    float ss = 0.f;
    for (int c = lane; c < d; c += 32) {
      const float x = to_f32(src[h * d + c]);
      r[c] = x;
      ss = fmaf(x, x, ss);
    }
    __syncwarp();
    const float* gain = h < hq ? q_gain : k_gain;
    const float inv = gain != nullptr ? 1.f / sqrtf(group_sum<32>(ss) / d + eps) : 1.f;
    const int kvh = h < hq ? 0 : (h - hq) % hkv;
    for (int c = lane; c < d; c += 32) {
      float y = r[c];
      if (!is_v) {
        auto val = [&](int e) { return gain != nullptr ? r[e] * inv * gain[e] : r[e]; };
        y = val(c);
        if (c < rot) {
          const int i = interleaved ? c >> 1 : (c < half ? c : c - half);
          const bool second = interleaved ? (c & 1) : c >= half;
          const int pc = interleaved ? c ^ 1 : (second ? c - half : c + half);
          y = second ? fmaf(y, cs[i], val(pc) * sn[i]) : fmaf(y, cs[i], -val(pc) * sn[i]);
        }
      }
      if (h < hq) q_out[t * q_stride + h * d + c] = __float2bfloat16_rn(y);
      else if (!is_v && k_out != nullptr) k_out[t * k_stride + kvh * d + c] = __float2bfloat16_rn(y);
      if (h >= hq && cache_row >= 0) {
        const float* scale = is_v ? v_scale : k_scale;
        (is_v ? vc : kc)[cache_row + static_cast<int64_t>(kvh) * page_size * d + c] =
            CacheElem<E>::from(y, scale != nullptr ? 1.f / scale[kvh] : 1.f);
      }
    }
    __syncwarp();
  }
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
  const int ctas = T > 2 * kSlotThreads ? 8 : 1;
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
                            len_after, used_after, unserved);
}

cudaError_t qk_norm_rope_launch(const void* qkv, int64_t qkv_stride, void* q_out, int64_t q_stride,
                                void* k_out, int64_t k_stride, int T, int hq, int hkv, int d,
                                const float* q_gain, const float* k_gain, float eps,
                                const rm_rope& rope, const int32_t* positions,
                                const rm_kv_cache& cache, const int64_t* slots, cudaStream_t st) {
  if (T < 1) return cudaSuccess;
  const int64_t n_slots = static_cast<int64_t>(cache.n_pages) * cache.page_size;
  auto go = [&](auto* kernel, auto* kc, auto* vc) {
    kernel<<<T, kRopeThreads, 0, st>>>(
        static_cast<const bf16*>(qkv), qkv_stride, static_cast<bf16*>(q_out), q_stride,
        static_cast<bf16*>(k_out), k_stride, hq, hkv, d, q_gain, k_gain, eps, rope.freqs,
        rope.rot_dim, rope.layout, rope.mscale, positions, kc, vc, cache.page_stride, n_slots,
        cache.page_size, cache.k_scale, cache.v_scale, slots);
    return cudaGetLastError();
  };
  if (cache.dtype == RM_E4M3)
    return go(qk_norm_rope_kernel<__nv_fp8_e4m3>, static_cast<__nv_fp8_e4m3*>(cache.k),
              static_cast<__nv_fp8_e4m3*>(cache.v));
  return go(qk_norm_rope_kernel<bf16>, static_cast<bf16*>(cache.k), static_cast<bf16*>(cache.v));
}

}  // namespace rmk
