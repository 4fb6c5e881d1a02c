// One query row of the cached attention in plain fp32, by one warp: the form
// that is right for any values, whatever lies in the keys it does not see.
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"

namespace rmk {

// Eight consecutive elements of a cache row as fp32.
__device__ __forceinline__ void load_kv8(const bf16* p, float* f) { Chunk8<bf16>::load(p, f); }
__device__ __forceinline__ void load_kv8(const __nv_fp8_e4m3* p, float* f) {
  const uint2 v = *reinterpret_cast<const uint2*>(p);
  const uint32_t w[2] = {v.x, v.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
        static_cast<__nv_fp8x2_storage_t>((w[i >> 1] >> ((i & 1) * 16)) & 0xffffu), __NV_E4M3);
    const float2 x = __half22float2(__half2(h));
    f[2 * i] = x.x;
    f[2 * i + 1] = x.y;
  }
}

// Running state of a row: o[i] of lane x belongs to dim x + 32 i.
template <int D> struct RowState {
  float m = -INFINITY, l = 0.f;
  float o[D / 32] = {};
};

// Adds keys [j0, j1) to the row.  qs: the query in shared memory, scaled so
// that the scores are base-2 logarithms; ptr(j, k, v) sets the key's and
// value's rows, or leaves them null for a key that is not seen.
template <int D, typename E, typename Ptr>
__device__ __forceinline__ void attend_keys(const float* qs, int64_t j0, int64_t j1, Ptr ptr,
                                            RowState<D>& r) {
  const int lane = threadIdx.x & 31;
  for (int64_t jb = j0; jb < j1; jb += 32) {
    const E *kp = nullptr, *vp = nullptr;
    if (jb + lane < j1) ptr(jb + lane, kp, vp);
    float s = -INFINITY;
    if (kp != nullptr) {
      s = 0.f;
#pragma unroll 4
      for (int c = 0; c < D / 8; ++c) {
        float f[8];
        load_kv8(kp + 8 * c, f);
#pragma unroll
        for (int e = 0; e < 8; ++e) s = fmaf(qs[8 * c + e], f[e], s);
      }
    }
    const uint32_t seen = __ballot_sync(0xffffffffu, kp != nullptr);
    if (seen == 0) continue;
    const float mn = fmaxf(r.m, group_max<32>(s));
    const float keep = r.l == 0.f ? 0.f : exp2f(r.m - mn);
    const float p = kp != nullptr ? exp2f(s - mn) : 0.f;
    r.m = mn;
    r.l = r.l * keep + group_sum<32>(p);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) r.o[i] *= keep;
    for (uint32_t left = seen; left != 0; left &= left - 1) {
      const int src = __ffs(left) - 1;
      const float pj = __shfl_sync(0xffffffffu, p, src);
      const E* vj = reinterpret_cast<const E*>(
          __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(vp), src));
#pragma unroll
      for (int i = 0; i < D / 32; ++i) r.o[i] = fmaf(pj, static_cast<float>(vj[lane + 32 * i]), r.o[i]);
    }
  }
}

}  // namespace rmk
