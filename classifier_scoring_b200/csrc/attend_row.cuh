// One query row of an attention in plain fp32, by one warp: a form that is
// right for any values, since it touches the keys that the row sees and no
// others.
#pragma once

#include <cfloat>

#include "common.cuh"

namespace rmk {

// Running state of a row: o[i] of lane x belongs to dim x + 32 i.
template <int D> struct RowState {
  float m = -INFINITY, l = 0.f;
  float o[D / 32] = {};
};

// Adds keys [j0, j1) to the row with query q; scale makes the scores base-2
// logarithms; ptr(j, k, v) sets the key's and value's rows.
template <int D, typename Ptr>
__device__ __forceinline__ void attend_keys(const bf16* q, float scale, int64_t j0, int64_t j1,
                                            Ptr ptr, RowState<D>& r) {
  const int lane = threadIdx.x & 31;
  for (int64_t jb = j0; jb < j1; jb += 32) {
    const bf16 *kp = nullptr, *vp = nullptr;
    if (jb + lane < j1) ptr(jb + lane, kp, vp);
    float s = -INFINITY;
    if (kp != nullptr) {
      s = 0.f;
#pragma unroll 4
      for (int c = 0; c < D / 8; ++c) {
        float f[8], x[8];
        Chunk8<bf16>::load(kp + 8 * c, f);
        Chunk8<bf16>::load(q + 8 * c, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) s = fmaf(x[e], f[e], s);
      }
      s *= scale;
    }
    const uint32_t seen = __ballot_sync(0xffffffffu, kp != nullptr);
    if (seen == 0) continue;
    // (scores of -inf alone: any finite reference makes their weights 0)
    const float mn = fmaxf(fmaxf(r.m, group_max<32>(s)), -FLT_MAX);
    const float keep = r.l == 0.f ? 0.f : exp2f(r.m - mn);
    const float p = kp != nullptr ? exp2f(s - mn) : 0.f;
    r.m = mn;
    r.l = r.l * keep + group_sum<32>(p);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) r.o[i] *= keep;
    for (uint32_t left = seen; left != 0; left &= left - 1) {
      const int src = __ffs(left) - 1;
      const float pj = __shfl_sync(0xffffffffu, p, src);
      const bf16* vj = reinterpret_cast<const bf16*>(
          __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(vp), src));
#pragma unroll
      for (int i = 0; i < D / 32; ++i) r.o[i] = fmaf(pj, to_f32(vj[lane + 32 * i]), r.o[i]);
    }
  }
}

}  // namespace rmk
