// Causal attention of packed sequences with a sliding window and sinks.
#include "attend_row.cuh"
#include "kernels.h"

namespace rmk {
namespace {

constexpr int kRowWarps = 4;

template <int D>
__global__ void __launch_bounds__(kRowWarps * 32)
    attn_window_row_kernel(const bf16* __restrict__ q, int64_t q_stride, const bf16* __restrict__ k,
                           int64_t k_stride, const bf16* __restrict__ v, int64_t v_stride,
                           const int32_t* __restrict__ offsets, int n, int hq, int hkv, int window,
                           int sinks, bf16* __restrict__ out, int64_t out_stride,
                           float scale_log2) {
  __shared__ float qs[kRowWarps][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t t = blockIdx.x;
  const int h = blockIdx.y * kRowWarps + warp;
  if (h >= hq || t >= offsets[n]) return;
  const int start = offsets[upper_index(offsets, n, t)];
  for (int c = lane; c < D; c += 32) qs[warp][c] = to_f32(q[t * q_stride + h * D + c]) * scale_log2;
  __syncwarp();
  const int kvh = h / (hq / hkv);
  const int64_t lo = window > 0 && t - window + 1 > start ? t - window + 1 : start;
  const int64_t sink_end = lo - start < sinks ? lo : start + static_cast<int64_t>(sinks);
  auto ptr = [&](int64_t j, const bf16*& kp, const bf16*& vp) {
    kp = k + j * k_stride + kvh * D;
    vp = v + j * v_stride + kvh * D;
  };
  RowState<D> r;
  attend_keys<D, bf16>(qs[warp], start, sink_end, ptr, r);
  attend_keys<D, bf16>(qs[warp], lo, t + 1, ptr, r);
  const float inv = 1.f / r.l;
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
    out[t * out_stride + h * D + lane + 32 * i] = __float2bfloat16_rn(r.o[i] * inv);
}

}  // namespace

cudaError_t attn_window_launch(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                               const void* v, int64_t v_stride, const int32_t* offsets, int n,
                               int T, int hq, int hkv, int d, int window, int sinks, void* out,
                               int64_t out_stride, cudaStream_t st) {
  if (T < 1) return cudaSuccess;
  const float scale_log2 = 1.4426950408889634f / sqrtf(static_cast<float>(d));
  auto go = [&](auto* kernel) {
    kernel<<<dim3(T, (hq + kRowWarps - 1) / kRowWarps), kRowWarps * 32, 0, st>>>(
        static_cast<const bf16*>(q), q_stride, static_cast<const bf16*>(k), k_stride,
        static_cast<const bf16*>(v), v_stride, offsets, n, hq, hkv, window, sinks,
        static_cast<bf16*>(out), out_stride, scale_log2);
    return cudaGetLastError();
  };
  return d == 64 ? go(attn_window_row_kernel<64>) : go(attn_window_row_kernel<128>);
}

}  // namespace rmk
