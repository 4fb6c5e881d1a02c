// Attention of one new token per sequence over a paged cache.
#include "attend_row.cuh"
#include "kernels.h"

namespace rmk {
namespace {

constexpr int kRowWarps = 4;

template <int D, typename E>
__global__ void __launch_bounds__(kRowWarps * 32)
    attn_decode_row_kernel(const bf16* __restrict__ q, int64_t q_stride, const E* __restrict__ kc,
                           const E* __restrict__ vc, int64_t page_stride, int n_pages, int P,
                           const float* __restrict__ k_scale, const float* __restrict__ v_scale,
                           const int32_t* __restrict__ table, int table_stride,
                           const int32_t* __restrict__ length, int hq, int hkv, int window,
                           int sinks, bf16* __restrict__ out, int64_t out_stride,
                           float scale_log2) {
  __shared__ float qs[kRowWarps][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t s = blockIdx.x;
  const int h = blockIdx.y * kRowWarps + warp;
  if (h >= hq) return;
  const int kvh = h / (hq / hkv);
  const float ks = k_scale != nullptr ? k_scale[kvh] : 1.f, vs = v_scale != nullptr ? v_scale[kvh] : 1.f;
  for (int c = lane; c < D; c += 32)
    qs[warp][c] = to_f32(q[s * q_stride + h * D + c]) * (scale_log2 * ks);
  __syncwarp();
  int64_t len = length[s];
  if (len > static_cast<int64_t>(table_stride) * P) len = static_cast<int64_t>(table_stride) * P;
  const int64_t lo = window > 0 && len - window > 0 ? len - window : 0;
  const int64_t sink_end = lo < sinks ? lo : sinks;
  auto ptr = [&](int64_t j, const E*& kp, const E*& vp) {
    const int page = table[s * table_stride + j / P];
    if (page < 0 || page >= n_pages) return;
    const int64_t at = page * page_stride + (static_cast<int64_t>(kvh) * P + j % P) * D;
    kp = kc + at;
    vp = vc + at;
  };
  RowState<D> r;
  attend_keys<D, E>(qs[warp], 0, sink_end, ptr, r);
  attend_keys<D, E>(qs[warp], lo, len, ptr, r);
  const float inv = r.l == 0.f ? 0.f : vs / r.l;
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
    out[s * out_stride + h * D + lane + 32 * i] = __float2bfloat16_rn(r.o[i] * inv);
}

}  // namespace

size_t attn_decode_workspace(int, int, const rm_kv_cache&) { return 16; }

cudaError_t attn_decode_launch(const void* q, int64_t q_stride, const rm_kv_cache& c,
                               const int32_t* table, int table_stride, const int32_t* length,
                               int n, int hq, int window, int sinks, void* out, int64_t out_stride,
                               void* workspace, cudaStream_t st) {
  (void)workspace;
  const float scale_log2 = 1.4426950408889634f / sqrtf(static_cast<float>(c.head_dim));
  auto go = [&](auto* kernel, auto* kc, auto* vc) {
    kernel<<<dim3(n, (hq + kRowWarps - 1) / kRowWarps), kRowWarps * 32, 0, st>>>(
        static_cast<const bf16*>(q), q_stride, kc, vc, c.page_stride, c.n_pages, c.page_size,
        c.k_scale, c.v_scale, table, table_stride, length, hq, c.n_kv_heads, window, sinks,
        static_cast<bf16*>(out), out_stride, scale_log2);
    return cudaGetLastError();
  };
  using F8 = __nv_fp8_e4m3;
  if (c.dtype == RM_E4M3) {
    const F8 *k = static_cast<const F8*>(c.k), *v = static_cast<const F8*>(c.v);
    return c.head_dim == 64 ? go(attn_decode_row_kernel<64, F8>, k, v)
                            : go(attn_decode_row_kernel<128, F8>, k, v);
  }
  const bf16 *k = static_cast<const bf16*>(c.k), *v = static_cast<const bf16*>(c.v);
  return c.head_dim == 64 ? go(attn_decode_row_kernel<64, bf16>, k, v)
                          : go(attn_decode_row_kernel<128, bf16>, k, v);
}

}  // namespace rmk
