// C ABI of the incremental-scoring steps (include/rm_ops.h): validation and
// launch.  Their kernels are launched with programmatic stream serialization
// (launched while the kernel ahead of them drains) and wait for that kernel
// before they touch global memory; only the decode kernel lets its dependent,
// the join, be launched early.
#include <atomic>
#include <cmath>

#include "common.cuh"
#include "host.h"
#include "kernels.h"

namespace rmk {
namespace {

// The SM count of a device, looked up once (0: not yet).
cudaError_t device_sms(int dev, int* out) {
  static std::atomic<int> known[kMaxDevices];
  const bool keep = dev >= 0 && dev < kMaxDevices;
  *out = keep ? known[dev].load(std::memory_order_relaxed) : 0;
  if (*out != 0) return cudaSuccess;
  const cudaError_t e = cudaDeviceGetAttribute(out, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess && keep) known[dev].store(*out, std::memory_order_relaxed);
  return e;
}

// An output pointer is memory of the current device: a call made with another
// device current, or with host buffers, is refused rather than left to fault.
// (One pointer a call: looking all of slot maps' eleven up took 2 us of 8.)
int check_on_device(const void* out, int* num_sms = nullptr) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  cudaPointerAttributes at;
  if (e == cudaSuccess) e = cudaPointerGetAttributes(&at, out);
  if (e == cudaSuccess && num_sms != nullptr) e = device_sms(dev, num_sms);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return set_error(RM_E_DEVICE, "no usable CUDA device: %s", cudaGetErrorString(e));
  }
  if ((at.type != cudaMemoryTypeDevice && at.type != cudaMemoryTypeManaged) || at.device != dev)
    return set_error(RM_E_INVAL, "pointer %p is not memory of the current device %d", out, dev);
  return RM_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

bool row_stride_ok(int64_t stride, int64_t row) { return stride >= row && stride % 8 == 0; }

int check_cache(const rm_kv_cache& c, bool attention) {
  if (c.k == nullptr || c.v == nullptr) return set_error(RM_E_INVAL, "NULL cache pages");
  if (c.dtype != RM_BF16 && c.dtype != RM_E4M3)
    return set_error(RM_E_INVAL, "the cache holds bf16 or e4m3");
  if (c.n_pages < 1 || c.page_size < 1 || c.page_size > 1024 || c.n_kv_heads < 1 || c.n_kv_heads > 65536 ||
      c.head_dim < 8 || c.head_dim % 8 != 0 || c.head_dim > 256)
    return set_error(RM_E_INVAL, "bad cache sizes");
  if (attention && c.head_dim != 64 && c.head_dim != 128)
    return set_error(RM_E_INVAL, "attention takes head_dim 64 or 128");
  const int64_t item = c.dtype == RM_E4M3 ? 1 : 2;
  const int64_t page = static_cast<int64_t>(c.n_kv_heads) * c.page_size * c.head_dim;
  if (c.page_stride < page || c.page_stride > (INT64_MAX / 4) / c.n_pages ||
      (c.page_stride * item) % 16 != 0 || !aligned16(c.k) || !aligned16(c.v))
    return set_error(RM_E_INVAL, "bad page_stride, or pages not 16-byte aligned");
  if ((c.k_scale == nullptr) != (c.v_scale == nullptr))
    return set_error(RM_E_INVAL, "k_scale and v_scale go together");
  if (c.dtype == RM_BF16 && c.k_scale != nullptr)
    return set_error(RM_E_INVAL, "scales belong to an e4m3 cache");
  return RM_OK;
}

bool heads_ok(int32_t hq, int32_t hkv) { return hkv >= 1 && hq >= hkv && hq % hkv == 0 && hq <= 65536; }

}  // namespace
}  // namespace rmk

using namespace rmk;

#define RM_LAUNCH(call)                                                          \
  do {                                                                           \
    cudaError_t e_ = (call);                                                     \
    if (e_ != cudaSuccess)                                                       \
      return set_error(RM_E_CUDA, "%s: %s", #call, cudaGetErrorString(e_));      \
  } while (0)
#define RM_CHECK(call)            \
  do {                            \
    const int r_ = (call);        \
    if (r_ != RM_OK) return r_;   \
  } while (0)

extern "C" {

int rm_rope_freqs(int32_t rot_dim, double base, int32_t scaling, double factor, double trained,
                  double fast, double slow, double* freqs) {
  if (freqs == nullptr || rot_dim < 2 || rot_dim % 2 != 0 || rot_dim > 256 || !(base > 1.0) ||
      !std::isfinite(base))
    return set_error(RM_E_INVAL, "bad rot_dim, base or NULL freqs");
  if (scaling < RM_ROPE_PLAIN || scaling > RM_ROPE_PARTS)
    return set_error(RM_E_INVAL, "unknown scaling %d", scaling);
  if (scaling != RM_ROPE_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor)))
    return set_error(RM_E_INVAL, "factor must be at least 1");
  if (scaling == RM_ROPE_BASE) {
    if (rot_dim < 4) return set_error(RM_E_INVAL, "RM_ROPE_BASE needs rot_dim > 2");
    base *= std::pow(factor, rot_dim / (rot_dim - 2.0));
    if (!std::isfinite(base)) return set_error(RM_E_INVAL, "factor too large");
  }
  if (scaling == RM_ROPE_PARTS &&
      (!(trained >= 1.0) || !std::isfinite(trained) || !(slow > 0.0) || !(fast > slow) ||
       !std::isfinite(fast)))
    return set_error(RM_E_INVAL, "RM_ROPE_PARTS needs trained >= 1 and fast > slow > 0");
  const double two_pi = 6.283185307179586476925;
  for (int32_t i = 0; i < rot_dim / 2; ++i) {
    double f = std::pow(base, -2.0 * i / rot_dim);
    if (scaling == RM_ROPE_LINEAR) f /= factor;
    if (scaling == RM_ROPE_PARTS) {
      const double turns = trained * f / two_pi;
      const double keep = std::fmin(1.0, std::fmax(0.0, (turns - slow) / (fast - slow)));
      f = f * keep + f / factor * (1.0 - keep);
    }
    freqs[i] = f;
  }
  return RM_OK;
}

int rm_op_kv_slots(const int32_t* len_before, const int32_t* n_new, int32_t n_seqs,
                   int32_t page_size, const int32_t* free_pages, int32_t n_free,
                   const int32_t* used_before, int32_t* block_table, int32_t table_stride,
                   int32_t T, int32_t* offsets, int32_t* positions, int64_t* slots,
                   int32_t* len_after, int32_t* used_after, int32_t* unserved, void* stream) {
  if (len_before == nullptr || n_new == nullptr || used_before == nullptr || block_table == nullptr ||
      offsets == nullptr || len_after == nullptr || used_after == nullptr || unserved == nullptr ||
      (n_free > 0 && free_pages == nullptr) ||
      (T > 0 && (positions == nullptr || slots == nullptr)))
    return set_error(RM_E_INVAL, "NULL argument");
  if (n_seqs < 1 || page_size < 1 || page_size > 1024 || n_free < 0 || table_stride < 1 || T < 0)
    return set_error(RM_E_INVAL, "bad sizes");
  if (n_seqs > 16384) return set_error(RM_E_RANGE, "at most 16384 sequences a call");
  RM_CHECK(check_on_device(offsets));
  RM_LAUNCH(kv_slots_launch(len_before, n_new, n_seqs, page_size, free_pages, n_free, used_before,
                            block_table, table_stride, T, offsets, positions, slots, len_after,
                            used_after, unserved, static_cast<cudaStream_t>(stream)));
  return RM_OK;
}

int rm_op_qk_norm_rope(const void* qkv, int64_t qkv_stride, void* q_out, int64_t q_stride,
                       void* k_out, int64_t k_stride, int32_t T, int32_t n_q_heads,
                       int32_t n_kv_heads, int32_t head_dim, const float* q_gain,
                       const float* k_gain, float eps, const rm_rope* rope,
                       const int32_t* positions, const rm_kv_cache* cache, const int64_t* slots,
                       void* stream) {
  if (T > 0 && (qkv == nullptr || q_out == nullptr)) return set_error(RM_E_INVAL, "NULL argument");
  if (T < 0 || !heads_ok(n_q_heads, n_kv_heads) || head_dim < 8 || head_dim % 8 != 0 || head_dim > 256)
    return set_error(RM_E_INVAL, "bad sizes");
  const int64_t d = head_dim;
  if (!row_stride_ok(qkv_stride, (n_q_heads + 2 * static_cast<int64_t>(n_kv_heads)) * d) ||
      !row_stride_ok(q_stride, n_q_heads * d) ||
      (k_out != nullptr && !row_stride_ok(k_stride, n_kv_heads * d)))
    return set_error(RM_E_INVAL, "row strides must cover a row and be multiples of 8 elements");
  if (!aligned16(qkv) || !aligned16(q_out) || !aligned16(k_out))
    return set_error(RM_E_INVAL, "qkv, q_out and k_out must be 16-byte aligned");
  if ((q_gain == nullptr) != (k_gain == nullptr))
    return set_error(RM_E_INVAL, "q_gain and k_gain go together");
  if (((reinterpret_cast<uintptr_t>(q_gain) | reinterpret_cast<uintptr_t>(k_gain)) & 3) != 0)
    return set_error(RM_E_INVAL, "q_gain and k_gain must be 4-byte aligned");
  if (q_gain != nullptr && !(eps >= 0.f)) return set_error(RM_E_INVAL, "eps must be >= 0");
  rm_rope r = {};
  if (rope != nullptr) {
    r = *rope;
    if (r.rot_dim < 0 || r.rot_dim % 2 != 0 || r.rot_dim > head_dim ||
        (r.layout != RM_ROPE_HALF && r.layout != RM_ROPE_INTERLEAVED))
      return set_error(RM_E_INVAL, "bad rotation");
    if (r.rot_dim > 0 && (r.freqs == nullptr || (T > 0 && positions == nullptr)))
      return set_error(RM_E_INVAL, "a rotation needs freqs and positions");
  }
  rm_kv_cache c = {};
  if (cache != nullptr) {
    RM_CHECK(check_cache(*cache, false));
    c = *cache;
    if (T > 0 && slots == nullptr) return set_error(RM_E_INVAL, "a cache write needs slots");
    if (c.n_kv_heads != n_kv_heads || c.head_dim != head_dim)
      return set_error(RM_E_INVAL, "the cache has other heads");
  }
  if (T == 0) return RM_OK;
  int sms = 0;
  RM_CHECK(check_on_device(q_out, &sms));
  RM_LAUNCH(qk_norm_rope_launch(qkv, qkv_stride, q_out, q_stride, k_out, k_stride, T, n_q_heads,
                                n_kv_heads, head_dim, q_gain, k_gain, eps, r, positions, c, slots,
                                sms, static_cast<cudaStream_t>(stream)));
  return RM_OK;
}

int rm_op_attn_window(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                      const void* v, int64_t v_stride, const int32_t* offsets, int32_t n_seqs,
                      int32_t T, int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim,
                      int32_t window, int32_t sinks, void* out, int64_t out_stride, void* stream) {
  if (offsets == nullptr || (T > 0 && (q == nullptr || k == nullptr || v == nullptr || out == nullptr)))
    return set_error(RM_E_INVAL, "NULL argument");
  if (n_seqs < 1 || T < 0 || !heads_ok(n_q_heads, n_kv_heads) || n_q_heads / n_kv_heads > 128 ||
      (head_dim != 64 && head_dim != 128) || window < 0 || sinks < 0)
    return set_error(RM_E_INVAL, "bad sizes (head_dim must be 64 or 128)");
  const int64_t rq = static_cast<int64_t>(n_q_heads) * head_dim;
  const int64_t rk = static_cast<int64_t>(n_kv_heads) * head_dim;
  if (!row_stride_ok(q_stride, rq) || !row_stride_ok(out_stride, rq) ||
      !row_stride_ok(k_stride, rk) || !row_stride_ok(v_stride, rk))
    return set_error(RM_E_INVAL, "row strides must cover a row and be multiples of 8 elements");
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out))
    return set_error(RM_E_INVAL, "q, k, v and out must be 16-byte aligned");
  if (T == 0) return RM_OK;
  RM_CHECK(check_on_device(out));
  RM_LAUNCH(attn_window_launch(q, q_stride, k, k_stride, v, v_stride, offsets, n_seqs, T, n_q_heads,
                               n_kv_heads, head_dim, window, sinks, out, out_stride,
                               static_cast<cudaStream_t>(stream)));
  return RM_OK;
}

size_t rm_attn_decode_workspace(int32_t n_seqs, int32_t n_q_heads, const rm_kv_cache* cache) {
  if (cache == nullptr || n_seqs < 1 || check_cache(*cache, true) != RM_OK ||
      !heads_ok(n_q_heads, cache->n_kv_heads))
    return 0;
  return attn_decode_workspace(n_seqs, n_q_heads, *cache);
}

int rm_op_attn_decode(const void* q, int64_t q_stride, const rm_kv_cache* cache,
                      const int32_t* block_table, int32_t table_stride, const int32_t* length,
                      int32_t n_seqs, int32_t n_q_heads, int32_t window, int32_t sinks, void* out,
                      int64_t out_stride, void* workspace, size_t workspace_bytes, void* stream) {
  if (q == nullptr || cache == nullptr || block_table == nullptr || length == nullptr ||
      out == nullptr || workspace == nullptr)
    return set_error(RM_E_INVAL, "NULL argument");
  RM_CHECK(check_cache(*cache, true));
  if (n_seqs < 1 || table_stride < 1 || !heads_ok(n_q_heads, cache->n_kv_heads) || window < 0 || sinks < 0)
    return set_error(RM_E_INVAL, "bad sizes");
  const int64_t rq = static_cast<int64_t>(n_q_heads) * cache->head_dim;
  if (!row_stride_ok(q_stride, rq) || !row_stride_ok(out_stride, rq))
    return set_error(RM_E_INVAL, "row strides must cover a row and be multiples of 8 elements");
  if (!aligned16(q) || !aligned16(out) || !aligned16(workspace))
    return set_error(RM_E_INVAL, "q, out and workspace must be 16-byte aligned");
  if (workspace_bytes < attn_decode_workspace(n_seqs, n_q_heads, *cache))
    return set_error(RM_E_RANGE, "workspace too small (rm_attn_decode_workspace)");
  int sms = 0;
  RM_CHECK(check_on_device(out, &sms));
  RM_LAUNCH(attn_decode_launch(q, q_stride, *cache, block_table, table_stride, length, n_seqs,
                               n_q_heads, window, sinks, out, out_stride, workspace, sms,
                               static_cast<cudaStream_t>(stream)));
  return RM_OK;
}

}  // extern "C"
