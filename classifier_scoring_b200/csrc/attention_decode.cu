// Attention of one new token per sequence over a paged cache.
//
// A step reads every visible key and value once (2 * len * d elements for a
// key-value head) and computes 4 * d operations per query head and key: it is
// bound by memory, and by latency when the batch is small.  The kernel
// therefore spreads the bytes evenly and keeps many of them in flight:
//  - the (sequence, kv head) units' key tiles, laid end to end, are cut into
//    one equal stretch per CTA whatever the lengths are, so a long context
//    beside short ones does not leave SMs idle and no length needs to be known
//    on the host.  A unit that a cut divides leaves its parts (running maximum,
//    sum, unnormalised output) in the workspace; a second kernel joins them in
//    stretch order.
//  - each warp of a CTA takes its own keys of every tile through a private
//    ring of cp.async stages, with no barrier between warps until a unit ends;
//    the ring runs across unit borders.
//  - the query heads that share a kv head are the rows of one mma.sync tile
//    (m16n8k16), so a key is read once for all of them.
#include <cuda_fp8.h>

#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace rmk {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kRows = 16;                       // query heads per unit (rows of an MMA tile)
constexpr int kCtasPerSm = 2;
constexpr int kMaxCtas = 148 * kCtasPerSm;      // the workspace has parts for this many

// Keys per warp and step, and ring depth: a stage holds 8 KB of keys and
// values (4 KB for 8-bit heads of 64), and two CTAs fit an SM.
template <int D, typename E> struct Shape {
  static constexpr int kKeys = D * sizeof(E) >= 256 ? 16 : 32;
  static constexpr int kTile = kWarps * kKeys;
  static constexpr int kRowBytes = D * sizeof(E);
  static constexpr int kHalf = kKeys * kRowBytes;       // the keys of a stage; its values follow
  static constexpr int kStages = 2 * kHalf >= 8192 ? 3 : 6;
  static constexpr int kRing = kWarps * kStages * 2 * kHalf;
  static constexpr int kSum = kRing;                    // float [kRows][D]
  static constexpr int kMl = kSum + kRows * D * 4;      // float [kWarps][kRows][2]
  static constexpr int kSmem = kMl + kWarps * kRows * 2 * 4;
};

struct Parts {            // workspace
  float* o;               // [ctas][2][kRows][D]
  float* ml;              // [ctas][2][kRows][2]
  int4* rec;              // [ctas]: unit that begins in the CTA's stretch and goes on behind it
};

struct DecodeArgs {
  const bf16* q;
  int64_t q_stride;
  const void* kc;
  const void* vc;
  int64_t page_stride;
  int n_pages, P;
  uint32_t div;                 // x / P = x * div >> shift for 0 <= x < 2^31
  int shift;
  const float* k_scale;
  const float* v_scale;
  const int32_t* table;
  int table_stride;
  const int32_t* length;
  int n, hq, hkv, window, sinks;
  bf16* out;
  int64_t out_stride;
  float scale_log2;
  int units;                    // per sequence: hkv * ceil(group / kRows)
  Parts parts;
};

// What a sequence's newest token sees: keys [0, nsink) and then, from the
// nsink-th on, keys j + skip; vis of them in tiles of `tile`, at least one
// (an empty sequence's row of zeros is written by somebody too).
struct Seen {
  int vis, nsink, skip, nt;
};
__device__ __forceinline__ Seen seen_of(const DecodeArgs& a, int s, int tile) {
  const int64_t cap = static_cast<int64_t>(a.table_stride) * a.P;
  int len = max(0, a.length[s]);
  if (len > cap) len = static_cast<int>(cap);
  const int lo = a.window > 0 && len > a.window ? len - a.window : 0;
  Seen r;
  r.nsink = min(lo, a.sinks);
  r.skip = lo - r.nsink;
  r.vis = len - r.skip;
  r.nt = max(1u, (static_cast<unsigned>(r.vis) + tile - 1) / tile);
  return r;
}

// Position in the laid-out tiles: sequence, unit of it, key tile of that.
struct Cursor {
  int s, u, t;
  Seen seen;
  __device__ __forceinline__ void next(const DecodeArgs& a, int tile) {
    if (++t < seen.nt) return;
    t = 0;
    if (++u < a.units) return;
    u = 0;
    if (++s < a.n) seen = seen_of(a, s, tile);
  }
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
// D += A B, fp32 accumulators; operands bf16 (bf16 caches) or fp16 (8-bit
// caches: every e4m3 value is an fp16 value)
template <typename E>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (sizeof(E) == 2)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// two e4m3 bytes (low half of x) as two fp16
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t x) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(x & 0xffffu), __NV_E4M3);
  return static_cast<uint32_t>(h.x) | (static_cast<uint32_t>(h.y) << 16);
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// Byte offset of 16-byte chunk c of row r in a stage: chunks of the eight
// rows that one ldmatrix reads lie in eight different bank groups.
template <int RowBytes> __device__ __forceinline__ int chunk_at(int r, int c) {
  return RowBytes >= 128 ? r * RowBytes + ((c ^ (r & 7)) << 4) : r * RowBytes + ((c ^ ((r >> 1) & 3)) << 4);
}

template <int D, typename E>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) attn_decode_kernel(const DecodeArgs a) {
  using SH = Shape<D, E>;
  constexpr bool kF8 = sizeof(E) == 1;
  constexpr int kKeys = SH::kKeys, kStages = SH::kStages;
  extern __shared__ __align__(1024) uint8_t sm[];
  __shared__ long long scan[kWarps];
  __shared__ int start_s;
  __shared__ long long start_rem;
  __shared__ uint32_t masks[kWarps][kStages];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // this CTA's stretch [t0, t1) of all tiles, and where it begins
  const int per = (a.n + kThreads - 1) / kThreads;
  const int i0 = min(a.n, tid * per), i1 = min(a.n, i0 + per);
  long long mine = 0;
  for (int i = i0; i < i1; ++i) mine += static_cast<long long>(seen_of(a, i, SH::kTile).nt) * a.units;
  long long upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += x;
  }
  if (lane == 31) scan[warp] = upto;
  __syncthreads();
  long long total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) upto += scan[w];
    total += scan[w];
  }
  const int c = blockIdx.x;
  const long long ctas = min(static_cast<long long>(gridDim.x), total);   // no empty stretch among these
  if (c >= ctas) {
    if (tid == 0) a.parts.rec[c] = make_int4(-1, 0, 0, 0);
    return;
  }
  const long long t0 = c * total / ctas, t1 = (c + 1) * total / ctas;
  if (t0 >= upto - mine && t0 < upto) {
    long long rem = t0 - (upto - mine);
    int i = i0;
    for (;; ++i) {
      const long long k = static_cast<long long>(seen_of(a, i, SH::kTile).nt) * a.units;
      if (rem < k) break;
      rem -= k;
    }
    start_s = i;
    start_rem = rem;
  }
  __syncthreads();
  Cursor use;
  use.s = start_s;
  use.seen = seen_of(a, use.s, SH::kTile);
  use.u = static_cast<int>(start_rem / use.seen.nt);
  use.t = static_cast<int>(start_rem % use.seen.nt);
  Cursor get = use;
  const int steps = static_cast<int>(t1 - t0);
  const int group = a.hq / a.hkv, mtiles = a.units / a.hkv;

  uint8_t* ring = sm + warp * kStages * 2 * SH::kHalf;
  const uint32_t ring_u = static_cast<uint32_t>(__cvta_generic_to_shared(ring));
  float* sum = reinterpret_cast<float*>(sm + SH::kSum);
  float* ml = reinterpret_cast<float*>(sm + SH::kMl);

  // The page of a lane's key is looked up one step before its rows are
  // fetched.
  int pg = -1;
  int64_t row_in_page = 0;
  auto lookup = [&](bool more) {
    pg = -1;
    if (!more) return;
    const unsigned j = static_cast<unsigned>(get.t) * SH::kTile + warp * kKeys + lane;
    if (lane < kKeys && j < static_cast<unsigned>(get.seen.vis)) {
      const int key = static_cast<int>(j) + (j < static_cast<unsigned>(get.seen.nsink) ? 0 : get.seen.skip);
      const int b = static_cast<int>((static_cast<unsigned long long>(key) * a.div) >> a.shift);
      row_in_page = static_cast<int64_t>(get.u / mtiles) * a.P + (key - b * a.P);
      pg = a.table[static_cast<int64_t>(get.s) * a.table_stride + b];
    }
    get.next(a, SH::kTile);
  };
  auto fetch = [&](int stage) {
    const bool ok = pg >= 0 && pg < a.n_pages;
    const int64_t at = ok ? pg * a.page_stride + row_in_page * D : 0;
    const uint32_t mask = __ballot_sync(0xffffffffu, ok);
    if (lane == 0) masks[warp][stage] = mask;
    const uint32_t dst = ring_u + stage * 2 * SH::kHalf;
    constexpr int kChunks = SH::kRowBytes / 16;
    const char* kb = static_cast<const char*>(a.kc);
    const char* vb = static_cast<const char*>(a.vc);
#pragma unroll
    for (int i = 0; i < kKeys * kChunks / 32; ++i) {
      const int r = (i * 32 + lane) / kChunks, ch = (i * 32 + lane) % kChunks;
      const int64_t off = __shfl_sync(0xffffffffu, at, r) * static_cast<int64_t>(sizeof(E)) + ch * 16;
      const int bytes = (mask >> r) & 1 ? 16 : 0;               // 0: the row is filled with zeros
      const uint32_t d = dst + chunk_at<SH::kRowBytes>(r, ch);
      cp16(d, kb + off, bytes);
      cp16(d + SH::kHalf, vb + off, bytes);
    }
  };

  uint32_t qf[D / 16][4];
  float sc[2], o[D / 8][4], m[2], l[2];
  auto begin_unit = [&]() {
    const int h = use.u / mtiles, r0 = (use.u % mtiles) * kRows;
    const int rows = min(kRows, group - r0);
    const bf16* q = a.q + use.s * a.q_stride + static_cast<int64_t>(h * group + r0) * D;
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int r = g + (x & 1) * 8;
        // 8-bit keys arrive four dims to a lane: dims 4t..4t+3 of a step are
        // the MMA's k = 2t, 2t+1, 2t+8, 2t+9, for the query as for the keys
        const int dim = ks * 16 + (kF8 ? 4 * t + (x >> 1) * 2 : 2 * t + (x >> 1) * 8);
        qf[ks][x] = r < rows ? *reinterpret_cast<const uint32_t*>(q + r * D + dim) : 0u;
      }
    const float ks = a.scale_log2 * (kF8 && a.k_scale != nullptr ? a.k_scale[h] : 1.f);
    sc[0] = sc[1] = ks;
    if (kF8) {
      // bf16 queries as fp16, times the power of two that brings the row's
      // largest to [2^13, 2^14): exact but for entries 2^-27 below it
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float top = 0.f;
#pragma unroll
        for (int k2 = 0; k2 < D / 16; ++k2)
          top = fmaxf(top, fmaxf(fmaxf(fabsf(bf16_lo(qf[k2][x])), fabsf(bf16_hi(qf[k2][x]))),
                                 fmaxf(fabsf(bf16_lo(qf[k2][x + 2])), fabsf(bf16_hi(qf[k2][x + 2])))));
        top = group_max<4>(top);
        const int e = top > 0.f && top < INFINITY ? 13 - ilogbf(top) : 0;
        sc[x] = ldexpf(ks, -e);
#pragma unroll
        for (int k2 = 0; k2 < D / 16; ++k2) {
          qf[k2][x] = pack_f16x2(ldexpf(bf16_lo(qf[k2][x]), e), ldexpf(bf16_hi(qf[k2][x]), e));
          qf[k2][x + 2] = pack_f16x2(ldexpf(bf16_lo(qf[k2][x + 2]), e), ldexpf(bf16_hi(qf[k2][x + 2]), e));
        }
      }
    }
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.f;
#pragma unroll
    for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
  };

  auto step = [&](int stage) {
    const uint32_t kb = ring_u + stage * 2 * SH::kHalf, vb = kb + SH::kHalf;
    const uint32_t mask = masks[warp][stage];
    float s[kKeys / 8][4];
#pragma unroll
    for (int i = 0; i < kKeys / 8; ++i) s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
    const int lr = lane & 7, lm = lane >> 3;
#pragma unroll
    for (int nt = 0; nt < kKeys / 8; ++nt) {
      if (kF8) {
#pragma unroll
        for (int k4 = 0; k4 < D / 64; ++k4) {                    // four 16-dim steps a load
          uint32_t b[4];
          ldsm4(kb + chunk_at<SH::kRowBytes>(nt * 8 + lr, k4 * 4 + lm), b);
#pragma unroll
          for (int x = 0; x < 4; ++x)
            mma<E>(s[nt], qf[k4 * 4 + x], e4m3x2_f16x2(b[x]), e4m3x2_f16x2(b[x] >> 16));
        }
      } else {
#pragma unroll
        for (int k2 = 0; k2 < D / 32; ++k2) {                    // two 16-dim steps a load
          uint32_t b[4];
          ldsm4(kb + chunk_at<SH::kRowBytes>(nt * 8 + lr, k2 * 4 + lm), b);
          mma<E>(s[nt], qf[k2 * 2], b[0], b[1]);
          mma<E>(s[nt], qf[k2 * 2 + 1], b[2], b[3]);
        }
      }
    }
    // base-2 scores of the lane's rows lane/4 and lane/4 + 8, keys 8 nt + 2t + {0, 1}
    const int t2 = (lane & 3) * 2;
    float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int nt = 0; nt < kKeys / 8; ++nt)
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const bool in = (mask >> (nt * 8 + t2 + (x & 1))) & 1;
        s[nt][x] = in ? s[nt][x] * sc[x >> 1] : -INFINITY;
        top[x >> 1] = fmaxf(top[x >> 1], s[nt][x]);
      }
    top[0] = group_max<4>(top[0]);
    top[1] = group_max<4>(top[1]);
    // The reference the exponentials are taken against follows the maximum
    // only when it falls 2^8 behind: a rescale of the output is then rare, and
    // P stays below 2^8 with the same relative rounding.
    if (__any_sync(0xffffffffu, top[0] > m[0] + 8.f || top[1] > m[1] + 8.f)) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const float mn = fmaxf(m[x], top[x]);
        const float keep = m[x] == -INFINITY ? 0.f : ex2_approx_ftz(m[x] - mn);
        m[x] = mn;
        l[x] *= keep;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          o[i][2 * x] *= keep;
          o[i][2 * x + 1] *= keep;
        }
      }
    }
    const float ref[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
#pragma unroll
    for (int nt = 0; nt < kKeys / 8; ++nt)
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const bool in = (mask >> (nt * 8 + t2 + (x & 1))) & 1;
        s[nt][x] = in ? ex2_approx_ftz(s[nt][x] - ref[x >> 1]) : 0.f;
        l[x >> 1] += s[nt][x];
      }
#pragma unroll
    for (int k16 = 0; k16 < kKeys / 16; ++k16) {
      uint32_t p[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const float lo = s[2 * k16 + (x >> 1)][(x & 1) * 2], hi = s[2 * k16 + (x >> 1)][(x & 1) * 2 + 1];
        p[x] = kF8 ? pack_f16x2(lo, hi) : pack_bf16x2(lo, hi);
      }
      // matrices 0, 1: keys 0..7, 8..15 of the first 16-byte chunk; 2, 3: of the next
      const int vr = k16 * 16 + (lm & 1) * 8 + lr;
#pragma unroll
      for (int c2 = 0; c2 < SH::kRowBytes / 32; ++c2) {
        uint32_t b[4];
        ldsm4t(vb + chunk_at<SH::kRowBytes>(vr, c2 * 2 + (lm >> 1)), b);
        if (kF8) {
          // a register holds dims 2c, 2c+1 of two keys: even dims make one
          // 8-dim tile, odd dims the next
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const uint32_t b0 = __byte_perm(b[2 * y], 0, 0x3120), b1 = __byte_perm(b[2 * y + 1], 0, 0x3120);
            mma<E>(o[c2 * 4 + y * 2], p, e4m3x2_f16x2(b0), e4m3x2_f16x2(b1));
            mma<E>(o[c2 * 4 + y * 2 + 1], p, e4m3x2_f16x2(b0 >> 16), e4m3x2_f16x2(b1 >> 16));
          }
        } else {
          mma<E>(o[c2 * 2], p, b[0], b[1]);
          mma<E>(o[c2 * 2 + 1], p, b[2], b[3]);
        }
      }
    }
  };

  // Joins the warps' states of a finished unit, in warp order, and writes the
  // output rows, or the unit's part when the stretch holds only part of it.
  auto end_unit = [&](long long unit0) {
    const int h = use.u / mtiles, r0 = (use.u % mtiles) * kRows;
    const int rows = min(kRows, group - r0);
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      l[x] = group_sum<4>(l[x]);
      if (t == 0) {
        ml[(warp * kRows + g + 8 * x) * 2] = m[x];
        ml[(warp * kRows + g + 8 * x) * 2 + 1] = l[x];
      }
    }
    __syncthreads();
    float w[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      float mt = -INFINITY;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) mt = fmaxf(mt, ml[(i * kRows + g + 8 * x) * 2]);
      w[x] = m[x] == -INFINITY ? 0.f : ex2_approx_ftz(m[x] - mt);
      if (l[x] != l[x]) w[x] = l[x];                       // a NaN seen before any maximum
    }
    for (int i = 0; i < kWarps; ++i) {
      if (warp == i) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          if (g + 8 * x >= rows) continue;
          float* dst = sum + (g + 8 * x) * D;
#pragma unroll
          for (int n8 = 0; n8 < D / 8; ++n8)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int dim = kF8 ? (n8 >> 1) * 16 + 4 * t + 2 * e + (n8 & 1) : n8 * 8 + 2 * t + e;
              const float v = o[n8][2 * x + e] * w[x];
              dst[dim] = i == 0 ? v : dst[dim] + v;
            }
        }
      }
      __syncthreads();
    }
    const bool whole = unit0 >= t0 && unit0 + use.seen.nt <= t1;
    const int slot = unit0 <= t0 ? 0 : 1;
    float* po = a.parts.o + static_cast<size_t>(c * 2 + slot) * kRows * D;
    float* pm = a.parts.ml + static_cast<size_t>(c * 2 + slot) * kRows * 2;
    const float vs = kF8 && a.v_scale != nullptr ? a.v_scale[h] : 1.f;
    for (int i = tid; i < rows * (D / 2); i += kThreads) {
      const int r = i / (D / 2), d2 = (i % (D / 2)) * 2;
      float mt = -INFINITY, lt = 0.f;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) mt = fmaxf(mt, ml[(k * kRows + r) * 2]);
#pragma unroll
      for (int k = 0; k < kWarps; ++k) {
        const float mk = ml[(k * kRows + r) * 2], lk = ml[(k * kRows + r) * 2 + 1];
        lt += mk == -INFINITY ? lk : lk * ex2_approx_ftz(mk - mt);
      }
      const float x0 = sum[r * D + d2], x1 = sum[r * D + d2 + 1];
      if (whole) {
        const float inv = lt == 0.f ? 0.f : vs / lt;
        *reinterpret_cast<uint32_t*>(a.out + use.s * a.out_stride + static_cast<int64_t>(h * group + r0 + r) * D + d2) =
            pack_bf16x2(x0 * inv, x1 * inv);
      } else {
        *reinterpret_cast<float2*>(po + r * D + d2) = make_float2(x0, x1);
        if (d2 == 0) {
          pm[r * 2] = mt;
          pm[r * 2 + 1] = lt;
        }
      }
    }
    __syncthreads();
  };

  lookup(steps > 0);
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) {
    if (i < steps) {
      fetch(i);
      lookup(i + 1 < steps);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  begin_unit();
  int stage = 0;
  int4 rec = make_int4(-1, 0, 0, 0);
  for (int i = 0; i < steps; ++i) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
    __syncwarp();
    if (i + kStages - 1 < steps) {
      fetch(stage == 0 ? kStages - 1 : stage - 1);           // the stage read one step ago
      lookup(i + kStages < steps);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    step(stage);
    stage = stage + 1 == kStages ? 0 : stage + 1;
    const bool last_of_unit = use.t + 1 == use.seen.nt;
    if (last_of_unit || i + 1 == steps) {
      const long long unit0 = t0 + i - use.t;
      end_unit(unit0);
      if (!last_of_unit && unit0 >= t0) {                     // goes on in the next stretches
        const long long end = unit0 + use.seen.nt;
        rec = make_int4(use.s, use.u, unit0 == t0 ? 0 : 1, static_cast<int>((end * ctas - 1) / total));
      }
    }
    use.next(a, SH::kTile);
    if (last_of_unit && i + 1 < steps) begin_unit();
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  if (tid == 0) a.parts.rec[c] = rec;
}

// The units that lie in several stretches: CTA (c, r) joins row r of the one
// that begins in stretch c and goes on, if any.  kJoinSplit groups of D
// threads take every kJoinSplit-th part, then add up in order.
constexpr int kJoinThreads = 256;
template <int D>
__global__ void __launch_bounds__(kJoinThreads) attn_decode_join_kernel(const DecodeArgs a, int f8) {
  constexpr int kGroups = kJoinThreads / D;
  __shared__ float w[kMaxCtas];
  __shared__ float red[kGroups][D];
  __shared__ float rmax[kJoinThreads / 32], rsum[kJoinThreads / 32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int c = blockIdx.x, r = blockIdx.y, tid = threadIdx.x;
  const int4 rec = a.parts.rec[c];
  if (rec.x < 0) return;
  const int group = a.hq / a.hkv, mtiles = a.units / a.hkv;
  const int h = rec.y / mtiles, r0 = (rec.y % mtiles) * kRows;
  if (r0 + r >= group) return;
  const int parts = rec.w - c + 1;                 // stretch c + i, i < parts
  auto slot = [&](int i) { return static_cast<size_t>((c + i) * 2 + (i == 0 ? rec.z : 0)); };
  float mt = -INFINITY;
  for (int i = tid; i < parts; i += kJoinThreads) mt = fmaxf(mt, a.parts.ml[(slot(i) * kRows + r) * 2]);
  mt = group_max<32>(mt);
  if ((tid & 31) == 0) rmax[tid >> 5] = mt;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kJoinThreads / 32; ++i) mt = fmaxf(mt, rmax[i]);
  float lt = 0.f;
  for (int i = tid; i < parts; i += kJoinThreads) {
    const float* p = a.parts.ml + (slot(i) * kRows + r) * 2;
    const float wi = p[0] == -INFINITY ? (p[1] != p[1] ? p[1] : 0.f) : ex2_approx_ftz(p[0] - mt);
    w[i] = wi;
    lt += wi * p[1];
  }
  lt = group_sum<32>(lt);
  if ((tid & 31) == 0) rsum[tid >> 5] = lt;
  __syncthreads();
  lt = 0.f;
#pragma unroll
  for (int i = 0; i < kJoinThreads / 32; ++i) lt += rsum[i];
  const int grp = tid / D, dim = tid % D;
  float acc = 0.f;
#pragma unroll 4
  for (int i = grp; i < parts; i += kGroups) acc = fmaf(w[i], a.parts.o[(slot(i) * kRows + r) * D + dim], acc);
  red[grp][dim] = acc;
  __syncthreads();
  if (grp == 0) {
#pragma unroll
    for (int i = 1; i < kGroups; ++i) acc += red[i][dim];
    const float vs = f8 && a.v_scale != nullptr ? a.v_scale[h] : 1.f;
    a.out[rec.x * a.out_stride + static_cast<int64_t>(h * group + r0 + r) * D + dim] =
        __float2bfloat16_rn(lt == 0.f ? 0.f : acc * (vs / lt));
  }
}

Parts parts_at(void* workspace, int d) {
  Parts p;
  p.o = static_cast<float*>(workspace);
  p.ml = p.o + static_cast<size_t>(kMaxCtas) * 2 * kRows * d;
  p.rec = reinterpret_cast<int4*>(p.ml + static_cast<size_t>(kMaxCtas) * 2 * kRows * 2);
  return p;
}

template <int D, typename E> cudaError_t launch(const DecodeArgs& a, int grid, cudaStream_t st) {
  using SH = Shape<D, E>;
  auto kernel = attn_decode_kernel<D, E>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SH::kSmem);
  if (e != cudaSuccess) return e;
  kernel<<<grid, kThreads, SH::kSmem, st>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // the join starts while the first kernel drains and waits for it
  PdlScope pdl(true);
  return launch_k(attn_decode_join_kernel<D>, dim3(grid, std::min(kRows, a.hq / a.hkv)), dim3(kJoinThreads), 0, st, a,
                  static_cast<int>(sizeof(E) == 1));
}

}  // namespace

size_t attn_decode_workspace(int, int, const rm_kv_cache& c) {
  return static_cast<size_t>(kMaxCtas) * (2 * kRows * (c.head_dim + 2) * sizeof(float) + sizeof(int4));
}

cudaError_t attn_decode_launch(const void* q, int64_t q_stride, const rm_kv_cache& c,
                               const int32_t* table, int table_stride, const int32_t* length,
                               int n, int hq, int window, int sinks, void* out, int64_t out_stride,
                               void* workspace, int num_sms, cudaStream_t st) {
  DecodeArgs a;
  a.q = static_cast<const bf16*>(q);
  a.q_stride = q_stride;
  a.kc = c.k;
  a.vc = c.v;
  a.page_stride = c.page_stride;
  a.n_pages = c.n_pages;
  a.P = c.page_size;
  // x / P for 0 <= x < 2^31 as x * ceil(2^shift / P) >> shift with 2^shift =
  // 2^31 * (the power of two from P on): the multiplier fits 32 bits and
  // exceeds 2^shift / P by less than 1, so the quotient is too large by less
  // than 2^31 / 2^shift <= 1 / P
  a.shift = 31;
  while ((1 << (a.shift - 31)) < c.page_size) ++a.shift;
  a.div = static_cast<uint32_t>(((1ull << a.shift) + c.page_size - 1) / c.page_size);
  a.k_scale = c.k_scale;
  a.v_scale = c.v_scale;
  a.table = table;
  a.table_stride = table_stride;
  a.length = length;
  a.n = n;
  a.hq = hq;
  a.hkv = c.n_kv_heads;
  a.window = window;
  a.sinks = sinks;
  a.out = static_cast<bf16*>(out);
  a.out_stride = out_stride;
  a.scale_log2 = 1.4426950408889634f / sqrtf(static_cast<float>(c.head_dim));
  const int group = hq / c.n_kv_heads;
  a.units = c.n_kv_heads * ((group + kRows - 1) / kRows);
  a.parts = parts_at(workspace, c.head_dim);
  // no more CTAs than tiles of the longest possible contexts
  const int64_t most = static_cast<int64_t>(n) * a.units *
                       std::max<int64_t>(1, (static_cast<int64_t>(table_stride) * c.page_size + 63) / 64);
  const int grid = static_cast<int>(std::min<int64_t>(most, std::min(kMaxCtas, num_sms * kCtasPerSm)));
  using F8 = __nv_fp8_e4m3;
  if (c.dtype == RM_E4M3) return c.head_dim == 64 ? launch<64, F8>(a, grid, st) : launch<128, F8>(a, grid, st);
  return c.head_dim == 64 ? launch<64, bf16>(a, grid, st) : launch<128, bf16>(a, grid, st);
}

}  // namespace rmk
