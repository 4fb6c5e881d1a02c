// Attention of one new token per sequence over a paged cache.
//
// A step reads every visible key and value once (2 * len * d elements for a
// key-value head) and computes 4 * d operations per query head and key: it is
// bound by memory, and by latency when the batch is small.  The kernel
// therefore spreads the bytes evenly and keeps many of them in flight:
//  - the (sequence, kv head) units' key tiles, laid end to end, are cut into
//    one equal stretch per CTA whatever the lengths are, so a long context
//    beside short ones does not leave SMs idle and no length needs to be known
//    on the host.  A unit that a cut divides leaves its parts (reference, sum,
//    unnormalised output) in the workspace; a second kernel joins them in
//    stretch order.
//  - each warp of a CTA takes its own keys of every tile through a private
//    ring of cp.async stages, with no barrier between warps until a unit ends;
//    the ring runs across unit borders.
//  - the query heads that share a kv head are the columns of mma.sync tiles
//    (m16n8k16: 16 keys by 8 heads for the scores, 16 dims by 8 heads for the
//    output), so a key is read once for all of them and a step's arithmetic
//    follows the head count, eight at a time.
// Measured on B200, among calls on other inputs (in brackets: replayed on the
// same ones): 24 contexts of up to 131071 tokens, 32 heads on 8 of 128 dims:
// 193 us (192), 6.3 TB/s (95% of a copy's rate); 64 contexts of 256 to 560
// tokens, 16 heads of 128: 42 us (42), 5.1 TB/s (the rings' ramp and two
// launches); 128 windows over e4m3 pages: 94 us (86), 5.4 TB/s (the conversions
// take 45% of the issue slots); one context of 500 tokens: 9.4 us (6.8),
// latency.
#include <cuda_fp8.h>

#include <algorithm>
#include <cfloat>

#include "common.cuh"
#include "kernels.h"
#include "paging.cuh"

namespace rmk {
namespace {

RMK_BOUNDS_UNIT(attention_decode)

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kUnitCost = 2;                    // a unit's beginning and end, in tiles
constexpr int kCtasPerSm = 2;
constexpr int kMaxCtas = 148 * kCtasPerSm;      // the workspace has parts for this many

// NH columns of eight query heads per unit.  Keys per warp and step, and ring
// depth: a stage holds 8 KB of keys and values (4 KB for 8-bit heads of 64),
// and two CTAs fit an SM.
template <int D, typename E, int NH> struct Shape {
  static constexpr int kRows = 8 * NH;                  // query heads of a unit
  static constexpr int kKeys = D * sizeof(E) >= 256 ? 16 : 32;
  static constexpr int kTile = kWarps * kKeys;
  static constexpr int kRowBytes = D * sizeof(E);
  static constexpr int kHalf = kKeys * kRowBytes;       // the keys of a stage; its values follow
  static constexpr int kStages = 2 * kHalf >= 8192 ? 3 : 6;
  static constexpr int kRing = kWarps * kStages * 2 * kHalf;
  static constexpr int kPitch = D + 4;                  // of a head's sums: heads 2t in different banks
  static constexpr int kSum = kRing;                    // float [kRows][kPitch]
  static constexpr int kMl = kSum + kRows * kPitch * 4; // float [kWarps][kRows][2]
  static constexpr int kSmem = kMl + kWarps * kRows * 2 * 4;
};

struct Parts {            // workspace
  float* o;               // [ctas][2][rows][D]
  float* ml;              // [ctas][2][rows][2]: reference, sum
  int4* rec;              // [ctas]: unit that begins in the CTA's stretch and goes on behind it
};

struct DecodeArgs {
  const bf16* q;
  int64_t q_stride;
  const void* kc;
  const void* vc;
  int64_t page_stride;
  int n_pages;
  PageDiv div;
  const float* k_scale;
  const float* v_scale;
  const int32_t* table;
  int table_stride;
  const int32_t* length;
  int n, hq, hkv, window, sinks;
  bf16* out;
  int64_t out_stride;
  float scale_log2;
  int units;                    // per sequence: hkv * ceil(group / rows of a unit)
  Parts parts;
};

// What a sequence's newest token sees: keys [0, nsink) and then, from the
// nsink-th on, keys j + skip; vis of them in tiles of `tile`, at least one
// (an empty sequence's row of zeros is written by somebody too).
struct Seen {
  int vis, nsink, skip, nt;
};
__device__ __forceinline__ Seen seen_of(const DecodeArgs& a, int s, int tile) {
  const int64_t cap = static_cast<int64_t>(a.table_stride) * a.div.P;
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

// Position in the laid-out tiles: sequence, unit of it, key tile of that, and
// the tile's place v.  A unit takes kUnitCost places before its first tile, so
// that stretches of many short units are no slower than others.
struct Cursor {
  int s, u, t;
  long long v;
  Seen seen;
  __device__ __forceinline__ void next(const DecodeArgs& a, int tile) {
    ++v;
    if (++t < seen.nt) return;
    t = 0;
    v += kUnitCost;
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
// four e4m3 bytes as fp16: bytes 0 and 1 in lo, 2 and 3 in hi
__device__ __forceinline__ void e4m3x4_f16(uint32_t x, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(x));
}
// the transpose of the 8 x 8 matrix of 16-bit elements that a warp holds, row
// lane / 4, columns 2 (lane % 4) and one more
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// The reference of a row's exponentials, from its running maximum.  bf16 caches
// take the maximum itself: the largest probability is then 1, which has no
// rounding, and bf16 has the small ones.  fp16 (8-bit caches) runs out at
// 2^-24, so there the largest is 2^15: weights down to 2^-32 of it keep the
// precision of bf16, those below 2^-40 are 0 (with a largest of 1: 2^-17 and
// 2^-25, and a long flat tail under one key was lost).  The sum and the output
// carry the same factor.  From |maximum| = 2^20 on its fp32 step is 1/8 and the
// subtraction would round, up to an overflow of fp16: the maximum itself.
template <typename E> __device__ __forceinline__ float reference(float top) {
  return sizeof(E) == 1 && fabsf(top) < 1048576.f ? top - 15.f : top;
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

template <int D, typename E, int NH>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) attn_decode_kernel(const DecodeArgs a) {
  using SH = Shape<D, E, NH>;
  constexpr bool kF8 = sizeof(E) == 1;
  constexpr int kKeys = SH::kKeys, kStages = SH::kStages, kRows = SH::kRows, kPitch = SH::kPitch;
  extern __shared__ __align__(1024) uint8_t sm[];
  __shared__ long long scan[kWarps];
  __shared__ int start_s;
  __shared__ long long start_rem;
  __shared__ uint32_t masks[kWarps][kStages];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_launch_dependents();
  pdl_wait();

  // this CTA's stretch [v0, v1) of all places, and where it begins
  const int per = (a.n + kThreads - 1) / kThreads;
  const int i0 = min(a.n, tid * per), i1 = min(a.n, i0 + per);
  auto places = [&](int i) { return static_cast<long long>(seen_of(a, i, SH::kTile).nt + kUnitCost) * a.units; };
  long long mine = 0;
  for (int i = i0; i < i1; ++i) mine += places(i);
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
  const long long v0 = c < ctas ? c * total / ctas : total, v1 = c < ctas ? (c + 1) * total / ctas : total;
  if (v0 < v1 && v0 >= upto - mine && v0 < upto) {
    long long rem = v0 - (upto - mine);
    int i = i0;
    for (;; ++i) {
      const long long k = places(i);
      if (rem < k) break;
      rem -= k;
    }
    start_s = i;
    start_rem = rem;
  }
  __syncthreads();
  Cursor use;
  use.v = v1;                                   // an empty stretch
  if (v0 < v1) {
    use.s = start_s;
    use.seen = seen_of(a, use.s, SH::kTile);
    const int len = use.seen.nt + kUnitCost;
    use.u = static_cast<int>(start_rem / len);
    const int at = static_cast<int>(start_rem % len);
    use.t = max(0, at - kUnitCost);
    use.v = v0 + max(0, kUnitCost - at);        // the first place of the stretch that holds a tile
  }
  if (use.v >= v1) {
    if (tid == 0) a.parts.rec[c] = make_int4(-1, 0, 0, 0);
    return;
  }
  Cursor get = use;
  const long long first = use.v;
  const int group = a.hq / a.hkv, mtiles = a.units / a.hkv;

  uint8_t* ring = sm + warp * kStages * 2 * SH::kHalf;
  const uint32_t ring_u = static_cast<uint32_t>(__cvta_generic_to_shared(ring));
  float* sum = reinterpret_cast<float*>(sm + SH::kSum);
  float* ml = reinterpret_cast<float*>(sm + SH::kMl);

  // The page of a lane's key is looked up one step before its rows are
  // fetched.
  int pg = -1;
  bool got = false;                             // a step is looked up
  int64_t row_in_page = 0;
  auto lookup = [&]() {
    pg = -1;
    got = get.v < v1;
    if (!got) return;
    const unsigned j = static_cast<unsigned>(get.t) * SH::kTile + warp * kKeys + lane;
    if (lane < kKeys && j < static_cast<unsigned>(get.seen.vis)) {
      const int key = static_cast<int>(j) + (j < static_cast<unsigned>(get.seen.nsink) ? 0 : get.seen.skip);
      const int b = a.div.floor(key);
      row_in_page = static_cast<int64_t>(get.u / mtiles) * a.div.P + (key - b * a.div.P);
      if (in_bounds(get.s < a.n && b < a.table_stride && key - b * a.div.P >= 0 && key - b * a.div.P < a.div.P))
        pg = a.table[static_cast<int64_t>(get.s) * a.table_stride + b];
    }
    get.next(a, SH::kTile);
  };
  auto fetch = [&](int stage) {
    const bool ok = pg >= 0 && pg < a.n_pages;
    const int64_t at = ok ? (pg * a.page_stride + row_in_page * D) * static_cast<int64_t>(sizeof(E)) : 0;
    const uint32_t mask = __ballot_sync(0xffffffffu, ok);
    if (lane == 0) masks[warp][stage] = mask;
    const uint32_t dst = ring_u + stage * 2 * SH::kHalf;
    constexpr int kChunks = SH::kRowBytes / 16;
    const char* kb = static_cast<const char*>(a.kc) + (lane % kChunks) * 16;
    const char* vb = static_cast<const char*>(a.vc) + (lane % kChunks) * 16;
#pragma unroll
    for (int i = 0; i < kKeys * kChunks / 32; ++i) {
      const int r = i * (32 / kChunks) + lane / kChunks;
      const int64_t off = __shfl_sync(0xffffffffu, at, r);
      const int bytes = (mask >> r) & 1 ? 16 : 0;               // 0: the row is filled with zeros
      const uint32_t d = dst + chunk_at<SH::kRowBytes>(r, lane % kChunks);
      cp16(d, kb + off, bytes);
      cp16(d + SH::kHalf, vb + off, bytes);
    }
  };

  // The lane's heads are columns 8 nh + 2t, + 1 (t = lane % 4) of the scores
  // and the output; the query operand holds head 8 nh + lane / 4.
  const int g = lane >> 2, t2 = (lane & 3) * 2;
  uint32_t qf[NH][D / 16][2];
  float sc[NH][2], m[NH][2], l[NH][2], o[D / 16][NH][4];
  // A unit's queries are asked for before the unit ahead of it is joined and
  // written, and made ready (8-bit caches) and its state reset behind that.
  auto load_queries = [&]() {
    const int h = use.u / mtiles, r0 = (use.u % mtiles) * kRows;
    const int rows = min(kRows, group - r0);
    const bf16* q = a.q + use.s * a.q_stride + static_cast<int64_t>(h * group + r0) * D;
#pragma unroll
    for (int nh = 0; nh < NH; ++nh) {
      const int r = nh * 8 + g;
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          // 8-bit keys arrive four dims to a lane: dims 4t..4t+3 of a step are
          // the MMA's k = 2t, 2t+1, 2t+8, 2t+9, for the query as for the keys
          const int dim = k * 16 + (kF8 ? 2 * t2 + x * 2 : t2 + x * 8);
          qf[nh][k][x] = r < rows ? *reinterpret_cast<const uint32_t*>(q + r * D + dim) : 0u;
        }
    }
  };
  auto begin_unit = [&]() {
    const float ks = a.scale_log2 * (kF8 && a.k_scale != nullptr ? a.k_scale[use.u / mtiles] : 1.f);
#pragma unroll
    for (int nh = 0; nh < NH; ++nh) {
      sc[nh][0] = sc[nh][1] = ks;
      if (kF8) {
        // bf16 queries as fp16, times the power of two that brings the head's
        // largest to [2^13, 2^14): exact but for entries 2^-27 below it
        float top = 0.f;
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
#pragma unroll
          for (int x = 0; x < 2; ++x) top = fmaxf(top, fmaxf(fabsf(bf16_lo(qf[nh][k][x])), fabsf(bf16_hi(qf[nh][k][x]))));
        top = group_max<4>(top);
        const int e = top > 0.f && top < INFINITY ? 13 - ilogbf(top) : 0;
        // 2^e as two factors: e may pass the exponents of fp32
        const float f0 = ldexpf(1.f, e >> 1), f1 = ldexpf(1.f, e - (e >> 1));
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
#pragma unroll
          for (int x = 0; x < 2; ++x)
            qf[nh][k][x] = pack_f16x2(bf16_lo(qf[nh][k][x]) * f0 * f1, bf16_hi(qf[nh][k][x]) * f0 * f1);
        const float back = ldexpf(ks, -e);
        sc[nh][0] = __shfl_sync(0xffffffffu, back, t2 * 4);
        sc[nh][1] = __shfl_sync(0xffffffffu, back, t2 * 4 + 4);
      }
      m[nh][0] = m[nh][1] = -INFINITY;
      l[nh][0] = l[nh][1] = 0.f;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) o[i][nh][0] = o[i][nh][1] = o[i][nh][2] = o[i][nh][3] = 0.f;
    }
  };

  const int lr = lane & 7, lm = lane >> 3;
  auto step = [&](int stage) {
    const uint32_t kb = ring_u + stage * 2 * SH::kHalf, vb = kb + SH::kHalf;
    const uint32_t keys = masks[warp][stage], mask = keys >> g;  // of keys g, g + 8, ...
    float s[kKeys / 16][NH][4];
#pragma unroll
    for (int kt = 0; kt < kKeys / 16; ++kt) {
#pragma unroll
      for (int nh = 0; nh < NH; ++nh) s[kt][nh][0] = s[kt][nh][1] = s[kt][nh][2] = s[kt][nh][3] = 0.f;
      const int kr = kt * 16 + (lm & 1) * 8 + lr;
      if (kF8) {
#pragma unroll
        for (int k2 = 0; k2 < D / 32; ++k2) {                    // two 16-dim steps a load
          uint32_t b[4], f[4];
          ldsm4(kb + chunk_at<SH::kRowBytes>(kr, k2 * 2 + (lm >> 1)), b);
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            e4m3x4_f16(b[2 * x], f[0], f[2]);
            e4m3x4_f16(b[2 * x + 1], f[1], f[3]);
#pragma unroll
            for (int nh = 0; nh < NH; ++nh) mma<E>(s[kt][nh], f, qf[nh][k2 * 2 + x][0], qf[nh][k2 * 2 + x][1]);
          }
        }
      } else {
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          uint32_t b[4];
          ldsm4(kb + chunk_at<SH::kRowBytes>(kr, k * 2 + (lm >> 1)), b);
#pragma unroll
          for (int nh = 0; nh < NH; ++nh) mma<E>(s[kt][nh], b, qf[nh][k][0], qf[nh][k][1]);
        }
      }
    }
    // base-2 scores: elements 0, 1 of key 16 kt + g, 2, 3 of key 16 kt + 8 + g.
    // Once a key is seen the maximum is above -inf: scores of -inf weigh nothing,
    // and a row of them alone ends as 0 / 0.  So a maximum of -inf stands for no
    // key seen, a sum of 0 and an output of 0; a NaN is in the output already.
    const float floor = keys != 0u ? -FLT_MAX : -INFINITY;
#pragma unroll
    for (int nh = 0; nh < NH; ++nh) {
      float top[2] = {floor, floor};
#pragma unroll
      for (int kt = 0; kt < kKeys / 16; ++kt)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const bool in = (mask >> (kt * 16 + (x >> 1) * 8)) & 1;
          s[kt][nh][x] = in ? s[kt][nh][x] * sc[nh][x & 1] : -INFINITY;
          top[x & 1] = fmaxf(top[x & 1], s[kt][nh][x]);
        }
#pragma unroll
      for (int w = 4; w < 32; w <<= 1) {
        top[0] = fmaxf(top[0], __shfl_xor_sync(0xffffffffu, top[0], w));
        top[1] = fmaxf(top[1], __shfl_xor_sync(0xffffffffu, top[1], w));
      }
      // The maximum seldom moves, and only then is the output rescaled.
      if (__any_sync(0xffffffffu, top[0] > m[nh][0] || top[1] > m[nh][1])) {
        float keep[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float mn = fmaxf(m[nh][x], top[x]);
          keep[x] = m[nh][x] == -INFINITY ? 0.f : ex2_approx_ftz(reference<E>(m[nh][x]) - reference<E>(mn));
          m[nh][x] = mn;
          l[nh][x] *= keep[x];
        }
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
          for (int x = 0; x < 4; ++x) o[i][nh][x] *= keep[x & 1];
      }
      const float ref[2] = {m[nh][0] == -INFINITY ? 0.f : reference<E>(m[nh][0]),
                            m[nh][1] == -INFINITY ? 0.f : reference<E>(m[nh][1])};
#pragma unroll
      for (int kt = 0; kt < kKeys / 16; ++kt)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          s[kt][nh][x] = ex2_approx_ftz(s[kt][nh][x] - ref[x & 1]);   // a masked key's is 2^-inf = 0
          l[nh][x & 1] += s[kt][nh][x];
        }
    }
#pragma unroll
    for (int kt = 0; kt < kKeys / 16; ++kt) {
      uint32_t p[NH][2];
#pragma unroll
      for (int nh = 0; nh < NH; ++nh)
#pragma unroll
        for (int x = 0; x < 2; ++x)
          p[nh][x] = transposed(kF8 ? pack_f16x2(s[kt][nh][2 * x], s[kt][nh][2 * x + 1])
                                    : pack_bf16x2(s[kt][nh][2 * x], s[kt][nh][2 * x + 1]));
      if (kF8) {
        const int vr = kt * 16 + (lm & 1) * 8 + lr;
#pragma unroll
        for (int d2 = 0; d2 < D / 32; ++d2) {                    // two 16-dim tiles a load
          uint32_t b[4], f[4];
          ldsm4t(vb + chunk_at<SH::kRowBytes>(vr, d2 * 2 + (lm >> 1)), b);
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            // a register holds dims 2g, 2g+1 of two keys: the tile's rows
            // 0..7 are the even dims, 8..15 the odd ones
            e4m3x4_f16(__byte_perm(b[2 * x], 0, 0x3120), f[0], f[1]);
            e4m3x4_f16(__byte_perm(b[2 * x + 1], 0, 0x3120), f[2], f[3]);
#pragma unroll
            for (int nh = 0; nh < NH; ++nh) mma<E>(o[d2 * 2 + x][nh], f, p[nh][0], p[nh][1]);
          }
        }
      } else {
        const int vr = kt * 16 + (lm >> 1) * 8 + lr;
#pragma unroll
        for (int dt = 0; dt < D / 16; ++dt) {
          uint32_t b[4];
          ldsm4t(vb + chunk_at<SH::kRowBytes>(vr, dt * 2 + (lm & 1)), b);
#pragma unroll
          for (int nh = 0; nh < NH; ++nh) mma<E>(o[dt][nh], b, p[nh][0], p[nh][1]);
        }
      }
    }
  };

  // Joins the warps' states of a finished unit, in warp order, and writes the
  // output rows, or the unit's part when the stretch holds only part of it.
  // As many warps as the buffer has room for write at once.
  auto end_unit = [&](int s, int u, long long unit0, bool whole) {
    const int h = u / mtiles, r0 = (u % mtiles) * kRows;
    const int rows = min(kRows, group - r0);
#pragma unroll
    for (int nh = 0; nh < NH; ++nh)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        m[nh][x] = reference<E>(m[nh][x]);                       // what the parts are joined by
#pragma unroll
        for (int w = 4; w < 32; w <<= 1) l[nh][x] += __shfl_xor_sync(0xffffffffu, l[nh][x], w);
        if (g == 0) {
          ml[(warp * kRows + nh * 8 + t2 + x) * 2] = m[nh][x];
          ml[(warp * kRows + nh * 8 + t2 + x) * 2 + 1] = l[nh][x];
        }
      }
    __syncthreads();
    const int room = rows * 4 <= kRows ? 4 : (rows * 2 <= kRows ? 2 : 1);
    for (int i = 0; i < kWarps; i += room) {
      if (warp >= i && warp < i + room) {
#pragma unroll
        for (int nh = 0; nh < NH; ++nh)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int r = nh * 8 + t2 + x;
            if (r >= rows) continue;
            float mt = -INFINITY;
#pragma unroll
            for (int k = 0; k < kWarps; ++k) mt = fmaxf(mt, ml[(k * kRows + r) * 2]);
            const float w = m[nh][x] == -INFINITY ? 0.f : ex2_approx_ftz(m[nh][x] - mt);
            float* dst = sum + ((warp - i) * rows + r) * kPitch;
#pragma unroll
            for (int dt = 0; dt < D / 16; ++dt)
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                const int dim = dt * 16 + (kF8 ? 2 * g + y : 8 * y + g);
                const float v = o[dt][nh][2 * y + x] * w;
                dst[dim] = i == 0 ? v : dst[dim] + v;
              }
          }
      }
      __syncthreads();
    }
    const int slot = unit0 + kUnitCost <= first ? 0 : 1;
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
        lt += mk == -INFINITY ? 0.f : lk * ex2_approx_ftz(mk - mt);
      }
      float x0 = 0.f, x1 = 0.f;
      for (int k = 0; k < room; ++k) {
        const float2 v = *reinterpret_cast<const float2*>(sum + (k * rows + r) * kPitch + d2);
        x0 += v.x;
        x1 += v.y;
      }
      if (whole) {
        const float inv = mt == -INFINITY ? 0.f : 1.f / lt;                   // no key: zeros
        *reinterpret_cast<uint32_t*>(a.out + s * a.out_stride + static_cast<int64_t>(h * group + r0 + r) * D + d2) =
            pack_bf16x2(x0 * inv * vs, x1 * inv * vs);
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

  lookup();
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) {
    if (got) {
      fetch(i);
      lookup();
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  load_queries();
  begin_unit();
  int stage = 0;
  int4 rec = make_int4(-1, 0, 0, 0);
  for (;;) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
    __syncwarp();
    if (got) {
      fetch(stage == 0 ? kStages - 1 : stage - 1);           // the stage read one step ago
      lookup();
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    step(stage);
    stage = stage + 1 == kStages ? 0 : stage + 1;
    const bool last_of_unit = use.t + 1 == use.seen.nt;
    const bool last = last_of_unit ? use.v + 1 + kUnitCost >= v1 : use.v + 1 >= v1;
    if (!last_of_unit && !last) {
      use.next(a, SH::kTile);
      continue;
    }
    const int s = use.s, u = use.u;
    const long long unit0 = use.v - use.t - kUnitCost;        // the unit's first place
    const bool begins = unit0 + kUnitCost >= first;           // its first tile is in this stretch
    if (!last_of_unit && begins) {                            // it goes on in the next stretches
      const long long end = unit0 + kUnitCost + use.seen.nt;
      rec = make_int4(s, u, unit0 + kUnitCost <= first ? 0 : 1, static_cast<int>((end * ctas - 1) / total));
    }
    if (!last) {
      use.next(a, SH::kTile);
      load_queries();
    }
    end_unit(s, u, unit0, begins && last_of_unit);
    if (last) break;
    begin_unit();
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  if (tid == 0) a.parts.rec[c] = rec;
}

// The units that lie in several stretches: CTA (c, r) joins row r of the one
// that begins in stretch c and goes on, if any.  kJoinSplit groups of D
// threads take every kJoinSplit-th part, then add up in order.
constexpr int kJoinThreads = 256;
template <int D, int NH>
__global__ void __launch_bounds__(kJoinThreads) attn_decode_join_kernel(const DecodeArgs a, int f8) {
  constexpr int kRows = 8 * NH;
  constexpr int kGroups = kJoinThreads / D;
  __shared__ float w[kMaxCtas];
  __shared__ float red[kGroups][D];
  __shared__ float rmax[kJoinThreads / 32], rsum[kJoinThreads / 32];
  pdl_wait();
  const int c = blockIdx.x, r = blockIdx.y, tid = threadIdx.x;
  const int4 rec = a.parts.rec[c];
  if (rec.x < 0) return;
  if (!in_bounds(rec.x < a.n && rec.y >= 0 && rec.y < a.units && rec.w >= c && rec.w < static_cast<int>(gridDim.x))) return;
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
    const float wi = p[0] == -INFINITY ? 0.f : ex2_approx_ftz(p[0] - mt);
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
        __float2bfloat16_rn(mt == -INFINITY ? 0.f : acc * (1.f / lt) * vs);
  }
}

constexpr int kMaxRows = 16;                    // query heads per unit

Parts parts_at(void* workspace, int d) {
  Parts p;
  p.o = static_cast<float*>(workspace);
  p.ml = p.o + static_cast<size_t>(kMaxCtas) * 2 * kMaxRows * d;
  p.rec = reinterpret_cast<int4*>(p.ml + static_cast<size_t>(kMaxCtas) * 2 * kMaxRows * 2);
  return p;
}

template <int D, typename E, int NH>
cudaError_t launch(DecodeArgs a, int num_sms, cudaStream_t st) {
  using SH = Shape<D, E, NH>;
  const int group = a.hq / a.hkv;
  a.units = a.hkv * ((group + SH::kRows - 1) / SH::kRows);
  // no more CTAs than tiles of the longest possible contexts
  const int64_t keys = static_cast<int64_t>(a.table_stride) * a.div.P;
  const int64_t most = static_cast<int64_t>(a.n) * a.units * ((keys + SH::kTile - 1) / SH::kTile + kUnitCost);
  const int grid = static_cast<int>(std::min<int64_t>(most, std::min(kMaxCtas, num_sms * kCtasPerSm)));
  auto kernel = attn_decode_kernel<D, E, NH>;
  static std::atomic<unsigned long long> allowed{0};
  cudaError_t e = allow_smem(kernel, SH::kSmem, allowed);
  if (e != cudaSuccess) return e;
  PdlScope pdl(true);
  e = launch_k(kernel, dim3(grid), dim3(kThreads), SH::kSmem, st, a);
  if (e != cudaSuccess) return e;
  // the join is launched while the first kernel drains, and waits for it
  return launch_k(attn_decode_join_kernel<D, NH>, dim3(grid, std::min(SH::kRows, group)), dim3(kJoinThreads), 0, st, a,
                  static_cast<int>(sizeof(E) == 1));
}

}  // namespace

cudaError_t bounds_errors_attention_decode(int32_t* out, bool reset) {
  cudaError_t e = cudaMemcpyFromSymbol(out, g_bounds_attention_decode, sizeof(int32_t));
  if (e == cudaSuccess && reset) {
    const int32_t zero = 0;
    e = cudaMemcpyToSymbol(g_bounds_attention_decode, &zero, sizeof(int32_t));
  }
  return e;
}

size_t attn_decode_workspace(int, int, const rm_kv_cache& c) {
  return static_cast<size_t>(kMaxCtas) * (2 * kMaxRows * (c.head_dim + 2) * sizeof(float) + sizeof(int4));
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
  a.div = page_div(c.page_size);
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
  a.parts = parts_at(workspace, c.head_dim);
  // up to eight query heads a kv head: one column tile, half the arithmetic
  const bool few = hq / c.n_kv_heads <= 8;
  auto go = [&](auto elem) {
    using E = decltype(elem);
    if (c.head_dim == 64) return few ? launch<64, E, 1>(a, num_sms, st) : launch<64, E, 2>(a, num_sms, st);
    return few ? launch<128, E, 1>(a, num_sms, st) : launch<128, E, 2>(a, num_sms, st);
  };
  return c.dtype == RM_E4M3 ? go(__nv_fp8_e4m3{}) : go(bf16{});
}

}  // namespace rmk
