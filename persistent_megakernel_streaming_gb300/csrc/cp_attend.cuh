// cp_attend.cuh -- what the attention kernels share: the plain path of rows
// next to masked non-finite values, and how a part's result is stored.
#pragma once
#include "cp_cache.cuh"
#include "cp_cache_ptx.cuh"
#include "cp_call.h"

namespace cp {
namespace cache {

using ptx::pdl_trigger;
using ptx::pdl_wait;

// Biased exponent of a bf16 pattern, 0 for infinities and NaN.
__device__ __forceinline__ int finite_exp(uint32_t h) {
  const int e = (int)(h >> 7) & 255;
  return e == 255 ? 0 : e;
}

// Whether 16 bytes of shared memory hold an element that is not finite.
template <bool E4M3>
__device__ __forceinline__ bool any_nonfinite(uint32_t addr) {
  const uint4 x = ptx::ld_shared_v4u(addr);
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  bool bad = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (E4M3) bad |= __vcmpeq4(w[i] & 0x7f7f7f7fu, 0x7f7f7f7fu) != 0;
    else bad |= __vcmpeq2(w[i] & 0x7f807f80u, 0x7f807f80u) != 0;
  }
  return bad;
}

// Whether 16 e4m3 bytes hold an element that is not zero.
__device__ __forceinline__ bool any_nonzero(uint4 x) { return ((x.x | x.y | x.z | x.w) & 0x7f7f7f7fu) != 0; }

// Over an e4m3 cache q enters the products in fp16, each row under a power of two that puts its largest element into
// [1, 4), but for rows of less than 2^kLeastExp. Elements below 2^-14 lose bits there. What a row has lost, times the
// scale of its scores and the largest key that it may meet (448 times the largest scale), bounds the error of a score (in
// powers of two); a block where that passes kMostLost computes its rows the plain way, from q as it is. kLeastLost
// stands in for a row that lost nothing, so that the same bound finds scores whose scale comes near the end of fp32.
// (Looking costs 16 sequences of 1 or 301 rows 1.3 % of their 141 us, 64 single rows 0.2 % of 143.)
constexpr float kMostLost = 0x1p-12f, kLeastLost = 0x1p-121f;
constexpr int kLeastExp = -100;    // of a row's power of two, which times the scale of the scores stays a normal float

// Whether fp16 pairs hold an element below fp16's normal range.
template <int N>
__device__ __forceinline__ bool any_small(const uint32_t* y) {
  __half2 m = __habs2(*reinterpret_cast<const __half2*>(y));
#pragma unroll
  for (int i = 1; i < N; ++i) m = __hmin2(m, __habs2(*reinterpret_cast<const __half2*>(y + i)));
  const uint32_t x = *reinterpret_cast<const uint32_t*>(&m);
  return !(x & 0x7c00u) || !(x & 0x7c000000u);
}
// What the fp16 pair y keeps not of the bf16 pair w times f (nothing of infinities and NaN).
__device__ __forceinline__ float left_out(uint32_t w, float f, uint32_t y) {
  const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&y));
  return fmaxf(fabsf(bf_lo(w) * f - h.x), 0.f) + fmaxf(fabsf(bf_hi(w) * f - h.y), 0.f);
}

// Most powers of two by which the reference of an e4m3 cache's value scales may rise: fp32 outputs follow it with
// their precision. Past it the rows that do not see the new value could lose theirs.
constexpr int kMostRise = 110;

// Four neighbouring elements of a row's result: the answer itself, rounded, or
// a part's average in fp32.
template <int D>
__device__ __forceinline__ void store4(const AttendParams& p, int part, bool whole, int64_t row, int head, int d,
                                       const float* x) {
  if (whole)
    *reinterpret_cast<uint2*>(p.out + row * p.o_row + head * p.o_head + d) = make_uint2(bf_pack(x[0], x[1]), bf_pack(x[2], x[3]));
  else
    *reinterpret_cast<float4*>(p.part_o + (((int64_t)part * p.b.rows + row) * p.q_heads + head) * D + d) =
        make_float4(x[0], x[1], x[2], x[3]);
}
__device__ __forceinline__ void store_lse(const AttendParams& p, int part, int64_t row, int head, float lse) {
  p.part_lse[((int64_t)part * p.b.rows + row) * p.q_heads + head] = lse;
}

// Rows i0 .. i1-1 of a sequence and kv head (row i: new row i / group, query
// head i % group of the kv head) over positions [t_begin, t_end), a warp a
// row: lanes share the head's elements, walk the positions the row sees and
// read no other, with a running maximum and sum. The matrix kernels multiply
// masked values by zero, which is wrong where one is infinite or NaN; a block
// that finds one next to a mask runs this instead. So does one over an e4m3
// cache whose positions' scales lie further apart than the 16-bit operands
// reach (a row may see only the small ones), or whose q is wider than fp16.
// Right and slow: 512 rows over 32768 bf16 positions 60 ms a call instead of
// 0.135 where one NaN stands behind the diagonal, 64 single rows over e4m3
// with one value 2^20 above the others 6.6 ms instead of 0.14.
template <int D, bool E4M3>
__device__ __noinline__ void plain_rows(const AttendParams& p, Seq s, int seq, int kv, int i0, int i1, int t_begin,
                                        int t_end, int part, bool whole, int warp, int warps, float* avg = nullptr,
                                        float* avg_lse = nullptr, int pitch = D) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const int32_t* table = p.b.table + (int64_t)seq * p.b.table_stride;
  for (int i = i0 + warp; i < i1; i += warps) {
    const int64_t row = s.row0 + i / p.group;
    const int head = kv * p.group + i % p.group;
    int lo, hi;
    visible(p, s.first + i / p.group, s.len, &lo, &hi);
    lo = max(lo, t_begin);
    hi = min(hi, t_end);
    const uint16_t* qp = p.q + row * p.q_row + head * p.q_head + lane * E;
    float q[E], acc[E] = {};
#pragma unroll
    for (int j = 0; j < E; ++j) q[j] = __uint_as_float((uint32_t)qp[j] << 16) * p.scale_log2;
    float m = -INFINITY, l = 0.f;
    for (int t = lo; t < hi; ++t) {
      const int page = page_of(table, p.b.width, p.c.pages, p.c.page_shift, t);
      float k[E] = {}, v[E] = {};
      if (page < 0) {
        set_status(p.c.status, CP_ERR_DEVICE_BOUNDS);
      } else {
        const int64_t at = slot_bytes(p.c, page, kv, t);
        if (E4M3) {
          const int64_t sc = slot_scale(p.c, page, kv, t);
          const float fk = pow2i((int)p.c.ks[sc] - 127), fv = pow2i((int)p.c.vs[sc] - 127);
#pragma unroll
          for (int j = 0; j < E; ++j) {
            float f[4];
            e4m3x4_f32(p.c.k[at + lane * E + j], f);
            k[j] = f[0] * fk;
            e4m3x4_f32(p.c.v[at + lane * E + j], f);
            v[j] = f[0] * fv;
          }
        } else {
#pragma unroll
          for (int j = 0; j < E; ++j) {
            k[j] = __uint_as_float((uint32_t) reinterpret_cast<const uint16_t*>(p.c.k + at)[lane * E + j] << 16);
            v[j] = __uint_as_float((uint32_t) reinterpret_cast<const uint16_t*>(p.c.v + at)[lane * E + j] << 16);
          }
        }
      }
      float d = 0.f;
#pragma unroll
      for (int j = 0; j < E; ++j) d += q[j] * k[j];
#pragma unroll
      for (int o = 16; o; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
      const float mn = fmaxf(m, d), ref = mn == -INFINITY ? 0.f : mn;
      const float a = ex2(m - ref), w = ex2(d - ref);
      l = l * a + w;
#pragma unroll
      for (int j = 0; j < E; ++j) acc[j] = acc[j] * a + w * v[j];
      m = mn;
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    if (whole) {
#pragma unroll
      for (int j = 0; j < E; ++j) p.out[row * p.o_row + head * p.o_head + lane * E + j] = (uint16_t)bf_pack(acc[j] * inv, 0.f);
    } else if (avg) {                    // a block that joins its parts in shared memory
#pragma unroll
      for (int j = 0; j < E; ++j) avg[(i - i0) * pitch + lane * E + j] = acc[j] * inv;
      if (lane == 0) avg_lse[i - i0] = l == 0.f ? -INFINITY : m + log2f(l);
    } else {
      const int64_t unit = ((int64_t)part * p.b.rows + row) * p.q_heads + head;
#pragma unroll
      for (int j = 0; j < E; ++j) p.part_o[unit * D + lane * E + j] = acc[j] * inv;
      if (lane == 0) p.part_lse[unit] = l == 0.f ? -INFINITY : m + log2f(l);
    }
  }
}

// Four neighbouring elements of a row of an item, weighed over its parts' blocks, which are a cluster: each holds its
// averages at shared address `at` of the element and its log-sum of the row at `at_lse`.
constexpr int kMostCluster = 8;
__device__ __forceinline__ void join4(uint32_t at, uint32_t at_lse, int parts, float* x) {
  float lse[kMostCluster], top = -INFINITY;
  float4 y[kMostCluster];
#pragma unroll
  for (int i = 0; i < kMostCluster; ++i) {
    lse[i] = -INFINITY;
    if (i < parts) {
      lse[i] = ptx::ld_cluster(ptx::mapa(at_lse, i));
      y[i] = ptx::ld_cluster_v4(ptx::mapa(at, i));
    }
    top = fmaxf(top, lse[i]);
  }
  float sum = 0.f;
  x[0] = x[1] = x[2] = x[3] = 0.f;
#pragma unroll
  for (int i = 0; i < kMostCluster; ++i)
    if (i < parts) {
      const float w = lse[i] == -INFINITY ? 0.f : ex2(lse[i] - top);
      sum += w;
      x[0] += w * y[i].x; x[1] += w * y[i].y; x[2] += w * y[i].z; x[3] += w * y[i].w;
    }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
  for (int j = 0; j < 4; ++j) x[j] *= inv;
}

}  // namespace cache
}  // namespace cp
