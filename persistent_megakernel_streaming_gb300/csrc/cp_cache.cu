// cp_cache.cu -- the paged K/V cache: its C ABI (checks and launches), the
// append kernel (QK-norm, RoPE, quantisation, write) and the read-back kernel.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <initializer_list>
#include <new>

#include "cp.h"
#include "cp_cache.cuh"
#include "cp_cache_ptx.cuh"
#include "cp_call.h"

using namespace cp;
using namespace cp::cache;

struct cp_cache {
  int device = 0;
  cp_cache_desc d{};
  CacheView view{};
  CacheMaps maps{};
};

namespace {

constexpr int kAppendThreads = 128;
constexpr int kReadThreads = 128;
constexpr int kMaxRowsPerBlock = 4;    // one warp finds one row's sequence

// ------------------------------------------------------------------ rows
// Where a row goes: its sequence's table entry resolved to byte offsets.
struct Slot {
  int64_t at;        // byte offset of head 0 in K and V, -1: the row is skipped
  int64_t scale;     // the same in the scales
  int pos;
  int row;
};

// One warp finds row r's sequence (the count of sequences that end at or
// before it: lanes test 32 starts at a time, so a batch of 64 costs two loads)
// and its place. The last lane-0 write is the block's; callers synchronise.
__device__ __forceinline__ void find_slot(const CacheView& c, const BatchView& b, int r, Slot* out) {
  const int lane = threadIdx.x & 31;
  int seq = 0;
#pragma unroll 8
  for (int i0 = 0; i0 < b.n; i0 += 32) {
    const int i = i0 + lane;
    const bool before = i < b.n && b.start[min(i, b.n - 1) + 1] <= r;
    seq += __popc(__ballot_sync(0xffffffffu, before));
  }
  if (lane) return;
  Slot s;
  s.at = s.scale = -1;
  s.row = r;
  s.pos = 0;
  if (r < b.rows && seq < b.n) {
    const Seq q = seq_of(b, seq, c.status);
    if (r >= q.row0 && r < q.row0 + q.n) {
      s.pos = q.first + (r - q.row0);
      const int page = page_of(b.table + (int64_t)seq * b.table_stride, b.width, c.pages, c.page_shift, s.pos);
      if (page >= 0) {
        s.at = slot_bytes(c, page, 0, s.pos);
        s.scale = slot_scale(c, page, 0, s.pos);
      } else {
        set_status(c.status, CP_ERR_DEVICE_BOUNDS);
        s.pos = max(s.pos, 0);
      }
    } else {
      s.row = -1;
    }
  } else {
    s.row = -1;
  }
  *out = s;
}

// ------------------------------------------------------------------ append
__device__ __forceinline__ uint32_t e4m3x4(const float* x, float f) {
  uint16_t a, b;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(a) : "f"(x[1] * f), "f"(x[0] * f));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(b) : "f"(x[3] * f), "f"(x[2] * f));
  return a | (uint32_t)b << 16;
}

// Bits of 1.9375 * 2^127: from here on the nearest e4m3 step is 2^128, past fp32 and bf16.
constexpr int kRoundsPast = 0x7f780000;

struct AppendParams {
  CacheView c;
  BatchView b;
  const uint16_t* qkv;
  uint16_t* q_out;
  const uint16_t* q_norm;
  const uint16_t* k_norm;
  int64_t qkv_row, q_row;
  int q_heads;
  int rope;
  float eps;
  int rows_per_block;
  uint64_t turn[64];   // base^(-2j/D) / (2 pi) as a 64-bit fraction of a turn
};

// A row is heads of D elements, D/8 lanes a head: a lane has elements 4l .. 4l+3
// and their rotation partners D/2 further, so that RoPE needs no other lane,
// and the norm's sum and the absolute maximum are shuffles over the head's
// lanes. The rotary angle is kept in turns as a 64-bit fraction, position *
// turn[j] modulo 2^64, which wraps exactly: far positions lose nothing, and no
// 64-bit float is needed. Each row's D/2 sines and cosines are made once; a
// group of lanes stays with its row, keeps its four of them in registers, and
// takes every n-th head, four loads in flight.
// One read of qkv, one write of q and of the pages; arithmetic in pairs of fp32
// (an element that lies within that arithmetic's error, some 2^-22, of the
// middle between two e4m3 steps may take the other one: 4 in a million do).
// Measured: 8191 rows of 16/8 heads of 128 into bf16 pages 31 us a call, 4.3
// TB/s (63 % of the copy rate: the last round of blocks is short of loads.
// Blocks of 256 threads and 8 rows 33 us, of 512 36, of 64 and 2 rows 31; 2 or
// 8 loads in flight and more resident blocks at fewer registers 1 to 25 %
// slower; the first loads ahead of the look-up no faster); e4m3 pages, 16/16
// heads, 9018 rows 45 us in a replayed graph, issue slots 65 % busy, 73 a call
// with the read-back behind it.
template <int D, bool E4M3>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int kLanes = D / 8;
  constexpr int kGroups = kAppendThreads / kLanes;
  __shared__ Slot slots[kMaxRowsPerBlock];
  __shared__ float2 cs[kMaxRowsPerBlock][4][kLanes];          // [row][element of a lane][lane]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nrow = p.rows_per_block;                          // a power of two
  if (warp < nrow) find_slot(p.c, p.b, blockIdx.x * nrow + warp, &slots[warp]);
  __syncthreads();
  if (p.rope) {
    for (int i = threadIdx.x; i < nrow * (D / 2); i += kAppendThreads) {
      const int t = i / (D / 2), j = i % (D / 2);
      const int64_t frac = (int64_t)((uint64_t)slots[t].pos * p.turn[j]);   // turns in [-1/2, 1/2) * 2^64
      float sn, co;
      sincospif((float)frac * 0x1p-63f, &sn, &co);
      cs[t][j % 4][j / 4] = make_float2(co, sn);
    }
    __syncthreads();
  }
  const int heads = p.q_heads + 2 * p.c.heads;
  const int l = lane % kLanes;
  const int group = threadIdx.x / kLanes;
  const int t = group & (nrow - 1), first = group / nrow, step = kGroups / nrow;
  const Slot s = slots[t];
  float2 turn[4];
  if (p.rope) {
#pragma unroll
    for (int i = 0; i < 4; ++i) turn[i] = cs[t][i][l];
  }
  uint2 gains[2][2];                       // q's and k's, of the lane's lower and upper elements
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint16_t* g = i ? p.k_norm : p.q_norm;
    if (!g) continue;
    gains[i][0] = *reinterpret_cast<const uint2*>(g + l * 4);
    gains[i][1] = *reinterpret_cast<const uint2*>(g + D / 2 + l * 4);
  }
  const uint16_t* src = p.qkv + (int64_t)s.row * p.qkv_row + l * 4;
  constexpr int U = 4;
  // shuffles are the whole warp's, so every group goes through the same rounds
  for (int h0 = 0; h0 < heads; h0 += U * step) {
    uint2 lo[U], hi[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int h = h0 + k * step + first;
      lo[k] = hi[k] = make_uint2(0, 0);
      if (h < heads && s.row >= 0) {
        lo[k] = *reinterpret_cast<const uint2*>(src + (int64_t)h * D);
        hi[k] = *reinterpret_cast<const uint2*>(src + (int64_t)h * D + D / 2);
      }
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int h = h0 + k * step + first;
      if (h0 + k * step >= heads) break;                      // for the whole block
      const bool on = h < heads && s.row >= 0;
      const bool is_q = h < p.q_heads, is_v = h >= p.q_heads + p.c.heads;
      // pairs of elements: the lower two pairs and their partners
      uint64_t xx[2] = {ptx::pair_of(bf_lo(lo[k].x), bf_hi(lo[k].x)), ptx::pair_of(bf_lo(lo[k].y), bf_hi(lo[k].y))};
      uint64_t yy[2] = {ptx::pair_of(bf_lo(hi[k].x), bf_hi(hi[k].x)), ptx::pair_of(bf_lo(hi[k].y), bf_hi(hi[k].y))};
      const bool normed = is_q ? p.q_norm != nullptr : !is_v && p.k_norm;
      if (__any_sync(0xffffffffu, normed)) {
        const uint64_t sq = ptx::fma2(xx[0], xx[0], ptx::fma2(xx[1], xx[1], ptx::fma2(yy[0], yy[0], ptx::mul2(yy[1], yy[1]))));
        float a, b;
        ptx::split_pair(sq, &a, &b);
        float ss = a + b;
#pragma unroll
        for (int o = kLanes / 2; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (normed) {
          const float r = rsqrtf(ss * (1.f / D) + p.eps);
          const uint64_t rr = ptx::pair_of(r, r);
          const uint2 g = is_q ? gains[0][0] : gains[1][0], f = is_q ? gains[0][1] : gains[1][1];
          xx[0] = ptx::mul2(ptx::mul2(xx[0], rr), ptx::pair_of(bf_lo(g.x), bf_hi(g.x)));
          xx[1] = ptx::mul2(ptx::mul2(xx[1], rr), ptx::pair_of(bf_lo(g.y), bf_hi(g.y)));
          yy[0] = ptx::mul2(ptx::mul2(yy[0], rr), ptx::pair_of(bf_lo(f.x), bf_hi(f.x)));
          yy[1] = ptx::mul2(ptx::mul2(yy[1], rr), ptx::pair_of(bf_lo(f.y), bf_hi(f.y)));
        }
      }
      if (p.rope && !is_v) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint64_t c = ptx::pair_of(turn[2 * i].x, turn[2 * i + 1].x), n = ptx::pair_of(turn[2 * i].y, turn[2 * i + 1].y);
          const uint64_t a = xx[i], m = ptx::pair_of(-turn[2 * i].y, -turn[2 * i + 1].y);
          xx[i] = ptx::fma2(yy[i], m, ptx::mul2(a, c));
          yy[i] = ptx::fma2(a, n, ptx::mul2(yy[i], c));
        }
      }
      float x[4], y[4];
      ptx::split_pair(xx[0], x, x + 1);
      ptx::split_pair(xx[1], x + 2, x + 3);
      ptx::split_pair(yy[0], y, y + 1);
      ptx::split_pair(yy[1], y + 2, y + 3);
      const int kv = is_v ? h - p.q_heads - p.c.heads : h - p.q_heads;
      uint8_t* const pages = is_v ? p.c.v : p.c.k;
      if (!E4M3 || is_q) {
        const uint2 w = make_uint2(bf_pack(x[0], x[1]), bf_pack(x[2], x[3]));
        const uint2 z = make_uint2(bf_pack(y[0], y[1]), bf_pack(y[2], y[3]));
        if (on && (is_q || s.at >= 0)) {
          uint16_t* dst = is_q ? p.q_out + (int64_t)s.row * p.q_row + (int64_t)h * D
                               : reinterpret_cast<uint16_t*>(pages + s.at + kv * p.c.head_b);
          *reinterpret_cast<uint2*>(dst + l * 4) = w;
          *reinterpret_cast<uint2*>(dst + l * 4 + D / 2) = z;
        }
      }
      if (E4M3 && __any_sync(0xffffffffu, !is_q)) {
        // the least e with max <= 448 * 2^e = 1.75 * 2^(e+8), from the maximum's bits: exact
        int top = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          top = max(top, max(__float_as_int(x[i]) & 0x7fffffff, __float_as_int(y[i]) & 0x7fffffff));
        if (top >= kRoundsPast) {
          // infinities are kept as NaN, and set no scale; what would round to 2^128 is kept as the step below
          top = 0;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float& z = i < 4 ? x[i] : y[i - 4];
            const bool no = (__float_as_int(z) & 0x7fffffff) >= 0x7f800000;
            z = no ? __int_as_float(0x7fc00000) : fminf(fmaxf(z, -0x1.ep127f), 0x1.ep127f);
            top = max(top, no ? 0 : __float_as_int(z) & 0x7fffffff);
          }
        }
#pragma unroll
        for (int o = kLanes / 2; o; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        int e = (top >> 23) - 127 - 8 + ((top & 0x7fffff) > 0x600000 ? 1 : 0);
        e = max(e, kMinExp);
        const float inv = pow2i(-e);
        if (on && !is_q && s.at >= 0) {
          uint8_t* dst = pages + s.at + kv * p.c.head_b + l * 4;
          *reinterpret_cast<uint32_t*>(dst) = e4m3x4(x, inv);
          *reinterpret_cast<uint32_t*>(dst + D / 2) = e4m3x4(y, inv);
          if (l == 0) (is_v ? p.c.vs : p.c.ks)[s.scale + kv * p.c.sc_head] = (uint8_t)(e + 127);
        }
      }
    }
  }
}

// ------------------------------------------------------------------ read back
struct ReadParams {
  CacheView c;
  BatchView b;
  uint16_t* k_out;
  uint16_t* v_out;
  int rows_per_block;
};

// 16 cached bytes a lane: 8 bf16 copied, or 16 e4m3 widened to fp32, scaled by
// the power of two and packed (exact: 4 significant bits). Bound by HBM: 12
// sequences, 96000 rows of 8 heads of 128, e4m3: 95 us, 6.2 TB/s, 92 % of the
// copy rate.
template <int D, bool E4M3>
__global__ void __launch_bounds__(kReadThreads) read_kernel(const __grid_constant__ ReadParams p) {
  constexpr int kElems = E4M3 ? 16 : 8;
  constexpr int kLanes = D / kElems;
  __shared__ Slot slots[kMaxRowsPerBlock];
  const int warp = threadIdx.x >> 5;
  const int nrow = p.rows_per_block;
  if (warp < nrow) find_slot(p.c, p.b, blockIdx.x * nrow + warp, &slots[warp]);
  __syncthreads();
  const int units = nrow * p.c.heads * 2 * kLanes;
#pragma unroll 4
  for (int u = threadIdx.x; u < units; u += kReadThreads) {
    const int l = u % kLanes, rest = u / kLanes;
    const int t = rest % nrow, hv = rest / nrow;       // rows of one head lie side by side in a page
    const int h = hv >> 1, is_v = hv & 1;
    const Slot s = slots[t];
    uint16_t* out = is_v ? p.v_out : p.k_out;
    if (s.at < 0 || !out) continue;
    const uint4 raw = *reinterpret_cast<const uint4*>((is_v ? p.c.v : p.c.k) + s.at + h * p.c.head_b + l * 16);
    uint4* dst = reinterpret_cast<uint4*>(out + ((int64_t)s.row * p.c.heads + h) * D + l * kElems);
    if (!E4M3) {
      dst[0] = raw;
    } else {
      const float sc = pow2i((int)(is_v ? p.c.vs : p.c.ks)[s.scale + h * p.c.sc_head] - 127);
      float f[16];
      e4m3x4_f32(raw.x, f); e4m3x4_f32(raw.y, f + 4); e4m3x4_f32(raw.z, f + 8); e4m3x4_f32(raw.w, f + 12);
      uint32_t w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = bf_pack(f[2 * i] * sc, f[2 * i + 1] * sc);
      dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
      dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
  }
}

// ------------------------------------------------------------------ copies of pages
struct CopyParams {
  CacheView c;
  const int32_t* moves;
  const int32_t* count;
  int capacity;
  int lane_shift;      // 16-byte units a position: a power of two
  int units;           // of a page, keys and values
  int pieces;          // blocks' shares of a page
  int scale_vec;       // positions' scales lie side by side, on 16-byte boundaries
};
constexpr int kCopyThreads = 256, kCopyUnits = 4 * kCopyThreads;

// A block takes pieces of 16 KB: four 16-byte loads a thread in flight, then the stores. Both leave L2 first, so that the
// tables and counts of the calls around this one stay there (200 sequences branched in two, e4m3: 28 -> 25 us for the
// four calls). Bound by HBM: 3940 pages of 262 KB 158 us, 6.5 TB/s.
__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const __grid_constant__ CopyParams p) {
  ptx::pdl_trigger();
  ptx::pdl_wait();
  int n = *p.count;
  if (n > p.capacity) {
    n = p.capacity;
    if (threadIdx.x == 0) set_status(p.c.status, CP_ERR_DEVICE_BOUNDS);
  }
  const int place_shift = p.lane_shift + p.c.page_shift, half = p.units >> 1;
  for (int64_t piece = blockIdx.x; piece < (int64_t)n * p.pieces; piece += gridDim.x) {
    const int move = (int)(piece / p.pieces), part = (int)(piece - (int64_t)move * p.pieces);
    const int from = p.moves[2 * (int64_t)move], to = p.moves[2 * (int64_t)move + 1];
    if ((uint32_t)from >= (uint32_t)p.c.pages || (uint32_t)to >= (uint32_t)p.c.pages) {
      if (threadIdx.x == 0) set_status(p.c.status, CP_ERR_DEVICE_BOUNDS);
      continue;
    }
    if (from == to) continue;
    const int64_t there = (int64_t)(to - from) * p.c.page_b;
    uint4 x[4];
    uint8_t* at[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int u = part * kCopyUnits + k * kCopyThreads + threadIdx.x;
      const int is_v = u >= half, w = is_v ? u - half : u;
      const int head = w >> place_shift, place = (w >> p.lane_shift) & ((1 << p.c.page_shift) - 1), l = w & ((1 << p.lane_shift) - 1);
      at[k] = u < p.units ? (is_v ? p.c.v : p.c.k) + (int64_t)from * p.c.page_b + head * p.c.head_b + place * p.c.tok_b + l * 16 : nullptr;
      if (at[k]) x[k] = __ldcs(reinterpret_cast<const uint4*>(at[k]));
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (at[k]) __stcs(reinterpret_cast<uint4*>(at[k] + there), x[k]);
    if (!p.c.ks || part) continue;
    // the page's scales: the first block's
    const int scales = p.c.heads << p.c.page_shift;
    const int64_t s_from = (int64_t)from * p.c.sc_page, s_there = (int64_t)(to - from) * p.c.sc_page;
    const int step = p.scale_vec ? 16 : 1;
    for (int i = threadIdx.x * step; i < 2 * scales; i += kCopyThreads * step) {
      const int is_v = i >= scales, w = is_v ? i - scales : i;
      const int head = w >> p.c.page_shift, place = w & ((1 << p.c.page_shift) - 1);
      uint8_t* a = (is_v ? p.c.vs : p.c.ks) + s_from + head * p.c.sc_head + place * p.c.sc_tok;
      if (p.scale_vec) *reinterpret_cast<uint4*>(a + s_there) = *reinterpret_cast<const uint4*>(a);
      else a[s_there] = *a;
    }
  }
}

// ------------------------------------------------------------------ checks
int check_desc(const cp_cache_desc* in, cp_cache_desc* d) {
  if (!in || !in->k || !in->v) return CP_ERR_INVALID_ARG;
  *d = *in;
  if (d->dtype != CP_CACHE_BF16 && d->dtype != CP_CACHE_E4M3) return CP_ERR_INVALID_ARG;
  if (d->kv_heads < 1 || d->head_dim < 1 || d->page_size < 1 || d->pages < 1) return CP_ERR_INVALID_ARG;
  if (d->head_dim != 64 && d->head_dim != 128) return CP_ERR_UNSUPPORTED;
  if (d->page_size != 16 && d->page_size != 32 && d->page_size != 64 && d->page_size != 128) return CP_ERR_UNSUPPORTED;
  if (d->kv_heads > 128) return CP_ERR_UNSUPPORTED;
  const bool e4m3 = d->dtype == CP_CACHE_E4M3;
  if (e4m3 ? (!d->k_scale || !d->v_scale) : (d->k_scale || d->v_scale)) return CP_ERR_INVALID_ARG;
  if (!d->token_stride) d->token_stride = d->head_dim;
  if (!d->head_stride) d->head_stride = (int64_t)d->page_size * d->head_dim;
  if (!d->page_stride) d->page_stride = (int64_t)d->kv_heads * d->page_size * d->head_dim;
  if (!d->scale_token_stride) d->scale_token_stride = 1;
  if (!d->scale_head_stride) d->scale_head_stride = d->page_size;
  if (!d->scale_page_stride) d->scale_page_stride = (int64_t)d->kv_heads * d->page_size;
  if (d->timeout_ns < 0) return CP_ERR_INVALID_ARG;
  if (!d->timeout_ns) d->timeout_ns = 2000000000ll;
  if (d->token_stride < 0 || d->head_stride < 0 || d->page_stride < 0 || d->scale_token_stride < 0 ||
      d->scale_head_stride < 0 || d->scale_page_stride < 0)
    return CP_ERR_INVALID_ARG;
  const int per16 = e4m3 ? 16 : 8;
  if (d->token_stride % per16 || d->head_stride % per16 || d->page_stride % per16 || !aligned16(d->k) || !aligned16(d->v))
    return CP_ERR_UNSUPPORTED;
  const int64_t most = ((int64_t)1 << 40) / (e4m3 ? 1 : 2);    // what a tensor map's strides reach
  if (d->token_stride >= most || d->head_stride >= most || d->page_stride >= most) return CP_ERR_UNSUPPORTED;
  if (!lie_apart(d->head_dim, {{d->page_size, d->token_stride}, {d->kv_heads, d->head_stride}, {d->pages, d->page_stride}}))
    return CP_ERR_INVALID_ARG;
  if (e4m3 && !lie_apart(1, {{d->page_size, d->scale_token_stride}, {d->kv_heads, d->scale_head_stride}, {d->pages, d->scale_page_stride}}))
    return CP_ERR_INVALID_ARG;
  return CP_OK;
}

// The tensor map of K or V: 64 bf16 columns a box in the 128-byte swizzle that
// the tensor core reads, or whole e4m3 rows as they lie; a page high.
int make_map(const cp_cache_desc& d, void* base, CUtensorMap* map) {
  void* fn = nullptr;
  cudaDriverEntryPointQueryResult found;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found) != cudaSuccess ||
      found != cudaDriverEntryPointSuccess)
    return CP_ERR_CUDA;
  const bool e4m3 = d.dtype == CP_CACHE_E4M3;
  const cuuint64_t es = e4m3 ? 1 : 2;
  const cuuint64_t dims[4] = {(cuuint64_t)d.head_dim, (cuuint64_t)d.page_size, (cuuint64_t)d.kv_heads, (cuuint64_t)d.pages};
  const cuuint64_t strides[3] = {(cuuint64_t)d.token_stride * es, (cuuint64_t)d.head_stride * es, (cuuint64_t)d.page_stride * es};
  const cuuint32_t box[4] = {(cuuint32_t)(e4m3 ? d.head_dim : 64), (cuuint32_t)d.page_size, 1, 1};
  const cuuint32_t steps[4] = {1, 1, 1, 1};
  const CUresult r = in_context([&] {
    return reinterpret_cast<decltype(&cuTensorMapEncodeTiled)>(fn)(
        map, e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, base, dims, strides, box, steps,
        CU_TENSOR_MAP_INTERLEAVE_NONE, e4m3 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  });
  return r == CUDA_SUCCESS ? CP_OK : CP_ERR_UNSUPPORTED;
}

CacheView view_of(const cp_cache_desc& d, int32_t* status) {
  const int64_t es = d.dtype == CP_CACHE_E4M3 ? 1 : 2;
  CacheView v{};
  v.k = static_cast<uint8_t*>(d.k);
  v.v = static_cast<uint8_t*>(d.v);
  v.ks = d.k_scale;
  v.vs = d.v_scale;
  v.page_b = d.page_stride * es;
  v.head_b = d.head_stride * es;
  v.tok_b = d.token_stride * es;
  v.sc_page = d.scale_page_stride;
  v.sc_head = d.scale_head_stride;
  v.sc_tok = d.scale_token_stride;
  v.pages = d.pages;
  v.heads = d.kv_heads;
  v.page_shift = d.page_size == 16 ? 4 : d.page_size == 32 ? 5 : d.page_size == 64 ? 6 : 7;
  v.status = status;
  return v;
}

int check_batch(const cp_cache_desc& d, const cp_batch* in, BatchView* b) {
  if (!in || !in->start || !in->length || !in->page_table) return CP_ERR_INVALID_ARG;
  if (in->sequences < 1 || in->sequences > 65535 || in->rows < 1 || in->table_width < 1) return CP_ERR_INVALID_ARG;
  if (in->max_new < 0 || in->max_length < 0 || in->table_stride < 0) return CP_ERR_INVALID_ARG;
  const int64_t held = (int64_t)in->table_width * d.page_size;
  if (in->max_length > held) return CP_ERR_INVALID_ARG;
  if (in->table_stride && in->sequences > 1 && in->table_stride < in->table_width) return CP_ERR_INVALID_ARG;
  b->start = in->start;
  b->length = in->length;
  b->table = in->page_table;
  b->table_stride = in->table_stride ? in->table_stride : in->table_width;
  b->n = in->sequences;
  b->rows = in->rows;
  b->width = in->table_width;
  b->max_new = in->max_new ? std::min(in->max_new, in->rows) : in->rows;
  // positions are 32-bit, with room for a tile past the last
  b->max_len = in->max_length ? in->max_length : (int)std::min<int64_t>(held, INT32_MAX - 1024);
  if (b->max_len > INT32_MAX - 1024) return CP_ERR_UNSUPPORTED;
  return CP_OK;
}

int check_append(const cp_cache_desc& d, const BatchView& b, const cp_append* a, AppendParams* p) {
  if (!a || !a->qkv || a->q_heads < 0) return CP_ERR_INVALID_ARG;
  if (a->q_heads > 1024) return CP_ERR_UNSUPPORTED;
  if ((a->q_heads > 0) != (a->q_out != nullptr)) return CP_ERR_INVALID_ARG;
  if (!(a->rms_eps >= 0.f) || !std::isfinite(a->rms_eps) || !(a->rope_base >= 0.f) || !std::isfinite(a->rope_base))
    return CP_ERR_INVALID_ARG;
  const int64_t wide = (int64_t)(a->q_heads + 2 * d.kv_heads) * d.head_dim, qw = (int64_t)a->q_heads * d.head_dim;
  p->qkv_row = a->qkv_stride ? a->qkv_stride : wide;
  p->q_row = a->q_stride ? a->q_stride : qw;
  if (p->qkv_row < wide || p->q_row < qw) return CP_ERR_INVALID_ARG;
  if (p->qkv_row % 8 || p->q_row % 8 || !aligned16(a->qkv) || !aligned16(a->q_out) || !aligned16(a->q_norm) ||
      !aligned16(a->k_norm))
    return CP_ERR_UNSUPPORTED;
  p->b = b;
  p->qkv = static_cast<const uint16_t*>(a->qkv);
  p->q_out = static_cast<uint16_t*>(a->q_out);
  p->q_norm = static_cast<const uint16_t*>(a->q_norm);
  p->k_norm = static_cast<const uint16_t*>(a->k_norm);
  p->q_heads = a->q_heads;
  p->eps = a->rms_eps;
  p->rope = a->rope_base > 0.f;
  if (p->rope) {
    // turns per position modulo one: 52 bits of them, position 2^31 is still good to 2^-24 turns. A power for j is that
    // of its multiple of 8 times that of the rest: 16 calls of pow, not 64, in each call
    double coarse[8], fine[8];
    for (int i = 0; i < 8; ++i) {
      coarse[i] = std::pow((double)a->rope_base, -16.0 * i / d.head_dim) / 6.283185307179586;
      fine[i] = std::pow((double)a->rope_base, -2.0 * i / d.head_dim);
    }
    for (int j = 0; j < d.head_dim / 2; ++j) {
      const double turns = coarse[j / 8] * fine[j % 8];
      p->turn[j] = (uint64_t)std::ldexp(turns - std::floor(turns), 64);
    }
  }
  return CP_OK;
}

int check_attend(const cp_cache_desc& d, const BatchView& b, const cp_attend* a, AttendParams* p) {
  if (!a || !a->q || !a->out || a->q_heads < 1 || a->window < 0) return CP_ERR_INVALID_ARG;
  if (a->q_heads % d.kv_heads) return CP_ERR_INVALID_ARG;
  if (a->q_heads / d.kv_heads > 64) return CP_ERR_UNSUPPORTED;
  if ((int64_t)b.rows * (a->q_heads / d.kv_heads) >= (1 << 30)) return CP_ERR_UNSUPPORTED;   // rows are counted in 32 bits
  if (!(a->scale >= 0.f) || !std::isfinite(a->scale)) return CP_ERR_INVALID_ARG;
  p->q_head = a->q_head_stride ? a->q_head_stride : d.head_dim;
  p->o_head = a->out_head_stride ? a->out_head_stride : d.head_dim;
  p->q_row = a->q_stride ? a->q_stride : (int64_t)a->q_heads * d.head_dim;
  p->o_row = a->out_stride ? a->out_stride : (int64_t)a->q_heads * d.head_dim;
  if (p->q_head < 0 || p->o_head < 0 || p->q_row < 0 || p->o_row < 0) return CP_ERR_INVALID_ARG;
  if (p->q_head % 8 || p->o_head % 8 || p->q_row % 8 || p->o_row % 8 || !aligned16(a->q) || !aligned16(a->out))
    return CP_ERR_UNSUPPORTED;
  if (!lie_apart(d.head_dim, {{b.rows, p->o_row}, {a->q_heads, p->o_head}})) return CP_ERR_INVALID_ARG;
  p->b = b;
  p->q = static_cast<const uint16_t*>(a->q);
  p->out = static_cast<uint16_t*>(a->out);
  p->q_heads = a->q_heads;
  p->group = a->q_heads / d.kv_heads;
  p->magic = (65535u + p->group) / p->group;
  const double scale = a->scale > 0.f ? (double)a->scale : 1.0 / std::sqrt((double)d.head_dim);
  p->scale_log2 = (float)(scale * 1.4426950408889634);
  if (!std::isfinite(p->scale_log2)) return CP_ERR_INVALID_ARG;
  p->causal = a->causal != 0;
  p->window = a->window;
  p->timeout_ns = d.timeout_ns;
  p->stall = d.debug_stall != 0;
  p->a = plan_attend(b, d.kv_heads, a->q_heads, d.head_dim, d.dtype == CP_CACHE_E4M3, p->causal != 0, p->window);
  return CP_OK;
}

// Rows per block, a power of two: one until every SM has two blocks, then up to four, which share the look-ups.
int rows_per_block(int rows) {
  int n = 1;
  while (n < kMaxRowsPerBlock && rows >= 304 * 2 * n) n *= 2;
  return n;
}

}  // namespace

extern "C" {

int cp_cache_check(const cp_cache_desc* desc, const cp_batch* batch, const cp_append* append, const cp_attend* attend,
                   size_t* workspace_bytes) {
  if (workspace_bytes) *workspace_bytes = 0;
  cp_cache_desc d;
  int st = check_desc(desc, &d);
  if (st) return st;
  if (!batch) return append || attend ? CP_ERR_INVALID_ARG : CP_OK;
  BatchView b{};
  if ((st = check_batch(d, batch, &b))) return st;
  AppendParams ap{};
  if (append && (st = check_append(d, b, append, &ap))) return st;
  AttendParams at{};
  if (attend) {
    if ((st = check_attend(d, b, attend, &at))) return st;
    if (workspace_bytes) *workspace_bytes = attend_workspace(at.a, b, at.q_heads, d.head_dim);
  }
  return CP_OK;
}

int cp_cache_create(const cp_cache_desc* desc, int device, cp_cache** out) {
  if (!out) return CP_ERR_INVALID_ARG;
  *out = nullptr;
  cp_cache_desc d;
  const int st = check_desc(desc, &d);
  if (st) return st;
  const int dev = check_device(device);
  if (dev) return dev;
  DeviceGuard guard(device);
  for (const void* ptr : {(const void*)d.k, (const void*)d.v, (const void*)d.k_scale, (const void*)d.v_scale})
    if (ptr && !on_device(ptr, device)) return CP_ERR_INVALID_ARG;
  cp_cache* c = new (std::nothrow) cp_cache();
  if (!c) return CP_ERR_NOMEM;
  c->device = device;
  c->d = d;
  int mapped = make_map(d, d.k, &c->maps.k);
  if (!mapped) mapped = make_map(d, d.v, &c->maps.v);
  if (mapped) {
    delete c;
    return mapped;
  }
  void* status = nullptr;
  if (cudaMalloc(&status, 16) != cudaSuccess) {
    delete c;
    return CP_ERR_NOMEM;
  }
  c->view = view_of(d, static_cast<int32_t*>(status));
  if (prepare_attend() != cudaSuccess || cudaMemset(status, 0, 16) != cudaSuccess || cudaDeviceSynchronize() != cudaSuccess) {
    cp_cache_destroy(c);
    return CP_ERR_CUDA;
  }
  *out = c;
  return CP_OK;
}

void cp_cache_destroy(cp_cache* c) {
  if (!c) return;
  {
    DeviceGuard g(c->device);
    cudaDeviceSynchronize();
    cudaFree(c->view.status);
  }
  delete c;
}

int cp_cache_status(cp_cache* c) {
  if (!c) return CP_ERR_INVALID_ARG;
  DeviceGuard g(c->device);
  if (cudaDeviceSynchronize() != cudaSuccess) return CP_ERR_CUDA;
  int32_t v = 0;
  if (cudaMemcpy(&v, c->view.status, 4, cudaMemcpyDeviceToHost) != cudaSuccess) return CP_ERR_CUDA;
  return v;
}

int cp_cache_clear_status(cp_cache* c) {
  if (!c) return CP_ERR_INVALID_ARG;
  DeviceGuard g(c->device);
  if (cudaDeviceSynchronize() != cudaSuccess) return CP_ERR_CUDA;
  if (cudaMemset(c->view.status, 0, 16) != cudaSuccess) return CP_ERR_CUDA;
  return cuda_err(cudaDeviceSynchronize());
}

int cp_cache_append(cp_cache* c, const cp_batch* batch, const cp_append* args, cp_stream_t stream) {
  if (!c) return CP_ERR_INVALID_ARG;
  BatchView b{};
  AppendParams p{};
  int st = check_batch(c->d, batch, &b);
  if (!st) st = check_append(c->d, b, args, &p);
  if (st) return st;
  DeviceGuard g(c->device);
  p.c = c->view;
  p.rows_per_block = rows_per_block(b.rows);
  const int grid = (b.rows - 1) / p.rows_per_block + 1;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool e4m3 = c->d.dtype == CP_CACHE_E4M3;
  if (c->d.head_dim == 128) {
    if (e4m3) append_kernel<128, true><<<grid, kAppendThreads, 0, s>>>(p);
    else append_kernel<128, false><<<grid, kAppendThreads, 0, s>>>(p);
  } else {
    if (e4m3) append_kernel<64, true><<<grid, kAppendThreads, 0, s>>>(p);
    else append_kernel<64, false><<<grid, kAppendThreads, 0, s>>>(p);
  }
  return cuda_err(cudaGetLastError());
}

int cp_cache_read(cp_cache* c, const cp_batch* batch, void* k_out, void* v_out, cp_stream_t stream) {
  if (!c || (!k_out && !v_out)) return CP_ERR_INVALID_ARG;
  BatchView b{};
  const int st = check_batch(c->d, batch, &b);
  if (st) return st;
  if (!aligned16(k_out) || !aligned16(v_out)) return CP_ERR_UNSUPPORTED;
  DeviceGuard g(c->device);
  ReadParams p{};
  p.c = c->view;
  p.b = b;
  p.k_out = static_cast<uint16_t*>(k_out);
  p.v_out = static_cast<uint16_t*>(v_out);
  p.rows_per_block = rows_per_block(b.rows);
  const int grid = (b.rows - 1) / p.rows_per_block + 1;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool e4m3 = c->d.dtype == CP_CACHE_E4M3;
  if (c->d.head_dim == 128) {
    if (e4m3) read_kernel<128, true><<<grid, kReadThreads, 0, s>>>(p);
    else read_kernel<128, false><<<grid, kReadThreads, 0, s>>>(p);
  } else {
    if (e4m3) read_kernel<64, true><<<grid, kReadThreads, 0, s>>>(p);
    else read_kernel<64, false><<<grid, kReadThreads, 0, s>>>(p);
  }
  return cuda_err(cudaGetLastError());
}

int cp_cache_copy(cp_cache* c, const int32_t* moves, int capacity, const int32_t* count, cp_stream_t stream) {
  if (!c || !moves || !count || capacity < 1) return CP_ERR_INVALID_ARG;
  DeviceGuard g(c->device);
  CopyParams p{};
  p.c = c->view;
  p.moves = moves;
  p.count = count;
  p.capacity = capacity;
  const int unit = c->d.head_dim * (c->d.dtype == CP_CACHE_E4M3 ? 1 : 2) / 16;
  while (1 << p.lane_shift < unit) ++p.lane_shift;
  p.units = 2 * c->d.kv_heads * c->d.page_size * unit;
  p.pieces = (p.units - 1) / kCopyUnits + 1;
  const bool aligned = aligned16(p.c.ks) && aligned16(p.c.vs) && p.c.sc_head % 16 == 0 && p.c.sc_page % 16 == 0;
  p.scale_vec = p.c.sc_tok == 1 && aligned;
  const int64_t grid = std::min<int64_t>((int64_t)capacity * p.pieces, kSms * 8);
  return cuda_err(launch_as(copy_kernel, dim3((unsigned)grid), 1, 1, true, kCopyThreads, 0, reinterpret_cast<cudaStream_t>(stream), p));
}

int cp_cache_attend(cp_cache* c, const cp_batch* batch, const cp_attend* args, void* workspace, size_t workspace_bytes,
                    cp_stream_t stream) {
  if (!c) return CP_ERR_INVALID_ARG;
  BatchView b{};
  AttendParams p{};
  int st = check_batch(c->d, batch, &b);
  if (!st) st = check_attend(c->d, b, args, &p);
  if (st) return st;
  const size_t need = attend_workspace(p.a, b, p.q_heads, c->d.head_dim);
  if (need && (!workspace || workspace_bytes < need)) return CP_ERR_INVALID_ARG;
  if (!aligned16(workspace)) return CP_ERR_UNSUPPORTED;
  DeviceGuard g(c->device);
  p.c = c->view;
  const size_t units = (size_t)b.rows * p.q_heads * kept_parts(p.a);
  p.part_o = static_cast<float*>(workspace);
  p.part_lse = p.part_o + units * c->d.head_dim;
  p.coarser = reinterpret_cast<int*>(p.part_lse + units);
  return cuda_err(launch_attend(p, c->maps, c->d.head_dim, c->d.dtype == CP_CACHE_E4M3, reinterpret_cast<cudaStream_t>(stream)));
}

int64_t cp_test_slot(const cp_cache_desc* desc, const int32_t* table, int table_width, int pos, int head) {
  cp_cache_desc d;
  if (check_desc(desc, &d) || !table || head < 0 || head >= d.kv_heads) return -1;
  const CacheView v = view_of(d, nullptr);
  const int page = page_of(table, table_width, v.pages, v.page_shift, pos);
  return page < 0 ? -1 : slot_bytes(v, page, head, pos) / (d.dtype == CP_CACHE_E4M3 ? 1 : 2);
}

}  // extern "C"
