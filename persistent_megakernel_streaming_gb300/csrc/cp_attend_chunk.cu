// cp_attend_chunk.cu -- attention of many new rows of a sequence (a piece of a
// prompt, or all of it) over the paged cache, on tcgen05.
//
// The rows of one sequence and kv head are packed row by row, query head by
// query head (row i: new row i / group, head i % group), and cut into tiles of
// 128; a block takes two tiles, so that each key and value it brings in serves
// 256 rows, and the two keep the tensor core busy in turn: while one tile's
// softmax runs, the other's products do.
//
// Warps 0-3 and 4-7: the softmax of tile 0 and tile 1, a thread a row. Warp
// 12: one thread issues every MMA. Warp 13 brings pages in through tensor maps,
// a lane a page. For each 128 positions S = Q K^T (128 x 128, fp32 in TMEM);
// the softmax threads read their row of S twice (maximum, then weights: the
// row does not fit their registers), write the weights as 16 bit over the S
// they have read, and O += P V reads them from there. O stays in TMEM for the
// whole pass; its reference maximum is only moved, and O rescaled, when a
// row's maximum has risen by 2^kLazy over it, since the sum and the weights of
// a part share the reference.
//
// bf16 pages land in the ring as the tensor core reads them. Tiles at the ends
// of what the block's rows see, and tiles that only some of them see, pass
// warps 8-11 first: values that nobody sees are zeroed (a page may hold
// anything there), and values that some row must not see are looked over for
// infinities and NaN. e4m3 pages land in a ring of their own and all pass
// warps 8-11, which widen them to fp16 (exact) into the operand ring. Scales
// and the handling of fp16's range are the step kernel's.
#include "cp_attend.cuh"

namespace cp {
namespace cache {
namespace {

using namespace ptx;

constexpr int kTile = 128;             // rows of a tile, and positions of one
constexpr int kThreadsC = 448;
constexpr int kHelper0 = 8;            // first of four helper warps
constexpr int kHelpers = 128;
constexpr int kMmaWarp = 12, kLoadWarp = 13;
constexpr int kScaleSlots = 8;         // tiles whose scales are held: more than the ring's
constexpr long long kWaitNs = 2000000000ll;

// Loads are counted K of tile 0, V of tile 0, K of tile 1, ...; load n is in slot n % kOps.
template <int D, bool E4M3>
struct Cfg {
  static constexpr int kOpBytes = kTile * D * 2;        // one operand tile
  static constexpr int kSlab = kTile * 128;             // 64 columns of it
  static constexpr int kOps = D == 64 ? 8 : E4M3 ? 3 : 4;
  static constexpr int kRawBytes = E4M3 ? kTile * D : 0;
  static constexpr int kRaws = E4M3 ? (D == 64 ? 4 : 2) : kOps;   // bf16: the operand ring itself
  static constexpr int kSmem = (2 + kOps) * kOpBytes + (E4M3 ? kRaws : 0) * kRawBytes + 1024;
};
// TMEM columns: the two tiles' scores (and weights), then their outputs
constexpr uint32_t kTmemS = 0, kTmemO = 256, kTmemCols = 512;

struct ChunkShared {
  uint64_t raw_full[8], raw_empty[8], op_full[8], op_empty[8];
  uint64_t q_full, s_full[2], p_full[2], o_full;
  uint32_t tmem;
  int abort;       // a wait gave up
  int bad;         // a value that some row must not see is not finite
  alignas(16) float fk[kScaleSlots][kTile];
  alignas(16) float fv[kScaleSlots][kTile];
  int vref[kScaleSlots];
};

// Bounded: after kWaitNs, or once another wait of the block gave up, false.
__device__ __forceinline__ bool wait_bar(ChunkShared& sh, uint32_t bar, uint32_t parity) {
  if (mb_try(bar, parity)) return true;
  const uint64_t t0 = gtime();
  for (;;) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (mb_try(bar, parity)) return true;
    if (*(volatile int*)&sh.abort) return false;
    if ((long long)(gtime() - t0) > kWaitNs) {
      *(volatile int*)&sh.abort = 1;
      return false;
    }
  }
}

// The same for a whole warp that goes on together.
__device__ __forceinline__ bool wait_warp(ChunkShared& sh, uint32_t bar, uint32_t parity) {
  return __all_sync(0xffffffffu, wait_bar(sh, bar, parity));
}

__device__ __forceinline__ uint64_t pack2(const uint32_t* x) { return pair_of(__uint_as_float(x[0]), __uint_as_float(x[1])); }
__device__ __forceinline__ void unpack2(uint64_t y, uint32_t* x) {
  float a, b;
  split_pair(y, &a, &b);
  x[0] = __float_as_uint(a);
  x[1] = __float_as_uint(b);
}
// Byte offset of 16-byte unit u (8 elements) of row r in an operand tile.
__device__ __forceinline__ uint32_t op_at(int r, int u) {
  return (uint32_t)((u >> 3) * (kTile * 128) + r * 128 + (((u & 7) ^ (r & 7)) << 4));
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(kThreadsC, 1) attend_chunk_kernel(const __grid_constant__ AttendParams p,
                                                                    const __grid_constant__ CacheMaps maps) {
  using C = Cfg<D, E4M3>;
  constexpr int NO = C::kOps, NR = C::kRaws;
  extern __shared__ uint8_t raw[];
  __shared__ ChunkShared sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // which sequence and which of its tile pairs: every warp counts the pairs, 32 sequences at a time
  int seq = -1, pair = 0;
  {
    int before = 0;
    const int want = blockIdx.x / p.c.heads;
    for (int i0 = 0; i0 < p.b.n && seq < 0; i0 += 32) {
      int pairs = 0;
      if (i0 + lane < p.b.n) {
        const Seq s = seq_of(p.b, i0 + lane, p.c.status);
        const int rows = s.n * p.group;
        if (rows > kStepRows || !p.a.use_step) pairs = (rows + kPairRows - 1) / kPairRows;
      }
      int sum = pairs;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += up;
      }
      const uint32_t has = __ballot_sync(0xffffffffu, before + sum > want);
      if (has) {
        const int at = __ffs(has) - 1;
        seq = i0 + at;
        const int end = __shfl_sync(0xffffffffu, before + sum, at);
        pair = end - 1 - want;            // the later rows of a sequence see more: they start first
      }
      before += __shfl_sync(0xffffffffu, sum, 31);
    }
  }
  if (seq < 0) return;
  const int kv = blockIdx.x % p.c.heads, part = blockIdx.y;
  const Seq s = seq_of(p.b, seq, p.c.status);
  const int nrows = s.n * p.group;
  const int row0 = pair * kPairRows;
  const int rows_here = min(kPairRows, nrows - row0);
  auto pos_of = [&](int i) { return s.first + min(i, nrows - 1) / p.group; };
  const Range range = item_range(p, pos_of(row0), pos_of(row0 + rows_here - 1), s.len, kChunkAlign);
  const int parts = parts_of(range, p.a.chunk_chunk);
  if (part >= max(parts, 1)) return;
  const bool whole = parts <= 1;
  const int t_begin = range.base + part * p.a.chunk_chunk;
  const int t_end = min(t_begin + p.a.chunk_chunk, range.hi);
  const int ntiles = t_end > t_begin ? (t_end - t_begin + kTile - 1) / kTile : 0;
  // tiles that stream i (tile of rows i) takes part in, and the positions that all its rows see
  int jb[2], je[2], all_lo[2], all_hi[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int f = row0 + i * kTile;
    jb[i] = je[i] = 0;
    all_lo[i] = all_hi[i] = 0;
    if (f < nrows) {
      const int first = pos_of(f), last = pos_of(f + kTile - 1);
      const Range r = item_range(p, first, last, s.len, kChunkAlign);
      const int a = max(r.lo, t_begin), b = min(r.hi, t_end);
      if (b > a) {
        jb[i] = (a - t_begin) / kTile;
        je[i] = (b - t_begin + kTile - 1) / kTile;
      }
      int d;
      visible(p, last, s.len, &all_lo[i], &d);
      visible(p, first, s.len, &d, &all_hi[i]);
    }
  }

  uint8_t* ops = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  const uint32_t q_s = saddr(ops), op_s = q_s + 2 * C::kOpBytes, raw_s = E4M3 ? op_s + NO * C::kOpBytes : op_s;

  if (threadIdx.x == 0) {
    for (int i = 0; i < NR; ++i) {
      mb_init(saddr(&sh.raw_full[i]), 1);
      mb_init(saddr(&sh.raw_empty[i]), kHelpers / 32);
    }
    for (int i = 0; i < NO; ++i) {
      mb_init(saddr(&sh.op_full[i]), kHelpers);
      mb_init(saddr(&sh.op_empty[i]), 1);
    }
    mb_init(saddr(&sh.q_full), 256);
    for (int i = 0; i < 2; ++i) {
      mb_init(saddr(&sh.s_full[i]), 1);
      mb_init(saddr(&sh.p_full[i]), 128);
    }
    mb_init(saddr(&sh.o_full), 1);
    sh.abort = 0;
    sh.bad = 0;
    mb_fence_init();
  }
  if (warp == kMmaWarp) {
    tm_alloc(saddr(&sh.tmem), kTmemCols);
    tm_relinquish();
  }
  tm_fence_before();
  __syncthreads();
  tm_fence_after();
  const uint32_t tmem = sh.tmem;

  // a softmax thread's row
  const int i = warp >> 2;                               // stream (warps 0-7)
  const int my = row0 + i * kTile + (warp & 3) * 32 + lane;
  const bool mine = warp < kHelper0 && my < nrows;
  const int64_t out_row = s.row0 + (mine ? my / p.group : 0);
  const int head = kv * p.group + (mine ? my % p.group : 0);
  float l = 0.f, m = -INFINITY;
  int vr = 0;
  constexpr float kBias = E4M3 ? 8.f : 0.f;
  constexpr float kLazy = E4M3 ? 6.f : 8.f;              // weights reach 2^(kBias + kLazy): inside fp16

  if (warp < kHelper0) {
    // ---------------------------------------------------------------- softmax
    float rs = p.scale_log2;
    {
      const uint32_t dst = q_s + i * C::kOpBytes;
      const int r = (warp & 3) * 32 + lane;
      const uint16_t* qp = p.q + out_row * p.q_row + (int64_t)head * p.q_head;
      if (!E4M3) {
#pragma unroll
        for (int u = 0; u < D / 8; ++u) {
          const uint4 x = mine ? *reinterpret_cast<const uint4*>(qp + u * 8) : make_uint4(0, 0, 0, 0);
          st_shared_v4u(dst + op_at(r, u), x);
        }
      } else {
        uint4 x[D / 8];
        int top = 0;
#pragma unroll
        for (int u = 0; u < D / 8; ++u) {
          x[u] = mine ? *reinterpret_cast<const uint4*>(qp + u * 8) : make_uint4(0, 0, 0, 0);
          const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) top = max(top, max(finite_exp(w[k] & 0xffffu), finite_exp(w[k] >> 16)));
        }
        const int e = min(max(top - 127, -100), 100);
        const float inv = pow2i(-e);
        rs = pow2i(e);
#pragma unroll
        for (int u = 0; u < D / 8; ++u) {
          const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
          uint32_t y[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) y[k] = hf_pack(bf_lo(w[k]) * inv, bf_hi(w[k]) * inv);
          st_shared_v4u(dst + op_at(r, u), make_uint4(y[0], y[1], y[2], y[3]));
        }
      }
      fence_proxy_async_smem();
      mb_arrive(saddr(&sh.q_full));
    }
    int lo = 0, hi = 0;
    if (mine) visible(p, s.first + my / p.group, s.len, &lo, &hi);
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;
    const uint32_t s_t = tmem + lanes + kTmemS + i * kTile, o_t = tmem + lanes + kTmemO + i * D;
    const int j0 = i ? jb[1] : jb[0], j1 = i ? je[1] : je[0];
    const int see_lo = i ? all_lo[1] : all_lo[0], see_hi = i ? all_hi[1] : all_hi[0];
    const uint64_t rs2 = pair_of(rs, rs);
    uint64_t sum[2] = {0, 0};              // two pairs of partial sums
    for (int j = j0; j < j1; ++j) {
      const int n = j - j0;
      const int t0 = t_begin + j * kTile;
      if (!wait_warp(sh, saddr(&sh.s_full[i]), n & 1)) break;
      if (E4M3 && !wait_warp(sh, saddr(&sh.op_full[(2 * j + 1) % NO]), ((2 * j + 1) / NO) & 1)) break;   // its scales
      tm_fence_after();
      const float* fk = sh.fk[j % kScaleSlots];
      const float* fv = sh.fv[j % kScaleSlots];
      const int vn = E4M3 ? sh.vref[j % kScaleSlots] : 0;
      const bool edge = t0 < see_lo || t0 + kTile > see_hi;
      uint32_t x0[32], x1[32];
      // 32 scores in place, times their keys' scales, masked ones minus infinity
      auto ready = [&](uint32_t* x, int c) {
        if (E4M3) {
#pragma unroll
          for (int k = 0; k < 32; k += 4) {
            float4 f = *reinterpret_cast<const float4*>(fk + c + k);
            unpack2(mul2(pack2(x + k), pair_of(f.x, f.y)), x + k);
            unpack2(mul2(pack2(x + k + 2), pair_of(f.z, f.w)), x + k + 2);
          }
        }
        if (edge) {
#pragma unroll
          for (int k = 0; k < 32; ++k)
            if (t0 + c + k < lo || t0 + c + k >= hi) x[k] = 0xff800000u;
        }
      };
      auto top_of = [&](const uint32_t* x, float top) {
        float a = top, b = __uint_as_float(x[0]);
#pragma unroll
        for (int k = 1; k < 31; k += 2) {
          a = fmaxf(a, __uint_as_float(x[k]));
          b = fmaxf(b, __uint_as_float(x[k + 1]));
        }
        return fmaxf(fmaxf(a, b), __uint_as_float(x[31]));
      };
      float top = -INFINITY;
      tm_ld32_start(s_t, x0);
#pragma unroll
      for (int c = 0; c < kTile; c += 64) {
        tm_ld32_wait(x0);
        tm_ld32_start(s_t + c + 32, x1);
        ready(x0, c);
        top = top_of(x0, top);
        tm_ld32_wait(x1);
        tm_ld32_start(s_t + (c + 64) % kTile, x0);       // the last one is the second pass's first
        ready(x1, c + 32);
        top = top_of(x1, top);
      }
      top *= rs;
      if (__any_sync(0xffffffffu, top > m + kLazy || vn != vr)) {
        const float mn = fmaxf(m, top);
        float f = mn == m ? 1.f : ex2(m - mn);
        const uint64_t f2 = pair_of(f, f);
        sum[0] = mul2(sum[0], f2);
        sum[1] = mul2(sum[1], f2);
        m = mn;
        if (E4M3) f *= pow2i(max(vr - vn, -127));
        vr = vn;
        if (n > 0) {
          tm_ld32_wait(x0);
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            float v[32];
            tm_ld32(o_t + c, v);
#pragma unroll
            for (int x = 0; x < 32; ++x) v[x] *= f;
            tm_st32(o_t + c, v);
          }
        }
      }
      const float ref = (m == -INFINITY ? 0.f : m) - kBias;
      const uint64_t ref2 = pair_of(-ref, -ref);
      auto weigh = [&](uint32_t* x, int c) {
        ready(x, c);
        uint32_t w[16];
#pragma unroll
        for (int k = 0; k < 32; k += 4) {
          float y[4];
          split_pair(fma2(pack2(x + k), rs2, ref2), y, y + 1);
          split_pair(fma2(pack2(x + k + 2), rs2, ref2), y + 2, y + 3);
#pragma unroll
          for (int q = 0; q < 4; ++q) y[q] = ex2(y[q]);
          uint64_t a = pair_of(y[0], y[1]), b = pair_of(y[2], y[3]);
          sum[0] = add2(sum[0], a);
          sum[1] = add2(sum[1], b);
          if (E4M3) {
            const float4 f = *reinterpret_cast<const float4*>(fv + c + k);
            split_pair(mul2(a, pair_of(f.x, f.y)), y, y + 1);
            split_pair(mul2(b, pair_of(f.z, f.w)), y + 2, y + 3);
          }
          w[k / 2] = E4M3 ? hf_pack(y[0], y[1]) : bf_pack(y[0], y[1]);
          w[k / 2 + 1] = E4M3 ? hf_pack(y[2], y[3]) : bf_pack(y[2], y[3]);
        }
        tm_st16(s_t + c / 2, w);
      };
#pragma unroll
      for (int c = 0; c < kTile; c += 64) {
        tm_ld32_wait(x0);
        tm_ld32_start(s_t + c + 32, x1);
        weigh(x0, c);
        tm_ld32_wait(x1);
        if (c + 64 < kTile) tm_ld32_start(s_t + c + 64, x0);
        weigh(x1, c + 32);
      }
      tm_wait_st();
      tm_fence_before();
      mb_arrive(saddr(&sh.p_full[i]));
    }
    float y[4];
    split_pair(sum[0], y, y + 1);
    split_pair(sum[1], y + 2, y + 3);
    l = (y[0] + y[1]) + (y[2] + y[3]);
  } else if (warp < kMmaWarp) {
    // ---------------------------------------------------------------- helpers
    const int tid = threadIdx.x - kHelper0 * 32;
    const int pair_lo = max(all_lo[0], all_lo[1]);
    const int pair_hi = rows_here > kTile ? min(all_hi[0], all_hi[1]) : all_hi[0];
    bool bad = false;
    if (!E4M3) {
      constexpr int UPR = D / 8, RPI = kHelpers / UPR;      // 16-byte units a row, rows an iteration
      const int u = tid % UPR;
      for (int j = 0; j < ntiles; ++j) {
        const int n = 2 * j + 1, t0 = t_begin + j * kTile;
        if (!wait_warp(sh, saddr(&sh.raw_full[n % NO]), (n / NO) & 1)) break;
        if (t0 < pair_lo || t0 + kTile > pair_hi) {         // also wherever a value is outside [range.lo, t_end)
          for (int r = tid / UPR; r < kTile; r += RPI) {
            const uint32_t at = op_s + (n % NO) * C::kOpBytes + op_at(r, u);
            if (t0 + r < range.lo || t0 + r >= t_end) st_shared_v4u(at, make_uint4(0, 0, 0, 0));
            else bad |= any_nonfinite<false>(at);
          }
          fence_proxy_async_smem();
        }
        mb_arrive(saddr(&sh.op_full[n % NO]));
      }
    } else {
      constexpr int UPR = D / 16, RPI = kHelpers / UPR, N = kTile / RPI;
      const int u = tid % UPR, r0 = tid / UPR;
      const int32_t* table = p.b.table + (int64_t)seq * p.b.table_stride;
      // each warp has the scale bytes (key | value << 8) of all of a tile: positions t0 + 32 h + lane
      uint32_t scale[4];
      auto load_scales = [&](int j) {
        int pg = -1;
        const int t8 = t_begin + j * kTile + (lane & 7) * 16;
        if (j < ntiles && t8 < t_end) pg = page_of(table, p.b.width, p.c.pages, p.c.page_shift, t8);
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          const int t = t_begin + j * kTile + h * 32 + lane;
          const int page = __shfl_sync(0xffffffffu, pg, h * 2 + lane / 16);
          scale[h] = 0;
          if (page >= 0 && t >= range.lo && t < t_end) {
            const int64_t so = slot_scale(p.c, page, kv, t);
            scale[h] = p.c.ks[so] | (uint32_t)p.c.vs[so] << 8;
          }
        }
      };
      int vref = -127;
      load_scales(0);
      for (int n = 0; n < 2 * ntiles; ++n) {
        const int j = n >> 1, is_v = n & 1, t0 = t_begin + j * kTile;
        if (!wait_warp(sh, saddr(&sh.raw_full[n % NR]), (n / NR) & 1)) break;
        if (n >= NO && !wait_warp(sh, saddr(&sh.op_empty[n % NO]), ((n / NO) & 1) ^ 1)) break;
        const uint32_t src = raw_s + (n % NR) * C::kRawBytes + u * 16, dst = op_s + (n % NO) * C::kOpBytes;
        const bool ends = is_v && (t0 < range.lo || t0 + kTile > t_end);
        const bool look = is_v && (t0 < pair_lo || t0 + kTile > pair_hi);
        uint4 x[N];
#pragma unroll
        for (int k = 0; k < N; ++k) {
          asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                       : "=r"(x[k].x), "=r"(x[k].y), "=r"(x[k].z), "=r"(x[k].w)
                       : "r"(src + (r0 + k * RPI) * D)
                       : "memory");
        }
        __syncwarp();
        if (lane == 0) mb_arrive(saddr(&sh.raw_empty[n % NR]));
#pragma unroll
        for (int k = 0; k < N; ++k) {
          const int r = r0 + k * RPI;
          if (ends && (t0 + r < range.lo || t0 + r >= t_end)) x[k] = make_uint4(0, 0, 0, 0);
          const uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
          if (look)
#pragma unroll
            for (int q = 0; q < 4; ++q) bad |= __vcmpeq4(w[q] & 0x7f7f7f7fu, 0x7f7f7f7fu) != 0;
          uint32_t y[8];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            y[2 * q] = e4m3x2_f16x2(w[q] & 0xffffu);
            y[2 * q + 1] = e4m3x2_f16x2(w[q] >> 16);
          }
          st_shared_v4u(dst + op_at(r, 2 * u), make_uint4(y[0], y[1], y[2], y[3]));
          st_shared_v4u(dst + op_at(r, 2 * u + 1), make_uint4(y[4], y[5], y[6], y[7]));
        }
        const int slot = j % kScaleSlots, w4 = warp & 3;
        if (!is_v) {
#pragma unroll
          for (int h = 0; h < 4; ++h)
            if (h == w4) sh.fk[slot][h * 32 + lane] = pow2i((int)(scale[h] & 255) - 127) * p.scale_log2;
        } else {
          int ev[4];
#pragma unroll
          for (int h = 0; h < 4; ++h) ev[h] = (int)(scale[h] >> 8) - 127;
          vref = max(vref, __reduce_max_sync(0xffffffffu, max(max(ev[0], ev[1]), max(ev[2], ev[3]))));
          if (tid == 0) sh.vref[slot] = vref;
#pragma unroll
          for (int h = 0; h < 4; ++h)
            if (h == w4) sh.fv[slot][h * 32 + lane] = pow2i(max(ev[h] - vref, -127));
          load_scales(j + 1);
        }
        fence_proxy_async_smem();
        mb_arrive(saddr(&sh.op_full[n % NO]));
      }
    }
    if (bad) *(volatile int*)&sh.bad = 1;
  } else if (warp == kLoadWarp) {
    // ---------------------------------------------------------------- loads
    // lane i < 128 / page size: the tile's i-th page. What is outside [range.lo, t_end), on no page or on a bad one
    // is asked for behind the pool's last page, which the tensor map returns as zeros.
    const int32_t* table = p.b.table + (int64_t)seq * p.b.table_stride;
    const int size = 1 << p.c.page_shift, boxes = kTile >> p.c.page_shift;
    auto page_at = [&](int j) {
      const int t = t_begin + j * kTile + lane * size;
      int pg = -1;
      if (j < ntiles && lane < boxes && t + size > range.lo && t < t_end) {
        pg = page_of(table, p.b.width, p.c.pages, p.c.page_shift, t);
        if (pg < 0) set_status(p.c.status, CP_ERR_DEVICE_BOUNDS);
      }
      return pg < 0 ? p.c.pages : pg;
    };
    int pg = page_at(0);
    for (int n = 0; n < 2 * ntiles; ++n) {
      const int j = n >> 1, is_v = n & 1;
      if (n >= NR &&
          !wait_warp(sh, E4M3 ? saddr(&sh.raw_empty[n % NR]) : saddr(&sh.op_empty[n % NO]), ((n / NR) & 1) ^ 1))
        break;
      const uint32_t bar = saddr(&sh.raw_full[n % NR]);
      if (lane == 0) mb_expect(bar, E4M3 ? C::kRawBytes : C::kOpBytes);
      __syncwarp();
      if (lane < boxes) {
        const void* map = is_v ? &maps.v : &maps.k;
        const uint32_t dst = raw_s + (n % NR) * (E4M3 ? C::kRawBytes : C::kOpBytes) + lane * size * (E4M3 ? D : 128);
        tma_load_4d(dst, map, 0, 0, kv, pg, bar);
        if (!E4M3 && D == 128) tma_load_4d(dst + C::kSlab, map, 64, 0, kv, pg, bar);
      }
      __syncwarp();
      if (is_v) pg = page_at(j + 1);
    }
    // what was asked for lands before the block may end, whatever ended the loop
    for (int n = max(0, 2 * ntiles - NR); n < 2 * ntiles; ++n) wait_warp(sh, saddr(&sh.raw_full[n % NR]), (n / NR) & 1);
  } else if (warp == kMmaWarp && lane == 0) {
    // ---------------------------------------------------------------- MMA
    const uint32_t id_s = idesc_m128(kTile, E4M3, false), id_o = idesc_m128(D, E4M3, true);
    bool ok = wait_bar(sh, saddr(&sh.q_full), 0);
    for (int j = -1; ok && j < ntiles; ++j) {
      const int nv = 2 * j + 1, nk = 2 * j + 2;       // V of tile j, K of tile j + 1
      if (j >= 0) ok = wait_bar(sh, saddr(&sh.op_full[nv % NO]), (nv / NO) & 1);
      bool k_here = j + 1 >= ntiles;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if (ok && j >= jb[x] && j < je[x]) {
          ok = wait_bar(sh, saddr(&sh.p_full[x]), (j - jb[x]) & 1);
          tm_fence_after();
          if (ok) {
            const uint32_t v = op_s + (nv % NO) * C::kOpBytes;
#pragma unroll
            for (int k = 0; k < kTile / 16; ++k)
              tm_mma_ts(tmem + kTmemO + x * D, tmem + kTmemS + x * kTile + k * 8, sdesc_sw128_cols(v + k * 2048, C::kSlab), id_o,
                        j > jb[x] || k > 0);
          }
        }
        if (ok && !k_here) {
          ok = wait_bar(sh, E4M3 ? saddr(&sh.op_full[nk % NO]) : saddr(&sh.raw_full[nk % NO]), (nk / NO) & 1);
          k_here = true;
        }
        if (ok && j + 1 >= jb[x] && j + 1 < je[x]) {
          const uint32_t a = q_s + x * C::kOpBytes, b = op_s + (nk % NO) * C::kOpBytes;
          tm_fence_after();
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t at = (k / 4) * C::kSlab + (k % 4) * 32;
            tm_mma(tmem + kTmemS + x * kTile, sdesc_sw128(a + at), sdesc_sw128(b + at), id_s, k > 0);
          }
          tm_commit(saddr(&sh.s_full[x]));
        }
      }
      if (!ok) break;
      if (j >= 0) tm_commit(saddr(&sh.op_empty[nv % NO]));
      if (j + 1 < ntiles) tm_commit(saddr(&sh.op_empty[nk % NO]));
    }
    tm_commit(saddr(&sh.o_full));
    // after a wait that gave up, the products in flight still end before TMEM is given back
    for (int x = 0; x < (1 << 20) && !mb_try(saddr(&sh.o_full), 0); ++x) {
    }
  }
  __syncwarp();
  __syncthreads();
  tm_fence_after();

  const bool failed = sh.abort != 0;
  if (failed && threadIdx.x == 0) set_status(p.c.status, CP_ERR_TIMEOUT);
  if (!failed && sh.bad) {
    plain_rows<D, E4M3>(p, s, seq, kv, row0, row0 + rows_here, t_begin, t_end, part, whole, warp, kThreadsC / 32);
  } else if (!failed && warp < kHelper0) {
    const uint32_t o_t = tmem + ((uint32_t)(warp & 3) << 21) + kTmemO + i * D;
    const bool any = i ? je[1] > jb[1] : je[0] > jb[0];
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const float e = E4M3 ? pow2i(min(max(vr, -126), 127)) : 1.f;
#pragma unroll 1
    for (int c = 0; c < D; c += 32) {
      float v[32];
      if (any) tm_ld32(o_t + c, v);
#pragma unroll
      for (int x = 0; x < 32; ++x) v[x] = any && inv != 0.f ? v[x] * inv * e : 0.f;
      if (mine && whole) {
        uint4* dst = reinterpret_cast<uint4*>(p.out + out_row * p.o_row + (int64_t)head * p.o_head + c);
#pragma unroll
        for (int x = 0; x < 4; ++x)
          dst[x] = make_uint4(bf_pack(v[8 * x], v[8 * x + 1]), bf_pack(v[8 * x + 2], v[8 * x + 3]),
                              bf_pack(v[8 * x + 4], v[8 * x + 5]), bf_pack(v[8 * x + 6], v[8 * x + 7]));
      } else if (mine) {
#pragma unroll
        for (int x = 0; x < 8; ++x) store4<D>(p, part, false, out_row, head, c + 4 * x, v + 4 * x);
      }
    }
    if (mine && !whole) store_lse(p, part, out_row, head, l == 0.f ? -INFINITY : m + log2f(l) - kBias);
    tm_fence_before();
  }
  __syncthreads();
  if (warp == kMmaWarp) {
    tm_fence_after();
    tm_dealloc(tmem, kTmemCols);
  }
}

}  // namespace

template <int D, bool E4M3>
static cudaError_t prepare() {
  return cudaFuncSetAttribute(attend_chunk_kernel<D, E4M3>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              Cfg<D, E4M3>::kSmem);
}
cudaError_t prepare_attend_chunk() {
  for (cudaError_t e : {prepare<64, false>(), prepare<64, true>(), prepare<128, false>(), prepare<128, true>()})
    if (e != cudaSuccess) return e;
  return cudaSuccess;
}

template <int D, bool E4M3>
static cudaError_t launch(const AttendParams& p, const CacheMaps& maps, cudaStream_t s) {
  const dim3 grid((unsigned)(p.c.heads * chunk_pairs(p.b, p.group)), p.a.chunk_parts);
  attend_chunk_kernel<D, E4M3><<<grid, kThreadsC, Cfg<D, E4M3>::kSmem, s>>>(p, maps);
  return cudaGetLastError();
}
cudaError_t launch_attend_chunk(const AttendParams& p, const CacheMaps& maps, int head_dim, bool e4m3, cudaStream_t s) {
  if (head_dim == 128) return e4m3 ? launch<128, true>(p, maps, s) : launch<128, false>(p, maps, s);
  return e4m3 ? launch<64, true>(p, maps, s) : launch<64, false>(p, maps, s);
}

}  // namespace cache
}  // namespace cp
