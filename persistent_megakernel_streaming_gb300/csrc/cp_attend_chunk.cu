// cp_attend_chunk.cu -- attention of many new rows of a sequence (a piece of a
// prompt, or all of it) over the paged cache, on tcgen05.
//
// The rows of one sequence and kv head are packed row by row, query head by
// query head (row i: new row i / group, head i % group), and cut into tiles of
// 128; a block takes two tiles, so that each key and value it brings in serves
// 256 rows, and the two keep the tensor core busy in turn: while one tile's
// softmax runs, the other's products do.
//
// Warps 0-3 and 4-7: the softmax of tile 0 and tile 1, a thread a row. Warps
// 8-11: producers. Warp 12: one thread issues every MMA. For each 128
// positions S = Q K^T (128 x 128, fp32 in TMEM); the softmax threads read their
// row of S twice (maximum, then weights: the row does not fit the registers of
// 416 threads), write the weights as 16 bit over the S they have read, and
// O += P V reads them from there. O stays in TMEM for the whole pass; its
// reference maximum is only moved, and O rescaled, when a row's maximum has
// risen by 2^kLazy over it, since the sum and the weights of a part share the
// reference.
//
// Producers bring rows in by 16-byte copies (bf16, asynchronous) or through
// registers (e4m3, widened to fp16, which is exact), into the 128-byte swizzle:
// any strides, positions that nobody of the block sees become zeros without
// being read. Scales and the handling of fp16's range are the step kernel's.
#include "cp_attend.cuh"

namespace cp {
namespace cache {
namespace {

using namespace ptx;

constexpr int kTile = 128;             // rows of a tile, and positions of one
constexpr int kThreadsC = 416;
constexpr int kProducer0 = 8;          // first producer warp
constexpr int kMmaWarp = 12;
constexpr int kScaleSlots = 8;         // tiles whose scales are held: more than the ring's
constexpr long long kWaitNs = 2000000000ll;

template <int D>
struct Cfg {
  static constexpr int kStages = D == 128 ? 2 : 4;      // K and V tiles held each
  static constexpr int kOpBytes = kTile * D * 2;        // one operand tile
  static constexpr int kSlab = kTile * 128;             // 64 columns of it
  static constexpr int kLag = D == 128 ? 2 : 4;         // copies in flight behind the last issued
  static constexpr int kSmem = (2 + 2 * kStages) * kOpBytes + 1024;
};
// TMEM columns: the two tiles' scores (and weights), then their outputs
constexpr uint32_t kTmemS = 0, kTmemO = 256, kTmemCols = 512;

struct ChunkShared {
  uint64_t k_full[4], k_empty[4], v_full[4], v_empty[4];
  uint64_t q_full, s_full[2], p_full[2], o_full;
  uint32_t tmem;
  int abort;       // a wait gave up
  int bad;         // a value that some row must not see is not finite
  int top[4];      // producers' warps: largest value scale of a tile
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

template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void cp16z(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void mul4(float* v, const float* f) {
  const float4 y = *reinterpret_cast<const float4*>(f);
  v[0] *= y.x; v[1] *= y.y; v[2] *= y.z; v[3] *= y.w;
}
// Byte offset of 16-byte unit u (8 elements) of row r in an operand tile.
__device__ __forceinline__ uint32_t op_at(int r, int u) {
  return (uint32_t)((u >> 3) * (kTile * 128) + r * 128 + (((u & 7) ^ (r & 7)) << 4));
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(kThreadsC, 1) attend_chunk_kernel(const __grid_constant__ AttendParams p) {
  using C = Cfg<D>;
  constexpr int S = C::kStages;
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
  const Range range = item_range(p, pos_of(row0), pos_of(row0 + rows_here - 1), s.len);
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
      const Range r = item_range(p, first, last, s.len);
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
  const uint32_t q_s = saddr(ops), k_s = q_s + 2 * C::kOpBytes, v_s = k_s + S * C::kOpBytes;

  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      mb_init(saddr(&sh.k_full[i]), 128);
      mb_init(saddr(&sh.k_empty[i]), 1);
      mb_init(saddr(&sh.v_full[i]), 128);
      mb_init(saddr(&sh.v_empty[i]), 1);
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
  const bool mine = warp < kProducer0 && my < nrows;
  const int64_t out_row = s.row0 + (mine ? my / p.group : 0);
  const int head = kv * p.group + (mine ? my % p.group : 0);
  float l = 0.f, m = -INFINITY;
  int vr = 0;
  constexpr float kBias = E4M3 ? 8.f : 0.f;
  constexpr float kLazy = E4M3 ? 6.f : 8.f;              // weights reach 2^(kBias + kLazy): inside fp16

  if (warp < kProducer0) {
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
    for (int j = jb[i]; j < je[i]; ++j) {
      const int n = j - jb[i];
      const int t0 = t_begin + j * kTile;
      if (!wait_warp(sh, saddr(&sh.s_full[i]), n & 1)) break;
      if (E4M3 && !wait_warp(sh, saddr(&sh.v_full[j % S]), (j / S) & 1)) break;    // the tile's scales
      tm_fence_after();
      const bool edge = t0 < all_lo[i] || t0 + kTile > all_hi[i];
      const float* fk = sh.fk[j % kScaleSlots];
      const float* fv = sh.fv[j % kScaleSlots];
      float top = -INFINITY;
#pragma unroll
      for (int c = 0; c < kTile; c += 32) {
        float v[32];
        tm_ld32(s_t + c, v);
#pragma unroll
        for (int x = 0; x < 32; ++x) {
          if (E4M3 && x % 4 == 0) mul4(v + x, fk + c + x);
          if (edge && (t0 + c + x < lo || t0 + c + x >= hi)) v[x] = -INFINITY;
        }
#pragma unroll
        for (int x = 0; x < 32; ++x) top = fmaxf(top, v[x]);
      }
      top *= rs;
      const int vn = E4M3 ? sh.vref[j % kScaleSlots] : 0;
      if (__any_sync(0xffffffffu, top > m + kLazy || vn != vr)) {
        const float mn = fmaxf(m, top);
        float f = mn == m ? 1.f : ex2(m - mn);
        l *= f;
        m = mn;
        if (E4M3) f *= pow2i(max(vr - vn, -127));
        vr = vn;
        if (n > 0) {
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
#pragma unroll
      for (int c = 0; c < kTile; c += 32) {
        float v[32];
        uint32_t w[16];
        tm_ld32(s_t + c, v);
#pragma unroll
        for (int x = 0; x < 32; ++x) {
          if (E4M3 && x % 4 == 0) mul4(v + x, fk + c + x);
          if (edge && (t0 + c + x < lo || t0 + c + x >= hi)) v[x] = -INFINITY;
          v[x] = ex2(fmaf(v[x], rs, -ref));
          l += v[x];
          if (E4M3 && x % 4 == 3) mul4(v + x - 3, fv + c + x - 3);
        }
#pragma unroll
        for (int x = 0; x < 16; ++x) w[x] = E4M3 ? hf_pack(v[2 * x], v[2 * x + 1]) : bf_pack(v[2 * x], v[2 * x + 1]);
        tm_st16(s_t + c / 2, w);
      }
      tm_wait_st();
      tm_fence_before();
      mb_arrive(saddr(&sh.p_full[i]));
    }
  } else if (warp < kMmaWarp) {
    // ---------------------------------------------------------------- producers
    const int tid = threadIdx.x - kProducer0 * 32;
    const int32_t* table = p.b.table + (int64_t)seq * p.b.table_stride;
    const uint8_t* kb = p.c.k + (int64_t)kv * p.c.head_b;
    const uint8_t* vb = p.c.v + (int64_t)kv * p.c.head_b;
    const int mask = (1 << p.c.page_shift) - 1;
    const int pair_lo = max(all_lo[0], all_lo[1]);
    const int pair_hi = rows_here > kTile ? min(all_hi[0], all_hi[1]) : all_hi[0];
    // lanes 0-7 hold the pages of a tile's eight groups of 16 positions
    auto pages_of = [&](int j) {
      int pg = -1;
      const int t = t_begin + j * kTile + (lane & 7) * 16;
      if (j < ntiles && t < t_end) {
        pg = page_of(table, p.b.width, p.c.pages, p.c.page_shift, t);
        if (pg < 0) set_status(p.c.status, CP_ERR_DEVICE_BOUNDS);
      }
      return pg;
    };
    bool ok = true, bad = false;
    int pg = pages_of(0);
    if (!E4M3) {
      constexpr int UPR = D / 8, RPI = 128 / UPR, N = kTile / RPI;   // units a row, rows an iteration, iterations
      const int u = tid % UPR, r0 = tid / UPR;
      auto arrive = [&](int n) {       // load n: K of tile n / 2, then its V
        const int j = n >> 1;
        if (n & 1) {
          const int t0 = t_begin + j * kTile;
          if (t0 < pair_lo || t0 + kTile > pair_hi)
#pragma unroll 4
            for (int k = 0; k < N; ++k) bad |= any_nonfinite<false>(v_s + (j % S) * C::kOpBytes + op_at(r0 + k * RPI, u));
        }
        fence_proxy_async_smem();
        mb_arrive(saddr(n & 1 ? &sh.v_full[j % S] : &sh.k_full[j % S]));
      };
      for (int n = 0; n < 2 * ntiles; ++n) {
        const int j = n >> 1, is_v = n & 1;
        const int t0 = t_begin + j * kTile;
        const int next = is_v ? pages_of(j + 1) : 0;
        if (j >= S && !wait_warp(sh, saddr(is_v ? &sh.v_empty[j % S] : &sh.k_empty[j % S]), ((j / S) & 1) ^ 1)) {
          ok = false;
          break;
        }
        const uint32_t dst = (is_v ? v_s : k_s) + (j % S) * C::kOpBytes;
        const uint8_t* src = is_v ? vb : kb;
#pragma unroll
        for (int k = 0; k < N; ++k) {
          const int r = r0 + k * RPI, t = t0 + r;
          const int page = __shfl_sync(0xffffffffu, pg, (k * RPI + r0) / 16);
          const bool on = page >= 0 && t >= range.lo && t < t_end;
          const int64_t o = on ? (int64_t)page * p.c.page_b + (int64_t)(t & mask) * p.c.tok_b + u * 16 : 0;
          cp16z(dst + op_at(r, u), src + o, on);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        if (n >= C::kLag) {
          cp_wait<C::kLag>();
          arrive(n - C::kLag);
        }
        if (is_v) pg = next;
      }
      cp_wait<0>();
      if (ok)
        for (int n = max(0, 2 * ntiles - C::kLag); n < 2 * ntiles; ++n) arrive(n);
    } else {
      constexpr int UPR = D / 16, RPI = 128 / UPR, N = kTile / RPI;
      const int u = tid % UPR, r0 = tid / UPR;
      uint4 kx[N], vx[N];
      uint32_t scale = 0;            // key | value << 8 of position t0 + tid
      int vref = -127;
      auto load = [&](uint4* x, const uint8_t* src, int j, int pgj) {
        const int t0 = t_begin + j * kTile;
#pragma unroll
        for (int k = 0; k < N; ++k) {
          const int t = t0 + r0 + k * RPI;
          const int page = __shfl_sync(0xffffffffu, pgj, (k * RPI + r0) / 16);
          const bool on = j < ntiles && page >= 0 && t >= range.lo && t < t_end;
          x[k] = make_uint4(0, 0, 0, 0);
          if (on) x[k] = *reinterpret_cast<const uint4*>(src + (int64_t)page * p.c.page_b + (int64_t)(t & mask) * p.c.tok_b + u * 16);
        }
      };
      auto load_scale = [&](int j, int pgj) {
        const int t = t_begin + j * kTile + tid;
        const int page = __shfl_sync(0xffffffffu, pgj, tid / 16);
        uint32_t b = 0;
        if (j < ntiles && page >= 0 && t >= range.lo && t < t_end) {
          const int64_t so = slot_scale(p.c, page, kv, t);
          b = p.c.ks[so] | (uint32_t)p.c.vs[so] << 8;
        }
        return b;
      };
      auto widen = [&](const uint4* x, uint32_t dst) {
#pragma unroll
        for (int k = 0; k < N; ++k) {
          const uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
          uint32_t y[8];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            y[2 * q] = e4m3x2_f16x2(w[q] & 0xffffu);
            y[2 * q + 1] = e4m3x2_f16x2(w[q] >> 16);
          }
          const int r = r0 + k * RPI;
          st_shared_v4u(dst + op_at(r, 2 * u), make_uint4(y[0], y[1], y[2], y[3]));
          st_shared_v4u(dst + op_at(r, 2 * u + 1), make_uint4(y[4], y[5], y[6], y[7]));
        }
      };
      load(kx, kb, 0, pg);
      scale = load_scale(0, pg);
      for (int j = 0; j < ntiles; ++j) {
        const int t0 = t_begin + j * kTile;
        load(vx, vb, j, pg);
        const int next = pages_of(j + 1);
        if (j >= S && !wait_warp(sh, saddr(&sh.k_empty[j % S]), ((j / S) & 1) ^ 1)) break;
        widen(kx, k_s + (j % S) * C::kOpBytes);
        sh.fk[j % kScaleSlots][tid] = pow2i((int)(scale & 255) - 127) * p.scale_log2;
        fence_proxy_async_smem();
        mb_arrive(saddr(&sh.k_full[j % S]));
        const int ev = (int)(scale >> 8) - 127;
        const int top = __reduce_max_sync(0xffffffffu, ev);
        if (lane == 0) sh.top[warp - kProducer0] = top;
        load(kx, kb, j + 1, next);
        scale = load_scale(j + 1, next);
        if (j >= S && !wait_warp(sh, saddr(&sh.v_empty[j % S]), ((j / S) & 1) ^ 1)) break;
        if (t0 < pair_lo || t0 + kTile > pair_hi)
#pragma unroll
          for (int k = 0; k < N; ++k) {
            const uint32_t w[4] = {vx[k].x, vx[k].y, vx[k].z, vx[k].w};
#pragma unroll
            for (int q = 0; q < 4; ++q) bad |= __vcmpeq4(w[q] & 0x7f7f7f7fu, 0x7f7f7f7fu) != 0;
          }
        widen(vx, v_s + (j % S) * C::kOpBytes);
        asm volatile("bar.sync 1, 128;" ::: "memory");
        vref = max(vref, max(max(sh.top[0], sh.top[1]), max(sh.top[2], sh.top[3])));
        sh.fv[j % kScaleSlots][tid] = pow2i(max(ev - vref, -127));
        if (tid == 0) sh.vref[j % kScaleSlots] = vref;
        fence_proxy_async_smem();
        mb_arrive(saddr(&sh.v_full[j % S]));
        asm volatile("bar.sync 1, 128;" ::: "memory");     // sh.top is read before it is written again
        pg = next;
      }
    }
    if (bad) *(volatile int*)&sh.bad = 1;
  } else if (lane == 0) {
    // ---------------------------------------------------------------- MMA
    const uint32_t id_s = idesc_m128(kTile, E4M3, false), id_o = idesc_m128(D, E4M3, true);
    bool ok = wait_bar(sh, saddr(&sh.q_full), 0);
    for (int j = -1; ok && j < ntiles; ++j) {
      if (j >= 0) ok = wait_bar(sh, saddr(&sh.v_full[j % S]), (j / S) & 1);
      bool k_here = j + 1 >= ntiles;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if (ok && j >= jb[x] && j < je[x]) {
          ok = wait_bar(sh, saddr(&sh.p_full[x]), (j - jb[x]) & 1);
          tm_fence_after();
          if (ok) {
            const uint32_t v = v_s + (j % S) * C::kOpBytes;
#pragma unroll
            for (int k = 0; k < kTile / 16; ++k)
              tm_mma_ts(tmem + kTmemO + x * D, tmem + kTmemS + x * kTile + k * 8, sdesc_sw128_cols(v + k * 2048, C::kSlab), id_o,
                        j > jb[x] || k > 0);
          }
        }
        if (ok && !k_here) {
          ok = wait_bar(sh, saddr(&sh.k_full[(j + 1) % S]), ((j + 1) / S) & 1);
          k_here = true;
        }
        if (ok && j + 1 >= jb[x] && j + 1 < je[x]) {
          const uint32_t a = q_s + x * C::kOpBytes, b = k_s + ((j + 1) % S) * C::kOpBytes;
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
      if (j >= 0) tm_commit(saddr(&sh.v_empty[j % S]));
      if (j + 1 < ntiles) tm_commit(saddr(&sh.k_empty[(j + 1) % S]));
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
  } else if (!failed && warp < kProducer0) {
    const uint32_t o_t = tmem + ((uint32_t)(warp & 3) << 21) + kTmemO + i * D;
    const bool any = je[i] > jb[i];
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
  return cudaFuncSetAttribute(attend_chunk_kernel<D, E4M3>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::kSmem);
}
cudaError_t prepare_attend_chunk() {
  for (cudaError_t e : {prepare<64, false>(), prepare<64, true>(), prepare<128, false>(), prepare<128, true>()})
    if (e != cudaSuccess) return e;
  return cudaSuccess;
}
cudaError_t launch_attend_chunk(const AttendParams& p, int head_dim, bool e4m3, cudaStream_t s) {
  const dim3 grid((unsigned)(p.c.heads * chunk_pairs(p.b, p.group)), p.a.chunk_parts);
  if (head_dim == 128) {
    if (e4m3) attend_chunk_kernel<128, true><<<grid, kThreadsC, Cfg<128>::kSmem, s>>>(p);
    else attend_chunk_kernel<128, false><<<grid, kThreadsC, Cfg<128>::kSmem, s>>>(p);
  } else {
    if (e4m3) attend_chunk_kernel<64, true><<<grid, kThreadsC, Cfg<64>::kSmem, s>>>(p);
    else attend_chunk_kernel<64, false><<<grid, kThreadsC, Cfg<64>::kSmem, s>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace cache
}  // namespace cp
