// cp_linear_rows.cu -- projections of more than 8 or 16 rows with 4-bit weights,
// on tcgen05.
//
// A block takes up to FT times 128 rows of the weights (features), up to 192
// rows of x, and a share of the inputs; a cluster's blocks have the same
// features and rows and different inputs, and join their sums through
// distributed shared memory. For each record (128 features by 128 inputs) the
// weights are the A operand, widened to bf16 in registers and put into tensor
// memory (D[feature][row of x] += A[feature][128] B[row of x][128]); x is the B
// operand, brought in by tensor-map copies as it lies.
//
// One lane brings the records into a ring in shared memory, one x; the others
// widen: warp w has the 32 features of TMEM lanes 32 (w % 4) of every
// kGroups-th record; at the end they write the results. The records' products
// go in turn to two or four streams, each with an issuing lane and sums of its
// own: what a lane does between two records' products (waits, commits) takes
// about as long as they do, and with one lane nothing covers it (64 rows, 16384
// to 8192: 32 us). (Weights loaded ahead into the widening warps' own registers: a
// warp's outstanding loads share few scoreboards, and waiting for the oldest
// waits for the newest.)
//
// A call costs 4.2 us (64 rows) to 7 (112 rows of 256 features a block) and
// 0.225 a record of a block (64 of them, 64 rows, 16384 to 8192: 23.7 us on 128
// SMs, 3.1 TB/s, 725 TFLOP/s). A record of 64 rows is 336 clocks of the tensor
// core, 375 of issuing what widens it, and measured 430: both, and the hand-overs
// between them, which take 380 even where nothing is widened.
#include <cuda.h>

#include "cp_cache_ptx.cuh"
#include "cp_linear.cuh"

namespace cp {
namespace linear {
namespace {

using namespace ptx;

constexpr int kGroups = 4;               // of four widening warps
constexpr int kMostStreams = 4;
constexpr int kWidenWarps = 4 * kGroups, kMmaWarp = kWidenWarps, kWeightWarp = kMmaWarp + kMostStreams, kXWarp = kWeightWarp + 1;
constexpr int kThreads = (kXWarp + 1) * 32;
constexpr int kMostRows = 192;           // of x, a block
constexpr int kMostStages = 8;           // of x's ring: 128 inputs each
constexpr int kUnits = 8;                // records in the weights' ring, a power of two
constexpr int kMostSlots = 4;            // widened records in tensor memory, 64 columns each: the last 128 or 256 columns
constexpr uint32_t kTmemCols = 512;
constexpr int kMostCluster = 4;          // of 8, whose blocks have an SM each, few fit: 16 to 30 us where 4 take 6 to 10
constexpr int kRing = kUnits * kMostRecord;
constexpr int kSmem = 216 * 1024;        // both rings, and at the end the sums that the cluster joins

struct Plan {
  int ft;             // 128-feature pieces a block: 1, or up to as many as streams, which it divides
  int streams;        // 2 or 4: records' products by turns; stream s has the sums of piece s % ft
  int cluster;        // shares of the inputs
  int n;              // rows of x a block, a multiple of 16
  int chunks;         // blocks along the rows
  int stages;         // of x's ring
  int slots;          // 2 or 4
};

// A place in a ring and the parity of its turn round it, by counting: a quotient takes one warp 100 to 200 clocks, and
// with several of them for each unit the issuing warps were what the kernel waited for (64 rows, 16384 to 8192: 100 us).
struct Turn {
  int at = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void next(int n, int by = 1) {      // by up to n
    at += by;
    if (at >= n) {
      at -= n;
      parity ^= 1;
    }
  }
};

struct RowsShared {
  uint64_t w_full[kUnits], w_empty[kUnits], a_full[kMostSlots], a_empty[kMostSlots], b_full[kMostStages], b_empty[kMostStages], d_full;
  uint32_t tmem;
  long long timeout_ns;
  int abort;          // a wait gave up
};

// Bounded: after the timeout, or once another wait of the block gave up, false. The kernel in front takes as long as it
// takes: x comes behind it, and the time counts from its end.
__device__ __noinline__ bool wait_long(RowsShared& sh, uint32_t bar, uint32_t parity) {
  pdl_wait();
  const uint64_t t0 = gtime();
  for (;;) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (mb_try(bar, parity)) return true;
    if (*(volatile int*)&sh.abort) return false;
    if ((long long)(gtime() - t0) > sh.timeout_ns) {
      *(volatile int*)&sh.abort = 1;
      return false;
    }
  }
}
__device__ __forceinline__ bool wait_bar(RowsShared& sh, uint32_t bar, uint32_t parity) {
  return mb_try(bar, parity) || wait_long(sh, bar, parity);
}
__device__ __forceinline__ bool wait_warp(RowsShared& sh, uint32_t bar, uint32_t parity) {
  return __all_sync(0xffffffffu, wait_bar(sh, bar, parity));
}

// 16 rows by 4 x 256 bits: lane 4 g + c has 8 consecutive bytes, 32 bytes apart, of rows g (r[4 i], r[4 i + 1]) and g + 8.
__device__ __forceinline__ void tm_st_16x256b_x4(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const void* map, int c0, int c1, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(map), "r"(c0), "r"(c1), "r"(bar)
      : "memory");
}

// One lane of the warp, always the same. Behind this the compiler knows that one lane is left, and keeps what the
// products and copies are given in uniform registers, if it comes from uniform values: a product every 28 clocks (32
// rows of x; 42 for 64, 90 for 160). Behind `lane == 0`, or predicated in a warp that stays together, it took 100 to
// 130 whatever the rows, and the whole kernel 76 us instead of what stands above.
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(one)
      :
      : "memory");
  return one != 0;
}
// A in tensor memory, B in shared memory.
__device__ __forceinline__ void tm_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred P;\n\t"
      "setp.ne.b32 P, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, P;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// 16 columns from each of two addresses, under way together: v[0 .. 15], v[16 .. 31]. (The first load's registers are not
// the second's address.)
__device__ __forceinline__ void tm_ld16_two(uint32_t a, uint32_t b, float* v) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%32];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%33];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=&r"(r[0]), "=&r"(r[1]), "=&r"(r[2]), "=&r"(r[3]), "=&r"(r[4]), "=&r"(r[5]), "=&r"(r[6]), "=&r"(r[7]), "=&r"(r[8]), "=&r"(r[9]),
        "=&r"(r[10]), "=&r"(r[11]), "=&r"(r[12]), "=&r"(r[13]), "=&r"(r[14]), "=&r"(r[15]), "=&r"(r[16]), "=&r"(r[17]), "=&r"(r[18]),
        "=&r"(r[19]), "=&r"(r[20]), "=&r"(r[21]), "=&r"(r[22]), "=&r"(r[23]), "=&r"(r[24]), "=&r"(r[25]), "=&r"(r[26]), "=&r"(r[27]),
        "=&r"(r[28]), "=&r"(r[29]), "=&r"(r[30]), "=&r"(r[31])
      : "r"(a), "r"(b)
      : "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ uint32_t ld_shared_u32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t ld_shared_u16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a) : "memory");
  return v;
}

template <class T, bool ZERO>
__global__ void __launch_bounds__(kThreads, 1) many_rows_kernel(const __grid_constant__ ApplyParams p, const __grid_constant__ Plan plan,
                                                                const __grid_constant__ CUtensorMap map) {
  extern __shared__ __align__(1024) uint8_t raw[];
  __shared__ RowsShared sh;
  const Weights& w = p.w;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int S = plan.cluster, rank = blockIdx.x % S, piece0 = blockIdx.x / S * plan.ft;
  const int ft = plan.ft, n = plan.n;
  const int row0 = blockIdx.y * n;
  const int b0 = (int)((int64_t)w.per_piece * rank / S), b1 = (int)((int64_t)w.per_piece * (rank + 1) / S);   // records
  const uint32_t stage_bytes = (uint32_t)n * 256;    // two halves of 64 inputs
  const uint32_t x_ring = (saddr(raw) + 1023) & ~1023u, w_ring = x_ring + plan.stages * stage_bytes;
  const int slots = plan.slots;
  const uint32_t tmem_a = kTmemCols - slots * 64;

  if (warp == kWeightWarp) {
    if (lane < kUnits) {
      mb_init(saddr(&sh.w_full[lane]), 1);
      mb_init(saddr(&sh.w_empty[lane]), 4);
    } else if (lane < kUnits + kMostSlots) {
      mb_init(saddr(&sh.a_full[lane - kUnits]), 4);
      mb_init(saddr(&sh.a_empty[lane - kUnits]), 1);
    } else if (lane < kUnits + kMostSlots + kMostStages) {
      mb_init(saddr(&sh.b_full[lane - kUnits - kMostSlots]), 1);
      mb_init(saddr(&sh.b_empty[lane - kUnits - kMostSlots]), ft);
    } else if (lane == 31) {
      mb_init(saddr(&sh.d_full), plan.streams);
      sh.abort = 0;
      sh.timeout_ns = p.timeout_ns;
    }
    mb_fence_init();
  }
  pdl_trigger();
  if (warp == kMmaWarp) {
    tm_alloc(saddr(&sh.tmem), kTmemCols);
    tm_relinquish();
  }
  tm_fence_before();
  __syncthreads();
  tm_fence_after();
  constexpr uint32_t tmem = 0;             // all of it is the block's: it starts at its first column
  const int units = (b1 - b0) * ft;

  if (warp < kWidenWarps) {
    // ---------------------------------------------------------------- widen
    const int quarter = warp & 3, g = lane >> 2;
    const int slot_shift = slots == 4 ? 2 : 1, group_shift = w.group_shift;
    const uint32_t zeros = kRecordWords + w.groups * kRecordScales;
    // a group for each slot at most: each then waits for its own last unit's products, and a turn's parity says which
    const int groups = min(kGroups, slots);
    for (int u = (warp >> 2) < groups ? warp >> 2 : units; u < units; u += groups) {
      const int unit = u & (kUnits - 1), slot = u & (slots - 1);
      if (!wait_warp(sh, saddr(&sh.w_full[unit]), (uint32_t)(u / kUnits) & 1)) break;
      const uint32_t at = w_ring + unit * kMostRecord, own = quarter * 16 + g;
      const uint32_t to = tmem + ((uint32_t)(quarter * 32) << 16) + tmem_a + slot * 64;
      bool ok = true;
#pragma unroll
      for (int sub = 0; sub < 2; ++sub) {
        uint32_t r[2][16];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint4 words = ld_shared_v4u(at + sub * 4096 + (quarter * 2 + i) * 512 + lane * 16);
          const uint32_t v[4] = {words.x, words.y, words.z, words.w};
          Meta m;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (j == 0 || (j == 2 && group_shift == 5)) {
              const int grp = (sub * 64 + j * 16) >> group_shift;
              const uint32_t s = ld_shared_u32(at + kRecordWords + grp * kRecordScales + (own + i * 8) * 4);
              m = meta_of<ZERO>(s, ZERO ? ld_shared_u16(at + zeros + grp * kRecordZeros + (own + i * 8) * 2) : 0);
            }
            uint32_t a[4];
            widen(v[j], m, a);
            r[i][4 * j] = a[0];
            r[i][4 * j + 1] = a[2];
            r[i][4 * j + 2] = a[1];
            r[i][4 * j + 3] = a[3];
          }
        }
        // the first half is widened while the products out of the slot's last unit still run
        if (sub == 0) {
          ok = wait_warp(sh, saddr(&sh.a_empty[slot]), ((uint32_t)(u >> slot_shift) & 1) ^ 1);     // at first: free
          if (!ok) break;
          tm_fence_after();
        }
        tm_st_16x256b_x4(to + sub * 32, r[0]);
        tm_st_16x256b_x4(to + (16 << 16) + sub * 32, r[1]);
      }
      if (!ok) break;
      __syncwarp();
      if (lane == 0) mb_arrive(saddr(&sh.w_empty[unit]));
      tm_wait_st();
      tm_fence_before();
      __syncwarp();
      if (lane == 0) mb_arrive(saddr(&sh.a_full[slot]));
    }
  } else if (warp == kWeightWarp) {
    // ---------------------------------------------------------------- weights
    if (elect_one()) {
      // a last group of fewer pieces has its last one again: nothing else is to know of it but the results
      const int last = w.tiles / 8 - 1 - piece0;
      const uint8_t* from = w.records + record_at(w, piece0 * 8, b0 * kRecordK);
      const int64_t next_piece = (int64_t)w.per_piece * w.bytes;
      int asked = 0, f = 0;
      Turn unit;
      for (; asked < units; ++asked) {
        if (!wait_bar(sh, saddr(&sh.w_empty[unit.at]), unit.parity ^ 1)) break;
        const uint32_t bar = saddr(&sh.w_full[unit.at]);
        mb_expect(bar, w.bytes);
        bulk_g2s(w_ring + unit.at * kMostRecord, from + min(f, last) * next_piece, w.bytes, bar);
        unit.next(kUnits);
        if (++f == ft) {
          f = 0;
          from += w.bytes;
        }
      }
      // what was asked for lands before the block may end, whatever ended the loop
      for (int u = max(0, asked - kUnits); u < asked; ++u)
        for (int k = 0; k < (1 << 20) && !mb_try(saddr(&sh.w_full[u & (kUnits - 1)]), (uint32_t)(u / kUnits) & 1); ++k) {
        }
    }
  } else if (warp == kXWarp) {
    // ---------------------------------------------------------------- x
    if (elect_one()) {
      Turn stage;
      int asked = 0;
      pdl_wait();                          // x may be what the kernel in front writes; the weights are nobody's
      for (; asked < b1 - b0; ++asked) {
        const uint32_t bar = saddr(&sh.b_full[stage.at]), at = x_ring + stage.at * stage_bytes;
        if (!wait_bar(sh, saddr(&sh.b_empty[stage.at]), stage.parity ^ 1)) break;
        if (asked > 0 || !p.stall) {
          mb_expect(bar, stage_bytes);
          tma_load_2d(at, &map, (b0 + asked) * kRecordK, row0, bar);
          tma_load_2d(at + stage_bytes / 2, &map, (b0 + asked) * kRecordK + kBlockK, row0, bar);
        }
        stage.next(plan.stages);
      }
      // what was asked for lands before the block may end, whatever ended the loop
      for (int i = max(p.stall ? 1 : 0, asked - plan.stages); i < asked; ++i)
        for (int k = 0; k < (1 << 20) && !mb_try(saddr(&sh.b_full[i % plan.stages]), (i / plan.stages) & 1); ++k) {
        }
    }
  } else if (warp - kMmaWarp < plan.streams) {
    // ---------------------------------------------------------------- products
    if (elect_one()) {
      const int own = warp - kMmaWarp, streams = plan.streams, step = streams / ft;
      const uint32_t id = idesc_bf16_m128(n), stage_desc = stage_bytes >> 4, d = tmem + own * n;
      const uint64_t b_desc = sdesc_sw128(x_ring);
      Turn stage, slot;
      stage.next(plan.stages, own / ft);
      slot.at = own;
      for (int i = own / ft; i < b1 - b0; i += step) {
        if (!wait_bar(sh, saddr(&sh.b_full[stage.at]), stage.parity) || !wait_bar(sh, saddr(&sh.a_full[slot.at]), slot.parity)) break;
        tm_fence_after();
        const uint64_t x0 = b_desc + stage.at * stage_desc, x1 = x0 + stage_desc / 2;
        const uint32_t a = tmem + tmem_a + slot.at * 64;
#pragma unroll
        for (int k = 0; k < 8; ++k) tm_mma_ts(d, a + k * 8, (k < 4 ? x0 : x1) + 2 * (k & 3), id, i >= step || k > 0);
        tm_commit(saddr(&sh.a_empty[slot.at]));
        tm_commit(saddr(&sh.b_empty[stage.at]));
        slot.next(slots, streams);
        stage.next(plan.stages, step);
      }
      tm_commit(saddr(&sh.d_full));
      // the products in flight end before anything is read or given back, even after a wait that gave up
      for (int k = 0; k < (1 << 20) && !mb_try(saddr(&sh.d_full), 0); ++k) {
      }
    }
  }
  __syncwarp();
  __syncthreads();
  tm_fence_after();
  const bool failed = sh.abort != 0;
  if (failed && threadIdx.x == 0) atomicCAS(p.status, 0, (int)CP_ERR_TIMEOUT);

  pdl_wait();                              // what reads out or writes add in front of this is done
  // Results. Feature i of a piece is in TMEM lane i, row r of x in column r.
  const int rows_here = min(n, p.rows - row0), here = min(ft, w.tiles / 8 - piece0);
  float* sums = reinterpret_cast<float*>(raw + (x_ring - saddr(raw)));      // [row][features of the block]
  const int wide = plan.ft * 128;
  if (warp < kWidenWarps && !failed) {
    const int quarter = warp & 3, part = warp >> 2;
    const uint32_t lanes = (uint32_t)quarter << 21;
    const int turns = b1 - b0;                        // stream s had products if there are more than s / ft
    auto put = [&](int f, int c, const float* v) {
#pragma unroll
      for (int x = 0; x < 16; ++x) sums[(c + x) * wide + f * 128 + quarter * 32 + lane] = v[x];
    };
    for (int c = part * 16; c < n; c += 16 * kGroups) {
      float v[32], x[32];
      if (ft == 1) {                                  // two streams' sums of the piece at a time
        tm_ld16_two(tmem + lanes + c, tmem + lanes + n + c, v);
#pragma unroll
        for (int k = 0; k < 16; ++k) v[k] += turns > 1 ? v[16 + k] : 0.f;
        if (plan.streams > 2 && turns > 2) {
          tm_ld16_two(tmem + lanes + 2 * n + c, tmem + lanes + 3 * n + c, x);
#pragma unroll
          for (int k = 0; k < 16; ++k) v[k] += turns > 3 ? x[k] + x[16 + k] : x[k];
        }
        put(0, c, v);
      } else {                                        // two pieces'
        for (int f = 0; f < here; f += 2) {
          tm_ld16_two(tmem + lanes + f * n + c, tmem + lanes + (f + 1) * n + c, v);
          if (plan.streams > ft && turns > 1) {
            tm_ld16_two(tmem + lanes + (f + ft) * n + c, tmem + lanes + (f + ft + 1) * n + c, x);
#pragma unroll
            for (int k = 0; k < 32; ++k) v[k] += x[k];
          }
          put(f, c, v);
          if (f + 1 < here) put(f + 1, c, v + 16);
        }
      }
    }
    tm_fence_before();
  }
  if (S > 1) {
    __syncwarp();
    cluster_sync_all();
  } else {
    __syncthreads();
  }
  // each of the cluster's blocks takes every S-th row, four features a thread, and adds up in the blocks' order; all loads
  // from other blocks' memory are under way before the first is waited for. (Straight out of tensor memory, an element a
  // thread at a time, 320 rows, 2048 to 2 x 6144, took 17.4 us a call, this way 15.0; with the residual's lines fetched into
  // L2 ahead every call took 0.3 to 1 more.)
  const int lg = 31 - __clz(plan.ft) + (w.gated ? 4 : 5), items = (rows_here - rank + S - 1) / S << lg;
  if (!failed)
    for (int i = threadIdx.x; i < items; i += kThreads) {
      const int r = rank + (i >> lg) * S, f = (i & ((1 << lg) - 1)) * 4;
      const int feature = piece0 * (w.gated ? 64 : 128) + f;
      if (feature >= w.outs) continue;                                         // a last group of fewer pieces, too
      const float* own = sums + r * wide + (w.gated ? (f >> 4) * 32 + (f & 15) : f);
      float4 v[kMostCluster], u[kMostCluster];
      if (S == 1) {
        v[0] = *reinterpret_cast<const float4*>(own);
        if (w.gated) u[0] = *reinterpret_cast<const float4*>(own + kTileRows);
      } else {
#pragma unroll
        for (int k = 0; k < kMostCluster; ++k)
          if (k < S) {
            v[k] = ld_cluster_v4(mapa(saddr(own), k));
            if (w.gated) u[k] = ld_cluster_v4(mapa(saddr(own + kTileRows), k));
          }
      }
      float y[4] = {}, up[4] = {};
#pragma unroll
      for (int k = 0; k < kMostCluster; ++k)
        if (k < S) {
          y[0] += v[k].x; y[1] += v[k].y; y[2] += v[k].z; y[3] += v[k].w;
          if (w.gated) up[0] += u[k].x, up[1] += u[k].y, up[2] += u[k].z, up[3] += u[k].w;
        }
      if (w.gated)
#pragma unroll
        for (int k = 0; k < 4; ++k) y[k] = silu(y[k]) * up[k];
      finish<T>(p, row0 + r, feature, min(4, w.outs - feature), y);
    }
  if (S > 1) {
    __syncwarp();
    cluster_sync_all();
  }
  if (warp == kMmaWarp) {
    tm_fence_after();
    tm_dealloc(tmem, kTmemCols);
  }
}

int up_to(int a, int b) { return (a + b - 1) / b * b; }

// How a call is cut up: what costs least by a model of the measured times, in microseconds. A round of blocks takes
// kRoundUs to start and end; a record's products 8 times (12 + n / 2) clocks on the tensor core, and no less than what
// widening and the hand-overs take; joining moves a block's sums through distributed shared memory at 12 bytes a clock.
// Clusters leave SMs over. (64 rows, 16384 to 8192: one piece and two shares of the inputs a block 22.7 us, two pieces and
// four shares 22.9, one piece and no shares 36.5, and four 29.7; 320 rows, 2048 to 2 x 6144: three chunks of 112 rows and two
// pieces a block 15.0, one piece 19.8, two chunks of 160 rows 21.7, five of 64 25.3.)
constexpr double kRoundUs = 5, kRecordUs = 0.256, kClocksUs = 1900;
int blocks_at_once(int cluster) { return cluster == 1 ? 152 : cluster == 2 ? 148 : 144; }

Plan make_plan(const ApplyParams& p) {
  Plan best{};
  double least = 1e30;
  const int pieces = p.w.tiles / 8, fewest = (p.rows + kMostRows - 1) / kMostRows;
  for (int chunks = fewest; chunks <= fewest + 3; ++chunks) {
    Plan a{};
    a.n = up_to((p.rows + chunks - 1) / chunks, 16);
    a.chunks = (p.rows + a.n - 1) / a.n;
    a.streams = a.n <= 64 ? 4 : 2;
    a.stages = (kSmem - kRing) / (a.n * 256);
    if (a.stages > kMostStages) a.stages = kMostStages;
    a.slots = a.streams * a.n <= 256 ? 4 : 2;
    const double record = 8 * (12 + 0.5 * a.n) / kClocksUs;
    for (a.ft = 1; a.ft <= a.streams; a.ft *= 2)
      for (a.cluster = 1; a.cluster <= kMostCluster && a.cluster <= p.w.per_piece; a.cluster *= 2) {
        const int64_t blocks = (int64_t)((pieces + a.ft - 1) / a.ft) * a.cluster * a.chunks;
        const int64_t rounds = (blocks + blocks_at_once(a.cluster) - 1) / blocks_at_once(a.cluster);
        const int units = (p.w.per_piece + a.cluster - 1) / a.cluster * a.ft;
        const double join = a.cluster == 1 ? 0 : 1 + a.n * a.ft * 512. * (a.cluster - 1) / a.cluster / 12 / kClocksUs;
        const double us = rounds * (kRoundUs + units * (record > kRecordUs ? record : kRecordUs) + join);
        if (us < least) {
          least = us;
          best = a;
        }
      }
  }
  return best;
}

template <class T>
cudaError_t launch(const ApplyParams& p, const Plan& a, const CUtensorMap& map, cudaStream_t s) {
  const int groups = (p.w.tiles / 8 + a.ft - 1) / a.ft;
  const dim3 grid((unsigned)(groups * a.cluster), (unsigned)a.chunks);
  return p.w.zero ? launch_as(many_rows_kernel<T, true>, grid, a.cluster, 1, true, kThreads, kSmem + 1024, s, p, a, map)
                  : launch_as(many_rows_kernel<T, false>, grid, a.cluster, 1, true, kThreads, kSmem + 1024, s, p, a, map);
}

}  // namespace

template <class T, bool ZERO>
static cudaError_t prepare() {
  return cudaFuncSetAttribute(many_rows_kernel<T, ZERO>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem + 1024);
}
cudaError_t prepare_many_rows() {
  for (cudaError_t e : {prepare<float, false>(), prepare<float, true>(), prepare<__nv_bfloat16, false>(), prepare<__nv_bfloat16, true>()})
    if (e != cudaSuccess) return e;
  return cudaSuccess;
}

cudaError_t launch_many_rows(const ApplyParams& p, cudaStream_t s) {
  static const auto encode = [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      fn = nullptr;
    return reinterpret_cast<decltype(&cuTensorMapEncodeTiled)>(fn);
  }();
  if (!encode) return cudaErrorNotSupported;
  const Plan a = make_plan(p);
  // x: 64 inputs by the block's rows, in the 128-byte swizzle that the tensor core reads; zeros outside
  CUtensorMap map;
  const cuuint64_t dims[2] = {(cuuint64_t)p.w.width, (cuuint64_t)p.rows};
  const cuuint64_t strides[1] = {(cuuint64_t)p.x_row * 2};
  const cuuint32_t box[2] = {kBlockK, (cuuint32_t)a.n}, steps[2] = {1, 1};
  const CUresult made = in_context([&] {
    return encode(&map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<uint16_t*>(p.x), dims, strides, box, steps,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  });
  if (made != CUDA_SUCCESS) return cudaErrorInvalidValue;
  return p.f32 ? launch<float>(p, a, map, s) : launch<__nv_bfloat16>(p, a, map, s);
}

}  // namespace linear
}  // namespace cp
