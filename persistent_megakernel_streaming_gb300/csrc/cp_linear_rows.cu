// cp_linear_rows.cu -- projections of more than 16 rows with 4-bit weights, on
// tcgen05.
//
// A block takes up to FT times 128 rows of the weights (features), up to 256
// rows of x, and a share of the inputs; a cluster's blocks have the same
// features and rows and different inputs, and join their sums through
// distributed shared memory. For each 64 inputs and 128 features the weights
// are the A operand, widened to bf16 in registers and put into tensor memory
// (D[feature][row of x] += A[feature][64] B[row of x][64]); x is the B operand,
// brought in by tensor-map copies as it lies.
//
// Warps 0-7 widen: warp w has the 32 features of TMEM lanes 32 (w % 4), and
// every second piece of weights (128 features by 64 inputs), which it loads
// kAhead pieces ahead into registers; at the end they write the results. Warp
// 8 issues the products, warp 9 the copies of x.
#include <cuda.h>

#include "cp_cache_ptx.cuh"
#include "cp_linear.cuh"

namespace cp {
namespace linear {
namespace {

using namespace ptx;

constexpr int kWidenWarps = 8, kMmaWarp = 8, kLoadWarp = 9, kThreads = 320;
constexpr int kAhead = 4;
constexpr int kMostRows = 256;          // of x, a block
constexpr int kMostStages = 8;
constexpr int kSlots = 4;               // pieces of weights in tensor memory: columns 384 ..
constexpr uint32_t kTmemA = 384, kTmemCols = 512;
constexpr int kMostCluster = 8;
constexpr int kSmem = 200 * 1024;       // x's ring, and at the end the sums that the cluster joins

struct Plan {
  int ft;             // 128-feature pieces a block
  int cluster;        // shares of the inputs
  int n;              // rows of x a block, a multiple of 16
  int chunks;         // blocks along the rows
  int stages;
};

struct RowsShared {
  uint64_t a_full[kSlots], a_empty[kSlots], b_full[kMostStages], b_empty[kMostStages], d_full;
  uint32_t tmem;
  long long timeout_ns;
  int abort;          // a wait gave up
};

// Bounded: after the timeout, or once another wait of the block gave up, false.
__device__ __forceinline__ bool wait_bar(RowsShared& sh, uint32_t bar, uint32_t parity) {
  if (mb_try(bar, parity)) return true;
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

// A lane's part of a piece: two tiles' words, and their scales and zero points (of both halves of the 64 inputs).
struct Piece {
  uint4 w[2];
  uint32_t s[2][2];
  uint32_t z[2][2];
};

template <class T>
__global__ void __launch_bounds__(kThreads, 1) many_rows_kernel(const __grid_constant__ ApplyParams p, const __grid_constant__ Plan plan,
                                                                const __grid_constant__ CUtensorMap map) {
  extern __shared__ __align__(1024) uint8_t raw[];
  __shared__ RowsShared sh;
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  const Weights& w = p.w;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int S = plan.cluster, rank = blockIdx.x % S, piece0 = blockIdx.x / S * plan.ft;
  const int ft = min(plan.ft, w.tiles / 8 - piece0), n = plan.n;
  const int row0 = blockIdx.y * n;
  const int b0 = (int)((int64_t)w.blocks * rank / S), b1 = (int)((int64_t)w.blocks * (rank + 1) / S);
  const uint32_t stage_bytes = (uint32_t)n * 128;

  if (warp == kLoadWarp) {
    if (lane < kSlots) {
      mb_init(saddr(&sh.a_full[lane]), 4);
      mb_init(saddr(&sh.a_empty[lane]), 1);
    } else if (lane < kSlots + kMostStages) {
      mb_init(saddr(&sh.b_full[lane - kSlots]), 1);
      mb_init(saddr(&sh.b_empty[lane - kSlots]), 1);
    } else if (lane == 31) {
      mb_init(saddr(&sh.d_full), 1);
      sh.abort = 0;
      sh.timeout_ns = p.timeout_ns;
    }
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
  const int units = (b1 - b0) * ft;

  if (warp < kWidenWarps) {
    // ---------------------------------------------------------------- widen
    const int quarter = warp & 3, g = lane >> 2;
    const bool zeros = w.zero != nullptr;
    Piece ahead[kAhead];
    // piece u: block b0 + u / ft, features piece0 + u % ft
    auto load = [&](int u, Piece& x) {
      if (u >= units) return;
      const int b = b0 + u / ft, t = (piece0 + u % ft) * 8 + quarter * 2;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        x.w[i] = w.w[((int64_t)(t + i) * w.blocks + b) * 32 + lane];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int64_t at = meta_at(w, t + i, b * kBlockK + 32 * h, g);
          x.s[i][h] = w.scale[at];
          x.z[i][h] = zeros ? w.zero[at] : kNoZero;
        }
      }
    };
    auto put = [&](int u, const Piece& x) {
      const int slot = u % kSlots;
      if (u >= kSlots && !wait_warp(sh, saddr(&sh.a_empty[slot]), (u / kSlots - 1) & 1)) return false;
      tm_fence_after();
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t words[4] = {x.w[i].x, x.w[i].y, x.w[i].z, x.w[i].w};
        uint32_t r[16];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t a[4];
          widen(words[j], meta_of(x.s[i][j >> 1], x.z[i][j >> 1]), a);
          r[4 * j] = a[0];
          r[4 * j + 1] = a[2];
          r[4 * j + 2] = a[1];
          r[4 * j + 3] = a[3];
        }
        tm_st_16x256b_x4(tmem + ((uint32_t)(quarter * 32 + i * 16) << 16) + kTmemA + slot * 32, r);
      }
      tm_wait_st();
      tm_fence_before();
      __syncwarp();
      if (lane == 0) mb_arrive(saddr(&sh.a_full[slot]));
      return true;
    };
    const int first = warp >> 2;
#pragma unroll
    for (int k = 0; k < kAhead; ++k) load(first + 2 * k, ahead[k]);
    bool ok = true;
    for (int u = first; u < units && ok; u += 2 * kAhead) {
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int at = u + 2 * k;
        if (at < units && ok) {
          ok = put(at, ahead[k]);
          load(at + 2 * kAhead, ahead[k]);
        }
      }
    }
  } else if (warp == kLoadWarp) {
    // ---------------------------------------------------------------- x
    int asked = 0;
    for (int i = 0; i < b1 - b0; ++i) {
      const int stage = i % plan.stages;
      if (i >= plan.stages && !wait_warp(sh, saddr(&sh.b_empty[stage]), (i / plan.stages - 1) & 1)) break;
      asked = i + 1;
      if (i == 0 && p.stall) continue;
      if (lane == 0) {
        mb_expect(saddr(&sh.b_full[stage]), stage_bytes);
        tma_load_2d(saddr(ring) + stage * stage_bytes, &map, (b0 + i) * kBlockK, row0, saddr(&sh.b_full[stage]));
      }
      __syncwarp();
    }
    // what was asked for lands before the block may end, whatever ended the loop
    for (int i = max(p.stall ? 1 : 0, asked - plan.stages); i < asked; ++i)
      for (int k = 0; k < (1 << 20) && !__all_sync(0xffffffffu, mb_try(saddr(&sh.b_full[i % plan.stages]), (i / plan.stages) & 1)); ++k) {
      }
  } else {
    // ---------------------------------------------------------------- products
    const uint32_t lead = lane == 0, id = idesc_bf16_m128(n);
    const uint64_t b_desc = sdesc_sw128(saddr(ring));
    bool ok = true;
    for (int i = 0; i < b1 - b0 && ok; ++i) {
      const int stage = i % plan.stages;
      ok = wait_warp(sh, saddr(&sh.b_full[stage]), (i / plan.stages) & 1);
      const uint64_t b = b_desc + (uint64_t)(stage * (stage_bytes >> 4));
      for (int f = 0; f < ft && ok; ++f) {
        const int u = i * ft + f, slot = u % kSlots;
        ok = wait_warp(sh, saddr(&sh.a_full[slot]), (u / kSlots) & 1);
        if (!ok) break;
        tm_fence_after();
#pragma unroll
        for (int k = 0; k < 4; ++k)
          tm_mma_ts_lead(lead, tmem + f * n, tmem + kTmemA + slot * 32 + k * 8, b + 2 * k, id, i > 0 || k > 0);
        tm_commit_lead(lead, saddr(&sh.a_empty[slot]));
      }
      if (ok) tm_commit_lead(lead, saddr(&sh.b_empty[stage]));
    }
    tm_commit_lead(lead, saddr(&sh.d_full));
    // the products in flight end before anything is read or given back, even after a wait that gave up
    for (int k = 0; k < (1 << 20) && !__all_sync(0xffffffffu, mb_try(saddr(&sh.d_full), 0)); ++k) {
    }
  }
  __syncwarp();
  __syncthreads();
  tm_fence_after();
  const bool failed = sh.abort != 0;
  if (failed && threadIdx.x == 0) atomicCAS(p.status, 0, (int)CP_ERR_TIMEOUT);

  // Results. Feature i of a piece is in TMEM lane i, row r of x in column r.
  const int rows_here = min(n, p.rows - row0);
  T* out = static_cast<T*>(p.out);
  auto finish = [&](int r, int feature, float y) {
    if (p.add) y += load_out<T>(p.add, (int64_t)(row0 + r) * p.add_row + feature);
    store_out(out + (int64_t)(row0 + r) * p.out_row + feature, y);
  };
  float* sums = reinterpret_cast<float*>(ring);            // [row][features of the block]
  const int wide = plan.ft * 128;
  if (warp < kWidenWarps && !failed) {
    const int quarter = warp & 3, half = warp >> 2;
    const uint32_t lanes = (uint32_t)quarter << 21;
    for (int f = 0; f < ft; ++f) {
      for (int c = half * 16; c < n; c += 32) {
        float v[16];
        if (b1 > b0) {
          tm_ld16(tmem + lanes + f * n + c, v);
        } else {
#pragma unroll
          for (int x = 0; x < 16; ++x) v[x] = 0.f;
        }
        if (S > 1) {
#pragma unroll
          for (int x = 0; x < 16; ++x) sums[(c + x) * wide + f * 128 + quarter * 32 + lane] = v[x];
        } else if (w.gated) {
          const int feature = (piece0 + f) * 64 + quarter * 16 + (lane & 15);
#pragma unroll
          for (int x = 0; x < 16; ++x) {
            const float up = __shfl_xor_sync(0xffffffffu, v[x], 16);
            if (lane < 16 && feature < w.outs && c + x < rows_here) finish(c + x, feature, silu(v[x]) * up);
          }
        } else {
          const int feature = (piece0 + f) * 128 + quarter * 32 + lane;
#pragma unroll
          for (int x = 0; x < 16; ++x)
            if (feature < w.outs && c + x < rows_here) finish(c + x, feature, v[x]);
        }
      }
    }
    tm_fence_before();
  }
  if (S > 1) {
    __syncwarp();
    cluster_sync_all();
    // each of the cluster's blocks takes every S-th row, and adds up in the blocks' order
    const int per = w.gated ? wide / 2 : wide;
    if (!failed)
      for (int r = rank; r < rows_here; r += S)
        for (int i = threadIdx.x; i < per; i += kThreads) {
          const int at = w.gated ? (i >> 4) * 32 + (i & 15) : i;
          const uint32_t mine = saddr(sums + r * wide + at);
          float y = 0.f, up = 0.f;
          for (int k = 0; k < S; ++k) {
            const uint32_t from = mapa(mine, k);
            y += ld_cluster(from);
            if (w.gated) up += ld_cluster(from + 64);
          }
          if (w.gated) y = silu(y) * up;
          const int feature = piece0 * (w.gated ? 64 : 128) + i;
          if (feature < w.outs && i < ft * (w.gated ? 64 : 128)) finish(r, feature, y);
        }
    __syncwarp();
    cluster_sync_all();
  } else {
    __syncthreads();
  }
  if (warp == kMmaWarp) {
    tm_fence_after();
    tm_dealloc(tmem, kTmemCols);
  }
}

int up_to(int a, int b) { return (a + b - 1) / b * b; }

Plan make_plan(const ApplyParams& p) {
  Plan a{};
  a.chunks = (p.rows + kMostRows - 1) / kMostRows;
  a.n = up_to((p.rows + a.chunks - 1) / a.chunks, 16);
  a.chunks = (p.rows + a.n - 1) / a.n;
  const int pieces = p.w.tiles / 8;
  a.ft = 1;
  a.cluster = 1;
  while (a.cluster < kMostCluster && pieces * a.chunks * a.cluster * 2 <= 152 && p.w.blocks >= a.cluster * 4) a.cluster *= 2;
  a.stages = kSmem / (a.n * 128);
  if (a.stages > kMostStages) a.stages = kMostStages;
  return a;
}

template <class T>
cudaError_t launch(const ApplyParams& p, const Plan& a, const CUtensorMap& map, cudaStream_t s) {
  const int groups = (p.w.tiles / 8 + a.ft - 1) / a.ft;
  return launch_as(many_rows_kernel<T>, dim3((unsigned)(groups * a.cluster), (unsigned)a.chunks), a.cluster, 1, false, kThreads,
                   kSmem + 1024, s, p, a, map);
}

}  // namespace

cudaError_t prepare_many_rows() {
  cudaError_t e = cudaFuncSetAttribute(many_rows_kernel<float>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem + 1024);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(many_rows_kernel<__nv_bfloat16>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem + 1024);
}

cudaError_t launch_many_rows(const ApplyParams& p, bool f32, cudaStream_t s) {
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
  if (encode(&map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<uint16_t*>(p.x), dims, strides, box, steps,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  return f32 ? launch<float>(p, a, map, s) : launch<__nv_bfloat16>(p, a, map, s);
}

}  // namespace linear
}  // namespace cp
