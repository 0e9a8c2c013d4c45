// cp_linear.cu -- projections with 4-bit weights: the C ABI (checks, layout of
// the weights, launches) and the kernel for few rows.
#include <cuda_runtime.h>

#include <new>

#include "cp.h"
#include "cp_call.h"
#include "cp_linear.cuh"
#include "cp_ptx.cuh"

using namespace cp;
using namespace cp::linear;

struct cp_linear {
  int device = 0;
  Weights w{};
  int32_t* status = nullptr;
  long long timeout_ns = 0;
  int stall = 0;
  void* memory = nullptr;
};

namespace {

// ------------------------------------------------------------------ layout
struct PackParams {
  Weights w;
  const uint8_t* q;
  const uint16_t* scale;
  const uint8_t* zero;
  uint8_t* out;
  int* bad;
};

// A thread a lane's word; lanes 0 .. 7 of a tile write its scales and zero points too.
__global__ void pack_kernel(const PackParams p) {
  const Weights& w = p.w;
  const int64_t words = (int64_t)w.tiles * w.per_piece * 2 * 32, step = (int64_t)gridDim.x * blockDim.x;
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < words; i += step) {
    const int lane = (int)(i & 31), g = lane >> 2, c = lane & 3;
    const int64_t rest = i >> 5;
    const int t = (int)(rest % w.tiles), k0 = (int)(rest / w.tiles) * kBlockK;
    uint8_t* record = p.out + record_at(w, t, k0);
    uint32_t out[4];
    for (int j = 0; j < 4; ++j) {
      out[j] = 0;
      for (int a = 0; a < 4; ++a) {
        const int row = row_of(w, t, g + (a & 1) * 8), k = k0 + 16 * j + 4 * c + (a >> 1) * 2;
        if (row < 0 || k >= w.width) continue;
        const uint32_t two = p.q[(int64_t)row * (w.width / 2) + k / 2];
        out[j] |= (two & 15) << (4 * a) | (two >> 4) << (16 + 4 * a);
      }
    }
    *reinterpret_cast<uint4*>(record + word_in(t, k0, lane)) = make_uint4(out[0], out[1], out[2], out[3]);
    if (lane >= 8) continue;
    for (int k = k0; k < k0 + kBlockK; k += 32) {              // a group of more is written by each of its blocks, alike
      uint32_t s = 0, z = 0;
      for (int h = 0; h < 2; ++h) {
        const int row = row_of(w, t, lane + 8 * h);
        if (row < 0 || k >= w.width) continue;               // rows and inputs that are not there weigh nothing
        const int64_t at = (int64_t)row * (w.width >> w.group_shift) + (k >> w.group_shift);
        const uint32_t up = __bfloat16_as_ushort(__float2bfloat16_rn(64.f * __uint_as_float((uint32_t)p.scale[at] << 16)));
        if ((up & 0x7fff) == 0x7f80 && (p.scale[at] & 0x7fff) != 0x7f80) atomicOr(p.bad, 2);
        s |= up << (16 * h);
        if (p.zero) {
          z |= (uint32_t)p.zero[at] << (8 * h);
          if (p.zero[at] > 15) atomicOr(p.bad, 1);
        }
      }
      *reinterpret_cast<uint32_t*>(record + scale_in(w, t, k, lane)) = s;
      if (p.zero) *reinterpret_cast<uint16_t*>(record + zero_in(w, t, k, lane)) = (uint16_t)z;
    }
  }
}

// A lane's scales and zero points of a record.
__device__ __forceinline__ Meta load_meta(const Weights& w, const uint8_t* record, int t, int k, int g) {
  const uint32_t s = *reinterpret_cast<const uint32_t*>(record + scale_in(w, t, k, g));
  return w.zero ? meta_of<true>(s, *reinterpret_cast<const uint16_t*>(record + zero_in(w, t, k, g))) : meta_of<false>(s, 0);
}

__global__ void unpack_kernel(const Weights w, uint16_t* out) {
  const int64_t words = (int64_t)w.tiles * w.per_piece * 2 * 32, step = (int64_t)gridDim.x * blockDim.x;
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < words; i += step) {
    const int lane = (int)(i & 31), g = lane >> 2, c = lane & 3;
    const int64_t rest = i >> 5;
    const int t = (int)(rest % w.tiles), k0 = (int)(rest / w.tiles) * kBlockK;
    const uint8_t* record = w.records + record_at(w, t, k0);
    const uint4 v = *reinterpret_cast<const uint4*>(record + word_in(t, k0, lane));
    const uint32_t of[4] = {v.x, v.y, v.z, v.w};
    for (int j = 0; j < 4; ++j) {
      uint32_t a[4];
      widen(of[j], load_meta(w, record, t, k0 + 16 * j, g), a);
      for (int x = 0; x < 4; ++x) {
        const int row = row_of(w, t, g + (x & 1) * 8), k = k0 + 16 * j + 4 * c + (x >> 1) * 2;
        if (row < 0 || k >= w.width) continue;
        out[(int64_t)row * w.width + k] = (uint16_t)a[x];
        out[(int64_t)row * w.width + k + 1] = (uint16_t)(a[x] >> 16);
      }
    }
  }
}

// ------------------------------------------------------------------ few rows
__device__ __forceinline__ void mma(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// NT tiles of 8 rows of x; a block has TILES tiles of the weights (of a gated projection the gate's and the same of up),
// its WARPS warps every so manieth record, U records at a time, whose loads are all under way before the first is used;
// the first of them before the kernel in front has ended, since nobody writes weights. GROUPS of scales a record.
// Bound by the chain of loads, widening (13 operations a word of 8 weights) and products of a block, with nothing saturated (3
// rows, 2048 to 50001: half of the issue slots, 3 TB/s of DRAM in ncu, warps waiting for loads), and by how many blocks an SM
// holds: three of 8 warps, even where registers spill for it (us with that bound and without: 3 rows, 2048 to
// 50001 13.6 and 15.5; 1 row, 8192 to 28672 in groups of 64 26.1 and 29.0; 2 rows, 6144 to 12288 in groups of 32 12.6 and
// 16.6), but for 4 tiles with zero points of small groups (16.9 becomes 20.3); two of 16 with 2 tiles; with 1 the compiler
// does better unbound (2.4 and 2.6).
template <int NT, int WARPS, int TILES, int GROUPS, bool ZERO>
constexpr int kBlocksAnSm = NT > 1 || TILES == 1 ? 0 : WARPS == 16 ? 2 : TILES == 4 && ZERO && GROUPS > 1 ? 2 : 3;

template <int NT, int WARPS, int TILES, int U, int GROUPS, bool ZERO>
__global__ void __launch_bounds__(WARPS * 32, kBlocksAnSm<NT, WARPS, TILES, GROUPS, ZERO>) few_rows_kernel(const __grid_constant__ ApplyParams p) {
  __shared__ float part[WARPS][TILES * kTileRows][8 * NT + 1];
  const Weights& w = p.w;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int t0 = blockIdx.x * TILES;
  const uint8_t* words = w.records + record_at(w, t0, 0) + word_in(t0, 0, lane);
  const uint8_t* scales = w.records + record_at(w, t0, 0) + scale_in(w, t0, 0, g);
  const uint8_t* zeros = w.records + record_at(w, t0, 0) + zero_in(w, t0, 0, g);
  // a lane without a row of x takes the last again: its columns of the products are left out
  const uint16_t* x_row[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) x_row[n] = p.x + (int64_t)min(n * 8 + g, p.rows - 1) * p.x_row + 4 * c;
  ptx::pdl_trigger();
  float acc[TILES][NT][4] = {};
  for (int first = warp; first < w.per_piece; first += WARPS * U) {
    uint4 word[U][TILES][2];
    uint32_t scale[U][TILES][GROUPS], zero[U][TILES][GROUPS];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t at = (int64_t)min(first + u * WARPS, w.per_piece - 1) * w.bytes;   // past the last: it again, its scales and x as zeros
#pragma unroll
      for (int t = 0; t < TILES; ++t) {
        word[u][t][0] = *reinterpret_cast<const uint4*>(words + at + t * 512);
        word[u][t][1] = *reinterpret_cast<const uint4*>(words + at + t * 512 + 4096);
#pragma unroll
        for (int i = 0; i < GROUPS; ++i) {
          const bool past = u > 0 && first + u * WARPS >= w.per_piece;
          scale[u][t][i] = past ? 0 : *reinterpret_cast<const uint32_t*>(scales + at + t * 32 + i * kRecordScales);
          zero[u][t][i] = ZERO ? *reinterpret_cast<const uint16_t*>(zeros + at + t * 16 + i * kRecordZeros) : 0;
        }
      }
    }
    if (first == warp) ptx::pdl_wait();
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = (first + u * WARPS) * kRecordK;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint2 x[NT][4];
        const int k0 = k + h * kBlockK;
        if (k0 + kBlockK <= w.width) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) x[n][j] = *reinterpret_cast<const uint2*>(x_row[n] + k0 + 16 * j);
        } else {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              x[n][j] = k0 + 16 * j < w.width ? *reinterpret_cast<const uint2*>(x_row[n] + k0 + 16 * j) : make_uint2(0, 0);
        }
#pragma unroll
        for (int t = 0; t < TILES; ++t) {
          const uint4 v = word[u][t][h];
          const uint32_t four[4] = {v.x, v.y, v.z, v.w};
          Meta m;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            constexpr int kSteps = 8 / GROUPS;       // of 16 inputs, a group
            if ((h * 4 + j) % kSteps == 0 || j == 0) m = meta_of<ZERO>(scale[u][t][(h * 4 + j) / kSteps], zero[u][t][(h * 4 + j) / kSteps]);
            uint32_t a[4];
            widen(four[j], m, a);
#pragma unroll
            for (int n = 0; n < NT; ++n) mma(acc[t][n], a, x[n][j].x, x[n][j].y);
          }
        }
      }
    }
  }
  ptx::pdl_wait();                                   // a warp without records has not waited yet
#pragma unroll
  for (int t = 0; t < TILES; ++t)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) part[warp][t * kTileRows + g + (i >> 1) * 8][n * 8 + 2 * c + (i & 1)] = acc[t][n][i];
  __syncthreads();
  constexpr int kAll = TILES * kTileRows;
  const int per = w.gated ? kAll / 2 : kAll;
  for (int i = threadIdx.x; i < per * p.rows; i += WARPS * 32) {
    const int f = i & (per - 1), r = i / per;        // per is a power of two
    const int n = blockIdx.x * per + f;
    if (n >= w.outs) continue;
    const int at = w.gated ? (f >> 4) * 32 + (f & 15) : f;
    float y = 0.f;
#pragma unroll
    for (int k = 0; k < WARPS; ++k) y += part[k][at][r];
    if (TILES > 1 && w.gated) {
      float up = 0.f;
#pragma unroll
      for (int k = 0; k < WARPS; ++k) up += part[k][(at + kTileRows) & (kAll - 1)][r];
      y = silu(y) * up;
    }
    if (p.f32) finish<float>(p, r, n, 1, &y);
    else finish<__nv_bfloat16>(p, r, n, 1, &y);
  }
}

template <int NT, int WARPS, int TILES, int U, int GROUPS>
cudaError_t launch_few(const ApplyParams& p, cudaStream_t s) {
  const dim3 grid(p.w.tiles / TILES);
  return p.w.zero ? launch_as(few_rows_kernel<NT, WARPS, TILES, U, GROUPS, true>, grid, 1, 1, true, WARPS * 32, 0, s, p)
                  : launch_as(few_rows_kernel<NT, WARPS, TILES, U, GROUPS, false>, grid, 1, 1, true, WARPS * 32, 0, s, p);
}
template <int NT, int WARPS, int TILES, int U>
cudaError_t launch_few(const ApplyParams& p, cudaStream_t s) {
  return p.w.groups == 1 ? launch_few<NT, WARPS, TILES, U, 1>(p, s)
                         : p.w.groups == 2 ? launch_few<NT, WARPS, TILES, U, 2>(p, s) : launch_few<NT, WARPS, TILES, U, 4>(p, s);
}
// Nine to sixteen rows: two fragments a word, and no tensor memory to fill, win while the weights are few. (Records of
// 4 MB: 3.3 to 3.7 us here, 5.8 to 6.1 in the other kernel; of 6 MB 6.6 and 8.1; of 13 MB 8.7 to 9.5 and 8.6; of 34 MB 18
// to 20 and 14.)
constexpr int kFewRows = 8, kSomeRows = 16;
constexpr int64_t kSomeBytes = 8 << 20;
// Up to 8 rows: as many warps a block as leaves one round of blocks, for the more of them the sooner a block ends; where
// there are many rounds, more of the weights a block, so that x is read less often. Measured, us (16 warps and 1 tile; 16
// and 2; 8, 2 and two records at a time; 8 and 4): 1 row, 2048 to 4096 2.4, 3.1, 3.6, 3.8; 4 rows, 6144 to 2048 4.5, 6.0,
// 5.7, 8.1; 8 rows, 8192 to 8192 15.5, 10.3, 14.4, 21.9; 5 rows, 2048 to 2 x 6144 gated -, 5.1, 4.4, 7; 5 rows, 1024
// to 12288 (a record for each of 8 warps) -, 4.0, 4.4, -; 3 rows, 4096 to 16384 -, 10.6, 12.8, 12.8, to 20480 -, 13.3, 13.7,
// 13.1; 1 row, 8192 to 28672 34.1, 26.6, 26.2, 24.3; 3 rows, 2048 to 50001 21.2, 16.4, 15.2, 13.8.
cudaError_t launch_few_rows(const ApplyParams& p, cudaStream_t s) {
  if (p.rows > kFewRows) return launch_few<2, 16, 2, 1>(p, s);
  const int pairs = p.w.tiles / 2;                   // blocks of two tiles; an SM holds 2 of 16 warps, 3 of 8
  if (pairs * 2 <= 304 && !p.w.gated) return launch_few<1, 16, 1, 1>(p, s);
  if (pairs <= 304) return launch_few<1, 16, 2, 1>(p, s);
  if (pairs <= 456 && p.w.per_piece > 8) return launch_few<1, 8, 2, 2>(p, s);
  if (pairs <= 608) return launch_few<1, 16, 2, 1>(p, s);        // two rounds
  return launch_few<1, 8, 4, 1>(p, s);
}

bool takes_few(const ApplyParams& p) {
  return p.rows <= kFewRows || (p.rows <= kSomeRows && (int64_t)(p.w.tiles / kPadTiles) * p.w.per_piece * p.w.bytes <= kSomeBytes);
}

// ------------------------------------------------------------------ checks
int check_desc(const cp_linear_desc* d, Weights* w) {
  if (!d || !d->q || !d->scale || d->features < 1 || d->width < 1 || d->group < 1) return CP_ERR_INVALID_ARG;
  if (d->group != 32 && d->group != 64 && d->group != 128) return CP_ERR_UNSUPPORTED;
  if (d->width % d->group || (d->gated && d->features % 2) || d->timeout_ns < 0) return CP_ERR_INVALID_ARG;
  if (d->width > 1 << 20 || d->features > 1 << 24) return CP_ERR_UNSUPPORTED;
  w->features = d->features;
  w->width = d->width;
  w->group_shift = d->group == 32 ? 5 : d->group == 64 ? 6 : 7;
  w->gated = d->gated != 0;
  w->outs = d->gated ? d->features / 2 : d->features;
  const int tiles = (w->outs + kTileRows - 1) / kTileRows * (d->gated ? 2 : 1);
  w->tiles = (tiles + kPadTiles - 1) / kPadTiles * kPadTiles;
  w->zero = d->zero != nullptr;
  w->per_piece = (d->width + kRecordK - 1) / kRecordK;
  w->groups = kRecordK / d->group;
  w->bytes = kRecordWords + w->groups * (kRecordScales + (w->zero ? kRecordZeros : 0));
  return CP_OK;
}

int check_args(const Weights& w, const cp_linear_args* a, ApplyParams* p) {
  if (!a || !a->x || !a->out || a->rows < 1) return CP_ERR_INVALID_ARG;
  if (a->out_dtype != CP_OUT_BF16 && a->out_dtype != CP_OUT_F32) return CP_ERR_INVALID_ARG;
  if (a->rows > 65535) return CP_ERR_UNSUPPORTED;
  p->w = w;
  p->x = static_cast<const uint16_t*>(a->x);
  p->out = a->out;
  p->add = a->add;
  p->rows = a->rows;
  p->f32 = a->out_dtype == CP_OUT_F32;
  p->x_row = a->x_stride ? a->x_stride : w.width;
  p->out_row = a->out_stride ? a->out_stride : w.outs;
  p->add_row = a->add_stride ? a->add_stride : w.outs;
  if (p->x_row < 0 || p->out_row < 0 || p->add_row < 0 || (a->rows > 1 && p->x_row < w.width)) return CP_ERR_INVALID_ARG;
  const int64_t most = (int64_t)1 << 39;                       // what a tensor map's strides reach
  if (p->x_row >= most || p->out_row > most || p->add_row > most) return CP_ERR_UNSUPPORTED;
  if (p->x_row % 8 || !aligned16(a->x)) return CP_ERR_UNSUPPORTED;
  const uintptr_t es = a->out_dtype == CP_OUT_BF16 ? 2 : 4;
  if (reinterpret_cast<uintptr_t>(a->out) % es || reinterpret_cast<uintptr_t>(a->add) % es) return CP_ERR_UNSUPPORTED;
  if (!lie_apart(w.outs, {{a->rows, p->out_row}})) return CP_ERR_INVALID_ARG;
  const auto four = [es](const void* at, int64_t row) { return reinterpret_cast<uintptr_t>(at) % (4 * es) == 0 && row % 4 == 0; };
  p->by_four = four(a->out, p->out_row) && (!a->add || four(a->add, p->add_row));
  return CP_OK;
}

}  // namespace

extern "C" {

int cp_linear_check(const cp_linear_desc* desc, const cp_linear_args* args) {
  Weights w{};
  const int st = check_desc(desc, &w);
  if (st || !args) return st;
  ApplyParams p{};
  return check_args(w, args, &p);
}

int cp_linear_create(const cp_linear_desc* desc, int device, cp_linear** out) {
  if (!out) return CP_ERR_INVALID_ARG;
  *out = nullptr;
  PackParams p{};
  Weights& w = p.w;
  int st = check_desc(desc, &w);
  if (st) return st;
  if ((st = check_device(device))) return st;
  DeviceGuard guard(device);
  for (const void* ptr : {desc->q, desc->scale, desc->zero})
    if (ptr && !on_device(ptr, device)) return CP_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(desc->scale) % 2) return CP_ERR_UNSUPPORTED;
  cp_linear* l = new (std::nothrow) cp_linear();
  if (!l) return CP_ERR_NOMEM;
  l->device = device;
  const size_t bytes = (size_t)(w.tiles / kPadTiles) * w.per_piece * w.bytes;
  if (cudaMalloc(&l->memory, bytes + 256) != cudaSuccess) {          // records are multiples of 128 bytes
    cudaGetLastError();
    delete l;
    return CP_ERR_NOMEM;
  }
  p.out = static_cast<uint8_t*>(l->memory);
  p.bad = reinterpret_cast<int*>(p.out + bytes);
  p.q = static_cast<const uint8_t*>(desc->q);
  p.scale = static_cast<const uint16_t*>(desc->scale);
  p.zero = static_cast<const uint8_t*>(desc->zero);
  w.records = p.out;
  l->w = w;
  l->status = p.bad + 1;
  l->timeout_ns = desc->timeout_ns ? desc->timeout_ns : 2000000000ll;
  l->stall = desc->debug_stall;
  int bad = 0;
  // what the caller's streams still write into the arrays is waited for
  bool ok = cudaDeviceSynchronize() == cudaSuccess && cudaMemset(p.bad, 0, 8) == cudaSuccess && prepare_many_rows() == cudaSuccess;
  if (ok) {
    pack_kernel<<<1216, 256>>>(p);
    ok = cudaGetLastError() == cudaSuccess && cudaMemcpy(&bad, p.bad, 4, cudaMemcpyDeviceToHost) == cudaSuccess;
  }
  if (!ok || bad) {
    cp_linear_destroy(l);
    return bad & 1 ? CP_ERR_INVALID_ARG : bad ? CP_ERR_UNSUPPORTED : CP_ERR_CUDA;
  }
  *out = l;
  return CP_OK;
}

void cp_linear_destroy(cp_linear* l) {
  if (!l) return;
  {
    DeviceGuard g(l->device);
    cudaDeviceSynchronize();
    cudaFree(l->memory);
  }
  delete l;
}

int cp_linear_apply(cp_linear* l, const cp_linear_args* args, cp_stream_t stream) {
  if (!l) return CP_ERR_INVALID_ARG;
  ApplyParams p{};
  const int st = check_args(l->w, args, &p);
  if (st) return st;
  p.status = l->status;
  p.timeout_ns = l->timeout_ns;
  p.stall = l->stall;
  DeviceGuard g(l->device);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return cuda_err(takes_few(p) ? launch_few_rows(p, s) : launch_many_rows(p, s));
}

int cp_linear_status(cp_linear* l) {
  if (!l) return CP_ERR_INVALID_ARG;
  DeviceGuard g(l->device);
  if (cudaDeviceSynchronize() != cudaSuccess) return CP_ERR_CUDA;
  int32_t v = 0;
  if (cudaMemcpy(&v, l->status, 4, cudaMemcpyDeviceToHost) != cudaSuccess) return CP_ERR_CUDA;
  return v;
}

int cp_linear_clear_status(cp_linear* l) {
  if (!l) return CP_ERR_INVALID_ARG;
  DeviceGuard g(l->device);
  if (cudaDeviceSynchronize() != cudaSuccess) return CP_ERR_CUDA;
  if (cudaMemset(l->status, 0, 4) != cudaSuccess) return CP_ERR_CUDA;
  return cuda_err(cudaDeviceSynchronize());
}

int cp_linear_unpack(cp_linear* l, void* out, cp_stream_t stream) {
  if (!l || !out) return CP_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(out) % 2) return CP_ERR_UNSUPPORTED;
  DeviceGuard g(l->device);
  unpack_kernel<<<1216, 256, 0, reinterpret_cast<cudaStream_t>(stream)>>>(l->w, static_cast<uint16_t*>(out));
  return cuda_err(cudaGetLastError());
}

}  // extern "C"
