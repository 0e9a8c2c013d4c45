// cp_linear.cu -- projections with 4-bit weights: the C ABI (checks, layout of
// the weights, launches) and the kernel for up to 16 rows.
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
  return meta_of(s, w.zero ? *reinterpret_cast<const uint16_t*>(record + zero_in(w, t, k, g)) : kNoZero);
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
constexpr int kWarps = 8;

__device__ __forceinline__ void mma(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// NT tiles of 8 rows of x; a block has two tiles of the weights, of a gated projection the gate's and the same of up,
// its warps every eighth block of inputs.
template <class T, int NT>
__global__ void __launch_bounds__(kWarps * 32) few_rows_kernel(const __grid_constant__ ApplyParams p) {
  __shared__ float part[kWarps][2 * kTileRows][8 * NT + 1];
  const Weights& w = p.w;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int t0 = blockIdx.x * 2, row0 = blockIdx.y * 8 * NT;
  ptx::pdl_trigger();
  ptx::pdl_wait();
  float acc[2][NT][4] = {};
  for (int b = warp; b * kBlockK < w.width; b += kWarps) {
    uint2 x[NT][4];
    const int k = b * kBlockK;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int r = row0 + n * 8 + g;
      const uint16_t* src = p.x + (int64_t)r * p.x_row + k + 4 * c;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        x[n][j] = r < p.rows && k + 16 * j < w.width ? *reinterpret_cast<const uint2*>(src + 16 * j) : make_uint2(0, 0);
    }
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const uint8_t* record = w.records + record_at(w, t0 + t, k);
      const uint4 v = *reinterpret_cast<const uint4*>(record + word_in(t0 + t, k, lane));
      const uint32_t words[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int h = 0; h < 2; ++h) {                // groups of 32 have two in a block
        const Meta m = load_meta(w, record, t0 + t, k + 32 * h, g);
#pragma unroll
        for (int j = 2 * h; j < 2 * h + 2; ++j) {
          uint32_t a[4];
          widen(words[j], m, a);
#pragma unroll
          for (int n = 0; n < NT; ++n) mma(acc[t][n], a, x[n][j].x, x[n][j].y);
        }
      }
    }
  }
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) part[warp][t * kTileRows + g + (i >> 1) * 8][n * 8 + 2 * c + (i & 1)] = acc[t][n][i];
  __syncthreads();
  const int per = w.gated ? kTileRows : 2 * kTileRows;
  for (int i = threadIdx.x; i < per * 8 * NT; i += kWarps * 32) {
    const int f = i % per, r = i / per;
    const int n = blockIdx.x * per + f;
    if (n >= w.outs || row0 + r >= p.rows) continue;
    float y = 0.f, u = 0.f;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) y += part[k][f][r];
    if (w.gated) {
#pragma unroll
      for (int k = 0; k < kWarps; ++k) u += part[k][kTileRows + f][r];
      y = silu(y) * u;
    }
    if (p.add) y += load_out<T>(p.add, (row0 + r) * p.add_row + n);
    store_out(static_cast<T*>(p.out) + (row0 + r) * p.out_row + n, y);
  }
}

template <class T>
cudaError_t launch_few_rows(const ApplyParams& p, cudaStream_t s) {
  const dim3 grid(p.w.tiles / 2, p.rows <= 8 ? 1 : (p.rows + 15) / 16);
  return p.rows <= 8 ? launch_as(few_rows_kernel<T, 1>, grid, 1, 1, true, kWarps * 32, 0, s, p)
                     : launch_as(few_rows_kernel<T, 2>, grid, 1, 1, true, kWarps * 32, 0, s, p);
}

constexpr int kFewRows = 16;

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
  p->x_row = a->x_stride ? a->x_stride : w.width;
  p->out_row = a->out_stride ? a->out_stride : w.outs;
  p->add_row = a->add_stride ? a->add_stride : w.outs;
  if (p->x_row < 0 || p->out_row < 0 || p->add_row < 0) return CP_ERR_INVALID_ARG;
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
  const bool f32 = args->out_dtype == CP_OUT_F32;
  if (p.rows > kFewRows) return cuda_err(launch_many_rows(p, f32, s));
  return cuda_err(f32 ? launch_few_rows<float>(p, s) : launch_few_rows<__nv_bfloat16>(p, s));
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
