// cp_linear.cuh -- projections with 4-bit weights: how the weights lie, and the
// arithmetic that the kernels share.
//
// Rows of the weights are taken 16 at a time (a tile), inputs 64 at a time (a
// block). Lane 4 g + c of a warp holds rows g and g + 8 of a tile, one 16-byte
// word a block: its 32-bit word j has inputs 16 j + 4 c .. + 3, nibbles 0 to 3
// the even ones of (row g: 0, row g + 8: 0, row g: 2, row g + 8: 2), nibbles 4
// to 7 the odd ones behind them. By four masks and shifts a word becomes the
// four registers of an A fragment of a 16 x 8 x 16 product (whose inputs stand
// in an order of their own: a sum over k does not mind, and a lane's part of x
// is 8 consecutive bytes); and the tensor memory's stores of 16 rows by 256
// bits want just these lanes and inputs, in their own order, so that x comes
// as it lies there. Both kernels thus read the same words.
//
// A gated projection's tiles alternate: 16 rows of the gate, the same of up.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "cp.h"
#include "cp_call.h"

namespace cp {
namespace linear {

constexpr int kTileRows = 16, kBlockK = 64;
constexpr int kPadTiles = 8;                 // tiles come in eights: 128 rows

struct Weights {
  const uint4* w;            // [tiles][blocks][32 lanes]
  const uint32_t* scale;     // [tiles][groups][8]: bf16 of row g | of row g + 8 << 16
  const uint16_t* zero;      // [tiles][groups][8]: zero points, a byte each; or null
  int features, width, group_shift, gated;
  int tiles, blocks, groups; // groups: all that the blocks span
  int outs;                  // results a row
};

struct ApplyParams {
  Weights w;
  int32_t* status;           // sticky
  long long timeout_ns;
  int stall;                 // test: the first load is left out
  const uint16_t* x;
  int64_t x_row, out_row, add_row;
  void* out;
  const void* add;
  int rows;
};

// The row of the weights that is row i of tile t, or -1 behind the last.
__host__ __device__ __forceinline__ int row_of(const Weights& w, int t, int i) {
  if (!w.gated) {
    const int n = t * kTileRows + i;
    return n < w.features ? n : -1;
  }
  const int n = (t >> 1) * kTileRows + i, half = w.features >> 1;
  return n < half ? (t & 1) * half + n : -1;
}

__device__ __forceinline__ uint32_t bf2_sub(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t bf2_mul(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// What a lane multiplies its two rows' weights with: pairs of the same number.
struct Meta {
  uint32_t s[2];   // scales of rows g and g + 8
  uint32_t z[2];   // 128 + zero point
};
__device__ __forceinline__ Meta meta_of(uint32_t scale, uint32_t zero) {
  Meta m;
  m.s[0] = __byte_perm(scale, 0, 0x1010);
  m.s[1] = __byte_perm(scale, 0, 0x3232);
  const uint32_t a = zero & 0xffu, b = zero >> 8;
  m.z[0] = 0x43004300u | a | a << 16;
  m.z[1] = 0x43004300u | b | b << 16;
  return m;
}
constexpr uint32_t kNoZero = 0x0808u;

// A word's eight weights as bf16: a nibble in the low bits of 128 is 128 + q
// exactly, the difference q - z is exact, the product is the one rounding.
__device__ __forceinline__ void widen(uint32_t w, const Meta& m, uint32_t* a) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    a[i] = bf2_mul(bf2_sub((w >> (4 * i) & 0x000f000fu) | 0x43004300u, m.z[i & 1]), m.s[i & 1]);
}

// The place of a lane's scales and zero points: of tile t, input k.
__device__ __forceinline__ int64_t meta_at(const Weights& w, int t, int k, int g) {
  return ((int64_t)t * w.groups + (k >> w.group_shift)) * 8 + g;
}

template <class T>
__device__ __forceinline__ float load_out(const void* p, int64_t i);
template <>
__device__ __forceinline__ float load_out<float>(const void* p, int64_t i) { return static_cast<const float*>(p)[i]; }
template <>
__device__ __forceinline__ float load_out<__nv_bfloat16>(const void* p, int64_t i) {
  return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}
__device__ __forceinline__ void store_out(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_out(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// Exact to fp32's rounding: the type of the result may be fp32.
__device__ __forceinline__ float silu(float x) { return x / (1.f + expf(-x)); }

// Many rows: cp_linear_rows.cu. Once per device, with it current: its shared memory.
cudaError_t prepare_many_rows();
cudaError_t launch_many_rows(const ApplyParams& p, bool f32, cudaStream_t s);

}  // namespace linear
}  // namespace cp
