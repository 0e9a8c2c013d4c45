// cp_linear.cuh -- projections with 4-bit weights: how the weights lie, and the
// arithmetic that the kernels share.
//
// Rows of the weights are taken 16 at a time (a tile), inputs 64 at a time (a
// block). Lane 4 g + c of a warp holds rows g and g + 8 of a tile and inputs
// 16 c .. 16 c + 15 of a block, one 16-byte word a block: 32-bit word j has
// inputs 16 c + 4 j .. + 3, nibbles 0 to 3 the even ones of (row g: 0, row
// g + 8: 0, row g: 2, row g + 8: 2), nibbles 4 to 7 the odd ones behind them.
// A word thus becomes, by four masks and shifts, the four registers of an A
// fragment of a 16 x 8 x 16 product whose inputs stand in an order of their
// own (a sum over k does not mind), while the lane's part of x is 32
// consecutive bytes. The tensor memory's 16-row stores have the same lanes, so
// that the kernel for many rows reads the same words.
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

// Exact to fp32's rounding: the type of the result may be fp32.
__device__ __forceinline__ float silu(float x) { return x / (1.f + expf(-x)); }

}  // namespace linear
}  // namespace cp
