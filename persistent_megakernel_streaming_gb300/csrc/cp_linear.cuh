// cp_linear.cuh -- projections with 4-bit weights: how the weights lie, and the
// arithmetic that the kernels share.
//
// Rows of the weights are taken 16 at a time (a tile), inputs 64 at a time (a
// block). Lane 4 g + c of a warp holds rows g and g + 8 of a tile, one 16-byte
// word a block: its 32-bit word j has inputs 16 j + 4 c .. + 3, nibbles 0 to 3
// the even ones of (row g: 0, row g + 8: 0, row g: 2, row g + 8: 2), nibbles 4
// to 7 the odd ones behind them. By masks a word becomes the four registers of
// an A fragment of a 16 x 8 x 16 product (whose inputs stand
// in an order of their own: a sum over k does not mind, and a lane's part of x
// is 8 consecutive bytes); and the tensor memory's stores of 16 rows by 256
// bits want just these lanes and inputs, in their own order, so that x comes
// as it lies there. Both kernels thus read the same words.
//
// A gated projection's tiles alternate: 16 rows of the gate, the same of up.
// Eight tiles make a piece. What a piece has for two blocks lies together, a
// record that one copy brings in: words, scales, zero points.
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

constexpr int kRecordK = 2 * kBlockK;        // inputs of a record
constexpr int kRecordWords = 8192;           // bytes: [2 blocks][8 tiles][32 lanes] words,
constexpr int kRecordScales = 256;           // then [groups][8 tiles][8]: bf16 64 * scale of row g | of row g + 8 << 16,
constexpr int kRecordZeros = 128;            // then the same: zero points, a byte each
constexpr int kMostRecord = kRecordWords + 4 * (kRecordScales + kRecordZeros);

struct Weights {
  const uint8_t* records;    // [tiles / 8][records of a piece]
  int features, width, group_shift, gated, zero;
  int tiles, per_piece;      // per_piece: records of a piece
  int groups;                // of a record: 1, 2 or 4
  int bytes;                 // of a record
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
  int f32;                   // out's type: fp32, or bf16
  int by_four;               // rows of out and add start where four results can be written at once
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

__device__ __forceinline__ uint32_t bf2_fma(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
__device__ __forceinline__ uint32_t bf2_mul(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// What a lane widens its two rows' weights with: pairs of the same number.
struct Meta {
  uint32_t s[2];   // 64 times the scales of rows g and g + 8
  uint32_t z[2];   // minus the zero points, over 64
};
constexpr uint32_t kUp127 = 0x7f007f00u, kUp123 = 0x7d007d00u, kDown127 = 0xff00ff00u;    // bf16 2^127, 2^123, -2^127
constexpr uint32_t kEight = 0xbe00be00u;     // -8 / 64: where there are no zero points
template <bool ZERO>
__device__ __forceinline__ Meta meta_of(uint32_t scale, uint32_t zero) {
  Meta m;
  m.s[0] = __byte_perm(scale, 0, 0x1010);
  m.s[1] = __byte_perm(scale, 0, 0x3232);
  m.z[0] = ZERO ? bf2_mul(__byte_perm(zero, 0, 0x4040), kDown127) : kEight;
  m.z[1] = ZERO ? bf2_mul(__byte_perm(zero, 0, 0x4141), kDown127) : kEight;
  return m;
}

// A word's eight weights as bf16. A nibble in a bf16's lowest bits is q 2^-133, in the next four q 2^-129: below the
// second smallest exponent a float is as a whole number, linear in its bits. One fused operation makes (q - z) / 64 of
// it, exactly; the product with 64 times the scale is the one rounding. (128 + q by setting bits, and a difference,
// takes two shifts and four operations of the integer pipe more a word: it bounds the kernels.)
__device__ __forceinline__ void widen(uint32_t w, const Meta& m, uint32_t* a) {
  const uint32_t v = w >> 8;
  a[0] = bf2_mul(bf2_fma(w & 0x000f000fu, kUp127, m.z[0]), m.s[0]);
  a[1] = bf2_mul(bf2_fma(w & 0x00f000f0u, kUp123, m.z[1]), m.s[1]);
  a[2] = bf2_mul(bf2_fma(v & 0x000f000fu, kUp127, m.z[0]), m.s[0]);
  a[3] = bf2_mul(bf2_fma(v & 0x00f000f0u, kUp123, m.z[1]), m.s[1]);
}

// The record of tile t and input k, and in it the places of a lane's word, and of its scales and zero points.
__host__ __device__ __forceinline__ int64_t record_at(const Weights& w, int t, int k) {
  return ((int64_t)(t >> 3) * w.per_piece + k / kRecordK) * w.bytes;
}
__host__ __device__ __forceinline__ int word_in(int t, int k, int lane) {
  return (k / kBlockK & 1) * 4096 + (t & 7) * 512 + lane * 16;
}
__host__ __device__ __forceinline__ int scale_in(const Weights& w, int t, int k, int g) {
  return kRecordWords + (k % kRecordK >> w.group_shift) * kRecordScales + ((t & 7) * 8 + g) * 4;
}
__host__ __device__ __forceinline__ int zero_in(const Weights& w, int t, int k, int g) {
  return kRecordWords + w.groups * kRecordScales + (k % kRecordK >> w.group_shift) * kRecordZeros + ((t & 7) * 8 + g) * 2;
}

template <class T>
__device__ __forceinline__ float load_out(const void* p, int64_t i);
template <>
__device__ __forceinline__ float load_out<float>(const void* p, int64_t i) { return static_cast<const float*>(p)[i]; }
template <>
__device__ __forceinline__ float load_out<__nv_bfloat16>(const void* p, int64_t i) {
  return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}
__device__ __forceinline__ void load_four(const float* p, float* v) {
  const float4 x = *reinterpret_cast<const float4*>(p);
  v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
}
__device__ __forceinline__ void load_four(const __nv_bfloat16* p, float* v) {
  const uint2 x = *reinterpret_cast<const uint2*>(p);
  v[0] = __uint_as_float(x.x << 16); v[1] = __uint_as_float(x.x & 0xffff0000u);
  v[2] = __uint_as_float(x.y << 16); v[3] = __uint_as_float(x.y & 0xffff0000u);
}
__device__ __forceinline__ void store_four(float* p, const float* v) { *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]); }
__device__ __forceinline__ void store_four(__nv_bfloat16* p, const float* v) {
  __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<uint32_t*>(&a), *reinterpret_cast<uint32_t*>(&b));
}
__device__ __forceinline__ void store_out(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_out(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// x / (1 + exp(-x)) to a few of fp32's half steps (the result may be fp32): the rounding of the exponent's product with
// log2(e) is put back as a factor, and the quotient is one approximate reciprocal. Where the exponential passes 2^64 the 1
// is nothing beside it, and the powers of two that would take it, or its reciprocal, out of range come last: results of
// gates down to -91.8 are normal numbers, those of -103 the last that are not 0 (320 rows, 2048 to 2 x 6144: 14.7 -> 14.9 us).
__device__ __forceinline__ float silu(float x) {
  const float y = fminf(fmaxf(-x, -200.f), 200.f);           // past these the result is x, or 0
  const float t = __fmul_rn(y, 1.44269502f), rest = __fmaf_rn(y, 1.92596303e-8f, __fmaf_rn(y, 1.44269502f, -t));
  const bool far = t > 64.f;
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(far ? t - 64.f : t));
  e = __fmul_rn(e, __fmaf_rn(rest, 0.693147182f, 1.f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(far ? e : 1.f + e));
  return __fmul_rn(x * r, far ? 0x1p-64f : 1.f);
}

// Results of one row from `feature` on, `n` of them (up to four): the residual added, rounded, written.
template <class T>
__device__ __forceinline__ void finish(const ApplyParams& p, int row, int feature, int n, float* y) {
  T* out = static_cast<T*>(p.out) + (int64_t)row * p.out_row + feature;
  const T* add = static_cast<const T*>(p.add) + (int64_t)row * p.add_row + feature;
  if (p.by_four && n == 4) {
    if (p.add) {
      float r[4];
      load_four(add, r);
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] += r[i];
    }
    store_four(out, y);
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < n) store_out(out + i, p.add ? y[i] + load_out<T>(add, i) : y[i]);
}

// Many rows: cp_linear_rows.cu. Once per device, with it current: its shared memory.
cudaError_t prepare_many_rows();
cudaError_t launch_many_rows(const ApplyParams& p, cudaStream_t s);

}  // namespace linear
}  // namespace cp
