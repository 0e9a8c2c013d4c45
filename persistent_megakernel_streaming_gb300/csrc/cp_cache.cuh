// cp_cache.cuh -- what the paged cache's kernels share: the cache's and the
// batch's view on the device, the look-ups with their bounds checks, and the
// element formats.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "cp.h"

namespace cp {
namespace cache {

constexpr int kMinExp = -110;    // smallest exponent of a stored scale (byte 17)

struct CacheView {
  uint8_t* k;
  uint8_t* v;
  uint8_t* ks;                          // scales (e4m3) or null
  uint8_t* vs;
  int64_t page_b, head_b, tok_b;        // bytes between pages, heads, positions
  int64_t sc_page, sc_head, sc_tok;     // the same of the scales
  int pages, heads, page_shift;         // page size 1 << page_shift
  int32_t* status;                      // sticky status word of the cache
};

struct BatchView {
  const int32_t* start;
  const int32_t* length;
  const int32_t* table;
  int64_t table_stride;
  int n, rows, width, max_new, max_len;
};

// One sequence of the batch as the kernels use it: rows row0 .. row0 + n - 1,
// len cached positions, row row0 + i at position first + i.
struct Seq {
  int row0, n, len, first;
};

__device__ __forceinline__ void set_status(int32_t* status, int code) { atomicCAS(status, 0, code); }

// Starts, lengths and row counts are device data: whatever they hold, the
// returned rows lie in [0, rows] and the positions in [0, max_len].
__device__ __forceinline__ Seq seq_of(const BatchView& b, int i, int32_t* status) {
  const int s0 = b.start[i], s1 = b.start[i + 1], l = b.length[i];
  Seq s;
  s.row0 = min(max(s0, 0), b.rows);
  const int end = min(max(s1, s.row0), b.rows);
  s.n = min(end - s.row0, b.max_new);
  s.len = min(max(l, 0), b.max_len);
  if (s.row0 != s0 || end != s1 || s.n != end - s.row0 || s.len != l) set_status(status, CP_ERR_DEVICE_BOUNDS);
  s.first = s.len - s.n;
  return s;
}

// Page of position `pos` in a table row of `width` entries, or -1: a position
// outside the table or a page outside the pool (run on the host by
// cp_test_slot too).
__host__ __device__ __forceinline__ int page_of(const int32_t* table, int width, int pages, int page_shift, int pos) {
  if (pos < 0 || (pos >> page_shift) >= width) return -1;
  const int p = table[pos >> page_shift];
  return (uint32_t)p < (uint32_t)pages ? p : -1;
}
// Byte offset of a position in K or V: 64-bit, a pool may pass 4 GB.
__host__ __device__ __forceinline__ int64_t slot_bytes(const CacheView& c, int page, int head, int pos) {
  return (int64_t)page * c.page_b + (int64_t)head * c.head_b + (int64_t)(pos & ((1 << c.page_shift) - 1)) * c.tok_b;
}
__host__ __device__ __forceinline__ int64_t slot_scale(const CacheView& c, int page, int head, int pos) {
  return (int64_t)page * c.sc_page + (int64_t)head * c.sc_head + (int64_t)(pos & ((1 << c.page_shift) - 1)) * c.sc_tok;
}

// 2^e for e in [-126, 127].
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }

__device__ __forceinline__ float bf_lo(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float bf_hi(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }
__device__ __forceinline__ uint32_t bf_pack(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t hf_pack(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two e4m3 bytes of the low 16 bits as fp16 (exact).
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)two));
  return r;
}
__device__ __forceinline__ void e4m3x4_f32(uint32_t four, float* f) {
  const uint32_t a = e4m3x2_f16x2(four & 0xffffu), b = e4m3x2_f16x2(four >> 16);
  const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&a));
  const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&b));
  f[0] = x.x; f[1] = x.y; f[2] = y.x; f[3] = y.y;
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// ------------------------------------------------------------------ attention
// How a call is cut up, from the host's bounds alone (so that a captured call
// keeps it): sequences of at most kStepRows rows a kv head go to the step
// kernel if it runs, the others to the chunk kernel. An item (a sequence, or a tile of its
// rows) whose visible positions are more than `chunk` is cut into parts of
// that many, each a block's; a last kernel joins the parts.
constexpr int kStepRows = 16;
constexpr int kSms = 152;

constexpr int kPairRows = 256;    // rows (times query heads) that a chunk block takes
constexpr int kStepAlign = 16, kChunkAlign = 128;   // where an item's parts may start

struct AttendPlan {
  int use_step, use_chunk;
  int step_chunk, step_parts;     // positions a part, most parts of an item
  int step_wide;                  // items of more than 8 rows
  int step_cluster;               // the parts of a step item are one cluster's blocks, which join them
  int chunk_chunk, chunk_parts;
  int chunk_cluster;              // the same of a chunk item's
  int chunk_span;                 // positions that the parts were made for
  int chunk_coarser;              // the kernel looks at the lengths and may take fewer, longer parts
};
// Nanoseconds of a chunk call: a tile of 128 positions 1700 (heads of 64: 1200), a block's start and end 9000.
constexpr int kTileNs128 = 1700, kTileNs64 = 1200, kBlockNs = 9000;
__host__ __device__ __forceinline__ float chunk_rounds_ns(int64_t blocks, int tiles, int head_dim) {
  return (float)((blocks + kSms - 1) / kSms) * (float)((int64_t)tiles * (head_dim == 128 ? kTileNs128 : kTileNs64) + kBlockNs);
}
AttendPlan plan_attend(const BatchView& b, int kv_heads, int q_heads, int head_dim, bool e4m3, bool causal,
                       int window);
// Most parts of an item that go through the workspace.
inline int kept_parts(const AttendPlan& a) {
  const int step = a.step_cluster ? 0 : a.step_parts;
  const int chunk = a.chunk_cluster ? 0 : a.chunk_parts;
  return step > chunk ? step : chunk;
}
// An upper bound of the chunk kernel's items a kv head: whole pairs and one more a sequence.
inline int64_t chunk_pairs(const BatchView& b, int group) {
  return (int64_t)b.rows * group / kPairRows + (b.n < b.rows ? b.n : b.rows);
}
size_t attend_workspace(const AttendPlan& a, const BatchView& b, int q_heads, int head_dim);

struct AttendParams {
  CacheView c;
  BatchView b;
  AttendPlan a;
  const uint16_t* q;
  uint16_t* out;
  float* part_o;                          // [parts][rows][q_heads][D]: a part's softmax average of v
  float* part_lse;                        // [parts][rows][q_heads]: log2 of its sum of exponentials
  int* coarser;                           // the chunk kernel's own choice of positions a part
  int64_t q_row, q_head, o_row, o_head;   // element strides
  int group;                              // query heads per kv head
  uint32_t magic;                         // x / group is x * magic >> 16, for x below 320
  int q_heads;
  float scale_log2;                       // scale * log2(e)
  int causal, window;
  int64_t timeout_ns;
  int stall;                              // test: the first load is left out
};

// Positions [lo, hi) that the row at position `pos` sees.
__device__ __forceinline__ void visible(const AttendParams& p, int pos, int len, int* lo, int* hi) {
  *hi = p.causal ? min(pos + 1, len) : len;
  *lo = p.window > 0 && pos >= p.window ? pos - p.window + 1 : 0;
}

// The positions some row of an item sees, from its first and last row's
// positions; `base` is where its parts start: a multiple of 16 for the step
// kernel (16 positions never cross a page), of its 128-position tile for the
// chunk kernel.
struct Range {
  int lo, hi, base;
};
__device__ __forceinline__ Range item_range(const AttendParams& p, int pos_first, int pos_last, int len, int align) {
  Range r;
  int d;
  visible(p, pos_first, len, &r.lo, &d);
  visible(p, pos_last, len, &d, &r.hi);
  r.base = min(r.lo, max(r.hi, 0)) & ~(align - 1);
  return r;
}
__device__ __forceinline__ int parts_of(const Range& r, int chunk) {
  return r.hi > r.base ? (r.hi - r.base - 1) / chunk + 1 : 0;     // a part may be nearly as long as positions reach
}

// Once per device, with it current: the kernels' shared-memory sizes.
cudaError_t prepare_attend();
cudaError_t prepare_attend_chunk();
// The chunk kernel reads pages through tensor maps of K and V (head_dim,
// position in the page, head, page).
struct CacheMaps {
  CUtensorMap k, v;
};
cudaError_t launch_attend_chunk(const AttendParams& p, const CacheMaps& maps, int head_dim, bool e4m3, cudaStream_t s);
cudaError_t launch_attend(const AttendParams& p, const CacheMaps& maps, int head_dim, bool e4m3, cudaStream_t s);

}  // namespace cache
}  // namespace cp
