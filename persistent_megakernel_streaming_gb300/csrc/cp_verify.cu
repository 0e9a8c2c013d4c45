// cp_verify.cu -- verification of drafted tokens against the target's logits.
//
// Two launches. The first reads every logit once and leaves the maximum and the
// sum of exponentials of each piece of a row. The second, a cluster for each
// sequence, joins them, settles which drafted tokens are taken, and draws the
// token behind them from one row: there it sums again, in 64-bit fixed point,
// so that the draw does not depend on the order of the sums. Over a small
// vocabulary the second reads the rows itself, and is the only one (but for a
// look through the starts of many sequences).
//
// Of 48 sequences of 7 drafted tokens over 131075 fp32 logits (378 MB) the
// first takes 61 us (6.2 TB/s), the second 34 to 38 behind it: 8 to settle what
// is taken, 12 for the exponentials, 4 to add them up, 6 for the weights.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cfloat>
#include <cstring>

#include "cp.h"
#include "cp_call.h"
#include "cp_ptx.cuh"

using namespace cp;

namespace {

// A piece of a row: its largest scaled logit, the sum of exp(x - m), and, of a greedy row, the largest's first place.
struct Piece {
  float m, s;
  int arg, pad;
};

constexpr int kStatThreads = 128, kPer = 32;
constexpr int kPiece = kStatThreads * kPer;      // logits of a row that a block takes; the last up to 16 bytes a thread more
// Three blocks an SM: the draw waits (for loads, barriers, other blocks) more than it computes. With 512 threads a block and
// two an SM 48 sequences over 131075 took 51 us behind the sums, with these 40. Reading small rows itself, it takes 512
// for up to as many sequences as SMs whose rows 256 would read in two turns (two warps a row): us with 512 and 256 for 1
// sequence of 4 drafted tokens over 4096 9.0 and 10.7, for 152 of 5 over 2048 9.0 and 9.7, for 64 of 3 over 4096 9.9 and 9.3,
// for 256 of 5 over 2048 18.9 and 15.7.
constexpr int kTokenThreads = 256, kWideThreads = 512;
constexpr int kWideMost = 152;
constexpr int kRowsKept = 32;                    // rows of a sequence whose pieces are joined once
constexpr int kMostCluster = 16, kMostSums = kMostCluster * kTokenThreads / 32;
// Vocabularies up to which the second launch reads the rows itself, us with one launch and with two: 1 sequence of 4 drafted
// tokens over 2048 8.3 and 10.2, over 4096 9.0 and 10.2, over 8192 12.5 and 10.2; 64 of 3 over 4096 9.9 and 14.3, over 8192
// 13.9 and 14.4; 256 of 5 over 4096 20.0 and 19.9; 1000 of 3 over 4096 40 and 44.
constexpr int kDirect = 4096;

// A start out of order leaves in doubt whose rows are whose, for every sequence. It is looked through once, by up to so many
// blocks, a word for each of their four warps.
constexpr int kOrderBlocks = 32;
constexpr size_t kOrderBytes = kOrderBlocks * sizeof(int4);
// Sequences up to which each block of a draw in one launch looks through start itself, us a call that way and with a launch in
// front that does: plain draws over 2048 logits, 512 11.5 and 12.1, 2048 31.3 and 30.7, 8192 134 and 113, 65535 2323 and 954;
// over 4, 2048 22.6 and 22.7, 65535 1978 and 608.
constexpr int kOwnOrder = 2048;

struct VerifyParams {
  const int32_t* start;
  const void* logits;
  const void* draft_logits;
  int64_t row, draft_row;
  const int32_t* draft;
  const float* temperature;
  const float* u_accept;
  const float* u_token;
  int32_t* accepted;
  int32_t* token;
  float* prob;
  int4* order;                         // [checks]: not 0 where a warp found start out of order
  Piece* pieces;                       // [2][rows][splits]: the target's, the draft's
  int n, rows, vocab, splits;
  int cluster, chunk;                  // blocks a sequence, logits a block
  int z_bits;                          // of the fixed point of their sums
  int direct;                          // one launch: the vocabulary is small
  int checks;                          // blocks that look through start; 0: each block of the draw does
};

// Scaled logits are finite: NaN and -infinity become the lowest number, whose exponential next to any other is 0; a
// row whose largest is that has no probabilities.
constexpr float kLowest = -FLT_MAX;
constexpr float kLog2e = 1.44269504f;
__device__ __forceinline__ float scaled(float l, float by) { return fminf(fmaxf(__fmul_rn(l, by), kLowest), FLT_MAX); }
__device__ __forceinline__ float scale_of(float temperature) {
  return temperature > 0.f ? fminf(__fdiv_rn(1.f, temperature), FLT_MAX) : 1.f;
}
__device__ __forceinline__ float exp_from(float x, float m) { return expf(__fsub_rn(x, m)); }
// The same in fewer steps, for a row's sum. The difference comes first: it is exact next to the largest, where the sum is
// made, and 0 at it. (x log2(e) - m log2(e) by one fused operation keeps the rounding of the second product, half a step of
// a number as large as the largest logit over the temperature, in every exponential of the sum.)
__device__ __forceinline__ float ex2_from(float x, float m) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(__fmul_rn(__fsub_rn(x, m), kLog2e)));
  return r;
}

__device__ __forceinline__ float warp_max(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
// One piece out of the warp's: the largest first, so that each lane's sum is scaled once.
__device__ __forceinline__ Piece join_warp(const Piece& a) {
  Piece r;
  r.m = warp_max(a.m);
  r.s = warp_sum(a.s * expf(a.m - r.m));
  r.arg = __reduce_min_sync(0xffffffffu, a.m == r.m ? a.arg : INT32_MAX);
  r.pad = 0;
  return r;
}

__device__ __forceinline__ float value(const float* p) { return *p; }
__device__ __forceinline__ float value(const __nv_bfloat16* p) { return __bfloat162float(*p); }

__device__ __forceinline__ void join(Piece* a, const Piece& b) {
  if (b.m > a->m || (b.m == a->m && b.arg < a->arg)) a->arg = b.arg;
  const float top = fmaxf(a->m, b.m);
  a->s = a->s * expf(a->m - top) + b.s * expf(b.m - top);
  a->m = top;
}

// The sequence that row r belongs to, by one warp; n: none.
__device__ __forceinline__ int sequence_of(const VerifyParams& p, int r) {
  const int lane = threadIdx.x & 31;
  int lo = 0, len = p.n;                 // of the sequences from lo on, `len`, those that end at or before r are counted
  while (len > 32) {
    const int step = (len + 31) / 32, i = lo + (lane + 1) * step;
    const int full = __popc(__ballot_sync(0xffffffffu, i <= lo + len && p.start[min(i, p.n)] <= r));
    lo += full * step;
    len = min(step, len - full * step);
  }
  return lo + __popc(__ballot_sync(0xffffffffu, lane < len && p.start[min(lo + lane, p.n - 1) + 1] <= r));
}

// Whether sequence i's rows are not some of the call's, in order.
__device__ __forceinline__ bool out_of_order(const VerifyParams& p, int i) {
  const int b = p.start[i], e = p.start[i + 1];
  return b < 0 || e < b || e > p.rows;
}
// Block b's share of them.
__device__ __forceinline__ void check_order(const VerifyParams& p, int b) {
  bool bad = false;
#pragma unroll 4
  for (int i = b * kStatThreads + threadIdx.x; i < p.n; i += p.checks * kStatThreads) bad |= out_of_order(p, i);
  bad = __any_sync(0xffffffffu, bad);
  if ((threadIdx.x & 31) == 0) reinterpret_cast<int*>(p.order + b)[threadIdx.x >> 5] = bad;
}
// Where no other launch can see to it.
__global__ void __launch_bounds__(kStatThreads) order_kernel(const __grid_constant__ VerifyParams p) {
  ptx::pdl_trigger();
  ptx::pdl_wait();
  check_order(p, blockIdx.x);
}

// A thread's logits of a piece, in registers: 16 bytes at a time from a 16-byte boundary on, so that `skew` elements
// in front of the row may belong to the first; what is not the row's is minus infinity. Few of them are wanted again, so
// that they leave L2 first (48 sequences of 7 over 131075: 100.5 -> 96.2 us a call).
template <class T>
struct Loads {
  static constexpr int kVec = 16 / sizeof(T), kVecs = kPer / kVec;
  uint4 raw[kVecs + 1];
  bool tail;                             // the block's: there is a last one behind the piece
  __device__ __forceinline__ static int index(int part, int skew, int v) {
    return part * kPiece + (v * kStatThreads + (int)threadIdx.x) * kVec - skew;
  }
  __device__ __forceinline__ void load(const T* row, int vocab, int part, int splits, int skew) {
    tail = part == splits - 1 && (part + 1) * kPiece - skew < vocab;
#pragma unroll
    for (int v = 0; v <= kVecs; ++v) {
      if (v == kVecs && !tail) break;
      const int i = index(part, skew, v);
      raw[v] = sizeof(T) == 4 ? make_uint4(0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u)
                              : make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u);
      if (i >= 0 && i + kVec <= vocab) {
        raw[v] = __ldcs(reinterpret_cast<const uint4*>(row + i));
      } else if (i + kVec > 0 && i < vocab) {
        T x[kVec];
#pragma unroll
        for (int k = 0; k < kVec; ++k) x[k] = i + k >= 0 && i + k < vocab ? row[i + k] : T(-INFINITY);
        memcpy(&raw[v], x, 16);
      }
    }
  }
  __device__ __forceinline__ float get(int v, int k) const {
    const uint32_t w[4] = {raw[v].x, raw[v].y, raw[v].z, raw[v].w};
    if (sizeof(T) == 4) return __uint_as_float(w[k & 3]);
    return __uint_as_float(k & 1 ? w[(k >> 1) & 3] & 0xffff0000u : w[(k >> 1) & 3] << 16);
  }
};

// Bound by HBM. A thread holds its 32 logits, so that their maximum comes first and nothing is rescaled; an exponential
// is a product, a difference, a product, and ex2. Where NaN or infinities spoil that, the piece is done again with clamped
// logits. Eight blocks of 128 threads an SM: us a call of 48 sequences of 7 over 131075 92.5, four of 256 94.5, two of 512
// 96.0; three of 256, where no register spills, 103; half as many logits a thread 98.9. (With one fused operation for product
// and difference, which loses the bits that ex2_from keeps; with it each 2.5 more.)
template <class T>
__global__ void __launch_bounds__(kStatThreads, 8) stats_kernel(const __grid_constant__ VerifyParams p) {
  __shared__ Piece warps[kStatThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int r = blockIdx.x / p.splits, part = blockIdx.x % p.splits, is_draft = blockIdx.y;
  const T* row = is_draft ? static_cast<const T*>(p.draft_logits) + r * p.draft_row : static_cast<const T*>(p.logits) + r * p.row;
  const int skew = (int)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
  // only then may the next launch start: it reads what lies in front of this one before it waits for this one
  ptx::pdl_wait();
  ptx::pdl_trigger();
  Loads<T> x;
  if (!is_draft) x.load(row, p.vocab, part, p.splits, skew);                 // on their way while the row's sequence is looked up
  if (!is_draft && blockIdx.x < p.checks) check_order(p, blockIdx.x);
  const int seq = sequence_of(p, r);                               // each warp for itself: no barrier
  if (seq >= p.n || p.start[seq] > r) return;                      // nobody's
  const float heat = p.temperature[seq];
  const bool greedy = !(heat > 0.f);
  if (is_draft) {
    if (greedy || r == p.start[seq + 1] - 1) return;               // not asked for
    x.load(row, p.vocab, part, p.splits, skew);
  }
  const float by = scale_of(heat);
  Piece a = {kLowest, 0.f, INT32_MAX, 0};
  constexpr int V = Loads<T>::kVecs, K = Loads<T>::kVec;
  auto each = [&](auto f) {
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int k = 0; k < K; ++k) f(x.get(v, k), v, k);
    if (x.tail)
#pragma unroll
      for (int k = 0; k < K; ++k) f(x.get(V, k), V, k);
  };
  each([&](float l, int, int) { a.m = fmaxf(a.m, __fmul_rn(l, by)); });
  a.m = warp_max(a.m);
  float s[4] = {};
  each([&](float l, int, int k) { s[k & 3] += ex2_from(__fmul_rn(l, by), a.m); });
  a.s = (s[0] + s[1]) + (s[2] + s[3]);
  if (__any_sync(0xffffffffu, !(a.s <= FLT_MAX)) || a.m == INFINITY) {
    a.m = kLowest;
    a.s = 0.f;
    each([&](float l, int, int) { a.m = fmaxf(a.m, scaled(l, by)); });
    a.m = warp_max(a.m);
    each([&](float l, int, int) { a.s += exp_from(scaled(l, by), a.m); });
  }
  if (greedy) {
    each([&](float l, int v, int k) {
      if (a.arg == INT32_MAX && scaled(l, by) == a.m) a.arg = Loads<T>::index(part, skew, v) + k;
    });
    a.arg = __reduce_min_sync(0xffffffffu, a.arg);
  }
  a.s = warp_sum(a.s);
  if (lane == 0) warps[warp] = a;
  __syncthreads();
  if (warp == 0) {
    a = {kLowest, 0.f, INT32_MAX, 0};
    if (lane < kStatThreads / 32) a = warps[lane];
    a = join_warp(a);
    if (lane == 0) p.pieces[((int64_t)is_draft * p.rows + r) * p.splits + part] = a;
  }
}

// The whole row's, by one warp; the first of its pieces may have been loaded.
__device__ __forceinline__ Piece piece_of(const VerifyParams& p, int is_draft, int r, int k) {
  if (k >= p.splits) return {kLowest, 0.f, INT32_MAX, 0};
  const int4 x = reinterpret_cast<const int4*>(p.pieces)[((int64_t)is_draft * p.rows + r) * p.splits + k];
  return {__int_as_float(x.x), __int_as_float(x.y), x.z, 0};
}
__device__ __forceinline__ Piece row_stats(const VerifyParams& p, int is_draft, int r, Piece first) {
  for (int k = (threadIdx.x & 31) + 32; k < p.splits; k += 32) join(&first, piece_of(p, is_draft, r, k));
  return join_warp(first);
}
__device__ __forceinline__ Piece row_stats(const VerifyParams& p, int is_draft, int r) {
  return row_stats(p, is_draft, r, piece_of(p, is_draft, r, threadIdx.x & 31));
}

// A thread's sum of fp32 numbers keeps what rounding loses (the exact error of a sum, Knuth): twice fp32's bits, in the
// thread's own order. From there on sums are whole numbers of 64-bit fixed point, so that any order gives the same:
// exponentials are at most 1, as many as the vocabulary has, and in units of 2^-z_bits cannot pass 2^63; weights sum to
// 1 and a few roundings, in units of 2^-62. FP64, and conversions to 64-bit whole numbers, run at 1/64 of fp32's rate:
// the draw over 2048 logits took 65 us with the one and 14 with the other.
typedef unsigned long long fixed;
constexpr int kWeightBits = 62;
__device__ __forceinline__ fixed to_fixed(float x, int bits) {       // x not negative; cut off below a unit
  const int b = __float_as_int(x), s = (b >> 23) - 150 + bits;
  const fixed m = (b & 0x7fffff) | 0x800000;
  return s >= 0 ? m << s : s > -24 ? m >> -s : 0;
}
struct Sum {
  float hi = 0.f, lo = 0.f;
  __device__ __forceinline__ void add(float x) {
    const float t = __fadd_rn(hi, x), z = __fsub_rn(t, hi);
    lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(t, z)), __fsub_rn(x, z)));
    hi = t;
  }
  __device__ __forceinline__ fixed value(int bits) const {
    const fixed l = to_fixed(fabsf(lo), bits);
    return to_fixed(hi, bits) + (lo < 0.f ? 0 - l : l);
  }
};
// The warp's sum (modulo 2^64), by 32-bit reductions of parts that leave room for 32 of them: 27, 27 and 10 bits.
__device__ __forceinline__ fixed warp_total(fixed x) {
  const uint32_t part = (1u << 27) - 1;
  const uint32_t a = __reduce_add_sync(0xffffffffu, (uint32_t)x & part), b = __reduce_add_sync(0xffffffffu, (uint32_t)(x >> 27) & part),
                 c = __reduce_add_sync(0xffffffffu, (uint32_t)(x >> 54));
  return a + ((fixed)b << 27) + ((fixed)c << 54);
}
__device__ __forceinline__ fixed warp_prefix(fixed x) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const fixed y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}
// 2^bits / x to fp32's rounding, x not 0.
__device__ __forceinline__ float inverse(fixed x, int bits) {
  const int lead = __clzll((long long)x);
  const fixed y = x << lead;                                         // [1, 2) as 1.63 bits: 24 of them and the next 32
  const float hi = (float)(uint32_t)(y >> 40) * 0x1p-23f, lo = (float)(uint32_t)(y >> 8) * 0x1p-55f;
  const float r = __frcp_rn(hi);
  return __fmul_rn(__fmaf_rn(r, __fmaf_rn(-lo, r, __fmaf_rn(-hi, r, 1.f)), r), __int_as_float((127 + bits - 63 + lead) << 23));
}
// The whole part of u x, u in [0, 1): u's bits times x, shifted.
__device__ __forceinline__ fixed times(float u, fixed x) {
  const int bits = __float_as_int(u), e = bits >> 23;
  const fixed m = e ? (bits & 0x7fffff) | 0x800000 : bits & 0x7fffff;
  const int down = 150 - max(e, 1);                                  // u = m 2^-down, 24 <= down
  const fixed lo = m * x, hi = __umul64hi(m, x);
  return down < 64 ? hi << (64 - down) | lo >> down : down < 128 ? hi >> (down - 64) : 0;
}

template <int WARPS>
struct TokenShared {
  int first;                            // the first refused row, or the last
  Piece rows[2][kRowsKept];             // the target's and the draft's rows
  int draft[kRowsKept];
  Piece pair[WARPS / 2];                // what one warp of a pair found out about the draft
  fixed z[2][kMostSums];                // each of the cluster's warps' sums of exponentials
  fixed w[2][kMostSums];                // and of weights, by turn
};

// One value of a warp to the same place of all of the cluster's blocks.
__device__ __forceinline__ void tell(fixed* slot, int cluster, fixed x) {
  const int lane = threadIdx.x & 31;
  if (lane < cluster) {
    const uint32_t at = ptx::mapa(ptx::saddr(slot), lane);
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(at), "l"(x) : "memory");
  }
}

// A row's share of a block: its logits from `src` on, `skew` elements past a 16-byte boundary.
template <class T>
struct Part {
  static constexpr int K = 16 / sizeof(T);
  const T* src;
  int size, skew;
  float m;
  __device__ __forceinline__ Part(const T* s, int n, float top)
      : src(s), size(n), skew((int)((reinterpret_cast<uintptr_t>(s) & 15) / sizeof(T))), m(top) {}
  __device__ __forceinline__ static float get(const uint4& raw, int k) {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    if (sizeof(T) == 4) return __uint_as_float(w[k & 3]);
    return __uint_as_float(k & 1 ? w[(k >> 1) & 3] & 0xffff0000u : w[(k >> 1) & 3] << 16);
  }
  // the v-th 16 bytes; minus infinity for what is not its
  __device__ __forceinline__ uint4 load(int v) const {
    const int i = v * K - skew;
    if (i >= 0 && i + K <= size) return *reinterpret_cast<const uint4*>(src + i);
    uint4 raw = sizeof(T) == 4 ? make_uint4(0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u)
                               : make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u);
    if (i + K > 0 && i < size) {
      T x[K];
#pragma unroll
      for (int k = 0; k < K; ++k) x[k] = i + k >= 0 && i + k < size ? src[i + k] : T(-INFINITY);
      memcpy(&raw, x, 16);
    }
    return raw;
  }
  // their exponentials: added to z and, if KEEP, left at kept[skew + i]. 0 for what is not there: m is above the lowest
  template <bool KEEP>
  __device__ __forceinline__ void take(int v, const uint4& raw, float by, Sum* z, float* kept) const {
    float e[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      e[k] = exp_from(scaled(get(raw, k), by), m);
      z[k & 1].add(e[k]);
    }
    if (KEEP && v * K < size + skew)
#pragma unroll
      for (int k = 0; k < K; k += 4) *reinterpret_cast<float4*>(kept + v * K + k) = make_float4(e[k], e[k + 1], e[k + 2], e[k + 3]);
  }
};

// What a block's chunk of exponentials takes in shared memory: room for the skew at the front and the last load's end.
__host__ __device__ __forceinline__ int kept_floats(int chunk) { return (chunk + 16 + 3) & ~3; }

// A whole row's maximum and sum by one warp, for vocabularies of up to kDirect: twice over it, the second time out of L1.
template <class T>
__device__ __forceinline__ Piece direct_stats(const T* row, int vocab, float by, bool greedy) {
  const int lane = threadIdx.x & 31;
  // each of a lane's logits, with its place, 32 loads under way at once; minus infinity behind the row
  auto each = [&](auto f) {
    for (int i0 = 0; i0 < vocab; i0 += 32 * 32) {
      float x[32];
#pragma unroll
      for (int u = 0; u < 32; ++u) x[u] = i0 + lane + 32 * u < vocab ? value(row + i0 + lane + 32 * u) : -INFINITY;
#pragma unroll
      for (int u = 0; u < 32; ++u) f(x[u], i0 + lane + 32 * u);
    }
  };
  Piece a = {kLowest, 0.f, INT32_MAX, 0};
  each([&](float l, int) { a.m = fmaxf(a.m, __fmul_rn(l, by)); });
  a.m = warp_max(a.m);
  float s[2] = {};
  each([&](float l, int i) { s[i >> 5 & 1] += ex2_from(__fmul_rn(l, by), a.m); });
  a.s = s[0] + s[1];
  if (__any_sync(0xffffffffu, !(a.s <= FLT_MAX)) || a.m == INFINITY) {     // NaN or infinities: clamped logits
    a.m = kLowest;
    a.s = 0.f;
    for (int i = lane; i < vocab; i += 32) a.m = fmaxf(a.m, scaled(value(row + i), by));
    a.m = warp_max(a.m);
    for (int i = lane; i < vocab; i += 32) a.s += exp_from(scaled(value(row + i), by), a.m);
  }
  if (greedy) {
    each([&](float l, int i) {
      if (i < a.arg && scaled(l, by) == a.m) a.arg = i;
    });
    a.arg = __reduce_min_sync(0xffffffffu, a.arg);
  }
  a.s = warp_sum(a.s);
  return a;
}

// The same where it is seldom called. (Written out at each of its four calls the kernel took 21.8 us between other kernels
// where it takes 8.2 behind itself: it waited for its instructions. This way 9.2 and 8.2.)
template <class T>
__device__ __noinline__ Piece direct_far(const T* row, int vocab, float by, bool greedy) { return direct_stats(row, vocab, by, greedy); }

// The two warps that share a row: a barrier of their own.
__device__ __forceinline__ void pair_sync(int id) { asm volatile("barrier.cta.sync %0, 64;" ::"r"(id) : "memory"); }

// What a sequence's blocks do. The first passes are short, so this is a chain of loads, sums over a warp, a block and a
// cluster, and barriers: 6 to 10 us from launch to launch for a few sequences over up to 4096, some 2 us each for the
// exponentials, their sum and the weights over 32000. KEEP: the exponentials of the block's logits stay in shared memory
// between the sum of them and the weights (64 sequences over 32000: 18.6 us, without 37.9); DIRECT: as many threads, and
// the rows' sums are made here.
template <class T, bool KEEP, int DIRECT>
__global__ void __launch_bounds__(DIRECT ? DIRECT : kTokenThreads, DIRECT == kWideThreads ? 1 : 3)
    token_kernel(const __grid_constant__ VerifyParams p) {
  extern __shared__ __align__(16) float kept[];       // exponentials of the block's chunk of the target's, and of the draft's
  constexpr int kThreads = DIRECT ? DIRECT : kTokenThreads, kWarps = kThreads / 32;
  __shared__ TokenShared<kWarps> sh;
  const int cluster = DIRECT ? 1 : p.cluster, rank = DIRECT ? 0 : blockIdx.x % p.cluster;
  const int seq = DIRECT ? blockIdx.x : blockIdx.x / p.cluster;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (!DIRECT) {
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");   // its memory may be written
  } else {
    ptx::pdl_trigger();
    ptx::pdl_wait();
  }
  const int r0 = p.start[seq], r1 = p.start[seq + 1];
  const float heat = p.temperature[seq], by = scale_of(heat), u_token = p.u_token[seq];
  const bool greedy = !(heat > 0.f);
  int4 order = {};
  bool bad = false;
  if (DIRECT) {
    if (p.checks) {
      if (lane < p.checks) order = p.order[lane];
    } else {
      for (int i = threadIdx.x; i < p.n; i += kThreads) bad |= out_of_order(p, i);
    }
    bad |= (order.x | order.y | order.z | order.w) != 0;
  } else {
    bad = out_of_order(p, seq);                                      // the others' are known behind the launch in front
  }
  if (threadIdx.x == 0) sh.first = r1 - 1;
  bad = __syncthreads_or(bad);
  const T* logits = static_cast<const T*>(p.logits);
  const T* drafts = greedy ? nullptr : static_cast<const T*>(p.draft_logits);
  bool waited = false;
  auto wait = [&] {                                                  // for the sums, in front of which all but them is read
    if (!waited) {
      ptx::pdl_wait();
      if (lane < p.checks) order = p.order[lane];
    }
    waited = true;
  };
  auto disorder = [&] { return __any_sync(0xffffffffu, (order.x | order.y | order.z | order.w) != 0) != 0; };
  // every block of the cluster does the same: a warp a row, or, where the rows are read here, one for the target's and one
  // for the draft's
  constexpr int kRowWarps = DIRECT ? 2 : 1;
  for (int r = r0 + warp / kRowWarps; r < r1 && !bad; r += kWarps / kRowWarps) {
    const bool last = r == r1 - 1;
    const int d = last ? -1 : p.draft[r];
    const bool in = (uint32_t)d < (uint32_t)p.vocab;
    const float u = last ? 0.f : fminf(fmaxf(p.u_accept[r], 0.f), 0x1.fffffep-1f);
    Piece a, b = {kLowest, 0.f, 0, 0};
    if (DIRECT) {
      const bool of_draft = warp & 1;
      a = b;
      if (!of_draft || (drafts && !last))
        a = direct_stats(of_draft ? drafts + r * p.draft_row : logits + r * p.row, p.vocab, by, greedy);
      if (of_draft && lane == 0) sh.pair[warp / 2] = a;
      pair_sync(1 + warp / 2);
      if (!of_draft) b = sh.pair[warp / 2];
      pair_sync(1 + warp / 2);
      if (of_draft) continue;
    } else {
      wait();
      a = piece_of(p, 0, r, lane);
      if (drafts && !last) b = piece_of(p, 1, r, lane);
      a = row_stats(p, 0, r, a);
      if (drafts && !last) b = row_stats(p, 1, r, b);
      bad = disorder();
    }
    const float xp = in ? scaled(value(logits + r * p.row + d), by) : 0.f;
    const float xq = in && drafts ? scaled(value(drafts + r * p.draft_row + d), by) : 0.f;
    const float pd = in && a.m > kLowest ? exp_from(xp, a.m) / a.s : 0.f;
    const float qd = !drafts ? 1.f : in && b.m > kLowest ? exp_from(xq, b.m) / b.s : 0.f;
    // u q < p of fp32 numbers, exactly: the product's rounding is a number of its own
    const float uq = __fmul_rn(u, qd);
    const bool less = uq < pd || (uq == pd && __fmaf_rn(u, qd, -uq) < 0.f);
    const bool yes = greedy ? a.m > kLowest && d == a.arg : less;
    if (lane == 0) {
      if (r - r0 < kRowsKept) {
        sh.rows[0][r - r0] = a;
        sh.rows[1][r - r0] = b;
        sh.draft[r - r0] = d;
      }
      if (!last && p.prob && rank == 0 && !bad) p.prob[r] = pd;
      if (!last && !yes) atomicMin(&sh.first, r);
    }
  }
  __syncwarp();
  if (!DIRECT) wait();
  if (!DIRECT) bad |= disorder();
  if (!DIRECT) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  if (bad || r0 == r1) {
    if (threadIdx.x == 0 && rank == 0) {
      p.accepted[seq] = bad ? -1 : 0;
      p.token[seq] = -1;
    }
    return;
  }
  __syncthreads();
  const int r = sh.first;
  const bool refused = r < r1 - 1, both = refused && drafts;
  Piece a, b = {kLowest, 0.f, 0, 0};
  int d;
  if (r - r0 < kRowsKept) {
    a = sh.rows[0][r - r0];
    if (both) b = sh.rows[1][r - r0];
    d = sh.draft[r - r0];
  } else {
    a = DIRECT ? direct_far(logits + r * p.row, p.vocab, by, greedy) : row_stats(p, 0, r);
    if (both) b = DIRECT ? direct_far(drafts + r * p.draft_row, p.vocab, by, false) : row_stats(p, 1, r);
    d = refused ? p.draft[r] : -1;
  }
  if (threadIdx.x == 0 && rank == 0) {
    p.accepted[seq] = r - r0;
    if (greedy || !(a.m > kLowest)) p.token[seq] = a.m > kLowest ? a.arg : -1;
  }
  if (greedy || !(a.m > kLowest)) return;                            // the whole cluster
  const bool with_q = b.m > kLowest;
  const int begin = min(rank * p.chunk, p.vocab), size = min(p.chunk, p.vocab - begin);
  const T* row = logits + r * p.row + begin;
  const T* draft_row = with_q ? drafts + r * p.draft_row + begin : row;
  const Part<T> of_p(row, size, a.m), of_q(draft_row, with_q ? size : 0, b.m);
  float* const put_q = kept + kept_floats(p.chunk);
  const float* kept_p = kept + of_p.skew;
  const float* kept_q = with_q ? put_q + of_q.skew : kept_p;
  // each warp's sums go to all blocks, and each warp adds them all up for itself: one barrier a sum
  const int sums = cluster * kWarps, own = rank * kWarps + warp;
  auto to_all = [&](fixed* slots, fixed x) {
    if (!DIRECT) tell(slots + own, cluster, x);
    else if (lane == 0) slots[own] = x;
  };
  auto meet = [] {
    __syncwarp();
    if (DIRECT) __syncthreads();
    else ptx::cluster_sync_all();
  };
  auto sum_below = [&](const fixed* slots, int n) {
    fixed x = 0;
    for (int k = lane; k < n; k += 32) x += slots[k];
    return warp_total(x);
  };
  // the token that a certain draft proposed weighs nothing where it was refused; its exponential is kept aside
  const int out = refused && !drafts && (uint32_t)(d - begin) < (uint32_t)size ? d - begin : -1;
  float aside = -1.f;
  // sums of both rows' exponentials; two of each, whose steps do not wait for one another
  Sum sum_p[2], sum_q[2];
  constexpr int U = sizeof(T) == 4 ? 4 : 2;
  for (int v0 = threadIdx.x; v0 * Part<T>::K < size + max(of_p.skew, of_q.skew); v0 += U * kThreads) {
    uint4 x[U], y[U];
#pragma unroll
    for (int u = 0; u < U; ++u) x[u] = of_p.load(v0 + u * kThreads);
    if (with_q)
#pragma unroll
      for (int u = 0; u < U; ++u) y[u] = of_q.load(v0 + u * kThreads);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      of_p.template take<KEEP>(v0 + u * kThreads, x[u], by, sum_p, kept);
      if (KEEP && out >= 0 && (out + of_p.skew) / Part<T>::K == v0 + u * kThreads) {
        aside = kept[out + of_p.skew];
        kept[out + of_p.skew] = 0.f;
      }
    }
    if (with_q)
#pragma unroll
      for (int u = 0; u < U; ++u) of_q.template take<KEEP>(v0 + u * kThreads, y[u], by, sum_q, put_q);
  }
  to_all(sh.z[0], warp_total(sum_p[0].value(p.z_bits) + sum_p[1].value(p.z_bits)));
  if (with_q) to_all(sh.z[1], warp_total(sum_q[0].value(p.z_bits) + sum_q[1].value(p.z_bits)));
  meet();
  const float rp = inverse(sum_below(sh.z[0], sums), p.z_bits);
  float rq = with_q ? inverse(sum_below(sh.z[1], sums), p.z_bits) : 0.f;      // 0 without a draft's logits: p - 0 p is p
  bool residual = true;
  auto weight = [&](int i) {
    float x, y;
    if (KEEP) {
      x = kept_p[i];
      y = kept_q[i];
    } else {
      x = residual && i == out ? 0.f : exp_from(scaled(value(row + i), by), a.m);
      y = with_q ? exp_from(scaled(value(draft_row + i), by), b.m) : 0.f;
    }
    return fmaxf(__fsub_rn(__fmul_rn(x, rp), __fmul_rn(y, rq)), 0.f);
  };
  // each thread a run of the block's logits, an odd number, so that a warp's lanes read from different banks
  const int run = (size + kThreads - 1) / kThreads | 1, begin_run = min((int)threadIdx.x * run, size), end_run = min(begin_run + run, size);
  fixed x, total;
  int turn = 0;
  for (;; ++turn) {
    Sum sum;
#pragma unroll 4
    for (int i = begin_run; i < end_run; ++i) sum.add(weight(i));
    x = sum.value(kWeightBits);
    to_all(sh.w[turn], warp_total(x));
    meet();
    total = sum_below(sh.w[turn], sums);
    if (total || turn) break;                                        // the same in every block
    // roundings left nothing: from p itself
    residual = false;
    rq = 0.f;
    if (KEEP && aside >= 0.f) kept[out + of_p.skew] = aside;
    __syncthreads();
  }
  // nobody reads another block's memory from here on. The warp, its thread, the thread's logit: each time the first whose
  // end passes `want`. A thread's sum and its logits' may differ in the last bits that it kept: should none of them pass,
  // the last that weighs anything is it
  const fixed want = times(fminf(fmaxf(u_token, 0.f), 0x1.fffffep-1f), total);
  fixed before = sum_below(sh.w[turn], own);
  if (want < before || want - before >= sh.w[turn][own]) return;
  auto first_above = [&](fixed y, bool* passed) {
    const fixed end = before + warp_prefix(y);
    const uint32_t some = __ballot_sync(0xffffffffu, y != 0), hit = __ballot_sync(0xffffffffu, end > want) & some;
    const int at = hit ? __ffs(hit) - 1 : some ? 31 - __clz(some) : -1;
    *passed = hit != 0;
    before = __shfl_sync(0xffffffffu, hit ? end - y : end, hit ? at : 31);
    return at;
  };
  bool passed;
  const int from = max(first_above(x, &passed), 0), i0 = (warp * 32 + from) * run, i1 = min(i0 + run, size);
  int token = i0;
  for (int t = i0; t < i1; t += 32) {
    const int at = first_above(t + lane < i1 ? to_fixed(weight(t + lane), kWeightBits) : 0, &passed);
    if (at >= 0) token = t + at;
    if (passed) break;
  }
  if (lane == 0) p.token[seq] = begin + token;
}

// ------------------------------------------------------------------ checks
constexpr int kResident = 3 * 152;
constexpr size_t kMostKept = 69 * 1024;        // bytes of exponentials in a block's shared memory: three blocks an SM
size_t kept_bytes(const VerifyParams& p) { return (size_t)kept_floats(p.chunk) * (p.draft_logits ? 8 : 4); }

int check(const cp_verify_args* a, VerifyParams* p, size_t* workspace) {
  if (!a || !a->start || !a->logits || !a->draft || !a->temperature || !a->u_accept || !a->u_token || !a->accepted || !a->token)
    return CP_ERR_INVALID_ARG;
  if (a->sequences < 1 || a->rows < 1 || a->vocab < 1) return CP_ERR_INVALID_ARG;
  if (a->dtype != CP_LOGITS_F32 && a->dtype != CP_LOGITS_BF16) return CP_ERR_INVALID_ARG;
  if (a->sequences > 65535 || a->rows > 1 << 20 || a->vocab > 1 << 24) return CP_ERR_UNSUPPORTED;
  p->row = a->logits_stride ? a->logits_stride : a->vocab;
  p->draft_row = a->draft_stride ? a->draft_stride : a->vocab;
  const int64_t most = (int64_t)1 << 40;
  if (p->row < 0 || p->draft_row < 0) return CP_ERR_INVALID_ARG;
  if (p->row > most || p->draft_row > most) return CP_ERR_UNSUPPORTED;
  const uintptr_t es = a->dtype == CP_LOGITS_F32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(a->logits) % es || reinterpret_cast<uintptr_t>(a->draft_logits) % es) return CP_ERR_UNSUPPORTED;
  p->start = a->start;
  p->logits = a->logits;
  p->draft_logits = a->draft_logits;
  p->draft = a->draft;
  p->temperature = a->temperature;
  p->u_accept = a->u_accept;
  p->u_token = a->u_token;
  p->accepted = a->accepted;
  p->token = a->token;
  p->prob = a->prob;
  p->n = a->sequences;
  p->rows = a->rows;
  p->vocab = a->vocab;
  p->cluster = 1;
  const auto splits = [a](int es) {                            // wherever a row starts within 16 bytes
    return std::max(1, (a->vocab + 16 / es - 1 - kStatThreads * (16 / es) + kPiece - 1) / kPiece);
  };
  p->splits = splits((int)es);
  if ((int64_t)p->rows * p->splits > 1 << 30) return CP_ERR_UNSUPPORTED;             // blocks
  p->direct = p->vocab <= kDirect;
  // blocks a sequence: more while there is work for them and room for all at once, or until a block's share can be kept
  // (16 blocks and 8, us: plain draws of 16 sequences over 131075 14.3 and 18.3, of 1 9.9 and 11.8, but 48 sequences of 7 92 and
  // 89; room for twice as many: 64 draws over 32000 13.6 -> 17.6)
  auto cut = [&] { p->chunk = (p->vocab + p->cluster - 1) / p->cluster; };
  for (cut(); !p->direct && p->cluster < kMostCluster &&
              ((p->chunk > 2048 && (int64_t)p->n * p->cluster * 2 <= kResident) || kept_bytes(*p) > kMostKept);
       cut())
    p->cluster *= 2;
  p->z_bits = 62;
  while (((int64_t)1 << (63 - p->z_bits)) < p->vocab) --p->z_bits;
  p->checks = p->direct && p->n <= kOwnOrder ? 0 : std::min(kOrderBlocks, (p->n + kStatThreads - 1) / kStatThreads);
  if (!p->direct) p->checks = (int)std::min<int64_t>(p->checks, (int64_t)p->rows * p->splits);
  *workspace = (p->checks ? kOrderBytes : 0) +
               (p->direct ? 0 : (size_t)2 * p->rows * std::max(splits(2), splits(4)) * sizeof(Piece));        // the same for both types
  return CP_OK;
}

template <class T, bool KEEP, int DIRECT>
cudaError_t launch_token(const VerifyParams& p, cudaStream_t s) {
  return launch_as(token_kernel<T, KEEP, DIRECT>, dim3((unsigned)(p.n * p.cluster)), p.cluster, 1, true, DIRECT ? DIRECT : kTokenThreads,
                   KEEP ? kept_bytes(p) : 0, s, p);
}
template <class T>
cudaError_t launch(const VerifyParams& p, cudaStream_t s) {
  const bool wide = p.n <= kWideMost && p.rows > 4 * p.n;
  if (p.direct) {
    if (p.checks) {
      const cudaError_t e = launch_as(order_kernel, dim3((unsigned)p.checks), 1, 1, true, kStatThreads, 0, s, p);
      if (e != cudaSuccess) return e;
    }
    return wide ? launch_token<T, true, kWideThreads>(p, s) : launch_token<T, true, kTokenThreads>(p, s);
  }
  const dim3 grid((unsigned)(p.rows * p.splits), p.draft_logits ? 2 : 1);
  const cudaError_t e = launch_as(stats_kernel<T>, grid, 1, 1, true, kStatThreads, 0, s, p);
  if (e != cudaSuccess) return e;
  return kept_bytes(p) <= kMostKept ? launch_token<T, true, 0>(p, s) : launch_token<T, false, 0>(p, s);
}

template <class T, bool KEEP, int DIRECT>
bool allow() {
  return cudaFuncSetAttribute(token_kernel<T, KEEP, DIRECT>, cudaFuncAttributeMaxDynamicSharedMemorySize, KEEP ? (int)kMostKept : 0) == cudaSuccess &&
         cudaFuncSetAttribute(token_kernel<T, KEEP, DIRECT>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess;
}

// Once per device: whether it is one that the kernels run on, and their shared memory.
int prepare(int device) {
  static std::atomic<int> done[64];
  if (device >= 0 && device < 64 && done[device].load(std::memory_order_acquire)) return CP_OK;
  const int st = check_device(device);
  if (st) return st;
  DeviceGuard g(device);
  const auto all = [](auto t) {
    using T = decltype(t);
    return allow<T, true, kWideThreads>() && allow<T, true, kTokenThreads>() && allow<T, true, 0>() && allow<T, false, 0>();
  };
  if (!all(0.f) || !all(__nv_bfloat16()))
    return CP_ERR_CUDA;
  if (device < 64) done[device].store(1, std::memory_order_release);
  return CP_OK;
}

}  // namespace

extern "C" {

int cp_verify_check(const cp_verify_args* args, size_t* workspace_bytes) {
  if (workspace_bytes) *workspace_bytes = 0;
  VerifyParams p{};
  size_t need = 0;
  const int st = check(args, &p, &need);
  if (!st && workspace_bytes) *workspace_bytes = need;
  return st;
}

int cp_verify(const cp_verify_args* args, int device, void* workspace, size_t workspace_bytes, cp_stream_t stream) {
  VerifyParams p{};
  size_t need = 0;
  const int st = check(args, &p, &need);
  if (st) return st;
  if (need && (!workspace || workspace_bytes < need)) return CP_ERR_INVALID_ARG;
  if (!aligned16(workspace)) return CP_ERR_UNSUPPORTED;
  const int dev = prepare(device);
  if (dev) return dev;
  DeviceGuard g(device);
  p.order = static_cast<int4*>(workspace);
  p.pieces = reinterpret_cast<Piece*>(static_cast<uint8_t*>(workspace) + kOrderBytes);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return cuda_err(args->dtype == CP_LOGITS_BF16 ? launch<__nv_bfloat16>(p, s) : launch<float>(p, s));
}

}  // extern "C"
