// cp_attend_chunk.cu -- attention of many new rows of a sequence (a piece of a
// prompt, or all of it) over the paged cache, on tcgen05.
//
// The rows of one sequence and kv head are packed row by row, query head by
// query head (row i: new row i / group, head i % group), and cut into tiles of
// 128; a block takes two tiles, so that each key and value it brings in serves
// 256 rows, and the two keep the tensor core busy in turn: while one tile's
// softmax runs, the other's products do.
//
// Warps 0-7 and 8-15: the softmax of tile 0 and tile 1, two threads a row with
// 64 of a tile's 128 positions each (more warps at less work each: what one
// tile's softmax takes is what the other tile's products have to cover). Behind
// them the helper warps, then the warp that issues every MMA, then the one that
// brings pages in through tensor maps, a lane a page. For each 128 positions
// S = Q K^T (128 x 128, fp32 in TMEM); the softmax threads read their part of
// it (over an e4m3 cache twice: there it does not fit their registers), write
// the weights as 16 bit over the S that they have read, and O += P V reads
// them from there. O stays in
// TMEM for the whole pass. The reference of a row's weights is its first
// tile's maximum; it is only moved, and O rescaled, when a later score has
// risen by 2^kLazy over it, since the sum and the weights of a part share the
// reference.
//
// bf16 pages land in the ring as the tensor core reads them. Tiles at the ends
// of what the block's rows see, and tiles that only some of them see, pass
// the helpers first: values that nobody sees are zeroed (a page may hold
// anything there), and values that some row must not see are looked over for
// infinities and NaN. e4m3 pages land in a ring of their own and all pass
// the helpers, which widen them to fp16 and multiply each row by its scale,
// relative to the largest that the block has met and 2^kUp up: exact as far
// as fp16 reaches, to rows 2^21 smaller; a block that meets one further apart
// computes its rows the plain way. The power taken out of a tile's keys multiplies its scores, the
// one of the values the result. Weights start at 2^kBias.
//
// Bound by the chain from a tile's scores through its softmax to its second
// product, and by the issuing warp: nothing of what it does between two groups
// of products is hidden (each clock of it is one of the tensor core's). 512
// rows of 16/8 heads of 128 behind 32256 positions, bf16: 135 us a call, 1010
// TFLOP/s, the tensor pipe busy 51 %, 128 of 152 SMs; two prompts of 4096:
// 150 us, 917 TFLOP/s, of which each block's start and end are 9 us. A second
// issuing warp hides the gaps alone, but pulls the two softmaxes into step:
// 186 us, with turns between the two 149.
#include <cfloat>
#include <type_traits>

#include "cp_attend.cuh"

namespace cp {
namespace cache {
namespace {

using namespace ptx;

constexpr int kTile = 128;             // rows of a tile, and positions of one
constexpr int kSoftWarps = 16;         // softmax: eight a tile of rows
constexpr int kHelper0 = 16;           // first helper warp
constexpr int kScaleSlots = 8;         // tiles whose scales are held: more than the ring's

// Loads are counted K of tile 0, V of tile 0, K of tile 1, ...; load n is in slot n % kOps.
template <int D, bool E4M3>
struct Cfg {
  // four helper warps widen e4m3; bf16 needs few, and the softmax threads the registers
  static constexpr int kHelpers = E4M3 ? 128 : 64;
  static constexpr int kMmaWarp = kHelper0 + kHelpers / 32, kLoadWarp = kMmaWarp + 1;
  static constexpr int kThreads = (kLoadWarp + 1) * 32;
  static constexpr int kOpBytes = kTile * D * 2;        // one operand tile
  static constexpr int kSlab = kTile * 128;             // 64 columns of it
  static constexpr int kOps = D == 64 ? 8 : 4;
  static constexpr int kRawBytes = E4M3 ? kTile * D : 0;
  static constexpr int kRaws = E4M3 ? (D == 64 ? 4 : 2) : kOps;   // bf16: the operand ring itself
  static constexpr int kTiles = (2 + kOps) * kOpBytes + (E4M3 ? kRaws : 0) * kRawBytes;
};
// TMEM columns: the two tiles' scores (and weights), then their outputs
constexpr uint32_t kTmemS = 0, kTmemO = 256, kTmemCols = 512;

// What the block computes: found by the load warp, and kept out of the others' registers.
struct Item {
  Seq s;
  int seq;                     // -1: nothing
  int kv, part, parts, whole;
  int row0, rows_here;         // the pair's rows
  int first_row, first_head;   // row i of them is new row first_row + (first_head + i) / group, head (first_head + i) % group
  int lo, t_begin, t_end, ntiles;       // first position that some row sees; the part's, and its tiles
  int jb[2], je[2], all_lo[2], all_hi[2];   // tiles that tile i of rows takes part in, and the positions that all its rows see
};

struct ChunkShared {
  uint64_t raw_full[8], raw_empty[8], op_full[8];
  uint64_t done[4];   // rounds of the MMA warp
  uint64_t q_full, s_full[2], p_full[2], o_full;
  uint32_t tmem;
  long long timeout_ns;
  int abort;       // a wait gave up
  int bad;         // a value that some row must not see is not finite
  int lost;        // e4m3: bits of the largest product of a row's scale and what fp16 left of its q out (kMostLost)
  int kref[kScaleSlots], vref[kScaleSlots];    // e4m3: exponents taken out of a tile's keys and values
  Item item;
  float row[2][kPairRows];     // what the two threads of a row tell each other; before that, [0]: e4m3's powers of
                               // two taken out of the rows of q, times the scale
};

// Dynamic shared memory: the tiles from a 1024-byte boundary on, then the rest. Without static shared memory the
// dynamic one starts on such a boundary; the largest size leaves 0.5 KB should it not.
template <int D, bool E4M3>
struct Smem {
  static constexpr int kMost = 227 * 1024, kWant = Cfg<D, E4M3>::kTiles + (int)sizeof(ChunkShared) + 1024;
  static_assert(Cfg<D, E4M3>::kTiles + (int)sizeof(ChunkShared) <= kMost, "tiles and barriers fit an SM");
  static constexpr int kBytes = kWant < kMost ? kWant : kMost;
};

// Bounded: after the cache's timeout, or once another wait of the block gave up, false.
__device__ __forceinline__ bool wait_bar(ChunkShared& sh, uint32_t bar, uint32_t parity) {
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

// The same for a whole warp that goes on together.
__device__ __forceinline__ bool wait_warp(ChunkShared& sh, uint32_t bar, uint32_t parity) {
  return __all_sync(0xffffffffu, wait_bar(sh, bar, parity));
}

__device__ __forceinline__ uint32_t hf_mul(uint32_t x, uint32_t f) {
  const __half2 y = __hmul2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&f));
  return *reinterpret_cast<const uint32_t*>(&y);
}
// Each lane that `need`s it waits for a barrier of its own. Tests without pause at first: the tensor core stands still
// meanwhile, and waking a suspended warp takes longer than most of these waits.
__device__ __forceinline__ bool wait_lanes(ChunkShared& sh, uint32_t bar, uint32_t parity, bool need) {
  bool ok = !need || mb_test(bar, parity);
#pragma unroll 1
  for (int i = 0; i < 4000 && !__all_sync(0xffffffffu, ok); ++i) ok = ok || mb_test(bar, parity);
  if (!ok) ok = wait_bar(sh, bar, parity);
  return __all_sync(0xffffffffu, ok);
}
// The two warps that share 32 rows: a barrier of their own, with the OR of a predicate.
__device__ __forceinline__ bool pair_or(int id, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %2, 64, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)x), "r"(id)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ uint64_t pack2(const uint32_t* x) { return pair_of(__uint_as_float(x[0]), __uint_as_float(x[1])); }
// Wait until the products that read operand load n are done: round i of the MMA warp reads K of tile i and V of
// tile i - 1.
__device__ __forceinline__ bool wait_done(ChunkShared& sh, int n) {
  const int i = (n + 1) >> 1;
  return wait_warp(sh, saddr(&sh.done[i & 3]), (i >> 2) & 1);
}
// Byte offset of 16-byte unit u (8 elements) of row r in an operand tile.
__device__ __forceinline__ uint32_t op_at(int r, int u) {
  return (uint32_t)((u >> 3) * (kTile * 128) + r * 128 + (((u & 7) ^ (r & 7)) << 4));
}

// Positions a part, by a whole warp: the plan's, made for sequences that all have the longest one's length and for more
// than one round of blocks, or longer ones if at the sequences' own lengths those are one round that costs less. Every
// block comes to the same. (16 sequences of 700 to 9000 e4m3 positions, four of them with 301 new rows: 150 us a call
// in the plan's parts, 141 in these. Choosing among several rounds too measured up to 7 % slower and 5 % faster.)
template <int D>
__device__ __forceinline__ int chosen_chunk(const AttendParams& p) {
  const int lane = threadIdx.x & 31;
  const int n = min(lane + 1, p.a.chunk_parts);
  const uint32_t tiles = ((p.a.chunk_span + n - 1) / n + kTile - 1) / kTile, magic = 0xffffffffu / tiles + 1;
  uint32_t blocks = 0, all = 0;
  for (int i0 = 0; i0 < p.b.n; i0 += 32) {
    uint32_t pairs = 0, len = 0;
    if (i0 + lane < p.b.n) {
      const Seq s = seq_of(p.b, i0 + lane, p.c.status);
      const int rows = s.n * p.group;
      if (rows > kStepRows || !p.a.use_step) pairs = (rows + kPairRows - 1) / kPairRows * p.c.heads;
      len = (min(s.len, p.a.chunk_span) + kTile - 1) / kTile;
    }
    for (uint32_t left = __ballot_sync(0xffffffffu, pairs > 0); left; left &= left - 1) {
      const int at = __ffs(left) - 1;
      const uint32_t items = __shfl_sync(0xffffffffu, pairs, at), of_one = __shfl_sync(0xffffffffu, len, at);
      blocks += items * (tiles == 1 ? of_one : __umulhi(of_one + tiles - 1, magic));
      all += items * of_one;
    }
  }
  // a round costs its longest block; several, of uneven blocks that follow one another closely, all work and half a block
  const float block = chunk_rounds_ns(1, tiles, D);
  const float even = ((float)all * (D == 128 ? kTileNs128 : kTileNs64) + (float)blocks * kBlockNs) * (1.f / kSms) + 0.5f * block;
  const float plan = __shfl_sync(0xffffffffu, even, 31);       // lane 31 has the plan's
  const uint32_t fits = __ballot_sync(0xffffffffu, blocks <= kSms && block < plan);
  const int chosen = __shfl_sync(0xffffffffu, (int)tiles, fits ? 31 - __clz(fits) : 31);
  return fits ? chosen * kTile : p.a.chunk_chunk;
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(Cfg<D, E4M3>::kThreads, 1) attend_chunk_kernel(const __grid_constant__ AttendParams p,
                                                                    const __grid_constant__ CacheMaps maps) {
  using C = Cfg<D, E4M3>;
  constexpr int NO = C::kOps, NR = C::kRaws, kHelpers = C::kHelpers, kMmaWarp = C::kMmaWarp, kLoadWarp = C::kLoadWarp;
  extern __shared__ __align__(1024) uint8_t raw[];
  uint8_t* ops = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  ChunkShared& sh = *reinterpret_cast<ChunkShared*>(ops + C::kTiles);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (ops + C::kTiles + sizeof(ChunkShared) > raw + Smem<D, E4M3>::kBytes) {
    set_status(p.c.status, CP_ERR_UNSUPPORTED);
    return;
  }
  if (warp == kHelper0) {                // a lane a barrier
    if (lane < 8) mb_init(saddr(&sh.raw_full[lane]), 1);
    else if (lane < 16) mb_init(saddr(&sh.raw_empty[lane - 8]), kHelpers / 32);
    else if (lane < 24) mb_init(saddr(&sh.op_full[lane - 16]), kHelpers / 32);
    else if (lane < 28) mb_init(saddr(&sh.done[lane - 24]), 1);
    if (lane < 2) {
      mb_init(saddr(&sh.s_full[lane]), 1);
      mb_init(saddr(&sh.p_full[lane]), 8);
    }
    if (lane == 2) mb_init(saddr(&sh.q_full), kSoftWarps);
    if (lane == 3) mb_init(saddr(&sh.o_full), 1);
    if (lane == 4) {
      sh.abort = sh.bad = sh.lost = 0;
      sh.timeout_ns = p.timeout_ns;
    }
    mb_fence_init();
  }
  if (warp == kMmaWarp) {
    tm_alloc(saddr(&sh.tmem), kTmemCols);
    tm_relinquish();
  }

  // The load warp finds the block's item alone: every warp doing so took the issue slots for 2 to 3 us a block.
  if (warp == kLoadWarp) {
    // which sequence and which of its tile pairs: the pairs are counted 32 sequences at a time
    int seq = -1, pair = 0;
    Seq s{};
    const int kv = blockIdx.x % p.c.heads, part = blockIdx.y, want = blockIdx.x / p.c.heads;
    int before = 0;
    for (int i0 = 0; i0 < p.b.n && seq < 0; i0 += 32) {
      int pairs = 0;
      Seq one{};
      if (i0 + lane < p.b.n) {
        one = seq_of(p.b, i0 + lane, p.c.status);
        const int rows = one.n * p.group;
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
        s.row0 = __shfl_sync(0xffffffffu, one.row0, at);
        s.n = __shfl_sync(0xffffffffu, one.n, at);
        s.len = __shfl_sync(0xffffffffu, one.len, at);
        s.first = __shfl_sync(0xffffffffu, one.first, at);
      }
      before += __shfl_sync(0xffffffffu, sum, 31);
    }
    Item& it = sh.item;
    if (seq >= 0) {
      const int nrows = s.n * p.group, row0 = pair * kPairRows, rows_here = min(kPairRows, nrows - row0);
      const int first_row = row0 / p.group, first_head = row0 - first_row * p.group;
      auto pos_of = [&](int i) { return s.first + first_row + (int)(((uint32_t)(first_head + min(i, rows_here - 1)) * p.magic) >> 16); };
      // lane 0 for the pair, lanes 1 and 2 for its tiles of rows
      const int f = lane == 2 ? kTile : 0;
      const int first = pos_of(f), last = pos_of(lane == 1 ? kTile - 1 : kPairRows - 1);
      const Range r = item_range(p, first, last, s.len, kChunkAlign);
      const Range range = {__shfl_sync(0xffffffffu, r.lo, 0), __shfl_sync(0xffffffffu, r.hi, 0), __shfl_sync(0xffffffffu, r.base, 0)};
      const int chunk = p.a.chunk_coarser ? chosen_chunk<D>(p) : p.a.chunk_chunk;
      const int parts = parts_of(range, chunk);
      const int t_begin = range.base + (part < parts ? part * chunk : 0);
      const int t_end = t_begin + min(chunk, range.hi - t_begin);
      if (part >= max(parts, 1)) seq = -1;
      if (lane == 1 || lane == 2) {
        const int x = lane - 1, a = max(r.lo, t_begin), b = min(r.hi, t_end);
        const bool any = f < rows_here && b > a;
        int d;
        it.jb[x] = any ? (a - t_begin) / kTile : 0;
        it.je[x] = any ? (b - t_begin + kTile - 1) / kTile : 0;
        visible(p, last, s.len, &it.all_lo[x], &d);
        visible(p, first, s.len, &d, &it.all_hi[x]);
      }
      if (lane == 0) {
        if (p.a.chunk_coarser) *p.coarser = chunk;
        it.s = s;
        it.kv = kv;
        it.part = part;
        it.parts = parts;
        it.whole = parts <= 1;
        it.row0 = row0;
        it.rows_here = rows_here;
        it.first_row = first_row;
        it.first_head = first_head;
        it.lo = range.lo;
        it.t_begin = t_begin;
        it.t_end = t_end;
        it.ntiles = t_end > t_begin ? (t_end - t_begin + kTile - 1) / kTile : 0;
      }
    }
    if (lane == 0) it.seq = seq;
  }
  tm_fence_before();
  __syncthreads();
  tm_fence_after();
  pdl_trigger();
  const Item& it = sh.item;
  if (it.seq < 0) {
    if (warp == kMmaWarp) tm_dealloc(sh.tmem, kTmemCols);
    return;
  }
  const uint32_t tmem = sh.tmem;

  const uint32_t q_s = saddr(ops), op_s = q_s + 2 * C::kOpBytes, raw_s = E4M3 ? op_s + NO * C::kOpBytes : op_s;

  // a softmax thread's row, and which half of a tile's positions (and later of its columns) is its
  const int i = warp >> 3, half = (warp >> 2) & 1;       // stream (warps 0-15)
  const int slot = (i * kTile + (warp & 3) * 32 + lane) & (kPairRows - 1);
  const int pair_id = 1 + i * 4 + (warp & 3);            // the named barrier of the row's two warps
  float l = 0.f, m = -INFINITY;
  int vr = 0;
  constexpr float kBias = E4M3 ? 8.f : 0.f;
  constexpr int kUp = 6;                                 // operands of e4m3 reach 448 * 2^kUp: inside fp16
  constexpr int kLeast = -15;                            // and the least, 2^-9, is still one of fp16's times this power
  constexpr float kLazy = E4M3 ? 6.f : 8.f;              // weights reach 2^(kBias + kLazy): inside fp16
  constexpr int kHalf = kTile / 2;

  if (warp < kSoftWarps) {
    // ---------------------------------------------------------------- softmax
    // a row of the pair: its new row and its head; the quotient by a multiplication, exact for sums below 320
    const int first_row = it.first_row, first_head = it.first_head, rows_here = it.rows_here;
    auto new_row = [&](int r) { return first_row + (int)(((uint32_t)(first_head + r) * p.magic) >> 16); };
    {
      // a thread's part of q: 16 of its pair of warps' 32 rows, a row's units side by side
      constexpr int UPR = D / 8, RPI = 32 / UPR, N = 16 / RPI;
      const int u = lane % UPR, base = (warp & 3) * 32 + half * 16 + lane / UPR;
      const uint16_t* src = p.q + (int64_t)it.s.row0 * p.q_row + (int64_t)(it.kv * p.group) * p.q_head + u * 8;
      uint4 x[N];
      float lost = 0.f;
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const int r = i * kTile + base + k * RPI, n = new_row(r);
        x[k] = make_uint4(0, 0, 0, 0);
        if (r < rows_here)
          x[k] = *reinterpret_cast<const uint4*>(src + (int64_t)n * p.q_row +
                                                 (int64_t)(first_head + r - (n - first_row) * p.group) * p.q_head);
      }
#pragma unroll
      for (int k = 0; k < N; ++k) {
        if (E4M3) {                        // in fp16, times a power of two of its row
          const uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
          int top = 0;
#pragma unroll
          for (int q = 0; q < 4; ++q) top = max(top, max(finite_exp(w[q] & 0xffffu), finite_exp(w[q] >> 16)));
#pragma unroll
          for (int o = UPR / 2; o; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
          const int e = min(max(top - 127, kLeastExp), 126);
          const float inv = pow2i(-e);
          uint32_t y[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) y[q] = hf_pack(bf_lo(w[q]) * inv, bf_hi(w[q]) * inv);
          x[k] = make_uint4(y[0], y[1], y[2], y[3]);
          const float scale = p.scale_log2 * pow2i(e);
          if (u == 0) sh.row[0][i * kTile + base + k * RPI] = scale;
          float out = 0.f;
          if (__any_sync(0xffffffffu, any_small<4>(y))) {
#pragma unroll
            for (int q = 0; q < 4; ++q) out += left_out(w[q], inv, y[q]);
#pragma unroll
            for (int o = UPR / 2; o; o >>= 1) out += __shfl_xor_sync(0xffffffffu, out, o);
          }
          lost = fmaxf(lost, scale * fmaxf(out, kLeastLost));
        }
        st_shared_v4u(q_s + i * C::kOpBytes + op_at(base + k * RPI, u), x[k]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mb_arrive(saddr(&sh.q_full));
      if (E4M3) {
        const int most = __reduce_max_sync(0xffffffffu, __float_as_int(lost));    // not negative: ordered as integers
        if (lane == 0) atomicMax(&sh.lost, most);
        pair_or(pair_id, false);
      }
    }
    const float row_scale = E4M3 ? sh.row[0][slot] : p.scale_log2;
    const int pos = slot < rows_here ? it.s.first + new_row(slot) : -1;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;
    const uint32_t s_t = tmem + lanes + kTmemS + i * kTile + half * kHalf;
    const uint32_t o_t = tmem + lanes + kTmemO + i * D + half * (D / 2);
    const int j0 = it.jb[i], j1 = it.je[i], t_begin = it.t_begin;
    const int see_lo = it.all_lo[i], see_hi = it.all_hi[i];
    uint64_t sum[2] = {0, 0};              // two pairs of partial sums
    for (int j = j0; j < j1; ++j) {
      const int n = j - j0;
      const int t0 = t_begin + j * kTile;
      bool ok = wait_warp(sh, saddr(&sh.s_full[i]), n & 1);
      if (E4M3) ok = ok && wait_warp(sh, saddr(&sh.op_full[(2 * j + 1) % NO]), ((2 * j + 1) / NO) & 1);    // its scales
      tm_fence_after();
      const int vn = E4M3 ? sh.vref[j % kScaleSlots] : 0;
      const bool edge = t0 < see_lo || t0 + kTile > see_hi;
      // never zero, which would make NaN of masked scores: a row of zeros over keys of zeros has 2^-219. At the least
      // normal float the others stay below 2^-100
      const float rs = E4M3 ? fmaxf(row_scale * pow2i(max(sh.kref[j % kScaleSlots] - kUp, -126)), FLT_MIN) : row_scale;
      // masked scores are minus infinity
      auto ready = [&](uint32_t* x, int c) {
        if (edge) {
          int lo, hi;
          visible(p, pos, it.s.len, &lo, &hi);
          lo -= t0 + half * kHalf + c;
          hi -= t0 + half * kHalf + c;
#pragma unroll
          for (int k = 0; k < 32; ++k)
            if (k < lo || k >= hi) x[k] = 0xff800000u;
        }
      };
      auto top_of = [&](const uint32_t* x) {
        float a = __uint_as_float(x[0]), b = __uint_as_float(x[1]);
#pragma unroll
        for (int k = 2; k < 32; k += 2) {
          a = fmaxf(a, __uint_as_float(x[k]));
          b = fmaxf(b, __uint_as_float(x[k + 1]));
        }
        return fmaxf(a, b);
      };
      // bf16's threads have the registers to read their 64 scores once, e4m3's read them twice
      constexpr bool kOnce = !E4M3;
      uint32_t x[kOnce ? 64 : 32];
      float top = -INFINITY;
      if (ok) {
        if (kOnce) {
          tm_ld32_start(s_t, x);
          tm_ld32_start(s_t + 32, x + (kOnce ? 32 : 0));
          tm_ld32_wait(x);
          tm_ld32_wait(x + (kOnce ? 32 : 0));
          ready(x, 0);
          ready(x + (kOnce ? 32 : 0), 32);
          top = fmaxf(top_of(x), top_of(x + (kOnce ? 32 : 0)));
        } else {
#pragma unroll 1
          for (int c = 0; c < kHalf; c += 32) {
            tm_ld32_start(s_t + c, x);
            tm_ld32_wait(x);
            ready(x, c);
            top = fmaxf(top, top_of(x));
          }
          tm_ld32_start(s_t, x);           // the first of the second pass
        }
        top *= rs;
      }
      if (pair_or(pair_id, !ok || top > m + kLazy || vn != vr)) {
        // move the reference, to what both threads of the row have seen (or end, if a wait gave up)
        if (pair_or(pair_id, !ok)) break;
        sh.row[half][slot] = top;
        pair_or(pair_id, false);
        const float mn = fmaxf(m, fmaxf(top, sh.row[half ^ 1][slot]));
        float f = mn == m ? 1.f : ex2(m - mn);
        const uint64_t f2 = pair_of(f, f);
        sum[0] = mul2(sum[0], f2);
        sum[1] = mul2(sum[1], f2);
        m = mn;
        if (E4M3) f *= pow2i(max(vr - vn, -127));          // a larger value scale
        vr = vn;
        if (n > 0) {
          if (!kOnce) tm_ld32_wait(x);
#pragma unroll 1
          for (int c = 0; c < D / 2; c += 16) {
            float v[16];
            uint32_t w[16];
            tm_ld16(o_t + c, v);
#pragma unroll
            for (int k = 0; k < 16; ++k) w[k] = __float_as_uint(v[k] * f);
            tm_st16(o_t + c, w);
          }
          if (!kOnce) tm_ld32_start(s_t, x);
        }
      }
      const float ref = (m == -INFINITY ? 0.f : m) - kBias;
      const uint64_t rs2 = pair_of(rs, rs), ref2 = pair_of(-ref, -ref);
      auto weigh = [&](uint32_t* x, int c) {
#pragma unroll
        for (int h = 0; h < 32; h += 16) {
          uint32_t w[8];
#pragma unroll
          for (int k = 0; k < 16; k += 4) {
            float y[4];
            split_pair(fma2(pack2(x + h + k), rs2, ref2), y, y + 1);
            split_pair(fma2(pack2(x + h + k + 2), rs2, ref2), y + 2, y + 3);
#pragma unroll
            for (int q = 0; q < 4; ++q) y[q] = ex2(y[q]);
            sum[0] = add2(sum[0], pair_of(y[0], y[1]));
            sum[1] = add2(sum[1], pair_of(y[2], y[3]));
            w[k / 2] = E4M3 ? hf_pack(y[0], y[1]) : bf_pack(y[0], y[1]);
            w[k / 2 + 1] = E4M3 ? hf_pack(y[2], y[3]) : bf_pack(y[2], y[3]);
          }
          if (!kOnce && h == 16 && c + 32 < kHalf) tm_ld32_start(s_t + c + 32, x);
          tm_st8(s_t + (c + h) / 2, w);
        }
      };
      if (kOnce) {
        weigh(x, 0);
        weigh(x + (kOnce ? 32 : 0), 32);
      } else {
#pragma unroll 1
        for (int c = 0; c < kHalf; c += 32) {
          tm_ld32_wait(x);
          ready(x, c);
          weigh(x, c);
        }
      }
      tm_wait_st();
      tm_fence_before();
      __syncwarp();
      if (lane == 0) mb_arrive(saddr(&sh.p_full[i]));
    }
    float y[4];
    split_pair(sum[0], y, y + 1);
    split_pair(sum[1], y + 2, y + 3);
    l = (y[0] + y[1]) + (y[2] + y[3]);
    // the row's other thread may still be to read this slot: the last move's maximum, or, without a tile, q's scale
    pair_or(pair_id, false);
    sh.row[half][slot] = l;                // met after the block's barrier
  } else if (warp < kMmaWarp) {
    // ---------------------------------------------------------------- helpers
    const int tid = threadIdx.x - kHelper0 * 32;
    const int pair_lo = it.all_lo[1], pair_hi = it.all_hi[0];         // seen by the last row, and by the first
    const int lo = it.lo, t_begin = it.t_begin, t_end = it.t_end, ntiles = it.ntiles;
    bool bad = false;
    if (!E4M3) {
      constexpr int UPR = D / 8, RPI = kHelpers / UPR;      // 16-byte units a row, rows an iteration
      const int u = tid % UPR;
      for (int j = 0; j < ntiles; ++j) {
        const int n = 2 * j + 1, t0 = t_begin + j * kTile;
        if (!wait_warp(sh, saddr(&sh.raw_full[n % NO]), (n / NO) & 1)) break;
        if (t0 < pair_lo || t0 + kTile > pair_hi) {         // also wherever a value is outside [lo, t_end)
          for (int r = tid / UPR; r < kTile; r += RPI) {
            const uint32_t at = op_s + (n % NO) * C::kOpBytes + op_at(r, u);
            if (t0 + r < lo || t0 + r >= t_end) st_shared_v4u(at, make_uint4(0, 0, 0, 0));
            else bad |= any_nonfinite<false>(at);
          }
          fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) mb_arrive(saddr(&sh.op_full[n % NO]));
      }
    } else {
      constexpr int UPR = D / 16, RPI = kHelpers / UPR, N = kTile / RPI;
      const int u = tid % UPR, r0 = tid / UPR;
      const int kv = it.kv;
      const int32_t* table = p.b.table + (int64_t)it.seq * p.b.table_stride;
      // each warp has the scale bytes of all of a tile: positions t0 + 32 h + lane. Pages are asked for two tiles
      // ahead and scales one, and nothing is done with them before their turn.
      uint8_t key_scale[4], value_scale[4];
      auto page_at = [&](int j) {
        const int t = t_begin + j * kTile + (lane & 7) * 16;
        return j < ntiles && t < t_end && (t >> p.c.page_shift) < p.b.width ? table[t >> p.c.page_shift] : -1;
      };
      auto load_scales = [&](int j, int pg) {
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          const int t = t_begin + j * kTile + h * 32 + lane;
          const int page = __shfl_sync(0xffffffffu, pg, h * 2 + lane / 16);
          key_scale[h] = value_scale[h] = 0;
          if ((uint32_t)page < (uint32_t)p.c.pages && j < ntiles && t >= lo && t < t_end) {
            const int64_t so = slot_scale(p.c, page, kv, t);
            key_scale[h] = p.c.ks[so];
            value_scale[h] = p.c.vs[so];
          }
        }
      };
      int pg = page_at(1);
      load_scales(0, page_at(0));
      int kref = -127, vref = -127;
      for (int n = 0; n < 2 * ntiles; ++n) {
        const int j = n >> 1, is_v = n & 1, t0 = t_begin + j * kTile;
        if (!wait_warp(sh, saddr(&sh.raw_full[n % NR]), (n / NR) & 1)) break;
        if (n >= NO && !wait_done(sh, n - NO)) break;
        const uint32_t src = raw_s + (n % NR) * C::kRawBytes + u * 16, dst = op_s + (n % NO) * C::kOpBytes;
        const bool ends = is_v && (t0 < lo || t0 + kTile > t_end);
        const bool look = is_v && (t0 < pair_lo || t0 + kTile > pair_hi);
        // every row by its scale next to the largest so far: a power of two, exact where fp16 reaches
        int e4[4], top = -127;
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          e4[h] = (int)(is_v ? value_scale[h] : key_scale[h]) - 127;
          top = max(top, e4[h]);
        }
        int& ref = is_v ? vref : kref;
        const int before = ref;
        ref = max(ref, __reduce_max_sync(0xffffffffu, top));
        if (is_v) bad |= before > -127 && ref - before > kMostRise;
        if (tid == 0) (is_v ? sh.vref : sh.kref)[j % kScaleSlots] = ref;
        uint4 x[N];
#pragma unroll
        for (int k = 0; k < N; ++k) x[k] = ld_shared_v4u(src + (r0 + k * RPI) * D);
        if (look)
#pragma unroll
          for (int k = 0; k < N; ++k) {
            const int r = r0 + k * RPI;
            if (ends && (t0 + r < lo || t0 + r >= t_end)) x[k] = make_uint4(0, 0, 0, 0);
            const uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
#pragma unroll
            for (int q = 0; q < 4; ++q) bad |= __vcmpeq4(w[q] & 0x7f7f7f7fu, 0x7f7f7f7fu) != 0;
          }
        // scales further apart than fp16 reaches, but for values of zeros, which have the least; a position's byte is
        // never 0
        int low = 0;
#pragma unroll
        for (int h = 0; h < 4; ++h) low = min(low, e4[h] - ref + kUp - kLeast);
        if (__any_sync(0xffffffffu, low < 0)) {
#pragma unroll
          for (int k = 0; k < N; ++k) {
            const int own = __shfl_sync(0xffffffffu, e4[(k * RPI) / 32], (r0 + k * RPI) % 32);
            bad |= own > -127 && own - ref + kUp < kLeast && any_nonzero(x[k]);
          }
        }
#pragma unroll
        for (int k = 0; k < N; ++k) {
          const int r = r0 + k * RPI;
          const int e = max(__shfl_sync(0xffffffffu, e4[(k * RPI) / 32], r % 32) - ref + kUp, -25);
          const uint32_t f = hf_pack(pow2i(e), pow2i(e));
          const uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
          uint32_t y[8];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            y[2 * q] = hf_mul(e4m3x2_f16x2(w[q] & 0xffffu), f);
            y[2 * q + 1] = hf_mul(e4m3x2_f16x2(w[q] >> 16), f);
          }
          st_shared_v4u(dst + op_at(r, 2 * u), make_uint4(y[0], y[1], y[2], y[3]));
          st_shared_v4u(dst + op_at(r, 2 * u + 1), make_uint4(y[4], y[5], y[6], y[7]));
        }
        __syncwarp();
        if (lane == 0) mb_arrive(saddr(&sh.raw_empty[n % NR]));
        if (is_v) {
          load_scales(j + 1, pg);
          pg = page_at(j + 2);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mb_arrive(saddr(&sh.op_full[n % NO]));
      }
    }
    if (bad) *(volatile int*)&sh.bad = 1;
  } else if (warp == kLoadWarp) {
    // ---------------------------------------------------------------- loads
    // lane i < 128 / page size: the tile's i-th page. What is outside [lo, t_end), on no page or on a bad one
    // is asked for behind the pool's last page, which the tensor map returns as zeros.
    const int32_t* table = p.b.table + (int64_t)it.seq * p.b.table_stride;
    const int lo = it.lo, t_begin = it.t_begin, t_end = it.t_end, ntiles = it.ntiles, kv = it.kv;
    const int size = 1 << p.c.page_shift, boxes = kTile >> p.c.page_shift;
    auto page_at = [&](int j) {
      const int t = t_begin + j * kTile + lane * size;
      int pg = -1;
      if (j < ntiles && lane < boxes && t + size > lo && t < t_end) {
        pg = page_of(table, p.b.width, p.c.pages, p.c.page_shift, t);
        if (pg < 0) set_status(p.c.status, CP_ERR_DEVICE_BOUNDS);
      }
      return pg < 0 ? p.c.pages : pg;
    };
    int pg = page_at(0), asked = 0;
    for (int n = 0; n < 2 * ntiles; ++n) {
      const int j = n >> 1, is_v = n & 1;
      if (n >= NR && !(E4M3 ? wait_warp(sh, saddr(&sh.raw_empty[n % NR]), ((n / NR) & 1) ^ 1) : wait_done(sh, n - NR))) break;
      const uint32_t bar = saddr(&sh.raw_full[n % NR]);
      // q goes first: when all blocks start at once, a ring's worth of K and V in front of it is 2 us
      if (n == 1 && !wait_warp(sh, saddr(&sh.q_full), 0)) break;
      asked = n + 1;                       // behind the last wait: what is counted here is on its way
      if (n == 0 && p.stall) continue;
      if (lane == 0) mb_expect(bar, E4M3 ? C::kRawBytes : C::kOpBytes);
      __syncwarp();
      if (lane < boxes) {
        const void* map = is_v ? &maps.v : &maps.k;
        const uint32_t dst = raw_s + (n % NR) * (E4M3 ? C::kRawBytes : C::kOpBytes) + lane * size * (E4M3 ? D : 128);
        tma_load_4d(dst, map, 0, 0, kv, pg, bar);
        if (!E4M3 && D == 128) tma_load_4d(dst + C::kSlab, map, 64, 0, kv, pg, bar);
      }
      __syncwarp();
      if (is_v) pg = page_at(j + 1);
    }
    // what was asked for lands before the block may end, whatever ended the loop
    for (int n = max(p.stall ? 1 : 0, asked - NR); n < asked; ++n)
      for (int k = 0; k < (1 << 20) && !__all_sync(0xffffffffu, mb_try(saddr(&sh.raw_full[n % NR]), (n / NR) & 1)); ++k) {
      }
  } else if (warp == kMmaWarp) {
    // ---------------------------------------------------------------- MMA
    // The instructions between two products matter: about four queued ones cover them, and one takes nearly as long
    // to issue as to run. The warp stays together and one lane issues, so that descriptors are uniform registers'.
    const uint32_t lead = lane == 0;
    const uint32_t id_s = idesc_m128(kTile, E4M3, false), id_o = idesc_m128(D, E4M3, true);
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    const int tiles = __shfl_sync(0xffffffffu, it.ntiles, 0);
    const int b0 = __shfl_sync(0xffffffffu, it.jb[0], 0), b1 = __shfl_sync(0xffffffffu, it.jb[1], 0);
    const int e0 = __shfl_sync(0xffffffffu, it.je[0], 0), e1 = __shfl_sync(0xffffffffu, it.je[1], 0);
    const uint32_t ops = __shfl_sync(0xffffffffu, op_s, 0), q0 = __shfl_sync(0xffffffffu, q_s, 0);
    const uint64_t q_desc = sdesc_sw128(q0), k_desc = sdesc_sw128(ops), v_desc = sdesc_sw128_cols(ops, C::kSlab);
    constexpr uint32_t kOpDesc = C::kOpBytes >> 4;
    const uint32_t ops_full = saddr(sh.op_full), k_full = E4M3 ? ops_full : saddr(sh.raw_full);
    const uint32_t s_full = saddr(sh.s_full), p_full = saddr(sh.p_full), done = saddr(sh.done);
    auto scores = [&](int x, int slot) {
      const uint64_t q = q_desc + x * kOpDesc, k0 = k_desc + slot * kOpDesc;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const uint32_t at = ((k / 4) * C::kSlab + (k % 4) * 32) >> 4;
        tm_mma_lead(lead, tm + kTmemS + x * kTile, q + at, k0 + at, id_s, k > 0);
      }
      tm_commit_lead(lead, s_full + 8 * x);
    };
    auto values = [&](int x, int slot, uint32_t more) {
      const uint64_t v = v_desc + slot * kOpDesc;
#pragma unroll
      for (int k = 0; k < kTile / 16; ++k)
        tm_mma_ts_lead(lead, tm + kTmemO + x * D, tm + kTmemS + x * kTile + (k / 4) * (kTile / 2) + (k % 4) * 8,
                       v + k * (2048 >> 4), id_o, k ? 1u : more);
    };
    // slots of V of tile j and K of tile j + 1, the parity of their turn round the ring, and of the streams' turns
    int sv = NO - 1, sk = 0;
    uint32_t rv = 1, rk = 0, rp0 = 0, rp1 = 0;
    bool ok = wait_warp(sh, saddr(&sh.q_full), 0);
    for (int j = -1; ok && j < tiles; ++j) {
      const bool v0 = j >= b0 && j < e0, v1 = j >= b1 && j < e1;                     // streams with values, and scores
      const bool s0 = j + 1 >= b0 && j + 1 < e0, s1 = j + 1 >= b1 && j + 1 < e1;
      // one wait for all that stream 0 needs, a lane a barrier
      const uint32_t bar = lane == 0 ? ops_full + 8 * sv : lane == 1 ? k_full + 8 * sk : p_full;
      const uint32_t par = lane == 0 ? rv : lane == 1 ? rk : rp0;
      ok = wait_lanes(sh, bar, par, lane == 0 ? j >= 0 : lane == 1 ? j + 1 < tiles : lane == 2 && v0);
      if (!ok) break;
      tm_fence_after();
      if (v0) {
        values(0, sv, j > b0);
        rp0 ^= 1;
      }
      if (s0) scores(0, sk);
      if (v1) {
        ok = wait_lanes(sh, p_full + 8, rp1, lane == 0);
        if (!ok) break;
        tm_fence_after();
        values(1, sv, j > b1);
        rp1 ^= 1;
      }
      if (s1) scores(1, sk);
      tm_commit_lead(lead, done + 8 * ((j + 1) & 3));
      // loads alternate K, V: V of tile j + 1 follows K of tile j + 1
      sv = sk + 1;
      rv = rk;
      if (sv == NO) sv = 0, rv ^= 1;
      sk = sv + 1;
      rk = rv;
      if (sk == NO) sk = 0, rk ^= 1;
    }
    tm_commit_lead(lead, saddr(&sh.o_full));
    // after a wait that gave up, the products in flight still end before TMEM is given back
    for (int x = 0; x < (1 << 20) && !__all_sync(0xffffffffu, mb_try(saddr(&sh.o_full), 0)); ++x) {
    }
  }
  __syncwarp();
  __syncthreads();
  tm_fence_after();

  const bool failed = sh.abort != 0;
  // rows of q that fp16 could not hold, next to the largest keys that the block met
  const bool far_q = E4M3 && !failed && it.ntiles > 0 &&
                     __int_as_float(sh.lost) * (448.f * pow2i(max(sh.kref[(it.ntiles - 1) % kScaleSlots], -126))) > kMostLost;
  if (failed && threadIdx.x == 0) set_status(p.c.status, CP_ERR_TIMEOUT);
  constexpr int kPitch = D + 4;
  static_assert(kPairRows * kPitch * 4 <= (2 + NO) * C::kOpBytes, "the rows fit the operands' memory");
  float* averages = reinterpret_cast<float*>(ops);
  const bool cluster = p.a.chunk_cluster && !it.whole;       // the item's parts are a cluster's blocks
  if (!failed && (sh.bad || far_q)) {
    plain_rows<D, E4M3>(p, it.s, it.seq, it.kv, it.row0, it.row0 + it.rows_here, it.t_begin, it.t_end, it.part, it.whole, warp,
                        C::kThreads / 32, cluster ? averages : nullptr, sh.row[0], kPitch);
  } else if (!failed && warp < kSoftWarps) {
    // rows leave through the operands' memory, so that a row is written at once and not by its threads piece by piece
    const int slot = threadIdx.x / 256 * kTile + (threadIdx.x & 127), half = (warp >> 2) & 1, i = warp >> 3;
    const int pair_id = 1 + i * 4 + (warp & 3);
    const uint32_t o_t = sh.tmem + ((uint32_t)(warp & 3) << 21) + kTmemO + i * D + half * (D / 2);
    const bool any = it.je[i] > it.jb[i], whole = it.whole;
    const int group = p.group, first_row = it.first_row, first_head = it.first_head, head0 = it.kv * group;
    const uint32_t magic = p.magic;
    auto place = [&](int r, int64_t* row, int* head) {
      const int q = (int)(((uint32_t)(first_head + r) * magic) >> 16);
      *row = it.s.row0 + first_row + q;
      *head = head0 + first_head + r - q * group;
    };
    l = sh.row[0][slot] + sh.row[1][slot];
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const float e = E4M3 ? pow2i(min(max(vr - kUp, -126), 127)) : 1.f;
    float* stage = averages + (i * kTile + (warp & 3) * 32) * kPitch;
    uint16_t* stage16 = reinterpret_cast<uint16_t*>(stage);
    constexpr int kPitch16 = D + 8;
#pragma unroll 1
    for (int c = 0; c < D / 2; c += 32) {
      float v[32];
      if (any) tm_ld32(o_t + c, v);
#pragma unroll
      for (int x = 0; x < 32; ++x) v[x] = any && inv != 0.f ? v[x] * inv * e : 0.f;
      if (whole) {
#pragma unroll
        for (int x = 0; x < 32; x += 8)
          *reinterpret_cast<uint4*>(stage16 + lane * kPitch16 + half * (D / 2) + c + x) =
              make_uint4(bf_pack(v[x], v[x + 1]), bf_pack(v[x + 2], v[x + 3]), bf_pack(v[x + 4], v[x + 5]), bf_pack(v[x + 6], v[x + 7]));
      } else {
#pragma unroll
        for (int x = 0; x < 32; x += 4)
          *reinterpret_cast<float4*>(stage + lane * kPitch + half * (D / 2) + c + x) = make_float4(v[x], v[x + 1], v[x + 2], v[x + 3]);
      }
    }
    const float lse = l == 0.f ? -INFINITY : m + log2f(l) - kBias;
    int64_t row;
    int head;
    if (slot < it.rows_here && !whole && !cluster && half == 0) {
      place(slot, &row, &head);
      store_lse(p, it.part, row, head, lse);
    }
    tm_fence_before();
    pair_or(pair_id, false);
    if (cluster && half == 0) sh.row[0][slot] = lse;
    // 16 of the rows a warp, their elements side by side, 16 bytes a lane; the next row's place by counting on
    const int rows0 = i * kTile + (warp & 3) * 32 + half * 16;
    auto rows_out = [&](auto per, auto store) {
      constexpr int LPR = D / decltype(per)::value, RPI = 32 / LPR;
      const int r0 = lane / LPR, d = lane % LPR * decltype(per)::value;
      int left = it.rows_here - (rows0 + r0);
      place(rows0 + r0, &row, &head);
      head -= head0;
#pragma unroll 4
      for (int k = 0; k < 16; k += RPI, left -= RPI) {
        if (left > 0) store(half * 16 + r0 + k, d);
        head += RPI;
        for (; head >= group; head -= group) ++row;
      }
    };
    if (whole) {
      const int64_t o_row = p.o_row, o_head = p.o_head;
      uint16_t* out = p.out + head0 * o_head;
      rows_out(std::integral_constant<int, 8>(), [&](int r, int d) {
        *reinterpret_cast<uint4*>(out + row * o_row + head * o_head + d) = *reinterpret_cast<const uint4*>(stage16 + r * kPitch16 + d);
      });
    } else if (!cluster) {
      float* part_o = p.part_o + ((int64_t)it.part * p.b.rows * p.q_heads + head0) * D;
      rows_out(std::integral_constant<int, 4>(), [&](int r, int d) {
        *reinterpret_cast<float4*>(part_o + (row * p.q_heads + head) * D + d) = *reinterpret_cast<const float4*>(stage + r * kPitch + d);
      });
    }
  }
  __syncthreads();
  if (cluster) {
    // each of the item's blocks joins every n-th row, out of all blocks' shared memory; they leave together
    cluster_sync_all();
    constexpr int LPR = D / 4, RPI = 32 / LPR;
    const int d = lane % LPR * 4;
#pragma unroll 1
    for (int r = it.part + it.parts * (warp * RPI + lane / LPR); r < it.rows_here; r += it.parts * (C::kThreads / 32) * RPI) {
      float x[4];
      join4(saddr(averages + r * kPitch + d), saddr(&sh.row[0][r]), it.parts, x);
      const int q = (int)(((uint32_t)(it.first_head + r) * p.magic) >> 16);
      store4<D>(p, 0, true, it.s.row0 + it.first_row + q, it.kv * p.group + it.first_head + r - q * p.group, d, x);
    }
    __syncwarp();
    cluster_sync_all();
  }
  if (warp == kMmaWarp) {
    tm_fence_after();
    tm_dealloc(sh.tmem, kTmemCols);
  }
}

}  // namespace

template <int D, bool E4M3>
static cudaError_t prepare() {
  return cudaFuncSetAttribute(attend_chunk_kernel<D, E4M3>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              Smem<D, E4M3>::kBytes);
}
cudaError_t prepare_attend_chunk() {
  for (cudaError_t e : {prepare<64, false>(), prepare<64, true>(), prepare<128, false>(), prepare<128, true>()})
    if (e != cudaSuccess) return e;
  return cudaSuccess;
}

template <int D, bool E4M3>
static cudaError_t launch(const AttendParams& p, const CacheMaps& maps, cudaStream_t s) {
  const dim3 grid((unsigned)(p.c.heads * chunk_pairs(p.b, p.group)), p.a.chunk_parts);
  return launch_as(attend_chunk_kernel<D, E4M3>, grid, 1, p.a.chunk_cluster ? p.a.chunk_parts : 1, false,
                   Cfg<D, E4M3>::kThreads, Smem<D, E4M3>::kBytes, s, p, maps);
}
cudaError_t launch_attend_chunk(const AttendParams& p, const CacheMaps& maps, int head_dim, bool e4m3, cudaStream_t s) {
  if (head_dim == 128) return e4m3 ? launch<128, true>(p, maps, s) : launch<128, false>(p, maps, s);
  return e4m3 ? launch<64, true>(p, maps, s) : launch<64, false>(p, maps, s);
}

}  // namespace cache
}  // namespace cp
