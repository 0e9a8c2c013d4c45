// cp_attend.cu -- attention of a batch's new rows over the paged cache: the
// plan of a call, the step kernel (up to 16 rows a kv head, bound by reading
// the cache once) and the kernel that joins an item's parts. Sequences with
// more rows go to cp_attend_chunk.cu.
#include <algorithm>

#include "cp_attend.cuh"

namespace cp {
namespace cache {

// ------------------------------------------------------------------ plan
constexpr int kStepBlocks = 2 * kSms; // step blocks resident at once
constexpr int kStepCluster = kMostCluster;
constexpr int kMaxStepChunk = 4096;   // positions a step block holds page numbers for

static int step_tile(int head_dim, bool e4m3) { return 4 * (e4m3 ? 32 : 16) * (128 / head_dim); }

AttendPlan plan_attend(const BatchView& b, int kv_heads, int q_heads, int head_dim, bool e4m3, bool causal,
                       int window) {
  AttendPlan a{};
  const int group = q_heads / kv_heads;
  a.use_chunk = (int64_t)b.max_new * group > kStepRows;
  // where every sequence may have max_new rows the chunk kernel takes what few may turn out shorter: an empty
  // launch of the step kernel costs 3 to 6 us
  a.use_step = group <= kStepRows && (!a.use_chunk || (int64_t)b.n * b.max_new > b.rows);
  // the most positions an item spans: all, or a window and the rows behind it
  const int64_t rows = std::min(b.max_new, kStepRows / std::min(group, kStepRows));
  int64_t span = b.max_len;
  if (window > 0) span = std::min<int64_t>(span, (int64_t)window + rows + kStepAlign - 1);
  const int tile = step_tile(head_dim, e4m3);
  const int64_t items = (int64_t)b.n * kv_heads;
  // two rounds of blocks if every sequence were the longest: 4, 8 and 16 rounds (a better balance, more starts and
  // joins) measured up to 4, 2 and 6 % slower on ragged batches of 64 and 10 to 20 % on few long or equal sequences
  const int64_t want = std::max<int64_t>(1, kStepBlocks * 2 / items);
  int64_t chunk = (span + want - 1) / want;
  chunk = std::min<int64_t>(std::max<int64_t>((chunk + tile - 1) / tile * tile, tile), kMaxStepChunk);
  // A call whose blocks are all resident at once may join an item's parts within a cluster, through shared memory,
  // and needs no second launch and no workspace: one sequence of 777 positions 18 -> 8.5 us a call. Longer
  // ones need more parts than a cluster has blocks.
  if (items * kStepCluster <= kStepBlocks && span <= kStepCluster * 512) {
    chunk = std::max<int64_t>((span + kStepCluster - 1) / kStepCluster + tile - 1, tile) / tile * tile;
    a.step_cluster = 1;
  }
  a.step_wide = rows * group > 8;
  a.step_chunk = (int)chunk;
  a.step_parts = a.use_step ? (int)std::max<int64_t>(1, (span + chunk - 1) / chunk) : 0;
  if (a.use_chunk) {
    // As many items as the rows make when every sequence has max_new of them, cut into the number of parts that costs
    // least on 152 SMs.
    const int64_t per = ((int64_t)b.max_new * group + kPairRows - 1) / kPairRows;
    const int64_t blocks = std::max<int64_t>(1, (int64_t)b.rows / b.max_new) * per * kv_heads;
    int64_t all = b.max_len;
    // a window spans itself and the item's rows; not causal, the rows up to the last of the sequence
    const int64_t ahead = causal ? std::min(b.max_new, (kPairRows + group - 1) / group + 1) : b.max_new;
    if (window > 0) all = std::min<int64_t>(all, (int64_t)window + ahead + kChunkAlign - 1);
    // In nanoseconds: rounds of blocks (chunk_rounds_ns), joining the parts of a cluster 2500, or through the workspace 3000 and the parts' results written and read again at 5 TB/s. Clusters
    // only where all blocks are resident at once: their blocks start and leave together (a ragged batch in two rounds
    // 169 us, in clusters 179).
    double best = 0;
    int64_t parts = 1;
    const double join_ns = 2.0 * b.rows * q_heads * head_dim * 4 / 5000;
    for (int64_t n = 1; n <= 32; ++n) {
      const double cost = chunk_rounds_ns(blocks * n, (int)(((all + n - 1) / n + 127) / 128), head_dim) +
                          (n == 1 ? 0 : n <= kMostCluster && blocks * n <= kSms ? 2500 : 3000 + n * join_ns);
      if (n == 1 || cost < best) best = cost, parts = n;
    }
    a.chunk_chunk = (int)(((all + parts - 1) / parts + 127) / 128 * 128);
    a.chunk_parts = (int)((all + a.chunk_chunk - 1) / a.chunk_chunk);
    a.chunk_span = (int)all;
    // a batch in more than one round, of items that one round holds: ragged, they may leave one of longer parts
    a.chunk_coarser = b.n > 1 && a.chunk_parts > 1 && blocks * a.chunk_parts > kSms && blocks <= kSms;
    a.chunk_cluster = a.chunk_parts > 1 && a.chunk_parts <= kMostCluster && blocks * a.chunk_parts <= kSms;
  }
  return a;
}

size_t attend_workspace(const AttendPlan& a, const BatchView& b, int q_heads, int head_dim) {
  const int parts = kept_parts(a);
  return parts > 1 ? (size_t)parts * b.rows * q_heads * (head_dim + 1) * sizeof(float) + 16 : 0;
}

namespace {

// ------------------------------------------------------------------ step kernel
constexpr int kStepWarps = 4;
constexpr int kStages = 3;
constexpr int kStageBytes = 8192;     // a warp's tile: K and V, 4 KB each
constexpr int kGroups = kMaxStepChunk / 16;
// e4m3: most powers of two between a value's scale and the largest. fp16 weights start at 2^8 and keep 11 bits down
// to 2^-14: 2^12 down, those a thousandth of a row's largest still do.
constexpr int kMostGap = 12;

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t a, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
// The 8 x 8 matrix of 16-bit elements whose row i lanes 4i .. 4i+3 hold, transposed.
__device__ __forceinline__ uint32_t transposed(uint32_t a) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
  return r;
}
template <bool HALF>
__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  if (HALF)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

constexpr int kStepSmem = kStepWarps * kStages * kStageBytes;
static_assert(kStepSmem >= kStepWarps * kStepRows * (128 + 4) * 4, "the ring holds the warps' averages");

struct StepShared {
  float scale_k[kStepWarps][64];      // e4m3: per position of the warp's tile, its key's scale times the softmax's
  float scale_v[kStepWarps][64];      // and its value's scale relative to the warp's reference
  int pages[kGroups];                 // page of each 16 positions of the part, -1: none
  float m[kStepWarps][kStepRows], l[kStepWarps][kStepRows];
  uint16_t rows_pad[8];
};

// The parts of an item, weighed by their sums, by the cluster whose blocks have them: each takes a share of the
// elements and reads the others' shared memory. Blocks without a part have left; the others leave together.
constexpr int kAvgAt = 10240;           // floats into the ring: behind the warps' averages
static_assert(kAvgAt >= kStepWarps * kStepRows * (128 + 4) && (kAvgAt + kStepRows * 129) * 4 <= kStepSmem, "the ring's plan");
template <int D>
__device__ __forceinline__ void join_cluster(const AttendParams& p, const Seq& s, int kv, int nrows, int parts, float* avg,
                                             float* avg_lse) {
  __syncwarp();
  ptx::cluster_sync_all();
  const uint32_t at = smem_u32(avg), at_lse = smem_u32(avg_lse);
  for (int u = blockIdx.x * (kStepWarps * 32) + threadIdx.x; u < nrows * (D / 4); u += parts * (kStepWarps * 32)) {
    const int r = u / (D / 4), d = u % (D / 4) * 4;
    float x[4];
    join4(at + (r * D + d) * 4, at_lse + r * 4, parts, x);
    store4<D>(p, 0, true, s.row0 + r / p.group, kv * p.group + r % p.group, d, x);
  }
  __syncwarp();
  ptx::cluster_sync_all();
}

// One block a (part, kv head, sequence); its four warps take the part's tiles
// in turn, each with a running maximum, sum and product of its own and its own
// ring of asynchronous copies, so that nothing in the loop waits for another
// warp; they are joined once at the end.
//
// The products are transposed, positions (and then columns of v) along the 16
// rows of the matrix instruction and the sequence's rows times the kv head's
// query heads along its columns: 8 of them, NT times. S^T = K q^T takes keys as
// they lie, O^T = V^T P^T values transposed on their way out of shared memory;
// S^T's layout is a transposition of 8 x 8 away from P^T's. (With the rows
// along the 16, steps of two heads spent twice the instructions and registers
// on rows that are not there: 64 sequences of 500 to 12001 e4m3 positions
// 151 us, now 140, the kernel alone; 5.8 TB/s.)
//
// K and V go to shared memory as they lie (16-byte units exchanged within a
// row so that ldmatrix meets no bank twice). e4m3 is widened to fp16 in
// registers (exact): q is fp16 times a power of two of its row, the key's
// scale multiplies the score, the value's scale the weight, relative to the
// largest seen (so that weight * scale stays in fp16's range; weights start
// at 2^8 to use it). A 4-byte fragment of e4m3 is four neighbouring elements
// where the instruction wants two and two: the sum over the head does not
// mind the order, so q is loaded in it, and two neighbouring columns of v
// become rows 8 apart.
//
// bf16 is bound by HBM: 64 sequences of one row, 16/8 heads of 128, 311 to
// 6000 positions 127 us a call, 6.5 TB/s, 96 % of the copy rate. e4m3 by the
// chain of conversions in front of each product, at 7.6 warps an SM: the 64
// sequences above 143 us a call, 85 % of the copy rate, with issue slots 44 %
// and the integer pipe 48 % busy (twice bf16's: widening is most of it).
template <int D, bool E4M3, int NT, bool CLUSTER>
__device__ __forceinline__ void step_block(const AttendParams& p) {
  constexpr int TK = (E4M3 ? 32 : 16) * (128 / D);    // positions a tile
  constexpr int ES = E4M3 ? 1 : 2;
  constexpr int UPR = D * ES / 16;                    // 16-byte units a row: 16, 8 or 4
  constexpr int MT = TK / 16;                         // score tiles of 16 positions
  constexpr int KS = D / 16;                          // steps over the head
  constexpr int RPL = 32 / UPR;                       // rows that one copy of the warp covers
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ StepShared sh;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  const int seq = blockIdx.z, kv = blockIdx.y, part = blockIdx.x;
  const Seq s = seq_of(p.b, seq, p.c.status);
  const int nrows = s.n * p.group;
  if (s.n == 0 || nrows > kStepRows) return;
  const Range range = item_range(p, s.first, s.first + s.n - 1, s.len, kStepAlign);
  const int parts = parts_of(range, p.a.step_chunk);
  if (part >= max(parts, 1)) return;
  const int t_begin = range.base + part * p.a.step_chunk;
  const int t_end = t_begin + min(p.a.step_chunk, range.hi - t_begin);    // positions end near those of 32 bits
  // every row sees [lo_all, hi_all) of the item; outside it a tile is masked by row
  int lo_all, hi_all, unused;
  visible(p, s.first + s.n - 1, s.len, &lo_all, &unused);
  visible(p, s.first, s.len, &unused, &hi_all);

  const int32_t* table = p.b.table + (int64_t)seq * p.b.table_stride;
  for (int i = threadIdx.x; i * 16 < t_end - t_begin; i += kStepWarps * 32) {
    const int pg = page_of(table, p.b.width, p.c.pages, p.c.page_shift, t_begin + i * 16);
    if (pg < 0) set_status(p.c.status, CP_ERR_DEVICE_BOUNDS);
    sh.pages[i] = pg;
  }
  __syncthreads();

  const uint32_t my_ring = smem_u32(ring) + warp * (kStages * kStageBytes);
  const int ntiles = t_end > t_begin ? (t_end - t_begin + TK - 1) / TK : 0;
  const int mine = ntiles > warp ? (ntiles - warp + kStepWarps - 1) / kStepWarps : 0;
  const uint8_t* kb = p.c.k + (int64_t)kv * p.c.head_b;
  const uint8_t* vb = p.c.v + (int64_t)kv * p.c.head_b;
  const int mask = (1 << p.c.page_shift) - 1;

  auto swz = [](int row, int unit) { return UPR == 4 ? unit ^ ((row >> 1) & 3) : unit ^ (row & 7); };
  // scale bytes of the lane's positions (two in a tile of 64): of the tile two on, and of the next
  uint8_t ks_next[2] = {0, 0}, vs_next[2] = {0, 0}, ks_cur[2] = {0, 0}, vs_cur[2] = {0, 0};
  // Tile i of this warp into its ring slot: rows outside [lo, t_end) or on no page are zeros.
  auto issue = [&](int i) {
    if (i < mine) {
      const int t0 = t_begin + (i * kStepWarps + warp) * TK;
      const uint32_t dst = my_ring + (i % kStages) * kStageBytes;
      const int u = lane % UPR, r0 = lane / UPR;
#pragma unroll
      for (int gr = 0; gr < TK / 16; ++gr) {
        const int tg = t0 + gr * 16;
        const int pg = tg < t_end ? sh.pages[(tg - t_begin) >> 4] : -1;
        const int64_t off = (int64_t)max(pg, 0) * p.c.page_b + (int64_t)((tg & mask) + r0) * p.c.tok_b + u * 16;
#pragma unroll
        for (int j = 0; j < 16 / RPL; ++j) {
          const int row = gr * 16 + j * RPL + r0, t = t0 + row;
          const bool on = pg >= 0 && t >= range.lo && t < t_end;
          const int64_t o = on ? off + (int64_t)(j * RPL) * p.c.tok_b : 0;
          const uint32_t d = dst + row * (UPR * 16) + swz(row, u) * 16;
          cp16(d, kb + o, on);
          cp16(d + kStageBytes / 2, vb + o, on);
        }
      }
      if (E4M3) {
#pragma unroll
        for (int x = 0; x < (TK + 31) / 32; ++x) {
          const int t = t0 + x * 32 + lane;
          ks_next[x] = vs_next[x] = 0;
          if (t >= range.lo && t < t_end) {
            const int pg = sh.pages[(t - t_begin) >> 4];
            if (pg >= 0) {
              const int64_t so = slot_scale(p.c, pg, kv, t);
              ks_next[x] = p.c.ks[so];
              vs_next[x] = p.c.vs[so];
            }
          }
        }
      }
    }
    cp_commit();
  };

  // q fragments, and for e4m3 the power of two taken out of each row; this thread's columns of the scores are rows
  // 8 n + 2 c and 8 n + 2 c + 1
  uint32_t qf[KS][NT][2];
  float qs[NT][2];
  int lo[NT][2], hi[NT][2];
  float lost = 0.f;                 // the most that a row's fp16 left of q out, times its scale (kMostLost)
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int r = n * 8 + g;
    const bool on = r < nrows;
    const uint16_t* qp = p.q + (int64_t)(s.row0 + (on ? r / p.group : 0)) * p.q_row +
                         (int64_t)(kv * p.group + (on ? r % p.group : 0)) * p.q_head;
    if (!E4M3) {
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        qf[k][n][0] = on ? *reinterpret_cast<const uint32_t*>(qp + k * 16 + 2 * c) : 0u;
        qf[k][n][1] = on ? *reinterpret_cast<const uint32_t*>(qp + k * 16 + 8 + 2 * c) : 0u;
      }
      qs[n][0] = qs[n][1] = p.scale_log2;
    } else {
      uint2 raw[KS];
      int top = 0;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        raw[k] = on ? *reinterpret_cast<const uint2*>(qp + k * 16 + 4 * c) : make_uint2(0u, 0u);
        const uint32_t w[2] = {raw[k].x, raw[k].y};
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          top = max(top, finite_exp(w[j] & 0xffffu));
          top = max(top, finite_exp(w[j] >> 16));
        }
      }
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int e = min(max(top - 127, kLeastExp), 126);
      const float inv = pow2i(-e);
      bool small = false;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        qf[k][n][0] = hf_pack(bf_lo(raw[k].x) * inv, bf_hi(raw[k].x) * inv);
        qf[k][n][1] = hf_pack(bf_lo(raw[k].y) * inv, bf_hi(raw[k].y) * inv);
        small |= any_small<2>(qf[k][n]);
      }
      float out = 0.f;
      if (__any_sync(0xffffffffu, small && on)) {
#pragma unroll
        for (int k = 0; k < KS; ++k) out += left_out(raw[k].x, inv, qf[k][n][0]) + left_out(raw[k].y, inv, qf[k][n][1]);
        out += __shfl_xor_sync(0xffffffffu, out, 1);
        out += __shfl_xor_sync(0xffffffffu, out, 2);
      }
      lost = fmaxf(lost, p.scale_log2 * pow2i(e) * fmaxf(out, kLeastLost));
#pragma unroll
      for (int j = 0; j < 2; ++j) qs[n][j] = p.scale_log2 * pow2i(__shfl_sync(0xffffffffu, e, (2 * c + j) * 4));
    }
    // the positions that the columns' rows see
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int row = n * 8 + 2 * c + j;
      lo[n][j] = hi[n][j] = 0;
      if (row < nrows) visible(p, s.first + row / p.group, s.len, &lo[n][j], &hi[n][j]);
    }
  }

  constexpr float kBias = E4M3 ? 8.f : 0.f;
  float m[NT][2], l[NT][2];
  float o[D / 16][NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    m[n][0] = m[n][1] = -INFINITY;
    l[n][0] = l[n][1] = 0.f;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) o[i][n][0] = o[i][n][1] = o[i][n][2] = o[i][n][3] = 0.f;
  }
  int ev_ref = -1000, ek_top = -126;
  bool bad = false;

#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) {
#pragma unroll
    for (int x = 0; x < 2; ++x) ks_cur[x] = ks_next[x], vs_cur[x] = vs_next[x];
    issue(i);
  }
  for (int it = 0; it < mine; ++it) {
    const int t0 = t_begin + (it * kStepWarps + warp) * TK;
    bool far[2] = {false, false};
    if (E4M3) {
      // this tile's scales to shared memory, where the lanes find the ones of their columns
      int ek[2], ev[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        ek[x] = (int)ks_cur[x] - 127;
        ek_top = max(ek_top, ek[x]);
        ev[x] = (int)vs_cur[x] - 127;
        ks_cur[x] = ks_next[x];
        vs_cur[x] = vs_next[x];
      }
      int top = -1000;
#pragma unroll
      for (int x = 0; x < (TK + 31) / 32; ++x) top = max(top, ev[x]);
      const int ref = max(ev_ref, __reduce_max_sync(0xffffffffu, top));
      if (ref != ev_ref) {
        bad |= ev_ref > -127 && ref - ev_ref > kMostRise;
        const float f = pow2i(max(ev_ref - ref, -127));
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
          for (int n = 0; n < NT; ++n) o[i][n][0] *= f, o[i][n][1] *= f, o[i][n][2] *= f, o[i][n][3] *= f;
        ev_ref = ref;
      }
#pragma unroll
      for (int x = 0; x < (TK + 31) / 32; ++x) {
        sh.scale_k[warp][x * 32 + lane] = pow2i(ek[x]);
        sh.scale_v[warp][x * 32 + lane] = pow2i(max(ev[x] - ref, -127));
        far[x] = ev[x] > -127 && ev[x] - ref < -kMostGap;      // a position's byte is never 0
      }
    }
    cp_wait<kStages - 2>();
    __syncwarp();
    const uint32_t tile = my_ring + (it % kStages) * kStageBytes;
    const uint32_t vtile = tile + kStageBytes / 2;
    const bool edge = t0 < lo_all || t0 + TK > hi_all;
    if (edge && nrows > p.group) {
      // a value that some row must not see may not be multiplied, not even by zero, unless it is finite
      const int u = lane % UPR, r0 = lane / UPR;
      for (int row = r0; row < TK; row += RPL)
        bad |= any_nonfinite<E4M3>(vtile + row * (UPR * 16) + u * 16);
    }
    if (E4M3 && __any_sync(0xffffffffu, far[0] || far[1])) {   // values of zeros have the least scale, and may be far
#pragma unroll
      for (int x = 0; x < (TK + 31) / 32; ++x)
        for (int u = 0; far[x] && u < UPR; ++u)
          bad |= any_nonzero(ptx::ld_shared_v4u(vtile + (x * 32 + lane) * (UPR * 16) + u * 16));
    }
    // scores
    float sc[MT][NT][4];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int n = 0; n < NT; ++n) sc[i][n][0] = sc[i][n][1] = sc[i][n][2] = sc[i][n][3] = 0.f;
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      if (!E4M3) {
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          uint32_t a[4];
          const int row = i * 16 + ((lane >> 3) & 1) * 8 + (lane & 7), unit = k * 2 + (lane >> 4);
          ldsm4(tile + row * (UPR * 16) + swz(row, unit) * 16, a);
#pragma unroll
          for (int n = 0; n < NT; ++n) mma16816<false>(sc[i][n], a, qf[k][n][0], qf[k][n][1]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < MT; i += 2) {
          uint32_t b[4];
          const int row = i * 16 + lane;
          ldsm4(tile + row * (UPR * 16) + swz(row, k) * 16, b);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t a[4] = {e4m3x2_f16x2(b[2 * h] & 0xffffu), e4m3x2_f16x2(b[2 * h + 1] & 0xffffu),
                                   e4m3x2_f16x2(b[2 * h] >> 16), e4m3x2_f16x2(b[2 * h + 1] >> 16)};
#pragma unroll
            for (int n = 0; n < NT; ++n) mma16816<true>(sc[i + h][n], a, qf[k][n][0], qf[k][n][1]);
          }
        }
      }
    }
    // scale, mask, running maximum
    float mx[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) mx[n][0] = m[n][0], mx[n][1] = m[n][1];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      float fk[2] = {1.f, 1.f};
      if (E4M3) fk[0] = sh.scale_k[warp][i * 16 + g], fk[1] = sh.scale_k[warp][i * 16 + 8 + g];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          sc[i][n][j] *= E4M3 ? qs[n][j & 1] * fk[j >> 1] : qs[n][j & 1];
          const int t = t0 + i * 16 + (j >> 1) * 8 + g;
          if (edge && (t < lo[n][j & 1] || t >= hi[n][j & 1])) sc[i][n][j] = -INFINITY;
          mx[n][j & 1] = fmaxf(mx[n][j & 1], sc[i][n][j]);
        }
    }
    float ref[NT][2];
    bool moved = false;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) mx[n][j] = fmaxf(mx[n][j], __shfl_xor_sync(0xffffffffu, mx[n][j], x));
        moved |= mx[n][j] > m[n][j];
        ref[n][j] = (mx[n][j] == -INFINITY ? 0.f : mx[n][j]) - kBias;
      }
    if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float f = mx[n][j] == m[n][j] ? 1.f : ex2(m[n][j] - mx[n][j]);
          l[n][j] *= f;
          m[n][j] = mx[n][j];
#pragma unroll
          for (int i = 0; i < D / 16; ++i) o[i][n][j] *= f, o[i][n][2 + j] *= f;
        }
    }
    // weights, and from (position, row) to (row, position)
    uint32_t pf[MT][NT][2];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      float fv[2] = {1.f, 1.f};
      if (E4M3) fv[0] = sh.scale_v[warp][i * 16 + g], fv[1] = sh.scale_v[warp][i * 16 + 8 + g];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          w[j] = ex2(sc[i][n][j] - ref[n][j & 1]);
          l[n][j & 1] += w[j];
        }
        pf[i][n][0] = transposed(E4M3 ? hf_pack(w[0] * fv[0], w[1] * fv[0]) : bf_pack(w[0], w[1]));
        pf[i][n][1] = transposed(E4M3 ? hf_pack(w[2] * fv[1], w[3] * fv[1]) : bf_pack(w[2], w[3]));
      }
    }
    // values times weights
#pragma unroll
    for (int i = 0; i < MT; i += E4M3 ? 2 : 1) {
#pragma unroll
      for (int d = 0; d < D / 16; ++d) {
        uint32_t b[4];
        if (!E4M3) {
          const int row = i * 16 + (lane >> 4) * 8 + (lane & 7), unit = d * 2 + ((lane >> 3) & 1);
          ldsm4t(vtile + row * (UPR * 16) + swz(row, unit) * 16, b);
#pragma unroll
          for (int n = 0; n < NT; ++n) mma16816<false>(o[d][n], b, pf[i][n][0], pf[i][n][1]);
        } else {
          const int row = i * 16 + lane;
          ldsm4t(vtile + row * (UPR * 16) + swz(row, d) * 16, b);
          // a register: two columns of position 2c, then of 2c + 1; split by column
#pragma unroll
          for (int j = 0; j < 4; ++j) b[j] = __byte_perm(b[j], 0, 0x3120);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t a[4] = {e4m3x2_f16x2(b[2 * h] & 0xffffu), e4m3x2_f16x2(b[2 * h] >> 16),
                                   e4m3x2_f16x2(b[2 * h + 1] & 0xffffu), e4m3x2_f16x2(b[2 * h + 1] >> 16)};
#pragma unroll
            for (int n = 0; n < NT; ++n) mma16816<true>(o[d][n], a, pf[(i + h) % MT][n][0], pf[(i + h) % MT][n][1]);
          }
        }
      }
    }
    __syncwarp();
    issue(it + kStages - 1);
  }
  cp_wait<0>();
  if (E4M3 && mine > 0) bad |= lost * (448.f * pow2i(__reduce_max_sync(0xffffffffu, ek_top))) > kMostLost;
  const bool whole = parts <= 1;
  // a cluster's parts: each block's averages and log-sums, where the others read them
  float* avg = reinterpret_cast<float*>(ring) + kAvgAt;
  float* avg_lse = avg + kStepRows * 128;
  if (__syncthreads_or(bad)) {
    plain_rows<D, E4M3>(p, s, seq, kv, 0, nrows, t_begin, t_end, part, whole, warp, kStepWarps, CLUSTER ? avg : nullptr, avg_lse);
    if (CLUSTER && !whole) join_cluster<D>(p, s, kv, nrows, parts, avg, avg_lse);
    return;
  }

  // join the warps: each leaves its average and its sum, the block weighs them
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) l[n][j] += __shfl_xor_sync(0xffffffffu, l[n][j], x);
      const int r = n * 8 + 2 * c + j;
      if (g == 0) {
        sh.m[warp][r] = m[n][j];
        sh.l[warp][r] = l[n][j];
      }
      const float f = l[n][j] == 0.f ? 0.f : 1.f / l[n][j];
      const float e = E4M3 ? pow2i(min(max(ev_ref, -126), 127)) : 1.f;
      float* dst = reinterpret_cast<float*>(ring) + (warp * kStepRows + r) * (D + 4);
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        if (E4M3) {
          *reinterpret_cast<float2*>(dst + i * 16 + 2 * g) = make_float2(o[i][n][j] * f * e, o[i][n][2 + j] * f * e);
        } else {
          dst[i * 16 + g] = o[i][n][j] * f;
          dst[i * 16 + 8 + g] = o[i][n][2 + j] * f;
        }
      }
    }
  __syncthreads();
  constexpr int TPR = kStepWarps * 32 / kStepRows;    // threads a row
  const int r = threadIdx.x / TPR, d0 = threadIdx.x % TPR * 4;
  if (r < nrows) {
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < kStepWarps; ++w) top = fmaxf(top, sh.m[w][r]);
    float fw[kStepWarps], sum = 0.f;
#pragma unroll
    for (int w = 0; w < kStepWarps; ++w) {
      fw[w] = sh.m[w][r] == -INFINITY ? sh.l[w][r] : sh.l[w][r] * ex2(sh.m[w][r] - top);
      sum += fw[w];
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int64_t row = s.row0 + r / p.group;
    const int head = kv * p.group + r % p.group;
#pragma unroll
    for (int d = d0; d < D; d += TPR * 4) {
      float x[4] = {};
#pragma unroll
      for (int w = 0; w < kStepWarps; ++w) {
        const float4 y = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(ring) + (w * kStepRows + r) * (D + 4) + d);
        const float f = fw[w] * inv;
        x[0] += y.x * f; x[1] += y.y * f; x[2] += y.z * f; x[3] += y.w * f;
      }
      if (CLUSTER && !whole) *reinterpret_cast<float4*>(avg + r * D + d) = make_float4(x[0], x[1], x[2], x[3]);
      else store4<D>(p, part, whole, row, head, d, x);
    }
    const float lse = sum == 0.f ? -INFINITY : top + log2f(sum) - kBias;
    if (!whole && d0 == 0) {
      if (CLUSTER) avg_lse[r] = lse;
      else store_lse(p, part, row, head, lse);
    }
  }
  if (CLUSTER && !whole) join_cluster<D>(p, s, kv, nrows, parts, avg, avg_lse);
}

// Behind the chunk kernel, whose results it does not need, it starts once that one's last blocks have, and fills the
// SMs that they leave. Its last block waits for that kernel's end, so that its own end stands for both.
template <int D, bool E4M3, int NT, bool CLUSTER>
__global__ void __launch_bounds__(kStepWarps * 32, 2) attend_step_kernel(const __grid_constant__ AttendParams p) {
  pdl_trigger();
  step_block<D, E4M3, NT, CLUSTER>(p);
  if (blockIdx.x + 1 == gridDim.x && blockIdx.y + 1 == gridDim.y && blockIdx.z + 1 == gridDim.z) pdl_wait();
}

// ------------------------------------------------------------------ join
// One warp a (row, query head) whose item was cut: the parts' averages weighed
// by their sums. Bound by reading the parts once, small next to the cache
// (largest where chunks are cut that fill no cluster: 11 us of a call of 141).
template <int D>
__global__ void __launch_bounds__(256) attend_join_kernel(const __grid_constant__ AttendParams p) {
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t unit = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int64_t row = unit / p.q_heads;
  const int head = (int)(unit % p.q_heads);
  if (row >= p.b.rows) return;
  int seq = 0;
#pragma unroll 4
  for (int i0 = 0; i0 < p.b.n; i0 += 32) {
    const int i = i0 + lane;
    seq += __popc(__ballot_sync(0xffffffffu, i < p.b.n && p.b.start[min(i, p.b.n - 1) + 1] <= row));
  }
  if (seq >= p.b.n) return;
  const Seq s = seq_of(p.b, seq, p.c.status);
  if (row < s.row0 || row >= s.row0 + s.n) return;
  const int nrows = s.n * p.group;
  int parts;
  if (p.a.use_step && nrows <= kStepRows) {
    parts = p.a.step_cluster ? 0 : parts_of(item_range(p, s.first, s.first + s.n - 1, s.len, kStepAlign), p.a.step_chunk);
  } else {
    const int i0 = ((int)(row - s.row0) * p.group + head % p.group) / kPairRows * kPairRows;
    const int i1 = min(i0 + kPairRows, nrows) - 1;
    parts = p.a.chunk_cluster
                ? 0
                : parts_of(item_range(p, s.first + i0 / p.group, s.first + i1 / p.group, s.len, kChunkAlign),
                           p.a.chunk_coarser ? *p.coarser : p.a.chunk_chunk);
  }
  if (parts <= 1) return;
  const int64_t n = (int64_t)p.b.rows * p.q_heads;
  float top = -INFINITY;
  for (int i = lane; i < parts; i += 32) top = fmaxf(top, p.part_lse[i * n + unit]);
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  constexpr int E = D / 32;
  float acc[E] = {}, sum = 0.f;
#pragma unroll 8
  for (int i = 0; i < parts; ++i) {
    const float lse = p.part_lse[i * n + unit];
    const float w = lse == -INFINITY ? 0.f : ex2(lse - top);
    sum += w;
    const float* src = p.part_o + (i * n + unit) * D + lane * E;
#pragma unroll
    for (int j = 0; j < E; ++j) acc[j] += w * src[j];
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  uint32_t w[E / 2];
#pragma unroll
  for (int j = 0; j < E / 2; ++j) w[j] = bf_pack(acc[2 * j] * inv, acc[2 * j + 1] * inv);
  uint16_t* dst = p.out + row * p.o_row + head * p.o_head + lane * E;
  if (E == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1 % (E / 2)]);
  else *reinterpret_cast<uint32_t*>(dst) = w[0];
}

template <int D, bool E4M3>
cudaError_t launch(const AttendParams& p, const CacheMaps& maps, cudaStream_t s) {
  // the longer blocks first: the step kernel's fill what they leave (a batch of both 150 us, the other way round 171)
  if (p.a.use_chunk) {
    const cudaError_t e = launch_attend_chunk(p, maps, D, E4M3, s);
    if (e != cudaSuccess) return e;
  }
  if (p.a.use_step) {
    const dim3 blocks(p.a.step_parts, p.c.heads, p.b.n);
    auto kernel = p.a.step_cluster ? (p.a.step_wide ? attend_step_kernel<D, E4M3, 2, true> : attend_step_kernel<D, E4M3, 1, true>)
                                   : (p.a.step_wide ? attend_step_kernel<D, E4M3, 2, false> : attend_step_kernel<D, E4M3, 1, false>);
    const cudaError_t e = launch_as(kernel, blocks, p.a.step_cluster ? p.a.step_parts : 1, 1, p.a.use_chunk != 0, kStepWarps * 32,
                                    kStepSmem, s, p);
    if (e != cudaSuccess) return e;
  }
  const int64_t units = (int64_t)p.b.rows * p.q_heads;
  const unsigned grid = (unsigned)((units + 7) / 8);
  if (kept_parts(p.a) > 1) {
    const cudaError_t e = launch_as(attend_join_kernel<D>, dim3(grid), 1, 1, true, 256, 0, s, p);
    if (e != cudaSuccess) return e;
  }
  return cudaGetLastError();
}

template <int D, bool E4M3>
cudaError_t prepare() {
  for (const void* f : {(const void*)attend_step_kernel<D, E4M3, 1, false>, (const void*)attend_step_kernel<D, E4M3, 1, true>,
                        (const void*)attend_step_kernel<D, E4M3, 2, false>, (const void*)attend_step_kernel<D, E4M3, 2, true>}) {
    const cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, kStepSmem);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t prepare_attend() {
  for (cudaError_t e : {prepare<64, false>(), prepare<64, true>(), prepare<128, false>(), prepare<128, true>()})
    if (e != cudaSuccess) return e;
  return prepare_attend_chunk();
}

cudaError_t launch_attend(const AttendParams& p, const CacheMaps& maps, int head_dim, bool e4m3, cudaStream_t s) {
  if (head_dim == 128) return e4m3 ? launch<128, true>(p, maps, s) : launch<128, false>(p, maps, s);
  return e4m3 ? launch<64, true>(p, maps, s) : launch<64, false>(p, maps, s);
}

}  // namespace cache
}  // namespace cp
