// cp_attend.cu -- attention of a batch's new rows over the paged cache.
#include "cp_cache.cuh"

namespace cp {
namespace cache {
namespace {

constexpr int kWarps = 8;

// One warp a (row, query head): lanes share the head's D elements and walk the
// visible positions with a running maximum and sum. Right for every case, and
// bound by the shuffles of each score's sum and by reading the cache once per
// query head.
template <int D, bool E4M3>
__global__ void __launch_bounds__(kWarps * 32) attend_rows_kernel(const __grid_constant__ AttendParams p) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t unit = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int r = (int)(unit / p.q_heads), h = (int)(unit % p.q_heads);
  if (r >= p.b.rows) return;
  int seq = 0;
  for (int i0 = 0; i0 < p.b.n; i0 += 32) {
    const int i = i0 + lane;
    seq += __popc(__ballot_sync(0xffffffffu, i < p.b.n && p.b.start[i + 1] <= r));
  }
  if (seq >= p.b.n) return;
  const Seq s = seq_of(p.b, seq, p.c.status);
  if (r < s.row0 || r >= s.row0 + s.n) return;
  int lo, hi;
  visible(p, s.first + r - s.row0, s.len, &lo, &hi);
  const int kv = h / p.group;
  const uint16_t* qp = p.q + r * p.q_row + h * p.q_head + lane * E;
  float q[E], acc[E] = {};
#pragma unroll
  for (int i = 0; i < E; ++i) q[i] = __uint_as_float((uint32_t)qp[i] << 16) * p.scale_log2;
  float m = -INFINITY, l = 0.f;
  const int32_t* table = p.b.table + (int64_t)seq * p.b.table_stride;
  for (int t = lo; t < hi; ++t) {
    const int page = page_of(table, p.b.width, p.c.pages, p.c.page_shift, t);
    float k[E] = {}, v[E] = {};
    if (page < 0) {
      set_status(p.c.status, CP_ERR_DEVICE_BOUNDS);
    } else {
      const int64_t at = slot_bytes(p.c, page, kv, t);
      if (E4M3) {
        const int64_t sc = slot_scale(p.c, page, kv, t);
        const float fk = pow2i((int)p.c.ks[sc] - 127), fv = pow2i((int)p.c.vs[sc] - 127);
#pragma unroll
        for (int i = 0; i < E; ++i) {
          float f[4];
          e4m3x4_f32(p.c.k[at + lane * E + i], f);
          k[i] = f[0] * fk;
          e4m3x4_f32(p.c.v[at + lane * E + i], f);
          v[i] = f[0] * fv;
        }
      } else {
#pragma unroll
        for (int i = 0; i < E; ++i) {
          k[i] = __uint_as_float((uint32_t) reinterpret_cast<const uint16_t*>(p.c.k + at)[lane * E + i] << 16);
          v[i] = __uint_as_float((uint32_t) reinterpret_cast<const uint16_t*>(p.c.v + at)[lane * E + i] << 16);
        }
      }
    }
    float d = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) d += q[i] * k[i];
#pragma unroll
    for (int o = 16; o; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
    const float mn = fmaxf(m, d), ref = mn == -INFINITY ? 0.f : mn;
    const float a = ex2(m - ref), w = ex2(d - ref);
    l = l * a + w;
#pragma unroll
    for (int i = 0; i < E; ++i) acc[i] = acc[i] * a + w * v[i];
    m = mn;
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  uint16_t* op = p.out + r * p.o_row + h * p.o_head + lane * E;
#pragma unroll
  for (int i = 0; i < E; ++i) op[i] = (uint16_t)bf_pack(acc[i] * inv, 0.f);
}

}  // namespace

cudaError_t launch_attend(const AttendParams& p, int head_dim, bool e4m3, cudaStream_t s) {
  const int64_t units = (int64_t)p.b.rows * p.q_heads;
  const unsigned grid = (unsigned)((units + kWarps - 1) / kWarps);
  if (head_dim == 128) {
    if (e4m3) attend_rows_kernel<128, true><<<grid, kWarps * 32, 0, s>>>(p);
    else attend_rows_kernel<128, false><<<grid, kWarps * 32, 0, s>>>(p);
  } else {
    if (e4m3) attend_rows_kernel<64, true><<<grid, kWarps * 32, 0, s>>>(p);
    else attend_rows_kernel<64, false><<<grid, kWarps * 32, 0, s>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace cache
}  // namespace cp
