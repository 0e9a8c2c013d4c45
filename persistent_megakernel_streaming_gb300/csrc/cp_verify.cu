// cp_verify.cu -- verification of drafted tokens against the target's logits.
//
// Two launches. The first reads every logit once and leaves the maximum and the
// sum of exponentials of each piece of a row. The second, for each sequence,
// joins them, settles which drafted tokens are taken, and draws the token
// behind them from one row: there it sums again, so exactly that the draw
// does not depend on the order of the sums (below).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cfloat>

#include "cp.h"
#include "cp_call.h"

using namespace cp;

namespace {

// A piece of a row: its largest scaled logit, the sum of exp(x - m), and, of a greedy row, the largest's first place.
struct Piece {
  float m, s;
  int arg, pad;
};

constexpr int kPiece = 8192;           // logits of a row that a block takes
constexpr int kStatThreads = 256;
constexpr int kTokenThreads = 1024;

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
  Piece* pieces;                       // [2][rows][splits]: the target's, the draft's
  int n, rows, vocab, splits;
};

// Scaled logits are finite: NaN and -infinity become the lowest number, whose exponential next to any other is 0; a
// row whose largest is that has no probabilities.
constexpr float kLowest = -FLT_MAX;
__device__ __forceinline__ float scaled(float l, float by) { return fminf(fmaxf(__fmul_rn(l, by), kLowest), FLT_MAX); }
__device__ __forceinline__ float scale_of(float temperature) {
  return temperature > 0.f ? fminf(__fdiv_rn(1.f, temperature), FLT_MAX) : 1.f;
}
__device__ __forceinline__ float exp_from(float x, float m) { return expf(__fsub_rn(x, m)); }

__device__ __forceinline__ float value(const float* p) { return *p; }
__device__ __forceinline__ float value(const __nv_bfloat16* p) { return __bfloat162float(*p); }

// Eight logits (16-byte aligned), and calls of f(x, index) for all of [begin, end) of a row, in steps of the calling
// group's `threads`: eight at a time where they are aligned.
__device__ __forceinline__ void load8(const float* p, float* x) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w; x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float* x) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ void join(float* m, float* s, float m2, float s2) {
  const float top = fmaxf(*m, m2);
  *s = *s * expf(*m - top) + s2 * expf(m2 - top);
  *m = top;
}

// The sequence that row r belongs to, by one warp; n: none.
__device__ __forceinline__ int sequence_of(const VerifyParams& p, int r) {
  const int lane = threadIdx.x & 31;
  int seq = 0;
#pragma unroll 8
  for (int i0 = 0; i0 < p.n; i0 += 32) {
    const int i = i0 + lane;
    const bool before = i < p.n && p.start[min(i, p.n - 1) + 1] <= r;
    seq += __popc(__ballot_sync(0xffffffffu, before));
  }
  return seq;
}

template <class T>
__global__ void __launch_bounds__(kStatThreads) stats_kernel(const __grid_constant__ VerifyParams p) {
  __shared__ int own;
  __shared__ float ms[8], ss[8];
  __shared__ int as[8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int r = blockIdx.x / p.splits, part = blockIdx.x % p.splits, is_draft = blockIdx.y;
  if (warp == 0) {
    const int seq = sequence_of(p, r);
    if (lane == 0) own = seq;
  }
  __syncthreads();
  const int seq = own;
  if (seq >= p.n || p.start[seq] > r) return;                      // nobody's
  const float heat = p.temperature[seq];
  const bool greedy = !(heat > 0.f);
  if (is_draft && (greedy || r == p.start[seq + 1] - 1)) return;   // not asked for
  const float by = scale_of(heat);
  const T* row = is_draft ? static_cast<const T*>(p.draft_logits) + r * p.draft_row : static_cast<const T*>(p.logits) + r * p.row;
  const int begin = part * kPiece, end = min(begin + kPiece, p.vocab);
  float m = kLowest, s = 0.f;
  int arg = INT32_MAX;
  // what lies in front of a 16-byte boundary, eight at a time behind it, and the rest
  const int skew = (int)((reinterpret_cast<uintptr_t>(row + begin) & 15) / sizeof(T));
  const int head = min(begin + (skew ? (int)(16 / sizeof(T)) - skew : 0), end), body = head + (end - head) / 8 * 8;
  for (int i = head + threadIdx.x * 8; i < body; i += kStatThreads * 8) {
    float x[8];
    load8(row + i, x);
    float top = kLowest;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      x[k] = scaled(x[k], by);
      top = fmaxf(top, x[k]);
    }
    if (top > m || i == head + (int)threadIdx.x * 8) {
      if (greedy && (top > m || arg == INT32_MAX)) {
#pragma unroll
        for (int k = 7; k >= 0; --k) arg = x[k] == top ? i + k : arg;
      }
      s *= expf(m - top);
      m = top;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) s += exp_from(x[k], m);
  }
  for (int i = threadIdx.x < (unsigned)(head - begin) ? begin + (int)threadIdx.x : body + (int)threadIdx.x - (head - begin); i < end;
       i = i < head ? end : i + kStatThreads) {
    const float x = scaled(value(row + i), by);
    if (greedy && (x > m || (x == m && i < arg))) arg = i;
    join(&m, &s, x, 1.f);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const float m2 = __shfl_xor_sync(0xffffffffu, m, o), s2 = __shfl_xor_sync(0xffffffffu, s, o);
    const int a2 = __shfl_xor_sync(0xffffffffu, arg, o);
    if (m2 > m || (m2 == m && a2 < arg)) arg = a2;
    // the same sum in both lanes: the larger lane's second
    const bool up = lane & o;
    float m1 = up ? m2 : m, s1 = up ? s2 : s;
    join(&m1, &s1, up ? m : m2, up ? s : s2);
    m = m1;
    s = s1;
  }
  if (lane == 0) {
    ms[warp] = m;
    ss[warp] = s;
    as[warp] = arg;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int k = 1; k < kStatThreads / 32; ++k) {
      if (ms[k] > m || (ms[k] == m && as[k] < arg)) arg = as[k];
      join(&m, &s, ms[k], ss[k]);
    }
    p.pieces[((int64_t)is_draft * p.rows + r) * p.splits + part] = {m, s, arg, 0};
  }
}

// The whole row's, by one warp.
__device__ __forceinline__ Piece row_stats(const VerifyParams& p, int is_draft, int r) {
  const int lane = threadIdx.x & 31;
  const Piece* at = p.pieces + ((int64_t)is_draft * p.rows + r) * p.splits;
  Piece a = {kLowest, 0.f, INT32_MAX, 0};
  for (int k = lane; k < p.splits; k += 32) {
    const Piece b = at[k];
    if (b.m > a.m || (b.m == a.m && b.arg < a.arg)) a.arg = b.arg;
    join(&a.m, &a.s, b.m, b.s);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    Piece b;
    b.m = __shfl_xor_sync(0xffffffffu, a.m, o);
    b.s = __shfl_xor_sync(0xffffffffu, a.s, o);
    b.arg = __shfl_xor_sync(0xffffffffu, a.arg, o);
    if (b.m > a.m || (b.m == a.m && b.arg < a.arg)) a.arg = b.arg;
    const bool up = lane & o;
    float m1 = up ? b.m : a.m, s1 = up ? b.s : a.s;
    join(&m1, &s1, up ? a.m : b.m, up ? a.s : b.s);
    a.m = m1;
    a.s = s1;
  }
  return a;
}

// A sum of fp32 numbers with its rounding errors kept: twice fp32's bits.
struct Sum {
  float hi = 0.f, lo = 0.f;
  __device__ __forceinline__ void add(float x) {
    const float t = __fadd_rn(hi, x), z = __fsub_rn(t, hi);
    lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(t, z)), __fsub_rn(x, z)));
    hi = t;
  }
  __device__ __forceinline__ double value() const { return (double)hi + (double)lo; }
};

__device__ __forceinline__ double warp_sum(double x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

template <class T>
__global__ void __launch_bounds__(kTokenThreads) token_kernel(const __grid_constant__ VerifyParams p) {
  constexpr int kWarps = kTokenThreads / 32;
  __shared__ int first;                // the first refused row, or the last
  __shared__ int found;
  __shared__ double sums[2][kWarps];
  const int seq = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int r0 = p.start[seq], r1 = p.start[seq + 1];
  // a start out of order leaves in doubt whose rows are whose, for every sequence
  bool out_of_order = false;
  for (int i = threadIdx.x; i < p.n; i += kTokenThreads) {
    const int b = p.start[i], e = p.start[i + 1];
    out_of_order |= b < 0 || e < b || e > p.rows;
  }
  const bool bad = __syncthreads_or(out_of_order);
  if (bad || r0 == r1) {
    if (threadIdx.x == 0) {
      p.accepted[seq] = bad ? -1 : 0;
      p.token[seq] = -1;
    }
    return;
  }
  const float heat = p.temperature[seq], by = scale_of(heat);
  const bool greedy = !(heat > 0.f);
  if (threadIdx.x == 0) {
    first = r1 - 1;
    found = INT32_MAX;
  }
  __syncthreads();
  const T* logits = static_cast<const T*>(p.logits);
  const T* drafts = static_cast<const T*>(p.draft_logits);
  for (int r = r0 + warp; r < r1 - 1; r += kWarps) {
    const int d = p.draft[r];
    const bool in = (uint32_t)d < (uint32_t)p.vocab;
    const Piece a = row_stats(p, 0, r);
    const float pd = in && a.m > kLowest ? exp_from(scaled(value(logits + r * p.row + d), by), a.m) / a.s : 0.f;
    float qd = 1.f;
    if (drafts && !greedy) {
      const Piece b = row_stats(p, 1, r);
      qd = in && b.m > kLowest ? exp_from(scaled(value(drafts + r * p.draft_row + d), by), b.m) / b.s : 0.f;
    }
    const double u = fminf(fmaxf(p.u_accept[r], 0.f), 0x1.fffffep-1f);
    const bool yes = greedy ? a.m > kLowest && d == a.arg : u * (double)qd < (double)pd;
    if (lane == 0) {
      if (p.prob) p.prob[r] = pd;
      if (!yes) atomicMin(&first, r);
    }
  }
  __syncthreads();
  const int r = first;
  const bool refused = r < r1 - 1;
  if (threadIdx.x == 0) p.accepted[seq] = r - r0;
  const Piece a = row_stats(p, 0, r);
  if (greedy || !(a.m > kLowest)) {
    if (threadIdx.x == 0) p.token[seq] = a.m > kLowest ? a.arg : -1;
    return;
  }
  const bool both = refused && drafts;
  const float qm = both ? row_stats(p, 1, r).m : 0.f;
  const int out = refused && !drafts ? p.draft[r] : -1;              // a certain draft's token, taken out
  const T* row = logits + r * p.row;
  const T* draft_row = both ? drafts + r * p.draft_row : nullptr;
  // sums of both rows' exponentials
  Sum zp, zq;
  for (int i = threadIdx.x; i < p.vocab; i += kTokenThreads) {
    zp.add(exp_from(scaled(value(row + i), by), a.m));
    if (both) zq.add(exp_from(scaled(value(draft_row + i), by), qm));
  }
  const double z0 = warp_sum(zp.value()), z1 = warp_sum(zq.value());
  if (lane == 0) {
    sums[0][warp] = z0;
    sums[1][warp] = z1;
  }
  __syncthreads();
  double tp = 0., tq = 0.;
  for (int k = 0; k < kWarps; ++k) {
    tp += sums[0][k];
    tq += sums[1][k];
  }
  const float rp = (float)(1. / tp), rq = both && qm > kLowest ? (float)(1. / tq) : 0.f;
  auto weight = [&](int i, bool residual) {
    const float x = __fmul_rn(exp_from(scaled(value(row + i), by), a.m), rp);
    if (!residual) return x;
    if (both) return fmaxf(__fsub_rn(x, __fmul_rn(exp_from(scaled(value(draft_row + i), by), qm), rq)), 0.f);
    return i == out ? 0.f : x;
  };
  // each warp a stretch of the vocabulary
  const int each = (p.vocab + kWarps - 1) / kWarps, begin = min(warp * each, p.vocab), end = min(begin + each, p.vocab);
  bool residual = true;
  double total = 0.;
  for (int turn = 0; turn < 2; ++turn) {
    Sum w;
    for (int i = begin + lane; i < end; i += 32) w.add(weight(i, residual));
    const double mine = warp_sum(w.value());
    __syncthreads();
    if (lane == 0) sums[0][warp] = mine;
    __syncthreads();
    total = 0.;
    for (int k = 0; k < kWarps; ++k) total += sums[0][k];
    if (total > 0.) break;
    residual = false;
  }
  const double want = fminf(fmaxf(p.u_token[seq], 0.f), 0x1.fffffep-1f) * total;
  double before = 0.;
  int my = -1;                                                       // the stretch that the draw falls into
  for (int k = 0; k < kWarps; ++k) {
    if (sums[0][k] > 0.) {
      my = k;
      if (before + sums[0][k] > want) break;
    }
    before += sums[0][k];
  }
  if (my != warp) return;
  before = 0.;
  for (int k = 0; k < my; ++k) before += sums[0][k];
  int last = 0;                                                      // rounding may put the draw behind all of them
  for (int i0 = begin; i0 < end; i0 += 32) {
    const int i = i0 + lane;
    const float w = i < end ? weight(i, residual) : 0.f;
    double c = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double up = __shfl_up_sync(0xffffffffu, c, o);
      if (lane >= o) c += up;
    }
    c += before;
    const uint32_t some = __ballot_sync(0xffffffffu, w > 0.f), hit = __ballot_sync(0xffffffffu, w > 0.f && c > want);
    if (some) last = i0 + 31 - __clz(some);
    if (hit) {
      last = i0 + __ffs(hit) - 1;
      break;
    }
    before = __shfl_sync(0xffffffffu, c, 31);
  }
  if (lane == 0) p.token[seq] = last;
}

// ------------------------------------------------------------------ checks
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
  p->splits = (a->vocab + kPiece - 1) / kPiece;
  if ((int64_t)p->rows * p->splits > 1 << 30) return CP_ERR_UNSUPPORTED;   // blocks
  *workspace = (size_t)2 * p->rows * p->splits * sizeof(Piece);
  return CP_OK;
}

template <class T>
cudaError_t launch(const VerifyParams& p, cudaStream_t s) {
  stats_kernel<T><<<dim3((unsigned)(p.rows * p.splits), p.draft_logits ? 2 : 1), kStatThreads, 0, s>>>(p);
  token_kernel<T><<<p.n, kTokenThreads, 0, s>>>(p);
  return cudaGetLastError();
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
  if (!workspace || workspace_bytes < need) return CP_ERR_INVALID_ARG;
  if (!aligned16(workspace)) return CP_ERR_UNSUPPORTED;
  const int dev = check_device(device);
  if (dev) return dev;
  DeviceGuard g(device);
  p.pieces = static_cast<Piece*>(workspace);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return cuda_err(args->dtype == CP_LOGITS_BF16 ? launch<__nv_bfloat16>(p, s) : launch<float>(p, s));
}

}  // extern "C"
