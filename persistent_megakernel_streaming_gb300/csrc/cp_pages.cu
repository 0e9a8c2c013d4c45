// cp_pages.cu -- which pages of a cache hold what: the C ABI (checks and
// launches) and the kernels that fork, grow, trim and compact sequences.
//
// All of it is whole numbers in an order that the calls define, so the results
// do not depend on how blocks are scheduled: counts are only added to, and
// whatever has an order (which free page goes to whom) comes from prefix sums.
#include <cuda_runtime.h>

#include <new>

#include "cp.h"
#include "cp_call.h"
#include "cp_ptx.cuh"

using namespace cp;

namespace {

// What a sequence grows by.
struct Plan {
  int len;           // new length, or -1: it stays as it is
  int had, want;     // pages
  int last;          // the partly filled page that it grows into, or -1
  int copies;        // whether it takes a page of its own for that: others hold it too
  int base, move;    // its first new page's place in the list, its place among the moves
};

struct PagesView {
  int32_t* refs;
  int32_t* table;
  int32_t* length;
  int64_t stride;
  int pages, sequences, width, shift;   // page size 1 << shift
  int32_t* status;
  // scratch
  int32_t* list;     // [pages] free pages in order
  int32_t* map;      // [pages] where a page is after a compaction; -1: nobody held it
  int32_t* tail;     // [pages] sequences that grow into a partly filled page; zeros between calls
  int32_t* keeper;   // [pages] the last of them, plus one; zeros between calls
  Plan* plan;        // [sequences]
  int32_t* marks;    // [sequences] pairs of a fork that name a sequence; zeros between calls
  int32_t* clash;    // [sequences] whether a pair of the fork gets in another's way
};

constexpr int kMostBlocks = 8;
constexpr int64_t kLow = ((int64_t)1 << 40) - 1;   // two counts in one sum

}  // namespace

struct cp_pages {
  int device = 0;
  PagesView view{};
  void* memory = nullptr;
};

namespace {

__device__ __forceinline__ void set_status(const PagesView& v) { atomicCAS(v.status, 0, (int)CP_ERR_DEVICE_BOUNDS); }

// Positions of a sequence; ones that its table cannot hold count as none.
__device__ __forceinline__ int length_of(const PagesView& v, int i) {
  const int l = v.length[i];
  if (l >= 0 && ((int64_t)l + (1 << v.shift) - 1) >> v.shift <= v.width) return l;
  set_status(v);
  return 0;
}
__device__ __forceinline__ int pages_for(const PagesView& v, int64_t length) {
  return (int)((length + (1 << v.shift) - 1) >> v.shift);
}
__device__ __forceinline__ bool in_pool(const PagesView& v, int page) { return (uint32_t)page < (uint32_t)v.pages; }

// ------------------------------------------------------------------ trim
// A block a sequence, bound by the launch: 1 us behind another kernel for up to 1000 sequences, 8.6 for 8192.
__global__ void __launch_bounds__(128) trim_kernel(const PagesView v, const int32_t* keep) {
  ptx::pdl_trigger();
  ptx::pdl_wait();
  const int i = blockIdx.x;
  const int want = keep[i], len = length_of(v, i);
  if (want < 0) {
    set_status(v);
    return;
  }
  if (want >= len) return;
  __syncthreads();                       // every thread has read the length
  const int held = pages_for(v, len);
  if (threadIdx.x == 0) v.length[i] = want;
  int32_t* row = v.table + (int64_t)i * v.stride;
  for (int k = pages_for(v, want) + threadIdx.x; k < held; k += 128) {
    const int page = row[k];
    row[k] = -1;
    if (!in_pool(v, page)) {
      set_status(v);
    } else if (atomicSub(v.refs + page, 1) <= 0) {
      atomicAdd(v.refs + page, 1);       // nobody held it
      set_status(v);
    }
  }
}

// ------------------------------------------------------------------ one cluster
// Growing and compacting need prefix sums over all sequences and all pages: one cluster of up to 8 blocks does them, a
// contiguous share of both to each block, and meets at cluster barriers, which order its memory accesses too. What bounds
// them is the chain of loads, scans and barriers: a thread that has one sequence, or four pages, keeps what it knows of
// them in registers from one to the next.
constexpr int kThreads = 1024;

// Exclusive prefix of x over the block's threads; *sum: of all. Synchronises.
__device__ __forceinline__ int64_t block_scan(int64_t x, int64_t* sum) {
  __shared__ int64_t warps[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t inc = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t up = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += up;
  }
  __syncthreads();
  if (lane == 31) warps[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    int64_t w = warps[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t up = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += up;
    }
    warps[lane] = w;
  }
  __syncthreads();
  *sum = warps[31];
  return inc - x + (warp ? warps[warp - 1] : 0);
}
// The block's share of n things, in steps of 4.
struct Share {
  int begin, end;
};
__device__ __forceinline__ Share share_of(int n) {
  const int64_t each = (((int64_t)n + gridDim.x - 1) / gridDim.x + 3) & ~3ll;
  return {(int)min((int64_t)n, each * blockIdx.x), (int)min((int64_t)n, each * (blockIdx.x + 1))};
}
// One value of each block told to all of the cluster, for after its next barrier.
struct Told {
  int64_t of[kMostBlocks];
};
__device__ __forceinline__ void tell(Told& t, int64_t x) {            // one warp, all lanes
  if (threadIdx.x < gridDim.x) {
    const uint32_t at = ptx::mapa(ptx::saddr(&t.of[blockIdx.x]), threadIdx.x);
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(at), "l"(x) : "memory");
  }
  __syncwarp();
}
// The sum of the blocks' before this one, and of all.
__device__ __forceinline__ int64_t before_me(const Told& t, int64_t* all) {
  int64_t mine = 0, sum = 0;
  for (int k = 0; k < (int)gridDim.x; ++k) {
    if (k < (int)blockIdx.x) mine += t.of[k];
    sum += t.of[k];
  }
  *all = sum;
  return mine;
}
// Every block's memory is there to be written, from the wait on.
__device__ __forceinline__ void arrive_early() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void wait_early() { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); }
__device__ __forceinline__ void meet() {
  __syncwarp();
  ptx::cluster_sync_all();
}

// Which of pages p .. p + 3 below `end` satisfy a predicate of (page, count): a bit each.
template <class F>
__device__ __forceinline__ uint32_t four(const PagesView& v, int p, int end, F f) {
  uint32_t bits = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (p + k < end && f(p + k, v.refs[p + k])) bits |= 1u << k;
  return bits;
}
template <class F>
__device__ __forceinline__ int64_t count_pages(const PagesView& v, Share pages, F f) {
  int64_t n = 0, sum;
  for (int p = pages.begin + threadIdx.x * 4; p < pages.end; p += kThreads * 4) n += __popc(four(v, p, pages.end, f));
  block_scan(n, &sum);
  return sum;
}
// For each such page of the share in ascending order, act(its rank, counted from `rank` on, page).
template <class F, class A>
__device__ __forceinline__ void each_page(const PagesView& v, Share pages, int64_t rank, F f, A act) {
  for (int p0 = pages.begin; p0 < pages.end; p0 += kThreads * 4) {
    const int p = p0 + threadIdx.x * 4;
    const uint32_t bits = four(v, p, pages.end, f);
    int64_t sum, at = rank + block_scan(__popc(bits), &sum);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (bits >> k & 1) act(at++, p + k);
    rank += sum;
  }
}

// ------------------------------------------------------------------ fork
// Whether pairs get in each other's way, for more of them than each looks through for itself: a sequence that one pair
// copies to, and no other pair names. Marks are counted, read and cleared by one cluster.
constexpr int kCopied = 1 << 20;         // more than there are pairs
__global__ void __launch_bounds__(kThreads) clash_kernel(const PagesView v, const int32_t* src, const int32_t* dst, int n) {
  ptx::pdl_trigger();
  ptx::pdl_wait();
  const int first = blockIdx.x * kThreads + threadIdx.x, step = gridDim.x * kThreads;
  auto is_one = [&](int s) { return (uint32_t)s < (uint32_t)v.sequences; };
  for (int i = first; i < n; i += step) {
    const int s = src[i], d = dst[i];
    if (is_one(s)) atomicOr(v.marks + s, kCopied);
    if (is_one(d)) atomicAdd(v.marks + d, 1);
  }
  meet();
  for (int i = first; i < n; i += step) v.clash[i] = !is_one(dst[i]) || __ldcg(v.marks + dst[i]) != 1;
  meet();
  for (int i = first; i < n; i += step) {
    if (is_one(src[i])) v.marks[src[i]] = 0;
    if (is_one(dst[i])) v.marks[dst[i]] = 0;
  }
}

// A block a pair; of pairs of 40 pages 2.8 us for 1, 3.3 for 8, 5.5 for 64, 8.7 for 200: a launch, four loads that wait for one
// another, and the counts.
// OWN: whether pairs get in each other's way is looked up among all of them by every block, so that no order between blocks
// is needed; otherwise the kernel in front says so.
template <bool OWN>
__global__ void __launch_bounds__(256) fork_kernel(const PagesView v, const int32_t* src, const int32_t* dst, int n) {
  ptx::pdl_trigger();
  ptx::pdl_wait();
  const int pair = blockIdx.x, s = src[pair], d = dst[pair];
  bool bad = (uint32_t)s >= (uint32_t)v.sequences || (uint32_t)d >= (uint32_t)v.sequences;
  if (OWN)
    for (int i = threadIdx.x; i < n; i += 256) bad |= (i != pair && dst[i] == d) || src[i] == d;
  else
    bad |= v.clash[pair] != 0;
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0) set_status(v);
    return;
  }
  const int len = length_of(v, s), held = pages_for(v, len);
  const int32_t* from = v.table + (int64_t)s * v.stride;
  int32_t* to = v.table + (int64_t)d * v.stride;
  bool left_out = v.length[d] != 0;      // nobody writes it before the barrier
  for (int i = threadIdx.x; i < held; i += 256) {
    const int page = from[i];
    left_out |= in_pool(v, page) && v.refs[page] < 1;    // nobody's: no call of this kernel makes it somebody's
  }
  if (__syncthreads_or(left_out)) {
    if (threadIdx.x == 0) set_status(v);
    return;
  }
  if (threadIdx.x == 0) v.length[d] = len;
  for (int i = threadIdx.x; i < held; i += 256) {
    const int page = from[i];
    to[i] = page;
    if (in_pool(v, page)) atomicAdd(v.refs + page, 1);
    else set_status(v);
  }
}

// ------------------------------------------------------------------ grow
__device__ __forceinline__ Plan ask_of(const PagesView& v, const int32_t* add, int i) {
  Plan a{};
  const int len = length_of(v, i), more = add[i];
  a.len = a.last = -1;
  a.had = a.want = pages_for(v, len);
  if (more == 0 || v.length[i] != len) return a;
  const int64_t to = (int64_t)len + more;
  if (more < 0 || to > INT32_MAX || (to + (1 << v.shift) - 1) >> v.shift > v.width) {
    set_status(v);
    return a;
  }
  if (len & ((1 << v.shift) - 1)) {
    const int page = v.table[(int64_t)i * v.stride + a.had - 1];
    if (!in_pool(v, page)) {
      set_status(v);
      return a;
    }
    if (v.refs[page] < 1) {
      set_status(v);
      return a;
    }
    a.last = page;
  }
  a.len = (int)to;
  a.want = pages_for(v, to);
  return a;
}

// The pages that a sequence takes: `n` from the list's place `at` on, behind the `had` it has.
struct Take {
  int64_t at;
  int had, n;
};

// ONE: no thread has more than one sequence, or more than four pages. From launch to launch 3.9 us for 1 sequence, 5.6 for
// 1024 of 8192 pages (some 4 more through scratch memory, as without ONE), 16.4 for 8200 of 40000.
template <bool ONE>
__global__ void __launch_bounds__(kThreads) grow_kernel(const PagesView v, const int32_t* add, int32_t* moves, int32_t* count) {
  __shared__ Told free_told, fresh_told, moved_told;
  __shared__ Take takes[kThreads];
  __shared__ int many;                   // some sequence of the block takes more pages than its own thread sees to
  const Share pages = share_of(v.pages), seqs = share_of(v.sequences);
  const int tid = threadIdx.x, my_page = pages.begin + tid * 4, my_seq = seqs.begin + tid;
  auto is_free = [](int, int refs) { return refs == 0; };
  arrive_early();
  ptx::pdl_trigger();
  ptx::pdl_wait();
  if (tid == 0) many = 0;
  const uint32_t bits = ONE ? four(v, my_page, pages.end, is_free) : 0;
  Plan own{};
  for (int i = my_seq; i < seqs.end; i += kThreads) {
    own = ask_of(v, add, i);
    if (!ONE) v.plan[i] = own;
    if (own.last >= 0) {
      atomicAdd(v.tail + own.last, 1);
      atomicMax(v.keeper + own.last, i + 1);
    }
  }
  int64_t free_here, my_free = 0;
  if (ONE) my_free = block_scan(__popc(bits), &free_here);
  else free_here = count_pages(v, pages, is_free);
  wait_early();
  if (tid < 32) tell(free_told, free_here);
  meet();
  // all that grow into a shared page take one of their own, but the last of them if nobody else holds it; none of them
  // grows if the page's count is less than they are
  int64_t fresh_here = 0, moved_here = 0;
  for (int i0 = seqs.begin; i0 < seqs.end || ONE; i0 += kThreads) {
    const int i = i0 + tid;
    Plan a = own;
    if (!ONE && i < seqs.end) a = v.plan[i];
    if (i >= seqs.end) a = Plan{-1, 0, 0, -1, 0, 0, 0};
    if (a.last >= 0) {
      const int sharers = __ldcg(v.tail + a.last), keeper = __ldcg(v.keeper + a.last), refs = v.refs[a.last];
      if (sharers > refs) {
        set_status(v);
        a.len = -1;
        a.want = a.had;
      } else {
        a.copies = !(sharers == refs && keeper == i + 1);
      }
    }
    int64_t sum;
    if (a.want - a.had > 2) many = 1;
    const int64_t fresh = a.want - a.had + a.copies;
    const int64_t at = block_scan((int64_t)a.copies << 40 | fresh, &sum);
    a.base = (int)min(fresh_here + (at & kLow), (int64_t)INT32_MAX);
    a.move = (int)(moved_here + (at >> 40));
    if (ONE) own = a;
    else if (i < seqs.end) v.plan[i] = a;
    fresh_here += sum & kLow;
    moved_here += sum >> 40;
    if (ONE) break;
  }
  if (tid < 32) {
    tell(fresh_told, fresh_here);
    tell(moved_told, moved_here);
  }
  meet();
  int64_t free_all, fresh_all, moved_all;
  const int64_t free0 = before_me(free_told, &free_all), fresh0 = before_me(fresh_told, &fresh_all), moved0 = before_me(moved_told, &moved_all);
  const bool enough = free_all >= fresh_all;
  if (blockIdx.x == 0 && tid == 0) *count = enough ? (int)moved_all : -(int)min(fresh_all - free_all, (int64_t)INT32_MAX);
  if (enough && free0 < fresh_all) {
    auto take = [&](int64_t at, int page) {
      if (at < fresh_all) v.list[at] = page;
    };
    if (ONE) {
      int64_t at = free0 + my_free;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (bits >> k & 1) take(at++, my_page + k);
    } else {
      each_page(v, pages, free0, is_free, take);
    }
  }
  meet();
  // what a sequence has is changed by its own thread; many pages are a warp's work, four sequences at a time, whose loads do
  // not wait for one another (40 of 80 sequences trimmed, the others compacted, 40 of 49 pages grown: 20 us for the three
  // calls, 31 where a warp took its lanes' sequences and compaction one page a thread after the other)
  const int lane = tid & 31;
  for (int i0 = seqs.begin; i0 < seqs.end; i0 += kThreads) {
    const int i = i0 + tid;
    Plan a = own;
    if (!ONE && i < seqs.end) a = v.plan[i];
    if (i >= seqs.end) a = Plan{-1, 0, 0, -1, 0, 0, 0};
    if (a.last >= 0) v.tail[a.last] = v.keeper[a.last] = 0;
    const bool grows = enough && a.len >= 0;
    const int64_t base = fresh0 + a.base;
    int32_t* row = v.table + (int64_t)i * v.stride;
    const int more = grows ? a.want - a.had : 0;
    if (grows) {
      v.length[i] = a.len;
      if (a.copies) {
        const int page = __ldcg(v.list + base);
        const int64_t m = moved0 + a.move;
        moves[2 * m] = a.last;
        moves[2 * m + 1] = page;
        row[a.had - 1] = page;
        v.refs[page] = 1;
        atomicSub(v.refs + a.last, 1);
      }
      if (more <= 2)
        for (int k = 0; k < more; ++k) {
          const int page = __ldcg(v.list + base + a.copies + k);
          row[a.had + k] = page;
          v.refs[page] = 1;
        }
    }
    if (!many) continue;
    takes[tid] = {base + a.copies, a.had, more > 2 ? more : 0};
    __syncthreads();
    const int here = min(seqs.end - i0, kThreads);
    for (int q = tid >> 5; q < here; q += 4 * (kThreads / 32)) {
      Take t[4];
      int most = 0;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int at = q + u * (kThreads / 32);
        t[u] = takes[min(at, here - 1)];
        if (at >= here) t[u].n = 0;
        most = max(most, t[u].n);
      }
      for (int k = lane; k < most; k += 32) {
        int page[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) page[u] = k < t[u].n ? __ldcg(v.list + t[u].at + k) : -1;
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (page[u] >= 0) {
            v.table[(int64_t)(i0 + q + u * (kThreads / 32)) * v.stride + t[u].had + k] = page[u];
            v.refs[page[u]] = 1;
          }
      }
    }
    __syncthreads();                       // all are done with this round's
  }
}

// ------------------------------------------------------------------ compact
// A sequence's entries, by `threads` threads of which this is the t-th: where the pages are now. One that names a page that
// nobody held stays as it is: what has moved there is not its.
__device__ __forceinline__ void remap(const PagesView& v, int i, int t, int threads) {
  const int held = pages_for(v, length_of(v, i));
  int32_t* row = v.table + (int64_t)i * v.stride;
  for (int k0 = t; k0 < held; k0 += 4 * threads) {
    int page[4], to[4];                  // loads first: those of four entries do not wait for one another
#pragma unroll
    for (int u = 0; u < 4; ++u) page[u] = k0 + u * threads < held ? row[k0 + u * threads] : -1;
#pragma unroll
    for (int u = 0; u < 4; ++u) to[u] = in_pool(v, page[u]) ? __ldcg(v.map + page[u]) : -1;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (k0 + u * threads >= held) break;
      if (to[u] < 0) set_status(v);
      else if (to[u] != page[u]) row[k0 + u * threads] = to[u];
    }
  }
}

// With n pages held, P(p) of them below page p: the free page p < n is the (p - P(p))-th hole, and the held page p >= n the
// (P(p) - P(n))-th that moves. One prefix sum settles both. 3.1 us of 576 pages, 4.5 of 8256, 12.5 of 65600.
template <bool ONE>
__global__ void __launch_bounds__(kThreads) compact_kernel(const PagesView v, int32_t* moves, int32_t* count, int tables) {
  __shared__ Told live_told, below_told;
  __shared__ int64_t below_n;              // P(n), where this block's share has page n
  const Share pages = share_of(v.pages);
  const int tid = threadIdx.x, my_page = pages.begin + tid * 4;
  auto is_live = [](int, int refs) { return refs != 0; };
  arrive_early();
  ptx::pdl_trigger();
  ptx::pdl_wait();
  if (tid == 0) below_n = 0;
  const uint32_t bits = ONE ? four(v, my_page, pages.end, is_live) : 0;
  int64_t live_here, my_live = 0;
  if (ONE) my_live = block_scan(__popc(bits), &live_here);
  else live_here = count_pages(v, pages, is_live);
  wait_early();
  if (tid < 32) tell(live_told, live_here);
  meet();
  int64_t all;
  const int64_t live0 = before_me(live_told, &all);
  const int n = (int)all;
  // holes to the list; what P(n) is, from the block that knows
  auto holes = [&](uint32_t b, int p, int64_t before) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int page = p + k;
      if (page >= pages.end) break;
      if (page == n) below_n = before;
      const bool live = b >> k & 1;
      if (!live && page < n) v.list[page - before] = page;
      before += live;
      v.map[page] = live && page < n ? page : -1;
    }
  };
  if (ONE) {
    holes(bits, my_page, live0 + my_live);
  } else {
    int64_t rank = live0;
    for (int p0 = pages.begin; p0 < pages.end; p0 += kThreads * 4) {
      const uint32_t b = four(v, p0 + tid * 4, pages.end, is_live);
      int64_t sum;
      const int64_t at = rank + block_scan(__popc(b), &sum);
      holes(b, p0 + tid * 4, at);
      rank += sum;
    }
  }
  __syncthreads();
  if (tid < 32) tell(below_told, below_n);
  meet();
  int64_t below;
  before_me(below_told, &below);
  if (n == v.pages) below = n;             // nothing lies behind
  if (blockIdx.x == 0 && tid == 0) *count = n - (int)below;
  auto move_on = [&](uint32_t b, int p, int64_t before) {
    // loads first: those of four pages do not wait for one another
    int64_t at[4];
    int to[4], refs[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      at[k] = before - below;
      before += b >> k & 1;
      if (p + k < n) b &= ~(1u << k);
      to[k] = b >> k & 1 ? __ldcg(v.list + at[k]) : 0;
      refs[k] = b >> k & 1 ? v.refs[p + k] : 0;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (!(b >> k & 1)) continue;
      moves[2 * at[k]] = p + k;
      moves[2 * at[k] + 1] = to[k];
      v.map[p + k] = to[k];
      v.refs[to[k]] = refs[k];
      v.refs[p + k] = 0;
    }
  };
  if (ONE) {
    move_on(bits, my_page, live0 + my_live);
  } else {
    int64_t rank = live0;
    for (int p0 = pages.begin; p0 < pages.end; p0 += kThreads * 4) {
      // what other blocks write below n is not looked at: pages from n on alone move, and change in their own turn alone
      const int p = p0 + tid * 4;
      const uint32_t b = four(v, p, pages.end, [n](int page, int refs) { return page >= n && refs != 0; });
      int64_t sum, at = block_scan(__popc(b), &sum);
      if (p0 == pages.begin) rank = max(below, live0);
      move_on(b, p, rank + at);
      rank += sum;
    }
  }
  if (!tables) return;
  meet();
  for (int i = blockIdx.x * (kThreads / 32) + (tid >> 5); i < v.sequences; i += gridDim.x * (kThreads / 32)) remap(v, i, tid & 31, 32);
}

// The tables, where they are too large for the one cluster: a block a sequence.
__global__ void __launch_bounds__(128) remap_kernel(const PagesView v) {
  ptx::pdl_trigger();
  ptx::pdl_wait();
  remap(v, blockIdx.x, threadIdx.x, 128);
}

// ------------------------------------------------------------------ checks
int check_desc(const cp_pages_desc* d, PagesView* v) {
  if (!d || !d->refs || !d->page_table || !d->length) return CP_ERR_INVALID_ARG;
  if (d->pages < 1 || d->page_size < 1 || d->sequences < 1 || d->table_width < 1 || d->table_stride < 0) return CP_ERR_INVALID_ARG;
  if (d->page_size != 16 && d->page_size != 32 && d->page_size != 64 && d->page_size != 128) return CP_ERR_UNSUPPORTED;
  if (d->pages > 1 << 30 || d->sequences > 65535) return CP_ERR_UNSUPPORTED;
  if (d->table_stride && d->sequences > 1 && d->table_stride < d->table_width) return CP_ERR_INVALID_ARG;
  v->refs = d->refs;
  v->table = d->page_table;
  v->length = d->length;
  v->stride = d->table_stride ? d->table_stride : d->table_width;
  v->pages = d->pages;
  v->sequences = d->sequences;
  v->width = d->table_width;
  v->shift = d->page_size == 16 ? 4 : d->page_size == 32 ? 5 : d->page_size == 64 ? 6 : 7;
  return CP_OK;
}

size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

// Blocks of the one cluster: the fewest whose threads get four pages and a sequence each (64 pages grown in 3.4 us, with 8
// blocks 5.0; 4096 in 3.9 and 5.0; 8192 in 4.7 and 4.9; some 0.5 more since), and all 8 where there are more.
int blocks_for(const PagesView& v) {
  int n = 1;
  while (n < kMostBlocks && (v.pages > n * 4 * kThreads || v.sequences > n * kThreads)) n *= 2;
  return n;
}

// Whether no thread of the cluster gets more than a sequence and four pages (shares are rounded up to four).
bool one_each(const PagesView& v, int blocks) {
  const auto share = [blocks](int n) { return ((n + blocks - 1) / blocks + 3) & ~3; };
  return share(v.pages) <= 4 * kThreads && share(v.sequences) <= kThreads;
}
// Pairs up to which each block of a fork looks through all of them itself, us of a fork and a trim behind it that way and
// with marks: 1024 10.4 and 11.5, 1536 12.9 and 13.2, 2048 16.9 and 14.3, 8192 69 and 35, 32000 1153 and 119.
constexpr int kOwnPairs = 1536;
// Table entries up to which the cluster that compacts rewrites them itself, us that way and with a launch of their own: 64
// entries 3.1 and 3.6, 1024 3.8 and 4.1, 2048 5.0 and 4.9, 8000 7.0 and 5.8, 32768 13.5 and 11.3, 262144 77 and 59.
constexpr int64_t kFewEntries = 1 << 11;

}  // namespace

extern "C" {

int cp_pages_check(const cp_pages_desc* desc) {
  PagesView v{};
  return check_desc(desc, &v);
}

int cp_pages_create(const cp_pages_desc* desc, int device, cp_pages** out) {
  if (!out) return CP_ERR_INVALID_ARG;
  *out = nullptr;
  PagesView v{};
  int st = check_desc(desc, &v);
  if (st) return st;
  if ((st = check_device(device))) return st;
  DeviceGuard guard(device);
  for (const void* ptr : {v.refs, v.table, v.length})
    if (!on_device(ptr, device)) return CP_ERR_INVALID_ARG;
  cp_pages* p = new (std::nothrow) cp_pages();
  if (!p) return CP_ERR_NOMEM;
  p->device = device;
  const size_t each = up256((size_t)v.pages * 4), plans = up256((size_t)v.sequences * sizeof(Plan));
  const size_t marks = up256((size_t)v.sequences * 4);
  const size_t bytes = 4 * each + plans + 2 * marks + 256;
  if (cudaMalloc(&p->memory, bytes) != cudaSuccess) {
    cudaGetLastError();
    delete p;
    return CP_ERR_NOMEM;
  }
  uint8_t* at = static_cast<uint8_t*>(p->memory);
  v.list = reinterpret_cast<int32_t*>(at);
  v.map = reinterpret_cast<int32_t*>(at + each);
  v.tail = reinterpret_cast<int32_t*>(at + 2 * each);
  v.keeper = reinterpret_cast<int32_t*>(at + 3 * each);
  v.plan = reinterpret_cast<Plan*>(at + 4 * each);
  v.marks = reinterpret_cast<int32_t*>(at + 4 * each + plans);
  v.clash = reinterpret_cast<int32_t*>(at + 4 * each + plans + marks);
  v.status = reinterpret_cast<int32_t*>(at + 4 * each + plans + 2 * marks);
  p->view = v;
  if (cudaMemset(p->memory, 0, bytes) != cudaSuccess || cudaDeviceSynchronize() != cudaSuccess) {
    cp_pages_destroy(p);
    return CP_ERR_CUDA;
  }
  *out = p;
  return CP_OK;
}

void cp_pages_destroy(cp_pages* p) {
  if (!p) return;
  {
    DeviceGuard g(p->device);
    cudaDeviceSynchronize();
    cudaFree(p->memory);
  }
  delete p;
}

int cp_pages_status(cp_pages* p) {
  if (!p) return CP_ERR_INVALID_ARG;
  DeviceGuard g(p->device);
  if (cudaDeviceSynchronize() != cudaSuccess) return CP_ERR_CUDA;
  int32_t v = 0;
  if (cudaMemcpy(&v, p->view.status, 4, cudaMemcpyDeviceToHost) != cudaSuccess) return CP_ERR_CUDA;
  return v;
}

int cp_pages_clear_status(cp_pages* p) {
  if (!p) return CP_ERR_INVALID_ARG;
  DeviceGuard g(p->device);
  if (cudaDeviceSynchronize() != cudaSuccess) return CP_ERR_CUDA;
  if (cudaMemset(p->view.status, 0, 4) != cudaSuccess) return CP_ERR_CUDA;
  return cuda_err(cudaDeviceSynchronize());
}

int cp_pages_fork(cp_pages* p, const int32_t* src, const int32_t* dst, int n, cp_stream_t stream) {
  if (!p || !src || !dst || n < 1 || n > p->view.sequences) return CP_ERR_INVALID_ARG;
  DeviceGuard g(p->device);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (n <= kOwnPairs) return cuda_err(launch_as(fork_kernel<true>, dim3(n), 1, 1, true, 256, 0, s, p->view, src, dst, n));
  const cudaError_t e = launch_as(clash_kernel, dim3(kMostBlocks), kMostBlocks, 1, true, kThreads, 0, s, p->view, src, dst, n);
  return cuda_err(e == cudaSuccess ? launch_as(fork_kernel<false>, dim3(n), 1, 1, true, 256, 0, s, p->view, src, dst, n) : e);
}

int cp_pages_trim(cp_pages* p, const int32_t* keep, cp_stream_t stream) {
  if (!p || !keep) return CP_ERR_INVALID_ARG;
  DeviceGuard g(p->device);
  return cuda_err(launch_as(trim_kernel, dim3(p->view.sequences), 1, 1, true, 128, 0, reinterpret_cast<cudaStream_t>(stream), p->view, keep));
}

int cp_pages_grow(cp_pages* p, const int32_t* add, int32_t* moves, int capacity, int32_t* count, cp_stream_t stream) {
  if (!p || !add || !moves || !count || capacity < p->view.sequences) return CP_ERR_INVALID_ARG;
  DeviceGuard g(p->device);
  const int n = blocks_for(p->view);
  return cuda_err(launch_as(one_each(p->view, n) ? grow_kernel<true> : grow_kernel<false>, dim3(n), n, 1, true, kThreads, 0,
                            reinterpret_cast<cudaStream_t>(stream), p->view, add, moves, count));
}

int cp_pages_compact(cp_pages* p, int32_t* moves, int capacity, int32_t* count, cp_stream_t stream) {
  if (!p || !moves || !count || capacity < p->view.pages / 2) return CP_ERR_INVALID_ARG;
  DeviceGuard g(p->device);
  int n = blocks_for(p->view);
  // a warp rewrites a sequence's entries, and moves are shared out: 80 of 49 pages with 1970 moves 17 us for the three calls, in
  // one block 20
  while (n < kMostBlocks && p->view.sequences > n * kThreads / 32) n *= 2;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int tables = (int64_t)p->view.sequences * p->view.width <= kFewEntries;
  cudaError_t e = launch_as(one_each(p->view, n) ? compact_kernel<true> : compact_kernel<false>, dim3(n), n, 1, true, kThreads, 0, s,
                            p->view, moves, count, tables);
  if (e == cudaSuccess && !tables) e = launch_as(remap_kernel, dim3(p->view.sequences), 1, 1, true, 128, 0, s, p->view);
  return cuda_err(e);
}

}  // extern "C"
