// Pages of a cache: copies, the rows of the next step (fork, reorder, free), growth and
// trimming with copy on write, and a dense pool again.
//
// refs[p] counts the table entries that name page p.  Everything that is decided depends
// on the inputs alone: counts are sums (integer atomics, whose order does not show), and
// free pages are handed out by rank, the lowest id first, to the rows in order.
#include <cooperative_groups.h>

#include <algorithm>

#include "common.cuh"
#include "launch.h"
#include "target_checks.h"

namespace dfl {
namespace {

namespace cg = cooperative_groups;

// ---------------------------------------------------------------------------
// copies
// ---------------------------------------------------------------------------
constexpr int kBuffers = 128;  // buffers of a launch: they travel as its parameters
constexpr int kChunk = 4096;   // bytes of a warp's turn
struct Buffers {
  char* data[kBuffers];
  int64_t stride[kBuffers];
  int32_t bytes[kBuffers];  // of a page, / 4
  int32_t n;
};

struct CopyList {
  const int32_t* src;
  const int32_t* dst;
  const int32_t* count_dev;  // or NULL: count
  int32_t count;
  int64_t n_pages;
  int32_t* status;
};

// One warp copies kChunk bytes of one page of one buffer at a time, 16 bytes a lane and load where
// addresses and size allow it.  Bound by memory: each byte once in and once out.
template <typename W>
__device__ __forceinline__ void copy_words(char* d, const char* s, int64_t from, int64_t to, int lane) {
  constexpr int U = 8;
  const W* sp = reinterpret_cast<const W*>(s);
  W* dp = reinterpret_cast<W*>(d);
  const int64_t b = from / (int)sizeof(W), e = to / (int)sizeof(W);
  for (int64_t i = b + lane; i < e; i += 32 * U) {
    W v[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i + 32 * u < e) v[u] = sp[i + 32 * u];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i + 32 * u < e) dp[i + 32 * u] = v[u];
  }
}

__device__ __forceinline__ void copy_pages(const CopyList& l, const Buffers& bufs, int* first) {
  // first[i]: chunks of a page in front of buffer i
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  if (threadIdx.x < 32) {
    int before = 0;
    for (int base = 0; base < bufs.n; base += 32) {
      const int i = base + lane;
      const int c = i < bufs.n ? (int)(((int64_t)bufs.bytes[i] * 4 + kChunk - 1) / kChunk) : 0;
      int incl = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += u;
      }
      if (i < bufs.n) first[i] = before + incl - c;
      before += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) first[bufs.n] = before;
  }
  __syncthreads();
  const int per = first[bufs.n];
  const int count = l.count_dev ? *l.count_dev : l.count;
  const int64_t total = (int64_t)count * per, step = (int64_t)gridDim.x * warps;
  for (int64_t u = (int64_t)blockIdx.x * warps + (threadIdx.x >> 5); u < total; u += step) {
    const int i = (int)(u / per), c = (int)(u - (int64_t)i * per);
    const int src = l.src[i], dst = l.dst[i];
    if (src < 0 || src >= l.n_pages || dst < 0 || dst >= l.n_pages) {
      if (lane == 0) flag_status(l.status, DFLASH_STATUS_PAGE);
      continue;
    }
    int lo = 0, hi = bufs.n;  // the buffer of chunk c
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (first[mid] <= c) lo = mid;
      else hi = mid;
    }
    const char* s = bufs.data[lo] + src * bufs.stride[lo];
    char* d = bufs.data[lo] + dst * bufs.stride[lo];
    const int64_t from = (int64_t)(c - first[lo]) * kChunk, bytes = (int64_t)bufs.bytes[lo] * 4;
    const int64_t to = min(from + kChunk, bytes);
    if ((((uint64_t)s | (uint64_t)d | (uint64_t)bytes) & 15u) == 0) copy_words<uint4>(d, s, from, to, lane);
    else copy_words<uint32_t>(d, s, from, to, lane);
  }
}

constexpr int kCopyThreads = 256;
__global__ void __launch_bounds__(kCopyThreads) k_pages_copy(CopyList l, const __grid_constant__ Buffers bufs) {
  __shared__ int first[kBuffers + 1];
  pdl_trigger();
  pdl_wait();
  l.src = after_wait(l.src);
  l.dst = after_wait(l.dst);
  if (l.count_dev) l.count_dev = after_wait(l.count_dev);
  copy_pages(l, bufs, first);
}

// ---------------------------------------------------------------------------
// rows of the table
// ---------------------------------------------------------------------------
struct Rows {
  int32_t n, width, stride, shift;
  int32_t* table;
  int32_t* lens;
};
// Pages of a length; -1: more than a row holds, or negative.
__device__ __forceinline__ int pages_of(int len, const Rows& t) {
  if (len < 0) return -1;
  const int p = (int)(((int64_t)len + (1 << t.shift) - 1) >> t.shift);
  return p <= t.width ? p : -1;
}

// A warp per row: those of `from` give their entries back, those of `to` take their parents'.
__global__ void __launch_bounds__(256) k_pages_reorder(int32_t* refs, int n_pages, Rows from, const int32_t* parents,
                                                       Rows to, int32_t* status) {
  pdl_trigger();
  pdl_wait();
  from.table = after_wait(from.table);
  from.lens = after_wait(from.lens);
  parents = after_wait(parents);
  const int lane = threadIdx.x & 31, w = (int)(blockIdx.x * 8 + (threadIdx.x >> 5));
  if (w >= from.n + to.n) return;
  const bool gives = w < from.n;
  const int row = gives ? w : w - from.n;
  int parent = gives ? row : parents[row], bad = 0;
  if (parent < -1 || parent >= from.n) {
    bad = DFLASH_STATUS_BOUNDS;
    parent = -1;
  }
  int len = parent >= 0 ? from.lens[parent] : 0, pages = pages_of(len, from);
  if (!gives && pages > to.width) pages = -1;
  if (pages < 0) {
    bad |= DFLASH_STATUS_BOUNDS;
    pages = gives && len > 0 ? from.width : 0;  // (what the row has is given back all the same)
    len = 0;
  }
  const int32_t* src = from.table + (int64_t)max(parent, 0) * from.stride;
  int32_t* dst = to.table + (int64_t)row * to.stride;
  const int end = gives ? pages : to.width;
  constexpr int U = 8;  // entries in flight
  for (int j0 = lane; j0 < end; j0 += 32 * U) {
    int es[U];
#pragma unroll
    for (int u = 0; u < U; ++u) es[u] = j0 + 32 * u < pages ? src[j0 + 32 * u] : -1;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = j0 + 32 * u;
      if (j >= end) break;
      int e = es[u];
      if (j < pages) {
        if (e >= 0 && e < n_pages) {
          atomicAdd(refs + e, gives ? -1 : 1);
        } else {
          bad |= gives && len == 0 ? 0 : DFLASH_STATUS_PAGE;
          e = -1;
        }
      }
      if (!gives) dst[j] = e;
    }
  }
  if (!gives && lane == 0) to.lens[row] = len;
  if (bad) flag_status(status, bad);
}

// ---------------------------------------------------------------------------
// growth and trimming
// ---------------------------------------------------------------------------
constexpr int kCluster = 8, kScanThreads = 1024;

// Sums over the threads of a cluster (ONE: of one CTA): each thread's exclusive prefix of v in (rank,
// thread) order, and the total.  64 bits: two counts ride in one word.
template <bool ONE>
struct Scan {
  uint64_t* warps;  // [32] of this CTA
  uint64_t* ctas;   // [1] of this CTA, read by its peers
  uint64_t prefix, total;
  __device__ __forceinline__ void run(uint64_t v) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint64_t incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t u = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += u;
    }
    if (lane == 31) warps[warp] = incl;
    __syncthreads();
    if (warp == 0) {
      uint64_t w = warps[lane], wi = w;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint64_t u = __shfl_up_sync(0xffffffffu, wi, o);
        if (lane >= o) wi += u;
      }
      warps[lane] = wi - w;
      if (lane == 31) *ctas = wi;
    }
    if (ONE) {
      __syncthreads();
      prefix = warps[warp] + incl - v;
      total = *ctas;
      return;
    }
    cg::cluster_group cl = cg::this_cluster();
    cl.sync();
    prefix = warps[warp] + incl - v;
    total = 0;
    for (int q = 0; q < kCluster; ++q) {
      const uint64_t c = *cl.map_shared_rank(ctas, q);
      if (q < (int)cl.block_rank()) prefix += c;
      total += c;
    }
  }
};

__device__ __forceinline__ int load_now(const int32_t* p) { return __ldcg(p); }  // (L2: other SMs' atomics show)

struct ResizeWs {
  int32_t* owner;    // [n_pages] lowest row that writes to a shared page
  int32_t* writers;  // [n_pages] how many rows do
  int32_t* free_;    // [n_pages] free pages, ascending
  int32_t* src;      // [rows] copies
  int32_t* dst;
  int32_t* count;    // [1]
};

// What a row asks for.
struct Ask {
  int old_len, new_len, have, need;
  bool ok, writes;
};
__device__ __forceinline__ Ask ask_of(const Rows& t, const int32_t* new_lens, int row) {
  Ask a;
  a.old_len = t.lens[row];
  a.new_len = new_lens[row];
  a.have = pages_of(a.old_len, t);
  a.need = pages_of(a.new_len, t);
  a.ok = a.have >= 0 && a.need >= 0;
  a.writes = a.ok && a.new_len > a.old_len && (a.old_len & ((1 << t.shift) - 1));
  return a;
}

// One cluster.  A thread has a stretch of rows and a stretch of pages, both contiguous, so that ranks
// are prefix sums over the threads.  Bound by latency: four cluster barriers (five where pages run out) and the loads
// between them (32 prompts
// of 8 samples, with the reorder in front and the copies behind it: 26.7 us, 31.1 when rows and entries were read again
// in each step and one at a time).
// ONE: a small pool and little to copy, one CTA, whose working arrays are in shared memory and which makes
// the copies itself: one launch in place of two.  A user's four candidates, 76 pages, 2 layers, with the reorder in
// front: 12.5 us, some 13 otherwise, and 20.6 against 23 of host time.
constexpr int kSmallPages = 2048, kSmallRows = 1024, kSmallBytes = 512 << 10;
template <bool ONE>
__device__ __forceinline__ void resize(int32_t* refs, int n_pages, Rows t, const int32_t* new_lens, ResizeWs ws,
                                       int32_t* free_pages, int32_t* status) {
  __shared__ uint64_t s_warps[2][32], s_cta[2];
  auto sync = [] {
    if constexpr (ONE) __syncthreads();
    else cg::this_cluster().sync();
  };
  // (working arrays: shared memory, or written by other SMs)
  auto get = [](const int32_t* p) { return ONE ? *p : load_now(p); };
  pdl_trigger();
  pdl_wait();
  t.table = after_wait(t.table);
  t.lens = after_wait(t.lens);
  new_lens = after_wait(new_lens);
  refs = after_wait(refs);
  const int rank = ONE ? 0 : (int)cg::this_cluster().block_rank();
  const int tid = rank * kScanThreads + threadIdx.x, threads = (ONE ? 1 : kCluster) * kScanThreads;
  const int lane = threadIdx.x & 31, gwarp = tid >> 5, gwarps = threads >> 5;
  int bad = 0;
  auto entry = [&](int row, int j) { return t.table + (int64_t)row * t.stride + j; };
  auto there = [&](int p) { return p >= 0 && p < n_pages; };
  if (tid == 0) *ws.count = 0;
  // 1: pages behind the new lengths go back; the counters of begun pages start anew.  A warp per row.
  for (int row = gwarp; row < t.n; row += gwarps) {
    const Ask a = ask_of(t, new_lens, row);
    if (!a.ok) {
      bad |= DFLASH_STATUS_BOUNDS;
      continue;
    }
    for (int j = a.need + lane; j < a.have; j += 32) {
      const int p = *entry(row, j);
      if (there(p)) atomicSub(refs + p, 1);
      else bad |= DFLASH_STATUS_PAGE;
      *entry(row, j) = -1;
    }
    if (a.writes && lane == 0) {
      const int p = *entry(row, a.have - 1);
      if (there(p)) {
        ws.owner[p] = INT32_MAX;
        ws.writers[p] = 0;
      } else {
        bad |= DFLASH_STATUS_PAGE;
      }
    }
  }
  sync();
  // 2: who writes to begun pages.  With a row per thread, what it has read of its row stays in registers.
  const bool own = t.n <= threads;
  Ask mine_a{0, 0, 0, 0, false, false};
  int mine_page = -1, mine_refs = 0;
  for (int row = tid; row < t.n; row += threads) {
    const Ask a = ask_of(t, new_lens, row);
    mine_a = a;
    if (!a.writes) continue;
    const int p = *entry(row, a.have - 1), n = there(p) ? load_now(refs + p) : 0;
    mine_page = p;
    mine_refs = n;
    if (n > 1) {
      atomicMin(ws.owner + p, row);
      atomicAdd(ws.writers + p, 1);
    }
  }
  auto ask = [&](int row) { return own ? mine_a : ask_of(t, new_lens, row); };
  // meanwhile the free pages are counted and listed
  const int per_p = (n_pages + threads - 1) / threads, p0 = min(tid * (int64_t)per_p, (int64_t)n_pages), p1 = min(p0 + per_p, n_pages);
  int mine = 0;
  uint32_t which = 0;  // of up to 32
#pragma unroll 4
  for (int p = p0; p < p1; ++p) {
    const bool is = load_now(refs + p) <= 0;
    mine += is;
    which |= (uint32_t)is << ((p - p0) & 31);
  }
  Scan<ONE> fs{s_warps[0], &s_cta[0], 0, 0};
  fs.run((uint64_t)mine);  // (its barrier ends 2)
  {
    int at = (int)fs.prefix;
    if (mine)
      for (int p = p0; p < p1; ++p)
        if (per_p <= 32 ? (which >> (p - p0)) & 1u : load_now(refs + p) <= 0) ws.free_[at++] = p;
  }
  // 3: what each row needs
  const int per_r = (t.n + threads - 1) / threads, r0 = min(tid * (int64_t)per_r, (int64_t)t.n), r1 = min(r0 + per_r, t.n);
  auto copies = [&](int row, const Ask& a) {
    if (!a.writes) return false;
    const int p = own ? mine_page : *entry(row, a.have - 1);
    if (!there(p)) return false;
    const int n = own ? mine_refs : load_now(refs + p);
    return n > 1 && !(n == get(ws.writers + p) && get(ws.owner + p) == row);
  };
  uint64_t sum = 0;  // pages << 16 | copies: up to 2^15 rows ask for 2^35 + 2^15 pages and 2^15 copies
  uint32_t own_copy = 0;  // a bit per row of this thread: its begun page has to be copied
  for (int row = r0; row < r1; ++row) {
    const Ask a = ask(row);
    if (!a.ok) continue;
    const bool c = copies(row, a);
    own_copy |= (uint32_t)c << (row - r0);
    sum += (uint64_t)(max(a.need - a.have, 0) + c) << 16 | (uint64_t)c;
  }
  Scan<ONE> rs{s_warps[1], &s_cta[1], 0, 0};
  if (free_pages && tid == 0) *free_pages = (int)fs.total;
  rs.run(sum);
  const int64_t n_free = (int64_t)fs.total;
  int64_t pages = (int64_t)(rs.prefix >> 16), made = (int64_t)(rs.prefix & 0xffffu);
  // 4: rows take their pages, behind those of the rows in front of them.  Once one does not get
  // its pages none behind it does (their sums only grow), so the copies that are made are the
  // first of the list.
  auto asks = [&](int row, const Ask& a) { return max(a.need - a.have, 0) + (int)((own_copy >> (row - r0)) & 1u); };
  uint32_t granted = 0, copied = 0;  // a bit per row of this thread
  int64_t sum_to = pages;
  for (int row = r0; row < r1; ++row) {
    const Ask a = ask(row);
    if (!a.ok) continue;
    const int n = asks(row, a);
    if (n == 0 || sum_to + n <= n_free) granted |= 1u << (row - r0);
    sum_to += n;
  }
  if ((int64_t)(rs.total >> 16) > n_free) {
    // Some rows are refused (the same answer in every thread).  One that does not get its copy still names the page
    // that it shares, which the row that would keep it must not write to then: that one is refused too.
    for (int row = r0; row < r1; ++row)
      if ((own_copy & ~granted) >> (row - r0) & 1u) ws.owner[own ? mine_page : *entry(row, ask(row).have - 1)] = -1;
    sync();
    for (int row = r0; row < r1; ++row) {
      const uint32_t bit = 1u << (row - r0);
      const Ask a = ask(row);
      if (a.writes && (granted & ~own_copy & bit)) {
        const int p = own ? mine_page : *entry(row, a.have - 1);
        if (there(p) && (own ? mine_refs : load_now(refs + p)) > 1 && get(ws.owner + p) < 0) granted &= ~bit;
      }
      if (a.ok && !(granted & bit)) bad |= DFLASH_STATUS_FULL;
    }
  }
  int given = 0;
  for (int row = r0; row < r1; ++row) {
    const Ask a = ask(row);
    if (!a.ok) continue;
    const int n = asks(row, a);
    if ((granted >> (row - r0)) & 1u) {
      int64_t at = pages;
      if ((own_copy >> (row - r0)) & 1u) {
        copied |= 1u << (row - r0);
        ws.src[made] = own ? mine_page : *entry(row, a.have - 1);
        ws.dst[made] = get(ws.free_ + at++);
        ++made;
      }
      for (int j = a.have; j < a.need; ++j) {
        const int p = get(ws.free_ + at++);
        *entry(row, j) = p;
        refs[p] = 1;
      }
      given += n;
    }
    pages += n;
  }
  if (copied) atomicAdd(ws.count, __popc(copied));
  if (given && free_pages) atomicSub(free_pages, given);
  sync();  // every row has looked at the begun pages' counts
  // 5: the copies' pages take the places of those that they are copies of; lengths
  made -= __popc(copied);
  for (int row = r0; row < r1; ++row) {
    if (!((granted >> (row - r0)) & 1u)) continue;
    if ((copied >> (row - r0)) & 1u) {
      const int p = ws.dst[made++];
      int32_t* e = entry(row, ask(row).have - 1);
      atomicSub(refs + (own ? mine_page : *e), 1);
      refs[p] = 1;
      *e = p;
    }
    t.lens[row] = ask(row).new_len;
  }
  if (bad) flag_status(status, bad);
}

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kScanThreads)
    k_pages_resize(int32_t* refs, int n_pages, Rows t, const int32_t* new_lens, ResizeWs ws, int32_t* free_pages,
                   int32_t* status) {
  resize<false>(refs, n_pages, t, new_lens, ws, free_pages, status);
}
__global__ void __launch_bounds__(kScanThreads) k_pages_resize_one(int32_t* refs, int n_pages, Rows t, const int32_t* new_lens,
                                                                   int32_t* free_pages, int32_t* status,
                                                                   const __grid_constant__ Buffers bufs) {
  __shared__ int32_t owner[kSmallPages], writers[kSmallPages], free_list[kSmallPages], src[kSmallRows], dst[kSmallRows], count;
  __shared__ int first[kBuffers + 1];
  resize<true>(refs, n_pages, t, new_lens, ResizeWs{owner, writers, free_list, src, dst, &count}, free_pages, status);
  __syncthreads();
  if (bufs.n > 0) copy_pages(CopyList{src, dst, &count, 0, n_pages, status}, bufs, first);
}

// ---------------------------------------------------------------------------
// a dense pool
// ---------------------------------------------------------------------------
struct CompactWs {
  int32_t* src;    // [n_pages] pages that move, ascending
  int32_t* dst;    // [n_pages] where to, ascending
  int32_t* to;     // [n_pages] of pages behind the dense part: where to, -1: not in use
  int32_t* count;  // [2] moves, pages in use
};

// One cluster: the count U of pages in use, then by rank the free pages below U and the pages in use from U on,
// which are as many.
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kScanThreads)
    k_pages_compact(const int32_t* refs, int32_t* new_refs, int n_pages, CompactWs ws, int32_t* used) {
  __shared__ uint64_t s_warps[2][32], s_cta[2];
  pdl_trigger();
  pdl_wait();
  refs = after_wait(refs);
  cg::cluster_group cl = cg::this_cluster();
  const int tid = (int)cl.block_rank() * kScanThreads + threadIdx.x, threads = kCluster * kScanThreads;
  const int per = (n_pages + threads - 1) / threads, p0 = min(tid * (int64_t)per, (int64_t)n_pages), p1 = min(p0 + per, n_pages);
  int mine = 0;
#pragma unroll 4
  for (int p = p0; p < p1; ++p) mine += refs[p] > 0;
  Scan<false> us{s_warps[0], &s_cta[0], 0, 0};
  us.run((uint64_t)mine);
  const int U = (int)us.total;
  uint64_t sum = 0;  // holes << 32 | movers
  for (int p = p0; p < p1; ++p) {
    const bool in = refs[p] > 0;
    if (p < U && !in) sum += 1ull << 32;
    if (p >= U && in) sum += 1;
  }
  Scan<false> ms{s_warps[1], &s_cta[1], 0, 0};
  ms.run(sum);
  int hole = (int)(ms.prefix >> 32), mover = (int)(ms.prefix & 0xffffffffu);
  const int moves = (int)(ms.total & 0xffffffffu);
  for (int p = p0; p < p1; ++p) {
    const bool in = refs[p] > 0;
    if (p < U) {
      if (!in) ws.dst[hole++] = p;
    } else if (in) {
      ws.src[mover++] = p;
    } else {
      ws.to[p] = -1;
    }
  }
  cl.sync();
  for (int i = tid; i < moves; i += threads) {
    const int a = load_now(ws.src + i), b = load_now(ws.dst + i);
    ws.to[a] = b;
    new_refs[b] = refs[a];
  }
  if (refs != new_refs)
    for (int p = p0; p < p1; ++p)
      if (p < U && refs[p] > 0) new_refs[p] = refs[p];
  cl.sync();  // (in place: the moved counts have been read)
  for (int p = max(p0, U); p < p1; ++p) new_refs[p] = 0;
  if (tid == 0) {
    ws.count[0] = moves;
    ws.count[1] = U;
    if (used) *used = U;
  }
}

// The table's entries and the pages themselves: a warp per row, then the copies.
__global__ void __launch_bounds__(kCopyThreads) k_pages_compact_move(CopyList l, const int32_t* to, const int32_t* used,
                                                                     int n_pages, Rows from, Rows into,
                                                                     const __grid_constant__ Buffers bufs, bool entries) {
  __shared__ int first[kBuffers + 1];
  pdl_trigger();
  pdl_wait();
  l.src = after_wait(l.src);
  l.dst = after_wait(l.dst);
  l.count_dev = after_wait(l.count_dev);
  from.table = after_wait(from.table);
  from.lens = after_wait(from.lens);
  to = after_wait(to);
  const int lane = threadIdx.x & 31, warps = kCopyThreads / 32, U = *after_wait(used);
  if (entries) {
    for (int row = (int)blockIdx.x * warps + (threadIdx.x >> 5); row < from.n; row += gridDim.x * warps) {
      int len = from.lens[row], pages = pages_of(len, from), bad = 0;
      if (pages < 0) {
        bad = DFLASH_STATUS_BOUNDS;
        pages = len = 0;
      }
      const int32_t* s = from.table + (int64_t)row * from.stride;
      int32_t* d = into.table + (int64_t)row * into.stride;
      constexpr int W = 4;  // entries in flight
      for (int j0 = lane; j0 < from.width; j0 += 32 * W) {
        int es[W];
#pragma unroll
        for (int u = 0; u < W; ++u) es[u] = j0 + 32 * u < pages ? s[j0 + 32 * u] : -1;
#pragma unroll
        for (int u = 0; u < W; ++u) es[u] = es[u] >= n_pages ? -1 : es[u] >= U ? to[es[u]] : es[u];
#pragma unroll
        for (int u = 0; u < W; ++u) {
          const int j = j0 + 32 * u;
          if (j >= from.width) break;
          if (j < pages && es[u] < 0) bad |= DFLASH_STATUS_PAGE;
          d[j] = max(es[u], -1);
        }
      }
      __syncwarp();
      if (lane == 0) into.lens[row] = len;
      if (bad) flag_status(l.status, bad);
    }
  }
  if (bufs.n > 0) copy_pages(l, bufs, first);
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
int check_pool(const char* call, const void* refs, int64_t n_pages) {
  if (!refs || (uintptr_t)refs % 4) return rfail(DFLASH_ERR_INVALID_ARG, call, "refs: 4-byte aligned, not null");
  if (n_pages < 1 || n_pages > (1 << 30)) return rfail(DFLASH_ERR_SHAPE, call, "n_pages outside 1..2^30");
  return DFLASH_OK;
}
int check_rows(const char* call, const dflash_page_rows* r) {
  if (!r || !r->table || !r->lens) return rfail(DFLASH_ERR_INVALID_ARG, call, "null rows, table or lens");
  if (r->rows < 1 || r->rows > 32768) return rfail(DFLASH_ERR_INVALID_ARG, call, "rows outside 1..32768");
  if (r->width < 1 || r->width > (1 << 20) || r->stride < r->width)
    return rfail(DFLASH_ERR_INVALID_ARG, call, "width outside 1..2^20 or stride below it");
  if (r->page_size < 8 || r->page_size > 1024 || !pow2(r->page_size))
    return rfail(DFLASH_ERR_SHAPE, call, "page_size: a power of two in 8..1024");
  return DFLASH_OK;
}
Rows rows_of(const dflash_page_rows* r) {
  int shift = 0;
  while ((1 << shift) < r->page_size) ++shift;
  return Rows{r->rows, r->width, r->stride, shift, r->table, r->lens};
}
int check_buffers(const char* call, const dflash_page_buffer* b, int32_t n) {
  if (n < 0 || n > 4096 || (n > 0 && !b)) return rfail(DFLASH_ERR_INVALID_ARG, call, "buffers: 0..4096 of them, not null");
  for (int i = 0; i < n; ++i)
    if (!b[i].data || (uintptr_t)b[i].data % 4 || b[i].page_stride % 4 || b[i].page_bytes % 4 || b[i].page_bytes < 4 ||
        b[i].page_bytes > (1 << 30) || b[i].page_stride < b[i].page_bytes || b[i].page_stride > ((int64_t)1 << 40))
      return rfail(DFLASH_ERR_INVALID_ARG, call, "a buffer: not null, multiples of 4, page_bytes 4..2^30, page_stride at least that");
  return DFLASH_OK;
}
Buffers buffers_of(const dflash_page_buffer* b, int from, int n) {
  Buffers o;
  o.n = std::min(kBuffers, n - from);
  for (int i = 0; i < o.n; ++i) {
    o.data[i] = (char*)b[from + i].data;
    o.stride[i] = b[from + i].page_stride;
    o.bytes[i] = (int32_t)(b[from + i].page_bytes / 4);
  }
  return o;
}
int64_t chunks_of(const Buffers& b) {
  int64_t c = 0;
  for (int i = 0; i < b.n; ++i) c += ((int64_t)b.bytes[i] * 4 + kChunk - 1) / kChunk;
  return c;
}
// CTAs for up to `most` copies: eight of 256 threads fill an SM
unsigned copy_grid(int64_t most, const Buffers& b) {
  return (unsigned)std::max<int64_t>(1, std::min<int64_t>((most * chunks_of(b) + 7) / 8, 152 * 8));
}
cudaError_t launch_copies(const CopyList& l, int64_t most, const dflash_page_buffer* b, int32_t n, cudaStream_t st) {
  for (int from = 0; from < n; from += kBuffers) {
    const Buffers bufs = buffers_of(b, from, n);
    if (cudaError_t e = launch_k(k_pages_copy, copy_grid(most, bufs), kCopyThreads, 0, st, l, bufs)) return e;
  }
  return cudaSuccess;
}
int64_t workspace_bytes(int64_t n_pages, int32_t rows) { return 4 * (3 * n_pages + 2 * (int64_t)rows + 2); }
int check_workspace(const char* call, const void* ws, int64_t bytes, int64_t n_pages, int32_t rows) {
  if (!ws || (uintptr_t)ws % 4 || bytes < workspace_bytes(n_pages, rows))
    return rfail(DFLASH_ERR_INVALID_ARG, call, "workspace: 4-byte aligned, at least dflash_pages_workspace bytes");
  return DFLASH_OK;
}

}  // namespace
}  // namespace dfl

using namespace dfl;

extern "C" {

DFLASH_API int dflash_pages_copy(const dflash_page_buffer* buffers, int32_t n_buffers, int64_t n_pages,
                                 const int32_t* src, const int32_t* dst, int32_t count, int32_t* status, void* stream) {
  const char* call = "dflash_pages_copy";
  if (int rc = check_buffers(call, buffers, n_buffers)) return rc;
  if (n_pages < 1 || n_pages > (1 << 30)) return rfail(DFLASH_ERR_SHAPE, call, "n_pages outside 1..2^30");
  if (count < 0 || (count > 0 && (!src || !dst))) return rfail(DFLASH_ERR_INVALID_ARG, call, "src, dst or count");
  if (count == 0) return DFLASH_OK;
  return rcheck(launch_copies(CopyList{src, dst, nullptr, count, n_pages, status}, count, buffers, n_buffers, (cudaStream_t)stream), call);
}

DFLASH_API int dflash_pages_reorder(int32_t* refs, int64_t n_pages, const dflash_page_rows* from,
                                    const int32_t* parents, const dflash_page_rows* to, int32_t* status, void* stream) {
  const char* call = "dflash_pages_reorder";
  if (int rc = check_pool(call, refs, n_pages)) return rc;
  if (int rc = check_rows(call, from)) return rc;
  if (int rc = check_rows(call, to)) return rc;
  if (!parents) return rfail(DFLASH_ERR_INVALID_ARG, call, "null parents");
  if (from->page_size != to->page_size) return rfail(DFLASH_ERR_SHAPE, call, "the page sizes differ");
  if (from->table == to->table || from->lens == to->lens) return rfail(DFLASH_ERR_INVALID_ARG, call, "to is from");
  return rcheck(launch_k(k_pages_reorder, (unsigned)((from->rows + to->rows + 7) / 8), 256, 0, (cudaStream_t)stream, refs,
                         (int)n_pages, rows_of(from), parents, rows_of(to), status),
                call);
}

DFLASH_API int64_t dflash_pages_workspace(int64_t n_pages, int32_t rows) {
  const char* call = "dflash_pages_workspace";
  if (n_pages < 1 || n_pages > (1 << 30)) return rfail(DFLASH_ERR_SHAPE, call, "n_pages outside 1..2^30");
  if (rows < 1 || rows > 32768) return rfail(DFLASH_ERR_INVALID_ARG, call, "rows outside 1..32768");
  return workspace_bytes(n_pages, rows);
}

DFLASH_API int dflash_pages_resize(int32_t* refs, int64_t n_pages, const dflash_page_rows* rows,
                                   const int32_t* new_lens, const dflash_page_buffer* buffers, int32_t n_buffers,
                                   int32_t* free_pages, void* workspace, int64_t workspace_bytes_, int32_t* status,
                                   void* stream) {
  const char* call = "dflash_pages_resize";
  if (int rc = check_pool(call, refs, n_pages)) return rc;
  if (int rc = check_rows(call, rows)) return rc;
  if (!new_lens) return rfail(DFLASH_ERR_INVALID_ARG, call, "null new_lens");
  if (new_lens == rows->lens) return rfail(DFLASH_ERR_INVALID_ARG, call, "new_lens is lens");
  if (int rc = check_buffers(call, buffers, n_buffers)) return rc;
  if (int rc = check_workspace(call, workspace, workspace_bytes_, n_pages, rows->rows)) return rc;
  cudaStream_t st = (cudaStream_t)stream;
  int32_t* w = (int32_t*)workspace;
  const ResizeWs ws{w, w + n_pages, w + 2 * n_pages, w + 3 * n_pages, w + 3 * n_pages + rows->rows,
                    w + 3 * n_pages + 2 * (int64_t)rows->rows};
  int64_t page = 0;  // bytes of a page in all buffers
  for (int i = 0; i < n_buffers; ++i) page += buffers[i].page_bytes;
  if (n_pages <= kSmallPages && rows->rows <= kSmallRows && n_buffers <= kBuffers && page * rows->rows <= kSmallBytes)
    return rcheck(launch_k(k_pages_resize_one, 1, kScanThreads, 0, st, refs, (int)n_pages, rows_of(rows), new_lens, free_pages,
                           status, buffers_of(buffers, 0, n_buffers)),
                  call);
  if (int rc = rcheck(launch_k(k_pages_resize, kCluster, kScanThreads, 0, st, refs, (int)n_pages, rows_of(rows), new_lens,
                               ws, free_pages, status),
                      call))
    return rc;
  return rcheck(launch_copies(CopyList{ws.src, ws.dst, ws.count, 0, n_pages, status}, rows->rows, buffers, n_buffers, st), call);
}

DFLASH_API int dflash_pages_compact(const int32_t* refs, int32_t* new_refs, int64_t n_pages,
                                    const dflash_page_rows* from, const dflash_page_rows* to,
                                    const dflash_page_buffer* buffers, int32_t n_buffers, int32_t* used,
                                    void* workspace, int64_t workspace_bytes_, int32_t* status, void* stream) {
  const char* call = "dflash_pages_compact";
  if (int rc = check_pool(call, refs, n_pages)) return rc;
  if (int rc = check_pool(call, new_refs, n_pages)) return rc;
  if (int rc = check_rows(call, from)) return rc;
  if (int rc = check_rows(call, to)) return rc;
  if (from->rows != to->rows || from->width != to->width || from->page_size != to->page_size)
    return rfail(DFLASH_ERR_SHAPE, call, "rows, width or page_size of from and to differ");
  if (from->table == to->table && from->stride != to->stride)
    return rfail(DFLASH_ERR_INVALID_ARG, call, "in place: the strides of from and to are the same");
  if (int rc = check_buffers(call, buffers, n_buffers)) return rc;
  if (int rc = check_workspace(call, workspace, workspace_bytes_, n_pages, from->rows)) return rc;
  cudaStream_t st = (cudaStream_t)stream;
  int32_t* w = (int32_t*)workspace;
  const CompactWs ws{w, w + n_pages, w + 2 * n_pages, w + 3 * n_pages};
  if (int rc = rcheck(launch_k(k_pages_compact, kCluster, kScanThreads, 0, st, refs, new_refs, (int)n_pages, ws, used), call))
    return rc;
  const CopyList l{ws.src, ws.dst, ws.count, 0, n_pages, status};
  for (int at = 0; at == 0 || at < n_buffers; at += kBuffers) {
    const Buffers bufs = buffers_of(buffers, at, n_buffers);
    const int64_t most = std::max<int64_t>(n_pages / 2, 1);  // moves: as many free pages as pages in use
    const unsigned grid = std::max(copy_grid(most, bufs), (unsigned)std::min((from->rows + 7) / 8, 152 * 8));
    if (int rc = rcheck(launch_k(k_pages_compact_move, grid, kCopyThreads, 0, st, l, ws.to, ws.count + 1, (int)n_pages,
                                 rows_of(from), rows_of(to), bufs, at == 0),
                        call))
      return rc;
  }
  return DFLASH_OK;
}

}  // extern "C"
