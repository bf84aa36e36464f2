// Attention of ragged new rows over paged or packed K/V on the sm_103a tensor
// cores (bf16, head_dim 64 or 128).
//
// Rows are (token, query head of one KV head's group) pairs: a tile of 128
// rows holds floor(128 / G) tokens x G heads.  A CTA works on NQ tiles of one
// sequence and KV head at a time (an item), 128 keys per step:
//   S = Q K^T        tcgen05, K tile as it lies in shared memory
//   P = 2^(S k - m)  one thread per row: S from TMEM, running maximum with lazy
//                    rescaling (O and l move only when the maximum grew by more
//                    than 2^8), P as bf16 back into S's own TMEM columns
//   O += P V         A = P from TMEM, B = V as it lies in the cache (rows of d:
//                    the N-contiguous operand form, no transposed copy)
// Rounding: P to bf16 once, because tcgen05 wants A in the type of B (half a
// step, at most 2^-8 of each probability, without a bias that the sums would
// keep); the maximum, l (of the unrounded P), O and the merges are fp32.
//
// Warps: 4 NQ softmax warps (tile x: warps 4x .. 4x+3), a TMA producer, the
// MMA issuer, a "fixer" and a scheduler.  Stretches of work overlap: the first S
// of the next one is issued behind the last product of its stream.
//   NQ = 2 (more than 128 rows): the two tiles share each K/V tile and alternate, one's
//          softmax under the other's two products.  Bound by that chain: about 3060
//          cycles for a key tile of both, of which the products alone are 2050.
//          8192 tokens, 32 over 8 heads of 128, all keys visible: 0.72 ms, 1.53
//          PFLOP/s (82% of a measured cuBLAS peak); causal 1.43; head dim 64 0.82.
//   NQ = 1: one tile, S double-buffered; bound by the K/V stream: 64 single tokens
//          over 4096, 8 KV heads of 128: 5.8 TB/s with pages of 16 (TMA boxes of 4 KB
//          are what limits it), 6.0 with pages of 64 (89% of a measured copy).  Few
//          short items are latency: 15 us for one block of 16 tokens over 4096.
//   KV8 (NQ = 2): an 8-bit cache.  Codes come by TMA, asked for by the scheduler warp; two warps (those of the
//          producer and the fixer) make V's, and for heads of 64 K's, fp16 in the ring.  For heads of 128 K's codes are
//          multiplied as they are (kind::f8f6f4) with q as a sum of two e4m3 numbers, the softmax warps' first
//          work on a stretch, so that K takes a quarter of the room and no conversion.  The softmax takes the
//          scales (softmax_tile8).  4 x 2048 new rows over 6000 tokens, 32 over 8 heads of 128: 0.86 ms, 1.10
//          PFLOP/s (56% of a measured cuBLAS peak), heads of 64 0.69 ms (0.68); 6 chunks of 145 to 477 rows over 1.9k to
//          4.8k 138 us, 0.67 PFLOP/s (whole items, two or one a CTA, leave a sixth of the SMs' time empty).
//          Bound by the softmax of two tiles in turn (0.84 ms when its parts were timed): with the softmax left out 0.69 ms, the converters 0.84, a
//          half or seven eighths of either product 0.86; the products alone are 0.48.
// V rows of hidden keys may hold anything, and 0 * NaN is NaN: in tiles with
// hidden keys the fixer zeroes the rows behind the sequence and puts non-finite
// numbers in the others to 0; the softmax warps then add those to the rows that
// see them (add_nonfinite).
//
// Work is laid out on the device from the lengths there, in one of three ways:
//   items   whole items, longest first (by key tiles, counted by binary search,
//           no sort), dealt to the persistent CTAs in snake order;
//   ranges  the concatenation of all items' key tiles cut into equal ranges,
//           one per CTA; the parts of a cut item meet in k_ragged_merge;
//   cluster few items of few key tiles (a verified block of one user): the key
//           tiles of an item dealt to a thread-block cluster, the parts meet in
//           distributed shared memory.  One launch, nothing to search.
// Every wait is bounded; an expired one sets DFLASH_STATUS_WAIT.
#include <cooperative_groups.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "common.cuh"
#include "kv8.h"
#include "launch.h"
#include "ragged.h"
#include "tc_ptx.cuh"

namespace dfl {

namespace {

using namespace tc;
namespace cg = cooperative_groups;

constexpr int KT = 128;          // keys per tile
constexpr int NW = 4;            // work descriptors in flight
constexpr uint32_t O_COL = 256;  // TMEM: S0 [0,128), S1 [128,256), O from 256
constexpr float kLn2 = 0.6931471805599453f, kLog2e = 1.4426950408889634f;

constexpr int kModeItems = 0, kModeRanges = 1, kModeCluster = 2;
constexpr int kMaxCluster = 16;

// The host's choices, the same for every CTA of a call.
struct Plan {
  int32_t mode;
  int32_t tpt;          // tokens per 128-row tile
  int32_t tok;          // tokens per item
  int32_t hgroup;       // items: KV heads dealt out together (bounds the K/V that is live in L2)
  int32_t cluster;      // cluster: CTAs of an item
  int32_t min_tiles_log2;  // ranges: log2 of the key tiles a CTA gets at least
  int32_t pad;          // ranges: what the start of an item costs, in key tiles
  int32_t ws_rows;      // rows of a partial
  int32_t slots;        // partials there is room for
  int32_t max_items;    // items of one KV head, and key tiles of all items (ranges), that there can be
  int32_t max_units;
};

// One stretch of key tiles [t0, t0 + max(nt)) of one item.
struct Work {
  int32_t b, start, n, len;
  int32_t kvh, i0, t0;
  int32_t nt[2];         // key tiles of each 128-row tile
  int32_t part;          // partial slot, or -1: the whole item
  int32_t clean_lo, clean_hi;  // keys that every row sees
  int32_t bad;           // set by the fixer, a bit per 128-row tile: values of V were put to 0
  int32_t done;
};

// Scales of an 8-bit tile's keys, a pair for each 16 of them.
struct __align__(16) TileScales {
  float2 key[KT / 16];  // K's, log2 of V's
  float most;           // the largest of V's logarithms
  int32_t pad[3];
};

template <int D, int NQ, bool KV8 = false>
struct Cfg {
  static constexpr int SLOT = KT * D * 2;                 // one K or V tile, one Q tile
  // 128 bytes of 32 rows for each softmax warp (NQ = 1: in the Q tile it has done with)
  static constexpr int STAGE = NQ == 2 ? 8 * 4096 : 0;
  // 8 bits: NC tiles of codes on their way to the converters, of K and V in turn, or only of V where K is multiplied
  // as it is (K8: its tiles are 2 of the ring's entries then, V's as fp16 the other 2)
  static constexpr bool K8 = KV8 && D == 128;
  static constexpr int NC = K8 ? 2 : 4;
  static constexpr int CODES = KV8 ? NC * KT * D : 0;
  static constexpr int RING = K8 ? 4 : (7 * 32768 - STAGE - CODES) / SLOT - 2;  // K/V tiles in flight
  static constexpr int RING_BYTES = K8 ? 2 * KT * D + 2 * SLOT : RING * SLOT;
  static constexpr int DATA = 2 * SLOT + RING_BYTES + STAGE + CODES;  // 224 KB
  static constexpr int THREADS = (4 * NQ + 4) * 32;
  // NQ = 2: registers of the softmax warps and of the other four; the launch's
  // 168 for all spilled 100 bytes in the key loop (452 -> 424 us for the packed
  // prompts of 1 to 8192 tokens).  8 x 200 + 4 x 104 = 12 x 168.
  static constexpr int R_SOFTMAX = 200, R_REST = 104;
  static constexpr int EXTRA = 768;  // barriers and descriptors
  // scales of as many tiles as the ring holds, the one that is being read and the next
  static constexpr int NSCALES = 8;
  static constexpr size_t SMEM = DATA + EXTRA + (KV8 ? NSCALES * sizeof(TileScales) + 2 * NC * 8 : 0);
};

__device__ __forceinline__ float max3(float a, float b, float c) {
  float m;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(a), "f"(b), "f"(c));
  return m;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint64_t f2pack(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 f2unpack(uint64_t r) {
  float2 v;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(v.x), "=f"(v.y) : "l"(r));
  return v;
}
__device__ __forceinline__ int warp_scan_i(int v, int lane) {  // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}
// eight scaled values as bf16
__device__ __forceinline__ uint4 pack8(const float* v, float f) {
  uint32_t u[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const __nv_bfloat162 b2 = __floats2bfloat162_rn(v[2 * q] * f, v[2 * q + 1] * f);
    u[q] = *reinterpret_cast<const uint32_t*>(&b2);
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}
// mbar_wait that looks at the clock only after some tries (for the wait that a
// call starts with: reading the clock takes longer)
__device__ __forceinline__ bool mbar_wait_short(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
#pragma unroll 1
  for (int i = 0; i < 32; ++i)
    if (mbar_try_wait(bar, parity)) return true;
  return mbar_wait(bar, parity, abort_flag);
}
template <int R> __device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R)); }
template <int R> __device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R)); }
// Arrival that publishes no memory (the tensor-memory fence in front of it
// orders what it hands over): unlike the default it does not wait for this
// thread's earlier stores, 300 cycles a key tile where P is handed over.
__device__ __forceinline__ void mbar_arrive_relaxed(uint64_t* bar) {
  asm volatile("mbarrier.arrive.relaxed.cta.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ int cdiv(int a, int b) { return (a + b - 1) / b; }

// ---------------------------------------------------------------------------
// the layout of the work
// ---------------------------------------------------------------------------
__device__ __forceinline__ int items_of(const Seq& s, const Plan& p) { return s.ok && s.n > 0 ? cdiv(s.n, p.tok) : 0; }
// Items of the sequence whose keys reach into tile c (1-based) or further:
// the last ones, as an item's keys end at its last token (or all at the length).
__device__ __forceinline__ int items_reaching(const Seq& s, int c, const Plan& p, int causal) {
  const int nq = items_of(s, p);
  if (nq == 0) return 0;
  const int y = KT * (c - 1) + 1;  // keys needed
  if (s.len < y) return 0;
  if (!causal) return nq;
  const int need = y - (s.len - s.n);
  const int first = need <= 0 ? 0 : cdiv(need, p.tok) - 1;
  return nq - min(first, nq - 1);
}
// ranges: a sequence's key tiles [first, first + count), taken for each of its
// items; in the units that are split evenly, `pad` empty ones lie in front of
// each item's tiles (a CTA that starts an item fills the pipeline anew)
__device__ __forceinline__ int tile_first(const Seq& s, int window) { return vis_lo(s.len - s.n, window) / KT; }
__device__ __forceinline__ int tile_count(const Seq& s, int window) { return cdiv(s.len, KT) - tile_first(s, window); }
__device__ __forceinline__ int64_t units_of(const Seq& s, const Plan& p, const AttnCall& a) {
  return s.ok && s.n > 0 ? (int64_t)items_of(s, p) * a.Hkv * (tile_count(s, a.window) + p.pad) : 0;
}
// The sum of the lanes' counts, or -1 where it is above what the host laid the
// work out for: sequences that overlap (starts that decrease somewhere).
__device__ __forceinline__ int sum_up_to(int64_t v, int most) {
  const unsigned c = (unsigned)min(v, (int64_t)INT32_MAX);
  const int64_t sum = ((int64_t)__reduce_add_sync(0xffffffffu, c >> 16) << 16) + __reduce_add_sync(0xffffffffu, c & 0xffffu);
  return sum > most ? -1 : (int)sum;
}
// The units' even split over the CTAs that take part: range c starts at start(c).
struct Ranges {
  int n, each, rest;
  __device__ __forceinline__ Ranges(int units, const Plan& p, int grid) {
    n = max(1, min(grid, units >> p.min_tiles_log2));
    each = units / n;
    rest = units - each * n;
  }
  __device__ __forceinline__ int start(int c) const { return c * each + min(c, rest); }
  // the range that holds unit u
  __device__ __forceinline__ int of(int u) const {
    const int head = rest * (each + 1);
    return u < head ? u / (each + 1) : rest + (u - head) / each;
  }
};

// Fills in everything of w that follows from its sequence, head and tokens;
// [t0, t0 + take) are the key tiles asked for.
__device__ __forceinline__ void make_work(Work& w, const Seq& s, int b, int kvh, int qi, int t0, int take, int part,
                                          const Plan& p, const AttnCall& a) {
  w.b = b;
  w.start = s.start;
  w.n = s.n;
  w.len = s.len;
  w.kvh = kvh;
  w.i0 = qi * p.tok;
  w.part = part;
  w.bad = 0;
  w.done = 0;
  const int ctx = s.len - s.n, i1 = min(w.i0 + p.tok, s.n);
  const int lo = vis_lo(ctx + w.i0, a.window) / KT;
  w.t0 = max(t0, lo);
  w.clean_lo = vis_lo(ctx + i1 - 1, a.window);
  w.clean_hi = vis_hi(ctx + w.i0, s.len, a.causal);
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int first = w.i0 + x * p.tpt, last = min(first + p.tpt, i1) - 1;
    int t = 0;
    if (last >= first) t = max(0, min(t0 + take, cdiv(vis_hi(ctx + last, s.len, a.causal), KT)) - w.t0);
    w.nt[x] = t;
  }
}

// Where a row's results go.  A partial is O (unscaled) in ws [2 grid][ws_rows][D]
// and (m, l) behind it, [2 grid][ws_rows].
template <int D>
__device__ __forceinline__ float* part_o(const AttnCall& a, const Plan& p, int slot, int row) {
  return a.ws + ((int64_t)slot * p.ws_rows + row) * D;
}
template <int D>
__device__ __forceinline__ float2* part_ml(const AttnCall& a, const Plan& p, int slot, int row) {
  return reinterpret_cast<float2*>(a.ws + (int64_t)p.slots * p.ws_rows * D) + (int64_t)slot * p.ws_rows + row;
}
// The statistics of a part as the merges take them.  A NaN score makes l NaN but
// never becomes the maximum, so m may still be -inf, which is what a part that saw
// no key has: NaN, it cannot be taken for one.
__device__ __forceinline__ float2 part_stats(float m, float l) { return make_float2(l != l ? l : m, l); }
// The natural log-sum-exp of a row: -inf where every score is, NaN where one is.
__device__ __forceinline__ float lse_of(float m, float l) { return (m + log2f(l)) * kLn2; }
// (m, l) of a partial (row r of tile x), or the log-sum-exp of packed row tok, head h
template <int D>
__device__ __forceinline__ void store_stats(const AttnCall& a, const Plan& p, int part, int x, int r, int tok, int h,
                                            float m, float l) {
  if (part >= 0) {
    *part_ml<D>(a, p, part, x * 128 + r) = part_stats(m, l);
  } else if (a.lse) {
    a.lse[(int64_t)tok * a.Hq + h] = lse_of(m, l);
  }
}

// Halves of a pair of bf16 with an exponent of ones (infinities and NaN): bits 15 and 31.
__device__ __forceinline__ uint32_t nonfinite_bits(uint32_t w) { return ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u; }
__device__ __forceinline__ uint32_t nonfinite_bits(uint4 q) {
  return nonfinite_bits(q.x) | nonfinite_bits(q.y) | nonfinite_bits(q.z) | nonfinite_bits(q.w);
}
__device__ __forceinline__ uint32_t finite_or_0(uint32_t w) { return w & ~((nonfinite_bits(w) >> 15) * 0xffffu); }

// Adds the values that the fixer put to 0 in a stretch's V tiles to the rows that
// see them: an infinity or a NaN times a probability, which is above 0, is itself.
// A row per lane, token i's; its O in TMEM.  V is read again from the cache, only
// in the tiles that the fixer looked at.  Those lie at the two edges of an item's
// keys, at most tok / 128 + 2 at each: what this takes does not grow with the length
// (one block of 16 over 4096: 14 us, 24 with one such key, 35 with 15).
template <int D>
__device__ __noinline__ void add_nonfinite(Ragged r, KVView kv, const Work& w, uint32_t tO, int i, int window,
                                           int causal) {
  const int pos = w.len - w.n + i, lo = vis_lo(pos, window), hi = vis_hi(pos, w.len, causal);
  const int lane = threadIdx.x & 31, T = max(w.nt[0], w.nt[1]);
  for (int t = 0; t < T; ++t) {
    const int kt = (w.t0 + t) * KT, in = min(KT, w.len - kt);
    if (kt >= w.clean_lo && kt + in <= w.clean_hi) {  // and so are all up to the edge
      t = max(t, w.clean_hi / KT - 1 - w.t0);
      continue;
    }
    for (int base = kt; base < kt + in; base += 32) {
      const int j = base + lane;
      const uint4* v = nullptr;
      uint32_t found = 0;
      if (j < kt + in) {
        int64_t at = (int64_t)(w.start + j) * kv.v_slot;
        bool there = true;
        if (kv.paged) {
          const int pg = r.table[(int64_t)w.b * r.table_stride + (j >> kv.page_shift)];
          there = pg >= 0 && pg < kv.n_pages;  // (otherwise zeros)
          at = pg * kv.page + (j & ((1 << kv.page_shift) - 1)) * kv.v_slot;
        }
        if (there) {
          v = reinterpret_cast<const uint4*>(reinterpret_cast<const bf16*>(kv.v) + at + w.kvh * kv.v_head);
          for (int c = 0; c < D / 8; ++c) found |= nonfinite_bits(v[c]);
        }
      }
      uint32_t todo = __ballot_sync(0xffffffffu, found != 0);
      while (todo) {
        const int src = __ffs(todo) - 1;
        todo &= todo - 1;
        const bf16* e = reinterpret_cast<const bf16*>(__shfl_sync(0xffffffffu, (unsigned long long)v, src));
        const bool see = base + src >= lo && base + src < hi;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          float o[32];
          tmem_ld32(tO + c, o);
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            const float x = __bfloat162float(e[c + k]);
            if (see && !isfinite(x)) o[k] += x;
          }
          tmem_st32(tO + c, o);
        }
      }
    }
  }
}

// One key tile of one row (a thread each): S from TMEM, m and l brought up to
// date, P into S's first 64 columns.
struct TileArgs {
  uint32_t tS, tO;     // this warp's lanes of S and O
  int hi, lo;          // keys of the tile that the row sees: [lo, hi)
  bool masked_hi, masked_lo;  // some row of the warp misses keys there
  bool valid;
  float sl2;
};
template <int D, int NQ>
__device__ __forceinline__ bool softmax_tile(const TileArgs& a, float& m, float& l, uint64_t* pv_done, uint32_t parity,
                                             volatile int* abort_flag) {
  float s[128];
  fence_after();
  const auto keep_of = [&](int c) {  // keys c .. c + 31 that the row sees, a bit each
    const int n = min(max(a.hi - c, 0), 32);
    return n == 32 ? 0xffffffffu : (1u << n) - 1u;
  };
  if (NQ == 1 && (a.masked_hi || a.masked_lo)) {
    // masks on their own, 32 columns a turn and back into TMEM: the code of the
    // 128 scores, run once an item, took 2100 cycles (it is not in the instruction
    // cache by then)
#pragma unroll 1
    for (int c = 0; c < 128; c += 32) {
      float v[32];
      tmem_ld32(a.tS + c, v);
      const int b = min(max(a.lo - c, 0), 32);
      const uint32_t keep = keep_of(c) & (b == 32 ? 0u : ~0u << b);
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] = (keep >> j) & 1u ? v[j] : -INFINITY;
      tmem_st32(a.tS + c, v);
    }
  }
  tmem_ld128(a.tS, s);
  if (NQ == 2 && a.masked_hi) {
#pragma unroll
    for (int c = 0; c < 128; c += 32) {
      const uint32_t keep = keep_of(c);
#pragma unroll
      for (int j = 0; j < 32; ++j) s[c + j] = (keep >> j) & 1u ? s[c + j] : -INFINITY;
    }
  }
  if (NQ == 2 && a.masked_lo) {
#pragma unroll
    for (int j = 0; j < 128; ++j) s[j] = j >= a.lo ? s[j] : -INFINITY;
  }
  float m0 = s[0], m1 = s[1], m2 = s[2], m3 = s[3];
#pragma unroll
  for (int j = 4; j < 124; j += 8) {
    m0 = max3(m0, s[j], s[j + 1]);
    m1 = max3(m1, s[j + 2], s[j + 3]);
    m2 = max3(m2, s[j + 4], s[j + 5]);
    m3 = max3(m3, s[j + 6], s[j + 7]);
  }
  m0 = max3(m0, s[124], s[125]);
  m1 = max3(m1, s[126], s[127]);
  const float mt = fmaxf(fmaxf(m0, m1), fmaxf(m2, m3)) * a.sl2;
  const bool grow = a.valid && mt > m + 8.f;
  if (__any_sync(0xffffffffu, grow && m != -INFINITY)) {
    const float f = grow && m != -INFINITY ? ex2(m - mt) : 1.f;
    // O holds the previous tile's product before it is scaled (NQ = 2: S of
    // this tile was issued behind it)
    if (NQ == 1 && !__all_sync(0xffffffffu, mbar_wait(pv_done, parity, abort_flag))) return false;
    fence_after();
#pragma unroll 1
    for (int c = 0; c < D; c += 32) {
      float o[32];
      tmem_ld32(a.tO + c, o);
#pragma unroll
      for (int j = 0; j < 32; ++j) o[j] *= f;
      tmem_st32(a.tO + c, o);
    }
    l *= f;
  }
  if (grow) m = mt;
  const float mref = m == -INFINITY ? 0.f : m;
  const uint64_t k2 = f2pack(a.sl2, a.sl2), c2 = f2pack(-mref, -mref);
  uint64_t sum0 = f2pack(0.f, 0.f), sum1 = sum0;
  auto probs = [&](int c) {  // 32 keys
    uint32_t pk[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      uint64_t e2;
      asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(e2) : "l"(f2pack(s[c + 2 * j], s[c + 2 * j + 1])), "l"(k2), "l"(c2));
      const float2 e = f2unpack(e2);
      const float p0 = ex2(e.x), p1 = ex2(e.y);
      if (j & 1) asm("add.rn.f32x2 %0, %0, %1;" : "+l"(sum1) : "l"(f2pack(p0, p1)));
      else asm("add.rn.f32x2 %0, %0, %1;" : "+l"(sum0) : "l"(f2pack(p0, p1)));
      const __nv_bfloat162 b2 = __floats2bfloat162_rn(p0, p1);
      pk[j] = *reinterpret_cast<const uint32_t*>(&b2);
    }
    tmem_st16u(a.tS + c / 2, pk);
  };
  probs(0);
  probs(32);
  probs(64);
  probs(96);
  const float2 s0 = f2unpack(sum0), s1 = f2unpack(sum1);
  l += (s0.x + s0.y) + (s1.x + s1.y);
  return true;
}
// (NQ = 1 does not inline it: 64 single tokens over 1k to 16k 237 -> 231 us with
// pages of 16, over 4096 178 -> 180 with pages of 64)
template <int D>
__device__ __noinline__ bool softmax_tile_call(const TileArgs a, float& m, float& l, uint64_t* pv_done, uint32_t parity,
                                               volatile int* abort_flag) {
  return softmax_tile<D, 1>(a, m, l, pv_done, parity, abort_flag);
}

// The same over an 8-bit cache (NQ = 2): scores of the codes times the key's scale, P in fp16 as p (vs / u) 2^7.  u is
// the row's own: the largest p vs of the keys that it sees was between u and 2^8 u when the row met it, so P <= 2^15,
// and neither a scale that the row does not see nor one with next to no probability takes bits from the others.  The
// tile's largest scale bounds p vs; only where that is above 2^8 u are the 16 keys' own looked at.  The scales
// come for 16 keys at a time and cost next to nothing: K's goes into the factor of its keys' scores (their maximum is
// taken before, the scale is positive), V's as a logarithm into the exponent, and l takes the sum of each 16 P's by
// the inverse of their weight.  (Two multiplications for each pair of keys, in a form of their own for tiles of
// several scales: 979 us where tiles of one scale took 793, 4 x 2048 rows over 8000.)  lu: log2 u, from m.  A weight
// below 2^-64 is taken as that: P is 0 in fp16 either way, and l does not lose the keys.
// a.sl2: scale log2(e) 2^-e of the row.
constexpr float kUnitLog8 = 7.f, kNoUnit = -1000.f;
template <int D>
__device__ __forceinline__ void softmax_tile8(const TileArgs& a, const TileScales& ts, float& m, float& l, float& lu) {
  float s[128];
  fence_after();
  tmem_ld128(a.tS, s);
  if (a.masked_hi) {
#pragma unroll
    for (int c = 0; c < 128; c += 32) {
      const int n = min(max(a.hi - c, 0), 32);
      const uint32_t keep = n == 32 ? 0xffffffffu : (1u << n) - 1u;
#pragma unroll
      for (int j = 0; j < 32; ++j) s[c + j] = (keep >> j) & 1u ? s[c + j] : -INFINITY;
    }
  }
  if (a.masked_lo) {
#pragma unroll
    for (int j = 0; j < 128; ++j) s[j] = j >= a.lo ? s[j] : -INFINITY;
  }
  // (never 0 nor infinite: a hidden key's -inf stays one, and a score of 0 is 0)
  float kq[KT / 16];
#pragma unroll
  for (int q = 0; q < KT / 16; ++q) kq[q] = fminf(fmaxf(a.sl2 * ts.key[q].x, 1.17549435e-38f), 3.4e38f);
  float mt = -INFINITY, top[KT / 16];
#pragma unroll
  for (int q = 0; q < KT / 16; ++q) {
    const float* v = s + 16 * q;
    float m0 = max3(v[0], v[1], v[2]), m1 = max3(v[3], v[4], v[5]);
    m0 = max3(m0, v[6], v[7]);
    m1 = max3(m1, v[8], v[9]);
    m0 = max3(m0, v[10], v[11]);
    m1 = max3(m1, v[12], v[13]);
    m0 = max3(m0, v[14], v[15]);
    top[q] = fmaxf(m0, m1) * kq[q];
    mt = fmaxf(mt, top[q]);
  }
  // (NaN, which is no growth, where both are -inf)
  if (__any_sync(0xffffffffu, a.valid && mt - m + fmaxf(ts.most - lu, 0.f) > 8.f)) {
    const bool grow = a.valid && mt > m + 8.f, first = m == -INFINITY;
    const float mn = grow ? mt : m, base = mn == -INFINITY ? 0.f : mn, shift = grow && !first ? m - mn : 0.f;
    float pv = -INFINITY;  // log2 of the largest p vs
#pragma unroll
    for (int q = 0; q < KT / 16; ++q) pv = fmaxf(pv, top[q] - base + ts.key[q].y);
    const float was = lu + shift;  // the unit so far, from the new maximum: O stays what it is where that will do
    const bool move = a.valid && pv > was + 8.f;
    lu = move ? pv : was;
    if (__any_sync(0xffffffffu, move && !first)) {
      const float f = move && !first ? ex2(was - lu) : 1.f;
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        float o[32];
        tmem_ld32(a.tO + c, o);
#pragma unroll
        for (int j = 0; j < 32; ++j) o[j] *= f;
        tmem_st32(a.tO + c, o);
      }
    }
    l *= ex2(shift);
    m = mn;
  }
  const float mref = m == -INFINITY ? 0.f : m;
#pragma unroll
  for (int c = 0; c < 128; c += 32) {
    uint32_t pk[16];
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const float k = kq[c / 16 + g], w = kUnitLog8 + fmaxf(ts.key[c / 16 + g].y - lu, -64.f);
      const uint64_t k2 = f2pack(k, k), c2 = f2pack(w - mref, w - mref);
      uint64_t sum = f2pack(0.f, 0.f);
#pragma unroll
      for (int j = 8 * g; j < 8 * g + 8; ++j) {
        uint64_t e2;
        asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(e2) : "l"(f2pack(s[c + 2 * j], s[c + 2 * j + 1])), "l"(k2), "l"(c2));
        const float2 e = f2unpack(e2), p = make_float2(ex2(e.x), ex2(e.y));
        asm("add.rn.f32x2 %0, %0, %1;" : "+l"(sum) : "l"(f2pack(p.x, p.y)));
        const __half2 h2 = __floats2half2_rn(p.x, p.y);
        pk[j] = *reinterpret_cast<const uint32_t*>(&h2);
      }
      const float2 both = f2unpack(sum);
      l = fmaf(both.x + both.y, ex2(-w), l);
    }
    tmem_st16u(a.tS + c / 2, pk);
  }
}

// A NaN among V's codes that the converters put to 0, given to the rows that see it (as
// add_nonfinite does).
template <int D>
__device__ __noinline__ void add_nan8(Ragged r, Kv8View kv, const Work& w, uint32_t tO, int i, int window, int causal) {
  const int pos = w.len - w.n + i, lo = vis_lo(pos, window), hi = vis_hi(pos, w.len, causal);
  const int lane = threadIdx.x & 31, T = max(w.nt[0], w.nt[1]);
  for (int t = 0; t < T; ++t) {
    const int kt = (w.t0 + t) * KT, in = min(KT, w.len - kt);
    if (kt >= w.clean_lo && kt + KT <= w.clean_hi) {  // what the converters left alone; and so are all up to the edge
      t = max(t, w.clean_hi / KT - 1 - w.t0);
      continue;
    }
    for (int base = kt; base < kt + in; base += 32) {
      const int j = base + lane;
      const uint32_t* v = nullptr;
      uint32_t found = 0;
      if (j < kt + in) {
        const int pg = r.table[(int64_t)w.b * r.table_stride + (j >> kv.page_shift)];
        if (pg >= 0 && pg < kv.n_pages) {
          v = reinterpret_cast<const uint32_t*>(kv.v + pg * kv.page + (j & ((1 << kv.page_shift) - 1)) * kv.slot + w.kvh * kv.head);
          for (int c = 0; c < D / 4; ++c) found |= nan_codes(v[c]);
        }
      }
      uint32_t todo = __ballot_sync(0xffffffffu, found != 0);
      while (todo) {
        const int src = __ffs(todo) - 1;
        todo &= todo - 1;
        const uint32_t* e = reinterpret_cast<const uint32_t*>(__shfl_sync(0xffffffffu, (unsigned long long)v, src));
        const bool see = base + src >= lo && base + src < hi;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          float o[32];
          tmem_ld32(tO + c, o);
#pragma unroll
          for (int k = 0; k < 32; ++k)
            if (see && (nan_codes(e[(c + k) / 4]) >> (8 * (k % 4) + 7)) & 1u) o[k] = __uint_as_float(0x7fffffffu);
          tmem_st32(tO + c, o);
        }
      }
    }
  }
}

// Sixteen codes as fp16, the first eight and the others.
__device__ __forceinline__ void codes_to_h16(const uint4& c, uint4& lo, uint4& hi) {
  e4m3x4_to_h4(c.x, lo.x, lo.y);
  e4m3x4_to_h4(c.y, lo.z, lo.w);
  e4m3x4_to_h4(c.z, hi.x, hi.y);
  e4m3x4_to_h4(c.w, hi.z, hi.w);
}

// A row of a Q tile (128 bytes of it in each of D / 64 blocks `block` bytes apart, its 16-byte chunks
// swizzled by row mod 8), bf16 to fp16 in place, times 2^e so that its largest finite element lies in
// [2^14, 2^15): fp16 then holds all of bf16's bits down to 2^-29 of that.  Returns e.
template <int D>
__device__ __forceinline__ int q_to_h16(uint8_t* row, int block, int swizzle) {
  auto chunk = [&](int c) { return reinterpret_cast<uint4*>(row + c / 8 * block + (((c & 7) ^ swizzle) << 4)); };
  uint32_t most2 = 0;  // largest magnitudes: finite bf16 order as integers do
#pragma unroll 4
  for (int c = 0; c < D / 8; ++c) {
    const uint4 u = *chunk(c);
    const uint32_t v[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t a = v[k] & 0x7fff7fffu;
      most2 = __vmaxu2(most2, a & ~((nonfinite_bits(a) >> 15) * 0xffffu));
    }
  }
  const uint32_t most = max(most2 & 0xffffu, most2 >> 16);
  const int e = most ? 14 - ilogbf(__uint_as_float(most << 16)) : 0, e0 = e / 2;
  const float f0 = ldexpf(1.f, e0), f1 = ldexpf(1.f, e - e0);  // two factors, either of them a normal number
#pragma unroll 4
  for (int c = 0; c < D / 8; ++c) {
    uint4* at = chunk(c);
    const uint4 u = *at;
    uint32_t v[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const __half2 h = __floats2half2_rn(__uint_as_float(v[k] << 16) * f0 * f1, __uint_as_float(v[k] & 0xffff0000u) * f0 * f1);
      v[k] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *at = make_uint4(v[0], v[1], v[2], v[3]);
  }
  return e;
}

// A row of a Q tile as above into two e4m3 pieces q1 + q2 (each a tile of its own, one in each 64-element
// block's place): 2^e q with its largest finite element in [2^7, 2^8), q1 its nearest code, q2 the code of what
// is left.  A code has 4 significant bits and a bf16 number 8, so the sum is exact for elements down to
// 2^-9 of the largest; smaller ones are off by at most 2^-17 of that (half a step of 2^-9, the largest being 2^7 or more).  Not finite: NaN.  Returns e.
template <int D>
__device__ __forceinline__ int q_to_e4m3(uint8_t* row, int block, int swizzle) {
  static_assert(D == 128, "a piece is a row of 128 bytes");
  uint4 u[D / 8];
  uint32_t most2 = 0;
#pragma unroll
  for (int c = 0; c < D / 8; ++c) {
    u[c] = *reinterpret_cast<const uint4*>(row + c / 8 * block + (((c & 7) ^ swizzle) << 4));
    const uint32_t v[4] = {u[c].x, u[c].y, u[c].z, u[c].w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t a = v[k] & 0x7fff7fffu;
      most2 = __vmaxu2(most2, a & ~((nonfinite_bits(a) >> 15) * 0xffffu));
    }
  }
  const uint32_t most = max(most2 & 0xffffu, most2 >> 16);
  const int e = most ? 7 - ilogbf(__uint_as_float(most << 16)) : 0, e0 = e / 2;
  const float f0 = ldexpf(1.f, e0), f1 = ldexpf(1.f, e - e0);
#pragma unroll
  for (int c = 0; c < D / 16; ++c) {  // 16 elements: a chunk of each piece
    uint32_t p1[4], p2[4];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint4 w4 = u[2 * c + k / 4];
      const uint32_t w = k % 4 == 0 ? w4.x : k % 4 == 1 ? w4.y : k % 4 == 2 ? w4.z : w4.w;
      float x = __uint_as_float(w << 16) * f0 * f1, y = __uint_as_float(w & 0xffff0000u) * f0 * f1;
      // (a conversion saturates: infinities by hand)
      x = nonfinite(x) ? __uint_as_float(0x7fffffffu) : x;
      y = nonfinite(y) ? __uint_as_float(0x7fffffffu) : y;
      const uint32_t c1 = f2_to_e4m3x2(x, y);
      uint32_t lo, hi;
      e4m3x4_to_h4(c1, lo, hi);
      const float2 r = __half22float2(*reinterpret_cast<const __half2*>(&lo));
      const uint32_t c2 = f2_to_e4m3x2(x - r.x, y - r.y);
      if (k & 1) {
        p1[k / 2] |= c1 << 16;
        p2[k / 2] |= c2 << 16;
      } else {
        p1[k / 2] = c1;
        p2[k / 2] = c2;
      }
    }
    const int at = (c ^ swizzle) << 4;
    *reinterpret_cast<uint4*>(row + at) = make_uint4(p1[0], p1[1], p1[2], p1[3]);
    *reinterpret_cast<uint4*>(row + block + at) = make_uint4(p2[0], p2[1], p2[2], p2[3]);
  }
  return e;
}

template <int D, int NQ, bool KV8>
__global__ void __launch_bounds__(Cfg<D, NQ, KV8>::THREADS, 1)
    k_ragged_tc(Ragged r, AttnCall a, typename std::conditional<KV8, Kv8View, KVView>::type kv, Plan p, const __grid_constant__ CUtensorMap mq,
                const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv) {
  using C = Cfg<D, NQ, KV8>;
  static_assert(!KV8 || (NQ == 2 && C::RING / 2 + 2 <= C::NSCALES), "8-bit tiles: two row tiles, scales of what is in flight");
  constexpr int SLOT = C::SLOT, RING = C::RING, NB = D / 64;
  constexpr int SW = 4 * NQ;  // the first warp behind the softmax
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sQ = smem;
  uint8_t* sR = sQ + 2 * SLOT;
  uint8_t* sS = sR + C::RING_BYTES;
  uint64_t* full = (uint64_t*)(sS + C::STAGE + C::CODES);
  uint64_t* empty = full + RING;
  uint64_t* v_fix = empty + RING;
  uint64_t* q_full = v_fix + RING;
  uint64_t* q_empty = q_full + 2;
  uint64_t* s_full = q_empty + 2;
  uint64_t* p_full = s_full + 2;
  uint64_t* pv_done = p_full + 2;
  uint64_t* w_full = pv_done + 2;
  uint64_t* w_empty = w_full + NW;
  uint64_t* all_done = w_empty + NW;
  uint32_t* tmem_slot = (uint32_t*)(all_done + 1);
  volatile int* abort_flag = (volatile int*)(tmem_slot + 1);
  Work* works = (Work*)(tmem_slot + 2);
  // 8 bits: scales of the last tiles, the tiles of codes, and (in place of what the fixer
  // signals) Q as fp16
  uint8_t* sC = sS + C::STAGE;
  TileScales* tscales = (TileScales*)(sC + C::CODES + C::EXTRA);
  uint64_t* c_full = (uint64_t*)(tscales + C::NSCALES);
  uint64_t* c_empty = c_full + C::NC;
  uint64_t* q_ready = v_fix;
  static_assert((3 * 12 + 10 + 2 * NW + 1) * 8 + 8 + NW * sizeof(Work) <= 768, "barriers and descriptors");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = a.Hq / a.Hkv;
  // entry i of the ring (K tiles even, V tiles odd): its slot, how often that was used before, where it lies
  constexpr bool K8 = C::K8;
  auto r_slot = [](uint32_t i) { return K8 ? (i & 1u) * 2u + ((i >> 1) & 1u) : i % RING; };
  auto r_use = [](uint32_t i) { return i / RING; };
  auto r_addr = [&](uint32_t slot) {
    if (K8) return sR + (slot < 2u ? slot * (KT * D) : 2u * (KT * D) + (slot - 2u) * SLOT);
    return sR + slot * SLOT;
  };

  if (tid == 0) {
    for (int s = 0; s < RING; ++s) {
      mbar_init(&full[s], KV8 ? 2 : 1);
      mbar_init(&empty[s], KV8 ? 1 : 2);  // the MMAs (seen by a softmax warp, or a commit) and the fixer
      mbar_init(&v_fix[s], KV8 ? 4 : 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&q_full[s], 1);
      mbar_init(&q_empty[s], NQ == 2 ? 1 : 4);
      mbar_init(&s_full[s], 1);
      mbar_init(&p_full[s], 4);
      mbar_init(&pv_done[s], 1);
    }
    for (int s = 0; KV8 && s < C::NC; ++s) {
      mbar_init(&c_full[s], 1);
      mbar_init(&c_empty[s], 2);
    }
    for (int s = 0; s < NW; ++s) {
      mbar_init(&w_full[s], 1);
      mbar_init(&w_empty[s], SW + 3);  // all warps but the scheduler
    }
    mbar_init(all_done, 1);
    *abort_flag = 0;
    mbar_fence_init();
  }
  if (warp == SW + 1) {
    tmem_alloc(tmem_slot, 512);
    fence_before();
  }
  if (warp == SW && lane < 3) {
    const CUtensorMap* m = lane == 0 ? &mq : lane == 1 ? &mk : &mv;
    asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)m) : "memory");
  }
  __syncthreads();
  fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_trigger();
  pdl_wait();

  auto give_up = [&]() {
    if (lane == 0) flag_status(r.status, DFLASH_STATUS_WAIT);
    *abort_flag = 1;
  };

  if (warp >= SW) {
  if constexpr (NQ == 2) regs_dec<C::R_REST>();
  if (KV8 && (warp == SW || warp == SW + 2)) {
    if constexpr (KV8) {
      // ---- converters: tiles of codes, which come by TMA, as fp16 into the ring.  A thread has 16 codes
      // of each of N keys.
      constexpr int PIECES = D / 16, KEYS = 64 / PIECES, N = KT / KEYS, H = 2;  // H pieces at a time (more code is fetched anew more often)
      const int cw = warp == SW ? 0 : 1, ct = cw * 32 + lane, piece = ct % PIECES, key = ct / PIECES;
      r.table = after_wait(r.table);
      uint32_t it = 0, c_it = 0;  // tiles of the ring, of codes
      bool ok = true;
      // where the piece's two 16-byte chunks lie in a tile, less the key's row (keys of a thread agree mod 8).
      // D = 128: lanes of the second block store their chunks in turn, so that no two of a phase meet in a bank.
      const bool swap = D == 128 && piece >= 4;
      const int block = piece / 4 * (SLOT / NB), c0 = 2 * (piece % 4) + swap, c1 = 2 * (piece % 4) + !swap;
      const int at0 = block + ((c0 ^ (key & 7)) << 4), at1 = block + ((c1 ^ (key & 7)) << 4);
      for (int k = 0; ok; ++k) {
        const int ws = k % NW;
        if (!__all_sync(0xffffffffu, mbar_wait(&w_full[ws], (uint32_t)(k / NW) & 1u, abort_flag))) {
          ok = false;
          break;
        }
        Work& w = works[ws];
        const int T = max(w.nt[0], w.nt[1]);
        if (w.done) break;
        const int len = w.len, lo_out = vis_lo(w.len - w.n + w.i0, a.window);
        const int32_t* tab = r.table + (int64_t)w.b * r.table_stride;
        const int64_t s_at = w.kvh * kv.s_head;
        const int tile0 = w.t0;
        // the scales of 16 keys of a tile, a lane each (lanes 0 .. 7).  Their loads depend on one
        // another and would hold the warp up, so the table is read two tiles ahead and the scales one.
        auto entry_of = [&](int t) {
          const int first = (tile0 + t) * KT + 16 * lane;
          return lane < KT / 16 && t < T && first < len ? tab[first >> kv.page_shift] : -1;
        };
        float ks = 1.f, vs = 0.f;
        auto look_up = [&](int t, int entry) {
          ks = 1.f;
          vs = 0.f;
          const int first = (tile0 + t) * KT + 16 * lane;
          if (lane < KT / 16 && t < T && first < len) {
            if (entry >= 0 && entry < kv.n_pages && first + 16 > lo_out) {
              ks = kv.ks[entry * kv.s_page + s_at];
              vs = kv.vs[entry * kv.s_page + s_at];
            }
          }
        };
        int ahead = -1;
        if (T > 0) {
          const int first = entry_of(0);
          ahead = entry_of(1);
          look_up(0, first);
        }
        auto wait_empty = [&](uint32_t e) {
          return r_use(e) == 0 || __all_sync(0xffffffffu, mbar_wait(&empty[r_slot(e)], (r_use(e) - 1) & 1u, abort_flag));
        };
        // The scales of tile t, for whoever sees its S: written when the K tile's entry is free, and told with
        // the tile (K8: as one of the two arrivals that it takes, the copy's being the other)
        auto put_scales = [&](int t) {
          TileScales& ts = tscales[((it >> 1) + t) % C::NSCALES];
          const float lv = scale_log2(vs), most = warp_max(lane < KT / 16 ? lv : kNoScaleLog2);
          if (lane < KT / 16) ts.key[lane] = make_float2(ks, lv);
          if (lane == 0) ts.most = most;
          look_up(t + 1, ahead);
          ahead = entry_of(t + 2);
          if (K8) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&full[r_slot(it + 2 * t)]);
          }
        };
        if (K8 && T > 0 && cw == 0) {
          if (!wait_empty(it)) {
            ok = false;
            break;
          }
          put_scales(0);
        }
        // K and V tiles in turn by the same few instructions (unrolled over both they were fetched anew each time)
#pragma unroll 1
        for (int u = K8 ? 1 : 0; u < 2 * T; u += K8 ? 2 : 1) {
          const int t = u >> 1, v = u & 1, kt = (tile0 + t) * KT;
          const uint32_t e = it + u, cs = c_it % C::NC;
          if (K8 && cw == 0 && t + 1 < T) {
            if (!wait_empty(e + 1)) {
              ok = false;
              break;
            }
            put_scales(t + 1);
          }
          // the ring's entry is free, and the codes are there
          if (!wait_empty(e) || !__all_sync(0xffffffffu, mbar_wait(&c_full[cs], c_it / C::NC & 1u, abort_flag))) {
            ok = false;
            break;
          }
          uint8_t* tile = r_addr(r_slot(e));
          ++c_it;
          if (v == 0 && cw == 0) put_scales(t);
          // keys that a row does not see (slots behind the sequence hold anything): 0 x NaN is NaN, such codes of V
          // become 0 here and are given to the rows that see them at the stretch's end (only for row tiles
          // that take this product)
          const bool edge = v && (kt < w.clean_lo || kt + KT > w.clean_hi);
#pragma unroll 1
          for (int i0 = 0; i0 < N; i0 += H) {
            uint4 q[H];
#pragma unroll
            for (int i = 0; i < H; ++i) q[i] = *reinterpret_cast<const uint4*>(sC + cs * (KT * D) + ((i0 + i) * 64 + ct) * 16);
            if (edge) {
              uint32_t found = 0;
#pragma unroll
              for (int i = 0; i < H; ++i) found |= nan_codes(q[i].x) | nan_codes(q[i].y) | nan_codes(q[i].z) | nan_codes(q[i].w);
              if (found) {
#pragma unroll
                for (int i = 0; i < H; ++i)
                  q[i] = make_uint4(without_nan(q[i].x), without_nan(q[i].y), without_nan(q[i].z), without_nan(q[i].w));
                atomicOr(&w.bad, (t < w.nt[0] ? 1 : 0) | (t < w.nt[1] ? 2 : 0));
              }
            }
            uint8_t* rows = tile + (key + KEYS * i0) * 128;
#pragma unroll
            for (int i = 0; i < H; ++i) {
              uint4 lo, hi;
              codes_to_h16(q[i], lo, hi);
              *reinterpret_cast<uint4*>(rows + KEYS * 128 * i + at0) = swap ? hi : lo;
              *reinterpret_cast<uint4*>(rows + KEYS * 128 * i + at1) = swap ? lo : hi;
            }
          }
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&c_empty[cs]);
            mbar_arrive(&full[r_slot(e)]);
          }
        }
        it += 2 * T;
        __syncwarp();
        if (lane == 0) mbar_arrive(&w_empty[ws]);
      }
      if (!ok) give_up();
    }
  } else if (warp == SW + 3) {
    // ---- scheduler
    r.starts = after_wait(r.starts);
    if (r.lens) r.lens = after_wait(r.lens);
    if (KV8) r.table = after_wait(r.table);
    int k = 0;
    bool ok = true;
    // 8 bits: this warp asks for the tiles too, Q and then K and V in turn (a copy per lane, the box of a page)
    uint32_t q_use[2] = {0, 0}, c_it = 0, k_it = 0;  // (k_it: K8, the ring's entry of the next K tile)
    Work last;
    auto produce = [&](const Work& w) {
      if constexpr (KV8) {
        const int page_rows = min(1 << kv.page_shift, KT), boxes = KT / page_rows, box = lane & (boxes - 1);
        const bool issuer = lane < boxes;
        const int32_t* tab = r.table + (int64_t)w.b * r.table_stride;
        const int T = max(w.nt[0], w.nt[1]), lo_out = vis_lo(w.len - w.n + w.i0, a.window);
        auto page_of = [&](int t) {
          const int pos = (w.t0 + t) * KT + box * page_rows;
          return t < T && issuer && pos < w.len ? tab[pos >> kv.page_shift] : -1;
        };
        int pg = page_of(0);
        for (int t = 0; t < T && ok; ++t) {
          const int kt = (w.t0 + t) * KT, pos = kt + box * page_rows, next = page_of(t + 1);
          const bool mine = issuer && pos < w.len;
          if (mine && (pg < 0 || pg >= kv.n_pages)) {
            // (a page that the window of every row has left behind may be gone)
            flag_status(pos + page_rows > lo_out ? r.status : nullptr, DFLASH_STATUS_PAGE);
            pg = kv.n_pages;  // just outside the map: zeros arrive
          }
          const uint32_t bytes = (uint32_t)__popc(__ballot_sync(0xffffffffu, mine)) * page_rows * D;
          for (int v = 0; v < 2; ++v) {
            const bool direct = K8 && v == 0;  // into the ring
            const uint32_t cs = c_it % C::NC, use = direct ? r_use(k_it) : c_it / C::NC;
            uint64_t *const there = direct ? &full[r_slot(k_it)] : &c_full[cs], *const free_ = direct ? &empty[r_slot(k_it)] : &c_empty[cs];
            if (use > 0 && !__all_sync(0xffffffffu, mbar_wait(free_, (use - 1) & 1u, abort_flag))) {
              ok = false;
              return;
            }
            uint8_t* const to = direct ? r_addr(r_slot(k_it)) : sC + cs * (KT * D);
            if (direct) k_it += 2;
            else ++c_it;
            if (lane == 0) mbar_expect_tx(there, bytes);
            __syncwarp();
            if (mine)
              tma_load_4d(to + box * page_rows * D, v ? &mv : &mk, there, 0, kt & ((1 << kv.page_shift) - 1), w.kvh, pg);
            if (t == 0 && v == 0) {
              for (int x = 0; x < 2; ++x) {
                if (w.nt[x] == 0) continue;
                if (q_use[x] > 0 && !__all_sync(0xffffffffu, mbar_wait(&q_empty[x], (q_use[x] - 1) & 1u, abort_flag))) {
                  ok = false;
                  return;
                }
                if (lane == 0) {
                  mbar_expect_tx(&q_full[x], (uint32_t)(G * p.tpt * 128 * NB));
                  for (int c = 0; c < NB; ++c)
                    tma_load_3d(sQ + x * SLOT + c * (SLOT / NB), &mq, &q_full[x], 64 * c, w.kvh * G, w.start + w.i0 + x * p.tpt);
                }
                ++q_use[x];
              }
            }
          }
          pg = next;
        }
      }
    };
    auto emit = [&](const Work& w) {
      const int s = k % NW;
      if (k >= NW && !__all_sync(0xffffffffu, mbar_wait(&w_empty[s], (uint32_t)(k / NW - 1) & 1u, abort_flag))) {
        ok = false;
        return;
      }
      if (lane == 0) {
        works[s] = w;
        mbar_arrive(&w_full[s]);
      }
      __syncwarp();
      ++k;
      if constexpr (KV8) {
        // the tiles of the stretch before: its successor is known by then, nobody waits for the search
        if (k > 1) produce(last);
        last = w;
      }
    };
    const int cta = blockIdx.x, grid = gridDim.x;
    const bool one = r.batch <= 32;  // then each lane keeps its sequence
    Seq mine{0, 0, 0, false};
    if (one && lane < r.batch) mine = load_seq(r, lane);
    auto seq_at = [&](int b) { return one ? mine : load_seq(r, b); };  // b = base + lane
    auto bcast = [&](const Seq& s, int src) {
      Seq o;
      o.start = __shfl_sync(0xffffffffu, s.start, src);
      o.n = __shfl_sync(0xffffffffu, s.n, src);
      o.len = __shfl_sync(0xffffffffu, s.len, src);
      o.ok = __shfl_sync(0xffffffffu, (int)s.ok, src) != 0;
      return o;
    };
    Work w;
    if (NQ == 1 && p.mode == kModeCluster) {
      // one item per sequence and KV head (its rows fit one tile); rank q of the
      // cluster takes an even share of its key tiles
      const int item = cta / p.cluster, q = cta - item * p.cluster, b = item / a.Hkv;
      const Seq s = load_seq(r, b);
      if (!s.ok && lane == 0 && item == b * a.Hkv && q == 0) flag_status(r.status, DFLASH_STATUS_BOUNDS);
      if (s.ok && s.n > 0) {
        const int T = tile_count(s, a.window), t = T * q / p.cluster;
        make_work(w, s, b, item - b * a.Hkv, 0, tile_first(s, a.window) + t, T * (q + 1) / p.cluster - t, 0, p, a);
        emit(w);
      }
    } else if (p.mode == kModeItems) {
      // items whose keys reach tile c: counted over the batch
      auto count = [&](int c) {
        int64_t s = 0;
        for (int b = lane; b < r.batch; b += 32) s += items_reaching(seq_at(b), c, p, a.causal);
        return sum_up_to(s, p.max_items);
      };
      int max_t = 0;
      for (int b = lane; b < r.batch; b += 32) {
        const Seq s = seq_at(b);
        if (!s.ok && cta == 0) flag_status(r.status, DFLASH_STATUS_BOUNDS);
        if (s.ok && s.n > 0) max_t = max(max_t, cdiv(s.len, KT));
      }
      max_t = __reduce_max_sync(0xffffffffu, max_t);
      const int found = count(1), pairs = max(found, 0), total = pairs * a.Hkv, per_group = pairs * p.hgroup;
      if (found < 0 && cta == 0) flag_status(r.status, DFLASH_STATUS_BOUNDS);
      for (int j = 0; ok && j < total; j += grid) {
        const int idx = j + (((j / grid) & 1) ? grid - 1 - cta : cta);
        if (idx >= total) continue;
        const int g = idx / per_group, heads = min(p.hgroup, a.Hkv - g * p.hgroup);
        const int rest = idx - g * per_group, pair = rest / heads;
        const int kvh = g * p.hgroup + rest - pair * heads;
        int c = 1, hi = max_t + 1;
        while (hi - c > 1) {
          const int mid = (c + hi) >> 1;
          if (count(mid) > pair) c = mid;
          else hi = mid;
        }
        int rank = pair - (c < max_t ? count(c + 1) : 0);
        for (int base = 0; base < r.batch; base += 32) {
          const int b = base + lane;
          int here = 0, first = 0;
          Seq s{0, 0, 0, false};
          if (b < r.batch) {
            s = seq_at(b);
            const int ge = items_reaching(s, c, p, a.causal);
            here = ge - items_reaching(s, c + 1, p, a.causal);
            first = items_of(s, p) - ge;
          }
          const int incl = warp_scan_i(here, lane), sum = __shfl_sync(0xffffffffu, incl, 31);
          if (rank < sum) {
            const int src = __ffs(__ballot_sync(0xffffffffu, incl > rank)) - 1;
            const int qi = __shfl_sync(0xffffffffu, first - (incl - here), src) + rank;
            make_work(w, bcast(s, src), base + src, kvh, qi, 0, INT32_MAX / 2, -1, p, a);
            emit(w);
            break;
          }
          rank -= sum;
        }
      }
    } else {
      int64_t sum = 0;
      for (int b = lane; b < r.batch; b += 32) {
        const Seq s = seq_at(b);
        if (!s.ok && cta == 0) flag_status(r.status, DFLASH_STATUS_BOUNDS);
        sum += units_of(s, p, a);
      }
      int units = sum_up_to(sum, p.max_units);
      if (units < 0) {
        if (cta == 0) flag_status(r.status, DFLASH_STATUS_BOUNDS);
        units = 0;
      }
      const Ranges rg(units, p, grid);
      int u = cta < rg.n ? rg.start(cta) : units;
      const int u1 = cta < rg.n ? rg.start(cta + 1) : units;
      int before = 0;  // units in front of the 32 sequences at `base`
      int seg = 0;
      for (int base = 0; base < r.batch && u < u1 && ok; base += 32) {
        const int b = base + lane;
        Seq s{0, 0, 0, false};
        if (b < r.batch) s = seq_at(b);
        const int mine_u = (int)units_of(s, p, a), incl = warp_scan_i(mine_u, lane);
        const int chunk_end = before + __shfl_sync(0xffffffffu, incl, 31);
        while (u < u1 && u < chunk_end && ok) {
          const int src = __ffs(__ballot_sync(0xffffffffu, before + incl > u)) - 1;
          const Seq q = bcast(s, src);
          const int off = u - (before + __shfl_sync(0xffffffffu, incl - mine_u, src));
          const int T = tile_count(q, a.window), item = off / (T + p.pad), qi = item / a.Hkv;
          const int t = off - item * (T + p.pad) - p.pad;  // < 0: in front of the item's tiles
          const int take = min(T, t + u1 - u) - max(t, 0);
          u += min(T - t, u1 - u);
          if (take <= 0) continue;
          const int part = take == T ? -1 : 2 * cta + (seg > 0);
          make_work(w, q, base + src, item - qi * a.Hkv, qi, tile_first(q, a.window) + max(t, 0), take, part, p, a);
          emit(w);
          ++seg;
        }
        before = chunk_end;
      }
    }
    w.done = 1;
    if (ok) emit(w);
    if (!ok) give_up();
    if (KV8 && (!ok || *abort_flag)) {
      // let this CTA's own copies land before leaving
      const uint64_t t0 = globaltimer_ns();
      for (int x = 0; x < 2; ++x) {
        while (q_use[x] > 0 && !mbar_try_wait(&q_full[x], (q_use[x] - 1) & 1u) && globaltimer_ns() - t0 < kWaitLimitNs) {
        }
      }
      for (uint32_t i = c_it > C::NC ? c_it - C::NC : 0; i < c_it; ++i) {
        while (!mbar_try_wait(&c_full[i % C::NC], i / C::NC & 1u) && globaltimer_ns() - t0 < kWaitLimitNs) {
        }
      }
      for (uint32_t i = k_it > 4 ? k_it - 4 : 0; i < k_it; i += 2) {  // (K8: the arrival of its scales may be missing)
        while (!mbar_try_wait(&full[r_slot(i)], r_use(i) & 1u) && globaltimer_ns() - t0 < kWaitLimitNs) {
        }
      }
    }
  } else if (!KV8 && warp == SW) {
    if constexpr (!KV8) {
    // ---- TMA producer: Q tiles, then K and V tiles in turn through one ring
    if (r.table) r.table = after_wait(r.table);
    uint32_t it = 0, q_use[2] = {0, 0};
    bool ok = true;
    const int page_rows = kv.paged ? min(1 << kv.page_shift, KT) : KT;
    const int boxes = KT / page_rows;
    // a copy per lane (the box of a page, one of its 128-byte halves), so that a
    // tile goes out in one instruction whatever the page size
    const int box = lane & (boxes - 1), half = lane / boxes;
    const bool issuer = half < NB;
    auto ring_wait = [&](uint32_t i) {
      return i < (uint32_t)RING ||
             __all_sync(0xffffffffu, mbar_wait(&empty[i % RING], (i / RING - 1) & 1u, abort_flag));
    };
    for (int k = 0; ok; ++k) {
      const int ws = k % NW;
      if (!__all_sync(0xffffffffu, mbar_wait_short(&w_full[ws], (uint32_t)(k / NW) & 1u, abort_flag))) {
        ok = false;
        break;
      }
      const Work w = works[ws];
      __syncwarp();
      if (lane == 0) mbar_arrive(&w_empty[ws]);
      if (w.done) break;
      const int T = max(w.nt[0], w.nt[1]);
      auto load_q = [&](int x, int buf) {
        if (q_use[buf] > 0 && !__all_sync(0xffffffffu, mbar_wait(&q_empty[buf], (q_use[buf] - 1) & 1u, abort_flag))) {
          ok = false;
          return;
        }
        if (lane == 0) {
          mbar_expect_tx(&q_full[buf], (uint32_t)(G * p.tpt * 128 * NB));
          for (int c = 0; c < NB; ++c)
            tma_load_3d(sQ + buf * SLOT + c * (SLOT / NB), &mq, &q_full[buf], 64 * c, w.kvh * G,
                        w.start + w.i0 + x * p.tpt);
        }
        ++q_use[buf];
      };
      const int32_t* tab = kv.paged ? r.table + (int64_t)w.b * r.table_stride : nullptr;
      // page of this lane's box of a tile; lanes past the sequence load nothing
      auto page_of = [&](int t) {
        const int pos = (w.t0 + t) * KT + box * page_rows;
        return kv.paged && t < T && issuer && pos < w.len ? tab[pos >> kv.page_shift] : -1;
      };
      int pg = page_of(0);  // on its way while Q is asked for
      if (NQ == 1) {
        // double-buffered: the buffers alternate over the stretches that have tiles
        if (w.nt[0] > 0) load_q(0, (int)((q_use[0] + q_use[1]) & 1u));
      } else {
        for (int x = 0; x < NQ && ok; ++x)
          if (w.nt[x] > 0) load_q(x, x);
      }
      // tiles of this lane whose page may be gone: the first, where the page lies in front of every row's
      // window (asked in the loop, single tokens over 1k to 16k took 402 us instead of 366)
      const int quiet = w.t0 * KT + (box + 1) * page_rows > vis_lo(w.len - w.n + w.i0, a.window) ? 0 : 1;
      for (int t = 0; t < T && ok; ++t) {
        const int kt = (w.t0 + t) * KT;
        const int next = page_of(t + 1);
        const bool mine = issuer && (!kv.paged || kt + box * page_rows < w.len);
        if (kv.paged && mine && (pg < 0 || pg >= kv.n_pages)) {
          flag_status(t >= quiet ? r.status : nullptr, DFLASH_STATUS_PAGE);
          pg = kv.n_pages;  // just outside the map: zeros arrive
        }
        const uint32_t bytes = (uint32_t)__popc(__ballot_sync(0xffffffffu, mine)) * page_rows * 128;
        for (int is_v = 0; is_v < 2 && ok; ++is_v, ++it) {
          const int st = it % RING;
          if (!ring_wait(it)) {
            ok = false;
            break;
          }
          if (lane == 0) mbar_expect_tx(&full[st], bytes);
          __syncwarp();
          if (mine) {
            const CUtensorMap* m = is_v ? &mv : &mk;
            uint8_t* dst = sR + st * SLOT + half * (SLOT / NB) + box * page_rows * 128;
            if (kv.paged) tma_load_4d(dst, m, &full[st], 64 * half, kt & ((1 << kv.page_shift) - 1), w.kvh, pg);
            else tma_load_4d(dst, m, &full[st], 64 * half, w.start + kt, w.kvh, 0);
          }
        }
        pg = next;
      }
    }
    if (!ok || *abort_flag) {
      // let this CTA's own copies land before leaving
      give_up();
      const uint64_t t0 = globaltimer_ns();
      for (uint32_t i = it > (uint32_t)RING ? it - RING : 0; i < it; ++i)
        while (!mbar_try_wait(&full[i % RING], (i / RING) & 1u) && globaltimer_ns() - t0 < kWaitLimitNs) {
        }
      for (int x = 0; x < 2; ++x)
        while (q_use[x] > 0 && !mbar_try_wait(&q_full[x], (q_use[x] - 1) & 1u) && globaltimer_ns() - t0 < kWaitLimitNs) {
        }
    }
    }
  } else if (warp == SW + 1) {
    // ---- MMA issuer: the whole warp decides, one elected lane issues.  The
    // tensor core takes MMAs little faster than it runs them (8 of them, one
    // product, in 512 cycles), so whatever this warp does between two products
    // is idle time, a commit 75 to 150 cycles of it (measured).  NQ = 2, which is
    // bound by this pipe, commits once per S: the softmax warps, who see it,
    // give the K/V and Q tiles back that were read in front of it.
    constexpr uint32_t idS = KV8 ? idesc_f16(128, KT) : idesc_bf16(128, KT);
    constexpr uint32_t idPV = (KV8 ? idesc_f16(128, D) : idesc_bf16(128, D)) | kIdescBMnMajor;
    uint32_t it = 0, fixpar = 0;
    uint32_t q_cnt0 = 0, q_cnt1 = 0;    // Q tiles used (NQ = 1: one count, the buffers alternate)
    uint32_t pv_cnt0 = 0, pv_cnt1 = 0;  // products P V of each stream
    uint32_t s_cnt = 0;                 // NQ = 1: S issued, the buffers alternate
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      if (ok && !__all_sync(0xffffffffu, mbar_wait(bar, parity & 1u, abort_flag))) ok = false;
      return ok;
    };
    auto ring_full = [&](uint32_t i) { return wait(&full[r_slot(i)], r_use(i)); };
    // (8 bits: the converters are one more stream of instructions in the SM, and code is fetched anew all the time; a
    // loop that is too short issues too slowly.  Chunked prefill with one, four and eight MMAs a turn: 143, 137, 140 us,
    // with both descriptors put together for each 163.)
    constexpr int MMA_UNROLL = 4;
    auto issue_s = [&](int qbuf, uint32_t st, int sbuf) {
      const uint32_t q0 = smem_u32(sQ + qbuf * SLOT), k0 = smem_u32(r_addr(st)), tS = tmem + sbuf * 128;
      if constexpr (K8) {  // both pieces of q (q_to_e4m3) times K's codes
        constexpr int N = D / 32;
        const uint32_t qd = (uint32_t)sdesc_sw128(q0), kd = (uint32_t)sdesc_sw128(k0);
        constexpr uint32_t hi = (uint32_t)(sdesc_sw128(0) >> 32);
#pragma unroll(MMA_UNROLL)
        for (int ks = 0; ks < 2 * N; ++ks)
          umma_e4m3_warp_lo(tS, qd + ks / N * (SLOT / NB / 16) + ks % N * 2, kd + ks % N * 2, hi, idS, ks > 0 ? 1u : 0u);
      } else if constexpr (KV8) {
        const uint32_t qd = (uint32_t)sdesc_sw128(q0), kd = (uint32_t)sdesc_sw128(k0);
        constexpr uint32_t hi = (uint32_t)(sdesc_sw128(0) >> 32);
#pragma unroll(MMA_UNROLL)
        for (int ks = 0; ks < D / 16; ++ks) umma_bf16_warp_lo(tS, qd + ks * 2, kd + ks * 2, hi, idS, ks > 0 ? 1u : 0u);
      } else {
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          umma_bf16_warp(tS, sdesc_sw128(q0 + (ks >> 2) * (SLOT / NB) + (ks & 3) * 32),
                         sdesc_sw128(k0 + (ks >> 2) * (SLOT / NB) + (ks & 3) * 32), idS, ks > 0 ? 1u : 0u);
        }
      }
      umma_commit_warp(&s_full[sbuf]);
    };
    auto issue_pv = [&](int x, uint32_t st, int sbuf, bool first) {
      const uint32_t v0 = smem_u32(r_addr(st)), tP = tmem + sbuf * 128, tO = tmem + O_COL + x * D;
      if constexpr (KV8) {
        const uint32_t vd = (uint32_t)sdesc_sw128_mn(v0, SLOT / NB);
        constexpr uint32_t hi = (uint32_t)(sdesc_sw128_mn(0, SLOT / NB) >> 32);
#pragma unroll(MMA_UNROLL)
        for (int ks = 0; ks < KT / 16; ++ks) umma_bf16_ts_warp_lo(tO, tP + ks * 8, vd + ks * 128, hi, idPV, first && ks == 0 ? 0u : 1u);
      } else {
#pragma unroll
        for (int ks = 0; ks < KT / 16; ++ks) {
          umma_bf16_ts_warp(tO, tP + ks * 8, sdesc_sw128_mn(v0 + ks * 2048, SLOT / NB), idPV, first && ks == 0 ? 0u : 1u);
        }
      }
    };
    int k = 0;
    // what this warp needs of a stretch
    struct Span {
      int nt0, nt1, T, t0, clean_lo, clean_hi;
    };
    // the next stretch with tiles; false at the end
    auto fetch = [&](Span& o) {
      for (;;) {
        const int ws = k % NW;
        if (!wait(&w_full[ws], (uint32_t)(k / NW))) return false;
        const Work& w = works[ws];
        o.nt0 = w.nt[0];
        o.nt1 = w.nt[1];
        o.T = max(o.nt0, o.nt1);
        o.t0 = w.t0;
        o.clean_lo = w.clean_lo;
        o.clean_hi = w.clean_hi;
        const int done = w.done;
        __syncwarp();
        if (lane == 0) mbar_arrive(&w_empty[ws]);
        ++k;
        if (done) return false;
        if (o.T > 0) return true;
      }
    };
    // V of tile t, whose ring entry is i
    auto wait_v = [&](const Span& w, int t, uint32_t i) {
      if (!ring_full(i)) return;
      const int kt = (w.t0 + t) * KT;
      if (!KV8 && (kt < w.clean_lo || kt + KT > w.clean_hi)) {  // the fixer looks at it first
        wait(&v_fix[i % RING], (fixpar >> (i % RING)) & 1u);
        fixpar ^= 1u << (i % RING);
      }
    };
    // S of a stretch's first tile: issued as soon as the tile before it in the
    // same stream lets go of the columns, ahead of the other stream's work on
    // the stretch before
    auto first_s = [&](int x, int nt, uint32_t ring) {
      if (nt == 0) return;
      if (NQ == 1) {
        if (!wait(&q_full[q_cnt0 & 1u], q_cnt0 >> 1) || !ring_full(ring)) return;
        issue_s((int)(q_cnt0 & 1u), r_slot(ring), (int)(s_cnt & 1u));
        umma_commit_warp(&empty[r_slot(ring)]);
        ++q_cnt0;
        ++s_cnt;
      } else {
        if (!wait(KV8 ? &q_ready[x] : &q_full[x], x ? q_cnt1 : q_cnt0) || !ring_full(ring)) return;
        issue_s(x, r_slot(ring), x);
        if (x) ++q_cnt1;
        else ++q_cnt0;
      }
    };
    Span w, nx;
    bool have = fetch(w);
    if (have) {
      first_s(0, w.nt0, it);
      if (NQ == 2) first_s(1, w.nt1, it);
    }
    while (have && ok) {
      bool more = false;
      for (int t = 0; t < w.T && ok; ++t) {
        const bool last = t + 1 == w.T;
        const uint32_t iv = it + 2 * t + 1, ik = it + 2 * (t + 1), sv = r_slot(iv), sk = r_slot(ik);
        if (last) more = fetch(nx);
        if (NQ == 1) {
          // S of the next tile in the stream goes ahead of this tile's product
          if (!last) {
            if (!ring_full(ik)) break;
            issue_s((int)((q_cnt0 + 1) & 1u), sk, (int)(s_cnt & 1u));  // the Q buffer in use
            umma_commit_warp(&empty[sk]);
            ++s_cnt;
          } else if (more) {
            first_s(0, nx.nt0, ik);
          }
          wait_v(w, t, iv);
          if (!wait(&p_full[pv_cnt0 & 1u], pv_cnt0 >> 1)) break;
          fence_after();
          issue_pv(0, sv, (int)(pv_cnt0 & 1u), t == 0);
          umma_commit_warp(&pv_done[0]);
          umma_commit_warp(&empty[sv]);
          ++pv_cnt0;
        } else {
          wait_v(w, t, iv);
#pragma unroll(KV8 ? 1 : 2)
          for (int x = 0; x < 2; ++x) {
            const int nt = x ? w.nt1 : w.nt0;
            uint32_t& cnt = x ? pv_cnt1 : pv_cnt0;
            if (ok && t < nt && wait(&p_full[x], cnt)) {
              ++cnt;
              fence_after();
              issue_pv(x, sv, x, t == 0);
              if (t + 1 < nt) {
                if (ring_full(ik)) issue_s(x, sk, x);
              } else {
                umma_commit_warp(&pv_done[x]);
              }
            }
            if (ok && last && more) first_s(x, x ? nx.nt1 : nx.nt0, ik);
          }
        }
      }
      it += 2 * w.T;
      w = nx;
      have = more;
    }
    if (!ok) give_up();
    umma_commit_warp(all_done);  // every product issued above has ended before TMEM is given back
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(all_done, 0) && globaltimer_ns() - t0 < kWaitLimitNs) {
    }
  } else if (!KV8 && warp == SW + 2) {
    // ---- fixer: V tiles with hidden keys
    uint32_t it = 0;
    bool ok = true;
    for (int k = 0; ok; ++k) {
      const int ws = k % NW;
      if (!__all_sync(0xffffffffu, mbar_wait(&w_full[ws], (uint32_t)(k / NW) & 1u, abort_flag))) {
        ok = false;
        break;
      }
      const Work w = works[ws];
      if (!w.done) {
        const int T = max(w.nt[0], w.nt[1]);
        // It follows the ring slot by slot, as one of the two readers a slot
        // waits for: a barrier it only looked at now and then could be more
        // than one phase away, which a parity cannot tell.
        for (uint32_t i = it; i < it + 2 * T; ++i) {
          const uint32_t st = i % RING;
          if (!__all_sync(0xffffffffu, mbar_wait(&full[st], (i / RING) & 1u, abort_flag))) {
            ok = false;
            break;
          }
          const int t = (int)(i - it) >> 1, kt = (w.t0 + t) * KT;
          if (((i - it) & 1u) == 0 || (kt >= w.clean_lo && kt + KT <= w.clean_hi)) {  // K, or nothing hidden
            if (lane == 0) mbar_arrive(&empty[st]);
            continue;
          }
          uint8_t* v = sR + st * SLOT;
          const int in = min(KT, w.len - kt);  // rows of the sequence
          // rows behind the sequence: zeros (8 lanes a row of 128 bytes)
          for (int e = in * 8 + lane; e < KT * 8; e += 32)
            for (int c = 0; c < NB; ++c)
              *reinterpret_cast<uint4*>(v + c * (SLOT / NB) + e * 16) = make_uint4(0, 0, 0, 0);
          if (kt < w.clean_lo || kt + in > w.clean_hi) {
            uint32_t found = 0;
            for (int e = lane; e < in * 8; e += 32)
              for (int c = 0; c < NB; ++c)
                found |= nonfinite_bits(*reinterpret_cast<const uint4*>(v + c * (SLOT / NB) + e * 16));
            if (__builtin_expect(__any_sync(0xffffffffu, found != 0), 0)) {
#pragma unroll 1
              for (int e = lane; e < in * 32; e += 32)
                for (int c = 0; c < NB; ++c) {
                  uint32_t* pair = reinterpret_cast<uint32_t*>(v + c * (SLOT / NB)) + e;
                  *pair = finite_or_0(*pair);
                }
              // (only for the row tiles that take this product: their warps all look
              // behind it, a tile that has ended already might see it in some)
              if (lane == 0) works[ws].bad |= (t < w.nt[0] ? 1 : 0) | (t < w.nt[1] ? 2 : 0);
            }
          }
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&v_fix[st]);
            mbar_arrive(&empty[st]);
          }
        }
        it += 2 * T;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&w_empty[ws]);
      if (w.done) break;
    }
    if (!ok) give_up();
  }
  } else {
    // ---- softmax: one thread per row
    if constexpr (NQ == 2) regs_inc<C::R_SOFTMAX>();
    const int x = warp >> 2, row = tid & 127;
    const uint32_t lrow = (uint32_t)((warp & 3) * 32) << 16, tO = tmem + lrow + O_COL + x * D;
    const float sl2 = a.scale * kLog2e;
    uint32_t cnt = 0;          // tiles of this warp's stream so far
    uint32_t it = 0;           // ring entries so far
    uint32_t q_cnt = 0, q_used = 0;  // stretches with tiles of this stream so far; the last one's number
    // cluster mode: this CTA's part, in the ring (idle by then: every tile that
    // was asked for has been read)
    float* c_o = reinterpret_cast<float*>(sR);
    float2* c_ml = reinterpret_cast<float2*>(sR + 128 * (D + 4) * 4);
    const int row_i = x * p.tpt + row / G, row_g = row % G;  // this row's token (in the item) and head (in the group)
    const bool teller = NQ == 2 && (warp & 3) == 0 && lane == 0;  // gives tiles back for its stream
    bool ok = true;
    for (int k = 0; ok; ++k) {
      const int ws = k % NW;
      if (!__all_sync(0xffffffffu, mbar_wait(&w_full[ws], (uint32_t)(k / NW) & 1u, abort_flag))) {
        ok = false;
        break;
      }
      const Work& w = works[ws];
      if (w.done) break;
      const int i = w.i0 + row_i, h = w.kvh * G + row_g;
      const bool valid = row < p.tpt * G && i < min(w.i0 + p.tok, w.n);
      const bool live = __any_sync(0xffffffffu, valid);
      int lo = 0, hi = INT32_MAX;  // padding rows ask for no mask
      if (valid) {
        const int pos = w.len - w.n + i;
        lo = vis_lo(pos, a.window);
        hi = vis_hi(pos, w.len, a.causal);
      }
      const int hi_min = __reduce_min_sync(0xffffffffu, hi);
      const int lo_max = __reduce_max_sync(0xffffffffu, lo);
      const int T = w.nt[x], nt_other = w.nt[x ^ 1];
      float m = -INFINITY, l = 0.f;
      float lu = kNoUnit, row_sl2 = 0.f;  // 8 bits: log2 of the unit of p vs, the row's factor of scores
      if constexpr (KV8) {
        if (T > 0) {
          if (!__all_sync(0xffffffffu, mbar_wait(&q_full[x], q_cnt & 1u, abort_flag))) {
            ok = false;
            break;
          }
          uint8_t* const q_row = sQ + x * SLOT + row * 128;
          if constexpr (K8) row_sl2 = ldexpf(sl2, -q_to_e4m3<D>(q_row, SLOT / NB, row & 7));
          else row_sl2 = ldexpf(sl2, -q_to_h16<D>(q_row, SLOT / NB, row & 7));
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) mbar_arrive(&q_ready[x]);
        }
      }
      auto kt_of = [&](int t) { return (w.t0 + t) * KT; };
      for (int t = 0; t < T; ++t, ++cnt) {
        const int sb = NQ == 2 ? x : (int)(cnt & 1u);
        const uint32_t par = NQ == 2 ? cnt & 1u : (cnt >> 1) & 1u;
        if (!__all_sync(0xffffffffu, mbar_wait(&s_full[sb], par, abort_flag))) {
          ok = false;
          break;
        }
        if (teller) {
          // S of this tile is through, and with it the product before it.  K
          // goes back with the later stream's S, V with its product.
          if (x == 1 || t >= nt_other) mbar_arrive_relaxed(&empty[r_slot(it + 2 * t)]);
          if (t > 0 && (x == 1 || t > nt_other)) mbar_arrive_relaxed(&empty[r_slot(it + 2 * t - 1)]);
          if (t + 1 == T) mbar_arrive_relaxed(&q_empty[x]);
        }
        // NQ = 1: every warp sees each of pv_done's phases, in order, before it
        // lets the next product start, so the parity is never ambiguous.  (NQ =
        // 2: S of this tile was issued behind the product before it.)
        auto prior_product = [&]() {
          if (NQ == 1 && cnt > 0) {
            ok = __all_sync(0xffffffffu, mbar_wait(&pv_done[x], (cnt - 1) & 1u, abort_flag));
          }
          return ok;
        };
        if (live) {
          const TileArgs ta{tmem + lrow + sb * 128, tO, hi - kt_of(t), lo - kt_of(t), hi_min < kt_of(t) + KT, lo_max > kt_of(t),
                            valid, KV8 ? row_sl2 : sl2};
          if constexpr (KV8) softmax_tile8<D>(ta, tscales[((it >> 1) + t) % C::NSCALES], m, l, lu);
          else if constexpr (NQ == 1) ok = softmax_tile_call<D>(ta, m, l, &pv_done[x], (cnt - 1) & 1u, abort_flag);
          else ok = softmax_tile<D, NQ>(ta, m, l, &pv_done[x], (cnt - 1) & 1u, abort_flag);
          if (!ok) break;
          tmem_wait_st();
          fence_before();
          if (!prior_product()) break;
        } else {
          if (!prior_product()) break;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive_relaxed(&p_full[sb]);
      }
      if (!ok) break;
      if (T > 0) {
        // the last product: NQ = 1 commits every one of them, NQ = 2 only this
        if (!__all_sync(0xffffffffu, mbar_wait(&pv_done[x], (NQ == 1 ? cnt - 1 : q_cnt) & 1u, abort_flag))) {
          ok = false;
          break;
        }
        if (teller && (x == 1 || T > nt_other)) mbar_arrive_relaxed(&empty[r_slot(it + 2 * T - 1)]);
        q_used = q_cnt;
        ++q_cnt;
        fence_after();
      }
      it += 2 * max(T, nt_other);
      // ---- epilogue: O and (m, l) of the rows.  The descriptor goes back in front
      // of the stores: behind them the arrival, a release, would wait for them.
      const int part = w.part, tok = w.start + i;
      const bool bad = T > 0 && ((*(volatile const int32_t*)&w.bad >> x) & 1);
      if (__builtin_expect(bad && live, 0)) {
        if constexpr (KV8) add_nan8<D>(r, kv, w, tO, i, a.window, a.causal);
        else add_nonfinite<D>(r, kv, w, tO, i, a.window, a.causal);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&w_empty[ws]);
      // Up to 8 rows of a warp (single tokens) each lane stores its own, which is
      // little code; more go through shared memory.
      const uint32_t rows = __ballot_sync(0xffffffffu, valid);
      const bool staged = NQ == 2 || (live && p.mode != kModeCluster && __popc(rows) > 8);
      if (NQ == 1 && T > 0 && !staged && lane == 0) mbar_arrive_relaxed(&q_empty[q_used & 1u]);
      if (live) {
        const float o_unit = KV8 ? exp2f(lu - kUnitLog8) : 1.f;
        const float inv = o_unit / l;  // (every row sees its own key: l is 0 only where all scores are -inf)
        if (NQ == 1 && p.mode == kModeCluster) {
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            float v[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = 0.f;
            if (T > 0) tmem_ld32(tO + c, v);
            if (valid) {
#pragma unroll
              for (int j = 0; j < 32; j += 4)
                *reinterpret_cast<float4*>(c_o + row * (D + 4) + c + j) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
            }
          }
          if (valid) c_ml[row] = part_stats(m, l);
        } else {
          if (valid) store_stats<D>(a, p, part, x, row, tok, h, m, l);
          // where this lane's own row starts, in 16-byte units
          const int64_t own =
              part >= 0 ? ((int64_t)part * p.ws_rows + x * 128 + row) * (D / 4)
                        : ((int64_t)tok * a.o_row + (int64_t)h * a.o_head) / 8;
          uint4* const base = reinterpret_cast<uint4*>(part >= 0 ? (void*)a.ws : a.out);
          if (!staged) {
            if (T > 0) {
              float v[D];
              if constexpr (D == 128) {
                tmem_ld128(tO, v);
              } else {
                tmem_ld32(tO, v);
                tmem_ld32(tO + 32, v + 32);
              }
              if (valid && part >= 0) {
#pragma unroll
                for (int j = 0; j < D / 4; ++j) base[own + j] = *reinterpret_cast<const uint4*>(v + 4 * j);
              } else if (valid) {
#pragma unroll
                for (int j = 0; j < D / 8; ++j) base[own + j] = pack8(v + 8 * j, inv);
              }
            }
          } else {
            // 128 bytes of each row at a time through shared memory, so that a store
            // covers whole lines (a row per lane took five times as long): row r's
            // 16-byte chunk c lies at chunk c ^ (r & 7).
            uint8_t* st = NQ == 2 ? sS + warp * 4096 : sQ + (q_used & 1u) * SLOT + warp * 4096;
            auto flush = [&](int at) {  // the staged 128 bytes of each row to 16-byte unit `at` of it
              __syncwarp();
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const int rr = 4 * k + (lane >> 3), c = lane & 7;
                const int64_t o = __shfl_sync(0xffffffffu, own, rr);
                const uint4 q = *reinterpret_cast<const uint4*>(st + rr * 128 + ((c ^ (rr & 7)) << 4));
                if ((rows >> rr) & 1u) base[o + at + c] = q;
              }
              __syncwarp();
            };
            auto put = [&](int c, uint4 q) { *reinterpret_cast<uint4*>(st + lane * 128 + ((c ^ (lane & 7)) << 4)) = q; };
            if (T > 0 && part >= 0) {
#pragma unroll 1
              for (int c = 0; c < D; c += 32) {
                float v[32];
                tmem_ld32(tO + c, v);
                if (KV8) {
#pragma unroll
                  for (int j = 0; j < 32; ++j) v[j] *= o_unit;
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) put(j, *reinterpret_cast<const uint4*>(v + 4 * j));
                flush(c / 4);
              }
            } else if (T > 0) {
#pragma unroll 1
              for (int c = 0; c < D; c += 64) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  float v[32];
                  tmem_ld32(tO + c + 32 * h, v);
#pragma unroll
                  for (int j = 0; j < 4; ++j) put(4 * h + j, pack8(v + 8 * j, inv));
                }
                flush(c / 8);
              }
            }
          }
        }
        fence_before();
      }
      if (NQ == 1 && T > 0 && staged) {
        fence_proxy_async();  // the next thing into this Q tile comes by TMA
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_empty[q_used & 1u]);
      }
    }
    if (!ok) give_up();
  }
  fence_before();
  __syncthreads();
  if (warp == SW + 1) {
    fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (NQ == 1 && p.mode == kModeCluster) {
    // ---- merge of the cluster's parts, in key order: rank q finishes the rows
    // [q R / S, (q + 1) R / S), a warp per row
    constexpr int CL = D / 32;
    cg::cluster_group cl = cg::this_cluster();
    cl.sync();  // every part is there
    const int S = p.cluster, q = (int)cl.block_rank(), item = (int)blockIdx.x / S, b = item / a.Hkv;
    const Seq s = load_seq(r, b);
    const int R = s.ok ? s.n * G : 0, kvh = item - b * a.Hkv;
    float* c_o = reinterpret_cast<float*>(sR);
    float2* c_ml = reinterpret_cast<float2*>(sR + 128 * (D + 4) * 4);
    for (int rr = q * R / S + warp; rr < (q + 1) * R / S; rr += C::THREADS / 32) {
      float2 ml = make_float2(-INFINITY, 0.f);
      if (lane < S) ml = *cl.map_shared_rank(c_ml + rr, lane);
      const float M = warp_max(ml.x);
      // a part that saw no key has weight 0; the NaN of a part with a NaN score stays one
      const float wt = ml.x == -INFINITY ? 0.f : exp2f(ml.x - M);
      const float L = warp_sum(wt == 0.f ? 0.f : ml.y * wt);
      float acc[CL];
#pragma unroll
      for (int j = 0; j < CL; ++j) acc[j] = 0.f;
      using Vec = typename std::conditional<CL == 4, float4, float2>::type;
#pragma unroll 4
      for (int u = 0; u < S; ++u) {
        // (a part that saw no key of this row holds zeros)
        const float wu = __shfl_sync(0xffffffffu, wt, u);
        const Vec t = *reinterpret_cast<const Vec*>(cl.map_shared_rank(c_o, u) + rr * (D + 4) + lane * CL);
        const float* v = reinterpret_cast<const float*>(&t);
#pragma unroll
        for (int j = 0; j < CL; ++j) acc[j] = fmaf(wu, v[j], acc[j]);
      }
      const int i = rr / G, h = kvh * G + rr % G;
      const float inv = 1.f / L;
      bf16* o = reinterpret_cast<bf16*>(a.out) + (int64_t)(s.start + i) * a.o_row + (int64_t)h * a.o_head + lane * CL;
#pragma unroll
      for (int j = 0; j < CL; j += 2)
        *reinterpret_cast<__nv_bfloat162*>(o + j) = __floats2bfloat162_rn(acc[j] * inv, acc[j + 1] * inv);
      if (a.lse && lane == 0)
        a.lse[(int64_t)(s.start + i) * a.Hq + h] = lse_of(M, L);
    }
    cluster_sync_relaxed();  // no CTA leaves while a peer reads its part
  }
}

// n floats from p, or zeros.  As predicated loads: under a branch the compiler
// waits for each of them before the next.
template <int n>
__device__ __forceinline__ void load_if(float* v, const float* p, bool yes) {
  static_assert(n == 2 || n == 4, "one vector load");
  if constexpr (n == 4) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %5, 0;\n\t"
        "mov.f32 %0, 0f00000000;\n\tmov.f32 %1, 0f00000000;\n\tmov.f32 %2, 0f00000000;\n\tmov.f32 %3, 0f00000000;\n\t"
        "@p ld.global.v4.f32 {%0, %1, %2, %3}, [%4];\n\t}"
        : "=&f"(v[0]), "=&f"(v[1]), "=&f"(v[2]), "=&f"(v[3])
        : "l"(p), "r"((uint32_t)yes)
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %3, 0;\n\t"
        "mov.f32 %0, 0f00000000;\n\tmov.f32 %1, 0f00000000;\n\t"
        "@p ld.global.v2.f32 {%0, %1}, [%2];\n\t}"
        : "=&f"(v[0]), "=&f"(v[1])
        : "l"(p), "r"((uint32_t)yes)
        : "memory");
  }
}

// Reads each part once, 7 us for single tokens and 19 (cold) for the 40 MB of 300
// row tiles of 128: bound by its chain of loads (lengths, cut, statistics, parts).
// Merge of the parts of each item that a range boundary cut.  CTA (c - 1, y):
// boundary c, if it is the first inside its item; RW rows per warp, parts in key
// order.
template <int D, int RW>
__global__ void __launch_bounds__(256, 4) k_ragged_merge(Ragged r, AttnCall a, Plan p, int grid) {
  constexpr int C = D / 32, rows_per_cta = 8 * RW;
  pdl_trigger();
  pdl_wait();
  r.starts = after_wait(r.starts);
  if (r.lens) r.lens = after_wait(r.lens);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int G = a.Hq / a.Hkv, c = blockIdx.x + 1;
  const bool one = r.batch <= 32;
  Seq mine_s{0, 0, 0, false};
  if (one && lane < r.batch) mine_s = load_seq(r, lane);
  int64_t sum = 0;
  for (int b = lane; b < r.batch; b += 32) sum += units_of(one ? mine_s : load_seq(r, b), p, a);
  const Ranges rg(max(sum_up_to(sum, p.max_units), 0), p, grid);
  if (c >= rg.n) return;
  const int u = rg.start(c), n = rg.n;
  int before = 0;
  for (int base = 0; base < r.batch; base += 32) {
    const int b = base + lane;
    Seq s{0, 0, 0, false};
    if (b < r.batch) s = one ? mine_s : load_seq(r, b);
    const int mine = (int)units_of(s, p, a), incl = warp_scan_i(mine, lane);
    const int end = before + __shfl_sync(0xffffffffu, incl, 31);
    if (u >= end) {
      before = end;
      continue;
    }
    const int src = __ffs(__ballot_sync(0xffffffffu, before + incl > u)) - 1;
    const int seq_u = before + __shfl_sync(0xffffffffu, incl - mine, src);
    const int start = __shfl_sync(0xffffffffu, s.start, src), sn = __shfl_sync(0xffffffffu, s.n, src);
    const int T = __shfl_sync(0xffffffffu, s.ok && s.n > 0 ? tile_count(s, a.window) + p.pad : 1, src);
    const int item = (u - seq_u) / T, i_begin = seq_u + item * T, i_end = i_begin + T;
    // no cut here (in front of the item's tiles), or not the item's first
    if (u <= i_begin + p.pad || rg.start(c - 1) > i_begin + p.pad) return;
    const int qi = item / a.Hkv, kvh = item - qi * a.Hkv, i0 = qi * p.tok;
    const int parts = rg.of(i_end - 1) - (c - 1) + 1;
    const int slot0 = 2 * (c - 1) + (rg.start(c - 1) < i_begin);
    auto slot_of = [&](int q) { return q == 0 ? slot0 : 2 * (c - 1 + q); };
    const int row0 = blockIdx.y * rows_per_cta + warp;
    // the token of a row of the item, or -1
    auto token = [&](int row) {
      const int x = row / 128, rr = row % 128, i = i0 + x * p.tpt + rr / G;
      return rr < p.tpt * G && i < min(i0 + p.tok, sn) ? start + i : -1;
    };
    auto put = [&](int row, int tok, float M, float L, const float* acc) {
      const float inv = 1.f / L;
      const int h = kvh * G + row % 128 % G;
      bf16* o = reinterpret_cast<bf16*>(a.out) + (int64_t)tok * a.o_row + (int64_t)h * a.o_head + lane * C;
#pragma unroll
      for (int j = 0; j < C; j += 2)
        *reinterpret_cast<__nv_bfloat162*>(o + j) = __floats2bfloat162_rn(acc[j] * inv, acc[j + 1] * inv);
      if (a.lse && lane == 0) a.lse[(int64_t)tok * a.Hq + h] = lse_of(M, L);
    };
    constexpr int PP = 32 / RW;
    if (RW > 1 && parts <= PP) {
      // all rows of the warp at once: the statistics a lane per (row, part), O two
      // parts of every row in flight
      const int k_ml = lane / PP, q_ml = lane % PP, row_ml = row0 + 8 * k_ml;
      float2 ml = make_float2(-INFINITY, 0.f);
      if (q_ml < parts && token(row_ml) >= 0) ml = *part_ml<D>(a, p, slot_of(q_ml), row_ml);
      float M = ml.x;
#pragma unroll
      for (int o = PP / 2; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
      // a part that saw no key has weight 0 and its sums were not written; the NaN of a part stays one
      const uint32_t saw = __ballot_sync(0xffffffffu, ml.y != 0.f);
      const float wt = ml.x == -INFINITY ? 0.f : exp2f(ml.x - M);
      float L = wt == 0.f ? 0.f : ml.y * wt;
#pragma unroll
      for (int o = PP / 2; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
      float acc[RW][C];
#pragma unroll
      for (int k = 0; k < RW; ++k)
#pragma unroll
        for (int j = 0; j < C; ++j) acc[k][j] = 0.f;
#pragma unroll 1
      for (int q0 = 0; q0 < parts; q0 += 2) {
        float v[2][RW][C], w[2][RW];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int k = 0; k < RW; ++k) {
            w[u][k] = __shfl_sync(0xffffffffu, wt, k * PP + ((q0 + u) & (PP - 1)));
            if (q0 + u >= parts) w[u][k] = 0.f;
            // (a weight that underflows still takes its sums along: 0 x NaN is NaN)
            load_if<C>(v[u][k], part_o<D>(a, p, slot_of(q0 + u), row0 + 8 * k) + lane * C,
                       q0 + u < parts && ((saw >> (k * PP + q0 + u)) & 1u));
          }
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int k = 0; k < RW; ++k)
#pragma unroll
            for (int j = 0; j < C; ++j) acc[k][j] = fmaf(w[u][k], v[u][k][j], acc[k][j]);
      }
#pragma unroll
      for (int k = 0; k < RW; ++k) {
        const float Mk = __shfl_sync(0xffffffffu, M, k * PP), Lk = __shfl_sync(0xffffffffu, L, k * PP);
        const int row = row0 + 8 * k, tok = token(row);
        if (tok >= 0) put(row, tok, Mk, Lk, acc[k]);
      }
      return;
    }
    for (int row = row0; row < (int)(blockIdx.y + 1) * rows_per_cta; row += 8) {
      const int tok = token(row);
      if (tok < 0) continue;
      float M = -INFINITY, L = 0.f, acc[C];
#pragma unroll
      for (int j = 0; j < C; ++j) acc[j] = 0.f;
      for (int base = 0; base < parts; base += 32) {
        float2 ml = make_float2(-INFINITY, 0.f);
        if (base + lane < parts) ml = *part_ml<D>(a, p, slot_of(base + lane), row);
        const int cnt = min(32, parts - base);
        // O of 8 parts at a time, the first 8 together with (m, l)
        float v[8][C];
        auto load = [&](int q0) {
#pragma unroll
          for (int q = 0; q < 8; ++q)
            load_if<C>(v[q], part_o<D>(a, p, slot_of(base + q0 + q), row) + lane * C, q0 + q < cnt);
        };
        load(0);
        const float Mn = fmaxf(M, warp_max(ml.x)), mref = Mn == -INFINITY ? 0.f : Mn;
        const float f = M == -INFINITY ? 0.f : exp2f(M - mref);
        // (weights as above)
        const uint32_t saw = __ballot_sync(0xffffffffu, ml.y != 0.f);
        const float wt = ml.x == -INFINITY ? 0.f : exp2f(ml.x - mref);
        M = Mn;
        L = L * f + warp_sum(wt == 0.f ? 0.f : ml.y * wt);
#pragma unroll
        for (int j = 0; j < C; ++j) acc[j] *= f;
        for (int q0 = 0; q0 < cnt; q0 += 8) {
          if (q0 > 0) load(q0);
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            const float wq = q0 + q < cnt ? __shfl_sync(0xffffffffu, wt, (q0 + q) & 31) : 0.f;
            const bool yes = q0 + q < cnt && ((saw >> (q0 + q)) & 1u);
#pragma unroll
            for (int j = 0; j < C; ++j) acc[j] = fmaf(wq, yes ? v[q][j] : 0.f, acc[j]);
          }
        }
      }
      put(row, tok, M, L, acc);
    }
    return;
  }
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
cudaError_t current_sms(int* sms) {
  static std::atomic<int> cached[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && cached[dev]) {
    *sms = cached[dev];
    return cudaSuccess;
  }
  e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess && dev < 64) cached[dev] = *sms;
  return e;
}

// Clusters of S CTAs of the NQ = 1 kernel that the current device runs at once.
template <int D>
int query_clusters(int S) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = S;
  cfg.blockDim = Cfg<D, 1>::THREADS;
  cfg.dynamicSmemBytes = Cfg<D, 1>::SMEM;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = S;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaFuncSetAttribute(k_ragged_tc<D, 1, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Cfg<D, 1>::SMEM) !=
          cudaSuccess ||
      cudaFuncSetAttribute(k_ragged_tc<D, 1, false>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, k_ragged_tc<D, 1, false>, &cfg) != cudaSuccess) {
    cudaGetLastError();
    n = 0;
  }
  return n;
}
int clusters_at_once(int d, int S) {
  static std::atomic<int> cached[64][2][kMaxCluster + 1];  // + 1; 0: not asked
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) {
    cudaGetLastError();
    return 0;
  }
  std::atomic<int>& c = cached[dev][d == 64][S];
  if (!c) c = 1 + (d == 64 ? query_clusters<64>(S) : query_clusters<128>(S));
  return c - 1;
}

struct HostPlan {
  Plan p;
  int nq;       // 128-row tiles per item
  int merge;    // parts may have to meet
};

HostPlan make_plan(const Ragged& r, const AttnCall& a, int sms, bool kv8 = false) {
  const int G = a.Hq / a.Hkv;
  HostPlan h{};
  Plan& p = h.p;
  p.tpt = std::min(128 / G, std::max(r.max_rows, 1));
  h.nq = !kv8 && (int64_t)r.max_rows * G <= (int64_t)p.tpt * G ? 1 : 2;
  p.tok = p.tpt * h.nq;
  p.ws_rows = h.nq == 1 ? p.tpt * G : 256;
  p.max_items = (int)std::min<int64_t>(std::min<int64_t>((int64_t)r.total / p.tok + std::min(r.batch, r.total), r.total),
                                       (int64_t)r.batch * ((r.max_rows + p.tok - 1) / p.tok));
  const int64_t items = (int64_t)p.max_items * a.Hkv;
  const int tiles = (r.max_len + KT - 1) / KT;
  // 2, 4 and 6 are within 2% of each other for chunks; single tokens of 64
  // sequences of 100 to 8000: 136 us without, 122 with 1, 124 with 3
  p.pad = h.nq == 2 || a.d == 64 ? 2 : 1;
  const int64_t units = items * (tiles + p.pad);
  p.max_units = (int)std::min<int64_t>(units, INT32_MAX);
  // Whole items where they fill the SMs one and a half times, or where the longest
  // ones of each wave (packed causal prompts: of the first, the others are short)
  // take no more key tiles than an even share and the 16 that cutting costs
  // (partials, their merge).  Causal prompt of 1024: 22 us whole, 38 cut; of 1500 29
  // and 53; 200 new tokens of 3 over 4096 62 and 65; 64 of 8 over 8192 111 and 79.
  const int64_t waves = a.causal && !r.lens ? 1 : (items + sms - 1) / sms;
  const bool whole = h.nq == 2 && (items >= 3 * sms / 2 || tiles * waves <= items * tiles / sms + 16);
  p.mode = whole || units > INT32_MAX ? kModeItems : kModeRanges;
  // cluster: a cluster per item, where all of them run at once and a CTA gets at
  // most 7 key tiles.  One user's block of 16, 8 KV heads: 15.8 us against 22.3
  // over 4096 tokens, 22.4 against 23.6 over 8192, 29 against 25 over 12288.
  // (Clusters that wait for others cost more than they save: two users' single
  // tokens over 1024, 16 clusters of 8, took 19.4 us against 13.8.)
  p.cluster = 1;
  if (h.nq == 1 && p.mode == kModeRanges) {
    const int64_t all = (int64_t)r.batch * a.Hkv;
    // (a window's keys may begin anywhere in a tile, but it has no more tiles than the sequence)
    const int64_t span = std::min<int64_t>(r.max_len, (int64_t)a.window + r.max_rows);
    const int64_t most = a.window ? std::min<int64_t>(tiles, (span + KT - 1) / KT + 1) : tiles;
    for (int S = 2; S <= kMaxCluster && S <= 2 * most && all * S <= sms; S *= 2)
      if (all <= clusters_at_once(a.d, S) && most <= 7 * S && most > 1) {
        p.mode = kModeCluster;
        p.cluster = S;
      }
  }
  // items: heads dealt out together while their K/V (both, bf16) stay within 48 MB of L2
  const int64_t per_head = std::max<int64_t>(1, (int64_t)(r.lens ? (int64_t)r.max_len * std::min(r.batch, r.total) : r.total) * a.d * 4);
  p.hgroup = (int)std::max<int64_t>(1, std::min<int64_t>(a.Hkv, (48ll << 20) / per_head));
  p.min_tiles_log2 = h.nq == 2 ? 2 : 0;
  p.slots = 2 * sms;
  h.merge = p.mode == kModeRanges && tiles > 1;
  return h;
}

enum Tile { kBf16, kCodes, kCodesSwizzled };
cudaError_t encode(CUtensorMap* m, const void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
                   const cuuint32_t* box, Tile tile = kBf16) {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return (PFN_cuTensorMapEncodeTiled_v12000)f;
  }();
  if (!fn) return cudaErrorNotSupported;
  const cuuint32_t one[4] = {1, 1, 1, 1};
  return fn(m, tile == kBf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, rank, const_cast<void*>(base), dims,
            strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, tile == kCodes ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? cudaSuccess
             : cudaErrorInvalidValue;
}

template <int D, int NQ, bool KV8 = false>
cudaError_t launch_tc(const Ragged& r, const AttnCall& a,
                      const typename std::conditional<KV8, Kv8View, KVView>::type& kv, const Plan& p, int sms,
                      const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, cudaStream_t st) {
  static std::atomic<bool> attr[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !attr[dev]) {
    e = cudaFuncSetAttribute(k_ragged_tc<D, NQ, KV8>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Cfg<D, NQ, KV8>::SMEM);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(k_ragged_tc<D, NQ, KV8>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    if (dev < 64) attr[dev] = true;
  }
  const int grid = p.mode == kModeCluster ? r.batch * a.Hkv * p.cluster : sms;
  return launch_kc(k_ragged_tc<D, NQ, KV8>, grid, Cfg<D, NQ, KV8>::THREADS, Cfg<D, NQ, KV8>::SMEM, st, p.cluster, r, a, kv, p, mq, mk,
                   mv);
}

cudaError_t encode_q(CUtensorMap* mq, const Ragged& r, const AttnCall& a, const HostPlan& h) {
  const cuuint64_t dims[3] = {(cuuint64_t)a.d, (cuuint64_t)a.Hq, (cuuint64_t)r.total};
  // (the stride of a dimension of one entry is never used, but may not be 0)
  const cuuint64_t strides[2] = {std::max<cuuint64_t>(a.q_head * 2, 16), (cuuint64_t)a.q_row * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)(a.Hq / a.Hkv), (cuuint32_t)h.p.tpt};
  return encode(mq, a.q, 3, dims, strides, box);
}

template <int D>
cudaError_t launch_d8(const Ragged& r, const AttnCall& a, const Kv8View& kv, const HostPlan& h, int sms, cudaStream_t st) {
  CUtensorMap mq, m[2];
  cudaError_t e = encode_q(&mq, r, a, h);
  for (int i = 0; i < 2 && e == cudaSuccess; ++i) {
    const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)1 << kv.page_shift, (cuuint64_t)a.Hkv, (cuuint64_t)kv.n_pages};
    // (the stride of a dimension of one entry is never used, but may not be 0)
    const cuuint64_t strides[3] = {(cuuint64_t)kv.slot, std::max<cuuint64_t>(kv.head, 16), std::max<cuuint64_t>(kv.page, 16)};
    const cuuint32_t box[4] = {(cuuint32_t)D, (cuuint32_t)std::min(1 << kv.page_shift, KT), 1, 1};
    e = encode(&m[i], i ? kv.v : kv.k, 4, dims, strides, box, i == 0 && Cfg<D, 2, true>::K8 ? kCodesSwizzled : kCodes);
  }
  if (e == cudaSuccess) e = launch_tc<D, 2, true>(r, a, kv, h.p, sms, mq, m[0], m[1], st);
  if (e != cudaSuccess || !h.merge) return e;
  return launch_k(k_ragged_merge<D, 4>, dim3(sms - 1, 256 / 32), 256, 0, st, r, a, h.p, sms);
}

template <int D>
cudaError_t launch_d(const Ragged& r, const AttnCall& a, const KVView& kv, const HostPlan& h, int sms, cudaStream_t st) {
  const int G = a.Hq / a.Hkv;
  CUtensorMap mq, mk, mv;
  if (cudaError_t e = encode_q(&mq, r, a, h)) return e;
  for (int i = 0; i < 2; ++i) {
    const cuuint64_t slot = (cuuint64_t)(i ? kv.v_slot : kv.k_slot) * 2, head = (cuuint64_t)(i ? kv.v_head : kv.k_head) * 2;
    const cuuint64_t dims[4] = {(cuuint64_t)D, kv.paged ? (cuuint64_t)1 << kv.page_shift : (cuuint64_t)kv.packed_rows,
                                (cuuint64_t)a.Hkv, kv.paged ? (cuuint64_t)kv.n_pages : 1};
    const cuuint64_t strides[3] = {slot, std::max<cuuint64_t>(head, 16),
                                   kv.paged ? std::max<cuuint64_t>(kv.page * 2, 16) : slot};
    const cuuint32_t box[4] = {64, (cuuint32_t)(kv.paged ? std::min(1 << kv.page_shift, KT) : KT), 1, 1};
    if (cudaError_t e = encode(i ? &mv : &mk, i ? kv.v : kv.k, 4, dims, strides, box)) return e;
  }
  cudaError_t e = h.nq == 1 ? launch_tc<D, 1>(r, a, kv, h.p, sms, mq, mk, mv, st)
                            : launch_tc<D, 2>(r, a, kv, h.p, sms, mq, mk, mv, st);
  if (e != cudaSuccess || !h.merge) return e;
  const int rows = h.nq == 1 ? r.max_rows * G : 256;
  // rows of a CTA: few enough CTAs that finding the cuts, which each does, is one wave
  return h.nq == 1 ? launch_k(k_ragged_merge<D, 1>, dim3(sms - 1, (rows + 7) / 8), 256, 0, st, r, a, h.p, sms)
                   : launch_k(k_ragged_merge<D, 4>, dim3(sms - 1, rows / 32), 256, 0, st, r, a, h.p, sms);
}

}  // namespace

cudaError_t attn_tc_workspace(const Ragged& r, const AttnCall& a, int64_t* bytes, bool kv8) {
  int sms = 0;
  // without a device (argument checks on a host) the largest part's count of SMs stands in
  if (current_sms(&sms) != cudaSuccess) {
    cudaGetLastError();
    sms = 152;
  }
  const HostPlan h = make_plan(r, a, sms, kv8);
  *bytes = h.merge ? (int64_t)h.p.slots * h.p.ws_rows * (a.d + 2) * 4 : 0;
  return cudaSuccess;
}

cudaError_t launch_attn_tc(const Ragged& r, const AttnCall& a, const KVView& kv, cudaStream_t st) {
  int sms = 0;
  if (cudaError_t e = current_sms(&sms)) return e;
  const HostPlan h = make_plan(r, a, sms);
  return a.d == 64 ? launch_d<64>(r, a, kv, h, sms, st) : launch_d<128>(r, a, kv, h, sms, st);
}

cudaError_t launch_attn_tc8(const Ragged& r, const AttnCall& a, const Kv8View& kv, cudaStream_t st) {
  int sms = 0;
  if (cudaError_t e = current_sms(&sms)) return e;
  const HostPlan h = make_plan(r, a, sms, true);
  return a.d == 64 ? launch_d8<64>(r, a, kv, h, sms, st) : launch_d8<128>(r, a, kv, h, sms, st);
}

}  // namespace dfl
