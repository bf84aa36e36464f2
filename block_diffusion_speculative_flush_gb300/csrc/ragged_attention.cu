// Target-side operators on ragged batches: new K/V rows into pages, and the
// attention of a chunk of new tokens over pages or of packed prompts on the
// CUDA cores.
//
//   o_i = sum_j p_ij v_j,  p_ij = exp(s_ij - m_i) / l_i,  s_ij = scale q_i . k_j
// over the keys j that row i sees, with the running maximum m and sum l of an
// online softmax (fp32, in the exp2 domain), one pass over K and V.
#include <cooperative_groups.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdio>
#include <type_traits>

#include "common.cuh"
#include "dflash.h"
#include "kernels.h"
#include "launch.h"
#include "ragged.h"
#include "target_checks.h"

namespace dfl {
namespace {

namespace cg = cooperative_groups;

// ---------------------------------------------------------------------------
// append
// ---------------------------------------------------------------------------
// One warp per new row: 16 bytes of K and of V per lane and step.  Bound by
// memory (2 reads and 2 writes of a row's Hkv d elements) for many rows: 6257 of
// 8 heads of 128 in 6.6 us, 7.7 TB/s, as they stay in L2.  64 rows are the
// latency of starts, length, table, row: 3 us.
__global__ void __launch_bounds__(256) k_kv_append(Ragged r, const uint4* k, const uint4* v, int64_t k_row,
                                                   int64_t k_head, int64_t v_row, int64_t v_head,
                                                   uint4* __restrict__ kp, uint4* __restrict__ vp, int64_t page_st,
                                                   int64_t slot_st, int64_t head_st, int page_shift, int n_pages,
                                                   int heads, int chunks) {
  pdl_trigger();
  pdl_wait();
  k = after_wait(k);  // the rows may be the previous kernel's
  v = after_wait(v);
  const int row = (int)(blockIdx.x * 8 + (threadIdx.x >> 5)), lane = threadIdx.x & 31;
  if (row >= r.total) return;
  const int b = seq_of_row(r, row);
  if (b >= r.batch) return;  // behind the last sequence
  const Seq s = load_seq(r, b);
  const int i = row - s.start;
  if (!s.ok && lane == 0) flag_status(r.status, DFLASH_STATUS_BOUNDS);
  if (!s.ok || i < 0 || i >= s.n) return;  // (in front of the first sequence: no one's row)
  const int pos = s.len - s.n + i;
  const int pg = r.table[(int64_t)b * r.table_stride + (pos >> page_shift)];
  if (pg < 0 || pg >= n_pages) {
    if (lane == 0) flag_status(r.status, DFLASH_STATUS_PAGE);
    return;
  }
  const int64_t base = (int64_t)pg * page_st + (int64_t)(pos & ((1 << page_shift) - 1)) * slot_st;
  for (int e = lane; e < heads * chunks; e += 32) {
    const int h = e / chunks, c = e - h * chunks;
    const uint4 a = k[(int64_t)row * k_row + h * k_head + c], w = v[(int64_t)row * v_row + h * v_head + c];
    kp[base + h * head_st + c] = a;
    vp[base + h * head_st + c] = w;
  }
}

// ---------------------------------------------------------------------------
// attention on the CUDA cores (fp32)
// ---------------------------------------------------------------------------
// Two kernels: k_attn_few for up to 64 packed rows of a sequence and KV head
// (single tokens, verified blocks, the first rows of a prompt), k_attn_tiles
// for more.  A row's arithmetic in k_attn_few depends on its own keys only
// (splits of the key axis start at fixed positions), so a block of tokens and
// single tokens give the same bits.
constexpr int kFewRows = 64;   // packed rows that k_attn_few takes
constexpr int kSplit = 256;    // keys of a split: one per thread of k_attn_few

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }

// Where position pos of sequence b (whose packed rows start at `start`) lies in
// K and V, in elements; false: on a page that does not exist.
__device__ __forceinline__ bool kv_at(const Ragged& r, const KVView& kv, int b, int start, int pos, int64_t& ko, int64_t& vo) {
  if (!kv.paged) {
    ko = (int64_t)(start + pos) * kv.k_slot;
    vo = (int64_t)(start + pos) * kv.v_slot;
    return true;
  }
  const int pg = r.table[(int64_t)b * r.table_stride + (pos >> kv.page_shift)], sl = pos & ((1 << kv.page_shift) - 1);
  ko = pg * kv.page + sl * kv.k_slot;
  vo = pg * kv.page + sl * kv.v_slot;
  return pg >= 0 && pg < kv.n_pages;
}

// Hidden keys among the scores and the probabilities of k_attn_few: V may hold
// anything there, and 0 x NaN is NaN, so their products are skipped.  Not every
// product with P = 0 is: a NaN that the row sees is its own, although its
// probability underflows.  The score of a hidden key is a NaN that no operation
// makes (theirs are 0x7fffffff), which a maximum passes over; its probability is
// -0, which exp2f never returns.
constexpr uint32_t kHidden = 0xffc0de00u;
__device__ __forceinline__ float masked_score(float s, bool see) { return see ? s : __uint_as_float(kHidden); }
__device__ __forceinline__ float masked_prob(float s, float mref) {
  return __float_as_uint(s) == kHidden ? -0.f : exp2f(s - mref);
}
__device__ __forceinline__ bool is_hidden(float p) { return __float_as_uint(p) == 0x80000000u; }

// The natural log-sum-exp of a row from (m, l) in the exp2 domain: -inf where every
// score is, NaN where one is.  (Every row sees its own key: l is never 0 for want of one.)
__device__ __forceinline__ float lse_of(float m, float l) { return (m + log2f(l)) * 0.6931471805599453f; }

// The splits of one row and four columns, taken in split order.
struct SplitMerge {
  float M = -INFINITY, L = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  __device__ __forceinline__ void max(float m) { M = fmaxf(M, m); }
  // (sums of a split that saw no key are zeros)
  __device__ __forceinline__ void add(float2 ml, float4 v) {
    const float mref = M == -INFINITY ? 0.f : M;
    const float f = ml.x == -INFINITY ? 0.f : exp2f(ml.x - mref);
    L = fmaf(f, ml.y, L);
    acc.x = fmaf(f, v.x, acc.x);
    acc.y = fmaf(f, v.y, acc.y);
    acc.z = fmaf(f, v.z, acc.z);
    acc.w = fmaf(f, v.w, acc.w);
  }
  __device__ __forceinline__ void store(const AttnCall& a, int tok, int h, int c) const {
    const float inv = 1.f / L;
    if (c < a.d)
      store4(reinterpret_cast<float*>(a.out) + (int64_t)tok * a.o_row + (int64_t)h * a.o_head + c,
             make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
    if (a.lse && c == 0)
      a.lse[(int64_t)tok * a.Hq + h] = lse_of(M, L);
  }
};

// BR packed rows (token, head of the group) x 256 keys per CTA; BR = 4 or 8 where
// a sequence and KV head has no more rows, else 16 (of 64 single tokens over 3900
// the CTAs of 16 took 292 us, those of 4 132).  Scores: a key per thread, its K
// row straight from memory, the rows of q broadcast from shared memory (a row at
// a time through shared-memory tiles, as many rows want it, left this kernel
// waiting for each 64 keys in turn).  Then a softmax, the rows dealt to the warps,
// and O = P V with the keys dealt to the warps.  Up to 8 splits are a thread-block
// cluster and meet in distributed shared memory, more meet through the workspace
// (k_attn_simt_merge, by the same arithmetic).
// Bound by latency where rows are few: the key's row, the softmax, V, each a chain
// of loads, then the merge; three blocks of 8 over 300 to 1500 tokens, 4 heads of
// 64: 11 us.  Many of them, 64 x 8 over 3900: 3.0 TB/s.
template <int DP, int BR> struct FewCfg {
  static constexpr int LQ = DP + 4, LP = BR + 4, LS = kSplit + 4;
  static constexpr int AREA = BR * (8 * DP > LS ? 8 * DP : LS);  // scores, later the warps' sums
  static constexpr size_t SMEM = sizeof(float) * (BR * LQ + AREA + kSplit * LP) + kSplit * 8 + BR * 8;
};
template <int DP, int BR>
__global__ void __launch_bounds__(256) k_attn_few(Ragged r, AttnCall a, KVView kv, int splits, int cluster) {
  using C = FewCfg<DP, BR>;
  constexpr int LQ = C::LQ, LP = C::LP, LS = C::LS;
  constexpr int COLS = DP / 4, SLICES = 32 / (COLS < 32 ? COLS : 32);  // column groups; key slices within a warp
  extern __shared__ float4 smem4[];
  float* sQ = reinterpret_cast<float*>(smem4);  // [BR][LQ]
  float* sS = sQ + BR * LQ;                     // [BR][LS] scores; later the warps' sums [8][BR][DP]
  float* sO = sS;
  float* sP = sS + C::AREA;                     // [256][LP]
  int64_t* sV = reinterpret_cast<int64_t*>(sP + kSplit * LP);        // [256] where the key's V lies, -1: nowhere
  float2* sML = reinterpret_cast<float2*>(sV + kSplit);              // [BR]
  pdl_trigger();
  pdl_wait();
  const int per = cluster > 1 ? cluster : splits;  // CTAs of 16 rows
  const int b = blockIdx.z, kvh = blockIdx.y, split = blockIdx.x % per, r0 = blockIdx.x / per * BR;
  const Seq s = load_seq(r, b);
  if (!s.ok) {
    if (threadIdx.x == 0) flag_status(r.status, DFLASH_STATUS_BOUNDS);
    return;
  }
  const int G = a.Hq / a.Hkv, R = s.n * G;
  if (r0 >= R) return;
  const bool idle = split > 0 && split * kSplit >= s.len;  // the merge does not look at it either
  if (idle && cluster == 1) return;
  cg::cluster_group cl = cg::this_cluster();
  if (idle) {
    cl.sync();
    cl.sync();
    return;
  }
  const int ctx = s.len - s.n, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // keys that any of the rows sees, within this split
  const int p_first = ctx + r0 / G, p_last = ctx + (min(r0 + BR, R) - 1) / G;
  const int k0 = split * kSplit;
  const int k_lo = max(k0, vis_lo(p_first, a.window));
  const int k_hi = min(k0 + kSplit, vis_hi(p_last, s.len, a.causal));
  const int pos = k0 + tid;
  int64_t ko = 0, vo = 0;
  bool here = pos >= k_lo && pos < k_hi, exists = false;
  if (here) {
    exists = kv_at(r, kv, b, s.start, pos, ko, vo);
    if (!exists) flag_status(r.status, DFLASH_STATUS_PAGE);
  }
  for (int e = tid; e < BR * COLS; e += 256) {
    const int rr = e / COLS, c = e % COLS * 4;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r0 + rr < R && c < a.d) {
      const int i = (r0 + rr) / G, g = (r0 + rr) % G;
      x = load4(reinterpret_cast<const float*>(a.q) + (int64_t)(s.start + i) * a.q_row + (int64_t)(kvh * G + g) * a.q_head + c);
    }
    *reinterpret_cast<float4*>(sQ + rr * LQ + c) = x;
  }
  sV[tid] = here && exists ? vo : -1;
  __syncthreads();
  // ---- scores
  float sc[BR];
#pragma unroll
  for (int i = 0; i < BR; ++i) sc[i] = 0.f;
  if (here && exists) {
    const float* kp = reinterpret_cast<const float*>(kv.k) + ko + kvh * kv.k_head;
#pragma unroll 8
    for (int c = 0; c < a.d; c += 4) {
      const float4 k4 = load4(kp + c);
#pragma unroll
      for (int i = 0; i < BR; ++i) {
        const float4 q4 = *reinterpret_cast<const float4*>(sQ + i * LQ + c);
        sc[i] = fmaf(q4.x, k4.x, sc[i]);
        sc[i] = fmaf(q4.y, k4.y, sc[i]);
        sc[i] = fmaf(q4.z, k4.z, sc[i]);
        sc[i] = fmaf(q4.w, k4.w, sc[i]);
      }
    }
  }
  const float sl2 = a.scale * 1.4426950408889634f;
  bool hidden = false;
#pragma unroll
  for (int i = 0; i < BR; ++i) {
    const int p = ctx + (r0 + i) / G;
    const bool see = here && r0 + i < R && pos >= vis_lo(p, a.window) && pos < vis_hi(p, s.len, a.causal);
    hidden |= !see;
    sS[i * LS + tid] = masked_score(sc[i] * sl2, see);
  }
  const bool guard = __syncthreads_or(hidden && here);
  // ---- softmax: warp w has rows w, w + 8
#pragma unroll
  for (int u = 0; u < (BR + 7) / 8; ++u) {
    const int i = warp + 8 * u;
    if (BR < 8 && i >= BR) break;
    float x[kSplit / 32], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int j = 0; j < kSplit / 32; ++j) {
      x[j] = sS[i * LS + lane + 32 * j];
      m = fmaxf(m, x[j]);
    }
    m = warp_max(m);
    const float mref = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int j = 0; j < kSplit / 32; ++j) {
      const float e = masked_prob(x[j], mref);
      l += e;
      sP[(lane + 32 * j) * LP + i] = e;
    }
    l = warp_sum(l);
    if (lane == 0) sML[i] = make_float2(m, l);
  }
  __syncthreads();
  // ---- O: warp w takes keys 32 w .. 32 w + 31 (its lanes' slices every SLICES-th)
  const int col = lane % COLS * 4, slice = lane / COLS;
  float acc[BR][4];
#pragma unroll
  for (int i = 0; i < BR; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
  const float* vp = reinterpret_cast<const float*>(kv.v) + kvh * kv.v_head + col;
  const bool in = col < a.d;
#pragma unroll 4
  for (int t = slice; t < 32; t += SLICES) {
    const int key = warp * 32 + t;
    const int64_t o = sV[key];
    float4 v4 = make_float4(0.f, 0.f, 0.f, 0.f);
    if (o >= 0 && in) v4 = load4(vp + o);
#pragma unroll
    for (int i4 = 0; i4 < BR; i4 += 4) {
      const float4 p4 = *reinterpret_cast<const float4*>(sP + key * LP + i4);
      const float pv[4] = {p4.x, p4.y, p4.z, p4.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (!guard || !is_hidden(pv[i])) {
          acc[i4 + i][0] = fmaf(pv[i], v4.x, acc[i4 + i][0]);
          acc[i4 + i][1] = fmaf(pv[i], v4.y, acc[i4 + i][1]);
          acc[i4 + i][2] = fmaf(pv[i], v4.z, acc[i4 + i][2]);
          acc[i4 + i][3] = fmaf(pv[i], v4.w, acc[i4 + i][3]);
        }
    }
  }
#pragma unroll
  for (int i = 0; i < BR; ++i) {
#pragma unroll
    for (int o = COLS; o < 32; o <<= 1)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] += __shfl_xor_sync(0xffffffffu, acc[i][j], o);
    if (slice == 0) *reinterpret_cast<float4*>(sO + (warp * BR + i) * DP + col) = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
  }
  __syncthreads();
  auto sum_warps = [&](int i, int c) {
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      const float4 t = *reinterpret_cast<const float4*>(sO + (w * BR + i) * DP + c);
      o.x += t.x;
      o.y += t.y;
      o.z += t.z;
      o.w += t.w;
    }
    return o;
  };
  if (cluster > 1) {
    float* sC = sP;  // [BR][DP], this split's sums (P has been used)
    for (int e = tid; e < BR * COLS; e += 256) {
      const int i = e / COLS, c = e % COLS * 4;
      *reinterpret_cast<float4*>(sC + i * DP + c) = sum_warps(i, c);
    }
    cl.sync();
    // rank q of the ns at work finishes every ns-th stretch of 256 column groups
    const int ns = max(1, min(splits, (s.len + kSplit - 1) / kSplit));
    for (int e = split * 32 + lane + warp * 32 * ns; e < BR * COLS; e += 8 * 32 * ns) {
      const int i = e / COLS, c = e % COLS * 4;
      if (r0 + i >= R) continue;
      SplitMerge m;
      for (int j = 0; j < ns; ++j) m.max(cl.map_shared_rank(sML, j)[i].x);
#pragma unroll 4
      for (int j = 0; j < ns; ++j)
        m.add(cl.map_shared_rank(sML, j)[i], *reinterpret_cast<const float4*>(cl.map_shared_rank(sC, j) + i * DP + c));
      m.store(a, s.start + (r0 + i) / G, kvh * G + (r0 + i) % G, c);
    }
    cl.sync();  // no CTA leaves while its sums are read
    return;
  }
  for (int e = tid; e < BR * COLS; e += 256) {
    const int i = e / COLS, c = e % COLS * 4;
    if (r0 + i >= R) continue;
    const float4 o = sum_warps(i, c);
    const float2 ml = sML[i];
    const int tok = s.start + (r0 + i) / G, h = kvh * G + (r0 + i) % G;
    if (splits > 1) {
      float* w = a.ws + (((int64_t)tok * a.Hq + h) * splits + split) * (a.d + 4);
      if (c == 0) *reinterpret_cast<float4*>(w) = make_float4(ml.x, ml.y, 0.f, 0.f);
      if (c < a.d) store4(w + 4 + c, o);
      continue;
    }
    const float inv = 1.f / ml.y;
    if (c < a.d)
      store4(reinterpret_cast<float*>(a.out) + (int64_t)tok * a.o_row + (int64_t)h * a.o_head + c,
             make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
    if (a.lse && c == 0)
      a.lse[(int64_t)tok * a.Hq + h] = lse_of(ml.x, ml.y);
  }
}

// 32 packed rows per CTA, 64 keys per step and group of 8 x 16 threads, each
// with 4 rows x 4 keys of the scores and 4 rows x DP / 16 columns of the output:
// 12 shared-memory passes for 64 products a thread.  A group's step (load, scores,
// softmax, product) is one chain between barriers: NG groups take every NG-th tile
// of keys, and their (m, l, O) meet in shared memory.  Bound by that chain still: a
// step of four groups takes about 20000 cycles, of which the FMAs need 8200.  The
// tiles with the most keys start first.  Causal prompts of 99 to 1200, 4 heads of
// 64: 61 us, 21 TFLOP/s, 28% of the fp32 pipe; one group before took 142.
constexpr int BK = 64;
template <int DP> struct TileCfg {
  static constexpr int NG = DP == 64 ? 4 : 2, BR = 32, LQ = DP + 4, LP = BK + 4;
  static constexpr int GROUP = BK * LQ + BK * DP + BR * LP;  // floats of a group's K, V and P
  static constexpr size_t SMEM = sizeof(float) * (BR * LQ + NG * GROUP);
};
template <int DP>
__global__ void __launch_bounds__(TileCfg<DP>::NG * 128) k_attn_tiles(Ragged r, AttnCall a, KVView kv) {
  using C = TileCfg<DP>;
  constexpr int RM = 4, BR = C::BR, LQ = C::LQ, LP = C::LP, NG = C::NG;
  extern __shared__ float4 smem4[];
  const int group = threadIdx.x >> 7, tid = threadIdx.x & 127;
  float* sQ = reinterpret_cast<float*>(smem4);
  float* sK = sQ + BR * LQ + group * C::GROUP;
  float* sV = sK + BK * LQ;
  float* sP = sV + BK * DP;
  auto group_sync = [&] { asm volatile("bar.sync %0, 128;" ::"r"(group + 1) : "memory"); };
  pdl_trigger();
  pdl_wait();
  // grid: (tile from the sequence's end, sequence, KV head), the head fastest
  const int kvh = (int)(blockIdx.x % a.Hkv), b = (int)(blockIdx.x / a.Hkv % r.batch);
  const int back = (int)(blockIdx.x / a.Hkv / r.batch);
  const Seq s = load_seq(r, b);
  if (!s.ok) {
    if (threadIdx.x == 0 && back == 0) flag_status(r.status, DFLASH_STATUS_BOUNDS);
    return;
  }
  const int G = a.Hq / a.Hkv, R = s.n * G, r0 = ((R + BR - 1) / BR - 1 - back) * BR;
  if (r0 < 0) return;
  const int ctx = s.len - s.n, tx = tid & 15, ty = tid >> 4;
  const int p_first = ctx + r0 / G, p_last = ctx + (min(r0 + BR, R) - 1) / G;
  const int k_lo = vis_lo(p_first, a.window), k_hi = vis_hi(p_last, s.len, a.causal);
  for (int e = threadIdx.x; e < BR * (DP / 4); e += NG * 128) {
    const int rr = e / (DP / 4), c = e % (DP / 4) * 4;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r0 + rr < R && c < a.d) {
      const int i = (r0 + rr) / G, g = (r0 + rr) % G;
      x = load4(reinterpret_cast<const float*>(a.q) + (int64_t)(s.start + i) * a.q_row + (int64_t)(kvh * G + g) * a.q_head + c);
    }
    *reinterpret_cast<float4*>(sQ + rr * LQ + c) = x;
  }
  int lo[RM], hi[RM];
  float m[RM], l[RM], acc[RM][DP / 16];
#pragma unroll
  for (int i = 0; i < RM; ++i) {
    const int rr = r0 + ty * RM + i, p = ctx + rr / G;
    lo[i] = vis_lo(p, a.window);
    hi[i] = rr < R ? vis_hi(p, s.len, a.causal) : 0;
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int c = 0; c < DP / 16; ++c) acc[i][c] = 0.f;
  }
  const float sl2 = a.scale * 1.4426950408889634f;
  const float* Kb = reinterpret_cast<const float*>(kv.k) + kvh * kv.k_head;
  const float* Vb = reinterpret_cast<const float*>(kv.v) + kvh * kv.v_head;
  __syncthreads();  // Q is there
  for (int t0 = (k_lo / BK + group) * BK; t0 < k_hi; t0 += NG * BK) {
    group_sync();
#pragma unroll 4
    for (int e = tid; e < BK * (DP / 4); e += 128) {
      const int kk = e / (DP / 4), c = e % (DP / 4) * 4, pos = t0 + kk;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
      if (pos >= k_lo && pos < k_hi && c < a.d) {
        int64_t ko, vo;
        if (kv_at(r, kv, b, s.start, pos, ko, vo)) {
          x = load4(Kb + ko + c);
          y = load4(Vb + vo + c);
        } else if (c == 0) {
          flag_status(r.status, DFLASH_STATUS_PAGE);
        }
      }
      *reinterpret_cast<float4*>(sK + kk * LQ + c) = x;
      *reinterpret_cast<float4*>(sV + kk * DP + c) = y;
    }
    group_sync();
    float sc[RM][4];
#pragma unroll
    for (int i = 0; i < RM; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) sc[i][j] = 0.f;
#pragma unroll 4
    for (int c = 0; c < DP; c += 4) {
      float4 q4[RM], k4[4];
#pragma unroll
      for (int i = 0; i < RM; ++i) q4[i] = *reinterpret_cast<const float4*>(sQ + (ty * RM + i) * LQ + c);
#pragma unroll
      for (int j = 0; j < 4; ++j) k4[j] = *reinterpret_cast<const float4*>(sK + (tx + 16 * j) * LQ + c);
#pragma unroll
      for (int i = 0; i < RM; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          sc[i][j] = fmaf(q4[i].x, k4[j].x, sc[i][j]);
          sc[i][j] = fmaf(q4[i].y, k4[j].y, sc[i][j]);
          sc[i][j] = fmaf(q4[i].z, k4[j].z, sc[i][j]);
          sc[i][j] = fmaf(q4[i].w, k4[j].w, sc[i][j]);
        }
    }
    bool masked = false;
#pragma unroll
    for (int i = 0; i < RM; ++i) {
      float mt = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int pos = t0 + tx + 16 * j;
        const bool see = pos >= lo[i] && pos < hi[i];
        masked |= !see;
        sc[i][j] = see ? sc[i][j] * sl2 : -INFINITY;
        mt = fmaxf(mt, sc[i][j]);
      }
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, o));
      const float mn = fmaxf(m[i], mt);
      const float mref = mn == -INFINITY ? 0.f : mn;
      const float f = m[i] == -INFINITY ? 0.f : exp2f(m[i] - mref);
      float ls = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float pv = exp2f(sc[i][j] - mref);
        ls += pv;
        sP[(ty * RM + i) * LP + tx + 16 * j] = pv;
      }
      m[i] = mn;
      l[i] = l[i] * f + ls;
#pragma unroll
      for (int c = 0; c < DP / 16; ++c) acc[i][c] *= f;
    }
    // P rows of this thread's row group come from the same half warp
    __syncwarp();
    auto product = [&](auto guarded) {
      int from[RM], keys[RM];  // keys [from, from + keys) of the tile are the row's
#pragma unroll
      for (int i = 0; i < RM; ++i) {
        from[i] = lo[i] - t0;
        keys[i] = max(hi[i] - lo[i], 0);
      }
#pragma unroll 2
      for (int kk = 0; kk < BK; kk += 4) {
        float4 p4[RM];
#pragma unroll
        for (int i = 0; i < RM; ++i) p4[i] = *reinterpret_cast<const float4*>(sP + (ty * RM + i) * LP + kk);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
#pragma unroll
          for (int cc = 0; cc < DP / 64; ++cc) {
            const float4 v4 = *reinterpret_cast<const float4*>(sV + (kk + u) * DP + cc * 64 + tx * 4);
#pragma unroll
            for (int i = 0; i < RM; ++i) {
              const float pv = u == 0 ? p4[i].x : u == 1 ? p4[i].y : u == 2 ? p4[i].z : p4[i].w;
              float* o = acc[i] + cc * 4;
              if (!decltype(guarded)::value || (unsigned)(kk + u - from[i]) < (unsigned)keys[i]) {
                o[0] = fmaf(pv, v4.x, o[0]);
                o[1] = fmaf(pv, v4.y, o[1]);
                o[2] = fmaf(pv, v4.z, o[2]);
                o[3] = fmaf(pv, v4.w, o[3]);
              }
            }
          }
        }
      }
    };
    // A row's hidden keys have P = 0, and V may be anything there: tiles with
    // some skip those products.  (Not every product with P = 0, as above.)
    if (__any_sync(0xffffffffu, masked)) product(std::true_type());
    else product(std::false_type());
  }
#pragma unroll
  for (int i = 0; i < RM; ++i)
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], o);
  // ---- the groups' parts meet in group order: (m, l) and O of groups 1.. in their K and V
  __syncthreads();
  if (group > 0) {
#pragma unroll
    for (int i = 0; i < RM; ++i) {
      const int rr = ty * RM + i;
      if (tx == 0) *reinterpret_cast<float2*>(sK + 2 * rr) = make_float2(m[i], l[i]);
#pragma unroll
      for (int cc = 0; cc < DP / 64; ++cc) store4(sV + rr * DP + cc * 64 + tx * 4, *reinterpret_cast<const float4*>(acc[i] + cc * 4));
    }
  }
  __syncthreads();
  if (group > 0) return;
#pragma unroll
  for (int i = 0; i < RM; ++i) {
    const int rr = r0 + ty * RM + i;
    if (rr >= R) continue;
#pragma unroll
    for (int g = 1; g < NG; ++g) {
      const float2 ml = *reinterpret_cast<const float2*>(sK + g * C::GROUP + 2 * (ty * RM + i));
      if (ml.y == 0.f) continue;  // no key, or none above -inf (a NaN score makes it NaN, m stays -inf)
      const float mn = fmaxf(m[i], ml.x), f = m[i] == -INFINITY ? 0.f : exp2f(m[i] - mn), e = exp2f(ml.x - mn);
      m[i] = mn;
      l[i] = l[i] * f + ml.y * e;
#pragma unroll
      for (int cc = 0; cc < DP / 64; ++cc) {
        const float4 v = load4(sV + g * C::GROUP + (ty * RM + i) * DP + cc * 64 + tx * 4);
        float* o = acc[i] + cc * 4;
        o[0] = o[0] * f + v.x * e;
        o[1] = o[1] * f + v.y * e;
        o[2] = o[2] * f + v.z * e;
        o[3] = o[3] * f + v.w * e;
      }
    }
    const int tok = s.start + rr / G, h = kvh * G + rr % G;
    const float inv = 1.f / l[i];
    float* o = reinterpret_cast<float*>(a.out) + (int64_t)tok * a.o_row + (int64_t)h * a.o_head;
#pragma unroll
    for (int cc = 0; cc < DP / 64; ++cc)
      if (cc * 64 + tx * 4 < a.d)
        store4(o + cc * 64 + tx * 4, make_float4(acc[i][cc * 4] * inv, acc[i][cc * 4 + 1] * inv,
                                                 acc[i][cc * 4 + 2] * inv, acc[i][cc * 4 + 3] * inv));
    if (a.lse && tx == 0)
      a.lse[(int64_t)tok * a.Hq + h] = lse_of(m[i], l[i]);
  }
}

// Merge of the splits' partials, in split order: one warp per (token, head),
// lanes over the columns.
__global__ void __launch_bounds__(256) k_attn_simt_merge(Ragged r, AttnCall a, int splits) {
  pdl_trigger();
  pdl_wait();
  const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31, tok = (int)(w / a.Hq), h = (int)(w % a.Hq);
  if (tok >= r.total) return;
  const int b = seq_of_row(r, tok);
  if (b >= r.batch) return;
  const Seq s = load_seq(r, b);
  if (!s.ok || tok < s.start || tok >= s.start + s.n) return;
  const int ns = max(1, min(splits, (s.len + kSplit - 1) / kSplit));
  const float* p = a.ws + w * splits * (a.d + 4);
  SplitMerge m;
  for (int j = lane; j < ns; j += 32) m.max(p[(int64_t)j * (a.d + 4)]);
  m.M = warp_max(m.M);
  const int col = 4 * lane < a.d ? 4 * lane : 0;
#pragma unroll 4
  for (int j = 0; j < ns; ++j) {
    const float* q = p + (int64_t)j * (a.d + 4);
    m.add(*reinterpret_cast<const float2*>(q), load4(q + 4 + col));
  }
  m.store(a, tok, h, 4 * lane);
}

bool few_rows(const Ragged& r, const AttnCall& a) { return (int64_t)r.max_rows * (a.Hq / a.Hkv) <= kFewRows; }
// (16 CTAs leave SMs of a GPC empty: one token each of 64 sequences over 3900 292 us
// through the workspace, 371 in clusters of 16; over 1900 151 and 155, of 1 16.5 and 13)
constexpr int kMaxSplitCluster = 8;
// CTAs of a cluster that holds all splits; 1: too many, they meet in the workspace
int split_cluster(int splits) {
  int c = 1;
  while (c < splits) c *= 2;
  return c <= kMaxSplitCluster ? c : 1;
}
int simt_splits(const Ragged& r, const AttnCall& a) { return few_rows(r, a) ? (r.max_len + kSplit - 1) / kSplit : 1; }

template <typename K>
cudaError_t allow_smem(K kernel, size_t smem, std::atomic<bool> (&done)[64]) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (dev < 64 && done[dev])) return e;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess && dev < 64) done[dev] = true;
  return e;
}

template <int DP>
cudaError_t launch_simt(const Ragged& r, const AttnCall& a, const KVView& kv, cudaStream_t st) {
  const int64_t rows = (int64_t)r.max_rows * (a.Hq / a.Hkv);
  if (!few_rows(r, a)) {
    using C = TileCfg<DP>;
    static std::atomic<bool> done[64];
    if (cudaError_t e = allow_smem(k_attn_tiles<DP>, C::SMEM, done)) return e;
    const int64_t tiles = (rows + C::BR - 1) / C::BR;
    return launch_k(k_attn_tiles<DP>, (unsigned)(tiles * r.batch * a.Hkv), C::NG * 128, C::SMEM, st, r, a, kv);
  }
  const int splits = simt_splits(r, a), cluster = split_cluster(splits);
  auto few = [&](auto br, std::atomic<bool> (&done)[64]) {
    constexpr int BR = decltype(br)::value;
    constexpr size_t smem = FewCfg<DP, BR>::SMEM;
    if (cudaError_t e = allow_smem(k_attn_few<DP, BR>, smem, done)) return e;
    return launch_kc(k_attn_few<DP, BR>, dim3((unsigned)((rows + BR - 1) / BR * (cluster > 1 ? cluster : splits)), a.Hkv, r.batch),
                     256, smem, st, cluster, r, a, kv, splits, cluster);
  };
  static std::atomic<bool> done4[64], done8[64], done16[64];
  const cudaError_t e = rows <= 4   ? few(std::integral_constant<int, 4>(), done4)
                        : rows <= 8 ? few(std::integral_constant<int, 8>(), done8)
                                    : few(std::integral_constant<int, 16>(), done16);
  if (e != cudaSuccess || splits == 1 || cluster > 1) return e;
  return launch_k(k_attn_simt_merge, (unsigned)(((int64_t)r.total * a.Hq + 7) / 8), 256, 0, st, r, a, splits);
}

}  // namespace

int64_t attn_simt_workspace(const Ragged& r, const AttnCall& a) {
  const int64_t splits = simt_splits(r, a);
  return splits == 1 || split_cluster((int)splits) > 1 ? 0 : (int64_t)r.total * a.Hq * splits * (a.d + 4) * 4;
}

cudaError_t launch_attn_simt(const Ragged& r, const AttnCall& a, const KVView& kv, cudaStream_t st) {
  return a.d <= 64 ? launch_simt<64>(r, a, kv, st) : launch_simt<128>(r, a, kv, st);
}

namespace {

AttnCall make_call(const dflash_attention* a) {
  return AttnCall{a->n_q_heads, a->n_kv_heads, a->head_dim, a->causal, a->window, a->scale, a->q.data, a->q.row_stride,
                  a->q.head_stride, a->out.data, a->out.row_stride, a->out.head_stride, a->lse, (float*)a->workspace};
}

int64_t workspace_of(const dflash_attention* a, const Ragged& r) {
  int64_t tc = 0;
  if (a->dtype == DFLASH_DTYPE_F32) return attn_simt_workspace(r, make_call(a));
  attn_tc_workspace(r, make_call(a), &tc);
  return tc;
}

int run_attention(const char* call, const dflash_attention* a, const Ragged& r, const KVView& kv, cudaStream_t st) {
  if (r.total == 0) return DFLASH_OK;
  if ((int64_t)r.total * a->n_q_heads > INT32_MAX) return rfail(DFLASH_ERR_SHAPE, call, "total_rows x n_q_heads above 2^31 - 1");
  const int64_t rows = (int64_t)r.max_rows * (a->n_q_heads / a->n_kv_heads);
  if (a->dtype == DFLASH_DTYPE_F32 && (rows + 31) / 32 * r.batch > INT32_MAX / a->n_kv_heads)
    return rfail(DFLASH_ERR_SHAPE, call, "max_rows x batch x n_q_heads / 32 above 2^31 - 1");
  const AttnCall c = make_call(a);
  const int64_t need = workspace_of(a, r);
  if (need > 0 && (!a->workspace || a->workspace_bytes < need || (uintptr_t)a->workspace % 32))
    return rfail(DFLASH_ERR_INVALID_ARG, call, "workspace: 32-byte aligned, at least dflash_attention_workspace bytes");
  return rcheck(a->dtype == DFLASH_DTYPE_F32 ? launch_attn_simt(r, c, kv, st) : launch_attn_tc(r, c, kv, st), call);
}

}  // namespace
}  // namespace dfl

using namespace dfl;

extern "C" {

DFLASH_API int dflash_kv_append(const dflash_kv_pages* pages, const dflash_ragged* batch, const dflash_heads* k,
                                const dflash_heads* v, void* stream) {
  const char* call = "dflash_kv_append";
  if (int rc = check_pages(call, pages)) return rc;
  if (int rc = check_ragged(call, batch, pages, true)) return rc;
  const bool rows = batch->total_rows > 0;
  if (int rc = check_heads(call, k, pages->dtype, pages->n_kv_heads, pages->head_dim, rows)) return rc;
  if (int rc = check_heads(call, v, pages->dtype, pages->n_kv_heads, pages->head_dim, rows)) return rc;
  if (!rows) return DFLASH_OK;
  const Ragged r = make_ragged(batch, pages);
  const int per = 16 / esize(pages->dtype);  // elements of 16 bytes
  int shift = 0;
  while ((1 << shift) < pages->page_size) ++shift;
  return rcheck(launch_k(k_kv_append, (unsigned)((r.total + 7) / 8), 256, 0, (cudaStream_t)stream, r,
                         (const uint4*)k->data, (const uint4*)v->data, k->row_stride / per, k->head_stride / per,
                         v->row_stride / per, v->head_stride / per, (uint4*)pages->k, (uint4*)pages->v,
                         pages->page_stride / per, pages->slot_stride / per, pages->head_stride / per, shift,
                         (int)pages->n_pages, (int)pages->n_kv_heads, (int)(pages->head_dim / per)),
                call);
}

DFLASH_API int64_t dflash_attention_workspace(const dflash_attention* a, const dflash_ragged* batch,
                                              const dflash_kv_pages* pages) {
  const char* call = "dflash_attention_workspace";
  if (int rc = check_attention(call, a, false, false)) return rc;
  if (int rc = check_ragged(call, batch, pages, false)) return rc;
  if (pages && (pages->page_size < 8 || pages->page_size > 1024 || !pow2(pages->page_size)))
    return rfail(DFLASH_ERR_SHAPE, call, "page_size: a power of two in 8..1024");
  const Ragged r = make_ragged(batch, pages);
  Ragged paged = r;
  static const int32_t there = 0;
  paged.lens = pages ? &there : nullptr;  // only its presence counts here
  return workspace_of(a, paged);
}

DFLASH_API int dflash_paged_attention(const dflash_attention* a, const dflash_ragged* batch,
                                      const dflash_kv_pages* pages, void* stream) {
  const char* call = "dflash_paged_attention";
  if (int rc = check_pages(call, pages)) return rc;
  if (int rc = check_ragged(call, batch, pages, true)) return rc;
  if (int rc = check_attention(call, a, true, batch->total_rows > 0)) return rc;
  if (a->dtype != pages->dtype || a->n_kv_heads != pages->n_kv_heads || a->head_dim != pages->head_dim)
    return rfail(DFLASH_ERR_SHAPE, call, "the pages' dtype, n_kv_heads or head_dim is not the attention's");
  int shift = 0;
  while ((1 << shift) < pages->page_size) ++shift;
  const KVView kv{pages->k, pages->v, pages->slot_stride, pages->head_stride, pages->slot_stride, pages->head_stride,
                  pages->page_stride, shift, (int32_t)pages->n_pages, 1, 0};
  return run_attention(call, a, make_ragged(batch, pages), kv, (cudaStream_t)stream);
}

DFLASH_API int dflash_prompt_attention(const dflash_attention* a, const dflash_ragged* batch, const dflash_heads* k,
                                       const dflash_heads* v, void* stream) {
  const char* call = "dflash_prompt_attention";
  if (int rc = check_ragged(call, batch, nullptr, true)) return rc;
  const bool rows = batch->total_rows > 0;
  if (int rc = check_attention(call, a, true, rows)) return rc;
  if (int rc = check_heads(call, k, a->dtype, a->n_kv_heads, a->head_dim, rows)) return rc;
  if (int rc = check_heads(call, v, a->dtype, a->n_kv_heads, a->head_dim, rows)) return rc;
  const KVView kv{k->data, v->data, k->row_stride, k->head_stride, v->row_stride, v->head_stride, 0, 0, 0, 0,
                  batch->total_rows};
  return run_attention(call, a, make_ragged(batch, nullptr), kv, (cudaStream_t)stream);
}

DFLASH_API int dflash_status_check(int32_t* status, void* stream) {
  const char* call = "dflash_status_check";
  if (!status) return rfail(DFLASH_ERR_INVALID_ARG, call, "null status");
  int32_t s = 0;
  cudaStream_t st = (cudaStream_t)stream;
  if (int rc = rcheck(cudaMemcpyAsync(&s, status, 4, cudaMemcpyDeviceToHost, st), call)) return rc;
  if (int rc = rcheck(cudaMemsetAsync(status, 0, 4, st), call)) return rc;
  if (int rc = rcheck(cudaStreamSynchronize(st), call)) return rc;
  if (!s) return DFLASH_OK;
  char buf[200];
  snprintf(buf, sizeof buf, "%s%s%s%s%s", s & DFLASH_STATUS_TOKEN ? "a token id outside the vocabulary; " : "",
           s & DFLASH_STATUS_BOUNDS ? "a sequence outside the batch's bounds; " : "",
           s & DFLASH_STATUS_PAGE ? "a page id outside the cache; " : "",
           s & DFLASH_STATUS_WAIT ? "a bounded wait expired; " : "",
           s & DFLASH_STATUS_FULL ? "no free page left; " : "");
  return rfail(DFLASH_ERR_DEVICE, call, buf);
}

}  // extern "C"
