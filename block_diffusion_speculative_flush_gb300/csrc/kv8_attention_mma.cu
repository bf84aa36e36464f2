// Attention of few rows (single tokens, verified blocks) over an 8-bit paged cache:
// bf16, head_dim 64 or 128.
//
// A warp copies its chunks of 16 keys (cp.async) into a ring of its own and waits for no other
// warp; each lane multiplies 16 bytes of each row that its place in the fragments has.  That works
// because a contraction may take its index in any order and a result its rows in any order:
//   S^T = K Q^T   A = 16 keys of K: lane (g, t) of the m16n8k16 fragment holds keys g and
//                 g + 8 at any 4 d's per step, here 16 bytes in a row of each
//   O^T = V^T P^T A = V^T, 16 d's by 16 keys: lane (g, t) holds keys 2t, 2t + 1, 2t + 8, 2t + 9 at
//                 the d's 16 g .. 16 g + 15, 16 bytes of each key's row
// with N = 8 rows (token, query head of the group) a fragment, so that a decode step's few rows
// fill it.  Codes become fp16 exactly (cvt).  P goes from the first product's result to the
// second one's operand by a transpose of 8 x 8 in registers (movmatrix).
//
// Numbers.  q is scaled by a power of two for its row, so that its largest element lies in
// [2^14, 2^15): fp16 holds bf16's 8 bits for elements down to 2^-29 of that, an error that
// fp32 sums of such products have too.  Scores: (S ks) (scale 2^-e log2 e), fp32.  P is
// rounded to fp16 once, as p (vs / u) 2^10 with p = 2^(s - m) <= 2^4 (the maximum moves only when it grew
// by more).  u is a row's own: the largest p vs of the keys that it sees was between u and 2^4 u when the row met it,
// so neither a scale that it does not see nor one with next to no probability takes bits from the others.
// Half a step is 2^-11 of P or less, below fp16's smallest normal number 2^-25, that is 2^-35 of the row's largest p vs.
// V's scale is a logarithm in the exponent of P, which l takes back: what it adds is P by the inverse of its weight.
// A weight below 2^-64 is taken as that: P is 0 in fp16 either way, and l does not lose the keys (scales lie
// up to 2^120 apart).  m, l, O and merges are fp32.
//
// Work, in one of two ways, by the host's bounds (few_cluster):
//   cluster  a thread-block cluster of 1 to 8 CTAs per (sequence, tile of rows, KV head) item, an even share of
//            its chunks each, the parts meet in distributed shared memory: all items at once, or in turn,
//            longest first (one launch, nothing to search);
//   ranges   the 16-key chunks of all items one after another, cut into even ranges, one per CTA; the parts of a cut
//            item meet in k_kv8_few_merge.
// The 8 warps of a CTA take its chunks in turn and meet in shared memory.  The order of every
// sum is fixed by the lengths.
//
// Bound by memory where calls are long: 64 single tokens over 1k to 16k, 8 KV heads of 128, pages of 16, 665 MB in
// 116 us, 5.7 TB/s (86% of a measured copy; loads in flight and issue slots keep it there).  Short calls are
// latency, the chain length -> table -> scales and codes -> products -> cluster: one user's block of 16 over 4096
// 18.2 us.
#include <cooperative_groups.h>

#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "kv8.h"
#include "launch.h"

namespace dfl {
namespace {

constexpr int kChunk = 16;  // keys of a chunk: never more than a page
constexpr int kWarps = 8;
constexpr int kMaxCluster = 8;
constexpr int kFewRows = 32;   // of a sequence and KV head, for this kernel in any case
constexpr int kMaxShare = 256;  // chunks of a CTA of a cluster where all run at once
constexpr int kSorted = 256;    // sequences that are put in order
namespace cg = cooperative_groups;
constexpr float kSlack = 4.f, kLn2 = 0.6931471805599453f, kLog2e = 1.4426950408889634f;
constexpr float kUnitLog2 = 10.f;  // of P in fp16
constexpr float kNoMax = -3.402823466e38f, kNoUnit = -1000.f;  // before the first key: finite, so that no difference is a NaN

struct FewPlan {
  int32_t cluster;    // CTAs of an item; 0: ranges
  int32_t in_turn;    // cluster: more CTAs than run at once
  int32_t tiles;      // cluster: tiles of rows that a sequence may have
  int32_t pad;        // what the start of an item costs, in chunks
  int32_t min_units;  // chunks that a CTA gets at least
  int32_t slots;      // partials there is room for
};

template <int D, int NB>
struct FewCfg {
  static constexpr int RB = 8 * NB;               // rows of a tile
  static constexpr int CTAS = NB <= 2 ? 2 : 1;    // of an SM
  static constexpr int BYTES = kChunk * 2 * D;    // codes of a chunk
  static constexpr int STAGES = (NB <= 2 ? 3 : 5) * (128 / D);
  static constexpr int SCALES = 64;               // of a warp's chunks: those looked up last and the 32 before
  static_assert(STAGES < 32, "a chunk in use was looked up at most once ago");
  static constexpr int LO = D + 4;                // floats of a row where the warps meet
  static constexpr int RING = kWarps * STAGES * BYTES, MEET = kWarps * RB * LO * 4, PART = RB * D * 4;
  static constexpr int AREA = RING > MEET + PART ? RING : MEET + PART;
  static constexpr bool QS = NB > 1;              // q's fragments in shared memory (registers otherwise)
  static constexpr int QF = QS ? NB * (D / 16) * 32 * 8 : 0;
  static constexpr size_t SMEM = AREA + QF + NB * 8 * 4 + kWarps * SCALES * 8 + kWarps * RB * 8 + RB * 8;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
template <int N> __device__ __forceinline__ void cp_async(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(N) : "memory");
}
template <int N> __device__ __forceinline__ void cp_async(uint32_t dst, const void* src, bool there) {
  // (size 0: zeros, the address is not looked at)
  asm volatile("cp.async.cg.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(N), "r"(there ? N : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// D += A B, m16n8k16, fp16 operands, fp32 sums
__device__ __forceinline__ void mma(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_h2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// ---------------------------------------------------------------------------
// the layout of the work
// ---------------------------------------------------------------------------
__device__ __forceinline__ int64_t few_tiles(const Seq& s, int G, int RB) {
  return s.ok && s.n > 0 ? ((int64_t)s.n * G + RB - 1) / RB : 0;
}
__device__ __forceinline__ int few_first(const Seq& s, int window) { return vis_lo(s.len - s.n, window) / kChunk; }
__device__ __forceinline__ int few_chunks(const Seq& s, int window) {
  return (s.len + kChunk - 1) / kChunk - few_first(s, window);
}
__device__ __forceinline__ int64_t warp_sum64(int64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ int64_t warp_scan64(int64_t v, int lane) {  // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}
struct FewRanges {
  int64_t units, each, rest;
  int n;
  __device__ __forceinline__ FewRanges(int64_t u, const FewPlan& p, int grid) {
    units = u;
    n = (int)max((int64_t)1, min((int64_t)grid, u / p.min_units));
    each = u / n;
    rest = u - each * n;
  }
  __device__ __forceinline__ int64_t start(int c) const { return c * each + min((int64_t)c, rest); }
  __device__ __forceinline__ int of(int64_t u) const {
    const int64_t head = rest * (each + 1);
    return (int)(u < head ? u / (each + 1) : rest + (u - head) / each);
  }
};
__device__ __forceinline__ Seq few_bcast(const Seq& s, int src) {
  Seq o;
  o.start = __shfl_sync(0xffffffffu, s.start, src);
  o.n = __shfl_sync(0xffffffffu, s.n, src);
  o.len = __shfl_sync(0xffffffffu, s.len, src);
  o.ok = __shfl_sync(0xffffffffu, (int)s.ok, src) != 0;
  return o;
}
// Partials: O in ws [slots][RB][D], (m, l) behind it, [slots][RB].
template <int D, int RB> __device__ __forceinline__ float* few_o(const AttnCall& a, int slot, int row) {
  return a.ws + ((int64_t)slot * RB + row) * D;
}
template <int D, int RB> __device__ __forceinline__ float2* few_ml(const AttnCall& a, const FewPlan& p, int slot, int row) {
  return reinterpret_cast<float2*>(a.ws + (int64_t)p.slots * RB * D) + (int64_t)slot * RB + row;
}
__device__ __forceinline__ float lse_of(float m, float l) { return (m + log2f(l)) * kLn2; }
// (m, l) for a merge: a part with a NaN score has l NaN, and m may still be -inf, what a part without a key
// has; NaN, it cannot be taken for one.
__device__ __forceinline__ float2 part_stats(float m, float l) { return make_float2(l != l ? l : m, l); }

template <int D> __device__ __forceinline__ void store_row(const AttnCall& a, int tok, int h, int lane, const float* v, float f) {
  constexpr int C = D / 32;
  bf16* o = reinterpret_cast<bf16*>(a.out) + (int64_t)tok * a.o_row + (int64_t)h * a.o_head + lane * C;
#pragma unroll
  for (int j = 0; j < C; j += 2) *reinterpret_cast<__nv_bfloat162*>(o + j) = __floats2bfloat162_rn(v[j] * f, v[j + 1] * f);
}

template <int D, int NB>
__global__ void __launch_bounds__(kWarps * 32, FewCfg<D, NB>::CTAS) k_kv8_few(Ragged r, AttnCall a, Kv8View kv, FewPlan plan) {
  using C = FewCfg<D, NB>;
  constexpr int RB = C::RB, S = C::STAGES, KS = D / 16, MT = D / 16;  // steps of the first product, tiles of the second
  constexpr int VB = D / 8, VW = VB / 4;                              // bytes and words of a lane's piece of a V row
  constexpr int CC = D / 32;                                          // columns of a lane where rows are put together
  extern __shared__ __align__(16) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  uint8_t* ring = smem + warp * S * C::BYTES;                     // this warp's stages
  float* meet = reinterpret_cast<float*>(smem);                   // [warps][RB][LO]
  float* part_o = reinterpret_cast<float*>(smem + C::MEET);       // [RB][D] this CTA's sums (cluster)
  uint2* s_qf = reinterpret_cast<uint2*>(smem + C::AREA);         // [NB][KS][32]
  float* s_rowf = reinterpret_cast<float*>(smem + C::AREA + C::QF);  // [RB]
  float2* scales = reinterpret_cast<float2*>(s_rowf + RB) + warp * C::SCALES;  // ks, log2 vs of a chunk's page
  float2* s_ml = reinterpret_cast<float2*>(s_rowf + RB) + kWarps * C::SCALES;  // [warps][RB]
  float2* part_ml = s_ml + kWarps * RB;                           // [RB]
  pdl_trigger();
  pdl_wait();
  r.starts = after_wait(r.starts);
  r.lens = after_wait(r.lens);
  r.table = after_wait(r.table);
  const int G = a.Hq / a.Hkv, cta = blockIdx.x, grid = gridDim.x;
  const float sl2 = a.scale * kLog2e;
  // One stretch of an item: rows rt RB .. of sequence b, chunks [c0, c0 + take) behind its first.  The rows' sums
  // end in memory, or (part >= 0) unscaled in a partial, or (part == -2) in this CTA's part_o and part_ml.
  auto stretch = [&](const Seq& s, int b, int rt, int kvh, int c0, int take, int part) {
    const int r0 = rt * RB, ctx = s.len - s.n, R = (int)min((int64_t)RB, (int64_t)s.n * G - r0);
    const int p_first = ctx + r0 / G, p_last = ctx + (r0 + R - 1) / G;
    const int k_lo = vis_lo(p_first, a.window), k_hi = vis_hi(p_last, s.len, a.causal);
    const int clean_lo = vis_lo(p_last, a.window), clean_hi = vis_hi(p_first, s.len, a.causal);
    const int first_key = (few_first(s, a.window) + c0 + warp) * kChunk;  // chunk i of this warp: + 128 i
    const int n_mine = take > warp ? (take - warp + kWarps - 1) / kWarps : 0;
    const int32_t* tab = r.table + (int64_t)b * r.table_stride;
    // pages and scales of this warp's next 32 chunks, one a lane
    int pg = -1;
    auto look_up = [&](int i0) {
      const int i = i0 + lane, key = first_key + kWarps * kChunk * i;
      float ks = 1.f, vs = 0.f;
      pg = -1;
      if (i < n_mine && key < k_hi && key + kChunk > k_lo) {
        pg = tab[key >> kv.page_shift];
        if (pg < 0 || pg >= kv.n_pages) {
          flag_status(r.status, DFLASH_STATUS_PAGE);
          pg = -1;
        } else {
          ks = kv.ks[pg * kv.s_page + kvh * kv.s_head];
          vs = kv.vs[pg * kv.s_page + kvh * kv.s_head];
        }
      }
      scales[i % C::SCALES] = make_float2(ks, scale_log2(vs));
    };
    // What this lane copies: 16 bytes of every RI-th row, as many lanes side by side as a row has, so that memory
    // sees whole rows (32 bytes of four rows in eight lanes, the pieces that a lane multiplies, reached half the
    // rate).  Row r's 16-byte chunk c lies at chunk c ^ (r mod 8) (64-byte rows: c ^ (r / 2 mod 4)), which no
    // reader meets another's bank at.
    constexpr int CH = D / 16, RI = 32 / CH, NI = kChunk / RI;  // chunks of a row, rows and instructions of a copy
    const int row_l = lane / CH, chunk_l = lane % CH;
    const uint8_t* k_base = kv.k + kvh * kv.head + row_l * kv.slot + 16 * chunk_l;
    const uint8_t* v_base = kv.v + kvh * kv.head + row_l * kv.slot + 16 * chunk_l;
    const int64_t rows_st = RI * kv.slot;
    auto place = [](int r, int c) { return r * D + ((D == 128 ? c ^ (r & 7) : c ^ ((r >> 1) & 3)) << 4); };
    const uint32_t dst0 = smem_addr(ring) + place(row_l, chunk_l), dst1 = smem_addr(ring) + place(row_l + RI, chunk_l);
    // what it reads: of K rows g and g + 8, of V rows 2t, 2t + 1, 2t + 8, 2t + 9
    const int k_at0 = place(g, D == 128 ? 2 * t : t), k_at1 = place(g, 2 * t + 1);
    const int v_at0 = kChunk * D + (D == 128 ? place(2 * t, g) : place(2 * t, g >> 1) + (g & 1) * 8);
    const int v_at1 = kChunk * D + (D == 128 ? place(2 * t + 1, g) : place(2 * t + 1, g >> 1) + (g & 1) * 8);
    uint32_t to = 0;  // the stage that is filled next
    auto issue = [&](int i) {  // chunk i
      if (i < n_mine) {
        if ((i & 31) == 0) look_up(i);
        const int page = __shfl_sync(0xffffffffu, pg, i & 31), key0 = first_key + kWarps * kChunk * i;
        const int64_t at = page * kv.page + (int64_t)(key0 & ((1 << kv.page_shift) - 1)) * kv.slot;
        const uint8_t* kp = k_base + at;
        const uint8_t* vp = v_base + at;
        if (page >= 0 && key0 >= k_lo && key0 + kChunk <= k_hi) {
#pragma unroll
          for (int q = 0; q < NI; ++q) {
            const uint32_t d = (q & 1 ? dst1 - RI * D : dst0) + to + q * RI * D;
            cp_async<16>(d, kp);
            cp_async<16>(d + kChunk * D, vp);
            kp += rows_st;
            vp += rows_st;
          }
        } else {  // (keys that no row of the tile sees arrive as zeros)
#pragma unroll
          for (int q = 0; q < NI; ++q) {
            const uint32_t d = (q & 1 ? dst1 - RI * D : dst0) + to + q * RI * D;
            const int key = key0 + q * RI + row_l;
            const bool seen = page >= 0 && key >= k_lo && key < k_hi;
            cp_async<16>(d, kp, seen);
            cp_async<16>(d + kChunk * D, vp, seen);
            kp += rows_st;
            vp += rows_st;
          }
        }
        to = to == (S - 1) * C::BYTES ? 0 : to + C::BYTES;
      }
      cp_commit();
    };
#pragma unroll 1
    for (int i = 0; i < S - 1; ++i) issue(i);
    // ---- q: lane (g, t) has rows g (+ 8 n) at the d's that it has of K
    uint32_t qf[C::QS ? 1 : NB][KS][2];
    float rowf[NB][2];  // of rows 2t, 2t + 1: scale 2^-e log2 e
    auto make_q = [&](int n, uint32_t (*f16)[2]) {
      const int row = 8 * n + g;
      uint4 w[D / 32];
#pragma unroll
      for (int c = 0; c < D / 32; ++c) w[c] = make_uint4(0, 0, 0, 0);
      if (row < R) {
        const int i = (r0 + row) / G, h = kvh * G + (r0 + row) % G;
        const bf16* q = reinterpret_cast<const bf16*>(a.q) + (int64_t)(s.start + i) * a.q_row + (int64_t)h * a.q_head;
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
#pragma unroll
          for (int k = 0; k < 2; ++k)
            w[2 * c + k] = *reinterpret_cast<const uint4*>(q + (D == 128 ? 32 * t + 16 * c : 16 * t) + 8 * k);
      }
      const uint32_t* ww = reinterpret_cast<const uint32_t*>(w);
      float most = 0.f;
#pragma unroll
      for (int k = 0; k < D / 8; ++k) {
        const float x = fabsf(__uint_as_float(ww[k] << 16)), y = fabsf(__uint_as_float(ww[k] & 0xffff0000u));
        most = fmaxf(most, fmaxf(nonfinite(x) ? 0.f : x, nonfinite(y) ? 0.f : y));
      }
      most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
      most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
      // most 2^e in [2^14, 2^15); 2^e in two factors, either of them a normal number
      const int e = most > 0.f ? 14 - ilogbf(most) : 0, e0 = e / 2;
      const float f0 = ldexpf(1.f, e0), f1 = ldexpf(1.f, e - e0);
#pragma unroll
      for (int k = 0; k < D / 8; ++k)
        f16[k / 2][k & 1] = pack_h2(__uint_as_float(ww[k] << 16) * f0 * f1, __uint_as_float(ww[k] & 0xffff0000u) * f0 * f1);
      return ldexpf(sl2, -e);
    };
    if constexpr (C::QS) {
      if (warp < NB) {  // a tile of rows a warp, for all of them
        uint32_t f16[KS][2];
        const float f = make_q(warp, f16);
#pragma unroll
        for (int k = 0; k < KS; ++k) s_qf[(warp * KS + k) * 32 + lane] = make_uint2(f16[k][0], f16[k][1]);
        if (t == 0) s_rowf[8 * warp + g] = f;
      }
      __syncthreads();
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        rowf[n][0] = s_rowf[8 * n + 2 * t];
        rowf[n][1] = s_rowf[8 * n + 2 * t + 1];
      }
    } else {
      const float f = make_q(0, qf[0]);
      // rows 2t, 2t + 1 of this tile are those of lanes g = 2t, 2t + 1
      rowf[0][0] = __shfl_sync(0xffffffffu, f, 8 * t);
      rowf[0][1] = __shfl_sync(0xffffffffu, f, 8 * t + 4);
    }
    float o[NB][MT][4], m[NB][2], l[NB][2], lu[NB][2];  // lu: log2 of the unit of p vs
#pragma unroll
    for (int n = 0; n < NB; ++n) {
#pragma unroll
      for (int k = 0; k < MT; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[n][k][j] = 0.f;
      m[n][0] = m[n][1] = kNoMax;
      lu[n][0] = lu[n][1] = kNoUnit;
      l[n][0] = l[n][1] = 0.f;
    }
    uint32_t from = 0;  // the stage that is read next
    auto scores = [&](const uint8_t* stage, const float2& sc, float (*x)[4]) {
      constexpr int CHAINS = NB == 1 ? 2 : 1;  // of dependent products a tile of rows
      float two[CHAINS][NB][4];
#pragma unroll
      for (int p = 0; p < CHAINS; ++p)
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
          for (int j = 0; j < 4; ++j) two[p][n][j] = 0.f;
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        const uint8_t* kp = stage + (c ? k_at1 : k_at0);
        const uint4 k0 = *reinterpret_cast<const uint4*>(kp), k8 = *reinterpret_cast<const uint4*>(kp + 8 * D);
        const uint32_t w0[4] = {k0.x, k0.y, k0.z, k0.w}, w8[4] = {k8.x, k8.y, k8.z, k8.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t a0, a1, a2, a3;
          e4m3x4_to_h4(w0[j], a0, a2);
          e4m3x4_to_h4(w8[j], a1, a3);
#pragma unroll
          for (int n = 0; n < NB; ++n) {
            if constexpr (C::QS) {
              const uint2 q = s_qf[(n * KS + 4 * c + j) * 32 + lane];
              mma(two[j % CHAINS][n], a0, a1, a2, a3, q.x, q.y);
            } else {
              mma(two[j % CHAINS][n], a0, a1, a2, a3, qf[n][4 * c + j][0], qf[n][4 * c + j][1]);
            }
          }
        }
      }
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) x[n][j] = (CHAINS == 2 ? two[0][n][j] + two[CHAINS - 1][n][j] : two[0][n][j]) * sc.x * rowf[n][j & 1];
    };
    auto sees = [&](int n, int j, int key) {  // row 2t + (j & 1) of tile n
      const int row = r0 + 8 * n + 2 * t + (j & 1), p = ctx + row / G;
      return row < r0 + R && key >= vis_lo(p, a.window) && key < vis_hi(p, s.len, a.causal);
    };
#pragma unroll 1
    for (int i = 0; i < n_mine; ++i) {
      cp_wait<S - 2>();
      __syncwarp();  // (what a lane reads has come through others; what is overwritten now has been read)
      issue(i + S - 1);
      const uint8_t* stage = ring + from;
      from = from == (S - 1) * C::BYTES ? 0 : from + C::BYTES;
      const float2 sc = scales[i % C::SCALES];
      const int key0 = first_key + kWarps * kChunk * i;
      const bool clean = key0 >= clean_lo && key0 + kChunk <= clean_hi;
      float x[NB][4];
      scores(stage, sc, x);
      if (!clean) {
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (!sees(n, j, key0 + g + (j >> 1) * 8)) x[n][j] = -INFINITY;
      }
      // ---- the maximum and the unit move when a score, or p vs, is more than 2^kSlack above them
      bool grow = false;
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) grow |= fmaxf(x[n][j], x[n][j + 2]) - m[n][j] + fmaxf(sc.y - lu[n][j], 0.f) > kSlack;
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float mx = fmaxf(x[n][j], x[n][j + 2]);
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
            // the unit so far, from the new maximum: O stays what it is where that will do.  (Before the first key
            // sums are 0 or NaN, and their factors 0.)
            const float mn = mx > m[n][j] + kSlack ? mx : m[n][j], shift = m[n][j] - mn, was = lu[n][j] + shift;
            const float top = mx - mn + sc.y, unit = top > was + kSlack ? top : was, f = ex2(was - unit);
            m[n][j] = mn;
            lu[n][j] = unit;
            l[n][j] *= ex2(shift);
#pragma unroll
            for (int k = 0; k < MT; ++k) {
              o[n][k][j] *= f;
              o[n][k][j + 2] *= f;
            }
          }
      }
      // ---- P, its sums, and P^T as the second product's operand
      uint32_t pb[NB][2];
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        float p[4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float w = fmaxf(sc.y - lu[n][j], -64.f) + kUnitLog2, c = w - m[n][j];
          p[j] = ex2(x[n][j] + c);
          p[j + 2] = ex2(x[n][j + 2] + c);
          l[n][j] = fmaf(p[j] + p[j + 2], ex2(-w), l[n][j]);
        }
        pb[n][0] = transpose8(pack_h2(p[0], p[1]));
        pb[n][1] = transpose8(pack_h2(p[2], p[3]));
      }
      // ---- O^T
      uint32_t vw[4][VW];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint8_t* vp = stage + (q & 1 ? v_at1 : v_at0) + (q >> 1) * 8 * D;
        if constexpr (VW == 4) {
          const uint4 v = *reinterpret_cast<const uint4*>(vp);
          vw[q][0] = v.x, vw[q][1] = v.y, vw[q][2] = v.z, vw[q][3] = v.w;
        } else {
          const uint2 v = *reinterpret_cast<const uint2*>(vp);
          vw[q][0] = v.x, vw[q][1] = v.y;
        }
      }
      if (!clean) {
        // A key that a row does not see may hold a NaN, and 0 x NaN is NaN: such codes become 0, and the rows
        // that do see them get the NaN by hand.
        uint32_t found = 0;
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int k = 0; k < VW; ++k) found |= nan_codes(vw[q][k]);
        if (__any_sync(0xffffffffu, found != 0)) {
#pragma unroll 1
          for (int st = 0; st < 4; ++st)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int key = key0 + 2 * st + (q & 1) + 8 * (q >> 1);
#pragma unroll
              for (int k = 0; k < VW; ++k) {
                const uint32_t bad = nan_codes(__shfl_sync(0xffffffffu, vw[q][k], 4 * g + st));
#pragma unroll
                for (int e = 0; e < 4; ++e)  // d VB g + 4 k + e: tile 2 k + e / 2, its row g + 8 (e & 1)
                  if ((bad >> (8 * e + 7)) & 1u)
#pragma unroll
                    for (int n = 0; n < NB; ++n)
#pragma unroll
                      for (int j = 0; j < 2; ++j)
                        if (sees(n, j, key)) o[n][2 * k + e / 2][2 * (e & 1) + j] = __uint_as_float(0x7fffffffu);
              }
            }
#pragma unroll
          for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int k = 0; k < VW; ++k) vw[q][k] = without_nan(vw[q][k]);
        }
      }
#pragma unroll
      for (int k = 0; k < VW; ++k) {
        const uint32_t e0 = __byte_perm(vw[0][k], vw[1][k], 0x5140), e1 = __byte_perm(vw[0][k], vw[1][k], 0x7362);
        const uint32_t f0 = __byte_perm(vw[2][k], vw[3][k], 0x5140), f1 = __byte_perm(vw[2][k], vw[3][k], 0x7362);
        uint32_t a0, a1, a2, a3, b0, b1, b2, b3;
        e4m3x4_to_h4(e0, a0, a1);
        e4m3x4_to_h4(f0, a2, a3);
        e4m3x4_to_h4(e1, b0, b1);
        e4m3x4_to_h4(f1, b2, b3);
#pragma unroll
        for (int n = 0; n < NB; ++n) {
          mma(o[n][2 * k], a0, a1, a2, a3, pb[n][0], pb[n][1]);
          mma(o[n][2 * k + 1], b0, b1, b2, b3, pb[n][0], pb[n][1]);
        }
      }
    }
    cp_wait<0>();
    // ---- the warps meet: O [row][d] and (m, l) of each
    __syncthreads();  // every warp has read its ring
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float sum = l[n][j];
        sum += __shfl_xor_sync(0xffffffffu, sum, 4);
        sum += __shfl_xor_sync(0xffffffffu, sum, 8);
        sum += __shfl_xor_sync(0xffffffffu, sum, 16);
        const int row = 8 * n + 2 * t + j;
        if (g == 0) s_ml[warp * RB + row] = part_stats(m[n][j] == kNoMax ? -INFINITY : m[n][j], sum);
        float* dst = meet + (warp * RB + row) * C::LO + VB * g;
        const float f = ex2(lu[n][j] - kUnitLog2);
#pragma unroll
        for (int k = 0; k < MT; k += 2)
          *reinterpret_cast<float4*>(dst + 2 * k) =
              make_float4(o[n][k][j] * f, o[n][k][j + 2] * f, o[n][k + 1][j] * f, o[n][k + 1][j + 2] * f);
      }
    __syncthreads();
    for (int row = warp; row < R; row += kWarps) {
      float2 ml = make_float2(-INFINITY, 0.f);
      if (lane < kWarps) ml = s_ml[lane * RB + row];
      const float M = warp_max(ml.x);
      // a warp that saw no key has weight 0, the NaN of one with a NaN score stays one
      const float wt = ml.x == -INFINITY ? 0.f : exp2f(ml.x - M);
      const float L = warp_sum(wt == 0.f ? 0.f : ml.y * wt);
      const uint32_t saw = __ballot_sync(0xffffffffu, ml.y != 0.f);
      float sum[CC];
#pragma unroll
      for (int j = 0; j < CC; ++j) sum[j] = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float ww = __shfl_sync(0xffffffffu, wt, w);
        const float* v = meet + (w * RB + row) * C::LO + lane * CC;
        // (a weight that underflows still takes its sums along: 0 x NaN is NaN)
#pragma unroll
        for (int j = 0; j < CC; ++j) sum[j] = fmaf(ww, (saw >> w) & 1u ? v[j] : 0.f, sum[j]);
      }
      const int tok = s.start + (r0 + row) / G, h = kvh * G + (r0 + row) % G;
      if (part == -1) {
        store_row<D>(a, tok, h, lane, sum, 1.f / L);
        if (a.lse && lane == 0) a.lse[(int64_t)tok * a.Hq + h] = lse_of(M, L);
      } else {
        float* w = (part >= 0 ? few_o<D, RB>(a, part, row) : part_o + row * D) + lane * CC;
#pragma unroll
        for (int j = 0; j < CC; ++j) w[j] = sum[j];
        if (lane == 0) *(part >= 0 ? few_ml<D, RB>(a, plan, part, row) : part_ml + row) = part_stats(M, L);
      }
    }
  };

  if (plan.cluster > 0) {
    // ---- rank q of the cluster takes an even share of the item's chunks; the ranks finish its rows in turn
    cg::cluster_group cl = cg::this_cluster();
    const int N = plan.cluster, item = cta / N, q = cta - item * N, rest = item / a.Hkv, kvh = item - rest * a.Hkv;
    const int turn = rest / plan.tiles, rt = rest - turn * plan.tiles;
    // Items that wait for their turn go longest first: sequence b is the turn-th by chunks.
    int b = turn;
    if (plan.in_turn && r.batch <= kSorted) {
      int* size = reinterpret_cast<int*>(smem);  // [kSorted]
      int* found = size + kSorted;
      int mine = -1;
      if (tid < r.batch) {
        const Seq s = load_seq(r, tid);
        mine = s.ok && s.n > 0 ? few_chunks(s, a.window) : 0;
      }
      size[tid] = mine;
      __syncthreads();
      if (tid < r.batch) {
        int before = 0;
#pragma unroll 4
        for (int j = 0; j < r.batch; ++j) before += size[j] > mine || (size[j] == mine && j < tid);
        if (before == turn) *found = tid;
      }
      __syncthreads();
      b = *found;
      __syncthreads();  // (the ring begins here)
    }
    const Seq s = load_seq(r, b);
    if (!s.ok && tid == 0 && rt == 0 && kvh == 0 && q == 0) flag_status(r.status, DFLASH_STATUS_BOUNDS);
    const int R = s.ok ? (int)max((int64_t)0, min((int64_t)RB, (int64_t)s.n * G - (int64_t)rt * RB)) : 0;
    if (R == 0) return;  // (the whole cluster: nobody waits)
    const int T = few_chunks(s, a.window), c0 = (int)((int64_t)T * q / N), c1 = (int)((int64_t)T * (q + 1) / N);
    stretch(s, b, rt, kvh, c0, c1 - c0, N == 1 ? -1 : -2);
    if (N == 1) return;
    cl.sync();
    for (int row = q + N * warp; row < R; row += N * kWarps) {
      float2 ml = make_float2(-INFINITY, 0.f);
      if (lane < N) ml = *cl.map_shared_rank(part_ml + row, lane);
      const float M = warp_max(ml.x), wt = ml.x == -INFINITY ? 0.f : exp2f(ml.x - M);
      const float L = warp_sum(wt == 0.f ? 0.f : ml.y * wt);
      const uint32_t saw = __ballot_sync(0xffffffffu, ml.y != 0.f);
      float sum[CC];
#pragma unroll
      for (int j = 0; j < CC; ++j) sum[j] = 0.f;
#pragma unroll 4
      for (int u = 0; u < N; ++u) {
        const float wu = __shfl_sync(0xffffffffu, wt, u);
        const float* v = cl.map_shared_rank(part_o, u) + row * D + lane * CC;
#pragma unroll
        for (int j = 0; j < CC; ++j) sum[j] = fmaf(wu, (saw >> u) & 1u ? v[j] : 0.f, sum[j]);
      }
      const int tok = s.start + (rt * RB + row) / G, h = kvh * G + (rt * RB + row) % G;
      store_row<D>(a, tok, h, lane, sum, 1.f / L);
      if (a.lse && lane == 0) a.lse[(int64_t)tok * a.Hq + h] = lse_of(M, L);
    }
    cl.sync();  // no CTA leaves while a peer reads its part
    return;
  }
  // ---- ranges: every warp lays the work out for itself
  const bool one = r.batch <= 32;
  Seq mine{0, 0, 0, false};
  if (one && lane < r.batch) mine = load_seq(r, lane);
  auto seq_at = [&](int b) { return one ? mine : load_seq(r, b); };
  auto units_of = [&](const Seq& s) {
    return s.ok && s.n > 0 ? few_tiles(s, G, RB) * a.Hkv * (few_chunks(s, a.window) + plan.pad) : (int64_t)0;
  };
  int64_t total = 0;
  for (int b = lane; b < r.batch; b += 32) {
    const Seq s = seq_at(b);
    if (!s.ok && cta == 0 && warp == 0) flag_status(r.status, DFLASH_STATUS_BOUNDS);
    total += units_of(s);
  }
  const FewRanges rg(warp_sum64(total), plan, grid);
  int64_t u = cta < rg.n ? rg.start(cta) : rg.units;
  const int64_t u1 = cta < rg.n ? rg.start(cta + 1) : rg.units;
  int64_t before = 0;
  int seg = 0;
  for (int base = 0; base < r.batch && u < u1; base += 32) {
    Seq ls{0, 0, 0, false};
    if (base + lane < r.batch) ls = seq_at(base + lane);
    const int64_t mine_u = units_of(ls), incl = warp_scan64(mine_u, lane);
    const int64_t chunk_end = before + __shfl_sync(0xffffffffu, incl, 31);
    while (u < u1 && u < chunk_end) {
      const int src = __ffs(__ballot_sync(0xffffffffu, before + incl > u)) - 1;
      const Seq s = few_bcast(ls, src);
      const int64_t off = u - (before + __shfl_sync(0xffffffffu, incl - mine_u, src));
      const int T = few_chunks(s, a.window);
      const int64_t item = off / (T + plan.pad);
      const int rt = (int)(item / a.Hkv), kvh = (int)(item - (int64_t)rt * a.Hkv);
      const int64_t at = off - item * (T + plan.pad) - plan.pad;  // < 0: in front of the item's chunks
      const int64_t most = u1 - u;
      const int c0 = (int)max(at, (int64_t)0), take = (int)(min((int64_t)T, at + most) - c0);
      u += min(T - at, most);
      if (take <= 0) continue;
      stretch(s, base + src, rt, kvh, c0, take, take == T ? -1 : 2 * cta + (seg > 0));
      ++seg;
      __syncthreads();  // the rings are free again
    }
    before = chunk_end;
  }
}

// Merge of the parts of each item that a range boundary cut, in key order.  CTA (c - 1, y): boundary c, if it
// is the first inside its item; a warp per row.
template <int D, int RB>
__global__ void __launch_bounds__(256) k_kv8_few_merge(Ragged r, AttnCall a, FewPlan plan, int grid) {
  constexpr int C = D / 32;
  pdl_trigger();
  pdl_wait();
  r.starts = after_wait(r.starts);
  r.lens = after_wait(r.lens);
  a.ws = after_wait(a.ws);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, G = a.Hq / a.Hkv, c = blockIdx.x + 1;
  const bool one = r.batch <= 32;
  Seq mine{0, 0, 0, false};
  if (one && lane < r.batch) mine = load_seq(r, lane);
  auto units_of = [&](const Seq& s) {
    return s.ok && s.n > 0 ? few_tiles(s, G, RB) * a.Hkv * (few_chunks(s, a.window) + plan.pad) : (int64_t)0;
  };
  int64_t total = 0;
  for (int b = lane; b < r.batch; b += 32) total += units_of(one ? mine : load_seq(r, b));
  const FewRanges rg(warp_sum64(total), plan, grid);
  if (c >= rg.n) return;
  const int64_t u = rg.start(c);
  int64_t before = 0;
  for (int base = 0; base < r.batch; base += 32) {
    Seq ls{0, 0, 0, false};
    if (base + lane < r.batch) ls = one ? mine : load_seq(r, base + lane);
    const int64_t mine_u = units_of(ls), incl = warp_scan64(mine_u, lane);
    const int64_t end = before + __shfl_sync(0xffffffffu, incl, 31);
    if (u >= end) {
      before = end;
      continue;
    }
    const int src = __ffs(__ballot_sync(0xffffffffu, before + incl > u)) - 1;
    const int64_t seq_u = before + __shfl_sync(0xffffffffu, incl - mine_u, src);
    const Seq s = few_bcast(ls, src);
    const int T = few_chunks(s, a.window) + plan.pad;
    const int64_t item = (u - seq_u) / T, i_begin = seq_u + item * T;
    // no cut here (in front of the item's chunks), or not the item's first
    if (u <= i_begin + plan.pad || rg.start(c - 1) > i_begin + plan.pad) return;
    const int rt = (int)(item / a.Hkv), kvh = (int)(item - (int64_t)rt * a.Hkv);
    const int parts = rg.of(i_begin + T - 1) - (c - 1) + 1;
    const int slot0 = 2 * (c - 1) + (rg.start(c - 1) < i_begin);
    auto slot_of = [&](int q) { return q == 0 ? slot0 : 2 * (c - 1 + q); };
    const int r0 = rt * RB, R = (int)min((int64_t)RB, (int64_t)s.n * G - r0), row = blockIdx.y * 8 + warp;
    if (row >= R) return;
    float M = -INFINITY, L = 0.f, acc[C];
#pragma unroll
    for (int j = 0; j < C; ++j) acc[j] = 0.f;
    for (int p0 = 0; p0 < parts; p0 += 32) {
      float2 ml = make_float2(-INFINITY, 0.f);
      if (p0 + lane < parts) ml = *few_ml<D, RB>(a, plan, slot_of(p0 + lane), row);
      const int cnt = min(32, parts - p0);
      const float Mn = fmaxf(M, warp_max(ml.x)), mref = Mn == -INFINITY ? 0.f : Mn;
      const float f = M == -INFINITY ? 0.f : exp2f(M - mref);
      const uint32_t saw = __ballot_sync(0xffffffffu, ml.y != 0.f);
      const float wt = ml.x == -INFINITY ? 0.f : exp2f(ml.x - mref);
      // (sums so far under a maximum of -inf are 0, or the NaN of a NaN score, which stays one)
      L = (M == -INFINITY ? L : L * f) + warp_sum(wt == 0.f ? 0.f : ml.y * wt);
#pragma unroll
      for (int j = 0; j < C; ++j) acc[j] *= M == -INFINITY ? 1.f : f;
      M = Mn;
#pragma unroll 4
      for (int q = 0; q < cnt; ++q) {
        const float wq = __shfl_sync(0xffffffffu, wt, q);
        const float* v = few_o<D, RB>(a, slot_of(p0 + q), row) + lane * C;
        const bool yes = (saw >> q) & 1u;
#pragma unroll
        for (int j = 0; j < C; ++j) acc[j] = fmaf(wq, yes ? v[j] : 0.f, acc[j]);
      }
    }
    const int tok = s.start + (r0 + row) / G, h = kvh * G + (r0 + row) % G;
    store_row<D>(a, tok, h, lane, acc, 1.f / L);
    if (a.lse && lane == 0) a.lse[(int64_t)tok * a.Hq + h] = lse_of(M, L);
    return;
  }
}

int rows_of(const Ragged& r, const AttnCall& a) {
  return (int)std::min<int64_t>((int64_t)r.max_rows * (a.Hq / a.Hkv), 1 << 20);
}
struct FewHost {
  int nb;
  FewPlan p;
};
// CTAs of a cluster per item, or 0 for ranges.  A cut item costs its rows' start and end again, and a launch that
// puts the parts together; 32 over 8 heads of 128, single tokens but for the last:
//   all at once, the largest share of a CTA kMaxShare (36 of 8 CTAs fit, not 38: 12 and 20 us).  One user over 300
//     tokens 6.6 us (ranges 11.4), over 16000 19 (27); 8 users over 8000 28 (43), over 16000 49 (65).
//   in turn, longest first, so that the last to end are short: one CTA an item while the longest (by the bound of
//     lengths) has at most 300 chunks for each item that a CTA's place gets, two up to 1000, and where items are
//     fewer than places four up to 2400: 16 users over 1k to 16k 37 us (ranges 47), 24 52 (61).  64 users over 1k to 16k
//     with one, two, four CTAs and ranges 136, 114, 139, 132 us (in the batch's order 150, 133, 136), over 1k to 8k
//     76, 87, 110, 90, over 100 to 2k 21, 38, 62, 32; 128 over 1k to 16k 226, 258, 313, 269; 128 blocks of 8 over 1k
//     to 8k 298, 378, 543, 369.  (A batch whose places are mostly empty has its few long sequences on few CTAs then.)
int few_cluster(const Ragged& r, const AttnCall& a, int rows, int tiles, int ctas) {
  const int64_t items = (int64_t)r.batch * tiles * a.Hkv;
  const int64_t span = a.window ? std::min<int64_t>(r.max_len, (int64_t)a.window + r.max_rows) : r.max_len;
  const int64_t chunks = (span + kChunk - 1) / kChunk + 1;
  int cluster = 0;
  for (int n = 1; n <= kMaxCluster && items * n <= (n == 8 ? ctas * 15 / 16 : ctas); n *= 2)
    if (chunks <= kMaxShare * n) cluster = n;
  while (cluster > 1 && chunks <= 4 * cluster) cluster /= 2;
  if (!cluster && rows <= kFewRows && items <= INT32_MAX / 8) {
    const int64_t live = std::min<int64_t>(r.batch, std::max(r.total, 1)) * tiles * a.Hkv, turn = live * 300 / ctas;
    cluster = chunks <= turn ? 1 : 3 * chunks <= 10 * turn ? 2 : live <= ctas && chunks <= 8 * turn ? 4 : 0;
  }
  return cluster;
}
FewHost few_plan(const Ragged& r, const AttnCall& a, int sms) {
  const int rows = rows_of(r, a);
  FewHost h;
  // what an item costs besides its chunks; 64 single tokens over 1k to 16k: 4 140 us, 16 134, 28 132, 44 130
  h.p.pad = 28;
  h.p.min_units = 8;
  h.nb = rows <= 8 ? 1 : 2;
  h.p.tiles = (rows + 8 * h.nb - 1) / (8 * h.nb);
  h.p.cluster = few_cluster(r, a, rows, h.p.tiles, 2 * sms);
  h.p.in_turn = h.p.cluster && (int64_t)r.batch * h.p.tiles * a.Hkv * h.p.cluster > 2 * sms;
  h.p.slots = 4 * sms;
  // A tile of rows converts the codes anew, so 32 rows a CTA (one an SM) where ranges are cut: 64 users' blocks of 8
  // over 2048 tokens 134 us (16 rows 152), 8 users' 34 (34).
  if (!h.p.cluster && rows > 16) {
    h.nb = 4;
    h.p.tiles = (rows + 31) / 32;
    h.p.slots = 2 * sms;
  }
  return h;
}

template <int D, int NB>
cudaError_t launch_few(const Ragged& r, const AttnCall& a, const Kv8View& kv, const FewPlan& p, int sms, cudaStream_t st) {
  using C = FewCfg<D, NB>;
  static std::atomic<bool> done[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !done[dev]) {
    e = cudaFuncSetAttribute(k_kv8_few<D, NB>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SMEM);
    if (e != cudaSuccess) return e;
    if (dev < 64) done[dev] = true;
  }
  if (p.cluster > 0)
    return launch_kc(k_kv8_few<D, NB>, r.batch * p.tiles * a.Hkv * p.cluster, kWarps * 32, C::SMEM, st, p.cluster, r, a, kv, p);
  const int grid = sms * C::CTAS;
  e = launch_k(k_kv8_few<D, NB>, grid, kWarps * 32, C::SMEM, st, r, a, kv, p);
  if (e != cudaSuccess) return e;
  const int rows = std::min(rows_of(r, a), C::RB);
  return launch_k(k_kv8_few_merge<D, C::RB>, dim3(grid - 1, (rows + 7) / 8), 256, 0, st, r, a, p, grid);
}
template <int D>
cudaError_t launch_few(const Ragged& r, const AttnCall& a, const Kv8View& kv, int sms, cudaStream_t st) {
  const FewHost h = few_plan(r, a, sms);
  return h.nb == 1   ? launch_few<D, 1>(r, a, kv, h.p, sms, st)
         : h.nb == 2 ? launch_few<D, 2>(r, a, kv, h.p, sms, st)
                     : launch_few<D, 4>(r, a, kv, h.p, sms, st);
}

}  // namespace

// Few rows, or many that are a short call: a KV head's rows of a sequence fill a quarter of the 128-row tiles or less,
// or all items run at once as clusters.  32 over 8 heads of 128, this and the tiles: 64 sequences of 32 rows over 2048
// 109 and 169 us, of 64 rows 236 and 167; 8 of 32 over 16000 109 and 133, of 48 167 and 132; one user's 64 rows over
// 4096 in clusters 18 and 35, 128 over 500 13 and 22.
bool kv8_few(const Ragged& r, const AttnCall& a, int sms) { return rows_of(r, a) <= kFewRows || few_plan(r, a, sms).p.cluster > 0; }
int64_t kv8_few_workspace(const Ragged& r, const AttnCall& a, int sms) {
  const FewHost h = few_plan(r, a, sms);
  return h.p.cluster ? 0 : (int64_t)h.p.slots * 8 * h.nb * (a.d + 2) * 4;
}
cudaError_t launch_kv8_few(const Ragged& r, const AttnCall& a, const Kv8View& kv, int sms, cudaStream_t st) {
  return a.d == 64 ? launch_few<64>(r, a, kv, sms, st) : launch_few<128>(r, a, kv, sms, st);
}

}  // namespace dfl
