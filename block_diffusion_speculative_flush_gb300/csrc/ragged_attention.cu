// Target-side operators on ragged batches: new K/V rows into pages, and the
// attention of a chunk of new tokens over pages or of packed prompts on the
// CUDA cores.
//
//   o_i = sum_j p_ij v_j,  p_ij = exp(s_ij - m_i) / l_i,  s_ij = scale q_i . k_j
// over the keys j that row i sees, with the running maximum m and sum l of an
// online softmax (fp32, in the exp2 domain), one pass over K and V.
#include <algorithm>
#include <cmath>
#include <cstdio>

#include "common.cuh"
#include "dflash.h"
#include "kernels.h"
#include "launch.h"
#include "ragged.h"

extern "C" int dflash__set_error(int code, const char* msg);

namespace dfl {
namespace {

// ---------------------------------------------------------------------------
// append
// ---------------------------------------------------------------------------
// One warp per new row: 16 bytes of K and of V per lane and step.  Bound by
// memory (2 reads and 2 writes of a row's Hkv d elements).
__global__ void __launch_bounds__(256) k_kv_append(Ragged r, const uint4* __restrict__ k, const uint4* __restrict__ v,
                                                   int64_t k_row, int64_t k_head, int64_t v_row, int64_t v_head,
                                                   uint4* kp, uint4* vp, int64_t page_st, int64_t slot_st,
                                                   int64_t head_st, int page_shift, int n_pages, int heads, int chunks) {
  pdl_trigger();
  pdl_wait();
  const int row = (int)(blockIdx.x * 8 + (threadIdx.x >> 5)), lane = threadIdx.x & 31;
  if (row >= r.total) return;
  const int b = seq_of_row(r, row);
  if (b >= r.batch) return;  // behind the last sequence
  const Seq s = load_seq(r, b);
  const int i = row - s.start;
  if (!s.ok || i < 0 || i >= s.n) {
    if (lane == 0) flag_status(r.status, DFLASH_STATUS_BOUNDS);
    return;
  }
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
// attention on the CUDA cores
// ---------------------------------------------------------------------------
constexpr int BK = 64;           // keys per tile
constexpr int kSimtSplit = 256;  // keys per split (a multiple of BK)

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }

// The CUDA-core attention works on 16 RM packed rows (token, head of the KV
// head's group) per CTA and 64 keys per step; threads are 16 x 16, each with
// RM rows x 4 keys of the scores and RM rows x DP / 16 columns of the output.
// A row's arithmetic depends on its own keys only (tiles and splits start at
// fixed positions), so a block of tokens and single tokens give the same bits.
template <int DP, int RM>
__global__ void __launch_bounds__(256) k_attn_simt_ragged(Ragged r, AttnCall a, KVView kv, int splits) {
  constexpr int BR = 16 * RM, LQ = DP + 4, LP = BK + 4;
  extern __shared__ float4 smem4[];
  float* sQ = reinterpret_cast<float*>(smem4);
  float* sK = sQ + BR * LQ;
  float* sV = sK + BK * LQ;
  float* sP = sV + BK * DP;
  pdl_trigger();
  pdl_wait();
  const int b = blockIdx.z, kvh = blockIdx.y, split = blockIdx.x % splits, rt = blockIdx.x / splits;
  const Seq s = load_seq(r, b);
  if (!s.ok) {
    if (threadIdx.x == 0) flag_status(r.status, DFLASH_STATUS_BOUNDS);
    return;
  }
  const int G = a.Hq / a.Hkv, R = s.n * G, r0 = rt * BR;
  if (r0 >= R) return;
  const int ctx = s.len - s.n;
  if (splits > 1 && split * kSimtSplit >= s.len && split > 0) return;  // the merge does not look at it either
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  // keys that any of the tile's rows sees, within this split
  const int p_first = ctx + r0 / G, p_last = ctx + (min(r0 + BR, R) - 1) / G;
  int k_lo = vis_lo(p_first, a.window), k_hi = vis_hi(p_last, s.len, a.causal);
  if (splits > 1) {
    k_lo = max(k_lo, split * kSimtSplit);
    k_hi = min(k_hi, (split + 1) * kSimtSplit);
  }
  const float* Q = reinterpret_cast<const float*>(a.q);
  for (int e = tid; e < BR * (DP / 4); e += 256) {
    const int rr = e / (DP / 4), c = e % (DP / 4) * 4;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r0 + rr < R && c < a.d) {
      const int i = (r0 + rr) / G, g = (r0 + rr) % G;
      x = load4(Q + (int64_t)(s.start + i) * a.q_row + (int64_t)(kvh * G + g) * a.q_head + c);
    }
    *reinterpret_cast<float4*>(sQ + rr * LQ + c) = x;
  }
  int lo[RM], hi[RM];
  float m[RM], l[RM], acc[RM][DP / 16];
#pragma unroll
  for (int i = 0; i < RM; ++i) {
    const int rr = r0 + ty * RM + i, p = ctx + rr / G;
    lo[i] = max(vis_lo(p, a.window), k_lo);
    hi[i] = rr < R ? min(vis_hi(p, s.len, a.causal), k_hi) : 0;
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int c = 0; c < DP / 16; ++c) acc[i][c] = 0.f;
  }
  const float sl2 = a.scale * 1.4426950408889634f;
  const float* Kb = reinterpret_cast<const float*>(kv.k) + kvh * kv.k_head;
  const float* Vb = reinterpret_cast<const float*>(kv.v) + kvh * kv.v_head;
  for (int t0 = k_lo / BK * BK; t0 < k_hi; t0 += BK) {
    __syncthreads();
    for (int e = tid; e < BK * (DP / 4); e += 256) {
      const int kk = e / (DP / 4), c = e % (DP / 4) * 4, pos = t0 + kk;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
      if (pos < k_hi && c < a.d) {
        int64_t ko, vo;
        bool ok = true;
        if (kv.paged) {
          const int pg = r.table[(int64_t)b * r.table_stride + (pos >> kv.page_shift)];
          const int sl = pos & ((1 << kv.page_shift) - 1);
          ok = pg >= 0 && pg < kv.n_pages;
          if (!ok && c == 0) flag_status(r.status, DFLASH_STATUS_PAGE);
          ko = pg * kv.page + sl * kv.k_slot;
          vo = pg * kv.page + sl * kv.v_slot;
        } else {
          ko = (int64_t)(s.start + pos) * kv.k_slot;
          vo = (int64_t)(s.start + pos) * kv.v_slot;
        }
        if (ok) {
          x = load4(Kb + ko + c);
          y = load4(Vb + vo + c);
        }
      }
      *reinterpret_cast<float4*>(sK + kk * LQ + c) = x;
      *reinterpret_cast<float4*>(sV + kk * DP + c) = y;
    }
    __syncthreads();
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
    // A key that a row does not see has P = 0; its V may still be NaN or
    // infinite, so tiles with hidden keys skip those products.
    const bool guard = __any_sync(0xffffffffu, masked);
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
            if (!guard || pv != 0.f) {
              o[0] = fmaf(pv, v4.x, o[0]);
              o[1] = fmaf(pv, v4.y, o[1]);
              o[2] = fmaf(pv, v4.z, o[2]);
              o[3] = fmaf(pv, v4.w, o[3]);
            }
          }
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < RM; ++i) {
    float ls = l[i];
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) ls += __shfl_xor_sync(0xffffffffu, ls, o);
    const int rr = r0 + ty * RM + i;
    if (rr >= R) continue;
    const int tok = s.start + rr / G, h = kvh * G + rr % G;
    if (splits > 1) {
      float* w = a.ws + (((int64_t)tok * a.Hq + h) * splits + split) * (a.d + 4);
      if (tx == 0) *reinterpret_cast<float4*>(w) = make_float4(m[i], ls, 0.f, 0.f);
#pragma unroll
      for (int cc = 0; cc < DP / 64; ++cc)
        if (cc * 64 + tx * 4 < a.d)
          *reinterpret_cast<float4*>(w + 4 + cc * 64 + tx * 4) =
              make_float4(acc[i][cc * 4], acc[i][cc * 4 + 1], acc[i][cc * 4 + 2], acc[i][cc * 4 + 3]);
      continue;
    }
    const float inv = m[i] == -INFINITY ? 0.f : 1.f / ls;
    float* o = reinterpret_cast<float*>(a.out) + (int64_t)tok * a.o_row + (int64_t)h * a.o_head;
#pragma unroll
    for (int cc = 0; cc < DP / 64; ++cc)
      if (cc * 64 + tx * 4 < a.d)
        store4(o + cc * 64 + tx * 4, make_float4(acc[i][cc * 4] * inv, acc[i][cc * 4 + 1] * inv,
                                                 acc[i][cc * 4 + 2] * inv, acc[i][cc * 4 + 3] * inv));
    if (a.lse && tx == 0)
      a.lse[(int64_t)tok * a.Hq + h] = m[i] == -INFINITY ? -INFINITY : (m[i] + log2f(ls)) * 0.6931471805599453f;
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
  const int ns = max(1, min(splits, (s.len + kSimtSplit - 1) / kSimtSplit));
  const float* p = a.ws + w * splits * (a.d + 4);
  float M = -INFINITY;
  for (int j = lane; j < ns; j += 32) M = fmaxf(M, p[(int64_t)j * (a.d + 4)]);
  M = warp_max(M);
  const float mref = M == -INFINITY ? 0.f : M;
  float L = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int j = 0; j < ns; ++j) {
    const float* q = p + (int64_t)j * (a.d + 4);
    if (q[0] == -INFINITY) continue;
    const float f = exp2f(q[0] - mref);
    L += q[1] * f;
    if (4 * lane < a.d) {
      const float4 v = *reinterpret_cast<const float4*>(q + 4 + 4 * lane);
      acc.x = fmaf(f, v.x, acc.x);
      acc.y = fmaf(f, v.y, acc.y);
      acc.z = fmaf(f, v.z, acc.z);
      acc.w = fmaf(f, v.w, acc.w);
    }
  }
  const float inv = M == -INFINITY ? 0.f : 1.f / L;
  if (4 * lane < a.d)
    store4(reinterpret_cast<float*>(a.out) + (int64_t)tok * a.o_row + (int64_t)h * a.o_head + 4 * lane,
           make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
  if (a.lse && lane == 0) a.lse[w] = M == -INFINITY ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
}

// Splits of the key axis: only where one row tile holds a sequence's rows
// (single tokens and verified blocks), where the length is what work there is.
int simt_splits(const Ragged& r, const AttnCall& a) {
  const int64_t rows = (int64_t)r.max_rows * (a.Hq / a.Hkv);
  if (!r.lens || rows > 64) return 1;
  return (r.max_len + kSimtSplit - 1) / kSimtSplit;
}

template <int DP, int RM>
cudaError_t launch_simt(const Ragged& r, const AttnCall& a, const KVView& kv, cudaStream_t st) {
  constexpr int BR = 16 * RM;
  constexpr size_t smem = sizeof(float) * (BR * (DP + 4) + BK * (DP + 4) + BK * DP + BR * (BK + 4));
  static bool attr[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !attr[dev]) {
    e = cudaFuncSetAttribute(k_attn_simt_ragged<DP, RM>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    if (dev < 64) attr[dev] = true;
  }
  const int splits = simt_splits(r, a);
  const int64_t tiles = ((int64_t)r.max_rows * (a.Hq / a.Hkv) + BR - 1) / BR;
  e = launch_k(k_attn_simt_ragged<DP, RM>, dim3((unsigned)(tiles * splits), a.Hkv, r.batch), 256, smem, st, r, a,
               kv, splits);
  if (e != cudaSuccess || splits == 1) return e;
  return launch_k(k_attn_simt_merge, (unsigned)(((int64_t)r.total * a.Hq + 7) / 8), 256, 0, st, r, a, splits);
}

}  // namespace

int64_t attn_simt_workspace(const Ragged& r, const AttnCall& a) {
  const int64_t splits = simt_splits(r, a);
  return splits == 1 ? 0 : (int64_t)r.total * a.Hq * splits * (a.d + 4) * 4;
}

cudaError_t launch_attn_simt(const Ragged& r, const AttnCall& a, const KVView& kv, cudaStream_t st) {
  const bool few = (int64_t)r.max_rows * (a.Hq / a.Hkv) <= 16;
  if (a.d <= 64) return few ? launch_simt<64, 1>(r, a, kv, st) : launch_simt<64, 4>(r, a, kv, st);
  return few ? launch_simt<128, 1>(r, a, kv, st) : launch_simt<128, 4>(r, a, kv, st);
}

namespace {

// ---------------------------------------------------------------------------
// argument checks
// ---------------------------------------------------------------------------
int rfail(int code, const char* call, const char* what) {
  char buf[256];
  snprintf(buf, sizeof buf, "%s: %s", call, what);
  return dflash__set_error(code, buf);
}
int rcheck(cudaError_t e, const char* call) {
  return e == cudaSuccess ? DFLASH_OK : rfail(DFLASH_ERR_CUDA, call, cudaGetErrorString(e));
}
int esize(int32_t dtype) { return dtype == DFLASH_DTYPE_F32 ? 4 : 2; }
bool pow2(int64_t x) { return x > 0 && (x & (x - 1)) == 0; }

int check_shape(const char* call, int32_t dtype, int32_t hkv, int32_t d) {
  if (dtype != DFLASH_DTYPE_F32 && dtype != DFLASH_DTYPE_BF16) return rfail(DFLASH_ERR_INVALID_ARG, call, "dtype");
  if (hkv < 1 || hkv > 1024) return rfail(DFLASH_ERR_SHAPE, call, "n_kv_heads outside 1..1024");
  if (dtype == DFLASH_DTYPE_BF16 ? (d != 64 && d != 128) : (d < 4 || d > 128 || d % 4))
    return rfail(DFLASH_ERR_SHAPE, call, "head_dim: bf16 64 or 128, fp32 a multiple of 4 up to 128");
  return DFLASH_OK;
}

// strides below 2^40 bytes keep every offset of 2^30 rows within 64 bits
bool stride_ok(int64_t s, int es) { return s >= 0 && (s * es) % 16 == 0 && s < ((int64_t)1 << 38); }

int check_heads(const char* call, const dflash_heads* h, int32_t dtype, int32_t heads, int32_t d, bool rows) {
  if (!h || (rows && !h->data)) return rfail(DFLASH_ERR_INVALID_ARG, call, "null rows");
  const int es = esize(dtype);
  if ((uintptr_t)h->data % 16 || !stride_ok(h->row_stride, es) || !stride_ok(h->head_stride, es))
    return rfail(DFLASH_ERR_INVALID_ARG, call, "rows: 16-byte aligned base, strides multiples of 16 bytes");
  if ((heads > 1 && h->head_stride < d) || h->row_stride < d)
    return rfail(DFLASH_ERR_INVALID_ARG, call, "rows: strides shorter than a head");
  return DFLASH_OK;
}

int check_pages(const char* call, const dflash_kv_pages* p) {
  if (!p || !p->k || !p->v) return rfail(DFLASH_ERR_INVALID_ARG, call, "null pages");
  if (int rc = check_shape(call, p->dtype, p->n_kv_heads, p->head_dim)) return rc;
  if (p->page_size < 8 || p->page_size > 1024 || !pow2(p->page_size))
    return rfail(DFLASH_ERR_SHAPE, call, "page_size: a power of two in 8..1024");
  if (p->n_pages < 1 || p->n_pages > INT32_MAX) return rfail(DFLASH_ERR_SHAPE, call, "n_pages outside 1..2^31 - 1");
  const int es = esize(p->dtype);
  if ((uintptr_t)p->k % 16 || (uintptr_t)p->v % 16 || !stride_ok(p->page_stride, es) ||
      !stride_ok(p->slot_stride, es) || !stride_ok(p->head_stride, es))
    return rfail(DFLASH_ERR_INVALID_ARG, call, "pages: 16-byte aligned bases, strides multiples of 16 bytes");
  if (p->slot_stride < p->head_dim || (p->n_kv_heads > 1 && p->head_stride < p->head_dim) ||
      (p->n_pages > 1 && p->page_stride < p->head_dim))
    return rfail(DFLASH_ERR_INVALID_ARG, call, "pages: strides shorter than a head");
  return DFLASH_OK;
}

// Host bounds of the batch; the device fields only have to be there.
int check_ragged(const char* call, const dflash_ragged* b, const dflash_kv_pages* pages, bool pointers) {
  if (!b) return rfail(DFLASH_ERR_INVALID_ARG, call, "null batch");
  if (b->batch < 1 || b->batch > 32768) return rfail(DFLASH_ERR_INVALID_ARG, call, "batch outside 1..32768");
  if (b->total_rows < 0 || b->total_rows > (1 << 30) || b->max_rows < 1 || b->max_rows > (1 << 24))
    return rfail(DFLASH_ERR_INVALID_ARG, call, "total_rows outside 0..2^30 or max_rows outside 1..2^24");
  if (pointers && !b->starts) return rfail(DFLASH_ERR_INVALID_ARG, call, "null starts");
  if (pages) {
    if (pointers && (!b->lens || !b->table)) return rfail(DFLASH_ERR_INVALID_ARG, call, "null lens or table");
    if (b->max_len < 1 || b->max_len > (1 << 30)) return rfail(DFLASH_ERR_INVALID_ARG, call, "max_len outside 1..2^30");
    if (b->table_width < 1 || b->table_stride < b->table_width)
      return rfail(DFLASH_ERR_INVALID_ARG, call, "table_width < 1 or table_stride below it");
  }
  return DFLASH_OK;
}

int check_attention(const char* call, const dflash_attention* a, bool pointers, bool rows) {
  if (!a) return rfail(DFLASH_ERR_INVALID_ARG, call, "null attention");
  if (int rc = check_shape(call, a->dtype, a->n_kv_heads, a->head_dim)) return rc;
  if (a->n_q_heads < 1 || a->n_q_heads % a->n_kv_heads || a->n_q_heads / a->n_kv_heads > 128)
    return rfail(DFLASH_ERR_SHAPE, call, "n_q_heads: a multiple of n_kv_heads, at most 128 per KV head");
  if ((a->causal != 0 && a->causal != 1) || a->window < 0 || a->window > (1 << 30))
    return rfail(DFLASH_ERR_INVALID_ARG, call, "causal 0 or 1, window 0 or 1..2^30");
  if (!(a->scale > 0.f) || !std::isfinite(a->scale)) return rfail(DFLASH_ERR_INVALID_ARG, call, "scale: finite, > 0");
  if (!pointers) return DFLASH_OK;
  if (int rc = check_heads(call, &a->q, a->dtype, a->n_q_heads, a->head_dim, rows)) return rc;
  if (int rc = check_heads(call, &a->out, a->dtype, a->n_q_heads, a->head_dim, rows)) return rc;
  if (rows && a->out.data == a->q.data) return rfail(DFLASH_ERR_INVALID_ARG, call, "out is q");
  return DFLASH_OK;
}

Ragged make_ragged(const dflash_ragged* b, const dflash_kv_pages* pages) {
  int64_t max_len = b->max_rows;
  if (pages) max_len = std::min<int64_t>(b->max_len, (int64_t)b->table_width * pages->page_size);
  return Ragged{b->batch, b->total_rows, std::min(b->max_rows, std::max(b->total_rows, 1)), (int32_t)max_len, b->starts,
                pages ? b->lens : nullptr, pages ? b->table : nullptr, b->table_stride, b->status};
}
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
  snprintf(buf, sizeof buf, "%s%s%s%s", s & DFLASH_STATUS_TOKEN ? "a token id outside the vocabulary; " : "",
           s & DFLASH_STATUS_BOUNDS ? "a sequence outside the batch's bounds; " : "",
           s & DFLASH_STATUS_PAGE ? "a page id outside the cache; " : "",
           s & DFLASH_STATUS_WAIT ? "a bounded wait expired; " : "");
  return rfail(DFLASH_ERR_DEVICE, call, buf);
}

}  // extern "C"
