// Attention of ragged new rows over an 8-bit paged cache: the CUDA-core path, and
// the entry points.
//
//   o_i = sum_j p_ij vs_j vc_j,  p_ij = exp(s_ij - m_i) / l_i,  s_ij = scale ks_j (q_i . kc_j)
// with codes kc, vc and the scales ks, vs of key j's page, over the keys that row i sees.
#include <algorithm>
#include <atomic>
#include <cmath>

#include "common.cuh"
#include "kv8.h"
#include "kv8_checks.h"
#include "launch.h"
#include "target_checks.h"

namespace dfl {
namespace {

constexpr int kTile = 256;  // keys of a step: one per thread

// Hidden keys among scores and probabilities: the score is a NaN that no operation
// makes (theirs are 0x7fffffff), which a maximum passes over; the probability is -0,
// which exp2f never returns.  V may hold anything there, so those products are left out;
// not every product with P = 0 is, a NaN that the row sees is its own.
constexpr uint32_t kHidden = 0xffc0de00u;
__device__ __forceinline__ float masked_prob(float s, float mref) {
  return __float_as_uint(s) == kHidden ? -0.f : exp2f(s - mref);
}
__device__ __forceinline__ bool is_hidden(float p) { return __float_as_uint(p) == 0x80000000u; }
// The natural log-sum-exp from (m, l) in the exp2 domain: -inf where every score is, NaN where one is.
__device__ __forceinline__ float lse_of(float m, float l) { return (m + log2f(l)) * 0.6931471805599453f; }

template <typename T> __device__ __forceinline__ float4 load4(const T* p);
template <> __device__ __forceinline__ float4 load4<float>(const float* p) { return *reinterpret_cast<const float4*>(p); }
template <> __device__ __forceinline__ float4 load4<bf16>(const bf16* p) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                     __uint_as_float(u.y & 0xffff0000u));
}
template <typename T> __device__ __forceinline__ void store4(T* p, float4 v);
template <> __device__ __forceinline__ void store4<float>(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
template <> __device__ __forceinline__ void store4<bf16>(bf16* p, float4 v) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

// Key tiles of one tile of rows, cut evenly into `splits` stretches.
struct Stretch {
  int t0, t1;
};
__device__ __forceinline__ Stretch stretch_of(int k_lo, int k_hi, int split, int splits) {
  const int a = k_lo / kTile, n = (k_hi + kTile - 1) / kTile - a;
  return Stretch{a + (int)((int64_t)n * split / splits), a + (int)((int64_t)n * (split + 1) / splits)};
}

// BR packed rows (token, head of the group) per CTA, 256 keys a step.  Scores: a key per
// thread, its codes straight from memory, the rows of q broadcast from shared memory.  Then
// the online softmax, the rows dealt to the warps, and O += P V with the keys dealt to
// the warps, whose sums meet at the end.  Where rows are few the keys are cut into splits
// that meet in k_kv8_simt_merge.
template <int DP, int BR> struct SimtCfg {
  static constexpr int LQ = DP + 4, LP = BR + 4, LS = kTile + 4;
  static constexpr int AREA = BR * (8 * DP > LS ? 8 * DP : LS);  // scores, at the end the warps' sums
  static constexpr size_t SMEM = sizeof(float) * (BR * LQ + AREA + kTile * LP + kTile + 3 * BR) + kTile * 8;
};
template <typename T, int DP, int BR>
__global__ void __launch_bounds__(256) k_kv8_simt(Ragged r, AttnCall a, Kv8View kv, int splits) {
  using C = SimtCfg<DP, BR>;
  constexpr int LQ = C::LQ, LP = C::LP, LS = C::LS;
  constexpr int COLS = DP / 4, SLICES = 32 / (COLS < 32 ? COLS : 32);  // column groups; key slices within a warp
  extern __shared__ float4 smem4[];
  float* sQ = reinterpret_cast<float*>(smem4);  // [BR][LQ]
  float* sS = sQ + BR * LQ;                     // [BR][LS]; at the end [8][BR][DP]
  float* sP = sS + C::AREA;                     // [256][LP]
  int64_t* sV = reinterpret_cast<int64_t*>(sP + kTile * LP);  // [256] where the key's V lies, -1: nowhere
  float* sVS = reinterpret_cast<float*>(sV + kTile);          // [256] its scale
  float* sM = sVS + kTile;                                    // [BR] running maximum, sum, and the step's factor
  float* sL = sM + BR;
  float* sF = sL + BR;
  pdl_trigger();
  pdl_wait();
  const int b = blockIdx.z, kvh = blockIdx.y, split = blockIdx.x % splits, r0 = blockIdx.x / splits * BR;
  const Seq s = load_seq(r, b);
  if (!s.ok) {
    if (threadIdx.x == 0) flag_status(r.status, DFLASH_STATUS_BOUNDS);
    return;
  }
  const int G = a.Hq / a.Hkv;
  const int64_t R = (int64_t)s.n * G;
  if (r0 >= R) return;
  const int ctx = s.len - s.n, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int p_first = ctx + r0 / G, p_last = ctx + (int)((min((int64_t)r0 + BR, R) - 1) / G);
  const int k_lo = vis_lo(p_first, a.window), k_hi = vis_hi(p_last, s.len, a.causal);
  const Stretch st = stretch_of(k_lo, k_hi, split, splits);
  for (int e = tid; e < BR * COLS; e += 256) {
    const int rr = e / COLS, c = e % COLS * 4;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r0 + rr < R && c < a.d) {
      const int i = (r0 + rr) / G, g = (r0 + rr) % G;
      x = load4(reinterpret_cast<const T*>(a.q) + (int64_t)(s.start + i) * a.q_row + (int64_t)(kvh * G + g) * a.q_head + c);
    }
    *reinterpret_cast<float4*>(sQ + rr * LQ + c) = x;
  }
  if (tid < BR) {
    sM[tid] = -INFINITY;
    sL[tid] = 0.f;
  }
  const float sl2 = a.scale * 1.4426950408889634f;
  const int col = lane % COLS * 4, slice = lane / COLS;
  const bool in = col < a.d;
  float acc[BR][4];
#pragma unroll
  for (int i = 0; i < BR; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
  for (int t = st.t0; t < st.t1; ++t) {
    const int pos = t * kTile + tid;
    const bool here = pos >= k_lo && pos < k_hi;
    bool exists = false;
    int64_t at = 0;
    float ks = 0.f, vs = 0.f;
    if (here) {
      const int pg = r.table[(int64_t)b * r.table_stride + (pos >> kv.page_shift)];
      exists = pg >= 0 && pg < kv.n_pages;
      if (exists) {
        at = pg * kv.page + (pos & ((1 << kv.page_shift) - 1)) * kv.slot + kvh * kv.head;
        ks = kv.ks[pg * kv.s_page + kvh * kv.s_head];
        vs = kv.vs[pg * kv.s_page + kvh * kv.s_head];
      } else {
        flag_status(r.status, DFLASH_STATUS_PAGE);
      }
    }
    __syncthreads();  // the last step's P and V have been used
    sV[tid] = exists ? at : -1;
    sVS[tid] = vs;
    float sc[BR];
#pragma unroll
    for (int i = 0; i < BR; ++i) sc[i] = 0.f;
    if (exists) {
      const uint8_t* kp = kv.k + at;
#pragma unroll 2
      for (int c = 0; c < a.d; c += 16) {
        const uint4 u = *reinterpret_cast<const uint4*>(kp + c);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float4 k4 = e4m3x4_to_f4(w[q]);
#pragma unroll
          for (int i = 0; i < BR; ++i) {
            const float4 q4 = *reinterpret_cast<const float4*>(sQ + i * LQ + c + 4 * q);
            sc[i] = fmaf(q4.x, k4.x, sc[i]);
            sc[i] = fmaf(q4.y, k4.y, sc[i]);
            sc[i] = fmaf(q4.z, k4.z, sc[i]);
            sc[i] = fmaf(q4.w, k4.w, sc[i]);
          }
        }
      }
    }
    bool hidden = false;
#pragma unroll
    for (int i = 0; i < BR; ++i) {
      const int p = ctx + (r0 + i) / G;
      const bool see = here && r0 + i < R && pos >= vis_lo(p, a.window) && pos < vis_hi(p, s.len, a.causal);
      hidden |= !see;
      // (the key's scale first: the product of both could overflow where the score does not)
      sS[i * LS + tid] = see ? sc[i] * ks * sl2 : __uint_as_float(kHidden);
    }
    const bool guard = __syncthreads_or(hidden && here);
#pragma unroll
    for (int u = 0; u < (BR + 7) / 8; ++u) {
      const int i = warp + 8 * u;
      if (BR < 8 && i >= BR) break;
      float x[kTile / 32], m = sM[i], l = 0.f;
      const float before = m;
#pragma unroll
      for (int j = 0; j < kTile / 32; ++j) {
        x[j] = sS[i * LS + lane + 32 * j];
        m = fmaxf(m, x[j]);
      }
      m = warp_max(m);
      const float mref = m == -INFINITY ? 0.f : m, f = before == -INFINITY ? 0.f : exp2f(before - mref);
#pragma unroll
      for (int j = 0; j < kTile / 32; ++j) {
        const float e = masked_prob(x[j], mref);
        l += e;
        sP[(lane + 32 * j) * LP + i] = e;
      }
      l = warp_sum(l);
      if (lane == 0) {
        // (a sum that is not 0 although the maximum is -inf is the NaN of a NaN score)
        sL[i] = before == -INFINITY ? sL[i] + l : sL[i] * f + l;
        sM[i] = m;
        sF[i] = before == -INFINITY ? 1.f : f;
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < BR; ++i) {
      const float f = sF[i];
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] *= f;
    }
#pragma unroll 4
    for (int q = slice; q < 32; q += SLICES) {
      const int key = warp * 32 + q;
      const int64_t o = sV[key];
      float4 v4 = make_float4(0.f, 0.f, 0.f, 0.f);
      if (o >= 0 && in) {
        v4 = e4m3x4_to_f4(*reinterpret_cast<const uint32_t*>(kv.v + o + col));
        const float vsc = sVS[key];
        v4.x *= vsc;
        v4.y *= vsc;
        v4.z *= vsc;
        v4.w *= vsc;
      }
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
  }
  __syncthreads();  // scores have been read
  float* sO = sS;
#pragma unroll
  for (int i = 0; i < BR; ++i) {
#pragma unroll
    for (int o = COLS; o < 32; o <<= 1)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] += __shfl_xor_sync(0xffffffffu, acc[i][j], o);
    if (slice == 0) *reinterpret_cast<float4*>(sO + (warp * BR + i) * DP + col) = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
  }
  __syncthreads();
  for (int e = tid; e < BR * COLS; e += 256) {
    const int i = e / COLS, c = e % COLS * 4;
    if (r0 + i >= R) continue;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      const float4 t = *reinterpret_cast<const float4*>(sO + (w * BR + i) * DP + c);
      o.x += t.x;
      o.y += t.y;
      o.z += t.z;
      o.w += t.w;
    }
    const int tok = s.start + (r0 + i) / G, h = kvh * G + (r0 + i) % G;
    if (splits > 1) {
      float* w = a.ws + (((int64_t)tok * a.Hq + h) * splits + split) * (a.d + 4);
      if (c == 0) *reinterpret_cast<float4*>(w) = make_float4(sM[i], sL[i], 0.f, 0.f);
      if (c < a.d) *reinterpret_cast<float4*>(w + 4 + c) = o;
      continue;
    }
    const float inv = 1.f / sL[i];
    if (c < a.d)
      store4(reinterpret_cast<T*>(a.out) + (int64_t)tok * a.o_row + (int64_t)h * a.o_head + c,
             make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
    if (a.lse && c == 0) a.lse[(int64_t)tok * a.Hq + h] = lse_of(sM[i], sL[i]);
  }
}

// Merge of the splits in their order: one warp per (token, head), lanes over the columns.
template <typename T>
__global__ void __launch_bounds__(256) k_kv8_simt_merge(Ragged r, AttnCall a, int splits) {
  pdl_trigger();
  pdl_wait();
  const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31, tok = (int)(w / a.Hq), h = (int)(w % a.Hq);
  if (tok >= r.total) return;
  const int b = seq_of_row(r, tok);
  if (b >= r.batch) return;
  const Seq s = load_seq(r, b);
  if (!s.ok || tok < s.start || tok >= s.start + s.n) return;
  const float* p = after_wait(a.ws) + w * splits * (a.d + 4);
  float M = -INFINITY, L = 0.f;
  for (int j = lane; j < splits; j += 32) M = fmaxf(M, p[(int64_t)j * (a.d + 4)]);
  M = warp_max(M);
  const float mref = M == -INFINITY ? 0.f : M;
  const int col = 4 * lane < a.d ? 4 * lane : 0;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int j = 0; j < splits; ++j) {
    const float* q = p + (int64_t)j * (a.d + 4);
    const float2 ml = *reinterpret_cast<const float2*>(q);
    const float4 v = *reinterpret_cast<const float4*>(q + 4 + col);
    // (a part without a key, or whose scores are all -inf, has zeros; the NaN of one with a NaN score stays one)
    const float f = ml.x == -INFINITY ? 1.f : exp2f(ml.x - mref);
    L = fmaf(f, ml.y, L);
    acc.x = fmaf(f, v.x, acc.x);
    acc.y = fmaf(f, v.y, acc.y);
    acc.z = fmaf(f, v.z, acc.z);
    acc.w = fmaf(f, v.w, acc.w);
  }
  const float inv = 1.f / L;
  if (4 * lane < a.d)
    store4(reinterpret_cast<T*>(a.out) + (int64_t)tok * a.o_row + (int64_t)h * a.o_head + 4 * lane,
           make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
  if (a.lse && lane == 0) a.lse[(int64_t)tok * a.Hq + h] = lse_of(M, L);
}

// Packed rows of a CTA.  fp32, 32 over 8 heads of 128: 64 single tokens over 4096 in 4 rows 288 us (8: 550), blocks
// of 16 of 8 users 468 (8: 470), 100 rows of 4 over 2000 682 (8: 658, 16: 723).
int simt_rows(const Ragged& r, const AttnCall& a) {
  return (int64_t)r.max_rows * (a.Hq / a.Hkv) <= 4 ? 4 : 8;
}
// Splits: CTAs for eight turns of each SM, so that uneven lengths even out, none of less than a tile.  64 single tokens over
// 4096: two turns 364 us, four 308, eight 288; blocks of 4 of 8 users 165, 151, 137.
int simt_splits(const Ragged& r, const AttnCall& a, int sms) {
  const int br = simt_rows(r, a);
  const int64_t ctas = ((int64_t)r.max_rows * (a.Hq / a.Hkv) + br - 1) / br * std::min(r.batch, std::max(r.total, 1)) * a.Hkv;
  const int64_t span = a.window ? std::min<int64_t>(r.max_len, (int64_t)a.window + r.max_rows) : r.max_len;
  return (int)std::max<int64_t>(1, std::min<int64_t>({(8 * sms + ctas - 1) / ctas, (span + kTile - 1) / kTile, 64}));
}

template <typename T, int DP, int BR>
cudaError_t launch_simt(const Ragged& r, const AttnCall& a, const Kv8View& kv, int splits, cudaStream_t st) {
  static std::atomic<bool> done[64];
  constexpr size_t smem = SimtCfg<DP, BR>::SMEM;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !done[dev]) {
    e = cudaFuncSetAttribute(k_kv8_simt<T, DP, BR>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    if (dev < 64) done[dev] = true;
  }
  const int64_t tiles = ((int64_t)r.max_rows * (a.Hq / a.Hkv) + BR - 1) / BR;
  e = launch_k(k_kv8_simt<T, DP, BR>, dim3((unsigned)(tiles * splits), a.Hkv, r.batch), 256, smem, st, r, a, kv, splits);
  if (e != cudaSuccess || splits == 1) return e;
  return launch_k(k_kv8_simt_merge<T>, (unsigned)(((int64_t)r.total * a.Hq + 7) / 8), 256, 0, st, r, a, splits);
}
template <typename T, int DP>
cudaError_t launch_simt(const Ragged& r, const AttnCall& a, const Kv8View& kv, int splits, cudaStream_t st) {
  const int br = simt_rows(r, a);
  return br == 4   ? launch_simt<T, DP, 4>(r, a, kv, splits, st)
                   : launch_simt<T, DP, 8>(r, a, kv, splits, st);
}

cudaError_t sms_of_device(int* sms) {
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

}  // namespace

int64_t kv8_simt_workspace(const Ragged& r, const AttnCall& a, int sms) {
  const int64_t splits = simt_splits(r, a, sms);
  return splits == 1 ? 0 : (int64_t)r.total * a.Hq * splits * (a.d + 4) * 4;
}

cudaError_t launch_kv8_simt(const Ragged& r, const AttnCall& a, const Kv8View& kv, bool is_bf16, int sms, cudaStream_t st) {
  const int splits = simt_splits(r, a, sms);
  if (is_bf16) return a.d <= 64 ? launch_simt<bf16, 64>(r, a, kv, splits, st) : launch_simt<bf16, 128>(r, a, kv, splits, st);
  return a.d <= 64 ? launch_simt<float, 64>(r, a, kv, splits, st) : launch_simt<float, 128>(r, a, kv, splits, st);
}

namespace {

// As check_attention, with the head dims of this cache.
int check_kv8_attention(const char* call, const dflash_attention* a, const dflash_kv8_pages* p, bool pointers, bool rows) {
  if (!a) return rfail(DFLASH_ERR_INVALID_ARG, call, "null attention");
  if (a->dtype != DFLASH_DTYPE_F32 && a->dtype != DFLASH_DTYPE_BF16) return rfail(DFLASH_ERR_INVALID_ARG, call, "dtype");
  if (a->n_kv_heads != p->n_kv_heads || a->head_dim != p->head_dim)
    return rfail(DFLASH_ERR_SHAPE, call, "the pages' n_kv_heads or head_dim is not the attention's");
  dflash_attention like = *a;
  like.dtype = DFLASH_DTYPE_F32;  // (whose head dims include the cache's)
  if (int rc = check_attention(call, &like, false, rows)) return rc;
  if (!pointers) return DFLASH_OK;
  if (int rc = check_heads(call, &a->q, a->dtype, a->n_q_heads, a->head_dim, rows)) return rc;
  if (int rc = check_heads(call, &a->out, a->dtype, a->n_q_heads, a->head_dim, rows)) return rc;
  if (rows && a->out.data == a->q.data) return rfail(DFLASH_ERR_INVALID_ARG, call, "out is q");
  return DFLASH_OK;
}

AttnCall kv8_call(const dflash_attention* a) {
  return AttnCall{a->n_q_heads, a->n_kv_heads, a->head_dim, a->causal, a->window, a->scale, a->q.data, a->q.row_stride,
                  a->q.head_stride, a->out.data, a->out.row_stride, a->out.head_stride, a->lse, (float*)a->workspace};
}

int kv8_sms() {
  int sms = 0;
  // without a device (argument checks on a host) the largest part's count of SMs stands in
  if (sms_of_device(&sms) != cudaSuccess) {
    cudaGetLastError();
    sms = 152;
  }
  return sms;
}

// The kernel of a call: bf16 with head_dim 64 or 128 runs on the tensor cores.
enum class Path { kSimt, kFew, kTiles };
Path kv8_path(const dflash_attention* a, const Ragged& r, const AttnCall& c, int sms) {
  if (a->dtype != DFLASH_DTYPE_BF16 || (a->head_dim != 64 && a->head_dim != 128)) return Path::kSimt;
  return kv8_few(r, c, sms) ? Path::kFew : Path::kTiles;
}
int64_t kv8_workspace(const dflash_attention* a, const Ragged& r, int sms) {
  const AttnCall c = kv8_call(a);
  int64_t bytes = 0;
  switch (kv8_path(a, r, c, sms)) {
    case Path::kSimt: return kv8_simt_workspace(r, c, sms);
    case Path::kFew: return kv8_few_workspace(r, c, sms);
    default: attn_tc_workspace(r, c, &bytes, true); return bytes;
  }
}

}  // namespace
}  // namespace dfl

using namespace dfl;

extern "C" {

DFLASH_API int64_t dflash_kv8_attention_workspace(const dflash_attention* a, const dflash_ragged* batch,
                                                  const dflash_kv8_pages* pages) {
  const char* call = "dflash_kv8_attention_workspace";
  if (int rc = check_kv8_pages(call, pages)) return rc;
  if (int rc = check_kv8_attention(call, a, pages, false, false)) return rc;
  const dflash_kv_pages like = kv8_as_pages(pages);
  if (int rc = check_ragged(call, batch, &like, false)) return rc;
  return kv8_workspace(a, make_ragged(batch, &like), kv8_sms());
}

DFLASH_API int dflash_kv8_attention(const dflash_attention* a, const dflash_ragged* batch,
                                    const dflash_kv8_pages* pages, void* stream) {
  const char* call = "dflash_kv8_attention";
  if (int rc = check_kv8_pages(call, pages)) return rc;
  const dflash_kv_pages like = kv8_as_pages(pages);
  if (int rc = check_ragged(call, batch, &like, true)) return rc;
  if (int rc = check_kv8_attention(call, a, pages, true, batch->total_rows > 0)) return rc;
  const Ragged r = make_ragged(batch, &like);
  if (r.total == 0) return DFLASH_OK;
  const int64_t rows = (int64_t)r.max_rows * (a->n_q_heads / a->n_kv_heads);
  if ((int64_t)r.total * a->n_q_heads > INT32_MAX || rows > INT32_MAX / 64)
    return rfail(DFLASH_ERR_SHAPE, call, "total_rows x n_q_heads above 2^31 - 1, or max_rows x heads of a group above 2^25");
  const int sms = kv8_sms();
  const int64_t need = kv8_workspace(a, r, sms);
  if (need > 0 && (!a->workspace || a->workspace_bytes < need || (uintptr_t)a->workspace % 32))
    return rfail(DFLASH_ERR_INVALID_ARG, call, "workspace: 32-byte aligned, at least dflash_kv8_attention_workspace bytes");
  const AttnCall c = kv8_call(a);
  const Kv8View kv = kv8_view(pages);
  cudaStream_t st = (cudaStream_t)stream;
  switch (kv8_path(a, r, c, sms)) {
    case Path::kSimt: return rcheck(launch_kv8_simt(r, c, kv, a->dtype == DFLASH_DTYPE_BF16, sms, st), call);
    case Path::kFew: return rcheck(launch_kv8_few(r, c, kv, sms, st), call);
    default: return rcheck(launch_attn_tc8(r, c, kv, st), call);
  }
}

}  // extern "C"
