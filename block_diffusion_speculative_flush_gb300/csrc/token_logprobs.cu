// Log probabilities of given tokens with the distribution's entropy and its
// top entries.  With c = log2(e) / T, d_v = (l_v - m) c for the running maximum
// m of l, s = sum 2^d and t = sum 2^d d:
//   log2 p(v) = d_v - log2 s,   H / ln 2 = log2 s - t / s.
// (The difference before the product: the largest entry's d is exactly 0, and a
// row of one possible token has entropy 0.)
// One pass over the logits: (m, s, t) per thread, rescaled when its maximum
// grows, and the top entries beside it.  Bound by reading the logits once.
//
// A row belongs to a cluster of 1..16 CTAs, as many as give every SM two CTAs
// when rows are few; each CTA streams its slice in 16-byte loads, four in
// flight per thread and the next four requested before they are used.  The
// slices meet through distributed shared memory: one launch at any row count.
// Arithmetic runs in packed pairs (5 instructions an element): at one element
// per instruction the issue slots, not memory, bounded the bf16 rows.
//
// Top entries: an element counts only if it reaches the CTA's threshold, a
// value that at least K of the CTA's entries reach; one compare per thread and
// 16 or 32 elements decides that none does, the common case.  The first
// threshold comes from the threads' maxima of the first batch: of each warp the
// r-th largest, r = ceil(K / warps), of these the smallest.  Each warp keeps
// its best 32 keys (value's order above, ~id below) sorted over its lanes and
// raises the threshold with its K-th.  In the end the keys that reach the
// threshold, little more than K, are ranked by counting the larger ones.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include <cmath>
#include <type_traits>

#include "common.cuh"
#include "dflash.h"
#include "launch.h"

extern "C" int dflash__set_error(int code, const char* msg);

namespace dfl {
namespace {

namespace cg = cooperative_groups;

constexpr int TH = 256, WARPS = TH / 32;
constexpr int U = 4;  // 16-byte loads of a batch
constexpr int kMaxCluster = 16;

__device__ __forceinline__ float lp_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// (m, s, t) of a set of entries; m = -inf: no entry above -inf.
struct Stat {
  float m, s, t;
};
// The union of the lanes' sets, in every lane.
__device__ __forceinline__ Stat warp_merge(Stat a, float c) {
  const float M = warp_max(a.m);
  // a side at -inf has s = t = 0 (or NaN, which stays)
  const float d = a.m == -INFINITY ? 0.f : (a.m - M) * c, f = exp2f(d);
  return Stat{M, warp_sum(a.s * f), warp_sum(f * (a.t + a.s * d))};
}
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t r) {
  float2 v;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(v.x), "=f"(v.y) : "l"(r));
  return v;
}
__device__ __forceinline__ float fmax3(float a, float b, float c) {
  float m;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(a), "f"(b), "f"(c));
  return m;
}
__device__ __forceinline__ float fmin3(float a, float b, float c) {
  float m;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(a), "f"(b), "f"(c));
  return m;
}

template <typename T> struct Elems;
template <> struct Elems<float> {
  static constexpr int E = 4;
  static __device__ __forceinline__ void get(const uint4& v, float* x) {
    x[0] = __uint_as_float(v.x);
    x[1] = __uint_as_float(v.y);
    x[2] = __uint_as_float(v.z);
    x[3] = __uint_as_float(v.w);
  }
  // largest and smallest of n vectors (NaN never wins)
  template <int n>
  static __device__ __forceinline__ void range(const uint4* v, float& hi, float& lo) {
    float h0 = -INFINITY, h1 = -INFINITY, l0 = INFINITY, l1 = INFINITY;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      float x[4];
      get(v[i], x);
      h0 = fmax3(h0, x[0], x[1]);
      h1 = fmax3(h1, x[2], x[3]);
      l0 = fmin3(l0, x[0], x[1]);
      l1 = fmin3(l1, x[2], x[3]);
    }
    hi = fmaxf(h0, h1);
    lo = fminf(l0, l1);
  }
};
template <> struct Elems<bf16> {
  static constexpr int E = 8;
  static __device__ __forceinline__ void get(const uint4& v, float* x) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  template <int n>
  static __device__ __forceinline__ void range(const uint4* v, float& hi, float& lo) {
    const __nv_bfloat162* b = reinterpret_cast<const __nv_bfloat162*>(v);
    __nv_bfloat162 h = __float2bfloat162_rn(-INFINITY), l = __float2bfloat162_rn(INFINITY);
#pragma unroll
    for (int i = 0; i < 4 * n; ++i) {
      h = __hmax2(h, b[i]);
      l = __hmin2(l, b[i]);
    }
    const float2 hf = __bfloat1622float2(h), lf = __bfloat1622float2(l);
    hi = fmaxf(hf.x, hf.y);
    lo = fminf(lf.x, lf.y);
  }
};

// Inserts key into the warp's list, sorted descending over the lanes.
__device__ __forceinline__ void list_insert(uint64_t& mine, uint64_t key, int lane) {
  const int pos = __popc(__ballot_sync(0xffffffffu, mine > key));
  const uint64_t up = __shfl_up_sync(0xffffffffu, mine, 1);
  if (lane == pos) mine = key;
  else if (lane > pos) mine = up;
}
// The k-th largest (0-based) of the lanes' values.
__device__ __forceinline__ float kth_of_lanes(float v, int k, int lane) {
#pragma unroll
  for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
    for (int o = size >> 1; o > 0; o >>= 1) {
      const float w = __shfl_xor_sync(0xffffffffu, v, o);
      const bool desc = (lane & size) == 0, low = (lane & o) == 0;
      v = desc == low ? fmaxf(v, w) : fminf(v, w);
    }
  return __shfl_sync(0xffffffffu, v, k);
}

template <typename T>
__global__ void __launch_bounds__(TH, 4) k_token_logprobs(dflash_logprobs a, int cluster, float c) {
  constexpr int E = Elems<T>::E, N = U * E;
  __shared__ uint64_t s_key[kMaxCluster * 32], s_out[32];
  __shared__ Stat s_stat[WARPS], s_cta, s_row;
  __shared__ float s_first[WARPS];
  __shared__ uint32_t s_tau, s_n;  // float_order of the threshold; keys gathered
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row = blockIdx.x / cluster, rank = blockIdx.x % cluster, K = a.top;
  if (tid == 0) {
    s_tau = float_order(-INFINITY);
    s_n = 0;
  }
  if (tid < 32) s_out[tid] = 0;
  __syncthreads();
  pdl_trigger();
  pdl_wait();
  const T* x = after_wait(reinterpret_cast<const T*>(a.logits)) + (int64_t)row * a.row_stride;
  // the token's own logit, requested first
  int tok = -1;
  float xt = 0.f;
  if (rank == 0 && tid == 0) {
    tok = after_wait(a.tokens)[row];
    if (tok >= 0 && tok < a.vocab) xt = to_f<T>(x[tok]);
  }
  // [0, head) single elements, nv vectors, then the tail
  const int head = min(a.vocab, (int)((16 - ((uintptr_t)x & 15)) & 15) / (int)sizeof(T));
  const int nv = (a.vocab - head) / E, per = (nv + cluster - 1) / cluster;
  const uint4* xv = reinterpret_cast<const uint4*>(x + head);
  const int v0 = min(nv, rank * per), v1 = min(nv, v0 + per);

  Stat st{-INFINITY, 0.f, 0.f};
  uint64_t list = 0, kth = 0;
  // adds n elements with maximum hi; clamp: -inf among them (2^-inf is 0, but
  // 0 (-inf) is not: the factor is kept finite; a NaN still comes in through p)
  auto add = [&](auto n_, const float* e, float hi, bool clamp) {
    constexpr int n = decltype(n_)::value;
    if (hi > st.m) {
      const float dm = (st.m - hi) * c, f = lp_ex2(dm);
      st.t = st.m == -INFINITY ? st.t : f * fmaf(st.s, dm, st.t);
      st.s *= f;
      st.m = hi;
    }
    const float mref = st.m == -INFINITY ? 0.f : st.m;
    const uint64_t m2 = pack2(mref, mref), c2 = pack2(c, c);
    uint64_t s2 = pack2(0.f, 0.f), t2 = s2;
#pragma unroll
    for (int i = 0; i < n; i += 2) {
      uint64_t d;
      asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(pack2(e[i], e[i + 1])), "l"(m2));
      asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(d), "l"(c2));
      float2 dd = unpack2(d);
      const uint64_t pp = pack2(lp_ex2(dd.x), lp_ex2(dd.y));
      if (clamp) d = pack2(fmaxf(dd.x, -1000.f), fmaxf(dd.y, -1000.f));
      asm("add.rn.f32x2 %0, %0, %1;" : "+l"(s2) : "l"(pp));
      asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(t2) : "l"(pp), "l"(d));
    }
    const float2 sf = unpack2(s2), tf = unpack2(t2);
    st.s += sf.x + sf.y;
    st.t += tf.x + tf.y;
  };
  // keys of the lanes' candidates (bit i: element i), re-read by id
  auto select = [&](uint32_t bits, auto id_of) {
    while (__any_sync(0xffffffffu, bits != 0)) {
      uint64_t key = 0;
      if (bits) {
        const int id = id_of(__ffs(bits) - 1);
        bits &= bits - 1;
        key = order_key(to_f<T>(x[id]), id);
      }
      uint32_t todo = __ballot_sync(0xffffffffu, key > kth);
      while (todo) {
        const uint64_t k2 = __shfl_sync(0xffffffffu, key, __ffs(todo) - 1);
        todo &= todo - 1;
        if (k2 > kth) {
          list_insert(list, k2, lane);
          kth = __shfl_sync(0xffffffffu, list, K - 1);
        }
      }
    }
    if (kth && lane == 0) atomicMax(&s_tau, (uint32_t)(kth >> 32));
  };

  if (v0 < v1) {
    uint4 cur[U], nxt[U];
    const uint32_t none = sizeof(T) == 4 ? 0xff800000u : 0xff80ff80u;  // -inf
    auto load = [&](uint4* d, int base) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int v = base + u * TH + tid;
        d[u] = v < v1 ? __ldcs(xv + v) : make_uint4(none, none, none, none);
      }
    };
    load(cur, v0);
    for (int base = v0; base < v1; base += U * TH) {
      load(nxt, base + U * TH);
      float hi, lo;
      Elems<T>::template range<U>(cur, hi, lo);
      if (!(hi >= -INFINITY)) hi = -INFINITY;  // nothing but NaN
      if (K > 0 && base == v0) {
        const float r = kth_of_lanes(hi, (K + WARPS - 1) / WARPS - 1, lane);
        if (lane == 0) s_first[warp] = r;
        __syncthreads();
        if (tid == 0) {
          float m = s_first[0];
          for (int w = 1; w < WARPS; ++w) m = fminf(m, s_first[w]);
          atomicMax(&s_tau, float_order(m));
        }
        __syncthreads();
      }
      {
        float e[N];
#pragma unroll
        for (int u = 0; u < U; ++u) Elems<T>::get(cur[u], e + u * E);
        if (lo > -INFINITY) add(std::integral_constant<int, N>(), e, hi, false);
        else add(std::integral_constant<int, N>(), e, hi, true);
      }
      if (K > 0) {
        const float tau = float_of_order(*(volatile uint32_t*)&s_tau);
        if (__any_sync(0xffffffffu, hi >= tau)) {
          uint32_t bits = 0;
#pragma unroll
          for (int u = 0; u < U; ++u) {
            float e[E];
            Elems<T>::get(cur[u], e);
#pragma unroll
            for (int i = 0; i < E; ++i) bits |= (e[i] >= tau ? 1u : 0u) << (u * E + i);
            if (base + u * TH + tid >= v1) bits &= ~(((1u << E) - 1u) << (u * E));
          }
          select(bits, [&](int i) { return head + (base + (i / E) * TH + tid) * E + i % E; });
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) cur[u] = nxt[u];
    }
  }
  if (rank == 0 && warp == 0) {
    // the elements outside the vectors: fewer than 2 E
    const int tail0 = head + nv * E, cnt = head + a.vocab - tail0;
    if (cnt > 0) {
      const int id = lane < head ? lane : tail0 + lane - head;
      const bool in = lane < cnt;
      const float e[2] = {in ? to_f<T>(x[id]) : -INFINITY, -INFINITY};
      add(std::integral_constant<int, 2>(), e, e[0] >= -INFINITY ? e[0] : -INFINITY, true);
      if (K > 0) select(in ? 1u : 0u, [&](int) { return id; });
    }
  }

  // ---- statistics: lanes, warps, CTAs
  st = warp_merge(st, c);
  if (lane == 0) s_stat[warp] = st;
  __syncthreads();
  // ---- top entries: the warps' keys that reach the threshold, ranked
  auto gather = [&](uint64_t key, uint32_t tau) {
    if (key && (uint32_t)(key >> 32) >= tau) s_key[atomicAdd(&s_n, 1u)] = key;
  };
  auto rank_of = [&](uint64_t key, int n) {
    int r = 0;
    for (int j = 0; j < n; ++j) r += s_key[j] > key;
    return r;
  };
  if (K > 0 && lane < K) gather(list, s_tau);
  if (warp == 0) {
    st = warp_merge(lane < WARPS ? s_stat[lane] : Stat{-INFINITY, 0.f, 0.f}, c);
    if (lane == 0) s_cta = st;
  }
  if (cluster > 1) {
    cg::cluster_group cl = cg::this_cluster();
    __syncthreads();
    if (tid < (int)s_n) {  // at most WARPS * 32 = TH
      const uint64_t key = s_key[tid];
      const int r = rank_of(key, (int)s_n);
      if (r < K) s_out[r] = key;
    }
    cl.sync();
    if (rank == 0) {
      uint32_t tau = lane < cluster ? *cl.map_shared_rank(&s_tau, lane) : 0u;
      tau = __reduce_max_sync(0xffffffffu, tau);
      uint64_t k0 = 0, k1 = 0;
      if (tid < cluster * K) k0 = *cl.map_shared_rank(&s_out[tid % K], tid / K);
      if (tid + TH < cluster * K) k1 = *cl.map_shared_rank(&s_out[(tid + TH) % K], (tid + TH) / K);
      if (warp == 0) {
        st = warp_merge(lane < cluster ? *cl.map_shared_rank(&s_cta, lane) : Stat{-INFINITY, 0.f, 0.f}, c);
        if (lane == 0) s_row = st;
      }
      if (tid == 0) s_n = 0;
      __syncthreads();
      gather(k0, tau);
      gather(k1, tau);
    }
    cl.sync();  // no CTA leaves while its shared memory is read
    if (rank != 0) return;
  } else {
    if (tid == 0) s_row = st;
    __syncthreads();
  }
  st = s_row;
  const float nan = __int_as_float(0x7fffffff);
  constexpr float ln2 = 0.6931471805599453f;
  // an all -inf row has no distribution
  const float ls = st.m == -INFINITY ? nan : log2f(st.s);
  if (tid == 0) {
    float lp = 0.f;
    if (tok >= 0 && tok < a.vocab) {
      lp = ((xt - st.m) * c - ls) * ln2;
    } else if (tok != -1) {
      lp = nan;
      if (a.status) atomicOr(a.status, DFLASH_STATUS_TOKEN);
    }
    a.logprobs[row] = lp;
    if (a.entropy) a.entropy[row] = (ls - st.t / st.s) * ln2;
  }
  if (K > 0) {
    const int n = (int)s_n;
    const int64_t o = (int64_t)row * K;
    for (int i = tid; i < n; i += TH) {
      const uint64_t key = s_key[i];
      const int r = rank_of(key, n);
      if (r >= K) continue;
      a.top_ids[o + r] = (int32_t)(0xffffffffu - (uint32_t)key);
      a.top_logprobs[o + r] = ((float_of_order((uint32_t)(key >> 32)) - st.m) * c - ls) * ln2;
    }
    if (tid >= n && tid < K) {  // fewer than K entries are not NaN
      a.top_ids[o + tid] = -1;
      a.top_logprobs[o + tid] = nan;
    }
  }
}

template <typename T>
cudaError_t launch_logprobs(const dflash_logprobs& a, int sms, cudaStream_t st) {
  // the smallest cluster that gives every SM two CTAs, while a CTA keeps at
  // least one full batch of its threads (4096 fp32 or 8192 bf16 elements)
  int cluster = 1;
  while (cluster < kMaxCluster && (int64_t)a.rows * cluster < 2 * sms &&
         (int64_t)a.vocab * (int)sizeof(T) >= (int64_t)cluster * 2 * TH * U * 16)
    cluster *= 2;
  static bool attr[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !attr[dev]) {
    e = cudaFuncSetAttribute(k_token_logprobs<T>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    if (dev < 64) attr[dev] = true;
  }
  const float c = (float)(1.4426950408889634 / (double)a.temperature);
  return launch_kc(k_token_logprobs<T>, (unsigned)(a.rows * cluster), TH, 0, st, cluster, a, cluster, c);
}

}  // namespace
}  // namespace dfl

using namespace dfl;

extern "C" DFLASH_API int dflash_token_logprobs(const dflash_logprobs* a, void* stream) {
  auto bad = [](const char* m) { return dflash__set_error(DFLASH_ERR_INVALID_ARG, m); };
  if (!a) return bad("dflash_token_logprobs: null argument");
  if (a->dtype != DFLASH_DTYPE_F32 && a->dtype != DFLASH_DTYPE_BF16) return bad("dflash_token_logprobs: dtype");
  if (a->rows < 0 || a->rows > (1 << 26) || a->vocab < 1 || a->vocab > (1 << 24) || a->row_stride < a->vocab ||
      a->row_stride >= ((int64_t)1 << 38))
    return bad("dflash_token_logprobs: rows outside 0..2^26, vocab outside 1..2^24 or row_stride below it");
  if (a->top < 0 || a->top > DFLASH_LOGPROBS_MAX_TOP || a->top > a->vocab)
    return bad("dflash_token_logprobs: top outside 0..32 or above vocab");
  if (!(a->temperature > 0.f) || !std::isfinite(a->temperature) || !std::isfinite(1.5f / a->temperature))
    return bad("dflash_token_logprobs: temperature: finite, > 0, with a finite reciprocal");
  if (a->rows == 0) return DFLASH_OK;
  if (!a->logits || !a->tokens || !a->logprobs || (a->top && (!a->top_ids || !a->top_logprobs)))
    return bad("dflash_token_logprobs: null pointer");
  if ((uintptr_t)a->logits % (a->dtype == DFLASH_DTYPE_F32 ? 4 : 2))
    return bad("dflash_token_logprobs: logits not aligned to their type");
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess)
    e = a->dtype == DFLASH_DTYPE_F32 ? launch_logprobs<float>(*a, sms, (cudaStream_t)stream)
                                     : launch_logprobs<bf16>(*a, sms, (cudaStream_t)stream);
  if (e != cudaSuccess) return dflash__set_error(DFLASH_ERR_CUDA, cudaGetErrorString(e));
  return DFLASH_OK;
}
