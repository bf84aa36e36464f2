// Log probabilities of given tokens with the distribution's entropy and its
// top entries.  With c = log2(e) / T, d_v = (l_v - m) c for the running maximum
// m of l, s = sum 2^d and t = sum 2^d d:
//   log2 p(v) = d_v - log2 s,   H / ln 2 = log2 s - t / s.
// (The difference before the product: the largest entry's d is exactly 0, and a
// row of one possible token has entropy 0.)
// One pass over the logits: (m, s, t) per thread, rescaled when its maximum
// grows, and the top entries beside it.  Bound by reading the logits once: 2047
// rows of 151936 bf16 in 98 us without top entries, 6.3 TB/s (94% of a measured
// copy), 116 with 5, 159 with 32.  16 rows of fp32 are latency: 6 us without, 12.5
// with 20.
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
// threshold is the K-th largest of the threads' maxima of the first batch (found
// among those that reach the smallest, over the warps, of each warp's r-th,
// r = ceil(K / warps)).  What reaches it goes into a shared buffer as a key
// (value's order above, ~id below); after 2, 4, 8, ... batches and in the end
// the keys are ranked by counting the larger ones, the best K stay and the K-th
// becomes the threshold.  (A row in ascending order fills the buffer between
// two rankings: what does not fit goes into sorted lists of 32, one per warp.)
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include <atomic>
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
constexpr int H = 4;       // batches looked at together
constexpr int CAP = TH;    // keys between two rankings (half of a buffer)
constexpr int kMaxCluster = 16;

__device__ __forceinline__ float lp_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 2^d is 0 in fp32 far above this: a d below it (a masked entry at the type's
// lowest value may be at -inf) is put here where it multiplies a 0.
constexpr float kFar = -1000.f;

// (m, s, t) of a set of entries; m = -inf: no entry above -inf.
struct Stat {
  float m, s, t;
};
// The union of the lanes' sets, in every lane.
__device__ __forceinline__ Stat warp_merge(Stat a, float c) {
  const float M = warp_max(a.m);
  // a side at -inf has s = t = 0 (or NaN, which stays)
  const float d = a.m == -INFINITY ? 0.f : fmaxf((a.m - M) * c, kFar), f = exp2f(d);
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
// The r-th largest (1-based) of the lanes' words.
__device__ __forceinline__ uint32_t rth_of_lanes(uint32_t v, int r, int lane) {
  uint32_t m = __reduce_max_sync(0xffffffffu, v);
  for (; r > 1; --r) {
    if (lane == __ffs(__ballot_sync(0xffffffffu, v == m)) - 1) v = 0;
    m = __reduce_max_sync(0xffffffffu, v);
  }
  return m;
}

template <typename T>
__global__ void __launch_bounds__(TH, 4) k_token_logprobs(dflash_logprobs a, int cluster, float c, float inv_t) {
  constexpr int E = Elems<T>::E, N = U * E;
  // keys of the running round: [0, CAP) in turn, [CAP, 2 CAP) the warps' lists
  __shared__ uint64_t s_key[2][2 * CAP], s_all[kMaxCluster * 32], s_out[32];
  __shared__ Stat s_stat[WARPS], s_cta, s_row;
  __shared__ uint32_t s_first[WARPS], s_max[TH];
  __shared__ uint4 s_stage[WARPS][H][U];
  __shared__ uint32_t s_tau, s_n[2], s_nlist[2], s_nall, s_nmax;  // float_order of the threshold; counts
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row = blockIdx.x / cluster, rank = blockIdx.x % cluster, K = a.top;
  if (tid == 0) {
    s_tau = float_order(-INFINITY);
    s_n[0] = s_n[1] = s_nlist[0] = s_nlist[1] = s_nall = s_nmax = 0;
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
  // adds n elements with maximum hi; clamp: some d may be below kFar (a NaN
  // still comes in through p)
  auto add = [&](auto n_, const float* e, float hi, bool clamp) {
    constexpr int n = decltype(n_)::value;
    if (hi > st.m) {
      const float dm = fmaxf((st.m - hi) * c, kFar), f = lp_ex2(dm);
      st.t = f * fmaf(st.s, dm, st.t);
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
      if (clamp) d = pack2(fmaxf(dd.x, kFar), fmaxf(dd.y, kFar));
      asm("add.rn.f32x2 %0, %0, %1;" : "+l"(s2) : "l"(pp));
      asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(t2) : "l"(pp), "l"(d));
    }
    const float2 sf = unpack2(s2), tf = unpack2(t2);
    st.s += sf.x + sf.y;
    st.t += tf.x + tf.y;
  };
  int side = 0;
  // the lanes' keys (0: none) into the warp's list
  auto insert = [&](uint64_t key) {
    uint32_t todo = __ballot_sync(0xffffffffu, key > kth);
    while (todo) {
      const uint64_t k2 = __shfl_sync(0xffffffffu, key, __ffs(todo) - 1);
      todo &= todo - 1;
      if (k2 > kth) {
        list_insert(list, k2, lane);
        kth = __shfl_sync(0xffffffffu, list, K - 1);
      }
    }
    if (kth && lane == 0) atomicMax(&s_tau, (uint32_t)(kth >> 32));
  };
  // The elements of a batch that reach tau, into the buffer; bit i of the result:
  // element i found it full.
  auto append = [&](const uint4* cur, int base, float tau) {
    uint32_t full = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int v = base + u * TH + tid;
      float e[E];
      Elems<T>::get(cur[u], e);
#pragma unroll
      for (int i = 0; i < E; ++i)
        if (e[i] >= tau && v < v1) {
          const uint32_t pos = atomicAdd(&s_n[side], 1u);
          if (pos < CAP) s_key[side][pos] = order_key(e[i], head + v * E + i);
          else full |= 1u << (u * E + i);
        }
    }
    return full;
  };
  // The batches of the lanes in `hits`, four at a time through shared memory:
  // the whole warp looks at one, an element a lane.
  auto look = [&](uint32_t hits, const uint4* cur, int base, auto each) {
    while (hits) {
      const int q = __popc(hits & ((1u << lane) - 1u));
      if (((hits >> lane) & 1u) && q < H) {
#pragma unroll
        for (int u = 0; u < U; ++u) s_stage[warp][q][u] = cur[u];
      }
      __syncwarp();
#pragma unroll 1
      for (int h = 0; h < H && hits; ++h) {
        const int src = __ffs(hits) - 1;
        hits &= hits - 1;
        const int v = base + (lane / E) * TH + warp * 32 + src;
        const float e = lane < N ? to_f<T>(reinterpret_cast<const T*>(s_stage[warp][h])[lane]) : 0.f;
        each(src, lane < N && v < v1, e, head + v * E + lane % E);
      }
      __syncwarp();
    }
  };
  auto candidates = [&](const uint4* cur, int base, float hi, float tau) {
    if constexpr (E == 4) {
      // 16 elements a lane: each lane offers its own.  What does not fit goes to the warps' lists
      const uint32_t full = append(cur, base, tau), hits = __ballot_sync(0xffffffffu, full != 0);
      if (hits)
        look(hits, cur, base, [&](int src, bool in, float e, int id) {
          const uint32_t bits = __shfl_sync(0xffffffffu, full, src);
          insert(in && ((bits >> lane) & 1u) ? order_key(e, id) : 0ull);
        });
    } else {
      // 32 elements a lane: unrolled as above they would not leave registers
      // enough for the sums (97 -> 187 us for 2047 rows)
      look(__ballot_sync(0xffffffffu, hi >= tau), cur, base, [&](int, bool in, float e, int id) {
        const bool yes = in && e >= tau;
        const uint32_t m = __ballot_sync(0xffffffffu, yes);
        if (!m) return;
        int pos = 0;
        if (lane == 0) pos = (int)atomicAdd(&s_n[side], (uint32_t)__popc(m));
        const int first = __shfl_sync(0xffffffffu, pos, 0);
        pos = first + __popc(m & ((1u << lane) - 1u));
        const uint64_t key = yes ? order_key(e, id) : 0ull;
        if (yes && pos < CAP) s_key[side][pos] = key;
        if (first + __popc(m) > CAP) insert(pos >= CAP ? key : 0ull);
      });
    }
  };
  // Ranks the round's keys; the best K go to dst in order (their count is the
  // result), and the K-th becomes the threshold.  The next round is the other side.
  auto rank_round = [&](uint64_t* dst) {
    if (__any_sync(0xffffffffu, list != 0)) {  // rare: the buffer overflowed
      uint32_t at = 0;
      const uint32_t m = __ballot_sync(0xffffffffu, list != 0);
      if (lane == 0) at = atomicAdd(&s_nlist[side], (uint32_t)__popc(m));
      at = __shfl_sync(0xffffffffu, at, 0);
      if (list) s_key[side][CAP + at + lane] = list;  // sorted: the first popc(m) lanes
      list = kth = 0;
    }
    __syncthreads();
    const int n = min((int)s_n[side], CAP), nl = (int)s_nlist[side], have = min(n + nl, K);
    const uint64_t* buf = s_key[side];
    for (int i = tid; i < n + nl; i += TH) {
      const uint64_t key = buf[i < n ? i : CAP + i - n];
      int r = 0;
#pragma unroll 8
      for (int j = 0; j < n; ++j) r += buf[j] > key;
      for (int j = 0; j < nl; ++j) r += buf[CAP + j] > key;
      if (r < K) dst[r] = key;
      if (r == K - 1) atomicMax(&s_tau, (uint32_t)(key >> 32));
    }
    side ^= 1;
    if (tid == 0) {
      s_n[side] = have;
      s_nlist[side] = 0;
    }
    __syncthreads();
    return have;
  };
  // first ranking of the candidates: after two batches; none of a slice of three
  // (16 rows of fp32 with 20 entries 13.4 -> 12.9 us; long rows with 32 159 us, 165
  // after four)
  int batch = 0, refresh = v1 - v0 <= 3 * U * TH ? 4 : 2;
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
        const uint32_t mine = float_order(hi), r = rth_of_lanes(mine, (K + WARPS - 1) / WARPS, lane);
        if (lane == 0) s_first[warp] = r;
        __syncthreads();
        uint32_t t = s_first[0];
#pragma unroll
        for (int w = 1; w < WARPS; ++w) t = min(t, s_first[w]);
        // of the maxima that reach it (K at least), the K-th is the threshold
        if (mine >= t) s_max[atomicAdd(&s_nmax, 1u)] = mine;
        __syncthreads();
        const int n = (int)s_nmax;
        if (tid < n) {
          const uint32_t v = s_max[tid];
          int r = 0;
#pragma unroll 8
          for (int j = 0; j < n; ++j) r += s_max[j] > v || (s_max[j] == v && j < tid);
          if (r == K - 1) atomicMax(&s_tau, v);
        }
        __syncthreads();
      }
      {
        float e[N];
#pragma unroll
        for (int u = 0; u < U; ++u) Elems<T>::get(cur[u], e + u * E);
        if ((lo - fmaxf(st.m, hi)) * c > kFar) add(std::integral_constant<int, N>(), e, hi, false);
        else add(std::integral_constant<int, N>(), e, hi, true);
      }
      if (K > 0) {
        const float tau = float_of_order(*(volatile uint32_t*)&s_tau);
        if (__any_sync(0xffffffffu, hi >= tau)) {
          candidates(cur, base, hi, tau);
        }
        if (++batch == refresh) {
          refresh *= 2;
          rank_round(s_key[side ^ 1]);
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
      if (K > 0) {
        uint64_t left = 0;
        if (in && e[0] >= float_of_order(*(volatile uint32_t*)&s_tau)) {
          const uint32_t pos = atomicAdd(&s_n[side], 1u);
          if (pos < CAP) s_key[side][pos] = order_key(e[0], id);
          else left = order_key(e[0], id);
        }
        if (__any_sync(0xffffffffu, left != 0)) insert(left);
      }
    }
  }

  // ---- statistics: lanes, warps, CTAs
  st = warp_merge(st, c);
  if (lane == 0) s_stat[warp] = st;
  __syncthreads();
  if (warp == 0) {
    st = warp_merge(lane < WARPS ? s_stat[lane] : Stat{-INFINITY, 0.f, 0.f}, c);
    if (lane == 0) s_cta = s_row = st;
  }
  // ---- top entries: of the CTA, then of the cluster
  int n = K > 0 ? rank_round(s_out) : 0;
  if (cluster > 1) {
    cg::cluster_group cl = cg::this_cluster();
    cl.sync();
    if (rank == 0) {
      // The first ceil(K / cluster) entries of every CTA, at most 32: K of them
      // at least, and the K-th largest is a threshold that K entries reach.
      uint32_t t = 0;
      if (K > 0) {
        const int r = (K + cluster - 1) / cluster;
        uint32_t v = 0;
        if (lane < cluster * r) v = (uint32_t)(*cl.map_shared_rank(&s_out[lane / cluster], lane % cluster) >> 32);
        int above = 0;
#pragma unroll 8
        for (int j = 0; j < 32; ++j) {
          const uint32_t o = __shfl_sync(0xffffffffu, v, j);
          above += o > v || (o == v && j < lane);
        }
        t = __shfl_sync(0xffffffffu, v, __ffs(__ballot_sync(0xffffffffu, above == K - 1)) - 1);
      }
      uint64_t kk[2] = {0, 0};
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int j = tid + i * TH;
        if (j < cluster * K) kk[i] = *cl.map_shared_rank(&s_out[j % K], j / K);
      }
      if (warp == 0) {
        st = warp_merge(lane < cluster ? *cl.map_shared_rank(&s_cta, lane) : Stat{-INFINITY, 0.f, 0.f}, c);
        if (lane == 0) s_row = st;
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (kk[i] && (uint32_t)(kk[i] >> 32) >= t) s_all[atomicAdd(&s_nall, 1u)] = kk[i];
    }
    cl.sync();  // no CTA leaves while its shared memory is read
    if (rank != 0) return;
  } else {
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
      lp = fmaf(xt - st.m, inv_t, -ls * ln2);
    } else if (tok != -1) {
      lp = nan;
      if (a.status) atomicOr(a.status, DFLASH_STATUS_TOKEN);
    }
    a.logprobs[row] = lp;
    if (a.entropy) a.entropy[row] = (ls - st.t / st.s) * ln2;
  }
  if (K > 0) {
    const int64_t o = (int64_t)row * K;
    auto put = [&](uint64_t k, int r) {
      a.top_ids[o + r] = (int32_t)(0xffffffffu - (uint32_t)k);
      a.top_logprobs[o + r] = fmaf(float_of_order((uint32_t)(k >> 32)) - st.m, inv_t, -ls * ln2);
    };
    if (cluster > 1) {
      n = (int)s_nall;
      for (int i = tid; i < n; i += TH) {
        const uint64_t k = s_all[i];
        int r = 0;
#pragma unroll 8
        for (int j = 0; j < n; ++j) r += s_all[j] > k;
        if (r < K) put(k, r);
      }
    } else if (tid < n) {
      put(s_out[tid], tid);
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
  static std::atomic<bool> attr[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !attr[dev]) {
    e = cudaFuncSetAttribute(k_token_logprobs<T>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    if (dev < 64) attr[dev] = true;
  }
  const float c = (float)(1.4426950408889634 / (double)a.temperature), inv_t = (float)(1 / (double)a.temperature);
  return launch_kc(k_token_logprobs<T>, (unsigned)(a.rows * cluster), TH, 0, st, cluster, a, cluster, c, inv_t);
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
