// Rotary positions of the rows of a ragged batch.
//
// The angle of pair i at position p is p f_i.  In fp32 that loses the fraction of
// a turn at far positions (2^20 f has 2^-4 radians left of its 24 bits at f = 1), so
// f_i is kept as a fraction of a turn in 0.64 fixed point: p f_i mod 1 is the low 64
// bits of the product, exact but for the 2^-53 relative rounding of f_i itself.  Its
// upper 32 bits go to fp32 (an error of at most pi 2^-24) and sincospif.
#include <cmath>

#include "common.cuh"
#include "launch.h"
#include "target_checks.h"

namespace dfl {
namespace {

struct RopeSide {
  const void* x;
  void* y;
  int64_t x_row, x_head, y_row, y_head;
};
struct RopeCall {
  RopeSide side[2];
  int32_t heads[2];
  int32_t d, rot, off, copy;  // copy: the elements that pass through are written too
  float amplitude, sign;
};
struct RopeTurns {
  uint64_t t[DFLASH_ROPE_MAX_DIM / 2];
};

template <int BYTES> struct Raw;
template <> struct Raw<16> { using type = uint4; };
template <> struct Raw<8> { using type = uint2; };
template <> struct Raw<4> { using type = uint32_t; };
template <> struct Raw<2> { using type = uint16_t; };

template <typename T, int V>
struct Vec {
  typename Raw<V * (int)sizeof(T)>::type raw;
  __device__ __forceinline__ void load(const T* p) { raw = *reinterpret_cast<const decltype(raw)*>(p); }
  __device__ __forceinline__ void store(T* p) const { *reinterpret_cast<decltype(raw)*>(p) = raw; }
  __device__ __forceinline__ void get(float* f) const {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < V; ++i) f[i] = reinterpret_cast<const float*>(&raw)[i];
    } else if constexpr (V == 1) {
      f[0] = __uint_as_float((uint32_t)raw << 16);
    } else {
#pragma unroll
      for (int i = 0; i < V; i += 2) {
        const uint32_t w = reinterpret_cast<const uint32_t*>(&raw)[i / 2];
        f[i] = __uint_as_float(w << 16);
        f[i + 1] = __uint_as_float(w & 0xffff0000u);
      }
    }
  }
  __device__ __forceinline__ void set(const float* f) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < V; ++i) reinterpret_cast<float*>(&raw)[i] = f[i];
    } else if constexpr (V == 1) {
      raw = __bfloat16_as_ushort(__float2bfloat16_rn(f[0]));
    } else {
#pragma unroll
      for (int i = 0; i < V; i += 2) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(f[i], f[i + 1]);
        reinterpret_cast<uint32_t*>(&raw)[i / 2] = *reinterpret_cast<const uint32_t*>(&b);
      }
    }
  }
};

// RPC rows per CTA: cos and sin of a row are worked out once, by as many threads as there are pairs, and serve
// all its heads from shared memory.  A thread has one place of a head (V elements; in the half layout V of
// each half) and goes through (row, head) pairs `step` apart, U of them in flight: no index is divided,
// and what it needs of cos and sin is two to four 16-byte loads.
// Bound by memory traffic and by instruction slots about alike: 10300 rows of 40 heads of 128, half of
// a head rotated: 211 MB.
constexpr int kRopeThreads = 256;
template <typename T, int V, bool IL, int RPC>
__global__ void __launch_bounds__(kRopeThreads) k_rope(Ragged r, RopeCall c, const __grid_constant__ RopeTurns turns) {
  __shared__ __align__(16) float2 cs[RPC * (DFLASH_ROPE_MAX_DIM / 2)];
  __shared__ int pos[RPC];
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, row0 = blockIdx.x * RPC, half = c.rot / 2;
  for (int k = warp; k < RPC; k += kRopeThreads / 32) {
    const int row = row0 + k;
    int p = -1;
    if (row < r.total) {
      const int b = seq_of_row(r, row);
      if (b < r.batch) {  // (otherwise behind the last sequence)
        const Seq s = load_seq(r, b);
        const int i = row - s.start;
        if (!s.ok && lane == 0) flag_status(r.status, DFLASH_STATUS_BOUNDS);
        if (s.ok && i >= 0 && i < s.n) p = s.len - s.n + i;
      }
    }
    if (lane == 0) pos[k] = p;
  }
  __syncthreads();
  for (int e = tid; e < RPC * half; e += kRopeThreads) {
    const int k = e / half, i = e - k * half;
    const uint64_t a = (uint64_t)(uint32_t)max(pos[k], 0) * turns.t[i];
    float sn, cn;
    sincospif((float)(int32_t)(a >> 32) * 4.656612873077392578125e-10f, &sn, &cn);  // half turns: 2^-31
    cs[e] = make_float2(cn * c.amplitude, sn * c.amplitude * c.sign);
  }
  __syncthreads();
  constexpr int U = 4, P = IL ? V / 2 : V;  // pairs of a vector
  const int turned = IL ? c.rot / V : half / V, per = turned + (c.copy ? (c.d - c.rot) / V : 0);
  const int heads = c.heads[0] + c.heads[1], step = kRopeThreads / per, h0 = tid / per, j = tid - h0 * per;
  if (h0 >= step) return;
  const bool turns_here = j < turned;
  int at = (j - turned) * V;  // elements in front of the rotated part, or behind it
  if (turns_here) at = c.off + j * V;
  else if (at >= c.off) at += c.rot;
  int k = h0 / heads, h = h0 - k * heads;  // row and head of the next vector
  while (k < RPC) {
    Vec<T, V> a[U], b[U];
    T* y[U];
    int row[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      row[u] = k < RPC && pos[min(k, RPC - 1)] >= 0 ? k : -1;
      if (row[u] >= 0) {
        const int w = h >= c.heads[0], g = w ? h - c.heads[0] : h;
        const T* x = reinterpret_cast<const T*>(w ? c.side[1].x : c.side[0].x) +
                     (int64_t)(row0 + k) * (w ? c.side[1].x_row : c.side[0].x_row) + g * (w ? c.side[1].x_head : c.side[0].x_head) + at;
        y[u] = reinterpret_cast<T*>(w ? c.side[1].y : c.side[0].y) +
               (int64_t)(row0 + k) * (w ? c.side[1].y_row : c.side[0].y_row) + g * (w ? c.side[1].y_head : c.side[0].y_head) + at;
        a[u].load(x);
        if (!IL && turns_here) b[u].load(x + half);
      }
      h += step;
      while (h >= heads) {
        h -= heads;
        ++k;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (row[u] < 0) continue;
      if (turns_here) {
        float2 t[P];
        const float2* src = cs + row[u] * half + j * P;
        if constexpr (P % 2 == 0) {  // (then half is even too)
#pragma unroll
          for (int q = 0; q < P; q += 2) *reinterpret_cast<float4*>(t + q) = *reinterpret_cast<const float4*>(src + q);
        } else {
#pragma unroll
          for (int q = 0; q < P; ++q) t[q] = src[q];
        }
        float f[V], g[V];
        a[u].get(f);
        if constexpr (IL) {
#pragma unroll
          for (int q = 0; q < P; ++q) {
            g[2 * q] = f[2 * q] * t[q].x - f[2 * q + 1] * t[q].y;
            g[2 * q + 1] = f[2 * q + 1] * t[q].x + f[2 * q] * t[q].y;
          }
          a[u].set(g);
        } else {
          b[u].get(g);
#pragma unroll
          for (int q = 0; q < V; ++q) {
            const float p = f[q] * t[q].x - g[q] * t[q].y;
            g[q] = g[q] * t[q].x + f[q] * t[q].y;
            f[q] = p;
          }
          a[u].set(f);
          b[u].set(g);
          b[u].store(y[u] + half);
        }
      }
      a[u].store(y[u]);
    }
  }
}

template <typename T, int V, bool IL>
cudaError_t launch_rope(const Ragged& r, const RopeCall& c, const RopeTurns& t, cudaStream_t st) {
  // Few rows: one a CTA, so that they spread over the SMs, as long as all CTAs run at once (three an SM).  40 heads
  // of 128: 64 rows 3.4 us (four a CTA 5.4), 456 4.3 (5.4), 608 7.1 (5.4), 2000 15.3 (13.0).
  if (r.total <= 456) return launch_k(k_rope<T, V, IL, 1>, (unsigned)r.total, kRopeThreads, 0, st, r, c, t);
  return launch_k(k_rope<T, V, IL, 4>, (unsigned)((r.total + 3) / 4), kRopeThreads, 0, st, r, c, t);
}
template <typename T>
cudaError_t launch_rope(const Ragged& r, const RopeCall& c, const RopeTurns& t, bool il, cudaStream_t st) {
  constexpr int W = 16 / (int)sizeof(T);
  // elements of a vector: as wide as the rotated part's borders allow
  const int unit = il ? c.rot | c.off : c.rot / 2 | c.off;
  if (il)
    return unit % W == 0       ? launch_rope<T, W, true>(r, c, t, st)
           : unit % (W / 2) == 0 ? launch_rope<T, W / 2, true>(r, c, t, st)
                                 : launch_rope<T, 2, true>(r, c, t, st);
  return unit % W == 0       ? launch_rope<T, W, false>(r, c, t, st)
         : unit % (W / 2) == 0 ? launch_rope<T, W / 2, false>(r, c, t, st)
                               : launch_rope<T, 1, false>(r, c, t, st);
}

bool positive(double x) { return x > 0 && std::isfinite(x); }

}  // namespace
}  // namespace dfl

using namespace dfl;

extern "C" {

DFLASH_API int dflash_rope_init(const dflash_rope_config* c, dflash_rope_table* table) {
  const char* call = "dflash_rope_init";
  if (!c || !table) return rfail(DFLASH_ERR_INVALID_ARG, call, "null config or table");
  if (c->rot_dim < 2 || c->rot_dim > DFLASH_ROPE_MAX_DIM || c->rot_dim % 2 || c->offset < 0 || c->offset % 2 ||
      c->offset > DFLASH_ROPE_MAX_DIM - c->rot_dim)
    return rfail(DFLASH_ERR_SHAPE, call, "rot_dim: even, 2..256; offset: even, offset + rot_dim at most 256");
  if ((c->layout != DFLASH_ROPE_HALF && c->layout != DFLASH_ROPE_INTERLEAVED) || c->scaling < DFLASH_ROPE_NONE ||
      c->scaling > DFLASH_ROPE_YARN)
    return rfail(DFLASH_ERR_INVALID_ARG, call, "layout or scaling");
  if (!(c->theta > 1) || !std::isfinite(c->theta)) return rfail(DFLASH_ERR_INVALID_ARG, call, "theta: finite, > 1");
  if (!(c->amplitude >= 0) || !std::isfinite((float)c->amplitude))
    return rfail(DFLASH_ERR_INVALID_ARG, call, "amplitude: finite, >= 0");
  const bool banded = c->scaling == DFLASH_ROPE_BANDS || c->scaling == DFLASH_ROPE_YARN;
  if (c->scaling != DFLASH_ROPE_NONE && !positive(c->factor)) return rfail(DFLASH_ERR_INVALID_ARG, call, "factor: finite, > 0");
  if (c->scaling == DFLASH_ROPE_YARN && c->factor < 1) return rfail(DFLASH_ERR_INVALID_ARG, call, "factor: >= 1 for YARN");
  if (banded && (!positive(c->original_len) || !positive(c->low) || !positive(c->high) || c->high <= c->low))
    return rfail(DFLASH_ERR_INVALID_ARG, call, "original_len > 0, 0 < low < high");
  const double R = c->rot_dim, two_pi = 6.283185307179586476925;
  double theta = c->theta;
  if (c->scaling == DFLASH_ROPE_NTK) {
    if (c->rot_dim == 2) return rfail(DFLASH_ERR_SHAPE, call, "NTK: rot_dim above 2");
    theta *= std::pow(c->factor, R / (R - 2));
    if (!std::isfinite(theta) || !(theta > 1)) return rfail(DFLASH_ERR_INVALID_ARG, call, "NTK: the stretched theta is not above 1");
  }
  double from = 0, to = 0;
  if (c->scaling == DFLASH_ROPE_YARN) {
    auto pair_of = [&](double turns) { return R * std::log(c->original_len / (two_pi * turns)) / (2 * std::log(theta)); };
    from = std::max(std::floor(pair_of(c->high)), 0.0);
    to = std::min(std::ceil(pair_of(c->low)), R - 1);
  }
  table->rot_dim = c->rot_dim;
  table->offset = c->offset;
  table->layout = c->layout;
  table->amplitude = (float)(c->amplitude > 0                     ? c->amplitude
                             : c->scaling == DFLASH_ROPE_YARN ? 0.1 * std::log(c->factor) + 1.0
                                                              : 1.0);
  for (int i = 0; i < DFLASH_ROPE_MAX_DIM / 2; ++i) {
    if (2 * i >= c->rot_dim) {
      table->turns[i] = 0;
      continue;
    }
    double f = std::pow(theta, -2.0 * i / R);
    if (c->scaling == DFLASH_ROPE_LINEAR) f /= c->factor;
    if (c->scaling == DFLASH_ROPE_BANDS) {
      const double u = c->original_len * f / two_pi;
      const double s = std::min(std::max((u - c->low) / (c->high - c->low), 0.0), 1.0);
      f *= (1 - s) / c->factor + s;
    }
    if (c->scaling == DFLASH_ROPE_YARN) {
      const double s = std::min(std::max((i - from) / std::max(to - from, 0.001), 0.0), 1.0);
      f = f / c->factor * s + f * (1 - s);
    }
    const double turn = f / two_pi;
    table->turns[i] = (uint64_t)std::ldexp(turn - std::floor(turn), 64);  // below 2^64: the fraction is below 1
  }
  return DFLASH_OK;
}

DFLASH_API int dflash_rope(const dflash_rope_table* table, const dflash_ragged* batch, const dflash_rope_call* a,
                           void* stream) {
  const char* call = "dflash_rope";
  if (!table || !a) return rfail(DFLASH_ERR_INVALID_ARG, call, "null table or call");
  if (int rc = check_ragged(call, batch, nullptr, true)) return rc;
  if (a->dtype != DFLASH_DTYPE_F32 && a->dtype != DFLASH_DTYPE_BF16) return rfail(DFLASH_ERR_INVALID_ARG, call, "dtype");
  if (batch->lens && (batch->max_len < 1 || batch->max_len > (1 << 30)))
    return rfail(DFLASH_ERR_INVALID_ARG, call, "max_len outside 1..2^30");
  if (table->rot_dim < 2 || table->rot_dim > DFLASH_ROPE_MAX_DIM || table->rot_dim % 2 || table->offset < 0 ||
      table->offset % 2 || table->offset > DFLASH_ROPE_MAX_DIM - table->rot_dim ||
      (table->layout != DFLASH_ROPE_HALF && table->layout != DFLASH_ROPE_INTERLEAVED))
    return rfail(DFLASH_ERR_INVALID_ARG, call, "table: not what dflash_rope_init made");
  if (a->head_dim < 8 || a->head_dim > DFLASH_ROPE_MAX_DIM || a->head_dim % 8 || table->offset + table->rot_dim > a->head_dim)
    return rfail(DFLASH_ERR_SHAPE, call, "head_dim: a multiple of 8 up to 256 that holds the rotated part");
  if (a->n_q_heads < 0 || a->n_q_heads > 1024 || a->n_k_heads < 0 || a->n_k_heads > 1024 || a->n_q_heads + a->n_k_heads == 0)
    return rfail(DFLASH_ERR_SHAPE, call, "heads outside 0..1024, or none");
  if (a->transpose != 0 && a->transpose != 1) return rfail(DFLASH_ERR_INVALID_ARG, call, "transpose: 0 or 1");
  const bool rows = batch->total_rows > 0;
  const dflash_heads* in[2] = {&a->q, &a->k};
  const dflash_heads* out[2] = {&a->q_out, &a->k_out};
  RopeCall c{};
  bool copy = false;
  for (int i = 0; i < 2; ++i) {
    c.heads[i] = i ? a->n_k_heads : a->n_q_heads;
    if (!c.heads[i]) continue;
    if (int rc = check_heads(call, in[i], a->dtype, c.heads[i], a->head_dim, rows)) return rc;
    if (int rc = check_heads(call, out[i], a->dtype, c.heads[i], a->head_dim, rows)) return rc;
    const bool same = in[i]->data == out[i]->data;
    if (same && rows && (in[i]->row_stride != out[i]->row_stride || in[i]->head_stride != out[i]->head_stride))
      return rfail(DFLASH_ERR_INVALID_ARG, call, "in place: the strides of input and output are the same");
    copy |= !same;
    c.side[i] = RopeSide{in[i]->data, out[i]->data, in[i]->row_stride, in[i]->head_stride, out[i]->row_stride, out[i]->head_stride};
  }
  if (!rows) return DFLASH_OK;
  c.d = a->head_dim;
  c.rot = table->rot_dim;
  c.off = table->offset;
  c.copy = copy;
  c.amplitude = table->amplitude;
  c.sign = a->transpose ? -1.f : 1.f;
  Ragged r = make_ragged(batch, nullptr);
  r.max_rows = batch->total_rows;
  r.max_len = batch->lens ? batch->max_len : batch->total_rows;
  r.lens = batch->lens;
  RopeTurns t;
  std::copy(table->turns, table->turns + DFLASH_ROPE_MAX_DIM / 2, t.t);
  const bool il = table->layout == DFLASH_ROPE_INTERLEAVED;
  cudaStream_t st = (cudaStream_t)stream;
  return rcheck(a->dtype == DFLASH_DTYPE_F32 ? launch_rope<float>(r, c, t, il, st) : launch_rope<bf16>(r, c, t, il, st), call);
}

}  // extern "C"
