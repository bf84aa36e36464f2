// New K/V rows into 8-bit pages with a scale for each page and KV head.
//
// For the new rows x of a page and head:  s = the smallest power of two with
// |x| <= 448 s, at least the page's scale if it holds rows in front of them;
// code = e4m3(x / s).  Powers of two make x / s exact, and a scale that grows only
// shifts the exponents of the codes that are there.
#include "common.cuh"
#include "kv8.h"
#include "launch.h"
#include "target_checks.h"
#include "kv8_checks.h"

namespace dfl {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;

template <typename T> struct Eight;  // eight elements
template <> struct Eight<bf16> {
  static constexpr int HOLD = 8;  // steps of a warp whose rows stay in registers
  uint4 a;
  __device__ __forceinline__ void load(const bf16* p) { a = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void get(float* f) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  // The running maximum of magnitudes: bits of a float without its sign order as integers do, two bf16 a word.
  __device__ __forceinline__ void most(uint32_t& m) const {
    m = __vmaxu2(__vmaxu2(__vmaxu2(m, a.x & 0x7fff7fffu), __vmaxu2(a.y & 0x7fff7fffu, a.z & 0x7fff7fffu)), a.w & 0x7fff7fffu);
  }
  static __device__ __forceinline__ uint32_t bits(uint32_t m) { return max(m << 16, m & 0xffff0000u); }
};
template <> struct Eight<float> {
  static constexpr int HOLD = 4;
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const float4*>(p);
    b = *reinterpret_cast<const float4*>(p + 4);
  }
  __device__ __forceinline__ void get(float* f) const {
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
    f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  }
  __device__ __forceinline__ void most(uint32_t& m) const {
    float f[8];
    get(f);
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(f[i]) & 0x7fffffffu);
  }
  static __device__ __forceinline__ uint32_t bits(uint32_t m) { return m; }
};

// The exponent of the smallest power of two s with most <= 448 s = 1.75 2^8 s.
__device__ __forceinline__ float scale_for(uint32_t u) {  // (bits of most)
  const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return __uint_as_float((uint32_t)(min(max(e, -60), 60) + 127) << 23);
}

// Pieces of a sequence: the pages that receive its new rows.
__device__ __forceinline__ int pieces_of(const Seq& s, int shift) {
  return s.ok && s.n > 0 ? ((s.len - 1) >> shift) - ((s.len - s.n) >> shift) + 1 : 0;
}

struct Rows8 {
  const void* x[2];
  int64_t row[2], head[2];
};

// A CTA takes 8 / WPT tasks of one piece, WPT warps each; a task is K or V of one head.
// d / 8 lanes a row.  The rows of up to HOLD steps stay in registers between the pass that
// finds the scale and the one that writes; longer pieces are read again.  Elements that are not finite are
// looked for only where the largest magnitude is one.
// Bound by instruction slots: a warp's way to its rows (lengths, page, scale: 300 instructions) and about 60 for
// 16 rows' bytes a lane.  As few warps a task as hold its rows.
template <typename T, int WPT>
__global__ void __launch_bounds__(kThreads) k_kv8_append(Ragged r, Rows8 x, Kv8View kv, int heads, int d, int per_lane) {
  constexpr int HOLD = Eight<T>::HOLD;
  __shared__ uint32_t most_w[kWarps];
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  r.starts = after_wait(r.starts);
  r.lens = after_wait(r.lens);
  // the piece's sequence and page: every warp finds it for itself
  int rest = blockIdx.x, b = -1, j = 0;
  Seq s{0, 0, 0, false};
  for (int base = 0; base < r.batch; base += 32) {
    Seq c{0, 0, 0, false};
    if (base + lane < r.batch) c = load_seq(r, base + lane);
    const int n = pieces_of(c, kv.page_shift);
    int incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += u;
    }
    const unsigned found = __ballot_sync(0xffffffffu, incl > rest);
    if (found) {
      const int src = __ffs(found) - 1;
      j = rest - __shfl_sync(0xffffffffu, incl - n, src);
      b = base + src;
      s.start = __shfl_sync(0xffffffffu, c.start, src);
      s.n = __shfl_sync(0xffffffffu, c.n, src);
      s.len = __shfl_sync(0xffffffffu, c.len, src);
      break;
    }
    rest -= __shfl_sync(0xffffffffu, incl, 31);
    if (rest < 0) break;  // (lengths that overflow: no one's piece)
  }
  // one warp tells of bad sequences, all of them: in the last CTA, which has the last piece or none
  if (blockIdx.x == gridDim.x - 1 && blockIdx.y == 0 && warp == 0)
    for (int i = lane; i < r.batch; i += 32)
      if (!load_seq(r, i).ok) flag_status(r.status, DFLASH_STATUS_BOUNDS);
  if (b < 0) return;
  const int first = s.len - s.n, page = (first >> kv.page_shift) + j, size = 1 << kv.page_shift;
  const int p0 = max(first, page << kv.page_shift), p1 = min(s.len, (page + 1) << kv.page_shift);
  const int s0 = p0 & (size - 1), n = p1 - p0, row0 = s.start + p0 - first;
  const int task = blockIdx.y * (kWarps / WPT) + warp / WPT, part = warp % WPT;
  const int pg = r.table[(int64_t)b * r.table_stride + page];  // on its way while the rows are asked for
  const bool live = task < 2 * heads;  // (a warp without a task still meets the barrier)
  const int w = task >= heads, h = live ? task - w * heads : 0;
  // (lane / lpr as lane per_lane / 2^16)
  const int lpr = d / 8, rpw = 32 * per_lane >> 16, mine = lane * per_lane >> 16, col = (lane - mine * lpr) * 8;
  const bool in = live && mine < rpw;
  const T* src = reinterpret_cast<const T*>(w ? x.x[1] : x.x[0]) + (int64_t)row0 * (w ? x.row[1] : x.row[0]) +
                 h * (w ? x.head[1] : x.head[0]) + col;
  const int64_t src_row = w ? x.row[1] : x.row[0];
  const int step = rpw * WPT, steps = (n + step - 1) / step, at = part * rpw + mine;
  Eight<T> hold[HOLD];
#pragma unroll
  for (int t = 0; t < HOLD; ++t)
    if (in && at + t * step < n) hold[t].load(src + (at + t * step) * src_row);
  if (pg < 0 || pg >= kv.n_pages) {
    if (threadIdx.x == 0) flag_status(r.status, DFLASH_STATUS_PAGE);
    return;
  }
  float* scale = (w ? kv.vs : kv.ks) + (int64_t)pg * kv.s_page + h * kv.s_head;
  const float old = s0 > 0 ? *scale : 0.f;
  // f(element, slot) over this lane's rows
  auto each = [&](auto f) {
#pragma unroll
    for (int t = 0; t < HOLD; ++t)
      if (in && at + t * step < n) f(hold[t], at + t * step);
#pragma unroll 2
    for (int t = HOLD; t < steps; ++t)
      if (in && at + t * step < n) {
        Eight<T> e;
        e.load(src + (int64_t)(at + t * step) * src_row);
        f(e, at + t * step);
      }
  };
  // the largest magnitude of the task's rows, over its warps
  auto over_task = [&](uint32_t m) {
    m = __reduce_max_sync(0xffffffffu, m);
    if (WPT > 1) {
      __syncthreads();
      if (lane == 0) most_w[warp] = m;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < WPT; ++i) m = max(m, most_w[warp - part + i]);
    }
    return m;
  };
  uint32_t m = 0;
  each([&](const Eight<T>& e, int) { e.most(m); });
  uint32_t most = over_task(Eight<T>::bits(m));
  const bool wild = most >= 0x7f800000u;
  if (WPT > 1 ? __syncthreads_or(wild) : wild) {  // not finite: the largest of the others
    uint32_t fin = 0;
    each([&](const Eight<T>& e, int) {
      float f[8];
      e.get(f);
#pragma unroll
      for (int i = 0; i < 8; ++i) fin = max(fin, nonfinite(f[i]) ? 0u : __float_as_uint(f[i]) & 0x7fffffffu);
    });
    most = over_task(fin);
  }
  if (!live) return;
  const float now = s0 > 0 ? fmaxf(scale_for(most), old) : scale_for(most);
  uint8_t* dst = (w ? kv.v : kv.k) + (int64_t)pg * kv.page + h * kv.head + col;
  // an old scale may be any number: a power of two's reciprocal is exact, others divide
  const bool exact = (__float_as_uint(now) & 0x807fffffu) == 0;
  const float inv = 1.f / now;
  auto write = [&](const Eight<T>& e, int slot) {
    float f[8];
    e.get(f);
    uint32_t c[2];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float q = exact ? f[i] * inv : f[i] / now;
      f[i] = wild && nonfinite(f[i]) ? __uint_as_float(0x7fffffffu) : q;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
      c[i] = (uint32_t)f2_to_e4m3x2(f[4 * i], f[4 * i + 1]) | (uint32_t)f2_to_e4m3x2(f[4 * i + 2], f[4 * i + 3]) << 16;
    *reinterpret_cast<uint2*>(dst + (s0 + slot) * kv.slot) = make_uint2(c[0], c[1]);
  };
  if (exact && !wild) {
    each([&](const Eight<T>& e, int slot) {
      float f[8];
      e.get(f);
      uint32_t c[2];
#pragma unroll
      for (int i = 0; i < 2; ++i)
        c[i] = (uint32_t)f2_to_e4m3x2(f[4 * i] * inv, f[4 * i + 1] * inv) |
               (uint32_t)f2_to_e4m3x2(f[4 * i + 2] * inv, f[4 * i + 3] * inv) << 16;
      *reinterpret_cast<uint2*>(dst + (s0 + slot) * kv.slot) = make_uint2(c[0], c[1]);
    });
  } else {
    each(write);
  }
  if (s0 > 0 && now != old) {
    // the rows in front of the new ones: their codes at the new scale
    const float f = old / now;
    for (int slot = at; slot < s0; slot += step)
      if (in) {
        uint2* p = reinterpret_cast<uint2*>(dst + slot * kv.slot);
        const uint2 c = *p;
        const float4 a = e4m3x4_to_f4(c.x), b4 = e4m3x4_to_f4(c.y);
        *p = make_uint2((uint32_t)f2_to_e4m3x2(a.x * f, a.y * f) | (uint32_t)f2_to_e4m3x2(a.z * f, a.w * f) << 16,
                        (uint32_t)f2_to_e4m3x2(b4.x * f, b4.y * f) | (uint32_t)f2_to_e4m3x2(b4.z * f, b4.w * f) << 16);
      }
  }
  if (part == 0 && lane == 0 && now != old) *scale = now;
}

template <typename T, int WPT>
cudaError_t launch(const Ragged& r, const Rows8& x, const Kv8View& kv, int heads, int d, cudaStream_t st) {
  const int64_t pieces = (int64_t)(r.total >> kv.page_shift) + 2ll * std::min(r.batch, r.total);
  const int per = kWarps / WPT;
  return launch_k(k_kv8_append<T, WPT>, dim3((unsigned)std::min<int64_t>(pieces, r.total), (2 * heads + per - 1) / per),
                  kThreads, 0, st, r, x, kv, heads, d, 65536 / (d / 8) + 1);
}
template <typename T>
cudaError_t launch(const Ragged& r, const Rows8& x, const Kv8View& kv, int heads, int d, cudaStream_t st) {
  // Warps a task: as few as hold its rows, those of a full page or the average sequence's, in registers.  bf16, 8
  // heads of 128, 8 x 300 rows: pages of 16 with 1, 2, 4 warps 4.0, 5.4, 8.1 us, pages of 64 13.5, 7.6, 4.1 (8: 6.0).
  constexpr int HOLD = Eight<T>::HOLD;
  const int rows = std::min(1 << kv.page_shift, std::max(1, r.total / r.batch)), steps = (rows * d / 8 + 31) / 32;
  return steps <= HOLD       ? launch<T, 1>(r, x, kv, heads, d, st)
         : steps <= 2 * HOLD ? launch<T, 2>(r, x, kv, heads, d, st)
         : steps <= 4 * HOLD ? launch<T, 4>(r, x, kv, heads, d, st)
                             : launch<T, 8>(r, x, kv, heads, d, st);
}

}  // namespace
}  // namespace dfl

using namespace dfl;

extern "C" DFLASH_API int dflash_kv8_append(const dflash_kv8_pages* pages, const dflash_ragged* batch, int32_t dtype,
                                            const dflash_heads* k, const dflash_heads* v, void* stream) {
  const char* call = "dflash_kv8_append";
  if (int rc = check_kv8_pages(call, pages)) return rc;
  if (dtype != DFLASH_DTYPE_F32 && dtype != DFLASH_DTYPE_BF16) return rfail(DFLASH_ERR_INVALID_ARG, call, "dtype");
  const dflash_kv_pages like = kv8_as_pages(pages);
  if (int rc = check_ragged(call, batch, &like, true)) return rc;
  const bool rows = batch->total_rows > 0;
  if (int rc = check_heads(call, k, dtype, pages->n_kv_heads, pages->head_dim, rows)) return rc;
  if (int rc = check_heads(call, v, dtype, pages->n_kv_heads, pages->head_dim, rows)) return rc;
  if (!rows) return DFLASH_OK;
  const Ragged r = make_ragged(batch, &like);
  const Rows8 x{{k->data, v->data}, {k->row_stride, v->row_stride}, {k->head_stride, v->head_stride}};
  const Kv8View kv = kv8_view(pages);
  cudaStream_t st = (cudaStream_t)stream;
  return rcheck(dtype == DFLASH_DTYPE_F32 ? launch<float>(r, x, kv, pages->n_kv_heads, pages->head_dim, st)
                                          : launch<bf16>(r, x, kv, pages->n_kv_heads, pages->head_dim, st),
                call);
}
