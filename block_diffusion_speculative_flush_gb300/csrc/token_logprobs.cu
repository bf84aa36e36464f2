// Log probabilities of given tokens with the distribution's entropy and its
// top entries.  With z = l / T, m = max z, s = sum e^(z - m) and
// t = sum e^(z - m) (z - m):
//   logp(v) = z_v - m - log s,   H = log s - t / s.
#include <cuda_bf16.h>

#include <cmath>

#include "common.cuh"
#include "dflash.h"
#include "launch.h"

extern "C" int dflash__set_error(int code, const char* msg);

namespace dfl {
namespace {

__device__ __forceinline__ uint64_t warp_max64(uint64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const uint64_t u = __shfl_xor_sync(0xffffffffu, v, o);
    v = u > v ? u : v;
  }
  return v;
}

// One CTA per row: a pass for the maximum, a pass for the sums, and a pass
// per top entry for the largest key below the last one.
template <typename T>
__global__ void __launch_bounds__(512) k_token_logprobs(dflash_logprobs a) {
  pdl_trigger();
  pdl_wait();
  __shared__ float red[16];
  __shared__ uint64_t red64[16];
  const int r = blockIdx.x, tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const T* x = reinterpret_cast<const T*>(a.logits) + (int64_t)r * a.row_stride;
  const float it = 1.f / a.temperature;
  float m = -INFINITY;
  for (int v = tid; v < a.vocab; v += 512) m = fmaxf(m, to_f<T>(x[v]) * it);
  m = warp_max(m);
  if (lane == 0) red[w] = m;
  __syncthreads();
  m = red[0];
  for (int i = 1; i < 16; ++i) m = fmaxf(m, red[i]);
  __syncthreads();
  float s = 0.f, t = 0.f;
  for (int v = tid; v < a.vocab; v += 512) {
    const float d = to_f<T>(x[v]) * it - m, e = expf(d);
    s += e;
    if (e != 0.f) t = fmaf(e, d, t);
  }
  s = block_sum(s, red);
  t = block_sum(t, red);
  const float ls = logf(s);
  if (tid == 0) {
    const int tok = a.tokens[r];
    float lp = 0.f;
    if (tok >= 0 && tok < a.vocab) {
      lp = to_f<T>(x[tok]) * it - m - ls;
    } else if (tok != -1) {
      lp = __int_as_float(0x7fffffff);
      if (a.status) atomicOr(a.status, DFLASH_STATUS_TOKEN);
    }
    a.logprobs[r] = lp;
    if (a.entropy) a.entropy[r] = ls - t / s;
  }
  uint64_t last = ~0ull;
  for (int k = 0; k < a.top; ++k) {
    uint64_t best = 0;
    for (int v = tid; v < a.vocab; v += 512) {
      const uint64_t key = order_key(to_f<T>(x[v]), v);
      if (key < last && key > best) best = key;
    }
    best = warp_max64(best);
    __syncthreads();
    if (lane == 0) red64[w] = best;
    __syncthreads();
    for (int i = 0; i < 16; ++i) best = red64[i] > best ? red64[i] : best;
    last = best;
    if (tid == 0) {
      const int64_t o = (int64_t)r * a.top + k;
      a.top_ids[o] = best ? (int32_t)(0xffffffffu - (uint32_t)best) : -1;
      a.top_logprobs[o] = best ? float_of_order((uint32_t)(best >> 32)) * it - m - ls : __int_as_float(0x7fffffff);
    }
  }
}

}  // namespace
}  // namespace dfl

using namespace dfl;

extern "C" DFLASH_API int dflash_token_logprobs(const dflash_logprobs* a, void* stream) {
  auto bad = [](const char* m) { return dflash__set_error(DFLASH_ERR_INVALID_ARG, m); };
  if (!a) return bad("dflash_token_logprobs: null argument");
  if (a->dtype != DFLASH_DTYPE_F32 && a->dtype != DFLASH_DTYPE_BF16) return bad("dflash_token_logprobs: dtype");
  if (a->rows < 0 || a->vocab < 1 || a->vocab > (1 << 24) || a->row_stride < a->vocab)
    return bad("dflash_token_logprobs: rows < 0, vocab outside 1..2^24 or row_stride below it");
  if (a->top < 0 || a->top > DFLASH_LOGPROBS_MAX_TOP || a->top > a->vocab)
    return bad("dflash_token_logprobs: top outside 0..32 or above vocab");
  if (!(a->temperature > 0.f) || !std::isfinite(a->temperature))
    return bad("dflash_token_logprobs: temperature: finite, > 0");
  if (a->rows == 0) return DFLASH_OK;
  if (!a->logits || !a->tokens || !a->logprobs || (a->top && (!a->top_ids || !a->top_logprobs)))
    return bad("dflash_token_logprobs: null pointer");
  if ((uintptr_t)a->logits % (a->dtype == DFLASH_DTYPE_F32 ? 4 : 2))
    return bad("dflash_token_logprobs: logits not aligned to their type");
  cudaError_t e = a->dtype == DFLASH_DTYPE_F32
                      ? launch_k(k_token_logprobs<float>, a->rows, 512, 0, (cudaStream_t)stream, *a)
                      : launch_k(k_token_logprobs<bf16>, a->rows, 512, 0, (cudaStream_t)stream, *a);
  if (e != cudaSuccess) return dflash__set_error(DFLASH_ERR_CUDA, cudaGetErrorString(e));
  return DFLASH_OK;
}
