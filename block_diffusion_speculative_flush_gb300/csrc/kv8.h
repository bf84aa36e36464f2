// Internal interface of the 8-bit paged cache: its view for kernels, and the
// conversions of e4m3 codes.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "ragged.h"

namespace dfl {

// The cache of one layer: code of page p, slot s, head h, element c at
// p * page + s * slot + h * head + c; its scale at p * s_page + h * s_head.
struct Kv8View {
  uint8_t* k;
  uint8_t* v;
  float* ks;
  float* vs;
  int64_t page, slot, head, s_page, s_head;
  int32_t page_shift, n_pages;
};

// Four codes (the lowest byte first) as fp16, two and two: exact, NaN stays NaN.
__device__ __forceinline__ void e4m3x4_to_h4(uint32_t c, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(c));
}
__device__ __forceinline__ float4 e4m3x4_to_f4(uint32_t c) {
  uint32_t lo, hi;
  e4m3x4_to_h4(c, lo, hi);
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo)), b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  return make_float4(a.x, a.y, b.x, b.y);
}
// Nearest codes, ties to even, beyond 448: 448; NaN: 0x7f.  a is the lower byte.
__device__ __forceinline__ uint16_t f2_to_e4m3x2(float a, float b) {
  uint16_t c;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(b), "f"(a));
  return c;
}
// Bit 7 of each byte that is a NaN, and the word with those bytes 0.
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }
__device__ __forceinline__ uint32_t without_nan(uint32_t w) { return w & ~((nan_codes(w) >> 7) * 0xffu); }
// log2 of a scale as the kernels add it to exponents; that of a page that is missing (its codes are zeros): the smallest.
constexpr float kNoScaleLog2 = -60.f;
__device__ __forceinline__ float scale_log2(float s) { return s > 0.f ? log2f(s) : kNoScaleLog2; }
// whether x is not finite (from its bits: fast-math flags do not change that)
__device__ __forceinline__ bool nonfinite(float x) { return (__float_as_uint(x) & 0x7f800000u) == 0x7f800000u; }

// The CUDA-core path (any rows, fp32 and bf16, head_dim a multiple of 16).
int64_t kv8_simt_workspace(const Ragged& r, const AttnCall& a, int sms);
cudaError_t launch_kv8_simt(const Ragged& r, const AttnCall& a, const Kv8View& kv, bool is_bf16, int sms, cudaStream_t st);

// Few rows on the tensor cores (bf16, head_dim 64 or 128).
bool kv8_few(const Ragged& r, const AttnCall& a, int sms);
int64_t kv8_few_workspace(const Ragged& r, const AttnCall& a, int sms);
cudaError_t launch_kv8_few(const Ragged& r, const AttnCall& a, const Kv8View& kv, int sms, cudaStream_t st);

// Many rows on the tensor cores (bf16, head_dim 64 or 128): attn_tc_workspace with kv8.
cudaError_t launch_attn_tc8(const Ragged& r, const AttnCall& a, const Kv8View& kv, cudaStream_t st);

}  // namespace dfl
