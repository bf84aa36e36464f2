// Internal interface of the target-side operators: ragged batches of new rows
// over paged or packed K/V.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "dflash.h"

namespace dfl {

// The ragged batch as kernels see it.  max_len is already capped by the table.
struct Ragged {
  int32_t batch, total, max_rows, max_len;
  const int32_t* starts;
  const int32_t* lens;   // NULL: packed prompts, a sequence's length is its row count
  const int32_t* table;
  int32_t table_stride;
  int32_t* status;
};

struct Seq {
  int32_t start, n, len;  // first packed row, new rows, length with them
  bool ok;                // within the batch's bounds; otherwise the sequence is skipped
};

// K/V of one layer: pages (slots of a page slot-stride apart), or packed rows
// (paged == 0: slot stride = row stride, position p of a sequence at its start + p).
struct KVView {
  const void* k;
  const void* v;
  int64_t k_slot, k_head, v_slot, v_head, page;  // strides in elements
  int32_t page_shift, n_pages, paged;
  int32_t packed_rows;  // rows of the packed arrays
};

struct AttnCall {
  int32_t Hq, Hkv, d, causal, window;
  float scale;
  const void* q;
  int64_t q_row, q_head;
  void* out;
  int64_t o_row, o_head;
  float* lse;
  float* ws;
};

__device__ __forceinline__ Seq load_seq(const Ragged& r, int b) {
  Seq s;
  s.start = r.starts[b];
  const int32_t end = r.starts[b + 1];
  s.len = r.lens ? r.lens[b] : end - s.start;
  s.ok = s.start >= 0 && end >= s.start && end <= r.total;
  s.n = s.ok ? end - s.start : 0;
  s.ok = s.ok && s.n <= r.max_rows && s.len >= s.n && s.len <= r.max_len;
  return s;
}
__device__ __forceinline__ void flag_status(int32_t* status, int bits) {
  if (status) atomicOr(status, bits);
}
// The sequence that owns packed row `row` (r.batch: behind the last one),
// found by the whole warp: the count of starts at or below the row.
__device__ __forceinline__ int seq_of_row(const Ragged& r, int row) {
  int c = 0;
  for (int j = 1 + (int)(threadIdx.x & 31); j <= r.batch; j += 32) c += r.starts[j] <= row;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
  return c;
}
// Keys [lo, hi) that a query at position p of a sequence of length len sees.
__device__ __forceinline__ int vis_lo(int p, int window) { return window && p >= window ? p - window + 1 : 0; }
__device__ __forceinline__ int vis_hi(int p, int len, int causal) { return causal ? p + 1 : len; }

// The CUDA-core path (fp32): bytes of workspace, and the launches.
int64_t attn_simt_workspace(const Ragged& r, const AttnCall& a);
cudaError_t launch_attn_simt(const Ragged& r, const AttnCall& a, const KVView& kv, cudaStream_t st);

// The tensor-core path (bf16, head_dim 64 or 128).
cudaError_t attn_tc_workspace(const Ragged& r, const AttnCall& a, int64_t* bytes, bool kv8 = false);
cudaError_t launch_attn_tc(const Ragged& r, const AttnCall& a, const KVView& kv, cudaStream_t st);

}  // namespace dfl
