// Arguments of the ragged quantize-append launch (host and device side).
#pragma once

#include "common.cuh"

namespace kvq {

struct RaggedParams {
  const Plan* const* plans;  // [batch] -> [n_kv] plans
  const void* k;             // [n_rows][n_kv][128]
  const void* v;
  int dtype;
  const int32_t* cu;      // [batch + 1] first row of each sequence
  const int64_t* slots;   // [n_rows]
  int batch, n_kv;
  int64_t n_rows;
  uint8_t* pool;
  int64_t n_pages;
  int64_t page_bytes;
  int span, span_shift;   // tokens per page
  int32_t* len;
  int tile_bytes;
  uint32_t* status;
  int rope;           // keys are pre-RoPE: rotate each to its position first
  double theta[64];
};

cudaError_t launch_append_ragged(const RaggedParams& p, int bits_v, cudaStream_t st);

}  // namespace kvq
