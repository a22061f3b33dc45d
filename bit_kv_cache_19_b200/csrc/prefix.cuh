// Arguments of the shared-prefix decode (host and device side).
#pragma once

#include "common.cuh"

namespace kvq {

constexpr int kPfxMaxGroups = 1024;

struct PrefixArgs {
  const Plan* const* plans;  // [batch] -> [n_kv]
  CacheMap pre;              // one row per prefix
  const int32_t* pre_len;    // [n_groups]
  const int32_t* group_start;  // [n_groups + 1]
  int n_groups;
  int64_t max_pre;
  CacheMap own;              // one row per sequence
  const int32_t* len;        // [batch]
  int64_t max_len;
  int batch, n_q, n_kv, bits_k, bits_v;
  const void* q;
  int q_dtype;
  void* out;
  int out_dtype;
  uint32_t* status;
};

size_t prefix_workspace_bytes(int batch, int n_q, int n_kv, int n_groups);
void set_prefix_stall(long long cycles);  // kvq_debug_decode_stall
cudaError_t launch_prefix_decode(const PrefixArgs& a, void* ws, size_t ws_bytes, cudaStream_t st);

}  // namespace kvq
