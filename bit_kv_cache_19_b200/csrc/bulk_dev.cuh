// Pass 1 of the bulk tile quantizers (quantize_append_kernel and the ragged
// append): one warp quantizes one token whose input type is known at compile
// time, value thresholds in registers where they fit.
#pragma once

#include "quant_dev.cuh"

namespace kvq {

// Element i of a row of the input type DT (KVQ_BF16 / FP16 / FP32) as fp32.
template <int DT>
__device__ __forceinline__ float in_elem(const void* base, size_t i) {
  if constexpr (DT == KVQ_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(base)[i]);
  else if constexpr (DT == KVQ_FP16) return __half2float(static_cast<const __half*>(base)[i]);
  else return static_cast<const float*>(base)[i];
}

// Code of a width-W value from the thresholds held in registers (W <= 3):
// the same binary search as code_of_w, its steps resolved by selects.
template <int W>
__device__ __forceinline__ uint32_t code_of_reg(const float (&t)[7], float z) {
  if constexpr (W == 1) {
    return t[0] < z ? 1u : 0u;
  } else if constexpr (W == 2) {
    const uint32_t c = t[1] < z ? 2u : 0u;
    return c + ((c ? t[2] : t[0]) < z ? 1u : 0u);
  } else {
    const uint32_t c2 = t[3] < z ? 4u : 0u;
    const uint32_t c1 = (c2 ? t[5] : t[1]) < z ? 2u : 0u;
    const float tl = c2 ? (c1 ? t[6] : t[4]) : (c1 ? t[2] : t[0]);
    return c2 + c1 + (tl < z ? 1u : 0u);
  }
}

// Pass 1 of the bulk path for one token (one warp), input type DT known at
// compile time: the arithmetic and decisions of warp_token_pass (fixed
// sum-of-squares tree, IEEE norm and reciprocal, the same butterfly graph),
// with the lane's value signs precomputed (bit q: coordinate lane + 32 q)
// and, for value widths <= 3, the thresholds in registers.
template <int BV, int DT>
__device__ __forceinline__ void bulk_token_pass(const Plan& pl, const float* thr,
                                                const float (&tv)[7], uint32_t vsgn,
                                                const void* k, const void* v, size_t row,
                                                int lane, int p, float* kz_row, uint32_t* words,
                                                bool clear, __half& kn, __half& vn,
                                                uint32_t& flags) {
  float kx[4], vx[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    kx[q] = in_elem<DT>(k, row + lane + 32 * q);
    vx[q] = in_elem<DT>(v, row + lane + 32 * q);
  }
  const bool kfin = __all_sync(0xffffffffu, isfinite(kx[0]) && isfinite(kx[1]) &&
                                                isfinite(kx[2]) && isfinite(kx[3]));
  const bool vfin = __all_sync(0xffffffffu, isfinite(vx[0]) && isfinite(vx[1]) &&
                                                isfinite(vx[2]) && isfinite(vx[3]));
  float kr;
  norm_and_recip(kx, kfin, kn, kr, flags);
  const bool klive = kfin && __half2float(kn) > 0.f;
#pragma unroll
  for (int q = 0; q < 4; ++q)
    kz_row[lane + 32 * q] = klive ? __fmul_rn(kx[q], kr) : __int_as_float(0x7fc00000);
  float vr;
  norm_and_recip(vx, vfin, vn, vr, flags);
  const bool vlive = vfin && __half2float(vn) > 0.f;
  float y[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const float x = vfin ? vx[q] : 0.f;
    y[q] = ((vsgn >> q) & 1u) ? -x : x;
  }
#pragma unroll
  for (int hh = 1; hh < 32; hh <<= 1) {
    const float sg = (lane & hh) ? -1.f : 1.f;
#pragma unroll
    for (int q = 0; q < 4; ++q) y[q] = __fmaf_rn(y[q], sg, __shfl_xor_sync(0xffffffffu, y[q], hh));
  }
  {
    const float a0 = __fadd_rn(y[0], y[1]), a1 = __fsub_rn(y[0], y[1]);
    const float a2 = __fadd_rn(y[2], y[3]), a3 = __fsub_rn(y[2], y[3]);
    y[0] = __fadd_rn(a0, a2);
    y[2] = __fsub_rn(a0, a2);
    y[1] = __fadd_rn(a1, a3);
    y[3] = __fsub_rn(a1, a3);
  }
  uint32_t* vwords = words + kHeadDim * pl.bits_k + ((slot_v(p) * BV) >> 5) + BV * lane;
  const int off = (slot_v(p) * BV) & 31;
  const bool spill = off + BV > 32;
  constexpr uint32_t mask = (1u << BV) - 1u;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint32_t* w = vwords + BV * 32 * q;
    const float z = __fmul_rn(y[q], vr);  // 0 for a dead token (vr = 0)
    uint32_t c;
    if constexpr (BV <= 3) c = code_of_reg<BV>(tv, z);
    else c = (uint32_t)code_of_w<BV>(thr, z);
    c = vlive ? c : 0u;  // a select, not a branch, in the unrolled loop
    if (clear) atomicAnd(w, ~(mask << off));
    atomicOr(w, c << off);
    if (spill) {
      if (clear) atomicAnd(w + 1, ~(mask >> (32 - off)));
      atomicOr(w + 1, c >> (32 - off));
    }
  }
}

}  // namespace kvq
