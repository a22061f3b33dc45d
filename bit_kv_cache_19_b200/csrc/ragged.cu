// Quantize-append of a packed ragged batch into paged caches: the new tokens
// of all sequences in one [tokens][n_kv][128] array, each going to its slot of
// the pool (kvq_pages_assign's slot map).
//
// The codes are those of kvq_quantize_append ("RoPE-Aware Bit Allocation for
// KV-Cache Quantization", abstract: Block-GTQ keys on TQ-MSE, uniform TQ-MSE
// values), token by token. What differs is how the work is found: an item is
// one (32-token tile, KV head) that new tokens fall into. A sequence of n tokens
// touches at most n / 32 + 2 tiles, so item numbers start at cu[b] / 32 + 2 b for
// sequence b, a bound that follows from cu alone: a CTA finds its sequence by
// bisection, without a prefix sum over lengths.
//
// What bounds it: instruction issue (69 % of slots; 17400 warp instructions per
// tile and KV head: norms, divisions and roots per token, shared atomics to pack),
// like the bulk quantizer. Measured: 52892 tokens of 24 sequences, 8 KV heads, K2V2,
// bf16: 300 us for 246 MB, 820 GB/s; one token for each of 16 sequences 10 us (the
// latency of one tile, with a copy that resets the lengths).
#include <algorithm>

#include "bulk_dev.cuh"
#include "ragged.cuh"
#include "splitk.cuh"

namespace kvq {

__constant__ float c_rthr[KVQ_CB_N_THR] = KVQ_CB_THR;

// The tokens of one item: rows [row, row + n) into positions [p_lo, p_lo + n)
// of the tile record at rec.
struct RaggedItem {
  int b, p_lo, n;
  int64_t row;
  int64_t pos;  // cache position of the first token (pre-RoPE keys only)
  uint8_t* rec;  // the tile's records (head 0); null: nothing to do
  bool clear;    // the tile already holds tokens
  uint32_t flags;
};

__device__ __forceinline__ int64_t ragged_item0(const int32_t* cu, int b) {
  return ((int64_t)max(cu[b], 0) >> 5) + 2 * (int64_t)b;
}

// Where a sequence's tiles begin follows from its first slot; its length is read
// only for the positions of pre-RoPE keys, which leaves one CTA free to advance
// it in the same launch otherwise (`advance`: the CTA of the item's KV head 0).
__device__ __forceinline__ RaggedItem ragged_item(const RaggedParams& p, int64_t item,
                                                  bool advance) {
  RaggedItem it;
  it.rec = nullptr;
  it.flags = 0;
  int lo = 0, n = p.batch;
  while (n > 1) {
    const int half = n >> 1;
    if (ragged_item0(p.cu, lo + half) <= item) lo += half;
    n -= half;
  }
  it.b = lo;
  const int64_t i = item - ragged_item0(p.cu, lo);
  const int64_t c0 = p.cu[lo], c1 = p.cu[lo + 1];
  if (c1 <= c0 || i < 0) return it;
  if (c0 < 0 || c1 > p.n_rows) {
    if (i == 0) it.flags = KVQ_FLAG_CAPACITY;
    return it;
  }
  const int64_t first = p.slots[c0];
  if (first == -1) return it;  // refused by the assignment
  const int p0 = (int)(first & (kTile - 1));
  const int64_t t_lo = i == 0 ? 0 : i * kTile - p0;  // the item's first token
  if (t_lo >= c1 - c0) return it;
  it.p_lo = i == 0 ? p0 : 0;
  it.n = (int)min((int64_t)(kTile - it.p_lo), c1 - c0 - t_lo);
  it.row = c0 + t_lo;
  it.clear = it.p_lo > 0;
  it.pos = 0;
  if (p.rope) {
    const int64_t len = p.len[lo];
    it.pos = len + t_lo;
    if (len < 0 || len + (c1 - c0) > 0x7FFFFFFF || (len & (kTile - 1)) != p0) {
      if (i == 0) it.flags = (len & (kTile - 1)) != p0 ? KVQ_FLAG_BAD_PAGE : KVQ_FLAG_CAPACITY;
      return it;
    }
  } else if (advance && i == 0 && threadIdx.x == 0) {
    const int64_t len = p.len[lo], to = len + (c1 - c0);  // read by this thread alone
    if ((len & (kTile - 1)) != p0) atomicOr(p.status, KVQ_FLAG_BAD_PAGE);
    else if (len < 0 || to > 0x7FFFFFFF) atomicOr(p.status, KVQ_FLAG_CAPACITY);
    else p.len[lo] = (int32_t)to;
  }
  const int64_t slot = p.slots[it.row];
  if (slot == -1) return it;
  const int64_t page = slot >> p.span_shift;
  const int in_page = (int)(slot & (p.span - 1)), lane = threadIdx.x & 31;
  // every warp looks at all of the tile's slots, a lane at one
  const bool run =
      __all_sync(0xffffffffu, lane >= it.n || p.slots[it.row + lane] == slot + lane);
  if (slot < 0 || page >= p.n_pages || (in_page & (kTile - 1)) != it.p_lo || !run) {
    it.flags = KVQ_FLAG_BAD_PAGE;
    return it;
  }
  it.rec = p.pool + page * p.page_bytes + (size_t)(in_page / kTile) * p.n_kv * p.tile_bytes;
  return it;
}

template <int BV, int DT>
__global__ void __launch_bounds__(256, 4) append_ragged_kernel(RaggedParams p) {
  __shared__ Plan s_plan;
  __shared__ float s_thr[KVQ_CB_N_THR];
  __shared__ float s_kz[kTile * kKzStride];
  __shared__ uint32_t s_words[kHeadDim * 16 + 1];  // + slack word for put_field
  __shared__ uint32_t s_flags;
  __shared__ double s_theta[64];
  __shared__ RotTables s_rot;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  for (int i = threadIdx.x; i < KVQ_CB_N_THR; i += blockDim.x) s_thr[i] = c_rthr[i];
  for (int i = threadIdx.x; i < 64; i += blockDim.x) s_theta[i] = p.theta[i];
  if (threadIdx.x == 0) s_flags = 0;
  float tv[7];  // value thresholds in registers (widths <= 3)
#pragma unroll
  for (int i = 0; i < 7; ++i) tv[i] = c_rthr[cb_t_off(BV) + min(i, (1 << BV) - 2)];
  uint32_t vsgn = 0;  // value signs of this lane's coordinates lane + 32 q
  const Plan* cur = nullptr;  // the plan in shared memory
  bool plan_ok = false;
  const int64_t n_items = ((int64_t)max(min((int64_t)p.cu[p.batch], p.n_rows), (int64_t)0) >> 5) +
                          2 * (int64_t)p.batch;
  for (int64_t item = blockIdx.x; item < n_items * p.n_kv; item += gridDim.x) {
    const int h = (int)(item % p.n_kv);
    const RaggedItem it = ragged_item(p, item / p.n_kv, DT >= 0 && h == 0);
    if (!it.rec) {
      if (it.flags && threadIdx.x == 0) atomicOr(p.status, it.flags);
      continue;
    }
    uint8_t* const rec = it.rec + (size_t)h * p.tile_bytes;
    __syncthreads();  // the previous item is done with the shared buffers
    if (p.plans[it.b] + h != cur) {
      cur = p.plans[it.b] + h;
      const uint32_t* src = reinterpret_cast<const uint32_t*>(cur);
      uint32_t* dst = reinterpret_cast<uint32_t*>(&s_plan);
      for (int i = threadIdx.x; i < KVQ_PLAN_BYTES / 4; i += blockDim.x) dst[i] = src[i];
      __syncthreads();
      plan_ok = s_plan.magic == KVQ_PLAN_MAGIC && s_plan.bits_k >= 1 && s_plan.bits_k <= 8 &&
                s_plan.bits_v == BV && p.tile_bytes == tile_bytes(s_plan.bits_k, BV) &&
                plan_sched_ok(s_plan, lane);
      if (plan_ok && s_plan.k_rot) rot_tables(s_plan, s_rot, threadIdx.x);
      vsgn = 0;
#pragma unroll
      for (int q = 0; q < 4; ++q) vsgn |= ((s_plan.v_sign[q] >> lane) & 1u) << q;
      __syncthreads();
    }
    if (!plan_ok) {
      if (threadIdx.x == 0) atomicOr(p.status, KVQ_FLAG_BAD_PLAN);
      continue;
    }
    const Plan& pl = s_plan;
    const int n_words = kHeadDim * (pl.bits_k + BV);
    uint32_t* gw = reinterpret_cast<uint32_t*>(rec);
    for (int i = threadIdx.x; i < n_words; i += blockDim.x) s_words[i] = it.clear ? gw[i] : 0u;
    __syncthreads();

    // ---- pass 1: one warp per new token
    const int p_hi = it.p_lo + it.n;
    uint32_t flags = 0;
    __half* norms = reinterpret_cast<__half*>(rec + 512 * (pl.bits_k + BV));
    for (int pp = it.p_lo + warp; pp < p_hi; pp += nw) {
      __half kn, vn;
      const size_t row = ((size_t)(it.row + (pp - it.p_lo)) * p.n_kv + h) * kHeadDim;
      if constexpr (DT >= 0)
        bulk_token_pass<BV, DT>(pl, s_thr, tv, vsgn, p.k, p.v, row, lane, pp,
                                s_kz + pp * kKzStride, s_words, it.clear, kn, vn, flags);
      else
        warp_token_pass<BV>(pl, s_thr, p.k, p.v, p.dtype, row, lane, pp, s_kz + pp * kKzStride,
                            s_words, it.clear, kn, vn, flags, p.rope ? s_theta : nullptr,
                            it.pos + (pp - it.p_lo));
      if (lane == 0) {
        norms[pp] = kn;
        norms[kTile + pp] = vn;
      }
    }
    if (flags) atomicOr(&s_flags, flags);
    __syncthreads();
    if (pl.k_rot) {  // ---- key rotation inside width groups, one warp per new token
      for (int pp = it.p_lo + warp; pp < p_hi; pp += nw)
        warp_rotate_row(s_kz + pp * kKzStride, pl, s_rot, pl.g, lane);
      __syncthreads();
    }
    // ---- pass 2: one warp per stored key block
    for (int r = warp; r < pl.n_ranks; r += nw)
      warp_block_pass(pl, s_thr, r, s_kz, it.p_lo, p_hi, lane, s_words, it.clear);
    __syncthreads();
    for (int i = threadIdx.x; i < n_words; i += blockDim.x) gw[i] = s_words[i];
  }
  __syncthreads();
  if (threadIdx.x == 0 && s_flags) atomicOr(p.status, s_flags);
}

// len += the sequence's tokens, unless the assignment refused them (pre-RoPE
// keys: every CTA of the append reads the lengths).
__global__ void ragged_len_kernel(RaggedParams p) {
  grid_dep_wait();
  const int b = blockIdx.x * blockDim.x + threadIdx.x;
  if (b >= p.batch) return;
  const int64_t c0 = p.cu[b], c1 = p.cu[b + 1], len = p.len[b];
  if (c1 <= c0 || c0 < 0 || c1 > p.n_rows || len < 0 || len + (c1 - c0) > 0x7FFFFFFF) return;
  if (p.slots[c0] != -1 && ((p.slots[c0] ^ len) & (kTile - 1)) == 0) p.len[b] = (int32_t)(len + (c1 - c0));
}

template <int BV>
static void launch_ragged_t(const RaggedParams& p, unsigned grid, cudaStream_t st) {
  if (p.rope) append_ragged_kernel<BV, -1><<<grid, 256, 0, st>>>(p);
  else if (p.dtype == KVQ_BF16) append_ragged_kernel<BV, KVQ_BF16><<<grid, 256, 0, st>>>(p);
  else if (p.dtype == KVQ_FP16) append_ragged_kernel<BV, KVQ_FP16><<<grid, 256, 0, st>>>(p);
  else append_ragged_kernel<BV, KVQ_FP32><<<grid, 256, 0, st>>>(p);
}

cudaError_t launch_append_ragged(const RaggedParams& p, int bits_v, cudaStream_t st) {
  int dev = 0, sms = 148;
  if (cudaGetDevice(&dev) == cudaSuccess)
    (void)cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  (void)cudaGetLastError();
  const int64_t items = (p.n_rows / kTile + 2 * (int64_t)p.batch) * p.n_kv;
  // resident CTAs; a multiple of n_kv, so that a CTA keeps its KV head and plan
  const int64_t most = std::max<int64_t>((int64_t)4 * sms / p.n_kv, 1) * p.n_kv;
  const unsigned grid = (unsigned)std::min<int64_t>(items, most);
  switch (bits_v) {
    case 1: launch_ragged_t<1>(p, grid, st); break;
    case 2: launch_ragged_t<2>(p, grid, st); break;
    case 3: launch_ragged_t<3>(p, grid, st); break;
    case 4: launch_ragged_t<4>(p, grid, st); break;
    case 5: launch_ragged_t<5>(p, grid, st); break;
    case 6: launch_ragged_t<6>(p, grid, st); break;
    case 7: launch_ragged_t<7>(p, grid, st); break;
    case 8: launch_ragged_t<8>(p, grid, st); break;
    default: return cudaErrorInvalidValue;
  }
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !p.rope) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((p.batch + 255) / 256));
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, ragged_len_kernel, p);
}

}  // namespace kvq
