// Block tables and slot maps from request lengths, on the GPU.
//
// No counterpart in the pages (they keep one cache per sequence); this is the
// device-side form of the page bookkeeping that kvq_pages describes, so that a
// serving step needs no host round trip (and can be captured in a graph).
// Mathematics: with span = 32 page_tiles tokens per page, sequence b needs
// need_b = ceil((len_b + n_new_b) / span) pages. Pages past need_b go to the tail
// of the ring of free ids (in sequence, then row order); then the missing
// need_b - held_b pages come from its head: the k-th page that sequence b takes
// is ring entry head + T_b + k, T the exclusive prefix sum of the takes. Token j
// of sequence b (token cu_b + j of the packed batch, cu the exclusive prefix sum
// of n_new) sits in slot page span + (len_b + j) mod span.
//
// What bounds it: a few integer operations per token and 12 bytes written (slot
// and position), so a batch of a decode step is one launch's latency, and a
// prefill chunk the store rate. Split: one CTA makes the three prefix sums (they
// are serial over the batch); a small step is finished by that CTA (one launch),
// a larger one by a grid over tokens and pages that resolves new pages from the
// ring itself, so that it waits for nothing but the sums. Measured: 5.2 us for 256
// one-token requests; 18 us, with a copy that resets the state, for 482499 tokens
// of 1000 requests.
#include <algorithm>

#include "pages.cuh"
#include "splitk.cuh"

namespace kvq {

constexpr int kScanThreads = 1024;
constexpr int kScanWarps = kScanThreads / 32;
constexpr int kSmallBatch = 768;  // sequences whose 48-byte records fit in static shared memory

struct Sum3 {  // tokens, returned pages, taken pages before a sequence
  long long tok, ret, take;
};
__device__ __forceinline__ Sum3 add3(const Sum3& a, const Sum3& b) {
  return {a.tok + b.tok, a.ret + b.ret, a.take + b.take};
}
__device__ __forceinline__ Sum3 shfl_up3(const Sum3& a, int d) {
  return {__shfl_up_sync(0xffffffffu, a.tok, d), __shfl_up_sync(0xffffffffu, a.ret, d),
          __shfl_up_sync(0xffffffffu, a.take, d)};
}

// Exclusive prefix over the CTA's threads; `total` gets the CTA's sum.
__device__ __forceinline__ Sum3 block_scan(Sum3 x, Sum3* warp_sum, Sum3& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Sum3 inc = x;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const Sum3 y = shfl_up3(inc, d);
    if (lane >= d) inc = add3(inc, y);
  }
  if (lane == 31) warp_sum[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    Sum3 w = warp_sum[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const Sum3 y = shfl_up3(w, d);
      if (lane >= d) w = add3(w, y);
    }
    warp_sum[lane] = w;
  }
  __syncthreads();
  total = warp_sum[kScanWarps - 1];
  const Sum3 before = warp ? warp_sum[warp - 1] : Sum3{0, 0, 0};
  return {before.tok + inc.tok - x.tok, before.ret + inc.ret - x.ret,
          before.take + inc.take - x.take};
}

// One sequence's request: its tokens, and the pages it takes or returns.
struct Request {
  long long n;  // tokens in the packed batch
  long long need;
  int held;
  int ret, take;
  bool ok;  // before the free pages are counted
};

__device__ __forceinline__ Request request_of(const PagesParams& p, int b, long long tok_before,
                                              bool have_tok, uint32_t& flags) {
  Request r;
  const int len = p.len[b], nn = p.n_new[b], held = p.held[b];
  r.n = max(nn, 0);
  r.held = held;
  r.need = ((long long)len + nn + p.span - 1) >> p.span_shift;
  const bool row = held >= 0 && held <= p.max_pages;
  const bool fits = len >= 0 && nn >= 0 && r.need <= p.max_pages;
  r.ok = row && fits && (!have_tok || tok_before + r.n <= p.n_slots);
  r.ret = r.ok && r.need < held ? held - (int)r.need : 0;
  r.take = r.ok && r.need > held ? (int)r.need - held : 0;
  if (have_tok) {
    if (!row) flags |= KVQ_FLAG_BAD_PAGE;
    else if (!r.ok) flags |= KVQ_FLAG_CAPACITY;
  }
  return r;
}

// Largest i in [0, n) with a[i] <= x (a ascending, a[0] <= x).
template <typename T, typename X>
__device__ __forceinline__ int last_le(const T* a, int n, X x) {
  int lo = 0;
  while (n > 1) {
    const int half = n >> 1;
    if ((X)a[lo + half] <= x) lo += half;
    n -= half;
  }
  return lo;
}

__device__ __forceinline__ long long ring_at(long long i, long long n) { return i >= n ? i - n : i; }

// Slot of token `tok` of the packed batch.
__device__ __forceinline__ void map_token(const PagesParams& p, const PagesMeta* meta,
                                          const int32_t* cu, int batch, long long head,
                                          long long tok) {
  const int b = last_le(cu, batch, (int)tok);
  const PagesMeta m = meta[b];
  const long long pos = (long long)m.len + (tok - m.cu);
  long long slot = -1;
  if (m.granted) {
    const int j = (int)(pos >> p.span_shift);
    const int page = j < m.held
                         ? p.table[(size_t)b * p.max_pages + j]
                         : p.free_ids[ring_at(head + m.take0 + (j - m.held), p.n_pages)];
    slot = ((long long)page << p.span_shift) + (pos & (p.span - 1));
  }
  p.slots[tok] = slot;
  if (p.pos) p.pos[tok] = (int32_t)pos;
}

// Table entry of the i-th page taken by this call.
__device__ __forceinline__ void fill_page(const PagesParams& p, const PagesMeta* meta, int batch,
                                          long long head, long long i) {
  int lo = 0, n = batch;
  while (n > 1) {
    const int half = n >> 1;
    if (meta[lo + half].take0 <= i) lo += half;
    n -= half;
  }
  const PagesMeta m = meta[lo];
  const int j = m.held + (int)(i - m.take0);
  if (m.granted && i - m.take0 < m.take)
    p.table[(size_t)lo * p.max_pages + j] = p.free_ids[ring_at(head + i, p.n_pages)];
}

// The prefix sums, the returned pages, the new ring and page counts; with SMALL
// also the table entries and the slots (one CTA). meta: per sequence, in shared
// memory when SMALL (batch <= kSmallBatch), else in the workspace.
template <bool SMALL>
__global__ void __launch_bounds__(kScanThreads) pages_scan_kernel(PagesParams p) {
  __shared__ Sum3 warp_sum[kScanWarps];
  __shared__ PagesMeta s_meta[SMALL ? kSmallBatch : 1];
  __shared__ int32_t s_cu[SMALL ? kSmallBatch : 1];
  __shared__ long long s_taken;
  __shared__ uint32_t s_flags;
  const int tid = threadIdx.x;
  if (!SMALL) grid_dep_launch();  // the map kernel's CTAs start, and wait for this one's end
  PagesMeta* const meta = SMALL ? s_meta : p.meta;
  if (tid == 0) {
    s_taken = 0;
    s_flags = 0;
  }
  const long long head = p.ring[0], count = p.ring[1];
  const bool ring_ok = head >= 0 && head < p.n_pages && count >= 0 && count <= p.n_pages;
  // consecutive sequences per thread, so that one scan covers any batch
  const int per = (p.batch + kScanThreads - 1) / kScanThreads;
  const int b0 = min(p.batch, tid * per), b1 = min(p.batch, b0 + per);
  uint32_t flags = 0;
  // a sequence whose tokens end past the slot array is refused, which changes
  // the page sums, so the token sum comes first
  Sum3 mine{0, 0, 0}, total;
  for (int b = b0; b < b1; ++b) mine.tok += max(p.n_new[b], 0);
  const long long tok0 = block_scan(mine, warp_sum, total).tok;
  const long long n_tok = total.tok;
  __syncthreads();
  long long t = tok0;
  mine = {0, 0, 0};
  for (int b = b0; b < b1; ++b) {
    const Request r = request_of(p, b, t, true, flags);
    t += r.n;
    mine.ret += r.ret;
    mine.take += r.take;
  }
  const Sum3 before = block_scan(mine, warp_sum, total);
  const long long n_ret = total.ret;
  // a ring or a row that cannot be what earlier calls left: nothing moves
  const bool sane = ring_ok && count + n_ret <= p.n_pages;
  if (!sane) flags |= KVQ_FLAG_BAD_PAGE;
  const long long avail = count + n_ret;
  long long ret0 = before.ret, take0 = before.take, taken = 0;
  t = tok0;
  for (int b = b0; b < b1; ++b) {
    uint32_t ignored = 0;
    const Request r = request_of(p, b, t, true, ignored);
    // the pages go in sequence order: once one sequence's do not fit, no later
    // sequence gets any either
    const bool granted = r.ok && sane && (r.take == 0 || take0 + r.take <= avail);
    if (r.ok && sane && !granted) flags |= KVQ_FLAG_CAPACITY;
    PagesMeta m;
    m.cu = t;
    m.take0 = take0;
    m.ret0 = ret0;
    m.held = r.held;
    m.len = p.len[b];
    m.take = granted ? r.take : 0;
    m.ret = granted ? r.ret : 0;
    m.granted = granted;
    meta[b] = m;
    const int32_t c = (int32_t)min(t, (long long)0x7FFFFFFF);
    p.cu[b] = c;
    if (SMALL) s_cu[b] = c;
    if (granted) {
      p.held[b] = (int32_t)r.need;
      if (r.take) taken = take0 + r.take;
    }
    t += r.n;
    ret0 += r.ret;
    take0 += r.take;
  }
  if (taken) atomicMax(&s_taken, taken);
  if (flags) atomicOr(&s_flags, flags);
  __syncthreads();
  const long long n_taken = s_taken;
  if (tid == 0) {
    const int32_t c = (int32_t)min(n_tok, (long long)0x7FFFFFFF);
    p.cu[p.batch] = c;
    if (sane) {
      p.ring[0] = (head + n_taken) % p.n_pages;
      p.ring[1] = avail - n_taken;
    }
    if (!SMALL) {
      p.head->head = head;
      p.head->n_tok = min(n_tok, (long long)p.n_slots);
      p.head->n_taken = n_taken;
    }
    if (s_flags) atomicOr(p.status, s_flags);
  }
  // returned pages, in sequence then row order, behind the free ones: a warp takes
  // the sequences of its lanes one after the other, 32 pages at a time (a search
  // for each page's sequence took 5 us of a 1000-request step)
  const int lane = tid & 31;
  for (int k = 0; k < per && sane && n_ret; ++k) {
    const int b = b0 + k;
    const bool mine_k = b < b1;
    const int back = mine_k ? meta[b].ret : 0;
    const int from = mine_k ? meta[b].held - back : 0;
    const long long to = mine_k ? head + count + meta[b].ret0 : 0;
    for (uint32_t any = __ballot_sync(0xffffffffu, back > 0); any; any &= any - 1) {
      const int src = __ffs(any) - 1;
      const int sb = __shfl_sync(0xffffffffu, b, src), n = __shfl_sync(0xffffffffu, back, src);
      const int f = __shfl_sync(0xffffffffu, from, src);
      const long long t0 = __shfl_sync(0xffffffffu, to, src);
      int32_t* const row = p.table + (size_t)sb * p.max_pages + f;
      for (int i = lane; i < n; i += 32) {
        p.free_ids[(t0 + i) % p.n_pages] = row[i];
        row[i] = -1;
      }
    }
  }
  if constexpr (SMALL) {
    __syncthreads();
    for (long long i = tid; i < n_taken; i += kScanThreads)
      fill_page(p, meta, p.batch, head, i);
    const long long n = min(n_tok, (long long)p.n_slots);
    for (long long i = tid; i < n; i += kScanThreads) map_token(p, meta, s_cu, p.batch, head, i);
  }
}

__global__ void __launch_bounds__(256) pages_map_kernel(PagesParams p) {
  grid_dep_wait();
  const long long head = p.head->head, n_tok = p.head->n_tok, n_taken = p.head->n_taken;
  const long long step = (long long)gridDim.x * blockDim.x;
  const long long first = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  for (long long i = first; i < n_tok; i += step) map_token(p, p.meta, p.cu, p.batch, head, i);
  for (long long i = first; i < n_taken; i += step) fill_page(p, p.meta, p.batch, head, i);
}

size_t pages_workspace_bytes(int batch) { return 256 + (size_t)batch * sizeof(PagesMeta); }

// One launch while the scan's CTA can also write the slots in about the time a
// second launch takes to start. One launch / two, us on the GPU: 256 requests of a
// token 5.2 / 7.8; 2160 slots of 9 requests 5.9 / 6.8; 4096 of 64 8.8 / 9.3; 6300 of 9
// 8.0 / 6.4; 16384 of 64 17.5 / 9.9.
constexpr int64_t kOneLaunchSlots = 4096;

cudaError_t launch_pages_assign(PagesParams p, void* ws, cudaStream_t st) {
  p.head = reinterpret_cast<PagesHead*>(ws);
  p.meta = reinterpret_cast<PagesMeta*>(reinterpret_cast<uint8_t*>(ws) + 256);
  if (p.batch <= kSmallBatch && p.n_slots <= kOneLaunchSlots) {
    pages_scan_kernel<true><<<1, kScanThreads, 0, st>>>(p);
    return cudaGetLastError();
  }
  pages_scan_kernel<false><<<1, kScanThreads, 0, st>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int64_t pages = p.n_slots / p.span + p.batch;
  const int64_t ctas = (std::max<int64_t>(p.n_slots, pages) + 255) / 256;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)std::min<int64_t>(std::max<int64_t>(ctas, 1), 148 * 8));
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, pages_map_kernel, p);
}

}  // namespace kvq
