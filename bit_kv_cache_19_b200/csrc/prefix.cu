// Decode attention for a batch whose sequences share long prefixes.
//
// Mathematics. Sequence b of prefix group g attends over the group's prefix
// tokens and its own: o = sum_t p_t v^_t, p = softmax of q . k^_t / sqrt(128)
// over both. Softmax over a union is the log-sum-exp-weighted mix of the parts'
// results, so each part gives records (m, l, o) with l = sum 2^(s - m) and
// o = sum 2^(s - m) v^ (base-2 logits s), and a merge adds them. The prefix's
// part is one product for all R = (sequences of the group) x G query rows of a
// KV head: S = Q K^T and O = P V with R rows instead of G, so its codes are
// unpacked once per 256 rows, not once per sequence. ("RoPE-Aware Bit
// Allocation for KV-Cache Quantization", abstract: decode attention directly on
// the packed cache; the pages have no batch and no sharing.)
//
// Operands are exact where the format is: K = the fp16 centroids of the codes,
// in plan order (position 2 r + e holds coordinate order[r] + 64 e), Q = q a^
// log2(e) / sqrt(128) scaled by a power of two per row; the token's key norm
// multiplies the fp32 logit. V = the centroids of the rotated values, P =
// 2^(s - m) times the value norm, in fp16. The inverse rotation comes after
// the merge. Rounding: for bf16 outputs Q and P are rounded to fp16 once (2^-11
// relative at most each, well under the output's 2^-9); for fp16 and fp32
// outputs both are split into two fp16 terms (hi + lo), two products each.
//
// Three launches (programmatic dependent launch between them):
//  1. prep: query rows into fp16 operand images (swizzled), the work schedule;
//  2. main: persistent, one CTA per SM. Units of work are (prefix, KV head, 256
//     query rows) and (sequence, KV head); the units' 128-token tiles form one
//     line of cost, cut evenly over the CTAs (a CTA takes a piece of one long
//     unit or many short ones), so ragged lengths need no tuning. Warp roles:
//     one warp streams 32-token records (bulk copies), six unpack codes into
//     fp16 tiles in shared memory, one thread issues tcgen05.mma, two warpgroups
//     run the softmax of two independent streams. A unit of more than 128 rows
//     puts one 128-row tile in each stream (both use every K/V tile); a smaller
//     one gives the streams alternate tiles. TMEM: S of both streams (P
//     overwrites it) and O of both, 512 columns.
//  3. combine: merges each row's records, undoes the value rotation.
// What bounds it: shared-memory bandwidth of unpacking (codebook lookups, tile
// stores, operand reads) at few rows; the exponentials and the tensor cores at
// 256 rows.
#include <algorithm>
#include <cstddef>

#include "prefix.cuh"
#include "quant_dev.cuh"
#include "splitk.cuh"
#include "tcgen.cuh"

namespace kvq {

__device__ __align__(16) const uint32_t g_plut[KVQ_LUT_BYTES / 4] = KVQ_LUT_IMAGE;
static_assert(KVQ_LUT_BYTES >= 512 * 16 + 128, "placeholder source of a refused page's tile");

constexpr int kTok = 128;       // tokens of a K/V tile
constexpr int kPThreads = 512;  // 2 softmax warpgroups, copy, MMA and 6 unpack warps
constexpr int kUnpackWarps = 6;
constexpr int kCopyWarp = 8, kMmaWarp = 9, kUnpackWarp0 = 10;
constexpr int kDescUsers = 8 + 1 + kUnpackWarps;  // warps that read a segment descriptor
constexpr uint32_t kPanel = 16384;                // 128 rows x 64 fp16, swizzled
constexpr uint32_t kTileBytes = 2 * kPanel;
constexpr uint32_t kQImage = 2 * kTileBytes;      // one unit's query image
constexpr int kSufRows = 16;                      // rows of a sequence's query image
constexpr uint32_t kSufImage = 2 * 2 * kSufRows * 128;  // 2 panels, hi and lo
constexpr int kMaxRing = 8;
constexpr int kNormSlots = 4;
// TMEM columns
constexpr uint32_t kColS = 0, kColO = 256;
// P is kept below 2^kPTop; a softmax reference moves when a tile would pass it,
// to leave the tile's largest P at 2^kPSet
constexpr float kPTop = 15.f, kPSet = 7.f;
// cost of a segment's start and of one tile (shared: 256 rows; else <= 128)
constexpr int kCostSeg = 3, kCostShared = 5, kCostAlt = 3;

// ---------------------------------------------------------------- workspace
struct PfxHead {
  int64_t total;    // cost of all units
  int64_t suffix0;  // cost of the prefix units
  int64_t n_punits;
};
struct PfxLayout {
  size_t head, gstart, gunit, gcost, scost, isc_p, isc_s, q_p, q_s, ml_p, ml_s, o_p, o_s, bytes;
};

static size_t up256(size_t x) { return (x + 255) / 256 * 256; }

// n_ctas bounds the main grid; rows per prefix unit are 256 or 128 by output
// type, and the layout covers both (units: the 128-row count; record rows: 256).
static PfxLayout pfx_layout(int batch, int n_q, int n_kv, int n_groups, int n_ctas) {
  const int G = n_q / n_kv;
  const size_t units = (size_t)n_kv * (n_groups + ((size_t)batch * G + 127) / 128);
  // incidences of (CTA, unit): one per step of a staircase
  const size_t inc_p = units + n_ctas, inc_s = (size_t)batch * n_kv + n_ctas;
  PfxLayout w;
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t a = at;
    at += up256(n);
    return a;
  };
  w.head = take(sizeof(PfxHead));
  w.gstart = take((size_t)(n_groups + 1) * 4);
  w.gunit = take((size_t)(n_groups + 1) * 4);
  w.gcost = take((size_t)(n_groups + 1) * 8);
  w.scost = take((size_t)(batch + 1) * 8);
  w.isc_p = take((size_t)batch * n_q * 4);
  w.isc_s = take((size_t)batch * n_q * 4);
  w.q_p = take(units * kQImage);
  w.q_s = take((size_t)batch * n_kv * kSufImage);
  w.ml_p = take(inc_p * 256 * 8);
  w.ml_s = take(inc_s * 2 * G * 8);
  w.o_p = take(inc_p * 256 * 512);
  w.o_s = take(inc_s * 2 * G * 512);
  w.bytes = at;
  return w;
}

struct PrefixParams {
  PrefixArgs a;
  int G, tile_bytes, n_ctas;
  int rows_unit;  // 256 or 128 rows per prefix unit
  PfxHead* head;
  int32_t *gstart, *gunit;
  int64_t *gcost, *scost;
  float *isc_p, *isc_s;
  uint8_t *q_p, *q_s;
  float2 *ml_p, *ml_s;
  float *o_p, *o_s;
  int ring, slot_bytes;
};

__device__ __forceinline__ int clamp_len(int32_t l, int64_t most) {
  return (int)min((int64_t)max(l, 0), most);
}
__device__ __forceinline__ int tiles_of(int len) { return (len + kTok - 1) / kTok; }

// Cost line of one group: n_kv blocks of nrt units, the last of `last` rows.
struct GroupCost {
  int tiles, nrt, last;
  int64_t full, lastc, block;  // costs: a full unit, the last one, one KV head
};
__device__ __forceinline__ GroupCost group_cost(int rows, int tiles, int rows_unit) {
  GroupCost c;
  c.tiles = tiles;
  c.nrt = (rows + rows_unit - 1) / rows_unit;
  c.last = rows - (c.nrt - 1) * rows_unit;
  const bool any = tiles > 0 && rows > 0;
  c.full = any ? kCostSeg + (int64_t)tiles * (rows_unit > 128 ? kCostShared : kCostAlt) : 0;
  c.lastc = any ? kCostSeg + (int64_t)tiles * (c.last > 128 ? kCostShared : kCostAlt) : 0;
  c.block = any ? (c.nrt - 1) * c.full + c.lastc : 0;
  return c;
}
__device__ __forceinline__ int64_t seq_cost(int tiles, int n_kv) {
  return tiles > 0 ? (int64_t)n_kv * (kCostSeg + (int64_t)tiles * kCostAlt) : 0;
}

// First position of CTA c's piece of the cost line.
__device__ __forceinline__ int64_t cut(int64_t total, int c, int n) { return total * c / n; }
// Number of a unit's tiles that start before position x of the cost line.
__device__ __forceinline__ int tiles_before(int64_t x, int64_t start, int tiles, bool shared) {
  const int64_t d = x - start - kCostSeg;
  if (d <= 0) return 0;
  const int64_t n = shared ? (d + kCostShared - 1) / kCostShared : (d + kCostAlt - 1) / kCostAlt;
  return (int)min(n, (int64_t)tiles);
}

// ---------------------------------------------------------------------- prep
// CTA 0: the schedule. CTA 1 + b n_kv + h: the query rows of sequence b, KV head
// h, for the prefix part (with the plan of the group's first sequence, which
// coded the prefix) and for the sequence's own part.
constexpr int kPrepThreads = 256;

struct PrepSmem {
  Plan plan;
  RotTables rot;
  int gstart[kPfxMaxGroups + 1];
  int gunit[kPfxMaxGroups + 1];
  int64_t warp_sum[8];
  alignas(16) float row[8][kHeadDim];
};

// Group starts made ascending in 0..batch, and the first unit of each group;
// by warp 0. Returns whether the starts were in order already.
__device__ __forceinline__ bool group_tables(const PrefixParams& p, PrepSmem& sm, int lane) {
  const int n = p.a.n_groups;
  int run = 0, units = 0;
  bool ok = true;
  for (int i0 = 0; i0 <= n; i0 += 32) {
    const int i = i0 + lane;
    const int raw = i <= n ? p.a.group_start[i] : 0;
    int v = i <= n ? min(max(raw, 0), p.a.batch) : 0;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, v, d);
      if (lane >= d) v = max(v, y);
    }
    v = max(v, run);
    run = __shfl_sync(0xffffffffu, v, 31);
    if (i <= n) {
      sm.gstart[i] = v;
      ok &= raw == v;
    }
  }
  __syncwarp();
  for (int i0 = 0; i0 < n; i0 += 32) {
    const int i = i0 + lane;
    const int rows = i < n ? (sm.gstart[i + 1] - sm.gstart[i]) * p.G : 0;
    const int u = (rows + p.rows_unit - 1) / p.rows_unit * p.a.n_kv;
    int s = u;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, s, d);
      if (lane >= d) s += y;
    }
    if (i < n) sm.gunit[i] = units + s - u;
    units += __shfl_sync(0xffffffffu, s, 31);
  }
  if (lane == 0) sm.gunit[n] = units;
  __syncwarp();
  return __all_sync(0xffffffffu, ok);
}

__device__ __forceinline__ int64_t block_sum_before(int64_t x, int64_t* warp_sum, int64_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t inc = x;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, inc, d);
    if (lane >= d) inc += y;
  }
  __syncthreads();
  if (lane == 31) warp_sum[warp] = inc;
  __syncthreads();
  int64_t before = 0;
  total = 0;
  for (int w = 0; w < kPrepThreads / 32; ++w) {
    if (w < warp) before += warp_sum[w];
    total += warp_sum[w];
  }
  return before + inc - x;
}

__device__ void prep_schedule(const PrefixParams& p, PrepSmem& sm) {
  const int tid = threadIdx.x, n = p.a.n_groups;
  uint32_t flags = 0;
  int64_t base = 0;
  for (int i0 = 0; i0 < n; i0 += kPrepThreads) {
    const int i = i0 + tid;
    int64_t c = 0;
    if (i < n) {
      const int raw = p.a.pre_len[i];
      if (raw > p.a.max_pre) flags |= KVQ_FLAG_CAPACITY;
      const int rows = (sm.gstart[i + 1] - sm.gstart[i]) * p.G;
      c = p.a.n_kv *
          group_cost(rows, tiles_of(clamp_len(raw, p.a.max_pre)), p.rows_unit).block;
    }
    int64_t total;
    const int64_t before = block_sum_before(c, sm.warp_sum, total);
    if (i < n) {
      p.gcost[i] = base + before;
      p.gstart[i] = sm.gstart[i];
      p.gunit[i] = sm.gunit[i];
    }
    base += total;
  }
  const int64_t suffix0 = base;
  for (int i0 = 0; i0 < p.a.batch; i0 += kPrepThreads) {
    const int i = i0 + tid;
    int64_t c = 0;
    if (i < p.a.batch) {
      const int raw = p.a.len[i];
      if (raw > p.a.max_len) flags |= KVQ_FLAG_CAPACITY;
      c = seq_cost(tiles_of(clamp_len(raw, p.a.max_len)), p.a.n_kv);
    }
    int64_t total;
    const int64_t before = block_sum_before(c, sm.warp_sum, total);
    if (i < p.a.batch) p.scost[i] = base + before;
    base += total;
  }
  if (tid == 0) {
    p.gcost[n] = suffix0;
    p.gstart[n] = sm.gstart[n];
    p.gunit[n] = sm.gunit[n];
    p.scost[p.a.batch] = base;
    p.head->total = base;
    p.head->suffix0 = suffix0;
    p.head->n_punits = sm.gunit[n];
  }
  if (flags) atomicOr(p.a.status, flags);
}

// One query row (a warp) as fp16 operand row `row` of the image at img (panel
// stride `panel`), its low part at img_lo; isc gets 2^-sigma.
__device__ __forceinline__ void prep_row(const PrefixParams& p, const PrepSmem& sm, bool plan_ok,
                                         float* buf, int b, int head, uint8_t* img, uint8_t* img_lo,
                                         uint32_t panel, int row, float* isc, int lane) {
  const Plan& pl = sm.plan;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int x = lane + 32 * i;
    const size_t qi = ((size_t)b * p.a.n_q + head) * kHeadDim + x;
    buf[x] = load_as_float(p.a.q, p.a.q_dtype, qi) * pl.a_hat[x & 63] * 0.12751743074f;
  }  // 0.12751743 = log2(e) / sqrt(128)
  __syncwarp();
  const bool rot = plan_ok && pl.k_rot != 0;
  if (rot) warp_rotate_row(buf, pl, sm.rot, nullptr, lane);
  const int nr = plan_ok ? pl.n_ranks : 0;
  float2 v[2];
  float mx = 0.f;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = lane + 32 * i;
    v[i] = make_float2(0.f, 0.f);
    if (r < nr) {
      const int j = pl.order[r] & 63;
      v[i] = rot ? make_float2(buf[2 * r], buf[2 * r + 1]) : make_float2(buf[j], buf[j + 64]);
    }
    mx = fmaxf(mx, fmaxf(fabsf(v[i].x), fabsf(v[i].y)));
  }
#pragma unroll
  for (int m = 16; m; m >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, m));
  const int sigma = (mx > 0.f && isfinite(mx)) ? 14 - ilogbf(mx) : 0;
  const float sc = ldexpf(1.f, min(sigma, 127));
  if (lane == 0) *isc = ldexpf(1.f, -min(sigma, 127));
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float x0 = v[i].x * sc, x1 = v[i].y * sc;  // rank lane + 32 i
    const uint32_t hi = pack_half2(x0, x1);
    const uint32_t at = i * panel + row * 128 + ((((uint32_t)lane >> 2) ^ (row & 7)) << 4) +
                        (lane & 3) * 4;
    *reinterpret_cast<uint32_t*>(img + at) = hi;
    if (img_lo) {
      const __half2 hh = *reinterpret_cast<const __half2*>(&hi);
      *reinterpret_cast<uint32_t*>(img_lo + at) =
          pack_half2(x0 - __low2float(hh), x1 - __high2float(hh));
    }
  }
  __syncwarp();
}

__device__ __forceinline__ bool load_plan(const PrefixParams& p, PrepSmem& sm, const Plan* src) {
  __syncthreads();
  const uint32_t* s = reinterpret_cast<const uint32_t*>(src);
  for (int i = threadIdx.x; i < KVQ_PLAN_BYTES / 4; i += kPrepThreads)
    reinterpret_cast<uint32_t*>(&sm.plan)[i] = s[i];
  __syncthreads();
  const bool ok = sm.plan.magic == KVQ_PLAN_MAGIC && sm.plan.bits_k == p.a.bits_k &&
                  sm.plan.bits_v == p.a.bits_v && plan_sched_ok(sm.plan, threadIdx.x & 31);
  if (ok && sm.plan.k_rot) rot_tables(sm.plan, sm.rot, threadIdx.x);
  if (!ok && threadIdx.x == 0) atomicOr(p.a.status, KVQ_FLAG_BAD_PLAN);
  __syncthreads();
  return ok;
}

template <bool SPLIT>
__global__ void __launch_bounds__(kPrepThreads) prefix_prep_kernel(const PrefixParams p) {
  __shared__ PrepSmem sm;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  grid_dep_launch();
  grid_dep_wait();
  if (warp == 0) {
    const bool ok = group_tables(p, sm, lane);
    if (!ok && lane == 0 && blockIdx.x == 0) atomicOr(p.a.status, KVQ_FLAG_BAD_PAGE);
  }
  __syncthreads();
  if (blockIdx.x == 0) {
    prep_schedule(p, sm);
    return;
  }
  const int bh = blockIdx.x - 1, b = bh / p.a.n_kv, h = bh - b * p.a.n_kv, n = p.a.n_groups;
  int g = 0;
  {  // the last group that starts at or before b
    int len = n + 1;
    while (len > 1) {
      const int half = len >> 1;
      if (sm.gstart[g + half] <= b) g += half;
      len -= half;
    }
  }
  const bool grouped = g < n && sm.gstart[g] <= b;
  const Plan* const own = p.a.plans[b] + h;
  const Plan* const pre = grouped ? p.a.plans[sm.gstart[g]] + h : own;
  bool ok = load_plan(p, sm, own);
  uint8_t* const img = p.q_s + (size_t)bh * kSufImage;
  for (int i = warp; i < p.G; i += kPrepThreads / 32)
    prep_row(p, sm, ok, sm.row[warp], b, h * p.G + i, img,
             SPLIT ? img + kSufImage / 2 : nullptr, kSufRows * 128, i,
             p.isc_s + (size_t)b * p.a.n_q + h * p.G + i, lane);
  if (!grouped) return;
  if (pre != own) {
    uint32_t sign[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) sign[i] = sm.plan.v_sign[i];
    ok = load_plan(p, sm, pre);
    // records of both parts are merged before the rotation is undone
    bool same = true;
#pragma unroll
    for (int i = 0; i < 4; ++i) same &= sign[i] == sm.plan.v_sign[i];
    if (!same && tid == 0) atomicOr(p.a.status, KVQ_FLAG_BAD_PLAN);
  }
  const int rows = (sm.gstart[g + 1] - sm.gstart[g]) * p.G;
  const int nrt = (rows + p.rows_unit - 1) / p.rows_unit;
  for (int i = warp; i < p.G; i += kPrepThreads / 32) {
    const int rr = (b - sm.gstart[g]) * p.G + i, rt = rr / p.rows_unit, r = rr % p.rows_unit;
    uint8_t* const u = p.q_p + (size_t)(sm.gunit[g] + h * nrt + rt) * kQImage;
    prep_row(p, sm, ok, sm.row[warp], b, h * p.G + i, SPLIT ? u : u + (r >> 7) * kTileBytes,
             SPLIT ? u + kTileBytes : nullptr, kPanel, r & 127,
             p.isc_p + (size_t)b * p.a.n_q + h * p.G + i, lane);
  }
}

// ---------------------------------------------------------------------- main
struct alignas(16) Desc {  // one segment: a run of tiles of one unit
  Plan plan;               // 16-byte aligned (bulk copy)
  float2* ml;
  float* o;
  const float* isc;
  int stop, shared, rows, tiles, tile0, len, b0, row0, h, qslot, sub;
};

struct alignas(128) MainSmem {
  uint8_t lut[KVQ_LUT_BYTES];
  Desc desc[2];
  alignas(16) float nk[kNormSlots][kTok];
  alignas(16) float nv[kNormSlots][kTok];
  int lg[kNormSlots][4];  // per record: the value norms are below 2^lg
  unsigned long long desc_full[2], desc_empty[2], ring_full[kMaxRing], ring_empty[kMaxRing];
  unsigned long long q_full[2], q_empty[2], k_full[2], k_empty[2], v_full[2], v_empty[2];
  unsigned long long s_full[2], p_ready[2], o_full[2], o_free[2], lut_full, drain;
  uint32_t tmem;
  int fail;
};
constexpr size_t kMainTiles = 6 * (size_t)kTileBytes;  // Q x 2, K x 2, V x 2
constexpr size_t kMaxSmem = 227 * 1024;
static_assert(offsetof(MainSmem, desc) % 16 == 0 && sizeof(Desc) % 16 == 0, "bulk destinations");

// Bounded wait that also gives up once another role has: the role then leaves
// its loop, and the CTA drains and ends with the TIMEOUT flag.
__device__ __forceinline__ bool wait_on(MainSmem& sm, unsigned long long* bar, uint32_t phase) {
  if (mbar_try_wait(bar, phase)) return true;
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, phase)) {
    if (clock64() - t0 > kWaitCycles || *(volatile int*)&sm.fail) {
      *(volatile int*)&sm.fail = 1;
      return false;
    }
  }
  return true;
}

// The same by a whole warp: every lane gets the same answer, so that a warp
// leaves its role as one.
__device__ __forceinline__ bool wait_warp(MainSmem& sm, unsigned long long* bar, uint32_t phase) {
  return __all_sync(0xffffffffu, wait_on(sm, bar, phase));
}

// Unit of work during the copy warp's walk along the cost line (warp-uniform).
struct Unit {
  bool suffix, shared;
  int g, b, h, rt;    // prefix: group, KV head, row tile; suffix: sequence, KV head
  int nrt, rows, len, tiles;
  int64_t start, cost, idx;
};

__device__ __forceinline__ Unit prefix_unit(const PrefixParams& p, int g, int h, int rt) {
  Unit u;
  const int b0 = p.gstart[g], rows = (p.gstart[g + 1] - b0) * p.G;
  u.suffix = false;
  u.g = g;
  u.b = b0;
  u.h = h;
  u.rt = rt;
  u.len = clamp_len(p.a.pre_len[g], p.a.max_pre);
  u.tiles = tiles_of(u.len);
  const GroupCost c = group_cost(rows, u.tiles, p.rows_unit);
  u.nrt = c.nrt;
  u.rows = rt == c.nrt - 1 ? c.last : p.rows_unit;
  u.shared = u.rows > 128;
  u.start = p.gcost[g] + h * c.block + rt * c.full;
  u.cost = rt == c.nrt - 1 ? c.lastc : c.full;
  u.idx = p.gunit[g] + h * c.nrt + rt;
  return u;
}
__device__ __forceinline__ Unit suffix_unit(const PrefixParams& p, int b, int h) {
  Unit u;
  u.suffix = true;
  u.shared = false;
  u.g = u.rt = u.nrt = 0;
  u.b = b;
  u.h = h;
  u.rows = p.G;
  u.len = clamp_len(p.a.len[b], p.a.max_len);
  u.tiles = tiles_of(u.len);
  u.cost = u.tiles > 0 ? kCostSeg + (int64_t)u.tiles * kCostAlt : 0;
  u.start = p.scost[b] + h * u.cost;
  u.idx = (int64_t)b * p.a.n_kv + h;
  return u;
}

// Largest i in [0, n) with a[i] <= x, by a warp (a ascending, a[0] <= x).
__device__ __forceinline__ int warp_last_le(const int64_t* a, int n, int64_t x, int lane) {
  int lo = 0;
  while (n > 1) {
    const int step = (n + 31) / 32;
    const bool le = lane * step < n && a[lo + lane * step] <= x;
    const int k = __popc(__ballot_sync(0xffffffffu, le)) - 1;
    lo += k * step;
    n = min(step, n - k * step);
  }
  return lo;
}

__device__ __forceinline__ Unit unit_at(const PrefixParams& p, int64_t x, int64_t suffix0,
                                        int lane) {
  if (x < suffix0) {
    const int g = warp_last_le(p.gcost, p.a.n_groups, x, lane);
    const int rows = (p.gstart[g + 1] - p.gstart[g]) * p.G;
    const GroupCost c =
        group_cost(rows, tiles_of(clamp_len(p.a.pre_len[g], p.a.max_pre)), p.rows_unit);
    const int64_t d = x - p.gcost[g];
    const int h = (int)(d / c.block);
    const int rt = (int)min((d - h * c.block) / c.full, (int64_t)c.nrt - 1);
    return prefix_unit(p, g, h, rt);
  }
  const int b = warp_last_le(p.scost, p.a.batch, x, lane);
  const Unit u = suffix_unit(p, b, 0);
  return u.cost > 0 ? suffix_unit(p, b, (int)min((x - u.start) / u.cost, (int64_t)p.a.n_kv - 1))
                    : u;
}

// 32 tokens of keys: one half step (<= 4 blocks of width W) of one record into
// rows 32 rec + (0..31) of the K tile. Lane (g, c): block c, tokens g + 8 i.
__device__ __forceinline__ void unpack_keys(const MainSmem& sm, const Plan& pl, const uint8_t* kw,
                                            int hs, uint8_t* tile, int rec, int lane) {
  const int g = lane >> 2, c = lane & 3;
  const int W = pl.hs_width[hs], r0 = pl.hs_rank0[hs], n = pl.hs_count[hs];
  const int cc = min(c, n - 1), rank = r0 + cc;
  const int off = pl.seg_off[r0] + 2 * W * cc + ((W * g) >> 2);
  const uint32_t sh = (uint32_t)(8 * W * g) & 31u;
  const uint8_t* wp = kw + 4 * off;
  const uint8_t* lut = sm.lut;
  const uint32_t w2 = 2u * (uint32_t)W;
  uint32_t A[4];
  if (W <= 3) {
    const uint32_t m7 = ((1u << w2) - 1u) << 7;
    const uint32_t lb = ((uint32_t)lane * 4u) | (W == 1 ? 0x4000u : W == 2 ? 0x2000u : 0u);
    const uint32_t v7 = funnel_r(*reinterpret_cast<const uint32_t*>(wp),
                                 *reinterpret_cast<const uint32_t*>(wp + 4), sh) << 7;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      A[i] = *reinterpret_cast<const uint32_t*>(lut + (((v7 >> (w2 * i)) & m7) | lb));
  } else {
    const uint32_t w0 = *reinterpret_cast<const uint32_t*>(wp);
    const uint32_t w1 = *reinterpret_cast<const uint32_t*>(wp + 4);
    const uint32_t x2 = W > 4 ? *reinterpret_cast<const uint32_t*>(wp + 8) : 0u;
    const unsigned long long v = ((unsigned long long)funnel_r(w1, x2, sh) << 32) |
                                 funnel_r(w0, w1, sh);
    if (W <= 5) {  // pair tables
      const uint8_t* tab = lut + (W == 4 ? 0x2800u : 0x2C00u);
      const uint32_t m = (1u << w2) - 1u;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        A[i] = *reinterpret_cast<const uint32_t*>(tab + 4u * ((uint32_t)(v >> (w2 * i)) & m));
    } else {  // single codes
      const uint8_t* tab = lut + 0x3C00u + 2u * (uint32_t)((1 << W) - 2);
      const uint32_t m = (1u << W) - 1u;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t f = (uint32_t)(v >> (w2 * i));
        A[i] = *reinterpret_cast<const uint16_t*>(tab + 2u * (f & m)) |
               ((uint32_t)*reinterpret_cast<const uint16_t*>(tab + 2u * ((f >> W) & m)) << 16);
      }
    }
  }
  if (c < n) {
    uint8_t* dst = tile + (rank >> 5) * kPanel + (32 * rec + g) * 128 +
                   ((((uint32_t)rank & 31u) >> 2 ^ (uint32_t)g) << 4) + (rank & 3) * 4;
#pragma unroll
    for (int i = 0; i < 4; ++i) *reinterpret_cast<uint32_t*>(dst + i * 8 * 128) = A[i];
  }
}

// 8 rotated value coordinates (rows 8 m .. 8 m + 7 of the V tile) of the 32
// tokens of record `rec`. Lane (g, c): coordinate 8 m + g, tokens 8 i + 2 c + (0, 1).
template <int BV>
__device__ __forceinline__ void unpack_values(const MainSmem& sm, const uint8_t* vw, int m,
                                              uint8_t* tile, int rec, int lane) {
  const int g = lane >> 2, c = lane & 3, row = 8 * m + g;
  const uint8_t* wp = vw + 4 * (row * BV + ((BV * c) >> 2));
  const uint32_t sh = (uint32_t)(8 * BV * c) & 31u;
  const uint8_t* lut = sm.lut;
  uint32_t F[4];
  if constexpr (BV <= 3) {
    constexpr uint32_t m7 = ((1u << (2 * BV)) - 1u) << 7;
    const uint32_t lb = ((uint32_t)lane * 4u) | (BV == 1 ? 0x4000u : BV == 2 ? 0x2000u : 0u);
    const uint32_t v7 = funnel_r(*reinterpret_cast<const uint32_t*>(wp),
                                 *reinterpret_cast<const uint32_t*>(wp + 4), sh) << 7;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      F[i] = *reinterpret_cast<const uint32_t*>(lut + (((v7 >> (2 * BV * i)) & m7) | lb));
  } else {
    const uint32_t w0 = *reinterpret_cast<const uint32_t*>(wp);
    const uint32_t w1 = *reinterpret_cast<const uint32_t*>(wp + 4);
    const uint32_t x2 = BV > 4 ? *reinterpret_cast<const uint32_t*>(wp + 8) : 0u;
    const unsigned long long v = ((unsigned long long)funnel_r(w1, x2, sh) << 32) |
                                 funnel_r(w0, w1, sh);
    if constexpr (BV <= 5) {
      const uint8_t* tab = lut + (BV == 4 ? 0x2800u : 0x2C00u);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        F[i] = *reinterpret_cast<const uint32_t*>(
            tab + 4u * ((uint32_t)(v >> (2 * BV * i)) & ((1u << (2 * BV)) - 1u)));
    } else {
      const uint8_t* tab = lut + 0x3C00u + 2u * (uint32_t)((1 << BV) - 2);
      constexpr uint32_t mm = (1u << BV) - 1u;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t f = (uint32_t)(v >> (2 * BV * i));
        F[i] = *reinterpret_cast<const uint16_t*>(tab + 2u * (f & mm)) |
               ((uint32_t)*reinterpret_cast<const uint16_t*>(tab + 2u * ((f >> BV) & mm)) << 16);
      }
    }
  }
  uint8_t* dst = tile + (rec >> 1) * kPanel + row * 128 + c * 4;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    *reinterpret_cast<uint32_t*>(dst + (((uint32_t)(4 * (rec & 1) + i) ^ (uint32_t)g) << 4)) = F[i];
}

// ---- the roles of the main kernel

template <bool SPLIT>
__device__ void copy_role(const PrefixParams& p, MainSmem& sm, uint8_t* qbuf, uint8_t* ring,
                          int lane) {
  const int64_t total = p.head->total, suffix0 = p.head->suffix0;
  const int64_t x0 = cut(total, blockIdx.x, p.n_ctas), x1 = cut(total, blockIdx.x + 1, p.n_ctas);
  const int bk = p.a.bits_k, bv = p.a.bits_v;
  uint32_t seg = 0, rc = 0;        // segments, ring slots issued
  uint32_t quse[2] = {0u, 0u};     // segments that used each query slot
  int qnext = 0;
  bool ok = true;
  if (x0 < x1) {
    Unit u = unit_at(p, x0, suffix0, lane);
    while (ok && u.start < x1) {
      const int t0 = tiles_before(x0, u.start, u.tiles, u.shared);
      const int t1 = tiles_before(x1, u.start, u.tiles, u.shared);
      if (t0 < t1) {
        // ---- descriptor, plan and query rows
        const uint32_t ds = seg & 1;
        if (!wait_warp(sm, &sm.desc_empty[ds], ((seg >> 1) & 1) ^ 1)) {
          ok = false;
          break;
        }
        const bool both = u.shared || SPLIT;
        const int qs = both ? 0 : qnext;
        if (lane == 0) {
          Desc& d = sm.desc[ds];
          const size_t inc = (size_t)blockIdx.x + (size_t)u.idx;
          d.ml = u.suffix ? p.ml_s + inc * 2 * p.G : p.ml_p + inc * 256;
          d.o = u.suffix ? p.o_s + inc * 2 * p.G * kHeadDim : p.o_p + inc * 256 * kHeadDim;
          d.isc = u.suffix ? p.isc_s : p.isc_p;
          d.stop = 0;
          d.shared = u.shared;
          d.rows = u.rows;
          d.tiles = t1 - t0;
          d.tile0 = t0;
          d.len = u.len;
          d.b0 = u.b;
          d.row0 = u.rt * p.rows_unit;
          d.h = u.h;
          d.qslot = qs;
          d.sub = u.suffix ? p.G : 128;
          mbar_expect_tx(&sm.desc_full[ds], KVQ_PLAN_BYTES);
          bulk_g2s(&d.plan, p.a.plans[u.b] + u.h, KVQ_PLAN_BYTES, &sm.desc_full[ds]);
        }
        __syncwarp();
        ++seg;
        for (int i = 0; i < (both ? 2 : 1) && ok; ++i) {
          const int s = qs + i;
          ok = wait_warp(sm, &sm.q_empty[s], (quse[s] & 1) ^ 1);
          if (!ok) break;
          // rows of this slot: the row tile of stream i, or all rows (hi, lo)
          const int rows = u.shared ? min(128, u.rows - 128 * i) : u.rows;
          const uint32_t bytes = (uint32_t)(rows + 7) / 8 * 1024;
          if (lane == 0) {
            const uint8_t* src = u.suffix ? p.q_s + (size_t)u.idx * kSufImage + i * (kSufImage / 2)
                                          : p.q_p + (size_t)u.idx * kQImage + i * kTileBytes;
            const uint32_t panel = u.suffix ? kSufRows * 128 : kPanel;
            mbar_expect_tx(&sm.q_full[s], 2 * bytes);
            bulk_g2s(qbuf + s * kTileBytes, src, bytes, &sm.q_full[s]);
            bulk_g2s(qbuf + s * kTileBytes + kPanel, src + panel, bytes, &sm.q_full[s]);
          }
          __syncwarp();
          ++quse[s];
        }
        if (!both) qnext ^= 1;
        // ---- packed records, keys then values of each tile; the pages of the
        //      next 32 records are looked up by the 32 lanes at once
        const CacheMap& cm = u.suffix ? p.a.own : p.a.pre;
        const int row = u.suffix ? u.b : u.g;
        const int n_rec = (u.len + kTile - 1) / kTile, mask = page_mask(cm);
        unsigned long long base = 0;
        for (int t = t0; t < t1 && ok; ++t) {
          if (((t - t0) & 7) == 0) {
            const int rec = 4 * t + lane;
            base = rec < n_rec
                       ? (unsigned long long)(uintptr_t)page_base(cm, row, rec) : 0ull;
          }
          for (int part = 0; part < 2 && ok; ++part)
            for (int r = 0; r < 4; ++r) {
              const int rec = 4 * t + r;
              const unsigned long long pb =
                  __shfl_sync(0xffffffffu, base, 4 * ((t - t0) & 7) + r);
              if (rec >= n_rec) break;
              const uint32_t slot = rc % p.ring;
              ok = wait_warp(sm, &sm.ring_empty[slot], ((rc / p.ring) & 1) ^ 1);
              if (!ok) break;
              if (lane == 0) {
                const uint8_t* src = reinterpret_cast<const uint8_t*>(g_plut);
                if (pb && !(pb & 15))
                  src = reinterpret_cast<const uint8_t*>((uintptr_t)pb) +
                        ((size_t)(rec & mask) * p.a.n_kv + u.h) * p.tile_bytes;
                else  // refused: placeholder bytes are streamed, the output is flagged
                  atomicOr(p.a.status, pb ? KVQ_FLAG_BAD_PLAN : KVQ_FLAG_BAD_PAGE);
                uint8_t* dst = ring + (size_t)slot * p.slot_bytes;
                if (part == 0) {
                  mbar_expect_tx(&sm.ring_full[slot], 512 * bk + 128);
                  bulk_g2s(dst, src, 512 * bk, &sm.ring_full[slot]);
                  bulk_g2s(dst + 512 * bk, src + 512 * (bk + bv), 128, &sm.ring_full[slot]);
                } else {
                  mbar_expect_tx(&sm.ring_full[slot], 512 * bv);
                  bulk_g2s(dst, src + 512 * bk, 512 * bv, &sm.ring_full[slot]);
                }
              }
              __syncwarp();
              ++rc;
            }
        }
      }
      // ---- next unit with any cost
      if (!u.suffix) {
        int g = u.g, h = u.h, rt = u.rt + 1;
        if (rt == u.nrt) {
          rt = 0;
          if (++h == p.a.n_kv) {
            h = 0;
            ++g;
            while (g < p.a.n_groups && p.gcost[g + 1] == p.gcost[g]) ++g;
          }
        }
        if (g < p.a.n_groups) {
          u = prefix_unit(p, g, h, rt);
          continue;
        }
        if (suffix0 >= x1) break;
        u = unit_at(p, suffix0, suffix0, lane);
        if (u.cost == 0) break;
        continue;
      }
      int b = u.b, h = u.h + 1;
      if (h == p.a.n_kv) {
        h = 0;
        const int64_t end = p.scost[b + 1];
        if (end >= x1) break;
        b = warp_last_le(p.scost, p.a.batch, end, lane);
      }
      u = suffix_unit(p, b, h);
    }
  }
  if (ok) {  // the end of the CTA's work
    const uint32_t ds = seg & 1;
    ok = wait_warp(sm, &sm.desc_empty[ds], ((seg >> 1) & 1) ^ 1);
    if (ok && lane == 0) {
      sm.desc[ds].stop = 1;
      mbar_arrive(&sm.desc_full[ds]);
    }
  }
  if (!ok) {  // let the copies in flight land before the CTA ends
    for (uint32_t i = 0; i < (uint32_t)p.ring && i < rc; ++i)
      (void)mbar_wait_bounded(&sm.ring_full[(rc - 1 - i) % p.ring], ((rc - 1 - i) / p.ring) & 1);
    for (int s = 0; s < 2; ++s)
      if (quse[s]) (void)mbar_wait_bounded(&sm.q_full[s], (quse[s] - 1) & 1);
    for (uint32_t i = 1; i <= 2 && i <= seg; ++i)
      (void)mbar_wait_bounded(&sm.desc_full[(seg - i) & 1], ((seg - i) >> 1) & 1);
  }
}

template <int BV>
__device__ void unpack_role(const PrefixParams& p, MainSmem& sm, uint8_t* kbuf, uint8_t* vbuf,
                            const uint8_t* ring, int uw, int lane) {
  uint32_t seg = 0, rc = 0, tile_no = 0;
  if (!wait_warp(sm, &sm.lut_full, 0)) return;
  for (;; ++seg) {
    const uint32_t ds = seg & 1;
    if (!wait_warp(sm, &sm.desc_full[ds], (seg >> 1) & 1)) return;
    const Desc& d = sm.desc[ds];
    if (d.stop) return;
    const Plan& pl = d.plan;
    const bool plan_ok = pl.magic == KVQ_PLAN_MAGIC && pl.bits_k == p.a.bits_k &&
                         pl.bits_v == BV && plan_sched_ok(pl, lane);
    if (!plan_ok && uw == 0 && lane == 0) atomicOr(p.a.status, KVQ_FLAG_BAD_PLAN);
    const int n_half = plan_ok ? pl.n_half : 0;
    const int n_rec = (d.len + kTile - 1) / kTile, norm_off = 512 * p.a.bits_k;
    const int tiles = d.tiles, tile0 = d.tile0, len = d.len;
    for (int t = 0; t < tiles; ++t, ++tile_no) {
      const uint32_t st = tile_no & 1, ph = (tile_no >> 1) & 1, ns = tile_no % kNormSlots;
      if (!wait_warp(sm, &sm.k_empty[st], ph ^ 1)) return;
      for (int r = 0; r < 4; ++r) {
        const int rec = 4 * (tile0 + t) + r;
        if (rec < n_rec) {
          const uint32_t slot = rc % p.ring;
          if (!wait_warp(sm, &sm.ring_full[slot], (rc / p.ring) & 1)) return;
          const uint8_t* w = ring + (size_t)slot * p.slot_bytes;
          if (uw == r) {  // norms: masked tokens 0; an exponent above the value norms
            const __half* nrm = reinterpret_cast<const __half*>(w + norm_off);
            const bool in = rec * kTile + lane < len;
            const float kn = in ? __half2float(nrm[lane]) : 0.f;
            const float vn = in ? __half2float(nrm[kTile + lane]) : 0.f;
            sm.nk[ns][32 * r + lane] = kn;
            sm.nv[ns][32 * r + lane] = vn;
            const uint32_t mx = __reduce_max_sync(0xffffffffu, __float_as_uint(vn));
            if (lane == 0) sm.lg[ns][r] = max((int)(mx >> 23) - 126, -24);
          }
          for (int hs = (uw + 2 * r) % kUnpackWarps; hs < n_half; hs += kUnpackWarps)
            unpack_keys(sm, pl, w, hs, kbuf + st * kTileBytes, r, lane);
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.ring_empty[slot]);
          ++rc;
        } else if (uw == r) {
          sm.nk[ns][32 * r + lane] = 0.f;
          sm.nv[ns][32 * r + lane] = 0.f;
          if (lane == 0) sm.lg[ns][r] = -24;
        }
      }
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.k_full[st]);
      if (!wait_warp(sm, &sm.v_empty[st], ph ^ 1)) return;
      for (int r = 0; r < 4; ++r) {
        if (4 * (tile0 + t) + r >= n_rec) break;
        const uint32_t slot = rc % p.ring;
        if (!wait_warp(sm, &sm.ring_full[slot], (rc / p.ring) & 1)) return;
        const uint8_t* w = ring + (size_t)slot * p.slot_bytes;
        for (int m = (uw + 2 * r) % kUnpackWarps; m < 16; m += kUnpackWarps)
          unpack_values<BV>(sm, w, m, vbuf + st * kTileBytes, r, lane);
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.ring_empty[slot]);
        ++rc;
      }
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.v_full[st]);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.desc_empty[ds]);
  }
}

// D fp32, A and B fp16 K-major, M = N = 128.
constexpr uint32_t kIdesc = (1u << 4) | (16u << 17) | (8u << 24);

template <bool SPLIT>
__device__ void mma_role(const PrefixParams& p, MainSmem& sm, const uint8_t* qbuf,
                         const uint8_t* kbuf, const uint8_t* vbuf, uint32_t tmem) {
  uint32_t quse[2] = {0u, 0u}, tile_base = 0;
  uint32_t items[2] = {0u, 0u}, segs[2] = {0u, 0u};  // P tiles consumed, segments, per stream
  const uint64_t qd = smem_desc(smem_addr(qbuf)), kd = smem_desc(smem_addr(kbuf)),
                 vd = smem_desc(smem_addr(vbuf));
  constexpr uint64_t kTileD = kTileBytes >> 4, kPanelD = kPanel >> 4;
  for (uint32_t seg = 0;; ++seg) {
    const uint32_t ds = seg & 1;
    if (!wait_on(sm, &sm.desc_full[ds], (seg >> 1) & 1)) return;
    const Desc& d = sm.desc[ds];
    if (d.stop) return;
    const bool shared = d.shared;
    const int tiles = d.tiles, n_items = shared ? 2 * tiles : tiles, q0 = d.qslot;
    const int ksteps = (min(max(d.plan.n_ranks, 1), 64) + 7) / 8;
    const bool both = shared || SPLIT;
    for (int i = 0; i < (both ? 2 : 1); ++i) {
      if (!wait_on(sm, &sm.q_full[q0 + i], quse[q0 + i] & 1)) return;
      ++quse[q0 + i];
    }
    auto qk = [&](int j) -> bool {
      const int s = j & 1, t = shared ? j >> 1 : j;
      const uint32_t no = tile_base + t, st = no & 1;
      if (!shared || s == 0)
        if (!wait_on(sm, &sm.k_full[st], (no >> 1) & 1)) return false;
      tc_fence_after();
      for (int part = 0; part < (SPLIT ? 2 : 1); ++part) {
        const uint64_t a = qd + (uint64_t)(SPLIT ? part : q0 + (shared ? s : 0)) * kTileD;
        for (int ks = 0; ks < ksteps; ++ks) {
          const uint64_t o = (uint64_t)(ks >> 2) * kPanelD + (uint64_t)(ks & 3) * 2;
          mma_ss(tmem + kColS + 128 * s, a + o, kd + st * kTileD + o, kIdesc, part > 0 || ks > 0);
        }
      }
      mma_commit(&sm.s_full[s]);
      if (!shared || s == 1) mma_commit(&sm.k_empty[st]);
      if (j == n_items - 1) {  // the segment's query rows are no longer needed
        mma_commit(&sm.q_empty[q0]);
        if (both) mma_commit(&sm.q_empty[q0 + 1]);
      }
      return true;
    };
    if (!qk(0)) return;
    if (n_items > 1 && !qk(1)) return;
    for (int j = 0; j < n_items; ++j) {
      const int s = j & 1, t = shared ? j >> 1 : j;
      const uint32_t no = tile_base + t, st = no & 1;
      if (!wait_on(sm, &sm.p_ready[s], items[s] & 1)) return;
      ++items[s];
      if (!shared || s == 0)
        if (!wait_on(sm, &sm.v_full[st], (no >> 1) & 1)) return;
      const bool first = j < 2;
      if (first) {  // the previous segment's O of this stream has been read
        if (!wait_on(sm, &sm.o_free[s], (segs[s] & 1) ^ 1)) return;
        ++segs[s];
      }
      tc_fence_after();
      for (int part = 0; part < (SPLIT ? 2 : 1); ++part)
        for (int ks = 0; ks < 8; ++ks)
          mma_ts(tmem + kColO + 128 * s, tmem + kColS + 128 * s + 64 * part + 8 * ks,
                 vd + st * kTileD + (uint64_t)(ks >> 2) * kPanelD + (uint64_t)(ks & 3) * 2, kIdesc,
                 !first || part > 0 || ks > 0);
      if (!shared || s == 1) mma_commit(&sm.v_empty[st]);
      if (j + 2 >= n_items) mma_commit(&sm.o_full[s]);
      else if (!qk(j + 2)) return;
    }
    tile_base += tiles;
    mbar_arrive(&sm.desc_empty[ds]);
  }
}

// Softmax of stream s (one warpgroup, thread = query row): logits from TMEM,
// running reference m and sum l, P back to TMEM, records at the end.
template <bool SPLIT>
__device__ void softmax_role(const PrefixParams& p, MainSmem& sm, uint32_t tmem, int s, int wq,
                             int lane) {
  uint32_t items = 0, segs = 0, tile_base = 0;
  const uint32_t lane_addr = (uint32_t)(32 * wq) << 16;
  const uint32_t ts = tmem + lane_addr + kColS + 128 * s, to = tmem + lane_addr + kColO + 128 * s;
  for (uint32_t seg = 0;; ++seg) {
    const uint32_t ds = seg & 1;
    if (!wait_warp(sm, &sm.desc_full[ds], (seg >> 1) & 1)) return;
    const Desc& d = sm.desc[ds];
    if (d.stop) return;
    const bool shared = d.shared;
    const int tiles = d.tiles, n = shared ? tiles : (tiles - s + 1) / 2;
    const int rows = shared ? min(128, d.rows - 128 * s) : d.rows;
    const int row = 32 * wq + lane;  // in this stream's tile
    const bool active = 32 * wq < rows, valid = row < rows;  // the warp has rows; this is one
    const int rr = d.row0 + (shared ? 128 * s : 0) + min(row, rows - 1);
    const int qi = (d.b0 + rr / p.G) * p.a.n_q + d.h * p.G + rr % p.G;
    const float isc = active ? d.isc[qi] : 1.f;
    const int len = d.len, tile0 = d.tile0;
    float* const rec_o = d.o + (size_t)(s * d.sub + row) * kHeadDim;
    float2* const rec_ml = d.ml + s * d.sub + row;
    float m = -INFINITY, l = 0.f;
    for (int i = 0; i < n; ++i, ++items) {
      const int t = shared ? i : 2 * i + s;
      const uint32_t ns = (tile_base + t) % kNormSlots;
      if (!wait_warp(sm, &sm.s_full[s], items & 1)) return;
      if (active) {
        tc_fence_after();
        float u[kTok];
#pragma unroll
        for (int c = 0; c < 4; ++c)
          tmem_ld32(ts + 32 * c, reinterpret_cast<uint32_t*>(u) + 32 * c);
        tmem_wait_ld();
        // logits times key norms, the row's maximum
        const float4* nk4 = reinterpret_cast<const float4*>(sm.nk[ns]);
        float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
        for (int c = 0; c < kTok / 4; ++c) {
          const float4 f = nk4[c];
          const float2 a = mul2(make_float2(u[4 * c], u[4 * c + 1]), make_float2(f.x, f.y));
          const float2 b = mul2(make_float2(u[4 * c + 2], u[4 * c + 3]), make_float2(f.z, f.w));
          u[4 * c] = a.x;
          u[4 * c + 1] = a.y;
          u[4 * c + 2] = b.x;
          u[4 * c + 3] = b.y;
        }
        const int nv = len - (tile0 + t) * kTok;
        if (nv < kTok) {  // the last tile: positions past the end
#pragma unroll
          for (int c = 0; c < kTok; ++c)
            if (c >= nv) u[c] = -INFINITY;
        }
#pragma unroll
        for (int c = 0; c < kTok; c += 4) {
          mx0 = fmaxf(fmaxf(mx0, u[c]), u[c + 1]);
          mx1 = fmaxf(fmaxf(mx1, u[c + 2]), u[c + 3]);
        }
        const float top = fmaxf(mx0, mx1) * isc +
                          (float)max(max(sm.lg[ns][0], sm.lg[ns][1]),
                                     max(sm.lg[ns][2], sm.lg[ns][3]));
        // the reference moves only when a product would pass 2^kPTop (or on NaN)
        const bool move = valid && !(top - m <= kPTop);
        if (__any_sync(0xffffffffu, move)) {
          const float m_new = move ? top - kPSet : m;
          const float alpha = move ? ex2(m - m_new) : 1.f;  // 0 from -inf
          l *= alpha;
          if (i > 0) {  // O holds this segment's earlier tiles
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint32_t o[32];
              tmem_ld32(to + 32 * c, o);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
              tmem_st32(to + 32 * c, o);
            }
          }
          m = m_new;
        }
        const float4* nv4 = reinterpret_cast<const float4*>(sm.nv[ns]);
        const float2 isc2 = make_float2(isc, isc), nm2 = make_float2(-m, -m);
        float2 l0 = make_float2(0.f, 0.f), l1 = l0;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t hi[32], lo[SPLIT ? 32 : 1];
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            const int k = 64 * half + 4 * c;
            const float4 f = nv4[16 * half + c];
            float2 a = fma2(make_float2(u[k], u[k + 1]), isc2, nm2);
            float2 b = fma2(make_float2(u[k + 2], u[k + 3]), isc2, nm2);
            a = make_float2(ex2(a.x), ex2(a.y));
            b = make_float2(ex2(b.x), ex2(b.y));
            l0 = add2(l0, a);
            l1 = add2(l1, b);
            a = mul2(a, make_float2(f.x, f.y));
            b = mul2(b, make_float2(f.z, f.w));
            hi[2 * c] = pack_half2(a.x, a.y);
            hi[2 * c + 1] = pack_half2(b.x, b.y);
            if constexpr (SPLIT) {
              const __half2 ha = *reinterpret_cast<const __half2*>(&hi[2 * c]);
              const __half2 hb = *reinterpret_cast<const __half2*>(&hi[2 * c + 1]);
              lo[2 * c] = pack_half2(a.x - __low2float(ha), a.y - __high2float(ha));
              lo[2 * c + 1] = pack_half2(b.x - __low2float(hb), b.y - __high2float(hb));
            }
          }
          tmem_st32(ts + 32 * half, hi);
          if constexpr (SPLIT) tmem_st32(ts + 64 + 32 * half, lo);
        }
        l += (l0.x + l0.y) + (l1.x + l1.y);
        tmem_wait_st();
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.p_ready[s]);
    }
    if (n > 0) {  // this stream's record of the segment
      if (!wait_warp(sm, &sm.o_full[s], segs & 1)) return;
      ++segs;
      if (active) {
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t o[32];
          tmem_ld32(to + 32 * c, o);
          tmem_wait_ld();
          if (valid) {
#pragma unroll
            for (int e = 0; e < 32; e += 8) st_global_v8(rec_o + 32 * c + e, o + e);
          }
        }
        if (valid) *rec_ml = make_float2(m, l);
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.o_free[s]);
    }
    tile_base += tiles;
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.desc_empty[ds]);
  }
}

template <int BV, bool SPLIT>
__global__ void __launch_bounds__(kPThreads, 1) prefix_main_kernel(const PrefixParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* const qbuf = smem_raw;
  uint8_t* const kbuf = qbuf + 2 * kTileBytes;
  uint8_t* const vbuf = kbuf + 2 * kTileBytes;
  MainSmem& sm = *reinterpret_cast<MainSmem*>(smem_raw + kMainTiles);
  uint8_t* const ring = smem_raw + kMainTiles + sizeof(MainSmem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  grid_dep_launch();
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.desc_full[i], 1);
      mbar_init(&sm.desc_empty[i], kDescUsers);
      mbar_init(&sm.q_full[i], 1);
      mbar_init(&sm.q_empty[i], 1);
      mbar_init(&sm.k_full[i], kUnpackWarps);
      mbar_init(&sm.k_empty[i], 1);
      mbar_init(&sm.v_full[i], kUnpackWarps);
      mbar_init(&sm.v_empty[i], 1);
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.p_ready[i], 4);
      mbar_init(&sm.o_full[i], 1);
      mbar_init(&sm.o_free[i], 4);
    }
    for (int i = 0; i < kMaxRing; ++i) {
      mbar_init(&sm.ring_full[i], 1);
      mbar_init(&sm.ring_empty[i], kUnpackWarps);
    }
    mbar_init(&sm.lut_full, 1);
    mbar_init(&sm.drain, 1);
    sm.fail = 0;
    fence_proxy_async();
    mbar_expect_tx(&sm.lut_full, KVQ_LUT_BYTES);
    bulk_g2s(sm.lut, g_plut, KVQ_LUT_BYTES, &sm.lut_full);
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&sm.tmem, 512);
    tmem_relinquish();
  }
  // operand columns and rows that no tile ever writes must be finite
  for (uint32_t i = tid; i < 4 * kTileBytes / 16; i += kPThreads)
    reinterpret_cast<uint4*>(kbuf)[i] = make_uint4(0u, 0u, 0u, 0u);
  fence_proxy_async();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem;
  grid_dep_wait();
  // registers: 256 x 184 + 256 x 72 = 512 x 128
  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
    softmax_role<SPLIT>(p, sm, tmem, warp >> 2, warp & 3, lane);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == kCopyWarp) {
      copy_role<SPLIT>(p, sm, qbuf, ring, lane);
    } else if (warp == kMmaWarp) {
      if (lane == 0) {
        mma_role<SPLIT>(p, sm, qbuf, kbuf, vbuf, tmem);
        mma_commit(&sm.drain);  // nothing of this CTA's is in flight after it
        (void)mbar_wait_bounded(&sm.drain, 0);
      }
      __syncwarp();
    } else {
      unpack_role<BV>(p, sm, kbuf, vbuf, ring, warp - kUnpackWarp0, lane);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
  if (tid == 0 && sm.fail) atomicOr(p.a.status, KVQ_FLAG_TIMEOUT);
}

// ------------------------------------------------------------------- combine
constexpr int kCombineWarps = 16;

// Running merge of records: lane holds coordinates 4 lane .. 4 lane + 3.
struct Merge {
  float m, l;
  float4 o;
};
__device__ __forceinline__ void merge_one(Merge& a, float2 ml, float4 o) {
  const float m = fmaxf(a.m, ml.x);
  if (m == -INFINITY) {
    a.l += ml.y;  // a NaN row keeps its NaN
    return;
  }
  const float wa = ex2(a.m - m), wb = ex2(ml.x - m);
  a.l = a.l * wa + ml.y * wb;
  a.o.x = a.o.x * wa + o.x * wb;
  a.o.y = a.o.y * wa + o.y * wb;
  a.o.z = a.o.z * wa + o.z * wb;
  a.o.w = a.o.w * wa + o.w * wb;
  a.m = m;
}

// CTAs whose pieces may hold tiles of a unit: the CTA of position x.
__device__ __forceinline__ int cta_of(int64_t x, int64_t total, int n) {
  int c = (int)(x * n / total);
  while (c > 0 && cut(total, c, n) > x) --c;
  while (c < n - 1 && cut(total, c + 1, n) <= x) ++c;
  return c;
}

// Adds the records of one row of a unit: CTA c's piece at incidence c + idx,
// `per` rows each; streams 0 and 1 at row and row + sub unless shared.
__device__ __forceinline__ void merge_unit(Merge& acc, const PrefixParams& p, int64_t total,
                                           int64_t start, int tiles, bool shared, int64_t idx,
                                           const float2* ml, const float* o, int per, int row,
                                           int sub, int part, int parts, int lane) {
  if (tiles == 0) return;
  const int w = shared ? kCostShared : kCostAlt;
  const int c0 = cta_of(start + kCostSeg, total, p.n_ctas);
  const int c1 = cta_of(start + kCostSeg + (int64_t)(tiles - 1) * w, total, p.n_ctas);
  constexpr int kBatch = 4;
  for (int c = c0 + part; c <= c1; c += parts * kBatch) {
    float2 m2[kBatch][2];
    float4 o2[kBatch][2];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int cc = c + i * parts;
      int n = 0;
      if (cc <= c1)
        n = tiles_before(cut(total, cc + 1, p.n_ctas), start, tiles, shared) -
            tiles_before(cut(total, cc, p.n_ctas), start, tiles, shared);
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        m2[i][s] = make_float2(-INFINITY, 0.f);
        o2[i][s] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (n > s && !(shared && s)) {
          const size_t at = (size_t)(cc + idx) * per + row + s * sub;
          m2[i][s] = ml[at];
          o2[i][s] = reinterpret_cast<const float4*>(o + at * kHeadDim)[lane];
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
#pragma unroll
      for (int s = 0; s < 2; ++s) merge_one(acc, m2[i][s], o2[i][s]);
  }
}

__global__ void __launch_bounds__(kCombineWarps * 32) prefix_combine_kernel(const PrefixParams p) {
  __shared__ Merge part_sum[kCombineWarps][32];
  __shared__ int s_g;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int b = blockIdx.x / p.a.n_kv, h = blockIdx.x - b * p.a.n_kv;
  grid_dep_launch();
  grid_dep_wait();
  if (tid == 0) {
    int g = 0, len = p.a.n_groups + 1;
    while (len > 1) {
      const int half = len >> 1;
      if (p.gstart[g + half] <= b) g += half;
      len -= half;
    }
    s_g = g < p.a.n_groups && p.gstart[g] <= b ? g : -1;
  }
  __syncthreads();
  const int g = s_g, parts = kCombineWarps / p.G;  // G <= 16
  const int head = warp / parts, part = warp % parts;
  const int64_t total = p.head->total;
  Merge acc{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
  if (head < p.G && total > 0) {
    if (g >= 0) {
      const int rr = (b - p.gstart[g]) * p.G + head;
      const Unit u = prefix_unit(p, g, h, rr / p.rows_unit);
      merge_unit(acc, p, total, u.start, u.tiles, u.shared, u.idx, p.ml_p, p.o_p, 256,
                 rr % p.rows_unit, 128, part, parts, lane);
    }
    const Unit u = suffix_unit(p, b, h);
    merge_unit(acc, p, total, u.start, u.tiles, false, u.idx, p.ml_s, p.o_s, 2 * p.G, head, p.G,
               part, parts, lane);
  }
  if (parts > 1) {
    part_sum[warp][lane] = acc;
    __syncthreads();
    if (part == 0)
      for (int i = 1; i < parts && head < p.G; ++i) {
        const Merge x = part_sum[warp + i][lane];
        merge_one(acc, make_float2(x.m, x.l), x.o);
      }
  }
  if (head >= p.G || part) return;
  // o = s . H o / (128 l): coordinates 4 lane + i, distances 1, 2 in the lane,
  // 4 .. 64 across lanes
  float y[4];
  y[0] = acc.o.x + acc.o.y;
  y[1] = acc.o.x - acc.o.y;
  y[2] = acc.o.z + acc.o.w;
  y[3] = acc.o.z - acc.o.w;
  {
    const float a = y[0], c = y[1];
    y[0] = a + y[2];
    y[2] = a - y[2];
    y[1] = c + y[3];
    y[3] = c - y[3];
  }
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const bool upper = (lane & d) != 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x = __shfl_xor_sync(0xffffffffu, y[i], d);
      y[i] = upper ? x - y[i] : y[i] + x;
    }
  }
  const Plan& pl = p.a.plans[b][h];
  // an empty row gives 0; a NaN sum stays NaN
  const float inv = acc.l == 0.f ? 0.f : 1.f / (128.f * acc.l);
  const uint32_t sg = pl.v_sign[lane >> 3] >> (4 * (lane & 7));
#pragma unroll
  for (int i = 0; i < 4; ++i) y[i] = ((sg >> i) & 1u ? -y[i] : y[i]) * inv;
  const size_t at = ((size_t)b * p.a.n_q + h * p.G + head) * kHeadDim + 4 * lane;
  if (p.a.out_dtype == KVQ_FP32) {
    *reinterpret_cast<float4*>(static_cast<float*>(p.a.out) + at) =
        make_float4(y[0], y[1], y[2], y[3]);
  } else if (p.a.out_dtype == KVQ_FP16) {
    *reinterpret_cast<uint2*>(static_cast<__half*>(p.a.out) + at) =
        make_uint2(pack_half2(y[0], y[1]), pack_half2(y[2], y[3]));
  } else {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(y[0], y[1]), hi = __floats2bfloat162_rn(y[2], y[3]);
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.a.out) + at) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
  }
}

// ------------------------------------------------------------------ launchers
constexpr int kFallbackCtas = 256;  // CTAs when no device answers (size queries)

static int main_ctas(cudaError_t* err) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  *err = e;
  return e == cudaSuccess ? sms : kFallbackCtas;
}

size_t prefix_workspace_bytes(int batch, int n_q, int n_kv, int n_groups) {
  cudaError_t e;
  const int n = main_ctas(&e);
  if (e != cudaSuccess) (void)cudaGetLastError();
  return pfx_layout(batch, n_q, n_kv, n_groups, n).bytes;
}

template <typename K>
static cudaError_t launch_pdl(K kernel, unsigned grid, unsigned block, size_t smem,
                              const PrefixParams& p, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <int BV, bool SPLIT>
static cudaError_t launch_main(const PrefixParams& p, cudaStream_t st) {
  const size_t smem = kMainTiles + sizeof(MainSmem) + (size_t)p.ring * p.slot_bytes;
  cudaError_t e = cudaFuncSetAttribute(prefix_main_kernel<BV, SPLIT>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMaxSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl(prefix_main_kernel<BV, SPLIT>, p.n_ctas, kPThreads, smem, p, st);
}

template <bool SPLIT>
static cudaError_t launch_all(const PrefixParams& p, cudaStream_t st) {
  cudaError_t e = launch_pdl(prefix_prep_kernel<SPLIT>, 1 + p.a.batch * p.a.n_kv, kPrepThreads, 0,
                             p, st);
  if (e != cudaSuccess) return e;
  switch (p.a.bits_v) {
    case 1: e = launch_main<1, SPLIT>(p, st); break;
    case 2: e = launch_main<2, SPLIT>(p, st); break;
    case 3: e = launch_main<3, SPLIT>(p, st); break;
    case 4: e = launch_main<4, SPLIT>(p, st); break;
    case 5: e = launch_main<5, SPLIT>(p, st); break;
    case 6: e = launch_main<6, SPLIT>(p, st); break;
    case 7: e = launch_main<7, SPLIT>(p, st); break;
    case 8: e = launch_main<8, SPLIT>(p, st); break;
    default: e = cudaErrorInvalidValue;
  }
  if (e != cudaSuccess) return e;
  return launch_pdl(prefix_combine_kernel, p.a.batch * p.a.n_kv, kCombineWarps * 32, 0, p, st);
}

cudaError_t launch_prefix_decode(const PrefixArgs& a, void* ws, size_t ws_bytes, cudaStream_t st) {
  cudaError_t e;
  PrefixParams p;
  p.a = a;
  p.n_ctas = main_ctas(&e);
  if (e != cudaSuccess) return e;
  const PfxLayout w = pfx_layout(a.batch, a.n_q, a.n_kv, a.n_groups, p.n_ctas);
  if (w.bytes > ws_bytes) return cudaErrorInvalidValue;
  const bool split = a.out_dtype != KVQ_BF16;
  p.G = a.n_q / a.n_kv;
  p.tile_bytes = tile_bytes(a.bits_k, a.bits_v);
  p.rows_unit = split ? 128 : 256;
  uint8_t* const s = static_cast<uint8_t*>(ws);
  p.head = reinterpret_cast<PfxHead*>(s + w.head);
  p.gstart = reinterpret_cast<int32_t*>(s + w.gstart);
  p.gunit = reinterpret_cast<int32_t*>(s + w.gunit);
  p.gcost = reinterpret_cast<int64_t*>(s + w.gcost);
  p.scost = reinterpret_cast<int64_t*>(s + w.scost);
  p.isc_p = reinterpret_cast<float*>(s + w.isc_p);
  p.isc_s = reinterpret_cast<float*>(s + w.isc_s);
  p.q_p = s + w.q_p;
  p.q_s = s + w.q_s;
  p.ml_p = reinterpret_cast<float2*>(s + w.ml_p);
  p.ml_s = reinterpret_cast<float2*>(s + w.ml_s);
  p.o_p = reinterpret_cast<float*>(s + w.o_p);
  p.o_s = reinterpret_cast<float*>(s + w.o_s);
  p.slot_bytes = 512 * std::max(a.bits_k, a.bits_v) + 128;  // keys carry the norms; values'
                                                            // last reads run past their words
  p.ring = (int)std::min<size_t>(kMaxRing,
                                 (kMaxSmem - kMainTiles - sizeof(MainSmem)) / p.slot_bytes);
  return split ? launch_all<true>(p, st) : launch_all<false>(p, st);
}

}  // namespace kvq
