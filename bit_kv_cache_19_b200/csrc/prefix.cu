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
// the merge. Rounding: a query row is a pair of fp16 terms (hi + lo, 22 bits, two
// products); P is one term for bf16 outputs (2^-11 of each weight, an eighth of the
// output's own 2^-8) and a pair for fp16 and fp32. Only a unit of more than 128 rows,
// whose second row tile takes the low parts' room, has one term per query element: for
// bf16 queries with bf16 outputs alone. 2^-11, an eighth of what a bf16 query element
// carries already, is then relative to each product q_i k_i, so a weight is off by up
// to 2^-11 sum |q_i k_i| / sqrt(128) of itself. Measured against 64 bits, relative to
// the norm: 2.2e-3 for 64 sequences behind 131072 tokens (512 rows), of which the
// output's own rounding is 1.7e-3; pairs there would unpack the prefix twice as often.
// With pairs (28 query rows on 4 KV heads, 16 sequences) 1.65e-3, 1.64e-3 of it the
// output's; one term had 1.71e-3 and 35.3 us instead of 36.1, and for 48 sequences
// behind three documents 59.5 instead of 61.3.
// Sums in tensor memory are fp32 and drop what falls below their last bit at every
// step of 16 terms. A logit's products are therefore issued from the small ones to the
// large: low parts first, then the blocks by energy (the other way round a logit lost
// 7e-7 of itself, now 1e-7; 257 tokens, fp32 outputs: 4.8e-7 to 1.2e-6 of the norm,
// now 4e-7 to 5e-7). O loses up to 2^-23 per 16 tokens that one CTA adds up (fp32
// outputs: 4.3e-7 of the norm behind 2048 tokens, 9.3e-6 for 64 sequences behind 131072;
// eager fp32: 7.9e-7, 8.5e-6).
//
// Three launches (programmatic dependent launch between them):
//  1. prep: query rows into fp16 operand images (swizzled), the work schedule;
//  2. main: persistent, one CTA per SM. Units of work are (prefix, KV head, 256
//     query rows) and (sequence, KV head); the units' 128-token tiles form one
//     line of cost, cut evenly over the CTAs (a CTA takes a piece of one long
//     unit or many short ones), so ragged lengths need no tuning. Warp roles:
//     one warp walks the units, one streams 32-token records, 13 unpack codes into
//     fp16 tiles in shared memory, one thread issues tcgen05.mma, two warpgroups
//     run the softmax of two independent streams. A unit of more than 128 rows
//     puts one 128-row tile in each stream (both use every K/V tile); a smaller
//     one gives the streams alternate tiles. TMEM: S of both streams (P
//     overwrites it) and O of both, 512 columns.
//  3. combine: merges each row's records, undoes the value rotation.
// What bounds it: no unit is near its peak, but the chain of a tile. A stream has one
// region of 128 columns for S and P, so Q K^T, softmax and P V take turns: about 4000
// cycles per 128-token tile at few rows (a softmax of 16 rows or fewer is one warp's
// work) and 6500 to 7000 at 256 rows (exponentials and tensor cores: 2048 each at their
// peak rates). Two halves of 64 tokens would fit the region and overlap; not built.
// Measured: 64 sequences behind one prefix of 131072 tokens, 16 query heads on 2 KV
// heads, K3V3: 154 us, 452 TFLOP/s of useful products; 48 sequences over three prefixes
// (32 on 8 heads, K2V2, 14.4 MB): 59 us. There 36 % of main's issue slots and 19 % of
// the tensor pipe's cycles are used; prep and combine take about 7 us each.
#include <algorithm>
#include <atomic>
#include <cstddef>

#include "prefix.cuh"
#include "quant_dev.cuh"
#include "splitk.cuh"
#include "tcgen.cuh"

namespace kvq {

__device__ __align__(16) const uint32_t g_plut[KVQ_LUT_BYTES / 4] = KVQ_LUT_IMAGE;
static_assert(KVQ_LUT_BYTES >= 512 * 16 + 128, "placeholder source of a refused page's tile");

constexpr int kTok = 128;       // tokens of a K/V tile
constexpr int kPThreads = 768;  // 2 softmax warpgroups, 3 single warps, 13 unpack warps
constexpr int kUnpackWarps = 13;
constexpr int kWalkWarp = 8, kMmaWarp = 9, kCopyWarp = 10, kUnpackWarp0 = 11;
constexpr int kDescUsers = 8 + 2 + kUnpackWarps;  // warps that read a segment descriptor
constexpr uint32_t kPanel = 16384;                // 128 rows x 64 fp16, swizzled
constexpr uint32_t kTileBytes = 2 * kPanel;
constexpr uint32_t kQImage = 2 * kTileBytes;      // one unit's query image
constexpr int kSufRows = 16;                      // rows of a sequence's query image
constexpr uint32_t kSufImage = 2 * 2 * kSufRows * 128;  // 2 panels, hi and lo
// A query slot (one tile) holds up to 64 rows as high and low parts, the low ones
// from row 64 on; more rows take both slots, for the two parts or, above 128, for
// the two row tiles
constexpr int kSlotRows = 64;
constexpr uint32_t kSlotLow = kSlotRows * 128;
constexpr int kMaxRing = 8;  // tiles in flight
constexpr int kNormSlots = 4;
// TMEM columns
constexpr uint32_t kColS = 0, kColO = 256;
// P is kept below 2^kPTop; a softmax reference moves when a tile would pass it,
// to leave the tile's largest P at 2^kPSet
constexpr float kPTop = 15.f, kPSet = 7.f;
// cost of a segment's start and of one tile (shared: 256 rows; else <= 128), near
// the cycles measured before queries were pairs (which add 256 tensor cycles to a tile
// of few rows): 4.6k to 5.3k, 6.5k to 7k and 4k; 4 : 6 for the tiles and 5 for
// the start took 153 us instead of 150 for a 131072-token prefix
constexpr int kCostSeg = 3, kCostShared = 5, kCostAlt = 3;
constexpr int kDescs = 4;  // segments in flight

// ---------------------------------------------------------------- workspace
struct PfxHead {
  int64_t total;    // cost of all units
  int64_t suffix0;  // cost of the prefix units
  int64_t n_cuts;   // CTAs that get a piece of the cost line
  int64_t pad;
};
// A unit of work: a row tile of a prefix (group g, first sequence b) and KV head,
// or a sequence's own tokens (suffix; sequence b).
struct alignas(16) Unit {
  int64_t start, cost, idx;  // position and length on the cost line; number
  int32_t suffix, shared;
  int32_t g, b, h, rt, nrt, rows, len, tiles;
};
// Prefix rows of a sequence: unit of KV head 0 (-1: no prefix), row tiles per KV
// head, first row in the group.
struct alignas(16) PfxRow {
  int32_t unit0, nrt, row0, pad;
};
// A unit's pieces: CTAs c0 .. c1 of the cost line.
struct alignas(16) PfxUnit {
  int64_t start;
  int32_t tiles, shared, c0, c1, pad[2];
};
struct PfxLayout {
  size_t head, cuts, first, row, unit_p, unit_s, gstart, gunit, gcost, scost, isc_p, isc_s, q_p, q_s, ml_p, ml_s, o_p, o_s, bytes;
};

static size_t up256(size_t x) { return (x + 255) / 256 * 256; }

// n_ctas bounds the main grid; rows per prefix unit are 256 or 128 by the types,
// and the layout covers both (units: the 128-row count; record rows: 256).
static PfxLayout pfx_layout(int batch, int n_q, int n_kv, int n_groups, int n_ctas) {
  const int G = n_q / n_kv;
  // a group without sequences has no unit, and no more groups have any than there
  // are sequences
  const size_t units =
      (size_t)n_kv * (std::min(n_groups, batch) + ((size_t)batch * G + 127) / 128);
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
  w.cuts = take((size_t)(n_ctas + 1) * 8);
  w.first = take((size_t)n_ctas * sizeof(Unit));
  w.row = take((size_t)batch * sizeof(PfxRow));
  w.unit_p = take(units * sizeof(PfxUnit));
  w.unit_s = take((size_t)batch * n_kv * sizeof(PfxUnit));
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
  int64_t* cuts;  // [n_ctas + 1] first position of each CTA's piece
  Unit* first;      // [n_ctas] first unit of each CTA's piece
  PfxRow* row;      // [batch]
  PfxUnit *unit_p, *unit_s;
  int32_t *gstart, *gunit;
  int64_t *gcost, *scost;
  float *isc_p, *isc_s;
  uint8_t *q_p, *q_s;
  float2 *ml_p, *ml_s;
  float *o_p, *o_s;
  int ring;  // tile slots (4 records each)
  long long stall_cycles;  // test hook (> 0): the products stop after so long a wait
};

__device__ __forceinline__ int clamp_len(int32_t l, int64_t most) {
  return (int)min((int64_t)max(l, 0), most);
}
// tiles and records of a length up to 2^31 - 1
__device__ __forceinline__ int tiles_of(int len) { return len / kTok + (len % kTok != 0); }
__device__ __forceinline__ int recs_of(int len) { return len / kTile + (len % kTile != 0); }

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

// Number of a unit's tiles that start before position x of the cost line.
__device__ __forceinline__ int tiles_before(int64_t x, int64_t start, int tiles, bool shared) {
  const int64_t d = x - start - kCostSeg;
  if (d <= 0) return 0;
  if (d >= (int64_t)tiles * (shared ? kCostShared : kCostAlt)) return tiles;
  const uint32_t e = (uint32_t)d;  // tiles < 2^24
  return (int)(shared ? (e + kCostShared - 1) / kCostShared : (e + kCostAlt - 1) / kCostAlt);
}

// Unit (h, rt) of group g: rows of the group in all, tiles and length of the
// prefix, the group's position on the cost line and first unit number.
__device__ __forceinline__ Unit make_prefix_unit(const PrefixParams& p, int g, int h, int rt,
                                                 int b0, int rows, int len, int64_t gcost,
                                                 int gunit) {
  Unit u;
  u.suffix = 0;
  u.g = g;
  u.b = b0;
  u.h = h;
  u.rt = rt;
  u.len = len;
  u.tiles = tiles_of(len);
  const GroupCost c = group_cost(rows, u.tiles, p.rows_unit);
  u.nrt = c.nrt;
  u.rows = rt == c.nrt - 1 ? c.last : p.rows_unit;
  u.shared = u.rows > 128;
  u.start = gcost + h * c.block + rt * c.full;
  u.cost = rt == c.nrt - 1 ? c.lastc : c.full;
  u.idx = gunit + h * c.nrt + rt;
  return u;
}
__device__ __forceinline__ Unit make_suffix_unit(const PrefixParams& p, int b, int h, int len,
                                                 int64_t scost) {
  Unit u;
  u.suffix = 1;
  u.shared = 0;
  u.g = u.rt = u.nrt = 0;
  u.b = b;
  u.h = h;
  u.rows = p.G;
  u.len = len;
  u.tiles = tiles_of(len);
  u.cost = u.tiles > 0 ? kCostSeg + (int64_t)u.tiles * kCostAlt : 0;
  u.start = scost + h * u.cost;
  u.idx = (int64_t)b * p.a.n_kv + h;
  return u;
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
  int64_t gcost[kPfxMaxGroups + 1];
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

// Largest i in [0, n) with a[i] <= x (a ascending, a[0] <= x).
__device__ __forceinline__ int last_at(const int64_t* a, int n, int64_t x) {
  int lo = 0;
  while (n > 1) {
    const int half = n >> 1;
    if (a[lo + half] <= x) lo += half;
    n -= half;
  }
  return lo;
}

__device__ __forceinline__ void prep_schedule(const PrefixParams& p, PrepSmem& sm) {
  const int tid = threadIdx.x, n = p.a.n_groups;
  uint32_t flags = 0;
  int64_t base = 0;
  // the first lengths are on their way while the groups are summed
  int raw_len = tid < p.a.batch ? p.a.len[tid] : 0;
#pragma unroll 1
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
      sm.gcost[i] = p.gcost[i] = base + before;
      p.gstart[i] = sm.gstart[i];
      p.gunit[i] = sm.gunit[i];
    }
    base += total;
  }
  const int64_t suffix0 = base;
#pragma unroll 1
  for (int i0 = 0; i0 < p.a.batch; i0 += kPrepThreads) {
    const int i = i0 + tid;
    int64_t c = 0;
    if (i < p.a.batch) {
      const int raw = i0 ? p.a.len[i] : raw_len;
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
  }
  __syncthreads();  // the sums are read below
  // no more pieces than tiles of the dearer kind; the CTAs past them get none
  const int64_t pieces = min((int64_t)p.n_ctas, max((int64_t)1, base / kCostShared));
  if (tid == 0) p.head->n_cuts = pieces;
#pragma unroll 1
  for (int c = tid; c <= p.n_ctas; c += kPrepThreads) {
    const int64_t x = c < pieces ? base * c / pieces : base;
    p.cuts[c] = x;
    if (c >= p.n_ctas || x >= base) continue;
    if (x >= suffix0) {
      const int i = last_at(p.scost, p.a.batch, x);
      Unit u = make_suffix_unit(p, i, 0, clamp_len(p.a.len[i], p.a.max_len), p.scost[i]);
      const int h = (int)((x - u.start) / u.cost);
      u.h = h;
      u.start += h * u.cost;
      u.idx += h;
      p.first[c] = u;
    } else {
      const int i = last_at(sm.gcost, n, x);
      const int rows = (sm.gstart[i + 1] - sm.gstart[i]) * p.G;
      const int len = clamp_len(p.a.pre_len[i], p.a.max_pre);
      const GroupCost gc = group_cost(rows, tiles_of(len), p.rows_unit);
      const int64_t d = x - sm.gcost[i];
      const int h = (int)(d / gc.block);
      const int rt = (int)min((d - h * gc.block) / gc.full, (int64_t)gc.nrt - 1);
      p.first[c] = make_prefix_unit(p, i, h, rt, sm.gstart[i], rows, len, sm.gcost[i], sm.gunit[i]);
    }
  }
  if (flags) atomicOr(p.a.status, flags);
}

// One query row (a warp) as fp16 operand row `row` of the image at img (panel
// stride `panel`), its low part `lo` bytes on (0: none); isc gets 2^-sigma.
__device__ __forceinline__ void prep_row(const PrefixParams& p, const PrepSmem& sm, bool plan_ok,
                                         float* buf, int b, int head, uint8_t* img, uint32_t lo,
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
  // 2^sigma puts the row's largest element in [2^14, 2^15); 0 for a zero, inf
  // or NaN row; at most 126, so that both powers are normal
  const int ex = (int)(__float_as_uint(mx) >> 23);  // biased exponent
  const int sigma = mx > 0.f && ex < 255 ? min(14 + 127 - ex, 126) : 0;
  const float sc = __int_as_float((127 + sigma) << 23);
  if (lane == 0) *isc = __int_as_float((127 - sigma) << 23);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float x0 = v[i].x * sc, x1 = v[i].y * sc;  // rank lane + 32 i
    const uint32_t hi = pack_half2(x0, x1);
    const uint32_t at = i * panel + row * 128 + ((((uint32_t)lane >> 2) ^ (row & 7)) << 4) +
                        (lane & 3) * 4;
    *reinterpret_cast<uint32_t*>(img + at) = hi;
    if (lo) {
      const __half2 hh = *reinterpret_cast<const __half2*>(&hi);
      *reinterpret_cast<uint32_t*>(img + lo + at) =
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

__global__ void __launch_bounds__(kPrepThreads) prefix_prep_kernel(const PrefixParams p) {
  __shared__ PrepSmem sm;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // dependents only after the wait: a kernel that starts before this call ends
  // (also one of another call, behind the combine) then still finds everything
  // before this call done
  grid_dep_wait();
  grid_dep_launch();
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
  // units without tiles have no piece: the merge finds these entries
  if (tid == 0) p.unit_s[bh] = PfxUnit{0, 0, 0, 0, -1, {0, 0}};
  if (grouped && b == sm.gstart[g])
    for (int u = tid; u < (sm.gunit[g + 1] - sm.gunit[g]) / p.a.n_kv; u += kPrepThreads)
      p.unit_p[sm.gunit[g] + h * ((sm.gunit[g + 1] - sm.gunit[g]) / p.a.n_kv) + u] =
          PfxUnit{0, 0, 0, 0, -1, {0, 0}};
  if (h == 0 && tid == 0) {
    const int rows = grouped ? (sm.gstart[g + 1] - sm.gstart[g]) * p.G : 0;
    p.row[b] = PfxRow{grouped ? sm.gunit[g] : -1, (rows + p.rows_unit - 1) / p.rows_unit,
                      grouped ? (b - sm.gstart[g]) * p.G : 0, 0};
  }
  uint32_t sign[4] = {0u, 0u, 0u, 0u};
  const Plan* held = nullptr;
  bool ok = false;
  // image 0: the sequence's own part; 1: the prefix part
#pragma unroll 1
  for (int part = 0; part < (grouped ? 2 : 1); ++part) {
    const Plan* const src = p.a.plans[part ? sm.gstart[g] : b] + h;
    if (src != held) {
      ok = load_plan(p, sm, src);
      held = src;
    }
    // records of both parts are merged before the rotation is undone
    bool same = true;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (part) same &= sign[i] == sm.plan.v_sign[i];
      sign[i] = sm.plan.v_sign[i];
    }
    if (!same && tid == 0) atomicOr(p.a.status, KVQ_FLAG_BAD_PLAN);
    const int rows = part ? (sm.gstart[g + 1] - sm.gstart[g]) * p.G : 0;
    const int nrt = (rows + p.rows_unit - 1) / p.rows_unit;
#pragma unroll 1
    for (int i = warp; i < p.G; i += kPrepThreads / 32) {
      const int rr = (b - sm.gstart[g]) * p.G + i, rt = rr / p.rows_unit, r = rr % p.rows_unit;
      uint8_t* img = p.q_s + (size_t)bh * kSufImage;
      uint32_t lo = kSufImage / 2;
      if (part) {
        img = p.q_p + (size_t)(sm.gunit[g] + h * nrt + rt) * kQImage;
        img += (r >> 7) * kTileBytes;
        lo = min(rows - rt * p.rows_unit, p.rows_unit) > 128 ? 0 : kTileBytes;
      }
      prep_row(p, sm, ok, sm.row[warp], b, h * p.G + i, img, lo,
               part ? kPanel : kSufRows * 128, part ? r & 127 : i,
               (part ? p.isc_p : p.isc_s) + (size_t)b * p.a.n_q + h * p.G + i, lane);
    }
  }
}

// ---------------------------------------------------------------------- main
struct alignas(16) Desc {  // one segment: a run of tiles of one unit
  Plan plan;               // 16-byte aligned (bulk copy)
  float2* ml;
  float* o;
  const float* isc;
  unsigned long long base[32];  // page bases of the first 32 records (0: refused)
  int suffix, row;              // cache map and its row
  int par;  // stream of the segment's first item
  int stop, shared, rows, tiles, tile0, len, b0, row0, h, qslot, sub;
};

struct alignas(128) MainSmem {
  uint8_t lut[KVQ_LUT_BYTES];
  Desc desc[kDescs];
  alignas(16) float nk[kNormSlots][kTok];
  alignas(16) float nv[kNormSlots][kTok];
  int lg[kNormSlots][4];  // per record: the value norms are below 2^lg
  unsigned long long desc_ready[kDescs], desc_full[kDescs], desc_empty[kDescs];
  unsigned long long ring_full[kMaxRing], ring_empty[kMaxRing];
  unsigned long long q_full[2], q_empty[2], k_full[2], k_empty[2], v_full, v_empty;
  unsigned long long s_full[2], p_ready[2], o_full[2], o_free[2], lut_full, drain;
  unsigned long long stall;  // nothing arrives on it
  uint32_t tmem;
  int fail;
};
constexpr size_t kMainTiles = 5 * (size_t)kTileBytes;  // Q x 2, K x 2, V
constexpr size_t kMaxSmem = 227 * 1024;
static_assert(offsetof(MainSmem, desc) % 16 == 0 && sizeof(Desc) % 16 == 0, "bulk destinations");

// Bounded wait that also gives up once another role has: the role then leaves
// its loop, and the CTA drains and ends with the TIMEOUT flag.
__device__ __forceinline__ bool wait_on(MainSmem& sm, unsigned long long* bar, uint32_t phase) {
  if (mbar_try_wait(bar, phase)) return true;
  const uint32_t t0 = (uint32_t)clock();
  while (!mbar_try_wait(bar, phase)) {
    if ((uint32_t)clock() - t0 > (uint32_t)kWaitCycles || *(volatile int*)&sm.fail) {
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

// Position in the ring of tile slots and its phase.
struct RingPos {
  uint32_t slot, phase;
  __device__ __forceinline__ void next(uint32_t ring) {
    if (++slot == ring) {
      slot = 0;
      phase ^= 1u;
    }
  }
};

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

// What a lane needs to unpack one half step (<= 4 blocks of width W) of a
// record: lane (g, c) = (lane / 4, lane mod 4) takes block c, tokens g + 8 i,
// i < 4, whose four 2W-bit fields are contiguous.
struct KeyStep {
  uint32_t src;   // byte offset of its first word in the record's key words
  uint32_t shw;   // first bit in that word | W << 8
  uint32_t dst;   // byte offset of token g's pair in the K tile, bit 31: no block
};
__device__ __forceinline__ KeyStep key_step(const Plan& pl, int hs, int lane) {
  const int g = lane >> 2, c = lane & 3;
  const int W = pl.hs_width[hs], r0 = pl.hs_rank0[hs], nb = pl.hs_count[hs];
  const int cc = min(c, nb - 1), rank = r0 + cc;
  KeyStep k;
  k.src = 4u * (uint32_t)(pl.seg_off[r0] + 2 * W * cc + ((W * g) >> 2));
  k.shw = ((uint32_t)(8 * W * g) & 31u) | (uint32_t)W << 8;
  k.dst = (uint32_t)(rank >> 5) * kPanel + (uint32_t)g * 128u +
          ((((uint32_t)rank & 31u) >> 2 ^ (uint32_t)g) << 4) + (uint32_t)(rank & 3) * 4u;
  if (c >= nb) k.dst |= 0x80000000u;
  return k;
}

// Least e with norm < 2^e (a stored norm: fp16, >= 0). 0 counts as 2^-64: such a
// token adds nothing to O, so that any reference suits it as long as its weight,
// below 2^(kPTop + 64), and the sum of 2^31 of them stay finite.
__device__ __forceinline__ int norm_exp(float norm) {
  return max((int)(__float_as_uint(norm) >> 23) - 126, -64);
}

// One half step of the four records whose key words are at w, into the K tile
// at dst (32 rows each). The records are independent lookup chains, which hides their latency; a tile's missing
// records repeat earlier ones (their positions are masked in the softmax).
__device__ __forceinline__ void unpack_keys(const KeyStep& k, const uint8_t* lut,
                                            const uint8_t* const (&w)[4], uint8_t* dst, int lane) {
  const uint32_t sh = k.shw & 31u, W = k.shw >> 8, w2 = 2u * W, mask = (1u << w2) - 1u;
  const bool store = !(k.dst >> 31);
  uint8_t* const to = dst + (k.dst & 0x7FFFFFFFu);
  if (W <= 3) {  // pair table replicated per lane, at most 24 bits
    const uint32_t lb = (uint32_t)lane * 4u | (W == 1 ? 0x4000u : W == 2 ? 0x2000u : 0u);
    const uint32_t m7 = mask << 7;
    uint32_t v[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const uint32_t* a = reinterpret_cast<const uint32_t*>(w[r] + k.src);
      v[r] = funnel_r(a[0], a[1], sh) << 7;
    }
    // every lookup before any store: the compiler cannot tell that the tile and
    // the table do not overlap, and would hold each store's later lookups back
    uint32_t x[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        x[i][r] = *reinterpret_cast<const uint32_t*>(lut + ((v[r] & m7) | lb));
        v[r] >>= w2;  // what falls below bit 7 is masked
      }
    if (store) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          *reinterpret_cast<uint32_t*>(to + r * 4096 + i * 1024) = x[i][r];
    }
    return;
  }
  if (W <= 5) {  // one pair table, at most 40 bits
    const uint8_t* tab = lut + (W == 4 ? 0x2800u : 0x2C00u);
    uint32_t lo[4], hi[4], x[4][4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const uint32_t* a = reinterpret_cast<const uint32_t*>(w[r] + k.src);
      const uint32_t a1 = a[1];
      lo[r] = funnel_r(a[0], a1, sh);
      hi[r] = funnel_r(a1, a[2], sh);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        x[i][r] = *reinterpret_cast<const uint32_t*>(
            tab + 4u * (funnel_r(lo[r], hi[r], w2 * i) & mask));
    if (store) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          *reinterpret_cast<uint32_t*>(to + r * 4096 + i * 1024) = x[i][r];
    }
    return;
  }
  // wider: two single-code lookups
  const uint8_t* tab = lut + 0x3C00u + 2u * (uint32_t)((1 << W) - 2);
  const uint32_t m1 = mask >> W;
#pragma unroll 1
  for (int r = 0; r < 4; ++r) {
    const uint32_t* a = reinterpret_cast<const uint32_t*>(
        (r == 0 ? w[0] : r == 1 ? w[1] : r == 2 ? w[2] : w[3]) + k.src);
    const uint32_t a1 = a[1];
    const unsigned long long v =
        ((unsigned long long)funnel_r(a1, a[2], sh) << 32) | funnel_r(a[0], a1, sh);
    uint32_t x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t f = (uint32_t)(v >> (w2 * i));
      x[i] = *reinterpret_cast<const uint16_t*>(tab + 2u * (f & m1)) |
             ((uint32_t)*reinterpret_cast<const uint16_t*>(tab + 2u * ((f >> W) & m1)) << 16);
    }
    if (store) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<uint32_t*>(to + r * 4096 + i * 1024) = x[i];
    }
  }
}

// The BV words of one rotated coordinate of a record (32 tokens).
template <int BV>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[BV + 1]) {
  if constexpr (BV % 4 == 0) {
#pragma unroll
    for (int i = 0; i < BV / 4; ++i) {
      const uint4 x = reinterpret_cast<const uint4*>(p)[i];
      w[4 * i] = x.x;
      w[4 * i + 1] = x.y;
      w[4 * i + 2] = x.z;
      w[4 * i + 3] = x.w;
    }
  } else if constexpr (BV % 2 == 0) {
#pragma unroll
    for (int i = 0; i < BV / 2; ++i) {
      const uint2 x = reinterpret_cast<const uint2*>(p)[i];
      w[2 * i] = x.x;
      w[2 * i + 1] = x.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < BV; ++i) w[i] = reinterpret_cast<const uint32_t*>(p)[i];
  }
  w[BV] = 0u;
}

// 32 tokens of one rotated value coordinate (a lane's row of the V tile) as
// fp16: the pair of tokens 8 i + 2 c + (0, 1) sits at bit (8 c + 2 i) BV, so
// the 16-byte chunk of tokens 8 i .. 8 i + 7 takes its four pairs from the
// four quarters of the words. Chunk i goes to dst + ((chunk0 + i) ^ sw) * 16.
template <int BV>
__device__ __forceinline__ void unpack_values(const uint8_t* lut, const uint8_t* src,
                                              uint32_t lane4, uint8_t* dst, uint32_t chunk0,
                                              uint32_t sw) {
  uint32_t w[BV + 1];
  load_words<BV>(src, w);
  constexpr uint32_t mask = (1u << (2 * BV)) - 1u;
  uint32_t x[4][4];  // every lookup before any store, as in unpack_keys
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int o = (8 * c + 2 * i) * BV, k = o >> 5, s = o & 31;
      const bool spill = s + 2 * BV > 32;
      if constexpr (BV <= 3) {  // table entries are 128 bytes apart, one copy per lane
        const uint32_t lb = lane4 | (BV == 1 ? 0x4000u : BV == 2 ? 0x2000u : 0u);
        const uint32_t v = spill ? funnel_r(w[k], w[k + 1], (s - 7) & 31)
                           : s >= 7 ? w[k] >> ((s - 7) & 31) : w[k] << ((7 - s) & 31);
        x[i][c] = *reinterpret_cast<const uint32_t*>(lut + ((v & (mask << 7)) | lb));
      } else {
        const uint32_t v = spill ? funnel_r(w[k], w[k + 1], s) : w[k] >> s;
        if constexpr (BV <= 5) {
          x[i][c] = *reinterpret_cast<const uint32_t*>(lut + (BV == 4 ? 0x2800u : 0x2C00u) +
                                                       4u * (v & mask));
        } else {
          const uint8_t* tab = lut + 0x3C00u + 2u * (uint32_t)((1 << BV) - 2);
          constexpr uint32_t m1 = (1u << BV) - 1u;
          x[i][c] =
              *reinterpret_cast<const uint16_t*>(tab + 2u * (v & m1)) |
              ((uint32_t)*reinterpret_cast<const uint16_t*>(tab + 2u * ((v >> BV) & m1)) << 16);
        }
      }
    }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    *reinterpret_cast<uint4*>(dst + (((chunk0 + i) ^ sw) << 4)) =
        make_uint4(x[i][0], x[i][1], x[i][2], x[i][3]);
}

// ---- the roles of the main kernel

// The unit with a cost that follows u on the cost line (there is one).
__device__ __forceinline__ Unit next_unit(const PrefixParams& p, const Unit& u, int64_t suffix0,
                                          int lane) {
  const int64_t x = u.start + u.cost;
  int i = u.suffix ? u.b : u.g, h = u.h, rt = 0;
  const bool suffix = x >= suffix0;
  if (!u.suffix && !suffix && u.rt + 1 < u.nrt) {
    rt = u.rt + 1;
  } else if (u.suffix != (int)suffix || ++h == p.a.n_kv) {
    h = 0;
    i = warp_last_le(suffix ? p.scost : p.gcost, suffix ? p.a.batch : p.a.n_groups, x, lane);
  }
  if (suffix)
    return make_suffix_unit(p, i, h, clamp_len(p.a.len[i], p.a.max_len), p.scost[i]);
  return make_prefix_unit(p, i, h, rt, p.gstart[i], (p.gstart[i + 1] - p.gstart[i]) * p.G,
                          clamp_len(p.a.pre_len[i], p.a.max_pre), p.gcost[i], p.gunit[i]);
}

// Walks the CTA's piece of the cost line: one descriptor, plan and query image
// per segment, ahead of the other roles.
__device__ __forceinline__ void walk_role(const PrefixParams& p, MainSmem& sm, uint8_t* qbuf,
                                          int lane) {
  const int64_t suffix0 = p.head->suffix0;
  const int n_cuts = (int)p.head->n_cuts;
  const int64_t x0 = p.cuts[blockIdx.x], x1 = p.cuts[blockIdx.x + 1];
  Unit u = p.first[blockIdx.x];  // of a CTA without a piece: not used
  uint32_t seg = 0;                // segments
  uint32_t items = 0;              // tiles of one stream so far
  uint32_t quse[2] = {0u, 0u};     // segments that used each query slot
  int qnext = 0;
  bool ok = true;
  bool more = x0 < x1;
#pragma unroll 1
  while (ok && more) {
    const int t0 = tiles_before(x0, u.start, u.tiles, u.shared);
    const int t1 = tiles_before(x1, u.start, u.tiles, u.shared);
    more = u.start + u.cost < x1;
    if (t0 >= t1) {
      if (more) u = next_unit(p, u, suffix0, lane);
      continue;
    }
    const int row = u.suffix ? u.b : u.g, n_rec = recs_of(u.len);
    const Plan* const plan = p.a.plans[u.b] + u.h;
    unsigned long long base = 0;
    if (4 * t0 + lane < n_rec)
      base = (unsigned long long)(uintptr_t)page_base(u.suffix ? p.a.own : p.a.pre, row,
                                                      4 * t0 + lane);
    const uint32_t ds = seg % kDescs;
    ok = wait_warp(sm, &sm.desc_empty[ds], ((seg / kDescs) & 1) ^ 1);
    if (!ok) break;
    const bool both = u.rows > kSlotRows;
    const int qs = both ? 0 : qnext;
    Desc& d = sm.desc[ds];
    d.base[lane] = base;
    __syncwarp();
    if (lane == 0) {
      const size_t inc = (size_t)blockIdx.x + (size_t)u.idx;
      d.ml = u.suffix ? p.ml_s + inc * 2 * p.G : p.ml_p + inc * 256;
      d.o = u.suffix ? p.o_s + inc * 2 * p.G * kHeadDim : p.o_p + inc * 256 * kHeadDim;
      d.isc = u.suffix ? p.isc_s : p.isc_p;
      d.suffix = u.suffix;
      d.row = row;
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
      d.par = (int)(items & 1);
      mbar_arrive(&sm.desc_ready[ds]);
      mbar_expect_tx(&sm.desc_full[ds], KVQ_PLAN_BYTES);
      bulk_g2s(&d.plan, plan, KVQ_PLAN_BYTES, &sm.desc_full[ds]);
    }
    __syncwarp();
    ++seg;
    items += (t1 - t0) << (u.shared ? 1 : 0);
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
      const int s = both ? i : qs;
      if (both || i == 0) {
        ok = wait_warp(sm, &sm.q_empty[s], (quse[0] * (s == 0) + quse[1] * (s == 1)) & 1 ^ 1);
        if (!ok) break;
        quse[0] += s == 0;
        quse[1] += s == 1;
      }
      // the row tile of stream i, or the high or low parts of all rows
      const int rows = u.shared ? min(128, u.rows - 128 * i) : u.rows;
      const uint32_t bytes = (uint32_t)(rows + 7) / 8 * 1024;
      if (lane == 0) {
        const uint8_t* src = u.suffix ? p.q_s + (size_t)u.idx * kSufImage + i * (kSufImage / 2)
                                      : p.q_p + (size_t)u.idx * kQImage + i * kTileBytes;
        const uint32_t panel = u.suffix ? kSufRows * 128 : kPanel;
        uint8_t* const dst = qbuf + s * kTileBytes + (both ? 0 : i * kSlotLow);
        if (both || i == 0) mbar_expect_tx(&sm.q_full[s], (both ? 2 : 4) * bytes);
        bulk_g2s(dst, src, bytes, &sm.q_full[s]);
        bulk_g2s(dst + kPanel, src + panel, bytes, &sm.q_full[s]);
      }
      __syncwarp();
    }
    if (!both) qnext ^= 1;
    if (t0 == 0) {  // the unit starts here: where its pieces lie, for the merge
      const int w = u.shared ? kCostShared : kCostAlt;
      const int c1 = warp_last_le(p.cuts, n_cuts,
                                  u.start + kCostSeg + (int64_t)(u.tiles - 1) * w, lane);
      if (lane == 0)
        (u.suffix ? p.unit_s : p.unit_p)[u.idx] =
            PfxUnit{u.start, u.tiles, u.shared, (int)blockIdx.x, c1, {0, 0}};
    }
    if (more) u = next_unit(p, u, suffix0, lane);
  }
  if (ok) {  // the end of the CTA's work
    const uint32_t ds = seg % kDescs;
    ok = wait_warp(sm, &sm.desc_empty[ds], ((seg / kDescs) & 1) ^ 1);
    if (ok && lane == 0) {
      sm.desc[ds].stop = 1;
      mbar_arrive(&sm.desc_ready[ds]);
      mbar_arrive(&sm.desc_full[ds]);
    }
  }
  // the copies land before the CTA ends, also when their readers have given up (the
  // end's descriptor took the slot of the fourth last segment, whose readers are done)
  if (quse[0]) (void)mbar_wait_bounded(&sm.q_full[0], (quse[0] - 1) & 1);
  if (quse[1]) (void)mbar_wait_bounded(&sm.q_full[1], (quse[1] - 1) & 1);
  for (uint32_t i = 1; i <= (ok ? kDescs - 1 : kDescs) && i <= seg; ++i)
    (void)mbar_wait_bounded(&sm.desc_full[(seg - i) % kDescs], ((seg - i) / kDescs) & 1);
}

// Streams the segments' records into the ring, a tile (up to four records, one
// bulk copy each) per slot.
__device__ __forceinline__ void copy_role(const PrefixParams& p, MainSmem& sm, uint8_t* ring,
                                          int lane) {
  const uint32_t n_ring = p.ring, tbytes = p.tile_bytes;
  RingPos rp{0u, 0u};
  uint32_t issued = 0;  // slots that copies have been issued to
  bool ok = true;
  for (uint32_t seg = 0; ok; ++seg) {
    const uint32_t ds = seg % kDescs;
    ok = wait_warp(sm, &sm.desc_ready[ds], (seg / kDescs) & 1);
    const Desc& d = sm.desc[ds];
    if (!ok || d.stop) break;
    const int tiles = d.tiles, n_rec = recs_of(d.len), row = d.row, h = d.h;
    const int rec0 = 4 * d.tile0;
    const bool suffix = d.suffix;
    const int mask = suffix ? page_mask(p.a.own) : page_mask(p.a.pre);
    const size_t rec_step = (size_t)p.a.n_kv * tbytes;
    // lane: the source of record lane of each run of 32 (8 tiles); the pages of
    // the next run are looked up a run ahead
    auto page_of = [&](int rec) -> unsigned long long {
      return rec < n_rec ? (unsigned long long)(uintptr_t)page_base(
                               suffix ? p.a.own : p.a.pre, row, rec) : 0ull;
    };
    auto source = [&](unsigned long long base, int rec) -> unsigned long long {
      if (rec >= n_rec) return 0ull;
      if (base && !(base & 15)) return base + (size_t)(rec & mask) * rec_step + (size_t)h * tbytes;
      // refused: placeholder bytes are streamed, the output is flagged
      atomicOr(p.a.status, base ? KVQ_FLAG_BAD_PLAN : KVQ_FLAG_BAD_PAGE);
      return (unsigned long long)(uintptr_t)g_plut;
    };
    unsigned long long src = source(d.base[lane], rec0 + lane), next = 0;
#pragma unroll 1
    for (int t = 0; t < tiles; ++t) {
      if ((t & 7) == 0) {
        if (t) src = source(next, rec0 + 4 * t + lane);
        next = t + 8 < tiles ? page_of(rec0 + 4 * (t + 8) + lane) : 0ull;
      }
      const int n = min(4, n_rec - rec0 - 4 * t);
      ok = wait_warp(sm, &sm.ring_empty[rp.slot], rp.phase ^ 1);
      if (!ok) break;
      uint8_t* const dst = ring + rp.slot * 4 * tbytes;
      if (lane == 0) mbar_expect_tx(&sm.ring_full[rp.slot], (uint32_t)n * tbytes);
      __syncwarp();
#pragma unroll 1
      for (int i = 0; i < n; ++i) {
        const unsigned long long a = __shfl_sync(0xffffffffu, src, (4 * (t & 7) + i) & 31);
        if (lane == 0)
          bulk_g2s(dst + i * tbytes, reinterpret_cast<const void*>((uintptr_t)a), tbytes,
                   &sm.ring_full[rp.slot]);
      }
      rp.next(n_ring);
      issued = min(issued + 1, n_ring);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.desc_empty[ds]);
  }
  // the copies land before the CTA ends, also when their readers have given up: the
  // last use of each slot had the ring's phase, or the one before
  for (uint32_t i = 0; i < issued; ++i)
    (void)mbar_wait_bounded(&sm.ring_full[i], i < rp.slot ? rp.phase : rp.phase ^ 1);
}

template <int BV>
__device__ __forceinline__ void unpack_role(const PrefixParams& p, MainSmem& sm, uint8_t* kbuf, uint8_t* vbuf,
                            const uint8_t* ring, int uw, int lane) {
  uint32_t seg = 0, tile_no = 0;
  const uint32_t n_ring = p.ring;
  RingPos rk{0u, 0u}, rv{0u, 0u};  // slots of the keys and of the values
  // values lag a tile behind the keys where the ring holds two tiles: V of a tile
  // is unpacked while its softmax runs, when the product before has freed the
  // V tile
  const int lag = n_ring > 1 ? 1 : 0;
  const uint32_t tbytes = p.tile_bytes;
  // not cut short when another role gives up: the copy must land before the CTA ends
  if (!__all_sync(0xffffffffu, mbar_wait_bounded(&sm.lut_full, 0))) {
    *(volatile int*)&sm.fail = 1;
    return;
  }
  for (;; ++seg) {
    const uint32_t ds = seg % kDescs;
    if (!wait_warp(sm, &sm.desc_full[ds], (seg / kDescs) & 1)) return;
    const Desc& d = sm.desc[ds];
    if (d.stop) return;
    const Plan& pl = d.plan;
    const bool plan_ok = pl.magic == KVQ_PLAN_MAGIC && pl.bits_k == p.a.bits_k &&
                         pl.bits_v == BV && plan_sched_ok(pl, lane);
    if (!plan_ok && uw == 0 && lane == 0) atomicOr(p.a.status, KVQ_FLAG_BAD_PLAN);
    const int n_half = plan_ok ? pl.n_half : 0;
    // half steps: the widest (slowest) ones first, one to each warp; the rest, the
    // narrowest, to the last warps, and the values' odd tasks to the first
    const int hs1 = 2 * kUnpackWarps - 1 - uw;
    const KeyStep k0 = key_step(pl, uw < n_half ? uw : 0, lane);
    const KeyStep k1 = key_step(pl, hs1 < n_half ? hs1 : 0, lane);
    const int n_steps = (uw < n_half) + (hs1 < n_half);
    const int n_rec = recs_of(d.len), key_bytes = 512 * p.a.bits_k;
    const int norm_off = key_bytes + 512 * BV;
    const int me = uw >= 3 && uw < 7 ? uw - 3 : 4;  // a record's norms, or none
    const int tiles = d.tiles, tile0 = d.tile0, len = d.len;
#pragma unroll 1
    for (int t = 0; t < tiles + lag; ++t) {
      if (t < tiles) {  // ---- keys of tile t
        const uint32_t no = tile_no + t, st = no & 1, ns = no % kNormSlots;
        const int rec0 = 4 * (tile0 + t), n = min(4, n_rec - rec0);  // records of the tile
        if (!wait_warp(sm, &sm.ring_full[rk.slot], rk.phase)) return;
        if (!wait_warp(sm, &sm.k_empty[st], ((no >> 1) & 1) ^ 1)) return;
        const uint8_t* const w0 = ring + rk.slot * 4 * tbytes;
        const uint8_t* w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = w0 + min(i, n - 1) * tbytes;
#pragma unroll 1
        for (int i = 0; i < n_steps; ++i)
          unpack_keys(i ? k1 : k0, sm.lut, w, kbuf + st * kTileBytes, lane);
        if (me < 4) {  // norms of record me: masked tokens 0
          const __half* nrm = reinterpret_cast<const __half*>(w0 + me * tbytes + norm_off);
          const bool in = (rec0 + me) * kTile + lane < len;
          const float kn = in ? __half2float(nrm[lane]) : 0.f;
          const float vn = in ? __half2float(nrm[kTile + lane]) : 0.f;
          sm.nk[ns][32 * me + lane] = kn;
          sm.nv[ns][32 * me + lane] = vn;
          const uint32_t mx = __reduce_max_sync(0xffffffffu, __float_as_uint(vn));
          if (lane == 0) sm.lg[ns][me] = norm_exp(__uint_as_float(mx));
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.k_full[st]);
        rk.next(n_ring);
      }
      if (t >= lag) {  // ---- values of tile t - lag: 32 coordinate rows of one record each
        const uint32_t no = tile_no + t - lag;
        const int n = min(4, n_rec - 4 * (tile0 + t - lag));
        if (!wait_warp(sm, &sm.v_empty, (no & 1) ^ 1)) return;
        const uint8_t* const w0 = ring + rv.slot * 4 * tbytes + key_bytes;
#pragma unroll 1
        for (int j = uw; j < 4 * n; j += kUnpackWarps) {
          const int rec = j >> 2, row = 32 * (j & 3) + lane;
          unpack_values<BV>(sm.lut, w0 + rec * tbytes + 4 * BV * row, (uint32_t)lane * 4u,
                            vbuf + (rec >> 1) * kPanel + row * 128, 4u * (rec & 1),
                            (uint32_t)lane & 7u);
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&sm.ring_empty[rv.slot]);
          mbar_arrive(&sm.v_full);
        }
        rv.next(n_ring);
      }
    }
    tile_no += tiles;
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.desc_empty[ds]);
  }
}

// D fp32, A and B fp16 K-major, M = N = 128.
constexpr uint32_t kIdesc = (1u << 4) | (16u << 17) | (8u << 24);

// A segment's items, in order (item = one stream's tile: of a shared segment the
// two row tiles of each tile in turn, else its tiles).
struct ItemCursor {
  uint32_t seg, j, n, tile0;  // segment, next item, items, number of its first tile
  bool shared;
  __device__ __forceinline__ uint32_t tile() const { return tile0 + (shared ? j >> 1 : j); }
  __device__ __forceinline__ bool first_use() const { return !shared || !(j & 1); }
  __device__ __forceinline__ bool last_use() const { return !shared || (j & 1); }
  __device__ __forceinline__ void load(const Desc& d) {
    tile0 += shared ? n >> 1 : n;
    shared = d.shared;
    n = (uint32_t)d.tiles << (shared ? 1 : 0);
    j = 0;
  }
};

// Step k: P V of item k - 2, then Q K of item k, through all segments in one
// sequence; item k belongs to stream k mod 2, so a stream starts a segment as soon
// as it has finished its part of the one before.
template <bool SPLIT>
__device__ __forceinline__ void mma_role(const PrefixParams& p, MainSmem& sm, const uint8_t* qbuf,
                         const uint8_t* kbuf, const uint8_t* vbuf, uint32_t tmem) {
  const bool elected = elect_one();
  // phases: bit s of quse (query slot s), items and segs (stream s)
  uint32_t quse = 0, items = 0, segs = 0;
  // low words of the operand descriptors (addresses in units of 16 bytes)
  const uint32_t qd = desc_lo(smem_addr(qbuf)), kd = desc_lo(smem_addr(kbuf)),
                 vd = desc_lo(smem_addr(vbuf));
  constexpr uint32_t kTileD = kTileBytes >> 4, kPanelD = kPanel >> 4;
  ItemCursor q{0u, 0u, 0u, 0u, false}, v{0u, 0u, 0u, 0u, false};
  uint32_t ksteps = 0;
  int q0 = 0;
  bool both = false;  // the segment's queries are in both slots
  const uint32_t stall_at = p.stall_cycles > 0 ? blockIdx.x & 7 : 0xffffffffu;
  bool more = true;
#pragma unroll 1
  for (uint32_t k = 0, issued = 0, done = 0;; ++k) {
    const int s = k & 1;
    if (k == stall_at) {  // test hook: a wait that runs out
      if (!__all_sync(0xffffffffu, mbar_wait_bounded(&sm.stall, 0, p.stall_cycles)))
        *(volatile int*)&sm.fail = 1;
      return;
    }
    if (k >= 2 && done < issued) {
      if (v.j == v.n) {  // the next segment's values
        if (v.n) {
          if (elected) mbar_arrive(&sm.desc_empty[v.seg % kDescs]);
          ++v.seg;
        }
        v.load(sm.desc[v.seg % kDescs]);
      }
      const uint32_t no = v.tile();
      if (!wait_warp(sm, &sm.p_ready[s], items >> s & 1)) return;
      items ^= 1u << s;
      if (v.first_use())
        if (!wait_warp(sm, &sm.v_full, no & 1)) return;
      const bool first = v.j < 2;
      if (first) {  // the previous segment's O of this stream has been read
        if (!wait_warp(sm, &sm.o_free[s], (segs >> s & 1) ^ 1)) return;
        segs ^= 1u << s;
      }
      tc_fence_after();
      if (elected) {
#pragma unroll 1
        for (int part = 0; part < (SPLIT ? 2 : 1); ++part) {
          const uint32_t a = tmem + kColS + 128 * s + 16 * part, o = tmem + kColO + 128 * s;
          if (first && part == 0) mma_ts<false>(o, a, vd, kIdesc);
          else mma_ts<true>(o, a, vd, kIdesc);
#pragma unroll
          for (uint32_t ks = 1; ks < 8; ++ks)
            mma_ts<true>(o, a + 32 * (ks >> 1) + 8 * (ks & 1),
                         vd + (ks >> 2) * kPanelD + (ks & 3) * 2, kIdesc);
        }
        if (v.last_use()) mma_commit(&sm.v_empty);
        if (v.j + 2 >= v.n) mma_commit(&sm.o_full[s]);
      }
      __syncwarp();
      ++v.j;
      ++done;
    }
    if (more && q.j == q.n) {  // the next segment's queries
      if (q.n) ++q.seg;
      const uint32_t ds = q.seg % kDescs;
      if (!wait_warp(sm, &sm.desc_full[ds], (q.seg / kDescs) & 1)) return;
      const Desc& d = sm.desc[ds];
      more = !d.stop;
      if (more) {
        q.load(d);
        q0 = d.qslot;
        both = d.rows > kSlotRows;
        ksteps = (min(max(d.plan.n_ranks, 1), 64) + 7) / 8;
#pragma unroll 1
        for (int i = q0; i < q0 + (both ? 2 : 1); ++i) {
          if (!wait_warp(sm, &sm.q_full[i], quse >> i & 1)) return;
          quse ^= 1u << i;
        }
      }
    }
    if (more) {
      const uint32_t no = q.tile(), st = no & 1;
      if (q.first_use())
        if (!wait_warp(sm, &sm.k_full[st], (no >> 1) & 1)) return;
      tc_fence_after();
      if (elected) {
        const uint32_t d = tmem + kColS + 128 * s, kt = kd + st * kTileD;
        // every step drops what falls below the sum's last bit, so the small terms come
        // first: low parts, then the narrow blocks (a plan's order is widest first)
        const uint32_t last = ksteps - 1, ol = (last >> 2) * kPanelD + (last & 3) * 2;
#pragma unroll 1
        for (int part = q.shared ? 0 : 1; part >= 0; --part) {
          const uint32_t a = qd + (both ? (q.shared ? q.j & 1 : part) * kTileD
                                        : q0 * kTileD + part * (kSlotLow >> 4));
          if (part || q.shared) mma_ss<false>(d, a + ol, kt + ol, kIdesc);
          else mma_ss<true>(d, a + ol, kt + ol, kIdesc);
#pragma unroll
          for (int ks = 6; ks >= 0; --ks)
            if (ks < (int)last) {
              const uint32_t o = (ks >> 2) * kPanelD + (ks & 3) * 2;
              mma_ss<true>(d, a + o, kt + o, kIdesc);
            }
        }
        mma_commit(&sm.s_full[s]);
        if (q.last_use()) mma_commit(&sm.k_empty[st]);
        if (q.j + 1 == q.n) {  // the segment's query rows are no longer needed
          mma_commit(&sm.q_empty[q0]);
          if (both) mma_commit(&sm.q_empty[1]);
        }
      }
      __syncwarp();
      ++q.j;
      ++issued;
    } else if (done == issued) {
      return;
    }
  }
}

template <int N>
struct IntC {
  __device__ constexpr operator int() const { return N; }
};

// Softmax of stream s (one warpgroup, 32 rows per warp). A chunk of 32 columns
// (one record) is held like a matrix fragment: lane (g, q) = (lane / 4, lane mod
// 4) has rows g + 8 k (k < 4) and columns 8 j + 2 q + (0, 1) (j < 4), so that a
// lane loads 8 key and 8 value norms per chunk; with a row per lane it would load
// 32 of each, and those loads alone took 2,000 shared-memory cycles per tile of
// 256 rows.
template <bool SPLIT>
__device__ __forceinline__ void softmax_role(const PrefixParams& p, MainSmem& sm, uint32_t tmem,
                                             int s, int wq, int lane) {
  uint32_t items = 0, segs = 0, tile_base = 0;
  const uint32_t lane_addr = (uint32_t)(32 * wq) << 16;
  const uint32_t ts = tmem + lane_addr + kColS + 128 * s, to = tmem + lane_addr + kColO + 128 * s;
  const int g = lane >> 2, q = lane & 3;
  // value of row `lane`, from the lane (lane mod 8, 0) that holds it as row 8 k + g
  auto by_row = [&](const float (&v)[4]) -> float {
    float r = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float x = __shfl_sync(0xffffffffu, v[k], (lane & 7) * 4);
      if (lane >> 3 == k) r = x;
    }
    return r;
  };
  for (uint32_t seg = 0;; ++seg) {
    const uint32_t ds = seg % kDescs;
    if (!wait_warp(sm, &sm.desc_full[ds], (seg / kDescs) & 1)) return;
    const Desc& d = sm.desc[ds];
    if (d.stop) return;
    const bool shared = d.shared;
    // the segment's items alternate between the streams from stream par on: this
    // stream has row tile f of a shared segment, else tiles f, f + 2, ...
    const int f = s ^ d.par, tiles = d.tiles, n = shared ? tiles : (tiles - f + 1) / 2;
    const int rows = shared ? min(128, d.rows - 128 * f) : d.rows;
    const bool active = 32 * wq < rows;  // the warp has rows
    float isc[4], m[4], l[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int row = 32 * wq + g + 8 * k;  // in this stream's tile
      const int rr = d.row0 + (shared ? 128 * f : 0) + min(row, rows - 1);
      isc[k] = active ? d.isc[(d.b0 + rr / p.G) * p.a.n_q + d.h * p.G + rr % p.G] : 1.f;
      // a row past the unit's has no reference to move: its numbers go nowhere
      m[k] = row < rows ? -INFINITY : INFINITY;
      l[k] = 0.f;
    }
    const int len = d.len, tile0 = d.tile0;
#pragma unroll 1
    for (int i = 0; i < n; ++i, ++items) {
      const int t = shared ? i : 2 * i + f;
      const uint32_t ns = (tile_base + t) % kNormSlots;
      if (!wait_warp(sm, &sm.s_full[s], items & 1)) return;
      if (active) {
        tc_fence_after();
        const int nvalid = len - (tile0 + t) * kTok;  // >= kTok but for the last tile
        // chunks in a loop that is not unrolled: with all 128 columns unrolled the
        // code of the roles outgrew the instruction cache. P = 2^(s - m) times the
        // value norm goes in place of the logits: the pairs of columns 32 c .. to
        // columns 32 c .. + 15 (low parts + 16 ..)
        auto chunks = [&](auto groups) {
          constexpr int K = groups;  // groups of 8 rows that hold any (1, or up to 4)
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t v[2][16];
          tmem_ld_frag(ts + 32 * c, v[0]);
          if constexpr (K > 2) tmem_ld_frag(ts + (16u << 16) + 32 * c, v[1]);
          const float2* nk2 = reinterpret_cast<const float2*>(&sm.nk[ns][32 * c + 2 * q]);
          const float2* nv2 = reinterpret_cast<const float2*>(&sm.nv[ns][32 * c + 2 * q]);
          const float lg = (float)sm.lg[ns][c];
          const float2 nk[4] = {nk2[0], nk2[4], nk2[8], nk2[12]};
          tmem_wait_ld16(v[0]);
          if constexpr (K > 2) tmem_wait_ld16(v[1]);
          float2 u[4][4];  // [row k][column group j]: logits times key norms
          bool move = false;
#pragma unroll
          for (int k = 0; k < K; ++k) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int e = 4 * j + 2 * (k & 1);
              u[k][j] = mul2(make_float2(__uint_as_float(v[k >> 1][e]),
                                         __uint_as_float(v[k >> 1][e + 1])), nk[j]);
            }
          }
          if (nvalid < 32 * c + 32) {  // the last tile: positions past the end
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                if (32 * c + 8 * j + 2 * q >= nvalid) u[k][j].x = -INFINITY;
                if (32 * c + 8 * j + 2 * q + 1 >= nvalid) u[k][j].y = -INFINITY;
              }
          }
#pragma unroll
          for (int k = 0; k < K; ++k) {
            const float a = fmaxf(fmaxf(u[k][0].x, u[k][0].y), u[k][1].x);
            const float b = fmaxf(fmaxf(u[k][1].y, u[k][2].x), u[k][2].y);
            const float top = fmaxf(fmaxf(a, b), fmaxf(u[k][3].x, u[k][3].y)) * isc[k] + lg;
            move |= 32 * wq + g + 8 * k < rows && !(top - m[k] <= kPTop);
          }
          // the reference, a whole number, moves only when a product would pass
          // 2^kPTop (or on NaN), to leave the largest product so far between
          // 2^(kPSet - 2) and 2^kPTop: O, l and this tile's earlier P are scaled by a
          // power of two. The bound above takes the chunk's largest value norm; what
          // decides is each token's own, or the reference would follow a heavy token
          // of small norm and leave the others' products below fp16's normal range
          if (nvalid > 32 * c && __any_sync(0xffffffffu, move)) {
            float alpha[4] = {1.f, 1.f, 1.f, 1.f};
            bool moved = false;
            float2 e[4];  // the value norms are below 2^e
#pragma unroll
            for (int j = 0; j < 4; ++j)
              e[j] = make_float2((float)norm_exp(nv2[4 * j].x), (float)norm_exp(nv2[4 * j].y));
#pragma unroll
            for (int k = 0; k < K; ++k) {
              float t = fmaxf(fmaf(u[k][0].x, isc[k], e[0].x), fmaf(u[k][0].y, isc[k], e[0].y));
#pragma unroll
              for (int j = 1; j < 4; ++j)
                t = fmaxf(t, fmaxf(fmaf(u[k][j].x, isc[k], e[j].x),
                                   fmaf(u[k][j].y, isc[k], e[j].y)));
              t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 1));
              t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 2));
              if (!(t - m[k] <= kPTop)) {
                const float m_new = ceilf(t) - kPSet;
                alpha[k] = ex2(m[k] - m_new);  // 0 from -inf
                l[k] *= alpha[k];
                m[k] = m_new;
                moved = true;
              }
            }
            if (__any_sync(0xffffffffu, moved)) {
              // what is read back below may have been stored by this tile's earlier
              // chunks (their P, and O and P of an earlier move): stores are
              // asynchronous, and only this wait orders a later load behind them
              tmem_wait_st();
              const float ar = by_row(alpha);
              if (i > 0) {  // O holds this segment's earlier tiles
#pragma unroll 1
                for (int k = 0; k < 16; ++k) {
                  uint32_t o[8];
                  tmem_ld8(to + 8 * k, o);
                  tmem_wait_ld8(o);
#pragma unroll
                  for (int e = 0; e < 8; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * ar);
                  tmem_st8(to + 8 * k, o);
                }
              }
              const __half2 ah = __float2half2_rn(ar);
#pragma unroll 1
              for (int k = 0; k < 4 * c; ++k) {  // columns 0 .. 31 of each earlier record
                uint32_t o[8];
                tmem_ld8(ts + 8 * k, o);
                tmem_wait_ld8(o);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  const __half2 x = __hmul2(*reinterpret_cast<const __half2*>(&o[e]), ah);
                  o[e] = *reinterpret_cast<const uint32_t*>(&x);
                }
                tmem_st8(ts + 8 * k, o);
              }
            }
          }
          uint32_t hi[2][8] = {};
          [[maybe_unused]] uint32_t lo[2][SPLIT ? 8 : 1] = {};
#pragma unroll
          for (int k = 0; k < K; ++k) {
            const float2 is = make_float2(isc[k], isc[k]), nm = make_float2(-m[k], -m[k]);
            float2 sum = make_float2(0.f, 0.f);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              float2 a = fma2(u[k][j], is, nm);
              a = make_float2(ex2(a.x), ex2(a.y));
              sum = add2(sum, a);
              a = mul2(a, nv2[4 * j]);
              const uint32_t h = pack_half2(a.x, a.y);
              hi[k >> 1][2 * j + (k & 1)] = h;
              if constexpr (SPLIT) {
                const __half2 hh = *reinterpret_cast<const __half2*>(&h);
                lo[k >> 1][2 * j + (k & 1)] =
                    pack_half2(a.x - __low2float(hh), a.y - __high2float(hh));
              }
            }
            l[k] += sum.x + sum.y;
          }
          tmem_st_frag(ts + 32 * c, hi[0]);
          if constexpr (K > 2) tmem_st_frag(ts + (16u << 16) + 32 * c, hi[1]);
          if constexpr (SPLIT) {
            tmem_st_frag(ts + 32 * c + 16, lo[0]);
            if constexpr (K > 2) tmem_st_frag(ts + (16u << 16) + 32 * c + 16, lo[1]);
          }
        }
        };
        if (rows - 32 * wq <= 8) chunks(IntC<1>{});
        else chunks(IntC<4>{});
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
        for (int k = 0; k < 4; ++k) {  // a row's sum is spread over four lanes
          l[k] += __shfl_xor_sync(0xffffffffu, l[k], 1);
          l[k] += __shfl_xor_sync(0xffffffffu, l[k], 2);
        }
        const float mr = by_row(m), lr = by_row(l);
        const int row = 32 * wq + lane;
        const size_t at = (size_t)(f * d.sub + row);
        float* const rec_o = d.o + at * kHeadDim;
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t o[32];
          tmem_ld32(to + 32 * c, o);
          tmem_wait_ld32(o);
          if (row < rows) {
#pragma unroll
            for (int e = 0; e < 32; e += 8) st_global_v8(rec_o + 32 * c + e, o + e);
          }
        }
        if (row < rows) d.ml[at] = make_float2(mr, lr);
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
      mbar_init(&sm.q_full[i], 1);
      mbar_init(&sm.q_empty[i], 1);
      mbar_init(&sm.k_full[i], kUnpackWarps);
      mbar_init(&sm.k_empty[i], 1);
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.p_ready[i], 4);
      mbar_init(&sm.o_full[i], 1);
      mbar_init(&sm.o_free[i], 4);
    }
    for (int i = 0; i < kDescs; ++i) {
      mbar_init(&sm.desc_ready[i], 1);  // the descriptor
      mbar_init(&sm.desc_full[i], 1);   // and its plan
      mbar_init(&sm.desc_empty[i], kDescUsers);
    }
    for (int i = 0; i < kMaxRing; ++i) {
      mbar_init(&sm.ring_full[i], 1);  // one expect_tx for the tile's records
      mbar_init(&sm.ring_empty[i], kUnpackWarps);
    }
    mbar_init(&sm.v_full, kUnpackWarps);
    mbar_init(&sm.v_empty, 1);
    mbar_init(&sm.lut_full, 1);
    mbar_init(&sm.drain, 1);
    mbar_init(&sm.stall, 1);
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
  for (uint32_t i = tid; i < 3 * kTileBytes / 16; i += kPThreads)
    reinterpret_cast<uint4*>(kbuf)[i] = make_uint4(0u, 0u, 0u, 0u);
  fence_proxy_async();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem;
  grid_dep_wait();
  // registers: 256 x 112 + 512 x 64 = 768 x 80
  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 112;");
    softmax_role<SPLIT>(p, sm, tmem, warp >> 2, warp & 3, lane);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    if (warp == kWalkWarp) {
      walk_role(p, sm, qbuf, lane);
    } else if (warp == kCopyWarp) {
      copy_role(p, sm, ring, lane);
    } else if (warp == kMmaWarp) {
      mma_role<SPLIT>(p, sm, qbuf, kbuf, vbuf, tmem);
      if (elect_one()) mma_commit(&sm.drain);  // nothing of this CTA's is in flight after it
      (void)mbar_wait_bounded(&sm.drain, 0);
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
// One CTA per (sequence, KV head), G x parts warps: `parts` warps share a query
// head's records and merge through shared memory. Registers are held to 64 so
// that two CTAs of 16 warps fit an SM; at 82 the 384 CTAs of a 48-sequence batch
// ran in three waves and took 20 us instead of one.
constexpr int kCombineMaxWarps = 32;
constexpr int kMaxCtas = 256;  // of the main grid

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

__global__ void __launch_bounds__(kCombineMaxWarps * 32) prefix_combine_kernel(
    const PrefixParams p, int parts) {
  extern __shared__ int64_t s_cuts[];  // [n_ctas + 1]
  __shared__ Merge part_sum[kCombineMaxWarps][32];
  __shared__ uint32_t s_list[3][2 * kMaxCtas];
  __shared__ int s_n[3];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int b = blockIdx.x / p.a.n_kv, h = blockIdx.x - b * p.a.n_kv;
  const int head = warp / parts, part = warp - head * parts;
  grid_dep_launch();
  grid_dep_wait();
  // three rounds of loads: tables; the prefix's unit; the records
  const PfxRow pr = p.row[b];
  const PfxUnit us = p.unit_s[blockIdx.x];
  const Plan* const pl = p.a.plans[b] + h;
  for (int i = tid; i <= p.n_ctas; i += blockDim.x) s_cuts[i] = p.cuts[i];
  // the prefix's units of the first and the last query head (rows of a sequence
  // may straddle two), and the suffix's
  const int ra = pr.row0 / p.rows_unit, rb = (pr.row0 + p.G - 1) / p.rows_unit;
  const int unit_a = pr.unit0 + h * pr.nrt + ra;
  PfxUnit ua{0, 0, 0, 0, -1, {0, 0}}, ub = ua;
  if (pr.unit0 >= 0) {
    ua = p.unit_p[unit_a];
    if (rb != ra) ub = p.unit_p[unit_a + 1];
  }
  const uint32_t sg = pl->v_sign[lane >> 3] >> (4 * (lane & 7));
  __syncthreads();
  // lists of their records, one warp each: (CTA c, stream s) as 2 (c + unit) + s,
  // CTA c's piece being at incidence c + unit; a shared unit's row is in one
  // stream, so its second stream's records are left out
  const int n_warps = p.G * parts;
#pragma unroll 1
  for (int l = warp; l < 3; l += n_warps) {
    const PfxUnit u = l == 0 ? ua : l == 1 ? ub : us;
    const int inc = l == 2 ? (int)blockIdx.x : unit_a + l, two = u.shared ? 0 : 1;
    int n = 0;
#pragma unroll 1
    for (int k0 = 0; k0 < (u.c1 - u.c0 + 1) << two; k0 += 32) {
      const int k = k0 + lane, c = u.c0 + (k >> two), s = k & two;
      const bool has = k < (u.c1 - u.c0 + 1) << two &&
                       tiles_before(s_cuts[c + 1], u.start, u.tiles, u.shared) -
                               tiles_before(s_cuts[c], u.start, u.tiles, u.shared) > s;
      const uint32_t got = __ballot_sync(0xffffffffu, has);
      if (has) s_list[l][n + __popc(got & ((1u << lane) - 1u))] = 2 * (c + inc) + s;
      n += __popc(got);
    }
    if (lane == 0) s_n[l] = n;
  }
  __syncthreads();
  Merge acc{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
  const int rr = pr.row0 + head, lp = rr / p.rows_unit - ra, row = rr % p.rows_unit;
  const bool shared = lp ? ub.shared : ua.shared;
  const int n_p = s_n[lp], n = n_p + s_n[2];
  constexpr int kBatch = 4;
#pragma unroll 1
  for (int k = part; k < n; k += parts * kBatch) {
    float2 m4[kBatch];
    float4 o4[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int kk = k + i * parts;
      m4[i] = make_float2(-INFINITY, 0.f);
      o4[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (kk < n) {
        const bool suf = kk >= n_p;
        const uint32_t e = suf ? s_list[2][kk - n_p] : s_list[lp][kk];
        const size_t at = suf ? (size_t)e * p.G + head
                              : (size_t)(e >> 1) * 256 + (shared ? 0 : (e & 1) * 128) + row;
        m4[i] = (suf ? p.ml_s : p.ml_p)[at];
        o4[i] = reinterpret_cast<const float4*>((suf ? p.o_s : p.o_p) + at * kHeadDim)[lane];
      }
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) merge_one(acc, m4[i], o4[i]);
  }
  if (parts > 1) {
    part_sum[warp][lane] = acc;
    __syncthreads();
    if (part) return;
    for (int i = 1; i < parts; ++i) {
      const Merge x = part_sum[warp + i][lane];
      merge_one(acc, make_float2(x.m, x.l), x.o);
    }
  }
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
  // an empty row gives 0; a NaN sum stays NaN
  const float inv = acc.l == 0.f ? 0.f : 1.f / (128.f * acc.l);
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
constexpr int kFallbackCtas = kMaxCtas;  // CTAs when no device answers (size queries)

static int main_ctas(cudaError_t* err) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  *err = e;
  return e == cudaSuccess ? std::min(sms, kMaxCtas) : kFallbackCtas;
}

size_t prefix_workspace_bytes(int batch, int n_q, int n_kv, int n_groups) {
  cudaError_t e;
  const int n = main_ctas(&e);
  if (e != cudaSuccess) (void)cudaGetLastError();
  return pfx_layout(batch, n_q, n_kv, n_groups, n).bytes;
}

template <typename K, typename... A>
static cudaError_t launch_pdl(cudaStream_t st, K kernel, unsigned grid, unsigned block, size_t smem,
                              const A&... args) {
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
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int BV, bool SPLIT>
static cudaError_t launch_main(const PrefixParams& p, cudaStream_t st) {
  const size_t smem = kMainTiles + sizeof(MainSmem) + (size_t)p.ring * 4 * p.tile_bytes;
  cudaError_t e = cudaFuncSetAttribute(prefix_main_kernel<BV, SPLIT>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMaxSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl(st, prefix_main_kernel<BV, SPLIT>, p.n_ctas, kPThreads, smem, p);
}

template <bool SPLIT>
static cudaError_t launch_all(const PrefixParams& p, cudaStream_t st) {
  cudaError_t e =
      launch_pdl(st, prefix_prep_kernel, 1 + p.a.batch * p.a.n_kv, kPrepThreads, 0, p);
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
  // warps per query head: up to 8, so many that about 32 warps per SM are at work
  // and a CTA has at most 32
  const int parts = std::max(1, std::min({8, kCombineMaxWarps / p.G,
                                          32 * p.n_ctas / (p.a.batch * p.a.n_q)}));
  return launch_pdl(st, prefix_combine_kernel, p.a.batch * p.a.n_kv, 32 * p.G * parts,
                    (size_t)(p.n_ctas + 1) * sizeof(int64_t), p, parts);
}

// Test hook: > 0 makes the warp that issues the products give up after so long a wait.
static std::atomic<long long> g_stall_cycles{0};
void set_prefix_stall(long long cycles) { g_stall_cycles.store(cycles > 0 ? cycles : 0); }

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
  // a query operand of two terms leaves no room for a second row tile: 256 rows to a
  // unit only where the queries come with bf16's 8 bits (see the top of the file)
  p.rows_unit = split || a.q_dtype != KVQ_BF16 ? 128 : 256;
  p.stall_cycles = g_stall_cycles.load();
  uint8_t* const s = static_cast<uint8_t*>(ws);
  p.head = reinterpret_cast<PfxHead*>(s + w.head);
  p.cuts = reinterpret_cast<int64_t*>(s + w.cuts);
  p.first = reinterpret_cast<Unit*>(s + w.first);
  p.row = reinterpret_cast<PfxRow*>(s + w.row);
  p.unit_p = reinterpret_cast<PfxUnit*>(s + w.unit_p);
  p.unit_s = reinterpret_cast<PfxUnit*>(s + w.unit_s);
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
  // the unpacking reads up to two words past a record's code words
  p.ring = (int)std::min<size_t>(
      kMaxRing, (kMaxSmem - kMainTiles - sizeof(MainSmem)) / (4 * (size_t)p.tile_bytes));
  return split ? launch_all<true>(p, st) : launch_all<false>(p, st);
}

}  // namespace kvq
