// What the kernels of the shared-prefix attention, and of the attention over a cache in pages
// (the same kernels, their keys fetched page by page), have in common: the decomposition into
// units, TMA loads over the caller's strides, and the tensor maps.
#pragma once
#include "internal.h"
#include "ptx.cuh"

namespace qi {
namespace pa {

constexpr int kKeys = 128;           // keys per tile
constexpr int kBox = 128 * 64 * 2;   // 128 rows x 64 dims, 128-byte swizzle (16 KB)
constexpr int kTile = 2 * kBox;      // K or V tile (32 KB)
constexpr float kRescaleLog2 = 8.0f; // rescale O only when its maximum grows by > 2^8
// Probabilities are 2^(s - m) with m the running maximum less kLift: fp16 ones lie between 2^7 and
// 2^15 times their ratio to the row's largest, so that the type's range below 1 serves the small ones
// too. Without it those below 2^-25 became zero, and thousands of such keys behind one of great
// weight and small value (a sink) left the row without its sum. The factor cancels in O / sum.
template <bool BF16>
constexpr float kLift = BF16 ? 0.f : 7.f;

// The decomposition, decided on the host from sizes alone.
struct Plan {
  int G;          // query heads per key head
  int tb;         // tokens per row block
  int nqb;        // row blocks per sequence
  int rb;         // sequences per prefix block (packed), else 1
  int npb;        // prefix blocks per key head (packed)
  int pt, ot;     // prefix tiles; own tiles at the largest own length
  int ct;         // tiles per chunk
  int nch;        // joint: chunks per unit; packed: chunks of the own keys
  int nchp;       // packed: chunks of the prefix
  int packed;
  int split;      // 1: partials and merge_partials
  int by_block;   // joint units ordered by row block, last first, before head and sequence
  int units_p;    // packed: units over the prefix (they come first)
  int units;
  int rows_p;     // rows of a prefix block's partial
  int rows_o;     // rows of a joint / own block's partial
  int few;        // blocks of at most kFewRows rows, by launch_few
  int join;       // joint units whose chunks are a cluster of CTAs and join their parts themselves
  int per;        // partials per unit
  int flow;       // a cache in pages: even pieces of all tiles, cut on the device (FlowParams); each CTA's
  int cost;       // ... of a unit beside its tiles, in 1/kLine of one
};

struct Params {
  Plan pl;
  Div d_nch, d_nchp, d_nqb, d_npb, d_tb, d_rb, d_ct;  // divisors: the plan's,
  Div d_B, d_hb, d_G, d_T, d_Hq;                      // B, Hkv B, G, T, Hq
  int B, T, Hq, Hkv, P, S, causal;
  const int* own_len;
  uint16_t* o;
  long long ob, orow, oh;  // element strides of o
  int o32;                 // o and its strides allow 32-byte stores
  float* part;             // partial O rows, 128 floats each
  float2* ml;              // (maximum in base-2 units, sum) of each partial row
  int* err;
};

// A cache in pages: no prefix, and own keys where the table says; S is the largest length.
struct PagedParams : Params {
  const int* table;  // page of key i of sequence b: table[b table_stride + (i >> page_log)]
  long long table_stride;
  const int* q_len;  // query rows of each sequence, or NULL: T
  int page_log, pages;
};
// ... whose tiles are dealt out when the kernel runs: every CTA gets the same share of all sequences' tiles
struct FlowParams : PagedParams {
  int per_slot;  // (sequence, row block) pairs to a sum
  Div d_slot;    // ... as a divisor
  Div d_pieces;  // pl.flow x the grid
  int4* rec;     // the block that each piece takes over (see Flow)
};
template <typename P>
constexpr bool kPaged = false;
template <>
constexpr bool kPaged<PagedParams> = true;
template <>
constexpr bool kPaged<FlowParams> = true;
template <typename P>
constexpr bool kFlow = false;
template <>
constexpr bool kFlow<FlowParams> = true;

struct Unit {
  int h, b0, t0;
  int tq;          // query rows of sequence b0
  int p0, pn;      // prefix tiles [p0, p0 + pn)
  int o0, on;      // own tiles of sequence b0
  int n;           // pn + on
  int len;         // own keys of sequence b0
  int rows;        // rows of the block (the MMA's other rows are ignored)
  bool clear;      // the last tile holds own rows at or past len
  long long slot;  // first partial row; of a share (FlowParams): -1 if the unit is a whole block
};

__device__ __forceinline__ int own_len_of(const Params& p, int b) {
  return p.own_len ? min(max(p.own_len[b], 0), p.S) : p.S;
}
template <typename P>
__device__ __forceinline__ int query_rows(const P& p, int b) {
  if constexpr (kPaged<P>) return p.q_len ? min(max(p.q_len[b], 0), p.T) : p.T;
  return p.T;
}
// own keys that token t of a sequence with `len` own keys and tq query rows sees
__device__ __forceinline__ int own_lim(const Params& p, int len, int t, int tq) {
  return p.causal ? min(max(len - tq + t + 1, 0), len) : len;
}
template <typename P>
__device__ __forceinline__ int own_tiles(const P& p, int len, int t0, int tb, int tq) {
  if (kPaged<P> && t0 >= tq) return 0;  // no row of the block
  return (own_lim(p, len, min(t0 + tb, tq) - 1, tq) + kKeys - 1) / kKeys;
}

template <typename P>
__device__ __forceinline__ Unit unit_of(const P& p, int u) {
  const Plan& pl = p.pl;
  Unit x;
  x.p0 = x.pn = x.o0 = x.on = x.len = 0;
  x.tq = p.T;
  x.clear = false;
  if (u < pl.units_p) {  // packed: prefix
    const int r = quot(p.d_nchp, u), c = u - r * pl.nchp;
    x.h = quot(p.d_npb, r);
    x.b0 = (r - x.h * pl.npb) * pl.rb;
    x.t0 = 0;
    x.p0 = c * pl.ct;
    x.pn = min(pl.ct, pl.pt - x.p0);
    x.rows = pl.rows_p;
    x.slot = static_cast<long long>(u) * pl.per * pl.rows_p;
  } else {
    const int v = u - pl.units_p;
    int r = quot(p.d_nch, v);
    const int c = v - r * pl.nch;
    int qb;
    if (pl.by_block) {  // causal: longest first over all heads and sequences
      const int k = quot(p.d_hb, r);
      qb = pl.nqb - 1 - k;
      r -= k * static_cast<int>(p.d_hb.d);
    } else {
      const int k = quot(p.d_nqb, r);
      qb = r - k * pl.nqb;
      r = k;
    }
    x.h = quot(p.d_B, r);
    x.b0 = r - x.h * p.B;
    x.t0 = qb * pl.tb;
    x.len = own_len_of(p, x.b0);
    const int pt = pl.packed ? 0 : pl.pt;
    x.tq = query_rows(p, x.b0);
    const int tiles = pt + own_tiles(p, x.len, x.t0, pl.tb, x.tq);
    const int lo = c * pl.ct;
    const int hi = min(lo + pl.ct, tiles);
    if (lo < hi) {
      x.p0 = min(lo, pt);
      x.pn = min(hi, pt) - x.p0;
      x.o0 = max(lo, pt) - pt;
      x.on = max(hi, pt) - pt - x.o0;
      // (rows past S read as zero, but not those of a page)
      x.clear = x.on > 0 && x.len < (x.o0 + x.on) * kKeys && (kPaged<P> || x.len < p.S);
    }
    x.rows = pl.rows_o;
    x.slot = (static_cast<long long>(pl.units_p) * pl.rows_p + static_cast<long long>(v) * pl.rows_o) * pl.per;
  }
  x.n = x.pn + x.on;
  return x;
}

// ------------------------------------------------------------------ even pieces of a cache in pages
//
// Sequences differ in length, and only the device knows by how much: units cut on the host for the
// longest leave some CTAs idle and others with a wave more. With FlowParams all blocks (sequence, head, row
// block) lie behind one another on a line, each as long as its tiles and a unit's overhead (pl.cost), which
// is cut into pl.flow x gridDim equal pieces: CTA c takes pieces c, c + gridDim, ..: whole blocks, whose rows
// it writes, and at either end a part of one, which it leaves as partials for merge_flow. A cut closer than
// kLeast tiles to an end of its block moves there. Every CTA works its cuts out for itself, from sums over the
// sequences. More rounds than one keep the CTAs, at any one time, on a stretch of the line whose keys stay
// in the L2 while the row blocks that share them pass by (figures: make_plan).
constexpr int kLeast = 2;
constexpr int kLineLog = 2, kLine = 1 << kLineLog;  // of the line to a tile
constexpr int kFlowThreads = 384;  // that add up: the smaller kernel's
constexpr int kMostRounds = 8;

struct FlowCut {
  int b, h, qb, j;  // sequence, head, row block, tile
};
__device__ __forceinline__ bool before(const FlowCut& x, const FlowCut& y) {
  return x.b != y.b ? x.b < y.b : x.h != y.h ? x.h < y.h : x.qb != y.qb ? x.qb < y.qb : x.j < y.j;
}
template <int SLOTS>
struct Flow {
  static constexpr int kSlots = SLOTS;
  int sum[SLOTS + 1];  // of one head's costs of all pairs before a slot's first, and of all (the plan sees to the range)
  int warp_sum[kFlowThreads / 32];
  FlowCut cut[2 * kMostRounds];  // begin and end of the CTA's pieces
  int from[kMostRounds];         // where the block that a piece begins in lies on the line
};
// partial rows of piece v: of the block that it takes over, 2 v; of the one that it leaves, 2 v + 1.
// rec[v] = (pair, head, whether that block ends here, piece that it began in) of the first, pair -1: none

// tiles of a pair, and whether it has rows at all
__device__ __forceinline__ int flow_tiles(const FlowParams& p, int e, bool& live) {
  const int b = quot(p.d_nqb, e), t0 = (e - b * p.pl.nqb) * p.pl.tb, len = own_len_of(p, b), tq = query_rows(p, b);
  live = t0 < tq;
  return own_tiles(p, len, t0, p.pl.tb, tq);
}
__device__ __forceinline__ int flow_cost(const FlowParams& p, int e) {
  bool live;
  const int n = flow_tiles(p, e, live);
  return live ? n * kLine + p.pl.cost : 0;
}
// costs of the pairs before pair e
template <typename F>
__device__ __forceinline__ int flow_upto(const FlowParams& p, const F& f, int e) {
  const int slot = quot(p.d_slot, e);
  int s = f.sum[slot];
  for (int x = slot * p.per_slot; x < e; ++x) s += flow_cost(p, x);
  return s;
}
// where on a line of `all` piece v begins: at floor(all v / pieces)
__device__ __forceinline__ int flow_at(const FlowParams& p, int all, int v) {
  const int n = static_cast<int>(p.d_pieces.d), each = quot(p.d_pieces, all);
  return each * v + quot(p.d_pieces, (all - each * n) * v);  // (n is below 2^15)
}

// Where piece v begins, by a warp: its lanes try 32 sequences, then 32 row blocks, at a time (one after the
// other, a lane's 9 steps for 6 sequences of 49 blocks came to 3 us, a launch's longest step). from: where the
// block that it begins in lies on the line.
template <typename F>
__device__ __forceinline__ FlowCut flow_cut(const FlowParams& p, const F& f, int all, int v, int& from) {
  const int nqb = p.pl.nqb, cost = p.pl.cost, lane = threadIdx.x & 31;
  const int pos = flow_at(p, all, v);
  from = pos;
  if (pos >= all) return {p.B, 0, 0, 0};
  // the last of n pairs, `step` apart from e0 on, with upto() mul <= most (the first one is)
  const auto find = [&](int e0, int n, int step, int mul, int most) {
    int lo = 0;
    while (n > 1) {
      const int each = (n + 31) >> 5, i = lane * each;
      const unsigned under = __ballot_sync(0xffffffffu, i < n && flow_upto(p, f, e0 + (lo + i) * step) * mul <= most);
      const int k = (31 - __clz(under)) * each;
      lo += k;
      n = min(each, n - k);
    }
    return lo;
  };
  FlowCut x{find(0, p.B, nqb, p.Hkv, pos), 0, 0, 0};
  const int e0 = x.b * nqb;
  const int base = flow_upto(p, f, e0), head = flow_upto(p, f, e0 + nqb) - base;
  int rest = pos - base * p.Hkv;
  x.h = rest / head;
  rest -= x.h * head;
  x.qb = find(e0, nqb, 1, 1, base + rest);
  const int begin = flow_upto(p, f, e0 + x.qb), length = flow_upto(p, f, e0 + x.qb + 1) - begin - cost;
  rest -= begin - base;
  from = pos - rest;
  x.j = (rest - cost) >> kLineLog;
  if (x.j < kLeast) {
    x.j = 0;
  } else if ((length >> kLineLog) - x.j < kLeast) {
    x.j = 0;
    if (++x.qb == nqb) {
      x.qb = 0;
      if (++x.h == p.Hkv) x.h = 0, ++x.b;
    }
  }
  return x;
}
// The piece in which a block began that lies at `from` and that a later one has the end of: the one before
// the first whose beginning is kLeast tiles into it.
__device__ __forceinline__ int flow_first(const FlowParams& p, int all, int from) {
  const int least = from + p.pl.cost + kLeast * kLine;
  // (floor(all w / n) >= least: an estimate, and steps from it)
  int w = static_cast<int>(__fdividef(static_cast<float>(least) * static_cast<float>(p.d_pieces.d), static_cast<float>(all)));
  while (flow_at(p, all, w) < least) ++w;
  while (w > 0 && flow_at(p, all, w - 1) >= least) --w;
  return w - 1;
}

// The CTA's pieces; all of its threads, of which the first kFlowThreads add up
template <typename F>
__device__ __forceinline__ void flow_pieces(const FlowParams& p, F& f) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int pairs = p.B * p.pl.nqb, slots = quot(p.d_slot, pairs + p.per_slot - 1);
  const int each = (slots + kFlowThreads - 1) / kFlowThreads, s0 = tid * each;
  int mine = 0, upto = 0;
  if (tid < kFlowThreads) {
    for (int s = s0; s < s0 + each && s < slots; ++s) {
      f.sum[s] = mine;
      for (int e = s * p.per_slot; e < (s + 1) * p.per_slot && e < pairs; ++e) mine += flow_cost(p, e);
    }
    upto = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, upto, d);
      if (lane >= d) upto += x;
    }
    if (lane == 31) f.warp_sum[warp] = upto;
  }
  __syncthreads();
  if (tid < kFlowThreads) {
    int at = upto - mine;
    for (int w = 0; w < warp; ++w) at += f.warp_sum[w];
    for (int s = s0; s < s0 + each && s < slots; ++s) f.sum[s] += at;
    if (tid == kFlowThreads - 1) f.sum[slots] = at + mine;
  }
  __syncthreads();
  const int all = f.sum[slots] * p.Hkv;
  for (int k = warp; k < 2 * p.pl.flow; k += static_cast<int>(blockDim.x) >> 5) {
    int from;
    const FlowCut x = flow_cut(p, f, all, (k >> 1) * static_cast<int>(gridDim.x) + static_cast<int>(blockIdx.x) + (k & 1), from);
    if (lane == 0) {
      f.cut[k] = x;
      if (!(k & 1)) f.from[k >> 1] = from;
    }
  }
  __syncthreads();
}
// What merge_flow is told of the CTA's pieces; a warp, which has the time
template <typename F>
__device__ __forceinline__ void flow_record(const FlowParams& p, const F& f) {
  const int r = threadIdx.x & 31;
  if (r < p.pl.flow) {
    const int pairs = p.B * p.pl.nqb, slots = quot(p.d_slot, pairs + p.per_slot - 1);
    const FlowCut a = f.cut[2 * r], z = f.cut[2 * r + 1];
    const bool one = a.b == z.b && a.h == z.h && a.qb == z.qb;  // the piece ends in the block that it begins in
    int4 rec = make_int4(-1, 0, 0, 0);
    if (a.j > 0 && !(one && a.j == z.j))
      rec = make_int4(a.b * p.pl.nqb + a.qb, a.h, one ? 0 : 1, flow_first(p, f.sum[slots] * p.Hkv, f.from[r]));
    p.rec[r * static_cast<int>(gridDim.x) + static_cast<int>(blockIdx.x)] = rec;
  }
  __syncwarp();
}

// The units of a CTA: unit blockIdx, blockIdx + grid, .., or those of its pieces
template <typename P, typename F>
struct Walk {
  int u;
  __device__ __forceinline__ Walk(const P&, const F*) : u(blockIdx.x) {}
  __device__ __forceinline__ bool more(const P& p) const { return u < p.pl.units; }
  __device__ __forceinline__ Unit unit(const P& p) const { return unit_of(p, u); }
  __device__ __forceinline__ void step(const P&) { u += gridDim.x; }
};
template <typename F>
struct Walk<FlowParams, F> {
  const F* f;
  int round = 0;
  FlowCut at, to;
  bool ends;  // the unit is the block's last
  int u = 0;
  __device__ __forceinline__ Walk(const FlowParams&, const F* flow) : f(flow), at(flow->cut[0]), to(flow->cut[1]) {}
  __device__ __forceinline__ bool more(const FlowParams& p) {
    for (;;) {
      while (before(at, to)) {
        const int tq = query_rows(p, at.b);
        if (at.qb * p.pl.tb < tq) return true;
        // no more rows
        at.qb = at.j = 0;
        if (tq == 0 || ++at.h == p.Hkv) at.h = 0, ++at.b;
      }
      if (++round >= p.pl.flow) return false;
      at = f->cut[2 * round];
      to = f->cut[2 * round + 1];
    }
  }
  __device__ __forceinline__ Unit unit(const FlowParams& p) {
    Unit x;
    x.b0 = at.b;
    x.h = at.h;
    x.t0 = at.qb * p.pl.tb;
    x.tq = query_rows(p, x.b0);
    x.len = own_len_of(p, x.b0);
    x.p0 = x.pn = 0;
    ends = !(at.b == to.b && at.h == to.h && at.qb == to.qb);
    const int stop = ends ? own_tiles(p, x.len, x.t0, p.pl.tb, x.tq) : to.j;
    x.o0 = at.j;
    x.n = x.on = stop - at.j;
    x.clear = x.on > 0 && x.len < stop * kKeys;
    x.rows = p.pl.rows_o;
    const long long v = static_cast<long long>(round) * gridDim.x + blockIdx.x;
    x.slot = at.j == 0 && ends ? -1 : (2 * v + (at.j == 0 ? 1 : 0)) * p.pl.rows_o;
    return x;
  }
  __device__ __forceinline__ void step(const FlowParams& p) {
    if (!ends) {
      at = to;
    } else {
      at.j = 0;
      if (++at.qb == p.pl.nqb) {
        at.qb = 0;
        if (++at.h == p.Hkv) at.h = 0, ++at.b;
      }
    }
  }
};

// 4-D tiled load: (dim, head, row, sequence); 5-D: (dim, head of the group, key head, token, sequence)
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int h, int row,
                                            int b) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(h), "r"(row), "r"(b)
      : "memory");
}
__device__ __forceinline__ void tma_load_5d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int g, int h,
                                            int t, int b) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(g), "r"(h), "r"(t), "r"(b)
      : "memory");
}

// One lane of a converged warp, always the same
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(one));
  return one != 0;
}

// The page that lane `lane` fetches for the tile of keys key0 .. key0 + 127 of a sequence: a tile is 128 >>
// page_log pages (or part of one), each two boxes of 64 dims, a lane a box. Pages behind the sequence and
// numbers that are none become `pages`, past the map's end, and read as zeros.
__device__ __forceinline__ int page_boxes(const PagedParams& p) { return p.page_log < 7 ? 256 >> p.page_log : 2; }
template <typename U>
__device__ __forceinline__ int page_of(const PagedParams& p, const U& un, int key0, int lane) {
  const int key = key0 + ((lane >> 1) << p.page_log);
  if (lane >= page_boxes(p) || key >= un.len) return p.pages;
  const int id = p.table[un.b0 * p.table_stride + (key >> p.page_log)];
  return static_cast<unsigned>(id) < static_cast<unsigned>(p.pages) ? id : p.pages;
}
// ... and its load, by the warp's lanes; `tile` has room for all boxes
__device__ __forceinline__ void load_pages(const PagedParams& p, const CUtensorMap* map, uint8_t* tile, uint64_t* bar,
                                           int h, int key0, int id, int lane) {
  if (lane < page_boxes(p))
    tma_load_4d(tile + (lane & 1) * kBox + ((lane >> 1) << (p.page_log + 7)), map, bar, (lane & 1) * 64, h,
                key0 & ((1 << p.page_log) - 1), id);
}

// ... of a tile of eight pages, by a lane that the pages are told to: by lanes, the boxes went out one in 130
// cycles, two warps' 32 a tile slower than its products (1024 rows behind 16384 in pages of 16, 234 us, this way
// 200; 6 x 777 rows 101 and 92; 16 x 300 rows over up to 1000, short units, 56 and 60). With fewer boxes a tile, or few
// rows, where HBM is the bound, the lanes are no slower and the code is shorter.
__device__ __forceinline__ void load_8_pages(const CUtensorMap* map, uint8_t* tile, uint64_t* bar, int h, int id) {
  int page[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) page[i] = __shfl_sync(0xffffffffu, id, 2 * i);
  if (elect_one()) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      tma_load_4d(tile + i * 2048, map, bar, 0, h, 0, page[i]);
      tma_load_4d(tile + i * 2048 + kBox, map, bar, 64, h, 0, page[i]);
    }
  }
  __syncwarp();
}

// Zeros for the rows of a V tile from r0 on, by a warp, in time for a product that it issues (a row's 128
// bytes stay within the row under the swizzle). The issuing warp does it, which would wait for P now: by the
// loading one, which then had to wait for its own load, the next unit's V came late
// (128 single tokens over up to 900 rows, 32 heads, 197 us; here 181; padded chunks of 777 rows, 98 and 95).
__device__ __forceinline__ void clear_rows(uint8_t* tile, int r0, int lane) {
  uint8_t* base = tile + r0 * 128;
  for (int i = lane; i < (kKeys - r0) * 8; i += 32) {
    *reinterpret_cast<uint4*>(base + i * 16) = make_uint4(0u, 0u, 0u, 0u);
    *reinterpret_cast<uint4*>(base + kBox + i * 16) = make_uint4(0u, 0u, 0u, 0u);
  }
  fence_proxy_async_smem();
  __syncwarp();
}

// 32 bytes, 32-byte aligned
__device__ __forceinline__ void store32(void* dst, const uint32_t (&r)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

template <bool BF16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  return BF16 ? pack_bf16x2(lo, hi) : pack_f16x2(lo, hi);
}

// Maps: Q over (dim, G, Hkv, T, B), once with the prefix block's box and once with
// the own / joint block's; K and V over (dim, Hkv, rows, sequences), prefix and own.
struct Maps {
  CUtensorMap qp, qo, pk, pv, k, v;
};


// The 8-bit prefix: maps over the codes (dim, key head, row; 16-byte piece i of row r lands at i ^ (r % 8)),
// scale bytes.
struct Maps8 {
  CUtensorMap k, v;
  const uint8_t* k_sf;
  const uint8_t* v_sf;
};

// Blocks of at most kFewRows rows (prefix_attention_few.cu); t8 NULL: 16-bit prefix. Each unit
// writes two partials; merge_partials joins them.
constexpr int kFewRows = 16;
constexpr int kFlowSlotsFew = 512;
cudaError_t launch_few(const Maps& tm, const Maps8* t8, const Params& p, bool bf16, float scale_log2, int sms,
                       cudaStream_t s);
cudaError_t launch_few(const Maps& tm, const PagedParams& p, bool bf16, float scale_log2, cudaStream_t s);  // pl.join
cudaError_t launch_few(const Maps& tm, const FlowParams& p, bool bf16, float scale_log2, cudaStream_t s);

// ------------------------------------------------------------------ what the host sides share (prefix_attention.cu)

struct Sizes {
  int B, T, Hq, Hkv, P, S, causal;
  bool from8, paged, ragged;  // ragged: of a cache in pages, whose chunks have lengths of their own
};

// workspace: the prefix in 16 bits (8-bit prefix only), partial O rows, their (max, sum), pieces' records
struct WsLayout {
  size_t pk, pv, part, ml, rec, total;
};

Plan plan_of(const Sizes& z, int sms);
WsLayout workspace_of(const Plan& pl);  // (without a prefix)
// what does not come from where the keys are
void set_params(Params* p, const Plan& pl, const Sizes& z, const Tensor4& o);
bool map_queries(CUtensorMap* m, const Tensor4& q, const Plan& pl, const Sizes& z);
// what launches without a status word report into, on the current device
cudaError_t status_word(int** word);
cudaError_t launch_merge(const PagedParams& p, bool bf16, cudaStream_t s);  // pl.split
// A stride of a dimension of size 1 is never followed: any legal value will do.
inline bool fix_stride(long long* s, int size) {
  if (size == 1) *s = 8;
  return *s > 0 && *s % 8 == 0 && *s < (1ll << 38);
}

// ------------------------------------------------------------------ parts joined by a cluster
//
// With pl.join the chunks of a row block are the CTAs of one cluster, one unit each, and their
// parts meet in distributed shared memory: no partials in memory and no second launch. Every
// CTA leaves part s of its unit at smem: row r of O (unnormalised, fp32) at float
// (s rows + r) kJoinPitch, its (maximum, sum) at kJoinMl + (s rows + r) 8 bytes; a part without
// a key has (-inf, 0), and its O is not read. CTA c writes output rows c, c + n, ..., adding the
// parts up in order.
constexpr int kJoinPitch = kHeadDim + 4;
constexpr int kJoinMl = 128 * kJoinPitch * 4;
constexpr int kJoinMost = 8;  // CTAs of a cluster that every GPU of this kind can place

template <bool BF16, typename P>
__device__ __forceinline__ void cluster_join(const P& p, const Unit& un, const uint8_t* smem, int rows) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int n = p.pl.nch, per = p.pl.per, parts = n * per;  // at most 16
  const uint32_t base = smem_u32(smem);
  for (int i = static_cast<int>(cluster_ctarank()) + n * warp; i < un.rows; i += n * warps) {
    float m = -INFINITY, l = 0.f;
    if (lane < parts) {
      const int c = per == 2 ? lane >> 1 : lane, s = per == 2 ? lane & 1 : 0;
      const uint32_t a = mapa_shared(base + kJoinMl + (s * rows + i) * 8, static_cast<uint32_t>(c));
      asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(m), "=f"(l) : "r"(a) : "memory");
    }
    float top = m;
#pragma unroll
    for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    const unsigned used = __ballot_sync(0xffffffffu, !(m == -INFINITY && l == 0.f));
    // (m = -inf with another sum is a row of NaN scores, which stays one)
    const float w = top == -INFINITY ? 1.f : fast_exp2(m - top);
    float den = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k = 0; k < parts; ++k) {
      if (!((used >> k) & 1u)) continue;
      const int c = per == 2 ? k >> 1 : k, s = per == 2 ? k & 1 : 0;
      const uint32_t a =
          mapa_shared(base + ((s * rows + i) * kJoinPitch + lane * 4) * 4, static_cast<uint32_t>(c));
      float4 v;
      asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                   : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                   : "r"(a)
                   : "memory");
      const float wk = __shfl_sync(0xffffffffu, w, k);
      den += __shfl_sync(0xffffffffu, l, k) * wk;
      acc.x += v.x * wk;
      acc.y += v.y * wk;
      acc.z += v.z * wk;
      acc.w += v.w * wk;
    }
    const float inv = den == 0.f ? 0.f : 1.f / den;
    const int tok = quot(p.d_G, i), g = i - tok * p.pl.G, t = un.t0 + tok;
    if (t < un.tq) {
      uint16_t* orow = p.o + un.b0 * p.ob + t * p.orow + static_cast<long long>(un.h * p.pl.G + g) * p.oh;
      reinterpret_cast<uint2*>(orow)[lane] =
          make_uint2(pack16<BF16>(acc.x * inv, acc.y * inv), pack16<BF16>(acc.z * inv, acc.w * inv));
    }
  }
}

// launch_dependent with clusters of `cluster` CTAs
template <typename... KArgs, typename... Args>
cudaError_t launch_clusters(void (*kernel)(KArgs...), int cluster, dim3 grid, dim3 block, size_t smem,
                            cudaStream_t stream, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<Args&&>(args)...);
}

}  // namespace pa
}  // namespace qi
