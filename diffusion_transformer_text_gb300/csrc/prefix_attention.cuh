// What the kernels of the shared-prefix attention have in common: the decomposition into
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

struct Unit {
  int h, b0, t0;
  int p0, pn;      // prefix tiles [p0, p0 + pn)
  int o0, on;      // own tiles of sequence b0
  int n;           // pn + on
  int len;         // own keys of sequence b0
  int rows;        // rows of the block (the MMA's other rows are ignored)
  bool clear;      // the last tile holds own rows at or past len
  long long slot;  // first partial row
};

__device__ __forceinline__ int own_len_of(const Params& p, int b) {
  return p.own_len ? min(max(p.own_len[b], 0), p.S) : p.S;
}
// own keys that token t of a sequence with `len` own keys sees
__device__ __forceinline__ int own_lim(const Params& p, int len, int t) {
  return p.causal ? min(max(len - p.T + t + 1, 0), len) : len;
}
__device__ __forceinline__ int own_tiles(const Params& p, int len, int t0, int tb) {
  return (own_lim(p, len, min(t0 + tb, p.T) - 1) + kKeys - 1) / kKeys;
}

__device__ __forceinline__ Unit unit_of(const Params& p, int u) {
  const Plan& pl = p.pl;
  Unit x;
  x.p0 = x.pn = x.o0 = x.on = x.len = 0;
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
    const int tiles = pt + own_tiles(p, x.len, x.t0, pl.tb);
    const int lo = c * pl.ct;
    const int hi = min(lo + pl.ct, tiles);
    if (lo < hi) {
      x.p0 = min(lo, pt);
      x.pn = min(hi, pt) - x.p0;
      x.o0 = max(lo, pt) - pt;
      x.on = max(hi, pt) - pt - x.o0;
      x.clear = x.on > 0 && x.len < (x.o0 + x.on) * kKeys && x.len < p.S;
    }
    x.rows = pl.rows_o;
    x.slot = (static_cast<long long>(pl.units_p) * pl.rows_p + static_cast<long long>(v) * pl.rows_o) * pl.per;
  }
  x.n = x.pn + x.on;
  return x;
}

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
cudaError_t launch_few(const Maps& tm, const Maps8* t8, const Params& p, bool bf16, float scale_log2, int sms,
                       cudaStream_t s);

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

template <bool BF16>
__device__ __forceinline__ void cluster_join(const Params& p, const Unit& un, const uint8_t* smem, int rows) {
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
    if (t < p.T) {
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
