// Shared-prefix attention for blocks of at most 16 query rows (single tokens, drafted
// tokens): the products transposed, so that keys and head dimensions, not the few query
// rows, fill the 128 lanes of the tensor cores.
//
//   S^T [128 keys x 16 rows]  = K [128 x 128] Q^T        (A = the K tile, B = Q, N = 16)
//   O^T [128 dims x 16 rows] += V^T [128 x 128] P^T      (A = the V tile read MN-major, B = P)
//
// With the query rows as MMA rows a tile of 128 keys costs two N = 128 products and 64
// exponentials a thread whatever the row count; here it costs two N = 16 products and 16
// exponentials, and what is left is to keep HBM busy: K and V of a tile, 64 KB, go through
// an SM in about 1.4 us at full bandwidth, half that in 8 bits. The 8-bit prefix (Q8) is
// read as the codes it is: two further warpgroups turn a tile's codes and scales into the
// 16-bit K and V tiles in shared memory, so HBM and L2 carry 8 bits a value.
//
// A thread of a softmax warpgroup owns one key of the tile and all 16 rows; a row's maximum
// is a warp reduction (redux) and an exchange between the four warps. The two softmax
// warpgroups take alternate tiles, each with its own running maximum, sums and O^T; both
// write their partial result, and merge_partials joins them like any other parts; with JOIN
// the chunks of a block are the CTAs of one cluster, O^T stays in tensor memory and
// cluster_join adds the parts through distributed shared memory, in a fixed order. A row
// whose maximum grows by more than 2^8 rescales O^T (each warp its quarter of the dims).
//
// Roles: warp 0 loads K and Q, warp 2 V (and clears V rows past own_len), warp 1 issues
// S^T, warp 3 O^T; warps 4-7 and 8-11 softmax; with Q8 warps 12-15 turn K codes and warps
// 16-19 V codes into 16 bits. Warps that meet at a named barrier never leave their loops
// early: a wait that expires only makes them skip the work.
//
// Measured, 16 sequences of one token over 8192 prefix + 256 own keys, 32 key heads: 16 bits
// 38.1 us with the merge (the packed 128-row kernel 43.7), 4.8 TB/s; 8-bit prefix 40.4 us,
// 2.9 TB/s (75 us with the prefix turned into 16 bits in memory first). One sequence over
// 131072 prefix rows: 16 bits 304 us, the copy rate; 8 bits 287 us, 57 % of it. There a tile of
// codes takes 2300 cycles where HBM would give it in 1400: converting it keeps four warps
// apiece for K and V busy for about 1800, 500 of them with the conversions themselves, the
// rest with waits for their stages and with shared memory, which carries the codes in and out
// and the 16-bit tiles in and out.
#include "prefix_attention.cuh"

namespace qi {
using namespace pa;
namespace {

constexpr int kR = kFewRows;                  // 16: N of both products
constexpr int kQTile = kR * 256;              // Q or P of a block: two 64-column boxes of 16 rows
constexpr int kQBox = kR * 128;
constexpr int kCode = kKeys * kHeadDim;       // a tile of codes (16 KB)
constexpr int kQBufs = 2;
constexpr int kSBufs = 4;                     // S^T, and P: two per softmax warpgroup
constexpr uint32_t kTmemCols = 128;
constexpr uint32_t kColS = 0;                 // S^T buffer b at 16 b
constexpr uint32_t kColO = 64;                // O^T of warpgroup s at 64 + 16 s

template <bool Q8>
struct Cfg {
  static constexpr int kSt = Q8 ? 2 : 3;   // 16-bit K tiles, and V tiles
  static constexpr int kCSt = Q8 ? 2 : 0;  // tiles of K codes, and of V codes
  static constexpr int kThreads = Q8 ? 640 : 384;
};

// mbarriers; [K, V] where a pair is meant
enum : int {
  kFull = 0,                     // [K, V][3] 16-bit tile in place (producer; with Q8 also 4 converting warps)
  kEmpty = kFull + 6,            // [K, V][3] ... read by its product
  kCFull = kEmpty + 6,           // [K, V][2] codes in place
  kCEmpty = kCFull + 4,          // [K, V][2] ... turned into 16 bits (4 warps)
  kVClean = kCEmpty + 4,         // [3] rows past own_len of a unit's last V tile cleared
  kQFull = kVClean + 3,
  kQEmpty = kQFull + kQBufs,
  kSFull = kQEmpty + kQBufs,
  kSFree = kSFull + kSBufs,      // S^T in registers (4 warps)
  kPFull = kSFree + kSBufs,      // P in shared memory (4 warps)
  kPDone = kPFull + kSBufs,      // the tile's O^T product complete
  kDrainQK = kPDone + kSBufs,
  kDrainPV = kDrainQK + 1,
  kNumBars = kDrainPV + 1
};
constexpr int kBarSlots = (kNumBars + 1) & ~1;  // what follows is read in 16-byte pieces
template <bool Q8>
__device__ __forceinline__ uint32_t bar_count(int i) {
  if (i < kFull + 6) return Q8 ? 5 : 1;
  return (i >= kCEmpty && i < kCEmpty + 4) || (i >= kSFree && i < kSFree + kSBufs) ||
                 (i >= kPFull && i < kPFull + kSBufs)
             ? 4
             : 1;
}

// per softmax warpgroup: maxima by [tile parity][warp][row], sums by [warp][row]; per warp:
// negated maximum, rescale factor and key limit by row
struct Exchange {
  float top[2][2][4][kR];
  float sum[2][4][kR];
  float nm[8][kR], alpha[8][kR];
  int lim[8][kR];
  uint32_t issued[3][5];
  uint32_t pad;
  float2 ml[2][kR];  // JOIN: each warpgroup's maxima and sums
};
template <bool Q8>
constexpr int smem_bytes() {
  using C = Cfg<Q8>;
  return 2 * C::kSt * kTile + 2 * C::kCSt * kCode + kQBufs * kQTile + kSBufs * kQTile + 1024 + kBarSlots * 8 + 16 +
         static_cast<int>(sizeof(Exchange));
}
static_assert(smem_bytes<true>() <= 227 * 1024 && smem_bytes<false>() <= 227 * 1024, "shared memory per block");

__device__ __forceinline__ void warpgroup_sync(int id) { asm volatile("bar.sync %0, 128;" ::"r"(id) : "memory"); }

// the largest of the warp's values, in every lane
__device__ __forceinline__ float redux_max(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}
// sum += the low half of a pair of 16-bit values. The row sums are those of the probabilities as the
// product uses them, after their rounding: the weights of a row add up to 1, and an error of the
// largest one (which is no power of two where the maximum has moved by less than kRescaleLog2) does not
// scale the row. Costs nothing here; the kernel of 128 rows, where it would take a third more
// instructions a probability (causal continuation 85 -> 91 us), adds them up before the rounding.
template <bool BF16>
__device__ __forceinline__ void add16(float& sum, uint32_t pair) {
  if (BF16)
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tadd.f32.bf16 %0, l, %0;\n\t}" : "+f"(sum) : "r"(pair));
  else
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tadd.f32.f16 %0, l, %0;\n\t}" : "+f"(sum) : "r"(pair));
}
__device__ __forceinline__ void load16f(const float* src, float (&v)[kR]) {
#pragma unroll
  for (int i = 0; i < kR / 4; ++i) {
    const float4 f = reinterpret_cast<const float4*>(src)[i];
    v[4 * i] = f.x, v[4 * i + 1] = f.y, v[4 * i + 2] = f.z, v[4 * i + 3] = f.w;
  }
}
__device__ __forceinline__ void store16f(float* dst, const float (&v)[kR]) {
#pragma unroll
  for (int i = 0; i < kR / 4; ++i)
    reinterpret_cast<float4*>(dst)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
}

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int h, int row) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(h), "r"(row)
      : "memory");
}

// 2^e as a half, for the exponents with which code * 2^e can be formed in half precision (codes
// have 4 significant bits: the product is exact or, below 2^-14, rounded once); kNoHalf else.
constexpr uint32_t kNoHalf = 0xFFFFu;
__device__ __forceinline__ uint32_t half_scale(uint32_t byte) {
  const int e = static_cast<int>(byte) - 127;
  return e < -24 || e > 15 ? kNoHalf : e >= -14 ? static_cast<uint32_t>(e + 15) << 10 : 1u << (e + 24);
}

// 8 codes times their scale, rounded to the 16-bit type: in half precision by half_scale's value
// if HALF, else in fp32 by the scale byte
template <bool BF16, bool HALF>
__device__ __forceinline__ uint4 codes_to_16bit(uint2 c, uint32_t scale) {
  const uint32_t w[4] = {c.x & 0xFFFFu, c.x >> 16, c.y & 0xFFFFu, c.y >> 16};
  uint32_t r[4];
  if (HALF) {
    const uint32_t pair = scale | (scale << 16);
    const __half2 s = *reinterpret_cast<const __half2*>(&pair);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 v =
          __hmul2(__half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w[i]), __NV_E4M3)), s);
      r[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
  } else {
    const float s = __uint_as_float(scale == 0 ? 0x00400000u : scale << 23);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f =
          __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w[i]), __NV_E4M3)));
      r[i] = pack16<BF16>(f.x * s, f.y * s);
    }
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

template <bool BF16, bool Q8, bool JOIN>
__global__ void __launch_bounds__(Cfg<Q8>::kThreads, 1)
    prefix_attn_few(const __grid_constant__ Maps tm, const __grid_constant__ Maps8 t8, const __grid_constant__ Params p,
                    float scale_log2) {
  using C = Cfg<Q8>;
  constexpr int kSt = C::kSt, kCSt = Q8 ? 2 : 1;
  constexpr uint32_t kIdescS = BF16 ? idesc_bf16_f32(128, kR) : idesc_f16_f32(128, kR);
  constexpr uint32_t kIdescO = kIdescS | (1u << 15);  // A MN-major
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sT = smem;                                // [K, V][kSt] 16-bit tiles
  uint8_t* sC = sT + 2 * kSt * kTile;                // [K, V][kCSt] codes
  uint8_t* sQ = sC + 2 * C::kCSt * kCode;
  uint8_t* sP = sQ + kQBufs * kQTile;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sP + kSBufs * kQTile);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + kBarSlots);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  Exchange& ex = *reinterpret_cast<Exchange*>(tmem_slot + 4);
  uint32_t(*const issued)[5] = ex.issued;  // loads into each stage, last tile + 1: [K, V][16-bit 3, codes 2], Q

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int total = p.pl.units;
  const auto give_up = [&](int code) {
    if (!*abort_flag) report_error(p.err, code);
    *abort_flag = 1;
  };

  if (threadIdx.x == 0) {
    for (int i = 0; i < kNumBars; ++i) mbar_init(&bars[i], bar_count<Q8>(i));
    *abort_flag = 0;
    for (int i = 0; i < 15; ++i) ex.issued[i / 5][i % 5] = 0;
    for (int i = 0; i < 2 * kR; ++i) ex.ml[i / kR][i % kR] = make_float2(-INFINITY, 0.f);
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tm.qp);
    prefetch_tmap(&tm.qo);
    prefetch_tmap(&tm.k);
    prefetch_tmap(Q8 ? &t8.k : &tm.pk);
  }
  if (warp == 2 && lane == 0) {
    prefetch_tmap(&tm.v);
    prefetch_tmap(Q8 ? &t8.v : &tm.pv);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  // rows past a block's stay finite: nothing they hold may move a maximum
  for (int i = threadIdx.x; i < kQBufs * kQTile / 16; i += C::kThreads)
    reinterpret_cast<uint4*>(sQ)[i] = make_uint4(0u, 0u, 0u, 0u);
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_dep_wait();
  grid_dep_launch_dependents();

  if (warp == 0 || warp == 2) {
    // ---------------- producers: K tiles and Q (warp 0), V tiles (warp 2). Lane 0 works; warp 2
    // clears V rows past own_len as a whole, so every lane walks the units.
    const int kv = warp == 0 ? 0 : 1;
    uint32_t t = 0, tc = 0, nq = 0;  // tiles; of which requested as codes; Q blocks
    uint64_t* full = &bars[kFull + 3 * kv];
    uint64_t* empty = &bars[kEmpty + 3 * kv];
    uint64_t* cfull = &bars[kCFull + 2 * kv];
    uint64_t* cempty = &bars[kCEmpty + 2 * kv];
    uint8_t* tiles = sT + kv * kSt * kTile;
    uint8_t* codes = sC + kv * kCSt * kCode;
    const CUtensorMap* pre_map = kv ? &tm.pv : &tm.pk;
    const CUtensorMap* own_map = kv ? &tm.v : &tm.k;
    const CUtensorMap* code_map = kv ? &t8.v : &t8.k;
    bool ok = true;
    for (int u = blockIdx.x; u < total; u += gridDim.x) {
      const Unit un = unit_of(p, u);
      if (un.n == 0) continue;
      if (lane == 0 && ok) {
        if (kv == 0) {
          const uint32_t qb = nq % kQBufs;
          ok = !*abort_flag && mbar_wait(&bars[kQEmpty + qb], ((nq / kQBufs) & 1u) ^ 1u);
          if (ok) {
            const CUtensorMap* mq = u < p.pl.units_p ? &tm.qp : &tm.qo;
            mbar_arrive_expect_tx(&bars[kQFull + qb], static_cast<uint32_t>(un.rows) * 256u);
            tma_load_5d(sQ + qb * kQTile, mq, &bars[kQFull + qb], 0, 0, un.h, un.t0, un.b0);
            tma_load_5d(sQ + qb * kQTile + kQBox, mq, &bars[kQFull + qb], 64, 0, un.h, un.t0, un.b0);
            issued[2][qb] = ++nq;
          }
        }
        // Codes are requested two tiles ahead of their turn. Of every tile, turned from codes or
        // loaded as it is, the producer and the converting warps each wait for the 16-bit stage and
        // then arrive on it: a barrier's parity tells the phases apart only to who sees them all,
        // and none of them can be passed over this way.
        const auto request = [&](int j) {
          const uint32_t cs = tc % kCSt;
          if (!mbar_wait(&cempty[cs], ((tc / kCSt) & 1u) ^ 1u)) return false;
          mbar_arrive_expect_tx(&cfull[cs], kCode);
          tma_load_3d(codes + cs * kCode, code_map, &cfull[cs], 0, un.h, (un.p0 + j) * kKeys);
          issued[kv][3 + cs] = ++tc;
          return true;
        };
        if (Q8 && ok && un.pn > 0) ok = request(0) && (un.pn < 2 || request(1));
        for (int j = 0; ok && j < un.n; ++j) {
          const uint32_t tt = t + j, st = tt % kSt;
          const bool pre = j < un.pn;
          ok = mbar_wait(&empty[st], ((tt / kSt) & 1u) ^ 1u);
          if (!ok) break;
          if (Q8 && pre) {
            mbar_arrive(&full[st]);
            if (j + 2 < un.pn) ok = request(j + 2);
          } else {
            const CUtensorMap* m = pre ? pre_map : own_map;
            const int row = (pre ? un.p0 + j : un.o0 + j - un.pn) * kKeys;
            const int bs = pre ? 0 : un.b0;
            mbar_arrive_expect_tx(&full[st], kTile);
            tma_load_4d(tiles + st * kTile, m, &full[st], 0, un.h, row, bs);
            tma_load_4d(tiles + st * kTile + kBox, m, &full[st], 64, un.h, row, bs);
            issued[kv][st] = tt + 1;
          }
        }
        if (!ok) give_up(kErrTimeoutProducer);
      }
      t += un.n;
      if (kv == 1 && un.clear) {
        const uint32_t last = t - 1, st = last % kSt;
        if (lane == 0 && ok && !mbar_wait(&full[st], (last / kSt) & 1u)) {
          give_up(kErrTimeoutProducer);
          ok = false;
        }
        if (__shfl_sync(0xffffffffu, static_cast<int>(ok), 0)) {
          const int r0 = un.len - (un.o0 + un.on - 1) * kKeys;
          const int n16 = (kKeys - r0) * 8;
          uint8_t* base = tiles + st * kTile + r0 * 128;
          for (int i = lane; i < n16; i += 32) {
            *reinterpret_cast<uint4*>(base + i * 16) = make_uint4(0u, 0u, 0u, 0u);
            *reinterpret_cast<uint4*>(base + kBox + i * 16) = make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0 && ok) mbar_arrive(&bars[kVClean + st]);
      }
    }
  } else if (warp == 1) {
    // ---------------- S^T issuer. The issuing warps walk as a whole, so that the descriptors are
    // uniform: by a lane alone a product was issued 900 cycles after its operands were there (the
    // other warps' instructions came first), now 400; 7 sequences of 5 tokens 11.5 us, now 10.9.
    {
      const uint64_t kdesc0 = sw128_kmajor_desc(smem_u32(sT));
      const uint64_t qdesc0 = sw128_kmajor_desc(smem_u32(sQ));
      uint32_t t = 0, ku = 0;
      bool ok = true;
      for (int u = blockIdx.x; ok && u < total; u += gridDim.x) {
        const Unit un = unit_of(p, u);
        if (un.n == 0) continue;
        const uint32_t qb = ku % kQBufs;
        ok = __all_sync(0xffffffffu, !*abort_flag && mbar_wait(&bars[kQFull + qb], (ku / kQBufs) & 1u));
        if (!ok) break;
        const uint64_t qd = qdesc0 + ((qb * kQTile) >> 4);
        for (int j = 0; j < un.n; ++j, ++t) {
          const uint32_t st = t % kSt, sb = t % kSBufs;
          ok = __all_sync(0xffffffffu, mbar_wait(&bars[kSFree + sb], ((t / kSBufs) & 1u) ^ 1u) &&
                                           mbar_wait(&bars[kFull + st], (t / kSt) & 1u));
          if (!ok) break;
          tc_fence_after();
          const uint64_t kd = kdesc0 + ((st * kTile) >> 4);
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < kHeadDim / 16; ++k)
              mma_ss(tmem + kColS + 16 * sb, kd + (((k >> 2) * kBox + (k & 3) * 32) >> 4),
                     qd + (((k >> 2) * kQBox + (k & 3) * 32) >> 4), kIdescS, k > 0 ? 1u : 0u);
            mma_commit(&bars[kSFull + sb]);
            mma_commit(&bars[kEmpty + st]);
            if (j + 1 == un.n) mma_commit(&bars[kQEmpty + qb]);
          }
          __syncwarp();
        }
        if (!ok) break;
        ++ku;
      }
      if (elect_one()) {
        if (!ok) give_up(kErrTimeoutMma);
        mma_commit(&bars[kDrainQK]);
        if (!mbar_wait(&bars[kDrainQK], 0)) report_error(p.err, kErrTimeoutDrain);
      }
      __syncwarp();
    }
  } else if (warp == 3) {
    // ---------------- O^T issuer: the first tile of each warpgroup in a unit overwrites its O^T
    // (which it has read: its P comes after)
    {
      const uint64_t vdesc0 = sw128_mnmajor_desc(smem_u32(sT + kSt * kTile), kBox, 1024);
      const uint64_t pdesc0 = sw128_kmajor_desc(smem_u32(sP));
      uint32_t t = 0, cleared = 0;
      bool ok = true;
      for (int u = blockIdx.x; ok && u < total; u += gridDim.x) {
        const Unit un = unit_of(p, u);
        for (int j = 0; j < un.n; ++j, ++t) {
          const uint32_t st = t % kSt, sb = t % kSBufs;
          ok = mbar_wait(&bars[kFull + 3 + st], (t / kSt) & 1u);
          if (un.clear && j + 1 == un.n) {
            ok = ok && mbar_wait(&bars[kVClean + st], (cleared >> st) & 1u);
            cleared ^= 1u << st;  // the stage's phase
          }
          ok = __all_sync(0xffffffffu, ok && mbar_wait(&bars[kPFull + sb], (t / kSBufs) & 1u));
          if (!ok) break;
          tc_fence_after();
          const uint64_t vd = vdesc0 + ((st * kTile) >> 4);
          const uint64_t pd = pdesc0 + ((sb * kQTile) >> 4);
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < kKeys / 16; ++k)
              mma_ss(tmem + kColO + 16 * (t & 1u), vd + ((k * 2048) >> 4),
                     pd + (((k >> 2) * kQBox + (k & 3) * 32) >> 4), kIdescO, (j > 1 || k > 0) ? 1u : 0u);
            mma_commit(&bars[kPDone + sb]);
            mma_commit(&bars[kEmpty + 3 + st]);
          }
          __syncwarp();
        }
        if (!ok) break;
      }
      if (elect_one()) {
        if (!ok) give_up(kErrTimeoutMma);
        mma_commit(&bars[kDrainPV]);
        if (!mbar_wait(&bars[kDrainPV], 0)) report_error(p.err, kErrTimeoutDrain);
      }
      __syncwarp();
    }
  } else if (warp < 12) {
    // ---------------- softmax: warpgroup s takes the tiles of parity s; thread = one key
    const int s = (warp - 4) >> 2;
    const int quarter = warp & 3, sw = warp - 4;
    const int key = quarter * 32 + lane;
    const int row16 = lane & 15;  // the row this lane keeps the maximum of
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t tO = tmem + lane_off + kColO + 16u * s;
    const int tok16 = quot(p.d_G, row16);
    // P: row i of key k at box k / 64, 16-byte piece ((k % 64) / 8) ^ (i % 8)
    uint8_t* const pcol = sP + (key >> 6) * kQBox + (key & 7) * 2;
    const uint32_t piece = static_cast<uint32_t>((key & 63) >> 3);
    uint32_t t = 0, turn = 0;
    bool ok = true;
    for (int u = blockIdx.x; u < total; u += gridDim.x) {
      const Unit un = unit_of(p, u);
      if (un.n == 0) continue;
      const int lim16 = own_lim(p, un.len, un.t0 + tok16);
      const int lim_least = own_lim(p, un.len, un.t0);
      if (lane < kR) ex.lim[sw][lane] = lim16;
      __syncwarp();
      float m_used = -INFINITY;
      float l[kR] = {};
      int cnt = 0;
      uint32_t last = 0;
      for (int j = static_cast<int>((t ^ s) & 1u); j < un.n; j += 2, ++cnt) {
        const uint32_t tt = t + j, sb = tt % kSBufs, ph = (tt / kSBufs) & 1u;
        last = tt;
        ok = ok && __all_sync(0xffffffffu, mbar_wait(&bars[kSFull + sb], ph));
        tc_fence_after();
        uint32_t r[kR];
        tmem_ld16(tmem + lane_off + kColS + 16 * sb, r);
        tmem_ld_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[kSFree + sb]);
        float x[kR];
#pragma unroll
        for (int i = 0; i < kR; ++i) x[i] = __uint_as_float(r[i]);
        // keys at or past a row's limit become -inf, whatever their scores are
        const bool pre = j < un.pn;
        const int k0 = (pre ? un.p0 + j : un.o0 + j - un.pn) * kKeys;
        if (k0 + kKeys > (pre ? p.P : lim_least)) {
#pragma unroll
          for (int i = 0; i < kR; ++i) {
            const int lim = pre ? p.P : ex.lim[sw][i];
            if (k0 + key >= lim) x[i] = -INFINITY;
          }
        }
        float w[kR];
#pragma unroll
        for (int i = 0; i < kR; ++i) w[i] = redux_max(x[i]);
        if (lane == 0) store16f(ex.top[s][turn][quarter], w);
        warpgroup_sync(1 + s);
        const float mx = fmaf(fmaxf(fmaxf(ex.top[s][turn][0][row16], ex.top[s][turn][1][row16]),
                                    fmaxf(ex.top[s][turn][2][row16], ex.top[s][turn][3][row16])), scale_log2, -kLift<BF16>);
        turn ^= 1u;
        const float m_new = fmaxf(m_used, mx);
        if (cnt == 0) {
          m_used = m_new;
        } else {
          // (the four warps see the same numbers, so they agree)
          const bool grow = m_new > m_used + kRescaleLog2;
          if (__any_sync(0xffffffffu, grow)) {
            const uint32_t tp = tt - 2;
            ok = ok && __all_sync(0xffffffffu, mbar_wait(&bars[kPDone + tp % kSBufs], (tp / kSBufs) & 1u));
            tc_fence_after();
            if (lane < kR) ex.alpha[sw][lane] = grow ? fast_exp2(m_used - m_new) : 1.0f;
            __syncwarp();
            float al[kR];
            load16f(ex.alpha[sw], al);
            uint32_t o[kR];
            tmem_ld16(tO, o);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < kR; ++i) {
              o[i] = __float_as_uint(__uint_as_float(o[i]) * al[i]);
              l[i] *= al[i];
            }
            tmem_st16(tO, o);
            tmem_st_wait();
            tc_fence_before();
            if (grow) m_used = m_new;
          }
        }
        if (lane < kR) ex.nm[sw][lane] = m_used == -INFINITY ? 0.f : -m_used;
        __syncwarp();
        float nm[kR];
        load16f(ex.nm[sw], nm);
        ok = ok && __all_sync(0xffffffffu, mbar_wait(&bars[kPDone + sb], ph ^ 1u));
        uint8_t* const dst = pcol + sb * kQTile;
#pragma unroll
        for (int i = 0; i < kR; ++i) {
          const uint32_t e = pack16<BF16>(fast_exp2(fmaf(x[i], scale_log2, nm[i])), 0.f);
          add16<BF16>(l[i], e);
          *reinterpret_cast<uint16_t*>(dst + i * 128 + ((piece ^ (i & 7u)) << 4)) = static_cast<uint16_t>(e);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[kPFull + sb]);
      }
      // this warpgroup's part of the block's rows
      const long long slot = un.slot + s * un.rows;
      if (cnt > 0) {
        // sums over the warp's lanes
#pragma unroll
        for (int d = 16; d; d >>= 1)
#pragma unroll
          for (int i = 0; i < kR; ++i) l[i] += __shfl_xor_sync(0xffffffffu, l[i], d);
        if (lane == 0) store16f(ex.sum[s][quarter], l);
        warpgroup_sync(1 + s);
        const float den = (ex.sum[s][0][row16] + ex.sum[s][1][row16]) + (ex.sum[s][2][row16] + ex.sum[s][3][row16]);
        if (quarter == 0 && lane < kR) {
          if (JOIN)
            ex.ml[s][lane] = make_float2(m_used, den);
          else if (lane < un.rows)
            p.ml[slot + lane] = make_float2(m_used, den);
        }
        ok = ok && __all_sync(0xffffffffu, mbar_wait(&bars[kPDone + last % kSBufs], (last / kSBufs) & 1u));
        if (JOIN) continue;  // O^T stays in tensor memory for the end of the kernel
        tc_fence_after();
        uint32_t o[kR];
        tmem_ld16(tO, o);
        tmem_ld_wait();
        tc_fence_before();
        float* out = p.part + slot * kHeadDim + key;  // key doubles as the dim this lane holds
#pragma unroll
        for (int i = 0; i < kR; ++i)
          if (i < un.rows) out[i * kHeadDim] = __uint_as_float(o[i]);
        // (the next unit's sums are stored after another warpgroup_sync)
      } else if (!JOIN && quarter == 0 && lane < un.rows) {
        p.ml[slot + lane] = make_float2(-INFINITY, 0.f);  // no tile: merge_partials passes it over
      }
      t += un.n;
    }
    if (!ok && lane == 0) give_up(kErrTimeoutEpilogue);
  } else if constexpr (Q8) {
    // ---------------- codes to 16 bits: warps 12..15 K, 16..19 V. A lane turns one row (key): its
    // four scale bytes stay with it, and eight lanes' pieces of one column lie in eight different
    // 16-byte places of a 128-byte line, of the codes (swizzled as the 16-bit tiles are) and of the
    // tile alike, so neither access meets itself in the banks. (Sixteen lanes a row, the scales by
    // way of shared memory: 3 to 6 % slower. K by way of tensor memory: 8 % slower. Half of the
    // codes by integer instructions instead of the converter: 17 % slower.)
    const int kv = warp >= 16 ? 1 : 0;
    const int row = (warp & 3) * 32 + lane;
    const uint32_t turn = static_cast<uint32_t>(row & 7) << 4;
    const uint32_t* sf4 = reinterpret_cast<const uint32_t*>(kv ? t8.v_sf : t8.k_sf);  // 4-byte aligned
    uint8_t* tiles = sT + kv * kSt * kTile + row * 128;
    const uint8_t* codes = sC + kv * kCSt * kCode + row * 128;
    const auto scales_of = [&](const Unit& un, int tile) -> uint32_t {
      const int r = tile * kKeys + row;
      return r < p.P ? sf4[static_cast<long long>(r) * p.Hkv + un.h] : 0u;  // past the end: zero codes
    };
    uint32_t t = 0, tc = 0;
    bool ok = true;
    for (int u = blockIdx.x; u < total; u += gridDim.x) {
      const Unit un = unit_of(p, u);
      uint32_t bytes = un.pn > 0 ? scales_of(un, un.p0) : 0u;
      for (int j = 0; j < un.n; ++j) {
        const uint32_t tt = t + j, st = tt % kSt, cs = tc % kCSt;
        ok = ok && __all_sync(0xffffffffu, mbar_wait(&bars[kEmpty + 3 * kv + st], ((tt / kSt) & 1u) ^ 1u));
        if (j >= un.pn) {  // an own tile: nothing to turn
          if (lane == 0 && ok) mbar_arrive(&bars[kFull + 3 * kv + st]);
          continue;
        }
        const uint32_t ahead = j + 1 < un.pn ? scales_of(un, un.p0 + j + 1) : 0u;
        ok = ok && __all_sync(0xffffffffu, mbar_wait(&bars[kCFull + 2 * kv + cs], (tc / kCSt) & 1u));
        if (ok) {
          const uint8_t* src = codes + cs * kCode;
          uint8_t* dst = tiles + st * kTile;
          // (all loads before the first store: nothing tells the compiler that the two do not overlap)
          uint4 c[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) c[i] = *reinterpret_cast<const uint4*>(src + ((i << 4) ^ turn));
          // fp16: in half precision, unless a scale of the warp's rows does not allow it
          uint32_t h[4], worst = 0;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t byte = (bytes >> (8 * i)) & 255u;
            h[i] = BF16 ? byte : half_scale(byte);
            worst = max(worst, h[i]);
          }
          const auto put = [&](int i, uint4 lo, uint4 hi) {  // pieces 2 i and 2 i + 1
            uint8_t* box = dst + (i >> 2) * kBox;
            *reinterpret_cast<uint4*>(box + (((2 * i & 7) << 4) ^ turn)) = lo;
            *reinterpret_cast<uint4*>(box + (((2 * i & 7) + 1) << 4 ^ turn)) = hi;
          };
          if (!BF16 && __any_sync(0xffffffffu, worst == kNoHalf)) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const uint32_t byte = (bytes >> (8 * (i >> 1))) & 255u;
              put(i, codes_to_16bit<BF16, false>(make_uint2(c[i].x, c[i].y), byte),
                  codes_to_16bit<BF16, false>(make_uint2(c[i].z, c[i].w), byte));
            }
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              put(i, codes_to_16bit<BF16, !BF16>(make_uint2(c[i].x, c[i].y), h[i >> 1]),
                  codes_to_16bit<BF16, !BF16>(make_uint2(c[i].z, c[i].w), h[i >> 1]));
          }
        }
        bytes = ahead;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && ok) {
          mbar_arrive(&bars[kFull + 3 * kv + st]);
          mbar_arrive(&bars[kCEmpty + 2 * kv + cs]);
        }
        ++tc;
      }
      t += un.n;
    }
    if (!ok && lane == 0) give_up(kErrTimeoutProducer);
  }

  tc_fence_before();
  __syncthreads();
  // Without a failure every load has been waited for by what it fed. After one, each producer
  // waits for its last loads into every stage before the block ends (bounded; a stage that has
  // moved on just costs the limit).
  if (*abort_flag && lane == 0 && (warp == 0 || warp == 2)) {
    const int kv = warp == 0 ? 0 : 1;
    for (int i = 0; i < kSt; ++i)
      if (issued[kv][i]) mbar_wait(&bars[kFull + 3 * kv + i], ((issued[kv][i] - 1) / kSt) & 1u);
    for (int i = 0; i < C::kCSt; ++i)
      if (issued[kv][3 + i]) mbar_wait(&bars[kCFull + 2 * kv + i], ((issued[kv][3 + i] - 1) / kCSt) & 1u);
    for (int i = 0; kv == 0 && i < kQBufs; ++i)
      if (issued[2][i]) mbar_wait(&bars[kQFull + i], ((issued[2][i] - 1) / kQBufs) & 1u);
  }
  __syncthreads();
  if (JOIN) {
    // the unit was the CTA's only one and all is done: its parts go where the tiles were
    if (warp >= 4 && warp < 12) {
      const int s = (warp - 4) >> 2, dim = (warp & 3) * 32 + lane;
      tc_fence_after();
      uint32_t o[kR];
      tmem_ld16(tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + kColO + 16u * s, o);
      tmem_ld_wait();
      tc_fence_before();
#pragma unroll
      for (int i = 0; i < kR; ++i)
        *reinterpret_cast<uint32_t*>(smem + ((s * kR + i) * kJoinPitch + dim) * 4) = o[i];
      if (dim < kR) *reinterpret_cast<float2*>(smem + kJoinMl + (s * kR + dim) * 8) = ex.ml[s][dim];
    }
    __syncthreads();
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  if (JOIN) {
    __syncwarp();
    cluster_sync();  // every CTA's parts are in its shared memory
    cluster_join<BF16>(p, unit_of(p, static_cast<int>(blockIdx.x)), smem, kR);
    cluster_sync();  // none leaves while another reads them
  }
}

template <bool BF16, bool Q8>
cudaError_t launch_as(const Maps& tm, const Maps8& t8, const Params& p, float scale_log2, int sms, cudaStream_t stream) {
  static std::atomic<unsigned long long> attr_done{0}, attr_done_join{0};
  constexpr int smem = smem_bytes<Q8>();
  constexpr int threads = Cfg<Q8>::kThreads;
  if (p.pl.join) {
    const cudaError_t e = ensure_smem_limit(prefix_attn_few<BF16, Q8, true>, smem, attr_done_join);
    if (e != cudaSuccess) return e;
    return launch_clusters(prefix_attn_few<BF16, Q8, true>, p.pl.nch, dim3(p.pl.units), dim3(threads), smem, stream, tm,
                           t8, p, scale_log2);
  }
  const cudaError_t e = ensure_smem_limit(prefix_attn_few<BF16, Q8, false>, smem, attr_done);
  if (e != cudaSuccess) return e;
  const int grid = p.pl.units < sms ? p.pl.units : sms;
  return launch_dependent(prefix_attn_few<BF16, Q8, false>, dim3(grid), dim3(threads), smem, stream, tm, t8, p,
                          scale_log2);
}

}  // namespace

cudaError_t pa::launch_few(const Maps& tm, const Maps8* t8, const Params& p, bool bf16, float scale_log2, int sms,
                           cudaStream_t s) {
  static const Maps8 none{};
  if (t8) {
    return bf16 ? launch_as<true, true>(tm, *t8, p, scale_log2, sms, s)
                : launch_as<false, true>(tm, *t8, p, scale_log2, sms, s);
  }
  return bf16 ? launch_as<true, false>(tm, none, p, scale_log2, sms, s)
              : launch_as<false, false>(tm, none, p, scale_log2, sms, s);
}

}  // namespace qi
