// Attention of a batch whose sequences share a prefix of keys (one prompt's K/V)
// and have keys of their own, on the 5th-generation tensor cores.
//
// Row (b, t, hq) of a batch of B sequences with T query rows and Hq heads sees the
// P prefix keys and the first lim(b, t) of sequence b's own keys of head hq / G
// (G = Hq / Hkv), lim = own_len[b], or with `causal` own_len[b] - T + t + 1 (the
// sequence's last query row sees all of its keys), clamped to 0 .. own_len[b]:
//   s_j = scale q.k_j,  o = sum_j 2^(s_j log2 e - m) v_j / sum_j 2^(s_j log2 e - m).
// A row without a key is zero. Keys are visited in 128-key tiles with a running
// maximum and sum, so scores never reach memory.
//
// Work unit: a block of up to 128 query rows of one key head against a run of key
// tiles. The G heads of a group and the tokens of a block share the key tiles, so
// they are the rows of one MMA. Two decompositions (make_plan):
//   joint   block = tb tokens of one sequence; its tiles are the prefix's, then the
//           sequence's own. For blocks that fill the 128 MMA rows.
//   packed  the prefix is visited once for rb sequences together (T G rows each),
//           and each sequence's own keys by units of their own. For few query rows
//           per sequence, where a joint unit would read the whole prefix for T G of
//           the MMA's 128 rows.
// Where the units would not fill the SMs, or leave a ragged last wave, a unit's
// tiles are cut into chunks. Up to kJoinMost chunks of a joint block can be one
// cluster that adds its parts in distributed shared memory (cluster_join, JOIN: one
// launch, one unit per CTA); otherwise each writes its unnormalised O with its
// maximum and sum, and merge_partials joins a row's parts. Both in a fixed order, no
// atomics. Blocks of at most 16 rows may go to the kernel of prefix_attention_few.cu.
//
// The inside of a unit is that of the block-causal kernel (attention.cu): one CTA
// per SM, K and V rings filled by TMA, S and the two key halves' O in tensor
// memory, P written back there as the A operand of P V, separate Q K^T and P V
// issuing threads, two softmax warpgroups of one key half each, an epilogue
// warpgroup. What differs: Q comes by a five-dimensional tensor map whose box
// gathers the block's (sequence, token, head of the group) rows; K and V by maps
// over the prefix and over the own keys with the caller's strides; and rows of an
// own V tile at or past own_len are set to zero in shared memory before the
// product, so that whatever the cache holds there (0 x NaN is NaN) cannot reach O.
// P is rounded to the operands' 16-bit type, as the tensor cores need it: an error
// of half a step of that type per term, as large as the rounding of the output (in
// fp16, of at most 2^-32 of the row's largest P where P is below 2^-21 of it; kLift).
//
// Measured: 4 x 4096 rows over 407 shared and 4096 own keys each, 32 heads: 900 to 960 us,
// 1260 to 1340 TFLOP/s, 65 to 70 % of the library product's rate, the clock at its power limit. A
// tile takes 1770 cycles from one S to the next: Q K^T is issued about 500 after S has been
// read, runs for 512 and more beside the other product, and is seen 150 later; the softmax
// (65 to load S, 310 for the maximum, 660 for the exponentials, 300 to wait for P's place and
// to store it) fills 1350 of them. Between two units 2500 cycles go to the epilogue's reads of
// tensor memory, which is what small cases show: 3 x 777 causal rows over 2048 + 1201 keys, 4
// key heads, 84.5 us, 62 %. 32 single tokens over 8192 shared rows, 8
// key heads: 26.6 us with the merge, 46 % of HBM: the CTAs with a prefix unit have 15 tiles, the others 8.
#include <climits>
#include <cstdarg>
#include <cstdio>
#include <mutex>

#include "../../include/qidit.h"
#include "prefix_attention.cuh"

namespace qi {
using namespace pa;
namespace {

constexpr int kRows = 128;                    // MMA rows: query rows per block at most
constexpr int kKStages = 2;  // (a third measured 1 % slower at 1024^2)
constexpr int kVStages = 2;
constexpr int kQBufs = 2;                     // the next unit's Q loads while this one's tiles run
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 0;                 // O_h at kColO + 128 h
constexpr uint32_t kColS = 256;
constexpr uint32_t kColP = 384;               // buffer b at kColP + 64 b, half h at + 32 h
constexpr int kThreads = 512;
// (152 for the softmax warps, with which they spill: 1 to 2.5 % slower; 168: 1 to 3 %)
constexpr uint32_t kRegsLow = 96, kRegsHigh = 160, kRegsEpi = 96;
static_assert(kRegsLow + 2 * kRegsHigh + kRegsEpi == 4 * 128, "register split must equal the launch allotment");
// setmaxnreg.dec may only lower and setmaxnreg.inc only raise the launch's 128
static_assert(kRegsLow <= 128 && kRegsHigh >= 128 && kRegsEpi <= 128 && kRegsLow % 8 == 0 && kRegsHigh % 8 == 0 &&
                  kRegsEpi % 8 == 0,
              "setmaxnreg direction and granularity");

// A unit's numbers for the softmax and epilogue warps, worked out once, by the K producer, which
// is ahead of them: each warp doing it itself between two units held the next unit's first
// tile up by 700 cycles.
constexpr int kMessages = 4;
struct __align__(16) Message {
  int n, pn, p0, o0;
  int t0, b0, len, rows;
  int h, u;
  long long slot;
};

// mbarriers, as in attention.cu
enum : int {
  kKFull = 0,
  kKEmpty = kKFull + kKStages,
  kVFull = kKEmpty + kKStages,
  kVEmpty = kVFull + kVStages,
  // rows past own_len of a unit's last V tile cleared; one per stage, so that the next one cannot
  // complete before the issuer has seen this one (units may have one tile each)
  kVClean = kVEmpty + kVStages,
  kQFull = kVClean + kVStages,
  kQEmpty = kQFull + kQBufs,
  kSFull = kQEmpty + kQBufs,
  kSFree = kSFull + 1,
  kPFull = kSFree + 1,
  kPvDone = kPFull + 4,
  kOFull = kPvDone + 4,
  kOEmpty = kOFull + 1,
  kLFull = kOEmpty + 1,  // the unit's row sums and maxima in shared memory (8 softmax warps)
  kLFree = kLFull + 1,   // ... read by the epilogue (4 warps)
  kUFull = kLFree + 1,   // [message] a unit's numbers in shared memory, from the K producer
  kUEmpty = kUFull + kMessages,  // [message] ... read by the softmax and epilogue warps (12)
  kDrainQK = kUEmpty + kMessages,
  kDrainPV = kDrainQK + 1,
  kNumBars = kDrainPV + 1
};
__device__ __forceinline__ uint32_t bar_count(int i) {
  if (i >= kUEmpty && i < kUEmpty + kMessages) return 12;
  if (i == kSFree || i == kLFull) return 8;
  if ((i >= kPFull && i < kPFull + 4) || i == kOEmpty || i == kLFree) return 4;
  return 1;
}
constexpr int kSmem = (kQBufs + kKStages + kVStages) * kTile + 1024 + kNumBars * 8 + 16 + 2 * 2 * kRows * 4 + 16 +
                      kMessages * static_cast<int>(sizeof(Message));
static_assert(kSmem <= 227 * 1024, "shared memory over the per-block limit");

template <bool BF16, bool JOIN>
__global__ void __launch_bounds__(kThreads, 1)
    prefix_attn_tc(const __grid_constant__ Maps tm, const __grid_constant__ Params p, float scale_log2) {
  constexpr uint32_t kIdescQK = BF16 ? idesc_bf16_f32(128, kKeys) : idesc_f16_f32(128, kKeys);
  constexpr uint32_t kIdescPV = BF16 ? idesc_bf16_f32_bmn(128, 128) : idesc_f16_f32_bmn(128, 128);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;
  uint8_t* sK = sQ + kQBufs * kTile;
  uint8_t* sV = sK + kKStages * kTile;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sV + kVStages * kTile);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + kNumBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  float* lsum = reinterpret_cast<float*>(tmem_slot + 4);  // [half][kRows]
  float* msum = lsum + 2 * kRows;
  Message* messages = reinterpret_cast<Message*>((reinterpret_cast<uintptr_t>(msum + 2 * kRows) + 15) & ~uintptr_t(15));

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int total = p.pl.units;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kNumBars; ++i) mbar_init(&bars[i], bar_count(i));
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tm.qp);
    prefetch_tmap(&tm.qo);
    prefetch_tmap(&tm.pk);
    prefetch_tmap(&tm.k);
  }
  if (warp == 2 && lane == 0) {
    prefetch_tmap(&tm.pv);
    prefetch_tmap(&tm.v);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_dep_wait();
  grid_dep_launch_dependents();

  if (warp < 4) {
    regs_release<kRegsLow>();
    if (warp == 2) {
      // ---------------- V tiles: lane 0 loads them; the whole warp clears the rows past
      // own_len of a sequence's last tile. Every lane walks the same units; lane 0's failure
      // only stops its waits and loads, so the warp meets at every cleared tile.
      uint32_t t = 0;
      bool ok = true;
      for (int u = blockIdx.x; u < total; u += gridDim.x) {
        const Unit un = unit_of(p, u);
        if (lane == 0 && ok) {
          for (int j = 0; j < un.n; ++j) {
            const uint32_t tt = t + j, st = tt % kVStages;
            if (*abort_flag || !mbar_wait(&bars[kVEmpty + st], ((tt / kVStages) & 1u) ^ 1u)) {
              if (!*abort_flag) report_error(p.err, kErrTimeoutProducer);
              *abort_flag = 1;
              t = tt;  // tiles issued, for the drain below
              ok = false;
              break;
            }
            const bool pre = j < un.pn;
            const CUtensorMap* m = pre ? &tm.pv : &tm.v;
            const int row = (pre ? un.p0 + j : un.o0 + j - un.pn) * kKeys;
            const int bs = pre ? 0 : un.b0;
            mbar_arrive_expect_tx(&bars[kVFull + st], kTile);
            tma_load_4d(sV + st * kTile, m, &bars[kVFull + st], 0, un.h, row, bs);
            tma_load_4d(sV + st * kTile + kBox, m, &bars[kVFull + st], 64, un.h, row, bs);
          }
        }
        if (ok) t += un.n;
        if (un.clear) {
          const uint32_t last = t - 1, st = last % kVStages;
          if (lane == 0 && ok && !mbar_wait(&bars[kVFull + st], (last / kVStages) & 1u)) {
            if (!*abort_flag) report_error(p.err, kErrTimeoutProducer);
            *abort_flag = 1;
            ok = false;
          }
          if (__shfl_sync(0xffffffffu, static_cast<int>(ok), 0)) {
            // rows r0 .. 127 of both 64-dim boxes (a row's 128 bytes stay within the row
            // under the swizzle)
            const int r0 = un.len - (un.o0 + un.on - 1) * kKeys;
            const int n16 = (kKeys - r0) * 8;
            uint8_t* base = sV + st * kTile + r0 * 128;
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
      if (lane == 0) {
        for (uint32_t i = t > kVStages ? t - kVStages : 0; i < t; ++i)
          if (!mbar_wait(&bars[kVFull + i % kVStages], (i / kVStages) & 1u)) report_error(p.err, kErrTimeoutDrain);
      }
    } else if (warp == 3) {
      // ---------------- P V issuer: nothing between its waits but what it must decide; a
      // flag read for every tile here cost 4 % of a 1024^2 image's time. The issuing warps walk
      // as a whole, so that the descriptors are uniform, and one lane issues: by a lane alone the
      // causal case above took 91.2 us.
      const uint64_t vdesc0 = sw128_mnmajor_desc(smem_u32(sV), kBox, 1024);
      uint32_t t = 0;
      uint32_t ku = 0, cleared = 0;
      bool ok = true;
      for (int u = blockIdx.x; ok && u < total; u += gridDim.x) {
        const Unit un = unit_of(p, u);
        if (un.n == 0) continue;
        ok = __all_sync(0xffffffffu, !*abort_flag);
        if (!ok) break;
        for (int j = 0; j < un.n; ++j, ++t) {
          const uint32_t b = t & 1u;
          const uint32_t st = t % kVStages;
          ok = (j > 0 || ku == 0 || mbar_wait(&bars[kOEmpty], (ku - 1) & 1u)) &&
               mbar_wait(&bars[kVFull + st], (t / kVStages) & 1u);
          if (un.clear && j + 1 == un.n) {
            ok = ok && mbar_wait(&bars[kVClean + st], (cleared >> st) & 1u);
            cleared ^= 1u << st;  // the stage's phase
          }
          const uint64_t vd = vdesc0 + ((st * kTile) >> 4);
          for (int h = 0; h < 2; ++h) {
            ok = __all_sync(0xffffffffu, ok && mbar_wait(&bars[kPFull + b * 2 + h], (t >> 1) & 1u));
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                mma_ts(tmem + kColO + 128u * h, tmem + kColP + b * 64 + h * 32 + k * 8,
                       vd + ((static_cast<uint32_t>(4 * h + k) * 2048) >> 4), kIdescPV, (j > 0 || k > 0) ? 1u : 0u);
              mma_commit(&bars[kPvDone + b * 2 + h]);
              if (h == 1) {
                mma_commit(&bars[kVEmpty + st]);
                if (j + 1 == un.n) mma_commit(&bars[kOFull]);
              }
            }
            __syncwarp();
          }
          if (!ok) break;
        }
        if (!ok) break;
        ++ku;
      }
      if (elect_one()) {
        if (!ok && !*abort_flag) report_error(p.err, kErrTimeoutMma);
        if (!ok) *abort_flag = 1;
        mma_commit(&bars[kDrainPV]);
        if (!mbar_wait(&bars[kDrainPV], 0)) report_error(p.err, kErrTimeoutDrain);
      }
      __syncwarp();
    } else if (warp == 0) {
      // ---------------- TMA producer of the K tiles and of each unit's Q rows (lane 0)
      if (lane == 0) {
      uint32_t t = 0;
      uint32_t nq = 0, nm = 0;
      bool ok = true;
      for (int u = blockIdx.x; ok && u < total; u += gridDim.x) {
        const Unit un = unit_of(p, u);
        const uint32_t mb = nm % kMessages;
        if (*abort_flag || !mbar_wait(&bars[kUEmpty + mb], ((nm / kMessages) & 1u) ^ 1u)) {
          if (!*abort_flag) report_error(p.err, kErrTimeoutProducer);
          *abort_flag = 1;
          break;
        }
        messages[mb] = {un.n, un.pn, un.p0, un.o0, un.t0, un.b0, un.len, un.rows, un.h, u, un.slot};
        mbar_arrive(&bars[kUFull + mb]);
        ++nm;
        if (un.n == 0) continue;
        const uint32_t qb = nq % kQBufs;
        if (*abort_flag || !mbar_wait(&bars[kQEmpty + qb], ((nq / kQBufs) & 1u) ^ 1u)) {
          if (!*abort_flag) report_error(p.err, kErrTimeoutProducer);
          *abort_flag = 1;
          break;
        }
        const CUtensorMap* mq = u < p.pl.units_p ? &tm.qp : &tm.qo;
        mbar_arrive_expect_tx(&bars[kQFull + qb], static_cast<uint32_t>(un.rows) * 256u);  // whole boxes, also past the ends
        tma_load_5d(sQ + qb * kTile, mq, &bars[kQFull + qb], 0, 0, un.h, un.t0, un.b0);
        tma_load_5d(sQ + qb * kTile + kBox, mq, &bars[kQFull + qb], 64, 0, un.h, un.t0, un.b0);
        ++nq;
        for (int j = 0; j < un.n; ++j, ++t) {
          const uint32_t st = t % kKStages;
          if (*abort_flag || !mbar_wait(&bars[kKEmpty + st], ((t / kKStages) & 1u) ^ 1u)) {
            if (!*abort_flag) report_error(p.err, kErrTimeoutProducer);
            *abort_flag = 1;
            ok = false;
            break;
          }
          const bool pre = j < un.pn;
          const CUtensorMap* m = pre ? &tm.pk : &tm.k;
          const int row = (pre ? un.p0 + j : un.o0 + j - un.pn) * kKeys;
          const int bs = pre ? 0 : un.b0;
          mbar_arrive_expect_tx(&bars[kKFull + st], kTile);
          tma_load_4d(sK + st * kTile, m, &bars[kKFull + st], 0, un.h, row, bs);
          tma_load_4d(sK + st * kTile + kBox, m, &bars[kKFull + st], 64, un.h, row, bs);
        }
      }
      for (uint32_t i = t > kKStages ? t - kKStages : 0; i < t; ++i)
        if (!mbar_wait(&bars[kKFull + i % kKStages], (i / kKStages) & 1u)) report_error(p.err, kErrTimeoutDrain);
      for (uint32_t i = nq > kQBufs ? nq - kQBufs : 0; i < nq; ++i)
        if (!mbar_wait(&bars[kQFull + i % kQBufs], (i / kQBufs) & 1u)) report_error(p.err, kErrTimeoutDrain);
      }
      __syncwarp();
    } else {
      // ---------------- Q K^T issuer
      const uint64_t qdesc0 = sw128_kmajor_desc(smem_u32(sQ));
      const uint64_t kdesc0 = sw128_kmajor_desc(smem_u32(sK));
      uint32_t t = 0;
      uint32_t ku = 0;
      bool ok = true;
      for (int u = blockIdx.x; ok && u < total; u += gridDim.x) {
        const Unit un = unit_of(p, u);
        if (un.n == 0) continue;
        const uint32_t qb = ku % kQBufs;
        ok = __all_sync(0xffffffffu, !*abort_flag && mbar_wait(&bars[kQFull + qb], (ku / kQBufs) & 1u));
        if (!ok) break;
        tc_fence_after();
        const uint64_t qdesc = qdesc0 + ((qb * kTile) >> 4);
        for (int j = 0; j < un.n; ++j, ++t) {
          const uint32_t st = t % kKStages;
          ok = __all_sync(0xffffffffu, (t < 1 || mbar_wait(&bars[kSFree], (t - 1) & 1u)) &&
                                           mbar_wait(&bars[kKFull + st], (t / kKStages) & 1u));
          if (!ok) break;
          tc_fence_after();
          const uint64_t kd = kdesc0 + ((st * kTile) >> 4);
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < kHeadDim / 16; ++k) {
              const uint32_t off = static_cast<uint32_t>(((k >> 2) * kBox + (k & 3) * 32) >> 4);
              mma_ss(tmem + kColS, qdesc + off, kd + off, kIdescQK, k > 0 ? 1u : 0u);
            }
            mma_commit(&bars[kSFull]);
            mma_commit(&bars[kKEmpty + st]);
            if (j + 1 == un.n) mma_commit(&bars[kQEmpty + qb]);
          }
          __syncwarp();
        }
        if (!ok) break;
        ++ku;
      }
      if (elect_one()) {
        if (!ok) {
          report_error(p.err, kErrTimeoutMma);
          *abort_flag = 1;
        }
        mma_commit(&bars[kDrainQK]);
        if (!mbar_wait(&bars[kDrainQK], 0)) report_error(p.err, kErrTimeoutDrain);
      }
      __syncwarp();
    }
  } else if (warp < 12) {
    regs_acquire<kRegsHigh>();
    // ---------------- softmax: warps 4..7 keys 0-63, warps 8..11 keys 64-127 of every
    // tile; thread = one query row's half
    const int h = warp >= 8 ? 1 : 0;
    const int quarter = warp & 3;
    const int rit = quarter * 32 + lane;
    const int tok = quot(p.d_G, rit);  // the row's token within a joint / own block
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t tO = tmem + lane_off + kColO + 128u * h;
    const uint64_t sc2 = f2_pack(scale_log2, scale_log2);
    uint32_t t = 0;
    uint32_t ku = 0, km = 0;
    bool ok = true;
    for (int u = blockIdx.x; u < total; u += gridDim.x, ++km) {
      const uint32_t mb = km % kMessages;
      ok = __all_sync(0xffffffffu, mbar_wait(&bars[kUFull + mb], (km / kMessages) & 1u));
      if (!ok) break;
      const Message un = messages[mb];
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[kUEmpty + mb]);
      if (un.n == 0) continue;
      const int lim_own = own_lim(p, un.len, un.t0 + tok, p.T);
      // A warp whose 32 rows lie past the block's has nothing to compute: it only keeps the
      // barriers' counts (its lanes of S, P and O hold whatever they held). It still waits
      // for every S, so it is never a phase ahead of the other warps on a P buffer.
      const bool idle = quarter * 32 >= un.rows;
      float m_used = -INFINITY;
      float l = 0.f;
      // keys of this half of the tile that the row sees, counted down by tile (few live values:
      // the loop runs at its register limit, and the tile numbers kept instead cost 1.5 %)
      int left = p.P - un.p0 * kKeys - h * 64;
      const int left_own = lim_own - un.o0 * kKeys - h * 64;
      const int n = un.n, pn = un.pn;
      for (int j = 0; j < n; ++j) {
        const uint32_t tt = t + j;
        const uint32_t b = tt & 1u;
        const bool last = j + 1 == n;
        ok = __all_sync(0xffffffffu, mbar_wait(&bars[kSFull], tt & 1u));
        if (!ok) break;
        if (idle) {
          if (last) {
            ok = __all_sync(0xffffffffu, mbar_wait(&bars[kLFree], (ku & 1u) ^ 1u));
            if (!ok) break;
          }
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&bars[kSFree]);
            mbar_arrive(&bars[kPFull + b * 2 + h]);
            if (last) mbar_arrive(&bars[kLFull]);
          }
          continue;
        }
        tc_fence_after();
        uint32_t r[2][32];
        tmem_ld32(tmem + lane_off + kColS + h * 64, r[0]);
        tmem_ld32(tmem + lane_off + kColS + h * 64 + 32, r[1]);
        tmem_ld_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[kSFree]);
        // keys at or past the row's limit become -inf, whatever their scores are
        if (j == pn) left = left_own;
        if (__any_sync(0xffffffffu, left < 64)) {
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (c * 32 + i >= left) r[c][i] = 0xff800000u;
        }
        left -= kKeys;
        float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int i = 0; i < 32; i += 2)
            mx4[(i >> 1) & 3] = fmax3(mx4[(i >> 1) & 3], __uint_as_float(r[c][i]), __uint_as_float(r[c][i + 1]));
        const float mx = fmaf(fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])), scale_log2, -kLift<BF16>);
        const float m_new = fmaxf(m_used, mx);
        if (j == 0) {
          m_used = m_new;
        } else {
          const bool mine = m_new > m_used + kRescaleLog2;
          if (__any_sync(0xffffffffu, mine)) {
            const uint32_t tp = tt - 1;
            if (!__all_sync(0xffffffffu, mbar_wait(&bars[kPvDone + (tp & 1u) * 2 + h], (tp >> 1) & 1u))) {
              ok = false;
              break;
            }
            tc_fence_after();
            const float alpha = mine ? fast_exp2(m_used - m_new) : 1.0f;
#pragma unroll 1
            for (int c = 0; c < 8; ++c) {
              uint32_t o[16];
              tmem_ld16(tO + c * 16, o);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
              tmem_st16(tO + c * 16, o);
            }
            if (mine) {
              l *= alpha;
              m_used = m_new;
            }
          }
        }
        const float base = m_used == -INFINITY ? 0.f : m_used;
        const uint64_t nm2 = f2_pack(-base, -base);
        uint64_t rs2[4] = {0ull, 0ull, 0ull, 0ull};
        uint32_t pk[2][16];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const uint64_t x2 =
                fma_f32x2(f2_pack(__uint_as_float(r[c][2 * i]), __uint_as_float(r[c][2 * i + 1])), sc2, nm2);
            float x0, x1;
            f2_unpack(x2, x0, x1);
            const float e0 = fast_exp2(x0);
            const float e1 = fast_exp2(x1);
            rs2[i & 3] = add_f32x2(rs2[i & 3], f2_pack(e0, e1));
            pk[c][i] = pack16<BF16>(e0, e1);
          }
        }
        if (tt >= 2) {
          ok = __all_sync(0xffffffffu, mbar_wait(&bars[kPvDone + b * 2 + h], ((tt - 2) >> 1) & 1u));
          if (!ok) break;
          tc_fence_after();
        }
        const uint32_t tP = tmem + lane_off + kColP + b * 64 + h * 32;
        tmem_st16(tP, pk[0]);
        tmem_st16(tP + 16, pk[1]);
        float s[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) f2_unpack(rs2[i], s[2 * i], s[2 * i + 1]);
        l += ((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7]));
        tmem_st_wait();
        tc_fence_before();
        if (last) {
          ok = __all_sync(0xffffffffu, mbar_wait(&bars[kLFree], (ku & 1u) ^ 1u));
          if (!ok) break;
          lsum[h * kRows + rit] = l;
          msum[h * kRows + rit] = m_used;
        }
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&bars[kPFull + b * 2 + h]);
          if (last) mbar_arrive(&bars[kLFull]);
        }
      }
      if (!ok) break;
      t += n;
      ++ku;
    }
    if (!ok) {
      if (lane == 0) report_error(p.err, kErrTimeoutEpilogue);
      *abort_flag = 1;
    }
  } else {
    regs_release<kRegsEpi>();
    // ---------------- epilogue (warps 12..15), thread = one row of the block
    const int quarter = warp & 3;
    const int rit = quarter * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const int tok = quot(p.d_G, rit);
    const int g = rit - tok * p.pl.G;
    bool ok = true;
    uint32_t ku = 0, km = 0;
    for (int u = blockIdx.x; ok && u < total; u += gridDim.x, ++km) {
      const uint32_t mb = km % kMessages;
      ok = __all_sync(0xffffffffu, mbar_wait(&bars[kUFull + mb], (km / kMessages) & 1u));
      if (!ok) break;
      const Message un = messages[mb];
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[kUEmpty + mb]);
      // where the row goes: token and sequence (a prefix block runs over sequences)
      int b = un.b0, tk = un.t0 + tok;
      if (u < p.pl.units_p) {
        const int q = quot(p.d_T, tok);
        b += q;
        tk = tok - q * p.T;
      }
      const bool mine = rit < un.rows && tk < p.T && b < p.B;
      uint16_t* orow = p.o + b * p.ob + tk * p.orow + static_cast<long long>(un.h * p.pl.G + g) * p.oh;
      if (un.n == 0) {
        if (JOIN) *reinterpret_cast<float2*>(smem + kJoinMl + rit * 8) = make_float2(-INFINITY, 0.f);
        // no key at all: a joint unit that is its row's only one writes zeros
        if (!JOIN && !p.pl.split && mine) {
#pragma unroll
          for (int i = 0; i < 16; ++i) reinterpret_cast<uint4*>(orow)[i] = make_uint4(0u, 0u, 0u, 0u);
        }
        continue;
      }
      ok = __all_sync(0xffffffffu, mbar_wait(&bars[kLFull], ku & 1u));
      if (!ok) break;
      const float m0 = msum[rit], m1 = msum[kRows + rit];
      const float l0 = lsum[rit], l1 = lsum[kRows + rit];
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[kLFree]);
      const float mm = fmaxf(m0, m1);
      // a half without a visible key has m = -inf and weight 0; in a row without one both
      // sums and O are 0 already (or NaN, if its scores are)
      const float a0 = mm == -INFINITY ? 1.f : fast_exp2(m0 - mm);
      const float a1 = mm == -INFINITY ? 1.f : fast_exp2(m1 - mm);
      const float den = l0 * a0 + l1 * a1;
      const float inv = JOIN || p.pl.split ? 1.f : (den == 0.f ? 0.f : 1.f / den);
      const float w0 = a0 * inv, w1 = a1 * inv;
      if (!JOIN && p.pl.split && mine) p.ml[un.slot + rit] = make_float2(mm, den);
      ok = __all_sync(0xffffffffu, mbar_wait(&bars[kOFull], ku & 1u));
      if (!ok) break;
      if (quarter * 32 >= un.rows) {  // none of the warp's rows are the block's
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[kOEmpty]);
        ++ku;
        continue;
      }
      tc_fence_after();
      if (JOIN) {
        // (the unit is the CTA's only one and its products are done: the rings are free)
        *reinterpret_cast<float2*>(smem + kJoinMl + rit * 8) = make_float2(mm, den);
      }
      // 16 columns of both halves at a time, the next ones loading while these are stored
      const uint32_t tO = tmem + lane_off + kColO;
      const uint64_t w00 = f2_pack(w0, w0), w11 = f2_pack(w1, w1);
      uint32_t oa[2][16], ob[2][16];
      tmem_ld16(tO, oa[0]);
      tmem_ld16(tO + 128, ob[0]);
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        tmem_ld_wait();
        if (c < 7) {
          tmem_ld16(tO + (c + 1) * 16, oa[(c + 1) & 1]);
          tmem_ld16(tO + 128 + (c + 1) * 16, ob[(c + 1) & 1]);
        } else {
          // O_0 and O_1 are in registers: the next unit's first P V may overwrite them
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars[kOEmpty]);
        }
        const uint32_t* x = oa[c & 1];
        const uint32_t* y = ob[c & 1];
        if (mine) {
          float ov[16];
#pragma unroll
          for (int i = 0; i < 8; ++i)
            f2_unpack(fma_f32x2(f2_pack(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])), w00,
                                mul_f32x2(f2_pack(__uint_as_float(y[2 * i]), __uint_as_float(y[2 * i + 1])), w11)),
                      ov[2 * i], ov[2 * i + 1]);
          if (JOIN) {
            float4* d = reinterpret_cast<float4*>(smem + (rit * kJoinPitch + c * 16) * 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) d[i] = make_float4(ov[4 * i], ov[4 * i + 1], ov[4 * i + 2], ov[4 * i + 3]);
          } else if (p.pl.split) {
            float* d = p.part + (un.slot + rit) * kHeadDim + c * 16;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              uint32_t r[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) r[k] = __float_as_uint(ov[8 * i + k]);
              store32(d + 8 * i, r);
            }
          } else {
            uint32_t r[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) r[k] = pack16<BF16>(ov[2 * k], ov[2 * k + 1]);
            if (p.o32) {  // (a row a lane: half the line accesses of 16-byte stores; eight 384^2 images 86.2 -> 85.1 us)
              store32(orow + c * 16, r);
            } else {
              uint4* d = reinterpret_cast<uint4*>(orow + c * 16);
              d[0] = make_uint4(r[0], r[1], r[2], r[3]);
              d[1] = make_uint4(r[4], r[5], r[6], r[7]);
            }
          }
        }
      }
      ++ku;
    }
    if (!ok) {
      if (lane == 0) report_error(p.err, kErrTimeoutEpilogue);
      *abort_flag = 1;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  if (JOIN) {
    __syncwarp();
    cluster_sync();  // every CTA's part is in its shared memory
    cluster_join<BF16>(p, unit_of(p, static_cast<int>(blockIdx.x)), smem, kRows);
    cluster_sync();  // none leaves while another reads it
  }
}

// Joins an output row's partials (prefix chunks in order, then own chunks) by their maxima
// and sums: kMergeWarps / W rows per block, W warps per row. Warp w of a row takes parts w,
// w + W, ...; the W sums are added in order. Chunks without a tile were not written; they are
// told from the lengths, as the units told them. What comes before the wait reads only what
// was complete before the attention kernel began.
constexpr int kMergeWarps = 8;
template <bool BF16, int W, typename P>
__global__ void __launch_bounds__(kMergeWarps * 32) merge_partials(const __grid_constant__ P p) {
  __shared__ float4 sacc[kMergeWarps][32];
  __shared__ float sden[kMergeWarps];
  const Plan& pl = p.pl;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int w = warp % W;
  const long long row = static_cast<long long>(blockIdx.x) * (kMergeWarps / W) + warp / W;
  bool in = row < static_cast<long long>(p.B) * p.T * p.Hq;  // below 2^31
  const int r = in ? static_cast<int>(row) : 0;
  const int bt = quot(p.d_Hq, r), hq = r - bt * p.Hq;
  const int b = quot(p.d_T, bt), t = bt - b * p.T;
  const int h = quot(p.d_G, hq), g = hq - h * pl.G;
  const int qb = quot(p.d_tb, t);
  const int tq = query_rows(p, b);
  if (kPaged<P>) in = in && t < tq;  // rows past a sequence's stay as they are
  const int ot = own_tiles(p, own_len_of(p, b), qb * pl.tb, pl.tb, tq);
  const long long hb = static_cast<long long>(h) * p.B + b;
  const long long unit_o =
      (pl.by_block ? (pl.nqb - 1 - qb) * static_cast<long long>(p.Hkv) * p.B + hb : hb * pl.nqb + qb) * pl.nch;
  const long long slot_o =
      (static_cast<long long>(pl.units_p) * pl.rows_p + unit_o * pl.rows_o) * pl.per + (t - qb * pl.tb) * pl.G + g;
  const int parts_o = quot(p.d_ct, ot + (pl.packed ? 0 : pl.pt) + pl.ct - 1) * pl.per;
  long long slot_p = 0;
  int parts_p = 0;
  if (pl.packed) {
    const int pb = quot(p.d_rb, b);
    slot_p =
        (static_cast<long long>(h) * pl.npb + pb) * pl.nchp * pl.per * pl.rows_p + ((b - pb * pl.rb) * p.T + t) * pl.G + g;
    parts_p = pl.nchp * pl.per;
  }
  const int n = in ? parts_p + parts_o : 0;
  const auto slot = [&](int i) {
    return i < parts_p ? slot_p + static_cast<long long>(i) * pl.rows_p
                       : slot_o + static_cast<long long>(i - parts_p) * pl.rows_o;
  };
  grid_dep_wait();
  grid_dep_launch_dependents();
  float m = -INFINITY;
  for (int i = lane; i < n; i += 32) m = fmaxf(m, p.ml[slot(i)].x);
#pragma unroll
  for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
  float den = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int i = w; i < n; i += W) {
    const long long s = slot(i);
    const float2 ml = p.ml[s];
    const float4 v = reinterpret_cast<const float4*>(p.part + s * kHeadDim)[lane];
    // a part in which the row sees no key has m = -inf and sum 0 (and O may not have been
    // written); m = -inf with another sum is a row of NaN scores, which stays one
    const bool none = ml.x == -INFINITY && ml.y == 0.f;
    const float a = m == -INFINITY ? 1.f : fast_exp2(ml.x - m);
    den += none ? 0.f : ml.y * a;
    acc.x += none ? 0.f : v.x * a;
    acc.y += none ? 0.f : v.y * a;
    acc.z += none ? 0.f : v.z * a;
    acc.w += none ? 0.f : v.w * a;
  }
  if (W > 1) {
    sacc[warp][lane] = acc;
    if (lane == 0) sden[warp] = den;
    __syncthreads();
    if (w != 0) return;
#pragma unroll
    for (int i = 1; i < W; ++i) {
      const float4 v = sacc[warp + i][lane];
      den += sden[warp + i];
      acc.x += v.x;
      acc.y += v.y;
      acc.z += v.z;
      acc.w += v.w;
    }
  }
  if (!in) return;
  const float inv = den == 0.f ? 0.f : 1.f / den;
  uint16_t* orow = p.o + b * p.ob + t * p.orow + static_cast<long long>(hq) * p.oh;
  reinterpret_cast<uint2*>(orow)[lane] =
      make_uint2(pack16<BF16>(acc.x * inv, acc.y * inv), pack16<BF16>(acc.z * inv, acc.w * inv));
}

// ---------------------------------------------------------------- host

qi_status op_fail(qi_status st, const char* fmt, ...) {
  char buf[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  set_last_error(buf);
  return st;
}

int ceil_div(int a, int b) { return (a + b - 1) / b; }

// Chooses the decomposition from sizes alone (own lengths, which only the device knows, count
// as S): the one whose busiest CTA has the least to do. Time is counted in units of a key
// tile of the 128-row kernel, about 0.9 us: a unit costs its tiles plus a fill and an
// epilogue that grows with its rows, splitting costs kMergeTiles for the partials and the
// second launch, a cluster's join by its rows. The few-row kernel reads an 8-bit prefix as it
// is; the other first has it turned into 16 bits (a launch, and kConvert a 2^20 values:
// written and read again). Over 90 random calls the choice was within 3 % (geometric mean;
// 55 % at worst, where a few-row tile comes from L2 in half the time) of the best of joint,
// packed and joined units of both kernels. Measured, 128-row against few-row kernel, us:
//   16 sequences, 32 key heads, 8192 + 256, 16-bit prefix   43.7 / 38.1      8-bit   75 / 40.6
//   32 sequences, groups of 4, 8192 + 512, 16-bit   29.3 / 31.7      8-bit   34.6 / 61.7
//   7 sequences of 5 tokens, 16 bits   12.6 / 11.0      8 sequences of 16 rows, 8 bits   26.1 / 44.1
//   one sequence over 8192 prefix rows, 32 heads   28.0 / 26.2
//   64 sequences, 2048 own keys   87.6 / 86.7      2 sequences, 8 heads, 300 + 40   7.4 / 6.4
// and a cluster's join against partials and a merge (few-row kernel): the 7 sequences 11.0 / 11.9,
// 4 sequences of 4 tokens, groups of 4, 1000 + 1000 keys 10.1 / 9.8, the last 6.4 / 7.0.
//
// Order of the joint units: head-major, so that the CTAs running at one time share a few
// heads' K/V in L2; with `causal`, whose units differ in length, last row blocks first
// over all heads and sequences, so that the CTAs' sums of lengths agree (3 x 777 rows over
// 2048 + 1201 keys, 4 key heads: 90.4 us, head-major 97.0, when chosen), as long as all K/V
// stay in half of the L2.
struct Rate {
  float tile, tile8, unit, row;  // a 16-bit tile, a tile of codes, a unit, each of its rows
  float of(int rows) const { return unit + row * static_cast<float>(rows); }
};
constexpr Rate kFullRate{1.f, 1.f, 1.5f, 1.f / 128}, kFewRate{0.7f, 1.5f, 0.6f, 0.09f};
constexpr float kMergeTiles = 3.f, kPartRows = 5300.f;  // and a unit per so many partial rows written and read
constexpr float kConvert = 0.5f, kConvertStart = 2.5f;
constexpr float kStart = 3.f;      // of a kernel whose CTAs walk the units
constexpr float kJoinTiles = 2.6f, kJoinRow = 1.f / 32;  // start of a CTA in a cluster and its join; each row
constexpr long long kL2Half = 64ll << 20;
// Of a unit, in 1/kLine of a tile, where pieces are cut: 2, 3, 4, 6 for full blocks: 6 x 777 rows 100, 94, 91, 90 us,
// 4 x 2048 180, 176, 171, 173; 4, 8, 12 for few rows: 128 single tokens over up to 900 rows, 32 heads, 214, 198, 191
// (6, 8, 10 since: 179, 180, 182), 200 x 4 rows 124, 122, 122
constexpr int kFullCost = 4, kFewCost = 8;
// The next four against other values: geometric mean over 8 random calls whose plan the value changes. Larger ones
// would do better for three of them.
constexpr float kFlowStart = 5.f;           // cutting them, and a second launch. 0: 29 % longer. 10: 39 % shorter, by few row blocks
                                            // whose pieces leave many parts (1 x 77 rows over 9008 keys 46 -> 14.5 us)
constexpr float kSpan = 80 << 20;           // bytes of keys and values that row blocks share in a round of pieces
constexpr float kPiece = 24.f;              // tiles of a piece at least. 12: 12 % longer, 48: 1 % longer
constexpr float kApart = 1.1f;             // pieces against units that meet in the L2
constexpr float kEvenFrom = 48.f;           // tiles a CTA from which unequal chunks are worth cutting. 12: 28 % longer, 192: 8 %
                                            // shorter (3 x 452 rows over up to 29394 keys 31 % longer, 3 x 85 over 58545 25 % shorter)
constexpr int kFewTiles = 4;                // so few in a unit, and their number does not matter. 1: 18 % longer, 8: 13 % shorter
                                            // (92 x 191 rows over up to 774 keys, 32 heads, 26 % longer)
Plan make_plan(const Sizes& z, int sms) {
  Plan a{};
  a.G = z.Hq / z.Hkv;
  a.by_block = z.causal && (static_cast<long long>(z.B) * z.S + z.P) * z.Hkv * kHeadDim * 4 <= kL2Half;
  a.pt = ceil_div(z.P, kKeys);
  a.ot = ceil_div(z.S, kKeys);
  a.per = 1;
  Plan best = a;
  float best_cost = 3e38f;
  const auto rows_of = [&](Plan& c, int most, bool pack) {
    c.tb = most / c.G < z.T ? most / c.G : z.T;
    c.nqb = ceil_div(z.T, c.tb);
    c.rows_o = c.tb * c.G;
    c.rb = 1;
    c.packed = 0;
    if (pack) {
      c.packed = 1;
      c.rb = most / c.rows_o < z.B ? most / c.rows_o : z.B;
      c.npb = ceil_div(z.B, c.rb);
      c.rows_p = c.rb * c.rows_o;
    }
  };
  const float convert = z.from8 && z.P > 0 ? kConvertStart + kConvert * static_cast<float>(z.P) * z.Hkv * kHeadDim / (1 << 20) : 0.f;
  // pieces can be cut: the line in an int (beyond it, seconds of work, units will do)
  const auto fits = [&](int nqb) { return static_cast<float>(z.B) * nqb * z.Hkv * ((a.ot + 4) * kLine) < 2e9f; };
  // single tokens, or chunks of lengths of their own (q_len) with enough tiles to cut; without q_len the lengths in the
  // cache may differ all the same, and units cut by the longest then leave CTAs idle
  const int nqb_full = z.paged ? ceil_div(z.T, kRows / a.G) : 0;
  const bool even = z.paged && fits(nqb_full) &&
                    (nqb_full == 1 ||
                     (z.ragged && z.B > 1 && static_cast<float>(nqb_full) * z.B * z.Hkv * (a.ot + 2) > kEvenFrom * sms));
  // what a causal chunk's row blocks see of the longest sequence, on average
  const float seen = z.paged && z.causal && z.T < z.S ? 1.f - 0.5f * static_cast<float>(z.T) / static_cast<float>(z.S)
                     : z.paged && z.causal            ? 0.5f
                                                      : 1.f;
  // joint units, every number of chunks that keeps the grid within a few waves
  const auto joint = [&](Plan c, Rate r, bool always_split, float more) {
    const int n = c.pt + c.ot;
    const long long blocks = static_cast<long long>(z.Hkv) * z.B * c.nqb;
    const float each = (c.pt * (z.from8 ? r.tile8 : r.tile) + c.ot * r.tile) / n;
    for (int nch = 1; nch <= n; ++nch) {
      if (nch > 1 && blocks * nch > 4ll * sms) break;  // (at most 4 x SMs rounds of this loop)
      if (even && (nch > 1 || (blocks > sms && n > kFewTiles))) break;
      c.ct = ceil_div(n, nch);
      if (ceil_div(n, c.ct) != nch) continue;
      c.nch = nch;
      c.split = always_split || nch > 1;
      const float waves = static_cast<float>((blocks * nch + sms - 1) / sms);
      const float parts = c.split ? kMergeTiles + static_cast<float>(blocks * nch) * c.rows_o * c.per / kPartRows : 0.f;
      const float cost = kStart + waves * (c.ct * seen * each + r.of(c.rows_o)) + parts + more;
      if (cost < best_cost && blocks * nch <= INT_MAX / 2) {
        best_cost = cost;
        c.units = static_cast<int>(blocks * nch);
        best = c;
      }
    }
  };
  // joint units whose chunks join in a cluster: one unit per CTA, counted by the whole bound (by what causal chunks see
  // 21 of 5483 random calls would change, 8 of which took 16 % less time, 0.49 to 1.14); clusters of more than two leave
  // some SMs of a processing cluster over (of 152: 138 to 144 CTAs in clusters of 3 to 6, 105 of 7)
  const auto joined = [&](Plan c, Rate r, int least, float more) {
    const int n = c.pt + c.ot;
    const long long blocks = static_cast<long long>(z.Hkv) * z.B * c.nqb;
    const float each = (c.pt * (z.from8 ? r.tile8 : r.tile) + c.ot * r.tile) / n;
    for (int nch = least; nch <= n && nch <= kJoinMost; ++nch) {
      c.ct = ceil_div(n, nch);
      if (ceil_div(n, c.ct) != nch || blocks * nch > INT_MAX / 2) continue;
      c.nch = nch;
      c.join = 1;
      const int slots = nch <= 2 ? sms : nch <= 6 ? sms * 9 / 10 : sms * 2 / 3;
      const float waves = static_cast<float>((blocks * nch + slots - 1) / slots);
      if (even && waves > 1.f) continue;
      const float cost = waves * (c.ct * each + r.of(c.rows_o) + kJoinTiles + kJoinRow * static_cast<float>(c.rows_o)) + more;
      if (cost < best_cost) {
        best_cost = cost;
        c.units = static_cast<int>(blocks * nch);
        best = c;
      }
    }
  };
  // the prefix once per rb sequences, own keys by sequence; CTA i has units i, i + SMs, ...
  const auto packed = [&](Plan c, Rate r, float more) {
    c.split = 1;
    const long long blocks = static_cast<long long>(z.Hkv) * z.B;
    const int most = c.pt > c.ot ? c.pt : c.ot;
    for (int ct = 1; ct <= most; ct += 1 + ct / 32) {
      c.ct = ct;
      c.nchp = ceil_div(c.pt, ct);
      c.nch = c.ot ? ceil_div(c.ot, ct) : 1;
      const long long up = static_cast<long long>(z.Hkv) * c.npb * c.nchp, uo = c.ot ? blocks * c.nch : 0;
      if (up + uo > INT_MAX / 2) continue;
      const float unit_p = r.of(c.rows_p) + (z.from8 ? r.tile8 : r.tile) * c.pt / c.nchp;
      const float unit_o = r.of(c.rows_o) + r.tile * c.ot / c.nch;
      float load = 0.f;
      for (long long i : {0ll, up % sms, (up + uo) % sms - 1, static_cast<long long>(sms) - 1}) {
        if (i < 0) continue;
        const long long np = (up - i + sms - 1) / sms, all = (up + uo - i + sms - 1) / sms;
        const float l = np * unit_p + (all - np) * unit_o;
        load = l > load ? l : load;
      }
      const float parts = (static_cast<float>(up) * c.rows_p + static_cast<float>(uo) * c.rows_o) * c.per / kPartRows;
      const float cost = kStart + load + kMergeTiles + parts + more;
      if (cost < best_cost) {
        best_cost = cost;
        c.units_p = static_cast<int>(up);
        c.units = static_cast<int>(up + uo);
        best = c;
      }
    }
  };
  // Even pieces of a cache in pages, where the sequences' shares of the work are known on the device alone
  // (single tokens, chunks of lengths of their own), or where units would leave a ragged wave. Row blocks that
  // share keys follow one another on the line, so the CTAs go over it in rounds of about kSpan bytes of keys, which
  // stay in the L2 meanwhile: 12 x 141 rows over up to 20000 keys (450 MB) in one round 300 us, in rounds of
  // 32, 64, 80, 128 MB 264, 264, 264, 254; all 20000 long 722, then 514, 515, 517, 594; 2048 rows over 32768 keys 768,
  // then 753, 753, 752, 807; 3 x 3461 rows (146 MB) 138, then 150, 144, 137, 139: more rounds are more parts to join.
  // Where the plan has units enough for even waves, chunks of one length keep them (kApart): CTAs that walk
  // neighbouring row blocks from the same key on meet in the L2, and pieces do not (3 x 2461 causal rows, 32 / 16
  // heads: 132 us, in pieces 140; 4 x 4096 image rows 810 and 882). Else pieces: 1024 rows behind 16384, 32 / 8
  // heads, 198 us, in units 209.
  const auto flow = [&](Plan c, Rate r) {
    const long long blocks = static_cast<long long>(z.B) * c.nqb * z.Hkv;
    if (!z.paged || !fits(c.nqb)) return;
    c.nch = c.ct = 1;
    c.cost = c.few ? kFewCost : kFullCost;
    const float each = static_cast<float>(blocks) * (c.ot * seen * r.tile + r.of(c.rows_o)) / sms * (even ? 1.f : kApart);
    const float cost = kStart + kFlowStart + each + kMergeTiles;
    if (cost < best_cost) {
      best_cost = cost;
      c.units = blocks * c.ot < sms ? static_cast<int>(blocks * c.ot) : sms;
      const float span = static_cast<float>(z.B) * c.ot * z.Hkv * (2 * kTile) / kSpan + 0.5f;
      c.flow = static_cast<int>(c.nqb == 1 ? 1.f : span < each / kPiece ? span : each / kPiece);
      c.flow = c.flow < 1 ? 1 : c.flow > kMostRounds ? kMostRounds : c.flow;
      best = c;
    }
  };
  Plan c = a;
  rows_of(c, kRows, false);
  flow(c, kFullRate);
  joint(c, kFullRate, false, convert);
  joined(c, kFullRate, z.paged ? 1 : 2, convert);
  const int rows_seq = z.T * a.G;
  // packed: only if two or more sequences' rows fit one block
  if (z.P > 0 && z.B > 1 && 2 * rows_seq <= kRows) {
    rows_of(c, kRows, true);
    packed(c, kFullRate, convert);
  }
  if (rows_seq <= kFewRows) {
    c = a;
    c.few = 1;
    c.per = 2;
    rows_of(c, kFewRows, false);
    if (!z.paged) joint(c, kFewRate, true, 0.f);
    c.per = 1;
    flow(c, kFewRate);
    c.per = 2;
    joined(c, kFewRate, 1, 0.f);
    if (z.P > 0 && z.B > 1) {
      rows_of(c, kFewRows, true);
      packed(c, kFewRate, 0.f);
    }
  }
  return best;
}

// make_plan weighs hundreds of candidates, which takes longer than a launch: each thread keeps
// the plans of the sizes it met last.
Plan plan_for(const Sizes& z, int sms) {
  struct Entry {
    Sizes z;
    int sms;
    Plan plan;
  };
  static thread_local Entry kept[16];
  unsigned h = static_cast<unsigned>(z.B);
  for (int v : {z.T, z.Hq, z.Hkv, z.P, z.S, z.causal * 16 + (z.from8 ? 1 : 0) + (z.paged ? 2 : 0) + (z.ragged ? 8 : 0), sms})
    h = h * 0x9E3779B1u + static_cast<unsigned>(v);
  Entry& e = kept[(h ^ (h >> 16)) & 15u];
  if (e.sms != sms || e.z.B != z.B || e.z.T != z.T || e.z.Hq != z.Hq || e.z.Hkv != z.Hkv || e.z.P != z.P ||
      e.z.S != z.S || e.z.causal != z.causal || e.z.from8 != z.from8 || e.z.paged != z.paged || e.z.ragged != z.ragged)
    e = Entry{z, sms, make_plan(z, sms)};
  return e.plan;
}

size_t align256(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }
size_t partial_rows(const Plan& pl) {
  if (pl.flow) return static_cast<size_t>(pl.units) * pl.flow * 2 * pl.rows_o;
  return pl.split ? (static_cast<size_t>(pl.units_p) * pl.rows_p +
                     static_cast<size_t>(pl.units - pl.units_p) * pl.rows_o) * pl.per
                  : 0;
}
WsLayout ws_layout(const Plan& pl, int P, int Hkv, bool from8) {
  WsLayout w{};
  const size_t pre = from8 && !pl.few ? align256(static_cast<size_t>(P) * Hkv * kHeadDim * 2) : 0;
  const size_t rows = partial_rows(pl);
  w.pk = 0;
  w.pv = pre;
  w.part = 2 * pre;
  w.ml = w.part + align256(rows * kHeadDim * 4);
  w.rec = w.ml + align256(rows * 8);
  w.total = w.rec + (pl.flow ? align256(static_cast<size_t>(pl.units) * pl.flow * sizeof(int4)) : 0);
  return w;
}

bool map_kv(CUtensorMap* m, const Tensor4& t, int heads, int rows, int batch) {
  const unsigned long long dims[4] = {kHeadDim, static_cast<unsigned long long>(heads),
                                      static_cast<unsigned long long>(rows), static_cast<unsigned long long>(batch)};
  const unsigned long long str[3] = {static_cast<unsigned long long>(t.head) * 2,
                                     static_cast<unsigned long long>(t.row) * 2,
                                     static_cast<unsigned long long>(t.batch) * 2};
  const unsigned box[4] = {64, 1, kKeys, 1};
  return encode_map_nd(m, t.data, false, 4, dims, str, box);
}

bool map_codes(CUtensorMap* m, const uint8_t* codes, int heads, int rows) {
  const unsigned long long dims[3] = {kHeadDim, static_cast<unsigned long long>(heads),
                                      static_cast<unsigned long long>(rows)};
  const unsigned long long str[2] = {kHeadDim, static_cast<unsigned long long>(heads) * kHeadDim};
  const unsigned box[3] = {kHeadDim, 1, kKeys};
  return encode_map_nd(m, codes, true, 3, dims, str, box);
}

// `stall` (test hook): the boxes bring half of the bytes that the kernels wait for, so Q never comes
bool map_q(CUtensorMap* m, const Tensor4& t, int G, int Hkv, int T, int B, int tb, int rb, bool stall) {
  const unsigned long long dims[5] = {kHeadDim, static_cast<unsigned long long>(G),
                                      static_cast<unsigned long long>(Hkv), static_cast<unsigned long long>(T),
                                      static_cast<unsigned long long>(B)};
  const unsigned long long str[4] = {
      static_cast<unsigned long long>(t.head) * 2, static_cast<unsigned long long>(t.head) * G * 2,
      static_cast<unsigned long long>(t.row) * 2, static_cast<unsigned long long>(t.batch) * 2};
  const unsigned box[5] = {stall ? 32u : 64u, static_cast<unsigned>(G), 1, static_cast<unsigned>(tb), static_cast<unsigned>(rb)};
  return encode_map_nd(m, t.data, false, 5, dims, str, box);
}

qi_status check_sizes(const qi_prefix_attn* a) {
  if (!a) return op_fail(QI_ERR_INVALID_ARG, "qi_prefix_attention: NULL argument");
  if (a->dtype != QI_DT_F16 && a->dtype != QI_DT_BF16)
    return op_fail(QI_ERR_INVALID_ARG, "qi_prefix_attention: dtype %d", a->dtype);
  constexpr int kMost = 1 << 24;
  if (a->B < 1 || a->B > 65535 || a->T < 1 || a->T > kMost || a->Hkv < 1 || a->Hkv > 65535 || a->Hq < a->Hkv ||
      a->Hq % a->Hkv != 0 || a->Hq / a->Hkv > kRows || a->P < 0 || a->P > kMost || a->S < 0 || a->S > kMost ||
      (a->P == 0 && a->S == 0) || (a->pk8 && static_cast<long long>(a->P) * a->Hkv >= (1ll << 26)) ||
      static_cast<long long>(a->B) * a->T * a->Hq >= (1ll << 31))
    return op_fail(QI_ERR_SHAPE, "qi_prefix_attention: B %d T %d Hq %d Hkv %d P %d S %d", a->B, a->T, a->Hq, a->Hkv,
                   a->P, a->S);
  return QI_OK;
}

template <bool BF16, typename P>
cudaError_t launch_merge_as(const P& p, cudaStream_t stream) {
  // Warps per row: as many as its parts keep busy, unless the rows alone fill the GPU (1024
  // rows of 16 parts, with the attention before it: 31.6 us at one warp a row, 29.4 at 4 or 8)
  const long long rows = static_cast<long long>(p.B) * p.T * p.Hq;
  const int parts = (p.pl.packed ? p.pl.nchp + p.pl.nch : p.pl.nch) * p.pl.per;
  const int w = rows > 16384 || parts < 4 ? 1 : parts < 16 ? 4 : 8;
  const auto kernel = w == 1   ? merge_partials<BF16, 1, P>
                      : w == 4 ? merge_partials<BF16, 4, P>
                               : merge_partials<BF16, 8, P>;
  const long long per = kMergeWarps / w;
  return launch_dependent(kernel, dim3(static_cast<unsigned>((rows + per - 1) / per)), dim3(kMergeWarps * 32), 0, stream,
                          p);
}

template <bool BF16>
cudaError_t launch(const Maps& tm, const Maps8* t8, const Params& p, float scale_log2, int sms, cudaStream_t stream) {
  cudaError_t e;
  if (p.pl.few) {
    e = launch_few(tm, t8, p, BF16, scale_log2, sms, stream);
  } else {
    static std::atomic<unsigned long long> attr_done{0}, attr_done_join{0};
    if (p.pl.join) {
      e = ensure_smem_limit(prefix_attn_tc<BF16, true>, kSmem, attr_done_join);
      if (e != cudaSuccess) return e;
      return launch_clusters(prefix_attn_tc<BF16, true>, p.pl.nch, dim3(p.pl.units), dim3(kThreads), kSmem, stream, tm, p,
                             scale_log2);
    }
    e = ensure_smem_limit(prefix_attn_tc<BF16, false>, kSmem, attr_done);
    if (e != cudaSuccess) return e;
    const int grid = p.pl.units < sms ? p.pl.units : sms;
    e = launch_dependent(prefix_attn_tc<BF16, false>, dim3(grid), dim3(kThreads), kSmem, stream, tm, p, scale_log2);
  }
  return e != cudaSuccess || !p.pl.split ? e : launch_merge_as<BF16>(p, stream);
}

// What does not come from where the keys are
void fill_params(Params* p, const Plan& pl, const Sizes& z, const Tensor4& o) {
  p->pl = pl;
  p->d_nch = make_div(pl.nch);
  p->d_nchp = make_div(pl.packed ? pl.nchp : 1);
  p->d_nqb = make_div(pl.nqb);
  p->d_npb = make_div(pl.packed ? pl.npb : 1);
  p->d_tb = make_div(pl.tb);
  p->d_rb = make_div(pl.rb);
  p->d_ct = make_div(pl.ct);
  p->d_Hq = make_div(z.Hq);
  p->d_B = make_div(z.B);
  p->d_hb = make_div(z.Hkv * z.B);
  p->d_G = make_div(pl.G);
  p->d_T = make_div(z.T);
  p->B = z.B;
  p->T = z.T;
  p->Hq = z.Hq;
  p->Hkv = z.Hkv;
  p->P = z.P;
  p->S = z.S;
  p->causal = z.causal;
  p->o = static_cast<uint16_t*>(const_cast<void*>(o.data));
  p->ob = o.batch;
  p->orow = o.row;
  p->oh = o.head;
  // (only strides that are followed: fix_stride has replaced the others)
  const auto by32 = [](long long stride, int size) { return size == 1 || stride % 16 == 0; };
  p->o32 = (reinterpret_cast<uintptr_t>(o.data) & 31) == 0 && by32(o.batch, z.B) && by32(o.row, z.T) && by32(o.head, z.Hq);
}

}  // namespace

std::atomic<bool> g_stall_prefix_attention{false};

namespace {

// What launches without a status word report into, one on each device; its address is looked up once
// per device. (Told to the kernels like a caller's word: a choice between the two within them, at
// places that never run, made the 8-bit decode 12 % slower.)
__device__ int g_expired;
cudaError_t expired_word(int** word) {
  static std::atomic<int*> cached[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const bool slot = dev >= 0 && dev < 64;
  *word = slot ? cached[dev].load(std::memory_order_relaxed) : nullptr;
  if (*word) return cudaSuccess;
  e = cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_expired);
  if (e == cudaSuccess && slot) cached[dev].store(*word, std::memory_order_relaxed);
  return e;
}

}  // namespace

Plan pa::plan_of(const Sizes& z, int sms) { return plan_for(z, sms); }
WsLayout pa::workspace_of(const Plan& pl) { return ws_layout(pl, 0, 0, false); }
void pa::set_params(Params* p, const Plan& pl, const Sizes& z, const Tensor4& o) { fill_params(p, pl, z, o); }
bool pa::map_queries(CUtensorMap* m, const Tensor4& q, const Plan& pl, const Sizes& z) {
  return map_q(m, q, pl.G, z.Hkv, z.T, z.B, pl.tb, 1, g_stall_prefix_attention.exchange(false));
}
cudaError_t pa::status_word(int** word) { return expired_word(word); }
cudaError_t pa::launch_merge(const PagedParams& p, bool bf16, cudaStream_t s) {
  return bf16 ? launch_merge_as<true>(p, s) : launch_merge_as<false>(p, s);
}

int device_sms() {
  static std::atomic<int> cached[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (dev >= 0 && dev < 64) {
    const int c = cached[dev].load(std::memory_order_relaxed);
    if (c > 0) return c;
  }
  int n = 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  if (dev >= 0 && dev < 64) cached[dev].store(n, std::memory_order_relaxed);
  return n;
}

}  // namespace qi

extern "C" size_t qi_prefix_attention_workspace(const qi_prefix_attn* a) {
  using namespace qi;
  if (check_sizes(a) != QI_OK) return 0;
  const int sms = device_sms();
  if (sms <= 0) return 0;
  const Plan pl = plan_for({a->B, a->T, a->Hq, a->Hkv, a->P, a->S, a->causal != 0, a->P > 0 && a->pk8 != nullptr, false, false}, sms);
  return ws_layout(pl, a->P, a->Hkv, a->P > 0 && a->pk8 != nullptr).total;
}

extern "C" qi_status qi_prefix_attention(const qi_prefix_attn* a, qi_stream_t stream) {
  using namespace qi;
  qi_status st = check_sizes(a);
  if (st != QI_OK) return st;
  const bool from8 = a->pk8 || a->pv8 || a->pk_sf || a->pv_sf;
  if (!a->q || !a->o || (a->S > 0 && (!a->k || !a->v)))
    return op_fail(QI_ERR_INVALID_ARG, "qi_prefix_attention: NULL q, o, k or v");
  if (a->P > 0 && from8 && (!a->pk8 || !a->pv8 || !a->pk_sf || !a->pv_sf || a->pk || a->pv))
    return op_fail(QI_ERR_INVALID_ARG, "qi_prefix_attention: give the prefix either as pk, pv or as all of pk8, pv8, pk_sf, pv_sf");
  if (a->P > 0 && !from8 && (!a->pk || !a->pv))
    return op_fail(QI_ERR_INVALID_ARG, "qi_prefix_attention: NULL prefix");
  if (!(a->scale > 0.f) || !(a->scale < 3e38f))
    return op_fail(QI_ERR_INVALID_ARG, "qi_prefix_attention: scale must be positive and finite");
  const auto tensor = [](const void* data, const qi_strides& s) { return Tensor4{data, s.batch, s.row, s.head}; };
  Tensor4 q = tensor(a->q, a->q_stride), o = tensor(a->o, a->o_stride), k = tensor(a->k, a->k_stride);
  Tensor4 v = tensor(a->v, a->v_stride), pk = tensor(a->pk, a->pk_stride), pv = tensor(a->pv, a->pv_stride);
  const auto good = [](Tensor4* t, int batch, int rows, int heads) {
    return (reinterpret_cast<uintptr_t>(t->data) & 15) == 0 && fix_stride(&t->batch, batch) &&
           fix_stride(&t->row, rows) && fix_stride(&t->head, heads);
  };
  const char* kAlign = "qi_prefix_attention: %s needs 16-byte alignment and strides that are positive multiples of 8";
  if (!good(&q, a->B, a->T, a->Hq)) return op_fail(QI_ERR_INVALID_ARG, kAlign, "q");
  if (!good(&o, a->B, a->T, a->Hq)) return op_fail(QI_ERR_INVALID_ARG, kAlign, "o");
  if (a->S > 0 && (!good(&k, a->B, a->S, a->Hkv) || !good(&v, a->B, a->S, a->Hkv)))
    return op_fail(QI_ERR_INVALID_ARG, kAlign, "k / v");
  if (a->P > 0 && !from8 && (!good(&pk, 1, a->P, a->Hkv) || !good(&pv, 1, a->P, a->Hkv)))
    return op_fail(QI_ERR_INVALID_ARG, kAlign, "pk / pv");
  if (a->P > 0 && from8 &&
      (((reinterpret_cast<uintptr_t>(a->pk8) | reinterpret_cast<uintptr_t>(a->pv8)) & 15) ||
       ((reinterpret_cast<uintptr_t>(a->pk_sf) | reinterpret_cast<uintptr_t>(a->pv_sf)) & 3)))
    return op_fail(QI_ERR_INVALID_ARG, "qi_prefix_attention: the 8-bit prefix needs 16-byte aligned codes and 4-byte aligned scales");
  if ((reinterpret_cast<uintptr_t>(a->own_len) | reinterpret_cast<uintptr_t>(a->status)) & 3)
    return op_fail(QI_ERR_INVALID_ARG, "qi_prefix_attention: own_len and status need 4-byte alignment");
  const int sms = device_sms();
  if (sms <= 0) return op_fail(QI_ERR_CUDA, "qi_prefix_attention: no CUDA device");
  const Plan pl = plan_for({a->B, a->T, a->Hq, a->Hkv, a->P, a->S, a->causal != 0, a->P > 0 && a->pk8 != nullptr, false, false}, sms);
  if (pl.units <= 0) return op_fail(QI_ERR_SHAPE, "qi_prefix_attention: too many rows and heads");
  const bool pre8 = a->P > 0 && from8;
  const bool convert = pre8 && !pl.few;  // the prefix goes through 16 bits in the workspace
  const WsLayout w = ws_layout(pl, a->P, a->Hkv, pre8);
  if (w.total > 0 && (!a->ws || a->ws_bytes < w.total || (reinterpret_cast<uintptr_t>(a->ws) & 255)))
    return op_fail(QI_ERR_INVALID_ARG, "qi_prefix_attention: needs a 256-byte aligned workspace of %zu bytes", w.total);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool bf16 = a->dtype == QI_DT_BF16;
  uint8_t* ws = static_cast<uint8_t*>(a->ws);
  if (convert) {
    // the prefix in 16 bits, once for all row blocks
    Kv8Args r{};
    r.B = 1;
    r.T = r.S = a->P;
    r.H = a->Hkv;
    r.k8 = const_cast<uint8_t*>(a->pk8);
    r.v8 = const_cast<uint8_t*>(a->pv8);
    r.k_sf = const_cast<uint8_t*>(a->pk_sf);
    r.v_sf = const_cast<uint8_t*>(a->pv_sf);
    const long long head = kHeadDim, row = static_cast<long long>(a->Hkv) * kHeadDim;
    r.k = pk = Tensor4{ws + w.pk, row, row, head};
    r.v = pv = Tensor4{ws + w.pv, row, row, head};
    const cudaError_t e = launch_kv8_read(r, bf16, s);
    if (e != cudaSuccess) return op_fail(QI_ERR_CUDA, "qi_prefix_attention: %s", cudaGetErrorString(e));
  }
  Maps tm;
  const bool stall = g_stall_prefix_attention.exchange(false);
  bool ok = map_q(&tm.qo, q, pl.G, a->Hkv, a->T, a->B, pl.tb, 1, stall) &&
            (pl.packed ? map_q(&tm.qp, q, pl.G, a->Hkv, a->T, a->B, pl.tb, pl.rb, stall) : (tm.qp = tm.qo, true));
  Maps8 t8;
  const Maps8* use8 = nullptr;
  if (pre8 && !convert) {
    ok = ok && map_codes(&t8.k, a->pk8, a->Hkv, a->P) && map_codes(&t8.v, a->pv8, a->Hkv, a->P);
    t8.k_sf = a->pk_sf;
    t8.v_sf = a->pv_sf;
    use8 = &t8;
    tm.pk = tm.pv = tm.qo;  // never loaded from
  } else if (a->P > 0) {
    ok = ok && map_kv(&tm.pk, pk, a->Hkv, a->P, 1) && map_kv(&tm.pv, pv, a->Hkv, a->P, 1);
  }
  if (a->S > 0) ok = ok && map_kv(&tm.k, k, a->Hkv, a->S, a->B) && map_kv(&tm.v, v, a->Hkv, a->S, a->B);
  if (!ok) return op_fail(QI_ERR_INVALID_ARG, "qi_prefix_attention: tensor map encoding failed (strides?)");
  if (a->P == 0) tm.pk = tm.k, tm.pv = tm.v;  // never loaded from
  if (a->S == 0) tm.k = tm.pk, tm.v = tm.pv;
  Params p{};
  fill_params(&p, pl, {a->B, a->T, a->Hq, a->Hkv, a->P, a->S, a->causal != 0, false, false, false}, o);
  p.own_len = a->S > 0 ? a->own_len : nullptr;
  p.part = reinterpret_cast<float*>(ws + w.part);
  p.ml = reinterpret_cast<float2*>(ws + w.ml);
  p.err = a->status;
  if (!p.err) {
    const cudaError_t e = expired_word(&p.err);
    if (e != cudaSuccess) return op_fail(QI_ERR_CUDA, "qi_prefix_attention: %s", cudaGetErrorString(e));
  }
  const float scale_log2 = a->scale * 1.4426950408889634f;
  const cudaError_t e = bf16 ? launch<true>(tm, use8, p, scale_log2, sms, s) : launch<false>(tm, use8, p, scale_log2, sms, s);
  if (e != cudaSuccess) return op_fail(QI_ERR_CUDA, "qi_prefix_attention: %s", cudaGetErrorString(e));
  return QI_OK;
}

extern "C" qi_status qi_prefix_attention_check(qi_stream_t stream) {
  using namespace qi;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int* word = nullptr;
  int code = 0;
  cudaError_t e = cudaStreamSynchronize(s);
  if (e == cudaSuccess) e = expired_word(&word);
  if (e == cudaSuccess) e = cudaMemcpyAsync(&code, word, sizeof(int), cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e == cudaSuccess && code != 0) {
    e = cudaMemsetAsync(word, 0, sizeof(int), s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  }
  if (e != cudaSuccess) return op_fail(QI_ERR_CUDA, "qi_prefix_attention_check: %s", cudaGetErrorString(e));
  if (code != 0)
    return op_fail(QI_ERR_DEVICE_TIMEOUT, "qi_prefix_attention: a kernel's bounded wait expired (device code %d)", code);
  return QI_OK;
}
