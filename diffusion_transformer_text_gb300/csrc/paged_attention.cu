// Attention of a chunk of new tokens over a cache in pages, on the 5th-generation tensor cores: the kernel for
// blocks of more than 16 rows (a block = up to 128 rows: tokens of one sequence times the heads of a group).
//
// Row (b, t, hq) sees the first lim rows of sequence b's pages of head hq / G, lim = kv_len[b], or with
// `causal` kv_len[b] - q_len[b] + t + 1:  s_j = scale q.k_j,  o = sum_j 2^(s_j log2 e - m) v_j / sum_j 2^(..),
// with a running maximum m and sum over 128-key tiles. A row without a key is zero.
//
// The inside of a unit is that of prefix_attention.cu: one CTA per SM, S and the two key halves' O in tensor
// memory, P written back there as the A operand of P V, two softmax warpgroups of one key half each, an
// epilogue warpgroup. What differs: K and V come page by page (every page of a tile its own boxes; page numbers are
// looked up a tile ahead), there is no prefix, and only the warp that loads K walks the units: the others follow its
// messages.
//
// What bounds it: from one S of a tile to the next 1640 cycles for 1024 of products (the tensor pipe is busy 59 to 64 %
// of the time: 4 x 4096 image rows over up to 4590 keys, 32 heads, 805-830 us, 1.4 PFLOP/s; 1024 rows behind 16384, 195
// us): issue, product, softmax, each after the other, of which the exponentials are 950 cycles of the 32 softmax
// lanes' 64 keys. Between units, with few tiles in each, instruction fetch: the kernel is longer than the SM's
// instruction cache, and whatever a unit's beginning or end runs comes from the L2 (6 x 777 rows over up to 3001
// keys: 0.45 million misses, 11 % of the warps' time is spent without an instruction). So the code is kept short: units
// walked by one warp and not by four (6 x 777 rows 94.5 -> 88 us, 16 x 300 66 -> 61), the epilogue in a loop that is not
// unrolled (16 x 300 rows 61 -> 56, and 60 since load_8_pages); a walk begun a unit ahead, to have its first pages and Q
// early, cost more than it gave (6 x 777 rows 94.5 -> 99).
//
// Units: whole row blocks in the order that prefix_attention.cu's plan gives (chunks of one length), even
// pieces of all tiles cut on the device (FlowParams: single tokens with many heads, chunks of unlike
// length), or a cluster of CTAs that joins a block's chunks (JOIN: small calls).
// Roundings: P to the operands' type; scores, maxima, sums (of P before its rounding), O and partial rows fp32.
#include <climits>
#include <cstdarg>
#include <cstdio>

#include "../../include/qidit.h"
#include "prefix_attention.cuh"

namespace qi {
using namespace pa;
namespace {

constexpr int kRows = 128;
constexpr int kKStages = 2;
constexpr int kVStages = 2;
constexpr int kQBufs = 2;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 0;    // O of key half h at kColO + 128 h
constexpr uint32_t kColS = 256;
constexpr uint32_t kColP = 384;  // buffer b at kColP + 64 b, half h at + 32 h
constexpr int kThreads = 512;
constexpr uint32_t kRegsLow = 96, kRegsHigh = 160, kRegsEpi = 96;
static_assert(kRegsLow + 2 * kRegsHigh + kRegsEpi == 4 * 128, "register split must equal the launch allotment");

// A unit's numbers for the other warps, worked out once, by the K producer, which is ahead of them
constexpr int kMessages = 4;
struct __align__(16) Message {
  int n, tq, o0, rows;  // n < 0: no more units
  int t0, b0, len, h;
  long long slot;
};

enum : int {
  kKFull = 0,
  kKEmpty = kKFull + kKStages,
  kVFull = kKEmpty + kKStages,
  kVEmpty = kVFull + kVStages,
  kQFull = kVEmpty + kVStages,
  kQEmpty = kQFull + kQBufs,
  kSFull = kQEmpty + kQBufs,
  kSFree = kSFull + 1,   // scores in registers (8 softmax warps)
  kPFull = kSFree + 1,   // [buffer][half of the keys] (4 warps)
  kPvDone = kPFull + 4,  // [buffer][half]
  kOFull = kPvDone + 4,
  kOEmpty = kOFull + 1,       // (4 warps)
  kLFull = kOEmpty + 1,       // the unit's row sums and maxima in shared memory (8 softmax warps)
  kLFree = kLFull + 1,        // ... read by the epilogue (4 warps)
  kUFull = kLFree + 1,        // [message]
  kUEmpty = kUFull + kMessages,  // [message] (15 warps)
  kDrainQK = kUEmpty + kMessages,
  kDrainPV = kDrainQK + 1,
  kNumBars = kDrainPV + 1
};
__device__ __forceinline__ uint32_t bar_count(int i) {
  if (i >= kUEmpty && i < kUEmpty + kMessages) return 15;
  if (i == kSFree || i == kLFull) return 8;
  if ((i >= kPFull && i < kPFull + 4) || i == kOEmpty || i == kLFree) return 4;
  return 1;
}
using FlowFull = Flow<2048>;
constexpr int kSmemBase = (kQBufs + kKStages + kVStages) * kTile + 1024 + kNumBars * 8 + 16 + 2 * 2 * kRows * 4 + 16 +
                          kMessages * static_cast<int>(sizeof(Message));
template <typename P>
constexpr int kSmem = kSmemBase + (kFlow<P> ? static_cast<int>(sizeof(FlowFull)) : 0);
static_assert(kSmem<FlowParams> <= 227 * 1024 && kThreads >= kFlowThreads, "shared memory over the per-block limit");

template <bool BF16, bool JOIN, typename P>
__global__ void __launch_bounds__(kThreads, 1)
    paged_attn_tc(const __grid_constant__ Maps tm, const __grid_constant__ P p, float scale_log2) {
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
  FlowFull* pieces = reinterpret_cast<FlowFull*>(messages + kMessages);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const auto give_up = [&](int code) {
    if (!*abort_flag) report_error(p.err, code);
    *abort_flag = 1;
  };

  if (threadIdx.x == 0) {
    for (int i = 0; i < kNumBars; ++i) mbar_init(&bars[i], bar_count(i));
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tm.qo);
    prefetch_tmap(&tm.k);
  }
  if (warp == 2 && lane == 0) prefetch_tmap(&tm.v);
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
  if constexpr (kFlow<P>) flow_pieces(p, *pieces);

  // the next unit's numbers
  uint32_t km = 0;
  const auto receive = [&](Message& un) {
    const uint32_t mb = km % kMessages;
    if (!__all_sync(0xffffffffu, mbar_wait(&bars[kUFull + mb], (km / kMessages) & 1u))) return false;
    un = messages[mb];
    ++km;
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars[kUEmpty + mb]);
    return true;
  };

  if (warp < 4) {
    regs_release<kRegsLow>();
    if (warp == 0) {
      // ---------------- K tiles, each unit's Q, and its numbers
      uint32_t t = 0, nq = 0, nm = 0;
      bool ok = true;
      for (Walk<P, FlowFull> w(p, pieces); ok && w.more(p); w.step(p)) {
        const Unit un = w.unit(p);
        const uint32_t mb = nm % kMessages, qb = nq % kQBufs;
        ok = __all_sync(0xffffffffu, !*abort_flag && mbar_wait(&bars[kUEmpty + mb], ((nm / kMessages) & 1u) ^ 1u));
        if (!ok) break;
        if (lane == 0) {
          messages[mb] = {un.n, un.tq, un.o0, un.rows, un.t0, un.b0, un.len, un.h, un.slot};
          mbar_arrive(&bars[kUFull + mb]);
        }
        ++nm;
        if (un.n == 0) continue;
        ok = __all_sync(0xffffffffu, !*abort_flag && mbar_wait(&bars[kQEmpty + qb], ((nq / kQBufs) & 1u) ^ 1u));
        if (!ok) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&bars[kQFull + qb], static_cast<uint32_t>(un.rows) * 256u);  // whole boxes, also past the ends
          tma_load_5d(sQ + qb * kTile, &tm.qo, &bars[kQFull + qb], 0, 0, un.h, un.t0, un.b0);
          tma_load_5d(sQ + qb * kTile + kBox, &tm.qo, &bars[kQFull + qb], 64, 0, un.h, un.t0, un.b0);
        }
        ++nq;
        int next = page_of(p, un, un.o0 * kKeys, lane);
        for (int j = 0; j < un.n; ++j) {
          const uint32_t st = t % kKStages;
          const int key0 = (un.o0 + j) * kKeys, id = next;
          if (j + 1 < un.n) next = page_of(p, un, key0 + kKeys, lane);
          ok = __all_sync(0xffffffffu, !*abort_flag && mbar_wait(&bars[kKEmpty + st], ((t / kKStages) & 1u) ^ 1u));
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(&bars[kKFull + st], kTile);
          __syncwarp();
          if (p.page_log == 4)
            load_8_pages(&tm.k, sK + st * kTile, &bars[kKFull + st], un.h, id);
          else
            load_pages(p, &tm.k, sK + st * kTile, &bars[kKFull + st], un.h, key0, id, lane);
          ++t;
        }
      }
      const uint32_t mb = nm % kMessages;
      ok = ok && __all_sync(0xffffffffu, !*abort_flag && mbar_wait(&bars[kUEmpty + mb], ((nm / kMessages) & 1u) ^ 1u));
      if (lane == 0) {
        if (ok) {
          messages[mb].n = -1;
          mbar_arrive(&bars[kUFull + mb]);
        } else {
          give_up(kErrTimeoutProducer);
        }
        for (uint32_t i = t > kKStages ? t - kKStages : 0; i < t; ++i)
          if (!mbar_wait(&bars[kKFull + i % kKStages], (i / kKStages) & 1u)) report_error(p.err, kErrTimeoutDrain);
        for (uint32_t i = nq > kQBufs ? nq - kQBufs : 0; i < nq; ++i)
          if (!mbar_wait(&bars[kQFull + i % kQBufs], (i / kQBufs) & 1u)) report_error(p.err, kErrTimeoutDrain);
      }
      __syncwarp();
    } else if (warp == 2) {
      // ---------------- V tiles
      uint32_t t = 0;
      bool ok = true;
      for (;;) {
        Message un;
        ok = ok && receive(un);
        if (!ok || un.n < 0) break;
        if (un.n == 0) continue;
        int next = page_of(p, un, un.o0 * kKeys, lane);
        for (int j = 0; j < un.n; ++j) {
          const uint32_t st = t % kVStages;
          const int key0 = (un.o0 + j) * kKeys, id = next;
          if (j + 1 < un.n) next = page_of(p, un, key0 + kKeys, lane);
          ok = __all_sync(0xffffffffu, !*abort_flag && mbar_wait(&bars[kVEmpty + st], ((t / kVStages) & 1u) ^ 1u));
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(&bars[kVFull + st], kTile);
          __syncwarp();
          if (p.page_log == 4)
            load_8_pages(&tm.v, sV + st * kTile, &bars[kVFull + st], un.h, id);
          else
            load_pages(p, &tm.v, sV + st * kTile, &bars[kVFull + st], un.h, key0, id, lane);
          ++t;
        }
      }
      if (lane == 0) {
        if (!ok) give_up(kErrTimeoutProducer);
        for (uint32_t i = t > kVStages ? t - kVStages : 0; i < t; ++i)
          if (!mbar_wait(&bars[kVFull + i % kVStages], (i / kVStages) & 1u)) report_error(p.err, kErrTimeoutDrain);
      }
      __syncwarp();
    } else if (warp == 1) {
      // ---------------- S = Q K^T (the issuing warps walk as a whole, so that the descriptors are uniform)
      const uint64_t qdesc0 = sw128_kmajor_desc(smem_u32(sQ));
      const uint64_t kdesc0 = sw128_kmajor_desc(smem_u32(sK));
      uint32_t t = 0, ku = 0;
      bool ok = true;
      for (;;) {
        Message un;
        ok = receive(un);
        if (!ok || un.n < 0) break;
        if (un.n == 0) continue;
        const uint32_t qb = ku % kQBufs;
        ok = __all_sync(0xffffffffu, !*abort_flag && mbar_wait(&bars[kQFull + qb], (ku / kQBufs) & 1u));
        if (!ok) break;
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
        if (!ok) give_up(kErrTimeoutMma);
        mma_commit(&bars[kDrainQK]);
        if (!mbar_wait(&bars[kDrainQK], 0)) report_error(p.err, kErrTimeoutDrain);
      }
      __syncwarp();
    } else {
      // ---------------- O += P V, a half of the keys at a time: a unit's first tile overwrites O
      if constexpr (kFlow<P>) flow_record(p, *pieces);  // (long before the first P)
      const uint64_t vdesc0 = sw128_mnmajor_desc(smem_u32(sV), kBox, 1024);
      uint32_t t = 0, ku = 0;
      bool ok = true;
      for (;;) {
        Message un;
        ok = receive(un);
        if (!ok || un.n < 0) break;
        if (un.n == 0) continue;
        const bool clear = un.len < (un.o0 + un.n) * kKeys;
        ok = __all_sync(0xffffffffu, !*abort_flag && (ku == 0 || mbar_wait(&bars[kOEmpty], (ku - 1) & 1u)));
        for (int j = 0; ok && j < un.n; ++j, ++t) {
          const uint32_t st = t % kVStages, b = t & 1u;
          ok = mbar_wait(&bars[kVFull + st], (t / kVStages) & 1u);
          // rows past the sequence's last, whatever they hold (0 x NaN is NaN)
          if (clear && j + 1 == un.n) {
            ok = __all_sync(0xffffffffu, ok);
            if (ok) clear_rows(sV + st * kTile, un.len - (un.o0 + j) * kKeys, lane);
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
        }
        if (!ok) break;
        ++ku;
      }
      if (elect_one()) {
        if (!ok) give_up(kErrTimeoutMma);
        mma_commit(&bars[kDrainPV]);
        if (!mbar_wait(&bars[kDrainPV], 0)) report_error(p.err, kErrTimeoutDrain);
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
    uint32_t ku = 0;
    bool ok = true;
    for (;;) {
      Message un;
      ok = receive(un);
      if (!ok || un.n < 0) break;
      if (un.n == 0) continue;
      const int lim_own = own_lim(p, un.len, un.t0 + tok, un.tq);
      // A warp whose 32 rows lie past the block's has nothing to compute: it only keeps the
      // barriers' counts (its lanes of S, P and O hold whatever they held). It still waits
      // for every S, so it is never a phase ahead of the other warps on a P buffer.
      const bool idle = quarter * 32 >= un.rows;
      float m_used = -INFINITY;
      float l = 0.f;
      // keys of this half of the tile that the row sees, counted down by tile
      int left = lim_own - un.o0 * kKeys - h * 64;
      const int n = un.n;
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
    uint32_t ku = 0;
    for (;;) {
      Message un;
      ok = receive(un);
      if (!ok || un.n < 0) break;
      const bool part = kFlow<P> ? un.slot >= 0 : p.pl.split;  // (unless JOIN) not all of the rows' keys
      const bool mine = rit < un.rows && un.t0 + tok < un.tq;
      uint16_t* orow = p.o + un.b0 * p.ob + (un.t0 + tok) * p.orow + static_cast<long long>(un.h * p.pl.G + g) * p.oh;
      if (un.n == 0) {
        if (JOIN) *reinterpret_cast<float2*>(smem + kJoinMl + rit * 8) = make_float2(-INFINITY, 0.f);
        // no key at all
        if (!JOIN && !part && mine) {
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
      // a half without a visible key has m = -inf and weight 0; in a row without one both sums and O are 0
      // already (or NaN, if its scores are)
      const float a0 = mm == -INFINITY ? 1.f : fast_exp2(m0 - mm);
      const float a1 = mm == -INFINITY ? 1.f : fast_exp2(m1 - mm);
      const float den = l0 * a0 + l1 * a1;
      const float inv = JOIN || part ? 1.f : (den == 0.f ? 0.f : 1.f / den);
      const float w0 = a0 * inv, w1 = a1 * inv;
      if (!JOIN && part && mine) p.ml[un.slot + rit] = make_float2(mm, den);
      ok = __all_sync(0xffffffffu, mbar_wait(&bars[kOFull], ku & 1u));
      if (!ok) break;
      ++ku;
      if (quarter * 32 >= un.rows) {  // none of the warp's rows are the block's
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[kOEmpty]);
        continue;
      }
      tc_fence_after();
      // (JOIN: the unit is the CTA's only one and its products are done: the rings are free)
      if (JOIN) *reinterpret_cast<float2*>(smem + kJoinMl + rit * 8) = make_float2(mm, den);
      // 16 columns of both at a time (not unrolled: see above)
      const uint32_t tO = tmem + lane_off + kColO;
      const uint64_t w00 = f2_pack(w0, w0), w11 = f2_pack(w1, w1);
      uint32_t x[16], y[16];
#pragma unroll 1
      for (int c = 0; c < 8; ++c) {
        tmem_ld16(tO + c * 16, x);
        tmem_ld16(tO + 128 + c * 16, y);
        tmem_ld_wait();
        if (c == 7) {
          // both are in registers: the next unit's first products may overwrite them
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars[kOEmpty]);
        }
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
          } else if (part) {
            float* d = p.part + (un.slot + rit) * kHeadDim + c * 16;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              uint32_t v[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) v[k] = __float_as_uint(ov[8 * i + k]);
              store32(d + 8 * i, v);
            }
          } else {
            uint32_t v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = pack16<BF16>(ov[2 * k], ov[2 * k + 1]);
            if (p.o32) {  // (a row a lane: half the line accesses of 16-byte stores)
              store32(orow + c * 16, v);
            } else {
              uint4* d = reinterpret_cast<uint4*>(orow + c * 16);
              d[0] = make_uint4(v[0], v[1], v[2], v[3]);
              d[1] = make_uint4(v[4], v[5], v[6], v[7]);
            }
          }
        }
      }
    }
    if (!ok && lane == 0) give_up(kErrTimeoutEpilogue);
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

constexpr int kMergeWarps = 8;
// Joins the parts of a block that was cut (see Flow): block x has the one that piece x took over and ended.
// A warp has ROWS rows, their loads in flight together, and W warps a row where parts are many: warp w takes
// parts w, w + W, .., and the W sums are added in order.
template <bool BF16, int ROWS, int W>
__global__ void __launch_bounds__(kMergeWarps * 32) merge_flow(const __grid_constant__ FlowParams p) {
  __shared__ float4 sacc[W > 1 ? kMergeWarps : 1][32];
  __shared__ float sden[kMergeWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, w = warp % W, last = static_cast<int>(blockIdx.x);
  const int r0 = (static_cast<int>(blockIdx.y) * (kMergeWarps / W) + warp / W) * ROWS;
  grid_dep_wait();
  grid_dep_launch_dependents();
  const int4 end = p.rec[last];
  if (end.x < 0 || !end.z) return;  // (the whole block)
  const int first = end.w, parts = last - first + 1;
  // part k: what piece `first` left, then what piece first + k took over (none, if it is empty)
  const auto slot = [&](int k) {
    return (2ll * (first + k) + (k == 0 ? 1 : 0)) * p.pl.rows_o;
  };
  const auto used = [&](int k) {
    if (k == 0) return true;
    const int4 x = p.rec[first + k];
    return x.x == end.x && x.y == end.y;
  };
  const int b = quot(p.d_nqb, end.x), t0 = (end.x - b * p.pl.nqb) * p.pl.tb, tq = query_rows(p, b);
  float m[ROWS], den[ROWS];
  float4 acc[ROWS];
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    m[i] = -INFINITY;
    den[i] = 0.f;
    acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  for (int k = lane; k < parts; k += 32) {
    const bool u = used(k);
#pragma unroll
    for (int i = 0; i < ROWS; ++i)
      if (r0 + i < p.pl.rows_o) {
        const float x = p.ml[slot(k) + r0 + i].x;  // (what an empty piece's holds is not used)
        m[i] = u ? fmaxf(m[i], x) : m[i];
      }
  }
#pragma unroll
  for (int i = 0; i < ROWS; ++i)
#pragma unroll
    for (int d = 16; d; d >>= 1) m[i] = fmaxf(m[i], __shfl_xor_sync(0xffffffffu, m[i], d));
#pragma unroll 2
  for (int k = w; k < parts; k += W) {
    if (!used(k)) continue;
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      if (r0 + i >= p.pl.rows_o) break;
      const long long s = slot(k) + r0 + i;
      const float2 ml = p.ml[s];
      const float4 v = reinterpret_cast<const float4*>(p.part + s * kHeadDim)[lane];
      // (a part in which the row sees no key; m = -inf with another sum is a row of NaN scores, which stays one)
      const bool none = ml.x == -INFINITY && ml.y == 0.f;
      const float a = m[i] == -INFINITY ? 1.f : fast_exp2(ml.x - m[i]);
      den[i] += none ? 0.f : ml.y * a;
      acc[i].x += none ? 0.f : v.x * a;
      acc[i].y += none ? 0.f : v.y * a;
      acc[i].z += none ? 0.f : v.z * a;
      acc[i].w += none ? 0.f : v.w * a;
    }
  }
  if (W > 1) {  // (ROWS is 1)
    sacc[warp][lane] = acc[0];
    if (lane == 0) sden[warp] = den[0];
    __syncthreads();
    if (w != 0) return;
#pragma unroll
    for (int i = 1; i < W; ++i) {
      const float4 v = sacc[warp + i][lane];
      den[0] += sden[warp + i];
      acc[0].x += v.x;
      acc[0].y += v.y;
      acc[0].z += v.z;
      acc[0].w += v.w;
    }
  }
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const int r = r0 + i, tok = quot(p.d_G, r), t = t0 + tok;
    if (r >= p.pl.rows_o || t >= tq) break;
    const float inv = den[i] == 0.f ? 0.f : 1.f / den[i];
    uint16_t* orow = p.o + b * p.ob + t * p.orow + static_cast<long long>(end.y * p.pl.G + r - tok * p.pl.G) * p.oh;
    reinterpret_cast<uint2*>(orow)[lane] = make_uint2(pack16<BF16>(acc[i].x * inv, acc[i].y * inv),
                                                      pack16<BF16>(acc[i].z * inv, acc[i].w * inv));
  }
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

bool map_pages(CUtensorMap* m, const Tensor4& t, int heads, int page_rows, int pages) {
  const unsigned long long dims[4] = {kHeadDim, static_cast<unsigned long long>(heads),
                                      static_cast<unsigned long long>(page_rows), static_cast<unsigned long long>(pages)};
  const unsigned long long str[3] = {static_cast<unsigned long long>(t.head) * 2,
                                     static_cast<unsigned long long>(t.row) * 2,
                                     static_cast<unsigned long long>(t.batch) * 2};
  const unsigned box[4] = {64, 1, static_cast<unsigned>(page_rows < kKeys ? page_rows : kKeys), 1};
  return encode_map_nd(m, t.data, false, 4, dims, str, box);
}

template <bool BF16, typename P>
cudaError_t launch_join(const Maps& tm, const P& p, float scale_log2, cudaStream_t stream) {
  static std::atomic<unsigned long long> attr_done{0};
  const cudaError_t e = ensure_smem_limit(paged_attn_tc<BF16, true, P>, kSmem<P>, attr_done);
  if (e != cudaSuccess) return e;
  return launch_clusters(paged_attn_tc<BF16, true, P>, p.pl.nch, dim3(p.pl.units), dim3(kThreads), kSmem<P>, stream, tm, p,
                         scale_log2);
}
template <bool BF16, typename P>
cudaError_t launch_walk(const Maps& tm, const P& p, float scale_log2, int grid, cudaStream_t stream) {
  static std::atomic<unsigned long long> attr_done{0};
  const cudaError_t e = ensure_smem_limit(paged_attn_tc<BF16, false, P>, kSmem<P>, attr_done);
  if (e != cudaSuccess) return e;
  return launch_dependent(paged_attn_tc<BF16, false, P>, dim3(grid), dim3(kThreads), kSmem<P>, stream, tm, p, scale_log2);
}

template <bool BF16>
cudaError_t launch(const Maps& tm, const FlowParams& f, float scale_log2, int sms, cudaStream_t stream) {
  const Plan& pl = f.pl;
  const PagedParams& p = f;
  if (pl.join)
    return pl.few ? launch_few(tm, p, BF16, scale_log2, stream) : launch_join<BF16>(tm, p, scale_log2, stream);
  if (!pl.flow) {
    const cudaError_t e = launch_walk<BF16>(tm, p, scale_log2, pl.units < sms ? pl.units : sms, stream);
    return e != cudaSuccess || !pl.split ? e : launch_merge(p, BF16, stream);
  }
  const cudaError_t e = pl.few ? launch_few(tm, f, BF16, scale_log2, stream)
                               : launch_walk<BF16>(tm, f, scale_log2, pl.units, stream);
  const int pieces = pl.units * pl.flow;
  if (e != cudaSuccess || pieces == 1) return e;
  // few rows may have many parts, many rows have two or three
  constexpr int kRowsEach = 4, kWarpsEach = 4;
  const auto kernel = pl.few ? merge_flow<BF16, 1, kWarpsEach> : merge_flow<BF16, kRowsEach, 1>;
  const int each = pl.few ? kMergeWarps / kWarpsEach : kMergeWarps * kRowsEach;
  return launch_dependent(kernel, dim3(pieces, static_cast<unsigned>(ceil_div(pl.rows_o, each))), dim3(kMergeWarps * 32), 0,
                          stream, f);
}

// a call's sizes, checked but for what the plan makes of them
qi_status check_paged(const qi_paged_attn* a) {
  constexpr const char* kName = "qi_paged_attention";
  if (!a) return op_fail(QI_ERR_INVALID_ARG, "%s: NULL argument", kName);
  if (a->dtype != QI_DT_F16 && a->dtype != QI_DT_BF16) return op_fail(QI_ERR_INVALID_ARG, "%s: dtype %d", kName, a->dtype);
  constexpr int kMost = 1 << 24;
  const int n = a->page_rows;
  if (a->B < 1 || a->B > 65535 || a->T < 1 || a->T > kMost || a->Hkv < 1 || a->Hkv > 65535 || a->Hq < a->Hkv ||
      a->Hq % a->Hkv != 0 || a->Hq / a->Hkv > kRows || static_cast<long long>(a->B) * a->T * a->Hq >= (1ll << 31))
    return op_fail(QI_ERR_SHAPE, "%s: B %d T %d Hq %d Hkv %d", kName, a->B, a->T, a->Hq, a->Hkv);
  if (n < 16 || n > 65536 || (n & (n - 1)) != 0 || a->pages < 1 || a->table_width < 1 || a->max_len < 1 ||
      a->max_len > kMost || a->max_len > static_cast<long long>(a->table_width) * n)
    return op_fail(QI_ERR_SHAPE, "%s: pages %d of %d rows, table of %d, max_len %d", kName, a->pages, n, a->table_width,
                   a->max_len);
  return QI_OK;
}
Sizes paged_sizes(const qi_paged_attn* a) {
  return {a->B, a->T, a->Hq, a->Hkv, 0, a->max_len, a->causal != 0, false, true, a->q_len != nullptr};
}

}  // namespace
}  // namespace qi

extern "C" size_t qi_paged_attention_workspace(const qi_paged_attn* a) {
  using namespace qi;
  if (check_paged(a) != QI_OK) return 0;
  const int sms = device_sms();
  if (sms <= 0) return 0;
  return workspace_of(plan_of(paged_sizes(a), sms)).total;
}

extern "C" qi_status qi_paged_attention(const qi_paged_attn* a, qi_stream_t stream) {
  using namespace qi;
  constexpr const char* kName = "qi_paged_attention";
  const qi_status st = check_paged(a);
  if (st != QI_OK) return st;
  if (!a->q || !a->k || !a->v || !a->o || !a->table || !a->kv_len)
    return op_fail(QI_ERR_INVALID_ARG, "%s: NULL q, k, v, o, table or kv_len", kName);
  if (!(a->scale > 0.f) || !(a->scale < 3e38f))
    return op_fail(QI_ERR_INVALID_ARG, "%s: scale must be positive and finite", kName);
  const auto tensor = [](const void* data, const qi_strides& s) { return Tensor4{data, s.batch, s.row, s.head}; };
  Tensor4 q = tensor(a->q, a->q_stride), o = tensor(a->o, a->o_stride);
  Tensor4 k = tensor(a->k, a->k_stride), v = tensor(a->v, a->v_stride);
  const auto good = [](Tensor4* t, int batch, int rows, int heads) {
    return (reinterpret_cast<uintptr_t>(t->data) & 15) == 0 && fix_stride(&t->batch, batch) &&
           fix_stride(&t->row, rows) && fix_stride(&t->head, heads);
  };
  if (!good(&q, a->B, a->T, a->Hq) || !good(&o, a->B, a->T, a->Hq) || !good(&k, a->pages, a->page_rows, a->Hkv) ||
      !good(&v, a->pages, a->page_rows, a->Hkv))
    return op_fail(QI_ERR_INVALID_ARG, "%s: tensors need 16-byte alignment and strides that are positive multiples of 8",
                   kName);
  if ((reinterpret_cast<uintptr_t>(a->table) | reinterpret_cast<uintptr_t>(a->kv_len) |
       reinterpret_cast<uintptr_t>(a->q_len) | reinterpret_cast<uintptr_t>(a->status)) & 3)
    return op_fail(QI_ERR_INVALID_ARG, "%s: table, kv_len, q_len and status need 4-byte alignment", kName);
  if (a->B > 1 && (a->table_stride < a->table_width || a->table_stride >= (1ll << 38)))
    return op_fail(QI_ERR_INVALID_ARG, "%s: table rows %lld apart", kName, a->table_stride);
  const int sms = device_sms();
  if (sms <= 0) return op_fail(QI_ERR_CUDA, "%s: no CUDA device", kName);
  const Sizes z = paged_sizes(a);
  const Plan pl = plan_of(z, sms);
  if (pl.units <= 0) return op_fail(QI_ERR_SHAPE, "%s: too many rows and heads", kName);
  const WsLayout w = workspace_of(pl);
  if (w.total > 0 && (!a->ws || a->ws_bytes < w.total || (reinterpret_cast<uintptr_t>(a->ws) & 255)))
    return op_fail(QI_ERR_INVALID_ARG, "%s: needs a 256-byte aligned workspace of %zu bytes", kName, w.total);
  Maps tm;
  if (!map_queries(&tm.qo, q, pl, z) ||
      !map_pages(&tm.k, k, a->Hkv, a->page_rows, a->pages) || !map_pages(&tm.v, v, a->Hkv, a->page_rows, a->pages))
    return op_fail(QI_ERR_INVALID_ARG, "%s: tensor map encoding failed (strides?)", kName);
  tm.qp = tm.qo;  // no prefix: never loaded from
  tm.pk = tm.k;
  tm.pv = tm.v;
  FlowParams p{};
  set_params(&p, pl, z, o);
  p.own_len = a->kv_len;
  p.q_len = a->q_len;
  p.table = a->table;
  p.table_stride = a->B > 1 ? a->table_stride : 0;
  p.pages = a->pages;
  while ((1 << p.page_log) < a->page_rows) ++p.page_log;
  uint8_t* ws = static_cast<uint8_t*>(a->ws);
  p.part = reinterpret_cast<float*>(ws + w.part);
  p.ml = reinterpret_cast<float2*>(ws + w.ml);
  p.err = a->status;
  if (!p.err) {
    const cudaError_t e = status_word(&p.err);
    if (e != cudaSuccess) return op_fail(QI_ERR_CUDA, "%s: %s", kName, cudaGetErrorString(e));
  }
  const float scale_log2 = a->scale * 1.4426950408889634f;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  p.rec = reinterpret_cast<int4*>(ws + w.rec);
  p.per_slot = ceil_div(a->B * pl.nqb, pl.few ? kFlowSlotsFew : FlowFull::kSlots);
  p.d_slot = make_div(p.per_slot);
  p.d_pieces = make_div(pl.flow ? pl.units * pl.flow : 1);
  const cudaError_t e = a->dtype == QI_DT_BF16 ? launch<true>(tm, p, scale_log2, sms, s)
                                               : launch<false>(tm, p, scale_log2, sms, s);
  return e == cudaSuccess ? QI_OK : op_fail(QI_ERR_CUDA, "%s: %s", kName, cudaGetErrorString(e));
}
