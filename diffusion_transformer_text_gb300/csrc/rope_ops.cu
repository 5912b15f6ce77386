// Between the projection and attention: RMSNorm of every head of q and k, the rotation by positions
// of up to four axes, and the store of q, k and v in the attention's 16-bit type, K and V into
// tensors or into the pages of a cache. One pass: each value is read once and written once.
//
// For a head's 128 values x, with r = 1 / sqrt(mean(x^2) + eps) and gain w (r = w = 1 without a norm):
//   out_i = r (x_i w_i cos a - x_j w_j sin a),  out_j = r (x_j w_j cos a + x_i w_i sin a)
// for the pair (i, j) of angle a: neighbours (2c, 2c + 1), or (c, c + C) with `halves`, c < C; dims past
// 2 C are not rotated. Everything is fp32 until the one rounding to the output's type.
//
// Angles. Pair c turns by turns[c] / 2^64 of a circle per position, so the low 64 bits of position
// times turns[c] are the angle modulo a circle, exactly, at any position: its high half, as a signed
// fraction of half a turn, goes to sincospif. (An fp32 angle is off by 2^-24 of itself: by a hundredth
// of a radian at position 200000.) A table of cosines would be read instead of computed, 512 bytes a token.
//
// A half warp holds a head, 8 values a lane, so the mean is four shuffles and, with neighbours as
// pairs, the rotation none. A block takes a few tokens: its threads first put the factors w cos a and
// +-w sin a of q's and k's dims, and where the rows come from and go, in shared memory; then each warp takes
// tasks of a few heads of one row, all loads of a task before the first use, its lanes' factors in registers.
//
// Bound by HBM at 16 and more heads: a video of 20280 tokens, 32 + 32 + 32 heads, bf16, 147.0 us, the copy
// rate; 4096 image rows from fp32, 48.2 us, 92 %; 15 padded prompts of up to 1499 rows, 24 + 8 + 8 heads, into pages
// 56.7 us, 91 %. By instructions and the latency of a block's steps with few heads: 15800 tokens of 2 + 1 + 1 heads 15.1
// us, 26 %. The factors in registers of every warp, worked out anew for each task, took the video 223 us (90 registers,
// an angle a warp); slots of any two heads, their row, kind and factors looked up for each slot, 190.
#include <cstdarg>
#include <cstdio>

#include "../../include/qidit.h"
#include "internal.h"
#include "ptx.cuh"
#include "values.cuh"

namespace qi {
namespace {

constexpr int kWarps = 8;    // a block's
constexpr int kTokens = 8;   // ... and tokens at most
constexpr int kBlocks = 4;   // blocks an SM has room for: without this limit of 64 registers a thread the
                             // video took 164 us instead of 149

// pairs of heads of a task
template <typename TI>
constexpr int kAhead = sizeof(TI) == 4 ? 2 : 4;

struct RopeParams {
  Tensor4 in[3], out[3];  // q, k, v; with a cache the batch stride of k's and v's out is that of a page
  const void* w[2];       // gains of q and k, or NULL: no norm
  const int* pos;
  const unsigned long long* turns;
  const int* start;
  const int* lens;
  const int* table;  // NULL: out of k and v are tensors
  long long table_stride;
  int table_width, pages, page_log;
  int T, axes, ends[4], C;  // ends: pairs up to and with each axis
  int plus_one, w_f32;
  float eps;
  int heads[3], tasks[4];  // a token's tasks: first of q, of k, of v, and their number
  int group;     // tokens of a block
  int tokens;    // B T
  Div d_tasks, d_T;
};

// A token's row of q, k or v: where its first head is, and goes (NULL: nothing to do)
struct Row {
  const void* src;
  void* dst;
};

__device__ __forceinline__ float gain(const RopeParams& p, int kind, int dim) {
  if (!p.w[kind]) return 1.f;
  const float w = p.w_f32 ? static_cast<const float*>(p.w[kind])[dim]
                          : __bfloat162float(static_cast<const __nv_bfloat16*>(p.w[kind])[dim]);
  return p.plus_one ? 1.f + w : w;
}

template <typename T>
constexpr int kPieces = sizeof(T) == 4 ? 2 : 1;  // 16-byte pieces of 8 values

// out_i = r (own_i x_i + other_i x_partner): a row's factors. A lane's 8 dims are four packed pairs, of
// dims (0, 2), (1, 3), (4, 6), (5, 7), so that partners stand in the same place of two pairs; two pairs
// a piece, a lane's pieces 256 bytes apart, so that neighbouring lanes read neighbouring banks.
struct Factors {
  ulonglong2 own[2][16], other[2][16];
  __device__ __forceinline__ static float& at(ulonglong2 (&a)[2][16], int dim) {
    return reinterpret_cast<float*>(&a[(dim >> 2) & 1][dim >> 3])[(dim & 1) * 2 + ((dim >> 1) & 1)];
  }
};

// 8 values as those pairs, and back
__device__ __forceinline__ void pair8(const float (&v)[8], uint64_t (&x)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int d = (i >> 1) * 4 + (i & 1);
    x[i] = f2_pack(v[d], v[d + 2]);
  }
}
__device__ __forceinline__ void unpair8(const uint64_t (&x)[4], float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int d = (i >> 1) * 4 + (i & 1);
    f2_unpack(x[i], v[d], v[d + 2]);
  }
}

template <typename TI, typename TO, bool HALVES>
__global__ void __launch_bounds__(kWarps * 32, kBlocks) qk_norm_rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int U = kAhead<TI>;
  __shared__ Factors factors[kTokens][2];
  __shared__ Row rows[kTokens][3];
  grid_dep_wait();
  grid_dep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, half = lane >> 4, l16 = lane & 15;
  const int tok0 = static_cast<int>(blockIdx.x) * p.group;

  // thread = a pair of kTokens / kGroups tokens; all that is read is asked for at once
  constexpr int kGroups = kWarps * 32 / (kHeadDim / 2), kEach = kTokens / kGroups;
  const int here = min(p.group, p.tokens - tok0), c = threadIdx.x & (kHeadDim / 2 - 1), n0 = threadIdx.x / (kHeadDim / 2);
  // (wraps only where start alone is past any cache, and then to a negative row)
  const auto row_of = [&](int tok) {
    const int b = quot(p.d_T, tok);
    return static_cast<int>(static_cast<uint32_t>(p.start ? p.start[b] : 0) + static_cast<uint32_t>(tok - b * p.T));
  };
  unsigned long long turn = 0;
  int at[kEach] = {};
  if (c < p.C) {
    turn = p.turns[c];
    const int axis = (c >= p.ends[0]) + (c >= p.ends[1]) + (c >= p.ends[2]);
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      const int n = n0 + j * kGroups;
      if (n < here) at[j] = p.pos ? p.pos[static_cast<long long>(tok0 + n) * p.axes + axis] : row_of(tok0 + n);
    }
  }
  // the pair's dims; those that are not rotated are paired anyhow, and turn by nothing
  const int di = !HALVES ? 2 * c : c < p.C ? c : c + p.C;
  const int dj = !HALVES ? 2 * c + 1 : c < p.C ? c + p.C : di + (kHeadDim / 2 - p.C);
  float wi[2], wj[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) wi[k] = gain(p, k, di), wj[k] = gain(p, k, dj);
  if (threadIdx.x < 3 * here) {
    const int n = threadIdx.x / 3, k = threadIdx.x - 3 * n, tok = tok0 + n, b = quot(p.d_T, tok), t = tok - b * p.T;
    long long to = b * p.out[k].batch + t * p.out[k].row;
    bool ok = !p.lens || t < p.lens[b];
    if (k > 0 && p.table) {
      const int row = row_of(tok), page = row >> p.page_log;
      const int id = row >= 0 && page < p.table_width ? p.table[b * p.table_stride + page] : -1;
      ok = ok && id >= 0 && id < p.pages;
      to = id * p.out[k].batch + (row & ((1 << p.page_log) - 1)) * p.out[k].row;
    }
    rows[n][k].src = static_cast<const TI*>(p.in[k].data) + b * p.in[k].batch + t * p.in[k].row;
    rows[n][k].dst = ok ? static_cast<TO*>(const_cast<void*>(p.out[k].data)) + to : nullptr;
  }
#pragma unroll
  for (int j = 0; j < kEach; ++j) {
    const int n = n0 + j * kGroups;
    if (n >= here) break;
    float cs, sn;
    const unsigned long long angle = static_cast<unsigned long long>(static_cast<long long>(at[j])) * turn;
    sincospif(static_cast<float>(static_cast<int>(angle >> 32)) * 0x1p-31f, &sn, &cs);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      Factors& f = factors[n][k];
      Factors::at(f.own, di) = wi[k] * cs;
      Factors::at(f.own, dj) = wj[k] * cs;
      Factors::at(f.other, di) = -wj[k] * sn;
      Factors::at(f.other, dj) = wi[k] * sn;
    }
  }
  __syncthreads();

  const int n8 = p.C >> 3;                          // HALVES: lanes of a half's pairs
  const bool turned = !HALVES || l16 < 2 * n8;      // HALVES: the lane's dims are rotated
  const int partner = HALVES && turned ? lane + (l16 < n8 ? n8 : -n8) : lane;
  const bool some_plain = p.C < kHeadDim / 2;

#pragma unroll 1
  for (int task = warp; task < here * p.tasks[3]; task += kWarps) {
    const int n = quot(p.d_tasks, task), r0 = task - n * p.tasks[3];
    const int kind = (r0 >= p.tasks[1]) + (r0 >= p.tasks[2]);
    const Row row = rows[n][kind];
    if (!row.dst) continue;
    const int h0 = (r0 - p.tasks[kind]) * 2 * U + half, left = p.heads[kind] - h0;  // heads 0, 2, 4, .. below left
    const TI* src = static_cast<const TI*>(row.src) + h0 * p.in[kind].head + l16 * 8;
    TO* dst = static_cast<TO*>(row.dst) + h0 * p.out[kind].head + l16 * 8;
    const long long is = 2 * p.in[kind].head, os = 2 * p.out[kind].head;
    uint4 raw[U][kPieces<TI>];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < kPieces<TI>; ++i) {
        raw[u][i] = make_uint4(0u, 0u, 0u, 0u);
        if (2 * u < left) raw[u][i] = reinterpret_cast<const uint4*>(src + u * is)[i];
      }
    if (kind == 2) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float v[8];
        from_pieces<TI>(raw[u], v);
        if (2 * u < left) store8(dst + u * os, v);
      }
      continue;
    }
    uint64_t own[4], other[4];
    Factors& f = factors[n][kind];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const ulonglong2 a = f.own[k][l16], o = f.other[k][l16];
      own[2 * k] = a.x, own[2 * k + 1] = a.y;
      other[2 * k] = o.x, other[2 * k + 1] = o.y;
    }
    const bool norm = p.w[kind] != nullptr;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (2 * u >= left + half) break;  // (the whole warp)
      float v[8];
      uint64_t x[4], y[4];
      from_pieces<TI>(raw[u], v);
      pair8(v, x);
      float r = 1.f;
      if (norm) {
        const uint64_t s2 =
            add_f32x2(fma_f32x2(x[0], x[0], mul_f32x2(x[1], x[1])), fma_f32x2(x[2], x[2], mul_f32x2(x[3], x[3])));
        float sa, sb;
        f2_unpack(s2, sa, sb);
        float ss = sa + sb;
#pragma unroll
        for (int d = 8; d; d >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
        r = rsqrtf(fmaf(ss, 1.f / kHeadDim, p.eps));
      }
      if (HALVES) {
        uint4 far[kPieces<TI>];
#pragma unroll
        for (int i = 0; i < kPieces<TI>; ++i) {
          far[i].x = __shfl_sync(0xffffffffu, raw[u][i].x, partner);
          far[i].y = __shfl_sync(0xffffffffu, raw[u][i].y, partner);
          far[i].z = __shfl_sync(0xffffffffu, raw[u][i].z, partner);
          far[i].w = __shfl_sync(0xffffffffu, raw[u][i].w, partner);
        }
        float w[8];
        from_pieces<TI>(far, w);
        pair8(w, y);
      } else {
        y[0] = x[1], y[1] = x[0], y[2] = x[3], y[3] = x[2];
      }
      // dims that are not rotated take nothing of a neighbour, whatever it holds (0 x infinity)
      if (some_plain) {
        float w[8];
        unpair8(y, w);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (HALVES ? !turned : 4 * l16 + (e >> 1) >= p.C) w[e] = 0.f;
        pair8(w, y);
      }
      const uint64_t rr = f2_pack(r, r);
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = mul_f32x2(fma_f32x2(x[i], own[i], mul_f32x2(y[i], other[i])), rr);
      unpair8(x, v);
      if (2 * u < left) store8(dst + u * os, v);
    }
  }
}

qi_status op_fail(qi_status st, const char* fmt, ...) {
  char buf[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  set_last_error(buf);
  return st;
}

bool misaligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

// A stride of a dimension of size 1 is never followed: any legal value will do.
bool good_stride(long long* s, int size, int multiple) {
  if (size == 1) *s = 8;
  return *s > 0 && *s % multiple == 0 && *s < (1ll << 38);
}

template <typename TI, typename TO>
cudaError_t launch_rope(RopeParams p, int sms, bool halves, cudaStream_t s) {
  int n = 0;
  for (int i = 0; i < 3; ++i) {
    p.tasks[i] = n;
    n += (p.heads[i] + 2 * kAhead<TI> - 1) / (2 * kAhead<TI>);
  }
  p.tasks[3] = n;
  p.d_tasks = make_div(n);
  // A block's tokens: as many as make one wave of blocks where they are few (1158 tokens of 24 heads, halves of
  // blocks in a second wave: 5.8 us, in one 4.3), else about kRounds tasks a warp (2, 3, 4, 6 on the video: 163, 148,
  // 148, 149 us; on 1499-row prompts 60, 59, 57, 57)
  constexpr int kRounds = 4;
  const int fill = (p.tokens + kBlocks * sms - 1) / (kBlocks * sms), most = kRounds * kWarps / n;
  p.group = fill < most ? fill : most;
  p.group = p.group < 1 ? 1 : p.group > kTokens ? kTokens : p.group;
  const unsigned grid = static_cast<unsigned>((static_cast<long long>(p.tokens) + p.group - 1) / p.group);
  return launch_dependent(halves ? qk_norm_rope_kernel<TI, TO, true> : qk_norm_rope_kernel<TI, TO, false>, dim3(grid),
                          dim3(kWarps * 32), 0, s, p);
}

}  // namespace
}  // namespace qi

extern "C" qi_status qi_qk_norm_rope(const qi_qk_rope* a, qi_stream_t stream) {
  using namespace qi;
  constexpr const char* kName = "qi_qk_norm_rope";
  if (!a) return op_fail(QI_ERR_INVALID_ARG, "%s: NULL argument", kName);
  if ((a->dtype != QI_DT_F16 && a->dtype != QI_DT_BF16) || (a->in_dtype != QI_DT_F32 && a->in_dtype != a->dtype))
    return op_fail(QI_ERR_INVALID_ARG, "%s: dtypes %d and %d", kName, a->in_dtype, a->dtype);
  const void* in[3] = {a->q, a->k, a->v};
  void* out[3] = {a->q_out, a->k_out, a->v_out};
  const qi_strides in_stride[3] = {a->q_stride, a->k_stride, a->v_stride};
  const qi_strides out_stride[3] = {a->q_out_stride, a->k_out_stride, a->v_out_stride};
  const int heads[3] = {a->Hq, a->Hkv, a->Hkv};
  constexpr int kMost = 1 << 24;
  if (a->B < 1 || a->B > 65535 || a->T < 1 || a->T > kMost || a->Hq < 0 || a->Hq > 65535 || a->Hkv < 0 || a->Hkv > 65535 ||
      static_cast<long long>(a->B) * a->T * (static_cast<long long>(a->Hq) + 2 * a->Hkv) >= (1ll << 31))
    return op_fail(QI_ERR_SHAPE, "%s: B %d T %d Hq %d Hkv %d", kName, a->B, a->T, a->Hq, a->Hkv);
  if (a->axes < 0 || a->axes > 4) return op_fail(QI_ERR_SHAPE, "%s: %d axes", kName, a->axes);
  RopeParams p{};
  long long pairs = 0;
  for (int i = 0; i < 4; ++i) {
    const int n = i < a->axes ? a->pairs[i] : 0;
    if (n < 0 || n > kHeadDim / 2) return op_fail(QI_ERR_SHAPE, "%s: %d pairs", kName, n);
    pairs += n;
    p.ends[i] = static_cast<int>(pairs);
  }
  if (pairs > kHeadDim / 2) return op_fail(QI_ERR_SHAPE, "%s: %lld pairs", kName, pairs);
  if (a->halves && pairs % 8 != 0)
    return op_fail(QI_ERR_SHAPE, "%s: with halves the pairs come in multiples of 8, got %lld", kName, pairs);
  if ((pairs > 0 && !a->turns) || (!a->q && !a->k && !a->v))
    return op_fail(QI_ERR_INVALID_ARG, "%s: NULL turns or nothing to do", kName);
  const bool paged = a->table != nullptr;
  if (paged) {
    const int n = a->page_rows;
    if (n < 16 || n > 65536 || (n & (n - 1)) != 0 || a->pages < 1 || a->table_width < 1)
      return op_fail(QI_ERR_SHAPE, "%s: pages %d of %d rows, table of %d", kName, a->pages, n, a->table_width);
    while ((1 << p.page_log) < n) ++p.page_log;
    p.table_stride = a->table_stride;
    if (a->B == 1) p.table_stride = 0;
    if (a->B > 1 && (a->table_stride < a->table_width || a->table_stride >= (1ll << 38)))
      return op_fail(QI_ERR_INVALID_ARG, "%s: table rows %lld apart", kName, a->table_stride);
    if (a->q && !a->k && !a->v) return op_fail(QI_ERR_INVALID_ARG, "%s: a table without k or v", kName);
  }
  if (!(a->eps >= 0.f) || !(a->eps < 3e38f)) return op_fail(QI_ERR_INVALID_ARG, "%s: eps", kName);
  const int in_multiple = a->in_dtype == QI_DT_F32 ? 4 : 8;
  for (int i = 0; i < 3; ++i) {
    if (!in[i]) continue;
    if (!out[i] || heads[i] < 1) return op_fail(QI_ERR_INVALID_ARG, "%s: NULL output or no heads", kName);
    p.heads[i] = heads[i];
    p.in[i] = {in[i], in_stride[i].batch, in_stride[i].row, in_stride[i].head};
    p.out[i] = {out[i], out_stride[i].batch, out_stride[i].row, out_stride[i].head};
    const bool page = paged && i > 0;
    if (misaligned(in[i], 16) || misaligned(out[i], 16) || !good_stride(&p.in[i].batch, a->B, in_multiple) ||
        !good_stride(&p.in[i].row, a->T, in_multiple) || !good_stride(&p.in[i].head, heads[i], in_multiple) ||
        !good_stride(&p.out[i].batch, page ? a->pages : a->B, 8) ||
        !good_stride(&p.out[i].row, page ? a->page_rows : a->T, 8) || !good_stride(&p.out[i].head, heads[i], 8))
      return op_fail(QI_ERR_INVALID_ARG, "%s: tensors need 16-byte alignment and positive strides of whole 16 bytes", kName);
  }
  if (misaligned(a->q_w, 16) || misaligned(a->k_w, 16) || misaligned(a->turns, 8) || misaligned(a->pos, 4) ||
      misaligned(a->start, 4) || misaligned(a->lens, 4) || misaligned(a->table, 4))
    return op_fail(QI_ERR_INVALID_ARG, "%s: gains need 16-byte, turns 8-byte, int32 arrays 4-byte alignment", kName);
  const int sms = device_sms();
  if (sms <= 0) return op_fail(QI_ERR_CUDA, "%s: no CUDA device", kName);
  p.w[0] = a->q_w;
  p.w[1] = a->k_w;
  p.pos = a->pos;
  p.turns = reinterpret_cast<const unsigned long long*>(a->turns);
  p.start = a->start;
  p.lens = a->lens;
  p.table = a->table;
  p.table_width = a->table_width;
  p.pages = a->pages;
  p.T = a->T;
  p.axes = a->axes;
  p.C = static_cast<int>(pairs);
  p.plus_one = a->plus_one != 0;
  p.w_f32 = a->w_f32 != 0;
  p.eps = a->eps;
  p.tokens = a->B * a->T;
  p.d_T = make_div(a->T);
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool f16 = a->dtype == QI_DT_F16, h = a->halves != 0;
  const cudaError_t e = a->in_dtype == QI_DT_F32
                            ? (f16 ? launch_rope<float, __half>(p, sms, h, s) : launch_rope<float, __nv_bfloat16>(p, sms, h, s))
                            : (f16 ? launch_rope<__half, __half>(p, sms, h, s)
                                   : launch_rope<__nv_bfloat16, __nv_bfloat16>(p, sms, h, s));
  return e == cudaSuccess ? QI_OK : op_fail(QI_ERR_CUDA, "%s: %s", kName, cudaGetErrorString(e));
}
