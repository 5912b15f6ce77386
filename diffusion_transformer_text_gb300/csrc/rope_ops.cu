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
// pairs, the rotation none. A warp walks the heads of one token (or a run of them, where tokens alone
// would not fill the GPU): its lanes work out two cosines and sines each, hand them round, and keep
// w cos a and w sin a of their own 8 dims in registers for all heads.
#include <cstdarg>
#include <cstdio>

#include "../../include/qidit.h"
#include "internal.h"
#include "ptx.cuh"
#include "values.cuh"

namespace qi {
namespace {

constexpr int kWarps = 8;  // a block's
constexpr int kAhead = 4;  // slots (two heads) whose loads a warp issues before it uses the first

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
  int T, heads[3], axes, ends[4], C;  // ends: pairs up to and with each axis
  int plus_one, w_f32;
  float eps;
  int slots[4];  // first slot of q, k and v, and their number; a slot is two heads
  int per, items;
  Div d_chunks, d_T;
};

// the lane's 8 gains; `first` < 128
__device__ __forceinline__ void load_gain(const RopeParams& p, int kind, int first, float (&w)[8]) {
  if (!p.w[kind]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = 1.f;
    return;
  }
  if (p.w_f32)
    load8(static_cast<const float*>(p.w[kind]) + first, w);
  else
    load8(static_cast<const __nv_bfloat16*>(p.w[kind]) + first, w);
  if (p.plus_one) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] += 1.f;
  }
}

template <typename T>
constexpr int kPieces = sizeof(T) == 4 ? 2 : 1;  // 16-byte pieces of 8 values

template <typename TI, typename TO, bool HALVES>
__global__ void __launch_bounds__(kWarps * 32) qk_norm_rope_kernel(const __grid_constant__ RopeParams p) {
  grid_dep_wait();
  grid_dep_launch_dependents();
  const int lane = threadIdx.x & 31, half = lane >> 4, l16 = lane & 15;
  const int item = static_cast<int>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (item >= p.items) return;
  const int tok = quot(p.d_chunks, item), chunk = item - tok * static_cast<int>(p.d_chunks.d);
  const int b = quot(p.d_T, tok), t = tok - b * p.T;
  if (p.lens && t >= p.lens[b]) return;
  // (wraps only where start alone is past any cache, and then to a negative row)
  const int row = static_cast<int>(static_cast<uint32_t>(p.start ? p.start[b] : 0) + static_cast<uint32_t>(t));

  // cosines and sines of pairs 2 lane and 2 lane + 1
  float cs[2], sn[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int c = 2 * lane + j;
    cs[j] = 1.f;
    sn[j] = 0.f;
    if (c < p.C) {
      int at = row;
      if (p.pos) {
        const int axis = (c >= p.ends[0]) + (c >= p.ends[1]) + (c >= p.ends[2]);
        at = p.pos[static_cast<long long>(tok) * p.axes + axis];
      }
      const unsigned long long angle = static_cast<unsigned long long>(static_cast<long long>(at)) * p.turns[c];
      sincospif(static_cast<float>(static_cast<int>(angle >> 32)) * 0x1p-31f, &sn[j], &cs[j]);
    }
  }
  // those of this lane's dims: co[i], and the sine with the sign that its partner's value takes
  float co[8], si[8];
  const int n8 = p.C >> 3;                       // HALVES: lanes of a half's pairs
  const bool first = l16 < n8;                   // HALVES: the lane holds the first of its pairs
  const bool turned = !HALVES || l16 < 2 * n8;   // HALVES: ... or any
  const int partner = HALVES && turned ? lane + (first ? n8 : -n8) : lane;
  if (HALVES) {
    const int src = turned ? 4 * (first ? l16 : l16 - n8) : 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float c = __shfl_sync(0xffffffffu, cs[e & 1], src + (e >> 1));
      const float s = __shfl_sync(0xffffffffu, sn[e & 1], src + (e >> 1));
      co[e] = turned ? c : 1.f;
      si[e] = turned ? (first ? -s : s) : 0.f;
    }
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float c = __shfl_sync(0xffffffffu, cs[k & 1], 2 * l16 + (k >> 1));
      const float s = __shfl_sync(0xffffffffu, sn[k & 1], 2 * l16 + (k >> 1));
      co[2 * k] = co[2 * k + 1] = c;
      si[2 * k] = -s;
      si[2 * k + 1] = s;
    }
  }
  // dims that are not rotated take nothing of a neighbour, whatever it holds (0 x infinity)
  const bool some_plain = p.C < kHeadDim / 2;

  // where k's and v's rows go: their tensors' row t, or a row of a page
  long long kv_batch = b, kv_row = t;
  bool kv_ok = true;
  if (p.table) {
    const int page = row >> p.page_log;
    kv_ok = row >= 0 && page < p.table_width;
    int id = -1;
    if (kv_ok) id = p.table[b * p.table_stride + page];
    kv_ok = kv_ok && id >= 0 && id < p.pages;
    kv_batch = id;
    kv_row = row & ((1 << p.page_log) - 1);
  }

  const int lo = chunk * p.per, hi = lo + p.per;
#pragma unroll 1
  for (int kind = 0; kind < 3; ++kind) {
    const int s0 = max(lo, p.slots[kind]) - p.slots[kind], s1 = min(hi, p.slots[kind + 1]) - p.slots[kind];
    if (s0 >= s1 || (kind > 0 && !kv_ok)) continue;
    const TI* src = static_cast<const TI*>(p.in[kind].data) + b * p.in[kind].batch + t * p.in[kind].row + l16 * 8;
    TO* dst = static_cast<TO*>(const_cast<void*>(p.out[kind].data)) + l16 * 8 +
              (kind == 0 ? b * p.out[0].batch + t * p.out[0].row : kv_batch * p.out[kind].batch + kv_row * p.out[kind].row);
    const long long ih = p.in[kind].head, oh = p.out[kind].head;
    const bool norm = kind < 2 && p.w[kind];
    float own[8], other[8];
    if (kind < 2) {
      load_gain(p, kind, l16 * 8, own);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float w = HALVES ? __shfl_sync(0xffffffffu, own[e], partner) : own[e ^ 1];
        other[e] = w * si[e];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) own[e] *= co[e];
    }
#pragma unroll 1
    for (int s = s0; s < s1; s += kAhead) {
      uint4 raw[kAhead][kPieces<TI>];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int h = 2 * (s + u) + half;
#pragma unroll
        for (int i = 0; i < kPieces<TI>; ++i) {
          raw[u][i] = make_uint4(0u, 0u, 0u, 0u);
          if (s + u < s1 && h < p.heads[kind]) raw[u][i] = reinterpret_cast<const uint4*>(src + h * ih)[i];
        }
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        if (s + u >= s1) break;
        const int h = 2 * (s + u) + half;
        float x[8];
        from_pieces<TI>(raw[u], x);
        if (kind < 2) {
          float r = 1.f;
          if (norm) {
            float ss = ((x[0] * x[0] + x[1] * x[1]) + (x[2] * x[2] + x[3] * x[3])) +
                       ((x[4] * x[4] + x[5] * x[5]) + (x[6] * x[6] + x[7] * x[7]));
#pragma unroll
            for (int d = 8; d; d >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
            r = rsqrtf(fmaf(ss, 1.f / kHeadDim, p.eps));
          }
          float y[8];
          if (HALVES) {
            uint4 far[kPieces<TI>];
#pragma unroll
            for (int i = 0; i < kPieces<TI>; ++i) {
              far[i].x = __shfl_sync(0xffffffffu, raw[u][i].x, partner);
              far[i].y = __shfl_sync(0xffffffffu, raw[u][i].y, partner);
              far[i].z = __shfl_sync(0xffffffffu, raw[u][i].z, partner);
              far[i].w = __shfl_sync(0xffffffffu, raw[u][i].w, partner);
            }
            from_pieces<TI>(far, y);
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = x[e ^ 1];
          }
          if (some_plain) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (HALVES ? !turned : 4 * l16 + (e >> 1) >= p.C) y[e] = 0.f;
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = fmaf(x[e], own[e], y[e] * other[e]) * r;
        }
        if (h < p.heads[kind]) store8(dst + h * oh, x);
      }
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
cudaError_t launch_rope(const RopeParams& p, bool halves, cudaStream_t s) {
  const unsigned grid = static_cast<unsigned>((static_cast<long long>(p.items) + kWarps - 1) / kWarps);
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
  int slots = 0;
  for (int i = 0; i < 3; ++i) {
    p.slots[i] = slots;
    if (!in[i]) continue;
    if (!out[i] || heads[i] < 1) return op_fail(QI_ERR_INVALID_ARG, "%s: NULL output or no heads", kName);
    slots += (heads[i] + 1) / 2;
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
  p.slots[3] = slots;
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
  // A warp takes up to kMostSlots slots of a token, fewer where tokens are few
  const long long tokens = static_cast<long long>(a->B) * a->T;
  constexpr int kMostSlots = 16;
  const long long want = (tokens * slots + sms * 32ll - 1) / (sms * 32ll);
  int per = want < 1 ? 1 : want > kMostSlots ? kMostSlots : static_cast<int>(want);
  if (per > slots) per = slots;
  const int chunks = (slots + per - 1) / per;
  p.per = (slots + chunks - 1) / chunks;
  p.d_chunks = make_div(chunks);
  p.d_T = make_div(a->T);
  p.items = static_cast<int>(tokens * chunks);
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool f16 = a->dtype == QI_DT_F16, h = a->halves != 0;
  const cudaError_t e = a->in_dtype == QI_DT_F32
                            ? (f16 ? launch_rope<float, __half>(p, h, s) : launch_rope<float, __nv_bfloat16>(p, h, s))
                            : (f16 ? launch_rope<__half, __half>(p, h, s)
                                   : launch_rope<__nv_bfloat16, __nv_bfloat16>(p, h, s));
  return e == cudaSuccess ? QI_OK : op_fail(QI_ERR_CUDA, "%s: %s", kName, cudaGetErrorString(e));
}
