// Memory-bound operators of batches that share a prompt: the 8-bit K/V cache (write,
// read back) and the residual RMSNorm that ends in an MXFP8 operand.
//
// Both work on groups of 8 consecutive values per thread (one 16-byte access of 16-bit
// data), so a block of 32 values that shares a scale is four neighbouring lanes: its
// largest magnitude takes two shuffles, and every load and store of a warp is contiguous.
#include <cstdarg>
#include <cstdio>

#include "../../include/qidit.h"
#include "internal.h"
#include "ptx.cuh"

namespace qi {
namespace {

// ---------------------------------------------------------------- values

template <typename T>
__device__ __forceinline__ void load8(const T* src, float (&v)[8]);
template <>
__device__ __forceinline__ void load8(const float* src, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(src)[0], b = reinterpret_cast<const float4*>(src)[1];
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
  v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
template <>
__device__ __forceinline__ void load8(const __half* src, float (&v)[8]) {
  const uint4 w = *reinterpret_cast<const uint4*>(src);
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}
template <>
__device__ __forceinline__ void load8(const __nv_bfloat16* src, float (&v)[8]) {
  const uint4 w = *reinterpret_cast<const uint4*>(src);
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(u[i] << 16);
    v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
}

// Stores 8 values in T and leaves in v what was stored.
__device__ __forceinline__ void store8(float* dst, float (&v)[8]) {
  reinterpret_cast<float4*>(dst)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(dst)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ uint4 pack8(const __half*, const float (&v)[8]) {
  return make_uint4(pack_f16x2(v[0], v[1]), pack_f16x2(v[2], v[3]), pack_f16x2(v[4], v[5]), pack_f16x2(v[6], v[7]));
}
__device__ __forceinline__ uint4 pack8(const __nv_bfloat16*, const float (&v)[8]) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                    pack_bf16x2(v[6], v[7]));
}
template <typename T>
__device__ __forceinline__ void store8(T* dst, float (&v)[8]) {
  *reinterpret_cast<uint4*>(dst) = pack8(dst, v);
}
__device__ __forceinline__ void round8(const float*, float (&)[8]) {}
__device__ __forceinline__ void round8(const __half*, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __half2float(__float2half_rn(v[i]));
}
__device__ __forceinline__ void round8(const __nv_bfloat16*, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __bfloat162float(__float2bfloat16_rn(v[i]));
}

// MXFP8 of a block of 32 values held by four neighbouring lanes (8 each): this lane's 8
// codes, and the block's scale byte. Same definition as mx_quant32; the scaling by a power
// of two is exact, so the only rounding is the one to E4M3 (nearest, ties to even).
__device__ __forceinline__ uint2 mx_quant8(const float (&v)[8], uint32_t& scale) {
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(v[i]));
  top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
  int e = top > 0.f ? ilogbf(top) - 8 : -127;
  e = max(-127, min(127, e));
  const float inv = ldexpf(1.f, -e);
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    c[i] = __nv_cvt_float2_to_fp8x2(make_float2(v[2 * i] * inv, v[2 * i + 1] * inv), __NV_SATFINITE, __NV_E4M3);
  scale = static_cast<uint32_t>(e + 127);
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// ---------------------------------------------------------------- 8-bit K/V cache

constexpr int kKv8Threads = 256;

// Thread = 8 values of one (row, head) of K and the same of V; blockIdx.y strides over sequences.
template <typename T>
__global__ void __launch_bounds__(kKv8Threads) kv8_write_kernel(const __grid_constant__ Kv8Args a) {
  grid_dep_wait();
  grid_dep_launch_dependents();
  const uint32_t i = blockIdx.x * kKv8Threads + threadIdx.x;
  const uint32_t part = i & 15u, th = i >> 4;
  const int t = static_cast<int>(th / static_cast<uint32_t>(a.H));
  const int h = static_cast<int>(th - static_cast<uint32_t>(t) * a.H);
  for (int b = blockIdx.y; b < a.B; b += gridDim.y) {
    const int n = a.lens ? min(a.lens[b], a.T) : a.T;
    const long long row = static_cast<long long>(a.pos ? a.pos[b] : 0) + t;
    const bool in = t < n && row >= 0 && row < a.S;
    // (the four lanes of a scale block share a row, so they are in or out together)
    float kv[8] = {}, vv[8] = {};
    if (in) {
      load8(static_cast<const T*>(a.k.data) + b * a.k.batch + t * a.k.row + h * a.k.head + part * 8, kv);
      load8(static_cast<const T*>(a.v.data) + b * a.v.batch + t * a.v.row + h * a.v.head + part * 8, vv);
    }
    uint32_t ks, vs;
    const uint2 kc = mx_quant8(kv, ks), vc = mx_quant8(vv, vs);
    if (in) {
      const long long at = (static_cast<long long>(b) * a.S + row) * a.H + h;
      reinterpret_cast<uint2*>(a.k8 + at * kHeadDim)[part] = kc;
      reinterpret_cast<uint2*>(a.v8 + at * kHeadDim)[part] = vc;
      if ((part & 3u) == 0) {
        a.k_sf[at * 4 + part / 4] = static_cast<uint8_t>(ks);
        a.v_sf[at * 4 + part / 4] = static_cast<uint8_t>(vs);
      }
    }
  }
}

// 8 codes times their scale, in fp32 (exact: 4 significant bits times a power of two)
__device__ __forceinline__ void mx_values8(uint2 c, uint32_t scale, float (&v)[8]) {
  const float s = ldexpf(1.f, static_cast<int>(scale) - 127);
  const uint32_t w[4] = {c.x & 0xFFFFu, c.x >> 16, c.y & 0xFFFFu, c.y >> 16};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w[i]), __NV_E4M3);
    const float2 f = __half22float2(__half2(h));
    v[2 * i] = f.x * s;
    v[2 * i + 1] = f.y * s;
  }
}

template <typename T>
__global__ void __launch_bounds__(kKv8Threads) kv8_read_kernel(const __grid_constant__ Kv8Args a) {
  grid_dep_wait();
  grid_dep_launch_dependents();
  const uint32_t i = blockIdx.x * kKv8Threads + threadIdx.x;
  const uint32_t part = i & 15u, th = i >> 4;
  const int t = static_cast<int>(th / static_cast<uint32_t>(a.H));
  const int h = static_cast<int>(th - static_cast<uint32_t>(t) * a.H);
  for (int b = blockIdx.y; b < a.B; b += gridDim.y) {
    const int n = a.lens ? min(a.lens[b], a.T) : a.T;
    const long long row = static_cast<long long>(a.pos ? a.pos[b] : 0) + t;
    if (t >= n || row < 0 || row >= a.S) continue;
    const long long at = (static_cast<long long>(b) * a.S + row) * a.H + h;
    const uint2 kc = reinterpret_cast<const uint2*>(a.k8 + at * kHeadDim)[part];
    const uint2 vc = reinterpret_cast<const uint2*>(a.v8 + at * kHeadDim)[part];
    float kv[8], vv[8];
    mx_values8(kc, a.k_sf[at * 4 + part / 4], kv);
    mx_values8(vc, a.v_sf[at * 4 + part / 4], vv);
    store8(static_cast<T*>(const_cast<void*>(a.k.data)) + b * a.k.batch + t * a.k.row + h * a.k.head + part * 8, kv);
    store8(static_cast<T*>(const_cast<void*>(a.v.data)) + b * a.v.batch + t * a.v.row + h * a.v.head + part * 8, vv);
  }
}

cudaError_t launch_kv8(void (*kernel)(Kv8Args), const Kv8Args& a, cudaStream_t s) {
  const unsigned x = static_cast<unsigned>((static_cast<long long>(a.T) * a.H * 16 + kKv8Threads - 1) / kKv8Threads);
  return launch_dependent(kernel, dim3(x, static_cast<unsigned>(a.B)), dim3(kKv8Threads), 0, s, a);
}

// ---------------------------------------------------------------- residual RMSNorm to MXFP8

// An fp32 value with an error term: hi + lo. Sums and products that keep the rounding
// error of each fp32 operation (Knuth's two-sum, the FMA remainder of a product), so that
// y is rounded to fp32 once and a code differs from the exact one only where the exact
// value lies within an fp32 half step of a border between two codes.
struct F2 {
  float hi, lo;
};
__device__ __forceinline__ F2 two_sum(float a, float b) {
  const float s = __fadd_rn(a, b);
  const float bb = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, bb)), __fsub_rn(b, bb))};
}
__device__ __forceinline__ F2 add(F2 a, F2 b) {
  F2 s = two_sum(a.hi, b.hi);
  s.lo += a.lo + b.lo;
  return s;
}
// 1 / sqrt(m), m = hi + lo > 0: rsqrtf and one Newton step of which only the correction is kept
__device__ __forceinline__ F2 inv_sqrt(F2 m) {
  const float r = rsqrtf(m.hi);
  const float t = __fmul_rn(r, r);
  const float te = __fmaf_rn(r, r, -t);
  const float u = __fmaf_rn(-m.hi, t, 1.f) - m.lo * t - m.hi * te;
  const float c = 0.5f * r * u;
  return {r, isfinite(c) ? c : 0.f};
}

struct NormParams {
  qi_add_rmsnorm a;
  int groups;  // ceil(rows / 128)
};

// One CTA per row; a thread holds NC groups of 8 values (group threadIdx.x + i blockDim.x).
template <typename TX, typename TD, int NC>
__global__ void add_rmsnorm_kernel(const __grid_constant__ NormParams p) {
  grid_dep_wait();
  grid_dep_launch_dependents();
  __shared__ F2 part[32];
  const qi_add_rmsnorm& a = p.a;
  const int r = blockIdx.x;
  const int groups8 = a.K / 8;
  float v[NC][8];
  F2 sum = {0.f, 0.f};
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = threadIdx.x + i * blockDim.x;
#pragma unroll
    for (int k = 0; k < 8; ++k) v[i][k] = 0.f;
    if (c < groups8) {
      load8(static_cast<const TX*>(a.x) + r * a.x_stride + c * 8, v[i]);
      if (a.delta) {
        float d[8];
        load8(static_cast<const TD*>(a.delta) + r * a.delta_stride + c * 8, d);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[i][k] = __fadd_rn(v[i][k], d[k]);
        round8(static_cast<const TX*>(nullptr), v[i]);
      }
      if (a.x_out) store8(static_cast<TX*>(a.x_out) + r * a.x_out_stride + c * 8, v[i]);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float sq = __fmul_rn(v[i][k], v[i][k]);
      sum = add(sum, F2{sq, __fmaf_rn(v[i][k], v[i][k], -sq)});
    }
  }
#pragma unroll
  for (int d = 16; d; d >>= 1)
    sum = add(sum, F2{__shfl_xor_sync(0xffffffffu, sum.hi, d), __shfl_xor_sync(0xffffffffu, sum.lo, d)});
  const int warps = (blockDim.x + 31) / 32;
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = sum;
  __syncthreads();
  sum = part[0];
  for (int i = 1; i < warps; ++i) sum = add(sum, part[i]);
  // mean + eps, with the division's remainder
  const float n = static_cast<float>(a.K);
  const float mh = __fdiv_rn(sum.hi, n);
  const F2 m = add(F2{mh, __fdiv_rn(__fmaf_rn(-mh, n, sum.hi) + sum.lo, n)}, F2{a.eps, 0.f});
  const F2 rs = inv_sqrt(m);
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = threadIdx.x + i * blockDim.x;
    const bool in = c < groups8;  // groups8 is a multiple of 16: the lanes of a scale block agree
    float g[8], gl[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) g[k] = 1.f, gl[k] = 0.f;
    if (in && a.w) {
      if (a.w_f32)
        load8(static_cast<const float*>(a.w) + c * 8, g);
      else
        load8(static_cast<const __nv_bfloat16*>(a.w) + c * 8, g);
      if (a.plus_one) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const F2 s = two_sum(1.f, g[k]);
          g[k] = s.hi;
          gl[k] = s.lo;
        }
      }
    }
    float y[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float q = __fmul_rn(v[i][k], rs.hi);
      const float qe = __fmaf_rn(v[i][k], rs.hi, -q) + v[i][k] * rs.lo;
      const float z = __fmul_rn(q, g[k]);
      y[k] = z + (__fmaf_rn(q, g[k], -z) + (qe * g[k] + q * gl[k]));
    }
    uint32_t scale;
    const uint2 codes = mx_quant8(y, scale);
    if (in) {
      reinterpret_cast<uint2*>(a.q + static_cast<size_t>(r) * a.K)[c] = codes;
      if ((c & 3) == 0) a.sf[mx_sf_offset(r, c / 4, p.groups)] = static_cast<uint8_t>(scale);
    }
  }
}

template <typename TX, typename TD>
cudaError_t launch_norm(const NormParams& p, cudaStream_t s) {
  const int groups8 = p.a.K / 8;
  const int threads = groups8 < 256 ? (groups8 + 31) / 32 * 32 : 256;
  const int nc = (groups8 + threads - 1) / threads;
  const dim3 grid(static_cast<unsigned>(p.a.rows)), block(static_cast<unsigned>(threads));
  if (nc <= 1) return launch_dependent(add_rmsnorm_kernel<TX, TD, 1>, grid, block, 0, s, p);
  if (nc <= 2) return launch_dependent(add_rmsnorm_kernel<TX, TD, 2>, grid, block, 0, s, p);
  if (nc <= 4) return launch_dependent(add_rmsnorm_kernel<TX, TD, 4>, grid, block, 0, s, p);
  return launch_dependent(add_rmsnorm_kernel<TX, TD, 8>, grid, block, 0, s, p);
}
template <typename TX>
cudaError_t launch_norm_d(const NormParams& p, cudaStream_t s) {
  switch (p.a.delta ? p.a.delta_dtype : p.a.x_dtype) {
    case QI_DT_F16: return launch_norm<TX, __half>(p, s);
    case QI_DT_BF16: return launch_norm<TX, __nv_bfloat16>(p, s);
    default: return launch_norm<TX, float>(p, s);
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

bool misaligned(const void* p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0; }

// A stride of a dimension of size 1 is never followed.
bool good_stride(long long* s, int size) {
  if (size == 1) *s = 8;
  return *s > 0 && *s % 8 == 0 && *s < (1ll << 38);
}

qi_status kv8_call(const char* name, int dtype, int B, int T, int S, int H, const qi_tensor4* k, const qi_tensor4* v,
                   const uint8_t* k8, const uint8_t* v8, const uint8_t* k_sf, const uint8_t* v_sf, const int* pos,
                   const int* lens, Kv8Args* a) {
  if (!k || !v || !k->data || !v->data || !k8 || !v8 || !k_sf || !v_sf)
    return op_fail(QI_ERR_INVALID_ARG, "%s: NULL argument", name);
  if (dtype != QI_DT_F16 && dtype != QI_DT_BF16) return op_fail(QI_ERR_INVALID_ARG, "%s: dtype %d", name, dtype);
  constexpr int kMost = 1 << 24;
  if (B < 1 || B > 65535 || T < 1 || T > kMost || S < 1 || S > kMost || H < 1 || H > 65535 ||
      static_cast<long long>(T) * H >= (1ll << 27))
    return op_fail(QI_ERR_SHAPE, "%s: B %d T %d S %d H %d", name, B, T, S, H);
  a->B = B;
  a->T = T;
  a->S = S;
  a->H = H;
  a->k = *k;
  a->v = *v;
  for (qi_tensor4* t : {&a->k, &a->v})
    if (misaligned(t->data, 16) || !good_stride(&t->batch, B) || !good_stride(&t->row, T) || !good_stride(&t->head, H))
      return op_fail(QI_ERR_INVALID_ARG,
                     "%s: k and v need 16-byte alignment and strides that are positive multiples of 8", name);
  if (misaligned(k8, 16) || misaligned(v8, 16) || misaligned(k_sf, 4) || misaligned(v_sf, 4) || misaligned(pos, 4) ||
      misaligned(lens, 4))
    return op_fail(QI_ERR_INVALID_ARG, "%s: codes need 16-byte, scales, pos and lens 4-byte alignment", name);
  a->k8 = const_cast<uint8_t*>(k8);
  a->v8 = const_cast<uint8_t*>(v8);
  a->k_sf = const_cast<uint8_t*>(k_sf);
  a->v_sf = const_cast<uint8_t*>(v_sf);
  a->pos = pos;
  a->lens = lens;
  return QI_OK;
}

}  // namespace

cudaError_t launch_kv8_write(const Kv8Args& a, bool bf16, cudaStream_t s) {
  return launch_kv8(bf16 ? kv8_write_kernel<__nv_bfloat16> : kv8_write_kernel<__half>, a, s);
}
cudaError_t launch_kv8_read(const Kv8Args& a, bool bf16, cudaStream_t s) {
  return launch_kv8(bf16 ? kv8_read_kernel<__nv_bfloat16> : kv8_read_kernel<__half>, a, s);
}

}  // namespace qi

extern "C" qi_status qi_kv8_write(int dtype, int B, int T, int S, int H, const qi_tensor4* k, const qi_tensor4* v,
                                  uint8_t* k8, uint8_t* v8, uint8_t* k_sf, uint8_t* v_sf, const int* pos,
                                  const int* lens, qi_stream_t stream) {
  qi::Kv8Args a{};
  const qi_status st =
      qi::kv8_call("qi_kv8_write", dtype, B, T, S, H, k, v, k8, v8, k_sf, v_sf, pos, lens, &a);
  if (st != QI_OK) return st;
  const cudaError_t e = qi::launch_kv8_write(a, dtype == QI_DT_BF16, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? QI_OK : qi::op_fail(QI_ERR_CUDA, "qi_kv8_write: %s", cudaGetErrorString(e));
}

extern "C" qi_status qi_kv8_read(int dtype, int B, int T, int S, int H, const uint8_t* k8, const uint8_t* v8,
                                 const uint8_t* k_sf, const uint8_t* v_sf, const int* pos, const int* lens,
                                 const qi_tensor4* k, const qi_tensor4* v, qi_stream_t stream) {
  qi::Kv8Args a{};
  const qi_status st = qi::kv8_call("qi_kv8_read", dtype, B, T, S, H, k, v, k8, v8, k_sf, v_sf, pos, lens, &a);
  if (st != QI_OK) return st;
  const cudaError_t e = qi::launch_kv8_read(a, dtype == QI_DT_BF16, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? QI_OK : qi::op_fail(QI_ERR_CUDA, "qi_kv8_read: %s", cudaGetErrorString(e));
}

extern "C" qi_status qi_add_rmsnorm_mxfp8(const qi_add_rmsnorm* args, qi_stream_t stream) {
  using namespace qi;
  if (!args || !args->x || !args->q || !args->sf)
    return op_fail(QI_ERR_INVALID_ARG, "qi_add_rmsnorm_mxfp8: NULL argument");
  NormParams p{*args, 0};
  qi_add_rmsnorm& a = p.a;
  const auto known = [](int d) { return d == QI_DT_F16 || d == QI_DT_BF16 || d == QI_DT_F32; };
  if (!known(a.x_dtype) || (a.delta && !known(a.delta_dtype)))
    return op_fail(QI_ERR_INVALID_ARG, "qi_add_rmsnorm_mxfp8: dtypes %d and %d", a.x_dtype, a.delta_dtype);
  if (a.rows < 1 || a.K < 128 || a.K > 16384 || a.K % 128 != 0)
    return op_fail(QI_ERR_SHAPE, "qi_add_rmsnorm_mxfp8: rows %d K %d (K a multiple of 128 up to 16384)", a.rows, a.K);
  if (!(a.eps >= 0.f) || !(a.eps < 3e38f)) return op_fail(QI_ERR_INVALID_ARG, "qi_add_rmsnorm_mxfp8: eps");
  const auto good = [&](const void* t, long long* stride, int dtype) {
    if (a.rows == 1) *stride = a.K;
    const int size = dtype == QI_DT_F32 ? 4 : 2;
    return !misaligned(t, 16) && *stride >= a.K && *stride * size % 16 == 0 && *stride < (1ll << 38);
  };
  if (!good(a.x, &a.x_stride, a.x_dtype) || (a.delta && !good(a.delta, &a.delta_stride, a.delta_dtype)) ||
      (a.x_out && !good(a.x_out, &a.x_out_stride, a.x_dtype)) || misaligned(a.w, 16) || misaligned(a.q, 16) ||
      misaligned(a.sf, 4))
    return op_fail(QI_ERR_INVALID_ARG,
                   "qi_add_rmsnorm_mxfp8: x, delta, x_out, w and q need 16-byte alignment, rows at least K apart in "
                   "multiples of 16 bytes");
  p.groups = (a.rows + 127) / 128;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = a.x_dtype == QI_DT_F16    ? launch_norm_d<__half>(p, s)
                        : a.x_dtype == QI_DT_BF16 ? launch_norm_d<__nv_bfloat16>(p, s)
                                                  : launch_norm_d<float>(p, s);
  return e == cudaSuccess ? QI_OK : op_fail(QI_ERR_CUDA, "qi_add_rmsnorm_mxfp8: %s", cudaGetErrorString(e));
}
