// Memory-bound operators of batches that share a prompt: the 8-bit K/V cache (write,
// read back) and the residual RMSNorm that ends in an MXFP8 operand.
//
// All work on groups of 8 or 16 consecutive values per thread, so a block of 32 values that
// shares a scale is four or two neighbouring lanes: its largest magnitude takes a shuffle or
// two, and every load and store of a warp is contiguous.
#include <cstdarg>
#include <cstdio>

#include "../../include/qidit.h"
#include "internal.h"
#include "ptx.cuh"

namespace qi {
namespace {

// ---------------------------------------------------------------- values

// 8 values of a 16-bit type from 16 bytes
template <typename T>
__device__ __forceinline__ void unpack8(uint4 w, float (&v)[8]);
template <>
__device__ __forceinline__ void unpack8<__half>(uint4 w, float (&v)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}
template <>
__device__ __forceinline__ void unpack8<__nv_bfloat16>(uint4 w, float (&v)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(u[i] << 16);
    v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
}
template <typename T>
__device__ __forceinline__ void load8(const T* src, float (&v)[8]) {
  unpack8<T>(*reinterpret_cast<const uint4*>(src), v);
}
template <>
__device__ __forceinline__ void load8(const float* src, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(src)[0], b = reinterpret_cast<const float4*>(src)[1];
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
  v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

__device__ __forceinline__ uint4 pack8(const __half*, const float (&v)[8]) {
  return make_uint4(pack_f16x2(v[0], v[1]), pack_f16x2(v[2], v[3]), pack_f16x2(v[4], v[5]), pack_f16x2(v[6], v[7]));
}
__device__ __forceinline__ uint4 pack8(const __nv_bfloat16*, const float (&v)[8]) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                    pack_bf16x2(v[6], v[7]));
}
template <typename T>
__device__ __forceinline__ void store8(T* dst, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(dst) = pack8(dst, v);
}

// 8 values in 16-byte pieces: one of a 16-bit type, two of fp32
template <typename T>
__device__ __forceinline__ void from_pieces(const uint4 (&u)[1], float (&v)[8]) {
  unpack8<T>(u[0], v);
}
template <typename T>
__device__ __forceinline__ void from_pieces(const uint4 (&u)[2], float (&v)[8]) {
  v[0] = __uint_as_float(u[0].x), v[1] = __uint_as_float(u[0].y), v[2] = __uint_as_float(u[0].z);
  v[3] = __uint_as_float(u[0].w), v[4] = __uint_as_float(u[1].x), v[5] = __uint_as_float(u[1].y);
  v[6] = __uint_as_float(u[1].z), v[7] = __uint_as_float(u[1].w);
}
// ... and back; v becomes what was stored
template <typename T>
__device__ __forceinline__ void to_pieces(const T* type, float (&v)[8], uint4 (&u)[1]) {
  u[0] = pack8(type, v);
  unpack8<T>(u[0], v);
}
__device__ __forceinline__ void to_pieces(const float*, float (&v)[8], uint4 (&u)[2]) {
  u[0] = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
  u[1] = make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7]));
}

// 2^n for -127 <= n <= 128 (2^128 = inf)
__device__ __forceinline__ float pow2(int n) {
  return __uint_as_float(n == -127 ? 0x00400000u : static_cast<uint32_t>(n + 127) << 23);
}

// The shared exponent of a block by its largest magnitude: floor(log2 top) - 8 from the exponent
// field; below 2^-119 (zero and subnormals among it) it clamps to -127; an infinity takes 127,
// as in mx_quant32.
__device__ __forceinline__ int mx_exponent(float top) {
  const int field = static_cast<int>(__float_as_uint(top) >> 23);
  return field == 255 ? 127 : max(field - 135, -127);
}
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

// The largest magnitude of 16 packed values, in fp32 (NaNs are passed over; NaN if all are)
__device__ __forceinline__ float absmax16(const uint32_t (&u)[8], const __half*) {
  __half2 m = __habs2(*reinterpret_cast<const __half2*>(&u[0]));
#pragma unroll
  for (int i = 1; i < 8; ++i) m = __hmax2(m, __habs2(*reinterpret_cast<const __half2*>(&u[i])));
  return __half2float(__hmax(__low2half(m), __high2half(m)));
}
__device__ __forceinline__ float absmax16(const uint32_t (&u)[8], const __nv_bfloat16*) {
  __nv_bfloat162 m = __habs2(*reinterpret_cast<const __nv_bfloat162*>(&u[0]));
#pragma unroll
  for (int i = 1; i < 8; ++i) m = __hmax2(m, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&u[i])));
  return __bfloat162float(__hmax(__low2bfloat16(m), __high2bfloat16(m)));
}

// MXFP8 of a block of 32 values held by two neighbouring lanes (16 each): this lane's 16 codes
// and the block's scale byte. Same definition as mx_quant32; the scaling by a power of two is
// exact, so the only rounding is the one to E4M3 (nearest, ties to even).
template <typename T>
__device__ __forceinline__ uint4 mx_quant16(uint4 a, uint4 b, uint32_t& scale) {
  const uint32_t u[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  float top = absmax16(u, static_cast<const T*>(nullptr));
  top = fmaxf(fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1)), 0.f);  // (a block of NaNs counts as zero)
  const int e = mx_exponent(top);
  const float inv = pow2(-e);
  float v[16];
  unpack8<T>(a, *reinterpret_cast<float(*)[8]>(v));
  unpack8<T>(b, *reinterpret_cast<float(*)[8]>(v + 8));
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] *= inv;
  scale = static_cast<uint32_t>(e + 127);
  return make_uint4(e4m3x4(v[0], v[1], v[2], v[3]), e4m3x4(v[4], v[5], v[6], v[7]), e4m3x4(v[8], v[9], v[10], v[11]),
                    e4m3x4(v[12], v[13], v[14], v[15]));
}

// The exponent of a block of 32 values held by four neighbouring lanes (8 each)
__device__ __forceinline__ int mx_exponent8(const float (&v)[8], float& top) {
  top = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(v[i]));
  top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
  return mx_exponent(top);
}

// ---------------------------------------------------------------- 8-bit K/V cache

constexpr int kKv8Threads = 256;
// Groups of K and of V per thread, a block's width apart: all their loads are issued before
// the first is used, so that a warp's loads cover HBM's latency.
constexpr int kKv8Groups = 2;       // write: 16 values each, 128 bytes in flight per thread
constexpr int kKv8ReadGroups = 4;   // read: 8 codes each

// Item i of a sequence, items being a head's 128 values in `1 << LOG` parts: row, head, part, and
// the cache row of the row, or -1 if it is passed over.
struct Kv8At {
  int t, h, part, row;
};
template <int LOG>
__device__ __forceinline__ Kv8At kv8_at(const Kv8Args& a, int i, int n, int pos) {
  Kv8At x;
  const int th = i >> LOG;
  x.part = i & ((1 << LOG) - 1);
  x.t = quot(a.d_H, th);
  x.h = th - x.t * a.H;
  // (pos + t wraps only where pos alone is past any cache, and then to a negative row)
  const int row = static_cast<int>(static_cast<uint32_t>(pos) + static_cast<uint32_t>(x.t));
  x.row = x.t < n && row >= 0 && row < a.S ? row : -1;
  return x;
}
__device__ __forceinline__ long long kv8_offset(const Tensor4& t, const Kv8At& x) {
  return x.t * t.row + x.h * t.head;
}

// Thread = kKv8Groups groups of 16 values of one (row, head) of K and the same of V; two lanes
// share a scale. Bound by issue (71 % of the issue slots) more than by HBM (51 %): with groups of
// 8 and the position worked out for each, 17.7 instructions a value and 26.4 us; now 9.4 and
// 20.3 us (16 prompts of up to 2048 rows, 8 heads; the bytes alone take 16.9 us).
template <typename T>
__global__ void __launch_bounds__(kKv8Threads) kv8_write_kernel(const __grid_constant__ Kv8Args a) {
  grid_dep_wait();
  grid_dep_launch_dependents();
  const int b = blockIdx.y;
  const int n = a.lens ? min(a.lens[b], a.T) : a.T;
  const int pos = a.pos ? a.pos[b] : 0;
  const T* kb = static_cast<const T*>(a.k.data) + b * a.k.batch;
  const T* vb = static_cast<const T*>(a.v.data) + b * a.v.batch;
  const int i0 = static_cast<int>(blockIdx.x) * (kKv8Threads * kKv8Groups) + threadIdx.x;
  uint4 w[kKv8Groups][4];
  Kv8At at[kKv8Groups];
#pragma unroll
  for (int u = 0; u < kKv8Groups; ++u) {
    const Kv8At x = at[u] = kv8_at<3>(a, i0 + u * kKv8Threads, n, pos);
#pragma unroll
    for (int j = 0; j < 4; ++j) w[u][j] = make_uint4(0u, 0u, 0u, 0u);
    if (x.row >= 0) {
      const uint4* ks = reinterpret_cast<const uint4*>(kb + kv8_offset(a.k, x) + x.part * 16);
      const uint4* vs = reinterpret_cast<const uint4*>(vb + kv8_offset(a.v, x) + x.part * 16);
      w[u][0] = ks[0];
      w[u][1] = ks[1];
      w[u][2] = vs[0];
      w[u][3] = vs[1];
    }
  }
#pragma unroll
  for (int u = 0; u < kKv8Groups; ++u) {
    uint4 codes[2];
    uint32_t sf[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      codes[c] = mx_quant16<T>(w[u][2 * c], w[u][2 * c + 1], sf[c]);
      // the head's four scale bytes come together in its first lane
      sf[c] |= __shfl_down_sync(0xffffffffu, sf[c], 2) << 8;
      sf[c] |= __shfl_down_sync(0xffffffffu, sf[c], 4) << 16;
    }
    // (a head's eight lanes are in or out together)
    if (at[u].row >= 0) {
      const long long o = (static_cast<long long>(b) * a.S + at[u].row) * a.H + at[u].h;
      reinterpret_cast<uint4*>(a.k8 + o * kHeadDim)[at[u].part] = codes[0];
      reinterpret_cast<uint4*>(a.v8 + o * kHeadDim)[at[u].part] = codes[1];
      if (at[u].part == 0) {
        reinterpret_cast<uint32_t*>(a.k_sf)[o] = sf[0];
        reinterpret_cast<uint32_t*>(a.v_sf)[o] = sf[1];
      }
    }
  }
}

// 8 codes times their scale, in fp32 (exact: 4 significant bits times a power of two)
__device__ __forceinline__ void mx_values8(uint2 c, uint32_t scale, float (&v)[8]) {
  const float s = pow2(static_cast<int>(scale) - 127);
  const uint32_t w[4] = {c.x & 0xFFFFu, c.x >> 16, c.y & 0xFFFFu, c.y >> 16};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w[i]), __NV_E4M3);
    const float2 f = __half22float2(__half2(h));
    v[2 * i] = f.x * s;
    v[2 * i + 1] = f.y * s;
  }
}

// Bound by HBM: 4 prompts of 1999 rows of 32 heads in 22.2 us, 6.2 TB/s, 91 % of the copy rate.
template <typename T>
__global__ void __launch_bounds__(kKv8Threads) kv8_read_kernel(const __grid_constant__ Kv8Args a) {
  grid_dep_wait();
  grid_dep_launch_dependents();
  const int b = blockIdx.y;
  const int n = a.lens ? min(a.lens[b], a.T) : a.T;
  const int pos = a.pos ? a.pos[b] : 0;
  T* kb = static_cast<T*>(const_cast<void*>(a.k.data)) + b * a.k.batch;
  T* vb = static_cast<T*>(const_cast<void*>(a.v.data)) + b * a.v.batch;
  const int i0 = static_cast<int>(blockIdx.x) * (kKv8Threads * kKv8ReadGroups) + threadIdx.x;
  uint2 kc[kKv8ReadGroups], vc[kKv8ReadGroups];
  uint32_t ks[kKv8ReadGroups], vs[kKv8ReadGroups];
  Kv8At at[kKv8ReadGroups];
#pragma unroll
  for (int u = 0; u < kKv8ReadGroups; ++u) {
    const Kv8At x = at[u] = kv8_at<4>(a, i0 + u * kKv8Threads, n, pos);
    if (x.row >= 0) {
      const long long o = (static_cast<long long>(b) * a.S + x.row) * a.H + x.h;
      kc[u] = reinterpret_cast<const uint2*>(a.k8 + o * kHeadDim)[x.part];
      vc[u] = reinterpret_cast<const uint2*>(a.v8 + o * kHeadDim)[x.part];
      ks[u] = a.k_sf[o * 4 + x.part / 4];
      vs[u] = a.v_sf[o * 4 + x.part / 4];
    }
  }
#pragma unroll
  for (int u = 0; u < kKv8ReadGroups; ++u) {
    if (at[u].row < 0) continue;
    float kv[8], vv[8];
    mx_values8(kc[u], ks[u], kv);
    mx_values8(vc[u], vs[u], vv);
    store8(kb + kv8_offset(a.k, at[u]) + at[u].part * 8, kv);
    store8(vb + kv8_offset(a.v, at[u]) + at[u].part * 8, vv);
  }
}

cudaError_t launch_kv8(void (*kernel)(Kv8Args), Kv8Args a, int parts, int per_block, cudaStream_t s) {
  a.d_H = make_div(a.H);
  const unsigned x = static_cast<unsigned>((static_cast<long long>(a.T) * a.H * parts + per_block - 1) / per_block);
  return launch_dependent(kernel, dim3(x, static_cast<unsigned>(a.B)), dim3(kKv8Threads), 0, s, a);
}

// ---------------------------------------------------------------- residual RMSNorm to MXFP8

// An fp32 value with an error term: hi + lo. Sums and products that keep the rounding
// error of each fp32 operation (Knuth's two-sum, the FMA remainder of a product).
// Where it matters (a value next to a border between two codes, see below) y keeps its error
// term up to the quantiser and is then rounded to odd (the last bit set if anything was lost),
// which makes the rounding to E4M3, and the block's exponent, those of the unrounded value:
// codes differ from the exact ones only by the error of the mean square. Squares are added in
// plain fp32 by twos (two roundings of a sum of terms >= 0), those sums with error terms, so the
// mean is off by less than 2^-23 of itself whatever the row, and y by less than 2^-24. (Chains of
// plain fp32 over all of a thread's values, which a channel far above the others robs of their
// squares: up to 2^-19 at 16384 columns.)
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
// two of them at once: (hi, lo) += x
__device__ __forceinline__ void add_two_sum(uint64_t& hi, uint64_t& lo, uint64_t x) {
  const uint64_t minus = f2_pack(-1.f, -1.f);
  const uint64_t s = add_f32x2(hi, x);
  const uint64_t xx = fma_f32x2(hi, minus, s);  // (a product with -1 is exact: these are differences)
  const uint64_t hh = fma_f32x2(xx, minus, s);
  lo = add_f32x2(lo, add_f32x2(fma_f32x2(hh, minus, hi), fma_f32x2(xx, minus, x)));
  hi = s;
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

// hi + lo (hi its nearest fp32) as the fp32 value between which and the exact one no other lies,
// with an odd last bit unless it is exact
__device__ __forceinline__ float round_odd(F2 x) {
  const uint32_t b = __float_as_uint(x.hi);
  // toward lo: away from zero if the signs agree (hi is not zero where lo is not)
  const uint32_t step = ((__float_as_uint(x.lo) ^ b) >> 31) ? 0xFFFFFFFFu : 1u;
  return __uint_as_float(x.lo == 0.f || (b & 1u) ? b : b + step);
}

// a if x is a number, else b. As one select: from the operator ?: the compiler makes a branch for each
// value, which 2000 rows of 12288 columns show as 84 us instead of 76.
__device__ __forceinline__ float if_number(float x, float a, float b) {
  float r;
  asm("{\n\t.reg .pred p;\n\tsetp.num.f32 p, %1, %1;\n\tselp.f32 %0, %2, %3, p;\n\t}" : "=f"(r) : "f"(x), "f"(a), "f"(b));
  return r;
}

constexpr uint32_t kNear = 16;  // fp32 steps around a border

struct NormParams {
  qi_add_rmsnorm a;
  int groups;          // ceil(rows / 128)
  float n_hi, n_lo;    // 1 / K
};

// The sum of `lanes` (a power of two) neighbouring lanes' values, in each of them
__device__ __forceinline__ F2 lanes_sum(F2 x, int lanes) {
  for (int d = lanes / 2; d; d >>= 1)
    x = add(x, F2{__shfl_xor_sync(0xffffffffu, x.hi, d), __shfl_xor_sync(0xffffffffu, x.lo, d)});
  return x;
}

// One CTA per row. The sum goes to shared memory (as it is stored, in TX) between the two
// passes over it: a thread reads back only what it wrote, so the one barrier is that of the
// reduction, and there is none in a CTA of one warp. 4503 rows of 4096, fp32 with an fp16 delta:
// 37.1 us at 128 threads a row, 80 % of the copy rate. The first pass alone (loads, the sum, its
// store) takes 28.5 us and the arithmetic without stores 26: a CTA's reduction and second pass
// overlap other CTAs' loads, but not wholly. 256 threads 37.4 us, 64 threads 48, one warp 66; rows
// staged by cp.async a row ahead 48 (fewer resident CTAs).
constexpr int kNormUnroll = 2;  // groups of 8 whose loads are issued together
template <typename TX, typename TD>
__global__ void add_rmsnorm_kernel(const __grid_constant__ NormParams p) {
  extern __shared__ __align__(16) uint8_t stash[];
  __shared__ F2 part[32];
  const qi_add_rmsnorm& a = p.a;
  const int groups8 = a.K / 8;
  const int threads = blockDim.x, r = blockIdx.x;
  constexpr int kX = sizeof(TX) / 2, kD = sizeof(TD) / 2;  // 16-byte pieces of a group
  // piece-major, so that a warp's accesses are contiguous
  const auto piece = [&](int c, int j) { return reinterpret_cast<uint4*>(stash) + j * groups8 + c; };
  grid_dep_wait();
  grid_dep_launch_dependents();
  const uint4* x = reinterpret_cast<const uint4*>(static_cast<const TX*>(a.x) + r * a.x_stride);
  const uint4* d = a.delta ? reinterpret_cast<const uint4*>(static_cast<const TD*>(a.delta) + r * a.delta_stride) : nullptr;
  TX* xo = a.x_out ? static_cast<TX*>(a.x_out) + r * a.x_out_stride : nullptr;
  uint64_t sq = 0ull, sq_lo = 0ull;  // two sums and their error terms
  for (int c0 = threadIdx.x; c0 < groups8; c0 += kNormUnroll * threads) {
    uint4 xr[kNormUnroll][kX], dr[kNormUnroll][kD];
#pragma unroll
    for (int i = 0; i < kNormUnroll; ++i) {
      const int c = c0 + i * threads;
      if (c < groups8) {
#pragma unroll
        for (int j = 0; j < kX; ++j) xr[i][j] = x[c * kX + j];
        if (d) {
#pragma unroll
          for (int j = 0; j < kD; ++j) dr[i][j] = d[c * kD + j];
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kNormUnroll; ++i) {
      const int c = c0 + i * threads;
      if (c < groups8) {
        float v[8];
        from_pieces<TX>(xr[i], v);
        if (d) {
          float f[8];
          from_pieces<TD>(dr[i], f);
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] = __fadd_rn(v[k], f[k]);
          to_pieces(static_cast<const TX*>(nullptr), v, xr[i]);
        }
#pragma unroll
        for (int j = 0; j < kX; ++j) {
          *piece(c, j) = xr[i][j];
          if (xo) reinterpret_cast<uint4*>(xo)[c * kX + j] = xr[i][j];
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint64_t lo = f2_pack(v[2 * h], v[2 * h + 1]), hi = f2_pack(v[2 * h + 4], v[2 * h + 5]);
          add_two_sum(sq, sq_lo, fma_f32x2(hi, hi, mul_f32x2(lo, lo)));
        }
      }
    }
  }
  F2 even, odd;
  f2_unpack(sq, even.hi, odd.hi);
  f2_unpack(sq_lo, even.lo, odd.lo);
  F2 sum = lanes_sum(add(even, odd), 32);
  if (threads > 32) {
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = sum;
    __syncthreads();
    const int lane = threadIdx.x & 31;
    sum = lanes_sum(part[lane & (threads / 32 - 1)], threads / 32);
  }
  // mean + eps
  const float mh = __fmul_rn(sum.hi, p.n_hi);
  const float ml = __fmaf_rn(sum.hi, p.n_hi, -mh) + (sum.hi * p.n_lo + sum.lo * p.n_hi);
  const F2 rs = inv_sqrt(add(F2{mh, ml}, F2{a.eps, 0.f}));
  const float r1 = rs.hi + rs.lo;
  const float bias = a.w && a.plus_one ? 1.f : 0.f;
  uint2* codes = reinterpret_cast<uint2*>(a.q + r * static_cast<size_t>(a.K));
  uint32_t* scales = reinterpret_cast<uint32_t*>(a.sf + mx_sf_offset(r, 0, p.groups));
  // (all lanes of a warp run the same rounds: the shuffles need them)
  for (int c = threadIdx.x; (c & ~31) < groups8; c += threads) {
    const bool in = c < groups8;  // groups8 is a multiple of 16: the lanes of a scale block agree
    float v[8] = {}, g[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) g[k] = 1.f;
    if (in) {
      uint4 u[kX];
#pragma unroll
      for (int j = 0; j < kX; ++j) u[j] = *piece(c, j);
      from_pieces<TX>(u, v);
      if (a.w) {
        if (a.w_f32)
          load8(static_cast<const float*>(a.w) + c * 8, g);
        else
          load8(static_cast<const __nv_bfloat16*>(a.w) + c * 8, g);
      }
    }
    // y in fp32: roundings of r1, of 1 + w and of the two products, at most 2 fp32 steps and one
    // of the statistics off, that is within kNear steps with room to spare
    float y[8], top;
#pragma unroll
    for (int k = 0; k < 8; ++k) y[k] = v[k] * r1 * (g[k] + bias);
    int e = mx_exponent8(y, top);
    float inv = pow2(-e);
    // Borders between codes, of the evenly spaced ones below 2^-6 too, and the powers of two at
    // which the exponent changes all have 19 or more zero bits at the end; so has one value in
    // 16000. If any lane's value is that near one, the warp takes the sums with error terms.
    uint32_t near = 0xFFFFFFFFu;
#pragma unroll
    for (int k = 0; k < 8; ++k) near = min(near, __float_as_uint(y[k]) * 8192u + kNear * 8192u);
    if (__any_sync(0xffffffffu, near <= 2 * kNear * 8192u && in)) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const F2 h = two_sum(g[k], bias);
        const float q = __fmul_rn(v[k], rs.hi);
        const float qe = __fmaf_rn(v[k], rs.hi, -q) + v[k] * rs.lo;
        const float z = __fmul_rn(q, h.hi);
        // (an infinite gain or a product past fp32's range stays an infinity: the sum with its error term
        // is no number)
        const F2 t = two_sum(z, __fmaf_rn(q, h.hi, -z) + (qe * h.hi + q * h.lo));
        y[k] = if_number(t.hi, round_odd(t), z);
      }
      e = mx_exponent8(y, top);
      inv = pow2(-e);
    }
    // the four scale bytes of 128 columns are neighbours: they come together in the first lane
    uint32_t scale = static_cast<uint32_t>(e + 127);
    scale |= __shfl_down_sync(0xffffffffu, scale, 4) << 8;
    scale |= __shfl_down_sync(0xffffffffu, scale, 8) << 16;
    if (in) {
      codes[c] = make_uint2(e4m3x4(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv),
                            e4m3x4(y[4] * inv, y[5] * inv, y[6] * inv, y[7] * inv));
      if ((c & 15) == 0) scales[(c >> 4) * static_cast<size_t>(p.groups) * 128] = scale;
    }
  }
}

template <typename TX, typename TD>
cudaError_t launch_norm(const NormParams& p, cudaStream_t s) {
  const int groups8 = p.a.K / 8;
  const int bytes = p.a.K * static_cast<int>(sizeof(TX));
  const auto kernel = add_rmsnorm_kernel<TX, TD>;
  static std::atomic<unsigned long long> attr_done{0};
  const cudaError_t e = ensure_smem_limit(kernel, 64 * 1024, attr_done);
  if (e != cudaSuccess) return e;
  // 128 threads a row where the rows alone fill the GPU; where they do not, as many as halve
  // the row's passes, to 512 (3 rows of 4096: 4.2 us with 128 threads, 2.9 with 512)
  const int most = p.a.rows >= 2 * device_sms() ? 128 : 512;
  int threads = 32;
  while (threads < most && threads < groups8) threads *= 2;
  return launch_dependent(kernel, dim3(static_cast<unsigned>(p.a.rows)), dim3(static_cast<unsigned>(threads)),
                          static_cast<size_t>(bytes), s, p);
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

qi_status kv8_call(const char* name, const qi_kv8* z, Kv8Args* a) {
  if (!z || !z->k || !z->v || !z->k8 || !z->v8 || !z->k_sf || !z->v_sf)
    return op_fail(QI_ERR_INVALID_ARG, "%s: NULL argument", name);
  if (z->dtype != QI_DT_F16 && z->dtype != QI_DT_BF16)
    return op_fail(QI_ERR_INVALID_ARG, "%s: dtype %d", name, z->dtype);
  constexpr int kMost = 1 << 24;
  if (z->B < 1 || z->B > 65535 || z->T < 1 || z->T > kMost || z->S < 1 || z->S > kMost || z->H < 1 || z->H > 65535 ||
      static_cast<long long>(z->T) * z->H >= (1ll << 26))
    return op_fail(QI_ERR_SHAPE, "%s: B %d T %d S %d H %d", name, z->B, z->T, z->S, z->H);
  a->B = z->B;
  a->T = z->T;
  a->S = z->S;
  a->H = z->H;
  a->k = {z->k, z->k_stride.batch, z->k_stride.row, z->k_stride.head};
  a->v = {z->v, z->v_stride.batch, z->v_stride.row, z->v_stride.head};
  for (Tensor4* t : {&a->k, &a->v})
    if (misaligned(t->data, 16) || !good_stride(&t->batch, z->B) || !good_stride(&t->row, z->T) ||
        !good_stride(&t->head, z->H))
      return op_fail(QI_ERR_INVALID_ARG,
                     "%s: k and v need 16-byte alignment and strides that are positive multiples of 8", name);
  if (misaligned(z->k8, 16) || misaligned(z->v8, 16) || misaligned(z->k_sf, 4) || misaligned(z->v_sf, 4) ||
      misaligned(z->pos, 4) || misaligned(z->lens, 4))
    return op_fail(QI_ERR_INVALID_ARG, "%s: codes need 16-byte, scales, pos and lens 4-byte alignment", name);
  a->k8 = z->k8;
  a->v8 = z->v8;
  a->k_sf = z->k_sf;
  a->v_sf = z->v_sf;
  a->pos = z->pos;
  a->lens = z->lens;
  return QI_OK;
}

}  // namespace

cudaError_t launch_kv8_write(const Kv8Args& a, bool bf16, cudaStream_t s) {
  return launch_kv8(bf16 ? kv8_write_kernel<__nv_bfloat16> : kv8_write_kernel<__half>, a, 8, kKv8Threads * kKv8Groups,
                    s);
}
cudaError_t launch_kv8_read(const Kv8Args& a, bool bf16, cudaStream_t s) {
  return launch_kv8(bf16 ? kv8_read_kernel<__nv_bfloat16> : kv8_read_kernel<__half>, a, 16,
                    kKv8Threads * kKv8ReadGroups, s);
}

}  // namespace qi

extern "C" qi_status qi_kv8_write(const qi_kv8* args, qi_stream_t stream) {
  qi::Kv8Args a{};
  const qi_status st = qi::kv8_call("qi_kv8_write", args, &a);
  if (st != QI_OK) return st;
  const cudaError_t e = qi::launch_kv8_write(a, args->dtype == QI_DT_BF16, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? QI_OK : qi::op_fail(QI_ERR_CUDA, "qi_kv8_write: %s", cudaGetErrorString(e));
}

extern "C" qi_status qi_kv8_read(const qi_kv8* args, qi_stream_t stream) {
  qi::Kv8Args a{};
  const qi_status st = qi::kv8_call("qi_kv8_read", args, &a);
  if (st != QI_OK) return st;
  const cudaError_t e = qi::launch_kv8_read(a, args->dtype == QI_DT_BF16, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? QI_OK : qi::op_fail(QI_ERR_CUDA, "qi_kv8_read: %s", cudaGetErrorString(e));
}

extern "C" qi_status qi_add_rmsnorm_mxfp8(const qi_add_rmsnorm* args, qi_stream_t stream) {
  using namespace qi;
  if (!args || !args->x || !args->q || !args->sf)
    return op_fail(QI_ERR_INVALID_ARG, "qi_add_rmsnorm_mxfp8: NULL argument");
  NormParams p{*args, 0, 0.f, 0.f};
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
  p.n_hi = static_cast<float>(1.0 / a.K);
  p.n_lo = static_cast<float>(1.0 / a.K - static_cast<double>(p.n_hi));
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = a.x_dtype == QI_DT_F16    ? launch_norm_d<__half>(p, s)
                        : a.x_dtype == QI_DT_BF16 ? launch_norm_d<__nv_bfloat16>(p, s)
                                                  : launch_norm_d<float>(p, s);
  return e == cudaSuccess ? QI_OK : op_fail(QI_ERR_CUDA, "qi_add_rmsnorm_mxfp8: %s", cudaGetErrorString(e));
}
