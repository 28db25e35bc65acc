// k_quant.cu -- 8-bit integer rows for the projections: quantisation with one
// scale per row (tg_quantize_rows) and the CUDA-core product
// (tg_linear_quantized with few rows).
#include <algorithm>

#include "tg_device.cuh"
#include "tg_internal.h"

namespace tg {
namespace {

// ---------------------------------------------------------------- quantisation
// amax = max |x|, scale = amax / 127, xq = rint(127 x / amax) (ties to even).
// Bound by HBM: each row is read once (held in registers) and written once.
// That leaves about ten instructions an element: t = fma(x, 127 / amax, 1.5 *
// 2^23) has the rounded integer in its low bits, and e = x * 127 / amax minus
// it says how near the border it was. The integer is the one of the exact
// quotient: 127 / amax is rounded (2^-24 relative), so the product is off by at
// most 127 * 2^-24 < 8e-6, and where |e| is within 1e-5 of a half (0.4% of bf16
// values: quotients of 8-bit mantissas often are ties) the side is decided
// exactly. (Each such quotient in fp64 instead: 171 us for 32768 x 6144.)
template <typename T>
struct Vec16;
template <>
struct Vec16<__nv_bfloat16> {
  static constexpr int kN = 8;
  // elements 4 i .. 4 i + 3 of a 16-byte vector
  static __device__ __forceinline__ void get4(const uint4& u, int i, float (&f)[4]) {
    const uint32_t a = i == 0 ? u.x : u.z, b = i == 0 ? u.y : u.w;
    f[0] = __uint_as_float(a << 16);
    f[1] = __uint_as_float(a & 0xFFFF0000u);
    f[2] = __uint_as_float(b << 16);
    f[3] = __uint_as_float(b & 0xFFFF0000u);
  }
  // running largest magnitudes, of the even and the odd elements (a NaN stays)
  using Top = __nv_bfloat162;
  static __device__ __forceinline__ Top none() { return __floats2bfloat162_rn(0.f, 0.f); }
  static __device__ __forceinline__ Top top(const uint4& u, Top m) {
    const Top* e = reinterpret_cast<const Top*>(&u);
    return __hmax2_nan(__hmax2_nan(m, __hmax2_nan(__habs2(e[0]), __habs2(e[1]))),
                       __hmax2_nan(__habs2(e[2]), __habs2(e[3])));
  }
  // as the bits of an fp32 magnitude
  static __device__ __forceinline__ uint32_t bits(Top m) {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(&m) & 0x7FFF7FFFu;
    return max(w << 16, w & 0xFFFF0000u);
  }
};
template <>
struct Vec16<float> {
  static constexpr int kN = 4;
  static __device__ __forceinline__ void get4(const uint4& u, int, float (&f)[4]) {
    f[0] = __uint_as_float(u.x);
    f[1] = __uint_as_float(u.y);
    f[2] = __uint_as_float(u.z);
    f[3] = __uint_as_float(u.w);
  }
  using Top = uint32_t;
  static __device__ __forceinline__ Top none() { return 0u; }
  static __device__ __forceinline__ Top top(const uint4& u, Top m) {
    return max(m, max(max(u.x & 0x7FFFFFFFu, u.y & 0x7FFFFFFFu), max(u.z & 0x7FFFFFFFu, u.w & 0x7FFFFFFFu)));
  }
  static __device__ __forceinline__ uint32_t bits(Top m) { return m; }
};

// The integer of 127 x / amax where the product x r may be on the wrong side of a
// border (amax within 2^+-64 of 1, r = 127 / amax rounded): c is the border, and
// the sign of 127 x - c amax comes from two exact parts of the product c amax.
__device__ __forceinline__ uint32_t quantize_exact(float x, float r, float amax) {
  constexpr float kMagic = 12582912.0f;
  float q = fmaf(x, r, kMagic) - kMagic;
  const float e = fmaf(x, r, -q);
  if (fabsf(e) > 0.49999f) {
    const float c = q + copysignf(0.5f, e);
    const float hi = c * amax, lo = fmaf(c, amax, -hi), d = fmaf(127.0f, x, -hi);
    q = d > lo ? c + 0.5f : d < lo ? c - 0.5f : rintf(c);
  }
  return __float_as_uint(q + kMagic);
}

struct QuantRow {
  float r;             // 127 / amax
  float shift;         // 1, or the power of two that brings amax near 1
  float r_near, amax;  // after it
};

// Four integers in a word.
__device__ __forceinline__ uint32_t quantize4(const float (&f)[4], const QuantRow& a) {
  constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23
  const float2 magic = make_float2(kMagic, kMagic), r = make_float2(a.r, a.r), one = make_float2(-1.f, -1.f);
  const float2 x = make_float2(f[0], f[1]), y = make_float2(f[2], f[3]);
  const float2 tx = ffma2(x, r, magic), ty = ffma2(y, r, magic);
  const float2 ex = ffma2(x, r, ffma2(tx, one, magic)), ey = ffma2(y, r, ffma2(ty, one, magic));
  uint32_t q[4] = {__float_as_uint(tx.x), __float_as_uint(tx.y), __float_as_uint(ty.x),
                   __float_as_uint(ty.y)};
  const float worst = fmaxf(fmax3f(fabsf(ex.x), fabsf(ex.y), fabsf(ey.x)), fabsf(ey.y));
  if (!(worst <= 0.49999f)) {  // (127 / amax infinite: NaN, or 1e7 and more)
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = quantize_exact(f[i] * a.shift, a.r_near, a.amax);
  }
  return __byte_perm(__byte_perm(q[0], q[1], 0x0040), __byte_perm(q[2], q[3], 0x0040), 0x5410);
}

// kWarps warps a row; the first kHold vectors of each thread stay in registers.
template <typename T, int kWarps, int kHold>
__global__ void __launch_bounds__(256) quantize_rows(const T* __restrict__ x, int64_t x_stride,
                                                     int64_t rows, int cols, int8_t* __restrict__ xq,
                                                     float* __restrict__ scale) {
  using V = Vec16<T>;
  constexpr int kThreads = kWarps * 32;
  __shared__ uint32_t s_max[8];
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x % kThreads;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (8 / kWarps) + threadIdx.x / kThreads;
  const bool on = row < rows;
  const uint4* src = reinterpret_cast<const uint4*>(x + (on ? row : 0) * x_stride);
  const int n_vec = on ? cols / V::kN : 0;
  uint4 u[kHold];
#pragma unroll
  for (int i = 0; i < kHold; ++i) {
    const int at = tid + i * kThreads;
    u[i] = at < n_vec ? __ldg(src + at) : make_uint4(0u, 0u, 0u, 0u);
  }
  typename V::Top top = V::none();
#pragma unroll
  for (int i = 0; i < kHold; ++i) top = V::top(u[i], top);
  for (int at = tid + kHold * kThreads; at < n_vec; at += kThreads) top = V::top(__ldg(src + at), top);
  uint32_t mx = __reduce_max_sync(0xFFFFFFFFu, V::bits(top));
  if constexpr (kWarps > 1) {
    if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = mx;
    __syncthreads();
    const int w0 = threadIdx.x / kThreads * kWarps;
    mx = s_max[w0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) mx = max(mx, s_max[w0 + w]);
  }
  if (!on) return;
  const bool finite = mx < 0x7F800000u;
  const float amax = __uint_as_float(mx);
  if (tid == 0) scale[row] = finite ? amax / 127.0f : __uint_as_float(0x7FC00000u);
  const bool zero = !finite || mx == 0;
  QuantRow a;
  a.r = 127.0f / amax;
  a.shift = amax < 5.4210109e-20f ? 1.8446744e19f : amax > 1.8446744e19f ? 5.4210109e-20f : 1.0f;  // 2^+-64
  a.amax = amax * a.shift;
  a.r_near = 127.0f / a.amax;
  uint32_t* dst = reinterpret_cast<uint32_t*>(xq + row * cols);
  auto put = [&](const uint4& w, int at) {
    uint32_t q[V::kN / 4];
#pragma unroll
    for (int i = 0; i < V::kN / 4; ++i) {
      float f[4];
      V::get4(w, i, f);
      q[i] = zero ? 0u : quantize4(f, a);
    }
    if constexpr (V::kN == 8) *reinterpret_cast<uint2*>(dst + 2 * at) = make_uint2(q[0], q[1]);
    else dst[at] = q[0];
  };
#pragma unroll
  for (int i = 0; i < kHold; ++i)
    if (tid + i * kThreads < n_vec) put(u[i], tid + i * kThreads);
  for (int at = tid + kHold * kThreads; at < n_vec; at += kThreads) put(__ldg(src + at), at);
}

// ---------------------------------------------------------------- product, few rows
// y[i, j] = (sum_k xq[i, k] wq[j, k]) xs[i] ws[j] (+ residual). One warp per
// four output channels and up to four rows of x: the lanes split k in
// 16-byte pieces, the weights stream from memory once, the rows of x come
// from the L1 cache. Sums of products of 8-bit integers in 32-bit integers
// are exact (k <= 131071).
constexpr int kGvCols = 4, kGvRows = 4;

__device__ __forceinline__ int dot16(const int4& a, const int4& b, int c) {
  c = __dp4a(a.x, b.x, c);
  c = __dp4a(a.y, b.y, c);
  c = __dp4a(a.z, b.z, c);
  return __dp4a(a.w, b.w, c);
}

template <typename T>
__global__ void __launch_bounds__(256) quant_gemv(const __grid_constant__ QuantGemmArgs g) {
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t n0 = (static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5)) * kGvCols;
  const int64_t m0 = static_cast<int64_t>(blockIdx.y) * kGvRows;
  if (n0 >= g.n) return;
  int acc[kGvRows][kGvCols] = {};
  const int rows = static_cast<int>(min(static_cast<int64_t>(kGvRows), g.m - m0));
  for (int kk = lane * 16; kk < g.k; kk += 512) {
    int4 w[kGvCols];
#pragma unroll
    for (int c = 0; c < kGvCols; ++c)
      w[c] = *reinterpret_cast<const int4*>(g.w + (n0 + c) * g.k + kk);
#pragma unroll
    for (int r = 0; r < kGvRows; ++r) {
      if (r < rows) {
        const int4 xv = *reinterpret_cast<const int4*>(g.x + (m0 + r) * g.k + kk);
#pragma unroll
        for (int c = 0; c < kGvCols; ++c) acc[r][c] = dot16(xv, w[c], acc[r][c]);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < kGvRows; ++r) {
    if (r >= rows) break;
#pragma unroll
    for (int c = 0; c < kGvCols; ++c) {
      const int sum = __reduce_add_sync(0xFFFFFFFFu, acc[r][c]);
      if (lane == c) {
        const int64_t at = (m0 + r) * g.n + n0 + c;
        float v = static_cast<float>(sum) * g.xs[m0 + r] * g.ws[n0 + c];
        if constexpr (sizeof(T) == 4) {
          if (g.residual) v += static_cast<const float*>(g.residual)[at];
          static_cast<float*>(g.y)[at] = v;
        } else {
          if (g.residual) v += __bfloat162float(static_cast<const __nv_bfloat16*>(g.residual)[at]);
          static_cast<__nv_bfloat16*>(g.y)[at] = __float2bfloat16_rn(v);
        }
      }
    }
  }
}

}  // namespace

template <typename T>
static cudaError_t run_quantize(const T* x, int64_t x_stride, int64_t rows, int cols, int8_t* xq,
                                float* scale, cudaStream_t st) {
  // as few warps a row as hold it in three or four vectors a thread (32768 x 6144
  // on 8 warps: 110 us with three, 119 with four of which one is empty)
  const int n_vec = cols / Vec16<T>::kN;
  auto go = [&](auto kern, int warps) {
    const int per = 8 / warps;
    return launch_pdl(kern, dim3(static_cast<unsigned>((rows + per - 1) / per)), dim3(256), 0, st, x,
                      x_stride, rows, cols, xq, scale);
  };
  if (n_vec <= 128) return go(quantize_rows<T, 1, 4>, 1);
  if (n_vec <= 256) return go(quantize_rows<T, 2, 4>, 2);
  if (n_vec <= 512) return go(quantize_rows<T, 4, 4>, 4);
  if (n_vec <= 768) return go(quantize_rows<T, 8, 3>, 8);
  return go(quantize_rows<T, 8, 4>, 8);
}

cudaError_t launch_quantize_rows(const void* x, int64_t x_stride, int64_t rows, int cols, bool bf16,
                                 int8_t* xq, float* scale, cudaStream_t st) {
  if (rows <= 0) return cudaSuccess;
  if (bf16)
    return run_quantize(static_cast<const __nv_bfloat16*>(x), x_stride, rows, cols, xq, scale, st);
  return run_quantize(static_cast<const float*>(x), x_stride, rows, cols, xq, scale, st);
}

cudaError_t launch_quant_gemm(const QuantGemmArgs& g, cudaStream_t st) {
  if (g.m <= 0) return cudaSuccess;
  // Up to four rows the warps' dot products need no tensor core (1 x 4096 x
  // 2048: 3.9 us, narrow 4.9). Above, the narrow tiles, whose k can be split,
  // until the wide ones fill a third of the SMs (512 x 2048, 16 wide tiles: k =
  // 1024 narrow 9.9 us, wide 9.5; 6144 18.8 and 21.6; 700 x 2048, 24: 10.2 and 9.5,
  // 22.6 and 23.8; 1024 x 2048, 32: 10.7 and 9.6, 24.7 and 22.7); to a wave of them
  // where a wide tile would be half empty (64 x 12288 x 2048, 48: 10.2 and 13.9).
  const int64_t wide_tiles = (g.m + 255) / 256 * ((g.n + 255) / 256);
  if (g.m > 4)
    return wide_tiles < (g.m <= 128 ? 64 : 24) ? launch_quant_gemm_narrow(g, st)
                                               : launch_quant_gemm_wide(g, st);
  const dim3 grid(static_cast<unsigned>((g.n + 8 * kGvCols - 1) / (8 * kGvCols)),
                  static_cast<unsigned>((g.m + kGvRows - 1) / kGvRows));
  if (g.bf16) TG_CUDA_TRY(launch_pdl(quant_gemv<__nv_bfloat16>, grid, dim3(256), 0, st, g));
  else TG_CUDA_TRY(launch_pdl(quant_gemv<float>, grid, dim3(256), 0, st, g));
  return cudaGetLastError();
}

}  // namespace tg
