// k_quant.cu -- 8-bit integer rows for the projections: quantisation with one
// scale per row (tg_quantize_rows) and the CUDA-core product
// (tg_linear_quantized with few rows).
#include "tg_device.cuh"
#include "tg_internal.h"

namespace tg {
namespace {

// ---------------------------------------------------------------- quantisation
// amax = max |x|, scale = amax / 127, xq = rint(127 x / amax) (ties to even).
// The integer is the one of the exact quotient: y = x * (127 / amax) in fp32
// is off by at most 127 * 1.5 * 2^-23 < 3e-5, so a y farther than 1e-4 from
// every half-integer rounds as the exact quotient does, and the few others
// are divided in fp64, where 127 x is exact and the rounded quotient (of a
// 31-bit by a 24-bit integer, at most 2^8 large) falls on the right side of
// the half-integer, or on it.
template <typename T>
struct Vec16;
template <>
struct Vec16<__nv_bfloat16> {
  static constexpr int kN = 8;
  static __device__ __forceinline__ void get(const uint4& u, float (&f)[8]) {
    const __nv_bfloat162* e = reinterpret_cast<const __nv_bfloat162*>(&u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 t = __bfloat1622float2(e[i]);
      f[2 * i] = t.x;
      f[2 * i + 1] = t.y;
    }
  }
};
template <>
struct Vec16<float> {
  static constexpr int kN = 4;
  static __device__ __forceinline__ void get(const uint4& u, float (&f)[4]) {
    f[0] = __uint_as_float(u.x);
    f[1] = __uint_as_float(u.y);
    f[2] = __uint_as_float(u.z);
    f[3] = __uint_as_float(u.w);
  }
};

__device__ __forceinline__ uint32_t abs_bits(float f) { return __float_as_uint(f) & 0x7FFFFFFFu; }

__device__ __forceinline__ int quantize_one(float x, float r, float amax) {
  const float y = x * r;
  const float q = rintf(y);
  if (fabsf(fabsf(y - q) - 0.5f) < 1e-4f || !(fabsf(y) < 128.0f))
    return static_cast<int>(rint(127.0 * static_cast<double>(x) / static_cast<double>(amax)));
  return static_cast<int>(q);
}

template <typename T>
__global__ void __launch_bounds__(256) quantize_rows(const T* __restrict__ x, int64_t x_stride,
                                                     int64_t rows, int cols, int8_t* __restrict__ xq,
                                                     float* __restrict__ scale) {
  using V = Vec16<T>;
  pdl_trigger();
  pdl_wait();
  __shared__ uint32_t s_max[8];
  const int64_t row = blockIdx.x;
  const uint4* src = reinterpret_cast<const uint4*>(x + row * x_stride);
  const int n_vec = cols / V::kN;
  uint32_t mx = 0;
  for (int i = threadIdx.x; i < n_vec; i += blockDim.x) {
    float f[V::kN];
    V::get(src[i], f);
#pragma unroll
    for (int j = 0; j < V::kN; ++j) mx = max(mx, abs_bits(f[j]));
  }
  mx = __reduce_max_sync(0xFFFFFFFFu, mx);
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = mx;
  __syncthreads();
  mx = 0;
  for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) mx = max(mx, s_max[w]);
  const bool finite = mx < 0x7F800000u;
  const float amax = __uint_as_float(mx);
  if (threadIdx.x == 0) scale[row] = finite ? amax / 127.0f : __uint_as_float(0x7FC00000u);
  const bool zero = !finite || mx == 0;
  const float r = 127.0f / amax;
  uint32_t* dst = reinterpret_cast<uint32_t*>(xq + row * cols);
  for (int i = threadIdx.x; i < n_vec; i += blockDim.x) {
    float f[V::kN];
    V::get(src[i], f);
#pragma unroll
    for (int j = 0; j < V::kN; j += 4) {
      uint32_t w = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        w |= (static_cast<uint32_t>(zero ? 0 : quantize_one(f[j + e], r, amax)) & 255u) << (8 * e);
      dst[i * (V::kN / 4) + j / 4] = w;
    }
  }
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

cudaError_t launch_quantize_rows(const void* x, int64_t x_stride, int64_t rows, int cols, bool bf16,
                                 int8_t* xq, float* scale, cudaStream_t st) {
  if (rows <= 0) return cudaSuccess;
  const dim3 grid(static_cast<unsigned>(rows));
  if (bf16)
    TG_CUDA_TRY(launch_pdl(quantize_rows<__nv_bfloat16>, grid, dim3(256), 0, st,
                           static_cast<const __nv_bfloat16*>(x), x_stride, rows, cols, xq, scale));
  else
    TG_CUDA_TRY(launch_pdl(quantize_rows<float>, grid, dim3(256), 0, st,
                           static_cast<const float*>(x), x_stride, rows, cols, xq, scale));
  return cudaGetLastError();
}

cudaError_t launch_quant_gemm(const QuantGemmArgs& g, cudaStream_t st) {
  if (g.m <= 0) return cudaSuccess;
  // Up to four rows the warps' dot products need no tensor core (1 x 4096 x
  // 2048: 3.9 us, narrow 4.9). Above, the narrow tiles until the wide ones
  // come near to a wave of CTA pairs (200 x 4096 x 2048, 16 wide tiles: narrow
  // 10.2 us, wide 14.2; 1024 x 4096 x 2048, 64: 14.7 and 14.6; 512 x 12288 x
  // 2048, 96: 26.1 and 21.3).
  const int64_t wide_tiles = (g.m + 255) / 256 * ((g.n + 255) / 256);
  if (g.m > 4) return wide_tiles < 64 ? launch_quant_gemm_narrow(g, st) : launch_quant_gemm_wide(g, st);
  const dim3 grid(static_cast<unsigned>((g.n + 8 * kGvCols - 1) / (8 * kGvCols)),
                  static_cast<unsigned>((g.m + kGvRows - 1) / kGvRows));
  if (g.bf16) TG_CUDA_TRY(launch_pdl(quant_gemv<__nv_bfloat16>, grid, dim3(256), 0, st, g));
  else TG_CUDA_TRY(launch_pdl(quant_gemv<float>, grid, dim3(256), 0, st, g));
  return cudaGetLastError();
}

}  // namespace tg
