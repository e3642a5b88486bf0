// Projections with 4-bit weights: y[r][n] = sum_k x[r][k] w[n][k],
// w[n][k] = code[n][k] * scale[n][k / group].
//
// One warp per weight row: lanes read the packed codes 8 at a time and
// carry up to 8 rows of x.

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "gdn_internal.cuh"

namespace gdn {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kRows = 8;

__device__ __forceinline__ float ld1(const float *p) { return __ldg(p); }
__device__ __forceinline__ float ld1(const __nv_bfloat16 *p) {
  return __bfloat162float(*p);
}
__device__ __forceinline__ void st1(float *p, float x) { *p = x; }
__device__ __forceinline__ void st1(__nv_bfloat16 *p, float x) {
  *p = __float2bfloat16_rn(x);
}

template <typename T>
__global__ void __launch_bounds__(128)
    quant_linear_kernel(const T *__restrict__ x, const uint8_t *__restrict__ qw,
                        const __half *__restrict__ sc, T *__restrict__ y,
                        int rows, int N, int K, int group) {
  const int lane = threadIdx.x & 31;
  const size_t n = (size_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (n >= (size_t)N) return;
  const uint32_t *wp = reinterpret_cast<const uint32_t *>(qw + n * (K / 2));
  const __half *sp = sc + n * (K / group);
  for (int r0 = 0; r0 < rows; r0 += kRows) {
    const int nr = min(kRows, rows - r0);
    float acc[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) acc[r] = 0.f;
    for (int k = 8 * lane; k < K; k += 256) {
      const uint32_t u = __ldg(wp + (k >> 3));
      const float s = __half2float(sp[k / group]);
      float w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = s * (float)((int)(u << (28 - 4 * i)) >> 28);
#pragma unroll
      for (int r = 0; r < kRows; ++r)
        if (r < nr) {
          const T *xp = x + (size_t)(r0 + r) * K + k;
#pragma unroll
          for (int i = 0; i < 8; ++i) acc[r] = fmaf(ld1(xp + i), w[i], acc[r]);
        }
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
#pragma unroll
      for (int d = 16; d; d >>= 1) acc[r] += __shfl_xor_sync(kFull, acc[r], d);
      if (r < nr && lane == 0) st1(y + (size_t)(r0 + r) * N + n, acc[r]);
    }
  }
}

}  // namespace

cudaError_t launch_quant_linear(const void *x, const unsigned char *qw,
                                const void *scales, void *y, int rows, int N,
                                int K, int group, bool bf16,
                                cudaStream_t stream) {
  if (rows == 0 || N == 0) return cudaSuccess;
  const unsigned blocks = (unsigned)(((size_t)N + 3) / 4);
  const __half *sc = static_cast<const __half *>(scales);
  if (bf16)
    quant_linear_kernel<<<blocks, 128, 0, stream>>>(
        static_cast<const __nv_bfloat16 *>(x), qw, sc,
        static_cast<__nv_bfloat16 *>(y), rows, N, K, group);
  else
    quant_linear_kernel<<<blocks, 128, 0, stream>>>(
        static_cast<const float *>(x), qw, sc, static_cast<float *>(y), rows, N,
        K, group);
  return cudaGetLastError();
}

}  // namespace gdn
