// Rows and weight blocks to e4m3 codes with one fp32 scale per 128 elements.
//
//   amax = max |x| over the finite elements of the group (1 x 128 of a row, or
//          128 x 128 of a matrix), at least 2^-100
//   scale = amax / 448,  code = e4m3(x * (448 / amax)), round to nearest even
//
// Both kernels read each input once and write each code once, so HBM bounds
// them: a thread holds its 16 elements per row in registers between the
// maximum and the conversion.
#include "fp8.cuh"
#include "launch.h"

namespace moe {
namespace fp8 {

// 16 consecutive elements as floats
template <typename T>
__device__ __forceinline__ void load16(const T* p, float (&v)[16]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 a = ldg_nc_v4(p + 4 * i);
      v[4 * i] = __uint_as_float(a.x);
      v[4 * i + 1] = __uint_as_float(a.y);
      v[4 * i + 2] = __uint_as_float(a.z);
      v[4 * i + 3] = __uint_as_float(a.w);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint4 a = ldg_nc_v4(p + 8 * i);
      const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float2 f;
        if constexpr (std::is_same<T, __half>::value)
          f = __half22float2(*reinterpret_cast<const __half2*>(&u[j]));
        else
          f = bf16x2_to_f32x2(u[j]);
        v[8 * i + 2 * j] = f.x;
        v[8 * i + 2 * j + 1] = f.y;
      }
    }
  }
}

__device__ __forceinline__ float amax16(const float (&v)[16]) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) m = fmaxf(m, finite_abs(v[i]));
  return m;
}

__device__ __forceinline__ uint4 codes16(const float (&v)[16], float r) {
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    c[i] = e4m3x4(code_arg(v[4 * i], r), code_arg(v[4 * i + 1], r), code_arg(v[4 * i + 2], r),
                  code_arg(v[4 * i + 3], r));
  return make_uint4(c[0], c[1], c[2], c[3]);
}

// One scale per row and 128 columns: 8 threads x 16 elements per group.
template <typename T>
__global__ void __launch_bounds__(256) quant_rows_kernel(const T* __restrict__ x, long long groups,
                                                         int K, int KB, uint8_t* __restrict__ q,
                                                         float* __restrict__ s) {
  pdl_wait();
  pdl_launch();
  const long long g = ((long long)blockIdx.x * 256 + threadIdx.x) >> 3;
  const int l8 = threadIdx.x & 7;
  const bool in = g < groups;
  long long row = 0;
  int kb = 0;
  if (groups <= 0x7fffffffLL) {          // a 32-bit division where it fits
    row = (uint32_t)g / (uint32_t)KB;
    kb = (int)((uint32_t)g - (uint32_t)row * (uint32_t)KB);
  } else {
    row = g / KB;
    kb = (int)(g - row * KB);
  }
  const int col = kb * kBlock + l8 * 16;
  const bool live = in && col < K;        // K % 16 == 0: all 16 or none
  const size_t at = (size_t)row * K + col;
  float v[16];
  if (live) {
    load16(x + at, v);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = 0.f;
  }
  float m = amax16(v);
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (live) *reinterpret_cast<uint4*>(q + at) = codes16(v, rscale_of(m));
  if (in && l8 == 0) s[g] = scale_of(m);
}

// One scale per 128 x 128 block: one CTA of 256 threads per block, 32 rows at
// a time, its 64 elements per thread held in registers.
template <typename T>
__global__ void __launch_bounds__(256) quant_blocks_kernel(const T* __restrict__ x, int rows, int K,
                                                           int KB, uint8_t* __restrict__ q,
                                                           float* __restrict__ s) {
  __shared__ float s_max[8];
  pdl_wait();
  pdl_launch();
  const int kb = blockIdx.x % KB;
  const int rb = blockIdx.x / KB;
  const int col = kb * kBlock + (threadIdx.x & 7) * 16;
  const int r0 = rb * kBlock + (threadIdx.x >> 3);
  float v[4][16];
  float m = 0.f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int r = r0 + 32 * j;
    if (r < rows && col < K) {
      load16(x + (size_t)r * K + col, v[j]);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) v[j][i] = 0.f;
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) m = fmaxf(m, amax16(v[j]));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = m;
  __syncthreads();
  m = s_max[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) m = fmaxf(m, s_max[i]);
  const float r = rscale_of(m);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int rr = r0 + 32 * j;
    if (rr < rows && col < K) *reinterpret_cast<uint4*>(q + (size_t)rr * K + col) = codes16(v[j], r);
  }
  if (threadIdx.x == 0) s[(size_t)rb * KB + kb] = scale_of(m);
}

template <typename T>
static cudaError_t run(const void* x, int rows, int K, int block, void* q, float* s,
                       cudaStream_t st) {
  const int KB = (K + kBlock - 1) / kBlock;
  if (block == 1) {
    const long long groups = (long long)rows * KB;
    const long long ctas = (groups * 8 + 255) / 256;
    if (ctas > 0x7fffffffLL) return cudaErrorNotSupported;
    launch_pdl(quant_rows_kernel<T>, (unsigned)ctas, 256, 0, st, (const T*)x, groups, K, KB,
               (uint8_t*)q, s);
  } else {
    const long long ctas = (long long)((rows + kBlock - 1) / kBlock) * KB;
    if (ctas > 0x7fffffffLL) return cudaErrorNotSupported;
    launch_pdl(quant_blocks_kernel<T>, (unsigned)ctas, 256, 0, st, (const T*)x, rows, K, KB,
               (uint8_t*)q, s);
  }
  return cudaGetLastError();
}

}  // namespace fp8

cudaError_t launch_quantize_fp8(const void* x, int dt, int rows, int K, int block, void* q,
                                float* s, cudaStream_t st) {
  if (dt == MOE_BF16) return fp8::run<__nv_bfloat16>(x, rows, K, block, q, s, st);
  if (dt == MOE_F16) return fp8::run<__half>(x, rows, K, block, q, s, st);
  return fp8::run<float>(x, rows, K, block, q, s, st);
}

}  // namespace moe
