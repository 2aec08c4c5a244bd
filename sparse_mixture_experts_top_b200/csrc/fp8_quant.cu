// Rows and weight blocks to e4m3 codes with one fp32 scale per 128 elements.
//
//   amax = max |x| over the finite elements of the group (1 x 128 of a row, or
//          128 x 128 of a matrix), at least 2^-100
//   scale = amax / 448,  code = e4m3(x * (448 / amax)), round to nearest even
//
// Both kernels read each input once and write each code once, so HBM bounds
// them: a thread holds its 16 elements per row in registers between the
// maximum and the conversion. 4096 x 7168 fp16 rows take 14.5 us and 90112 x
// 2048 fp32 weights in blocks 145 us on one B200, 0.94 and 0.97 of the measured
// HBM rate.
#include "fp8.cuh"
#include "launch.h"

namespace moe {
namespace fp8 {

// 16 consecutive elements as they are stored, the largest magnitude of the
// finite ones, and their codes. A thread with an infinity or a NaN (the
// largest bit pattern says so) goes through its elements one by one; the
// others need no test per element, and 16-bit magnitudes are compared two to
// an instruction, as integers.
template <typename T>
struct Elems {
  static constexpr bool kWide = sizeof(T) == 4;
  static constexpr uint32_t kInf = std::is_same<T, __half>::value ? 0x7C00u : 0x7F80u;
  uint32_t u[kWide ? 16 : 8];
  bool odd;                          // some element is not finite

  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < (kWide ? 4 : 2); ++i) {
      const uint4 a = ldg_nc_v4(reinterpret_cast<const uint4*>(p) + i);
      u[4 * i] = a.x;
      u[4 * i + 1] = a.y;
      u[4 * i + 2] = a.z;
      u[4 * i + 3] = a.w;
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < (kWide ? 16 : 8); ++i) u[i] = 0;
  }
  __device__ __forceinline__ float at(int i) const {
    if constexpr (kWide) return __uint_as_float(u[i]);
    const uint32_t h = u[i / 2] >> (i % 2 * 16) & 0xFFFFu;
    if constexpr (std::is_same<T, __half>::value) return __half2float(__ushort_as_half((uint16_t)h));
    return bf16_bits_to_f32(h);
  }
  __device__ __forceinline__ float amax() {
    float m = 0.f;
    if constexpr (kWide) {
#pragma unroll
      for (int i = 0; i < 16; ++i) m = fmaxf(m, fabsf(at(i)));     // passes over NaN
      odd = m > FLT_MAX;
    } else {
      uint32_t x = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) x = __vmaxu2(x, u[i] & 0x7FFF7FFFu);
      const uint32_t h = max(x & 0xFFFFu, x >> 16);
      odd = h >= kInf;
      m = std::is_same<T, __half>::value ? __half2float(__ushort_as_half((uint16_t)h))
                                         : bf16_bits_to_f32(h);
    }
    if (odd) {
      m = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) m = fmaxf(m, finite_abs(at(i)));
    }
    return m;
  }
  __device__ __forceinline__ uint4 codes(float r) const {
    uint32_t c[4];
    if (odd) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        c[i] = e4m3x4(code_arg(at(4 * i), r), code_arg(at(4 * i + 1), r),
                      code_arg(at(4 * i + 2), r), code_arg(at(4 * i + 3), r));
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        c[i] = e4m3x4(at(4 * i) * r, at(4 * i + 1) * r, at(4 * i + 2) * r, at(4 * i + 3) * r);
    }
    return make_uint4(c[0], c[1], c[2], c[3]);
  }
};

// One scale per row and 128 columns: 8 threads x 16 elements per group, UN
// groups per thread whose loads go out together.
template <typename T>
constexpr int row_groups() { return sizeof(T) == 4 ? 1 : 2; }

template <typename T>
__global__ void __launch_bounds__(256) quant_rows_kernel(const T* __restrict__ x, long long groups,
                                                         int K, int KB, uint8_t* __restrict__ q,
                                                         float* __restrict__ s) {
  constexpr int UN = row_groups<T>();
  pdl_wait();
  pdl_launch();
  const int l8 = threadIdx.x & 7;
  Elems<T> v[UN];
  size_t at[UN];
  bool live[UN];
#pragma unroll
  for (int j = 0; j < UN; ++j) {
    const long long g = ((long long)blockIdx.x * UN + j) * 32 + (threadIdx.x >> 3);
    long long row;
    int kb;
    if (groups <= 0x7fffffffLL) {          // a 32-bit division where it fits
      row = (uint32_t)g / (uint32_t)KB;
      kb = (int)((uint32_t)g - (uint32_t)row * (uint32_t)KB);
    } else {
      row = g / KB;
      kb = (int)(g - row * KB);
    }
    const int col = kb * kBlock + l8 * 16;
    live[j] = g < groups && col < K;        // K % 16 == 0: all 16 or none
    at[j] = (size_t)row * K + col;
    if (live[j]) v[j].load(x + at[j]); else v[j].zero();
  }
#pragma unroll
  for (int j = 0; j < UN; ++j) {
    float m = v[j].amax();
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (live[j]) *reinterpret_cast<uint4*>(q + at[j]) = v[j].codes(rscale_of(m));
    const long long g = ((long long)blockIdx.x * UN + j) * 32 + (threadIdx.x >> 3);
    if (g < groups && l8 == 0) s[g] = scale_of(m);
  }
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
  Elems<T> v[4];
  float m = 0.f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int r = r0 + 32 * j;
    if (r < rows && col < K) v[j].load(x + (size_t)r * K + col); else v[j].zero();
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) m = fmaxf(m, v[j].amax());
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
    if (rr < rows && col < K) *reinterpret_cast<uint4*>(q + (size_t)rr * K + col) = v[j].codes(r);
  }
  if (threadIdx.x == 0) s[(size_t)rb * KB + kb] = scale_of(m);
}

template <typename T>
static cudaError_t run(const void* x, int rows, int K, int block, void* q, float* s,
                       cudaStream_t st) {
  const int KB = (K + kBlock - 1) / kBlock;
  if (block == 1) {
    const long long groups = (long long)rows * KB;
    const long long per_cta = 32 * row_groups<T>();
    const long long ctas = (groups + per_cta - 1) / per_cta;
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
