// Products of e4m3 rows with e4m3 weights by weight-streaming kernels: few
// token rows per weight row, bound by the weights' bytes.
//
//   y[m][n] = sum_kb xs[m][kb] ws[n / 128][kb] sum_{k in kb} x[m][k] w[n][k]
//
// kb runs over the blocks of 128 along K. The products of one block are added
// by mma.sync m16n8k32 (e4m3 operands, fp32 accumulation; their products are
// exact), then the block's sum is scaled and added in fp32.
//
// A CTA takes 16 weight rows (GLU: 16 gate and 16 up rows) and up to 8 token
// rows at a time (a dense product of more rows: 32, so that the weights are
// read a quarter as often): its 8 warps share out the K blocks, so that even a narrow
// product has every block's loads in flight at once, and add their sums in
// order through shared memory. The MMA sums over k in any order, so each lane
// loads 16 consecutive codes of its row and feeds them as four registers of
// two MMAs, the same way for weights and tokens: 16-byte loads, no
// conversion, nothing staged.
//
// Bound by latency at these sizes (one B200: one row, N = 4096, K = 7168, 29 MB of
// codes, 8.9 us, 0.50 of the measured HBM rate; one token through 8 of 128 experts'
// gate|up, 25 MB, 10.0 us, 0.38): every warp has up to four k-blocks of weights on
// their way, three CTAs (gate|up) or two share an SM.
//
// gate|up: eight such CTAs form a cluster that covers 128 features, the block
// that shares one scale of the quantised result; the rows' largest magnitudes
// are exchanged through distributed shared memory.
#include <cooperative_groups.h>

#include "fp8.cuh"
#include "launch.h"

namespace moe {
namespace fp8s {

using namespace fp8;
namespace cg = cooperative_groups;

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kRows = 16;              // weight rows of one matrix per CTA (MMA M)
constexpr int kTok = 8;                // token rows at a time (MMA N)
constexpr int kCluster = kBlock / kRows;

struct Params {
  const uint8_t* x;          // token codes [.][K]
  const float* xs;           // [.][KB]
  const uint32_t* row_map;   // row of x of each sorted row; null: the row itself
  const int32_t* row_off;    // null: one dense product of M rows
  const int32_t* tile_off;
  int BM, M, E;
  int N;                     // output columns (GLU: features F)
  int K, KB;
  const uint8_t* w;          // [E][rows_per_group][K]
  const float* ws;           // [E][scale_rows][KB]
  int rows_per_group, scale_rows;
  void* out;                 // [.][N]: out_dt, or (GLU) codes
  float* out_s;              // GLU: [.][N / 128]
  int out_dt, act;
  int* status;               // fp16 range reports (null: none)
};

__device__ __forceinline__ void mma_e4m3(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The CTA's products of MATS matrices of 16 weight rows (the lane's two rows at
// wa, scales at wsc) with token rows [r0, r0 + nv), nv <= 8 NT, left in
// red[warp][mat][row][token] by each warp.
template <int MATS, int NT>
__device__ __forceinline__ void tile_products(const Params& p, const uint8_t* const (&wa)[MATS][2],
                                              const float* const (&wsc)[MATS], int r0, int nv,
                                              float* red) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  // rows past the tile repeat its last one; their results are not stored
  auto row_of = [&](int i) {
    const int r = r0 + min(i, nv - 1);
    return p.row_map ? (size_t)__ldg(p.row_map + r) : (size_t)r;
  };
  const uint8_t* xr[NT];
  const float* sc[NT][2];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    xr[t] = p.x + row_of(t * kTok + g) * p.K;
    sc[t][0] = p.xs + row_of(t * kTok + 2 * c) * p.KB;
    sc[t][1] = p.xs + row_of(t * kTok + 2 * c + 1) * p.KB;
  }
  float acc[MATS][NT][4];
#pragma unroll
  for (int m = 0; m < MATS; ++m)
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[m][t][i] = 0.f;
  const uint4 z = make_uint4(0, 0, 0, 0);
  // UN k-blocks' weights are loaded at once, before any token row is looked at
  constexpr int UN = MATS == 1 && NT == 1 ? 4 : MATS == 1 ? 2 : 1;
  for (int kb0 = warp; kb0 < p.KB; kb0 += kWarps * UN) {
    uint4 a[UN][MATS][2][2];
#pragma unroll
    for (int u = 0; u < UN; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int k0 = (kb0 + u * kWarps) * kBlock + h * 64 + c * 16;   // K % 16 == 0: all 16 or none
        const bool in = k0 < p.K;
#pragma unroll
        for (int m = 0; m < MATS; ++m) {
          a[u][m][h][0] = in ? ldg_nc_v4(wa[m][0] + k0) : z;
          a[u][m][h][1] = in ? ldg_nc_v4(wa[m][1] + k0) : z;
        }
      }
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      const int kb = kb0 + u * kWarps;
      if (kb >= p.KB) break;
      float sw[MATS];
#pragma unroll
      for (int m = 0; m < MATS; ++m) sw[m] = __ldg(wsc[m] + kb);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        uint4 b[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int k0 = kb * kBlock + h * 64 + c * 16;
          b[h] = k0 < p.K ? __ldg(reinterpret_cast<const uint4*>(xr[t] + k0)) : z;
        }
        const float t0 = __ldg(sc[t][0] + kb), t1 = __ldg(sc[t][1] + kb);
#pragma unroll
        for (int m = 0; m < MATS; ++m) {
          float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint4 &v0 = a[u][m][h][0], &v1 = a[u][m][h][1];
            mma_e4m3(d, v0.x, v1.x, v0.y, v1.y, b[h].x, b[h].y);
            mma_e4m3(d, v0.z, v1.z, v0.w, v1.w, b[h].z, b[h].w);
          }
          acc[m][t][0] = fmaf(d[0], sw[m] * t0, acc[m][t][0]);
          acc[m][t][1] = fmaf(d[1], sw[m] * t1, acc[m][t][1]);
          acc[m][t][2] = fmaf(d[2], sw[m] * t0, acc[m][t][2]);
          acc[m][t][3] = fmaf(d[3], sw[m] * t1, acc[m][t][3]);
        }
      }
    }
  }
#pragma unroll
  for (int m = 0; m < MATS; ++m)
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float* o = red + ((warp * MATS + m) * NT + t) * (kRows * kTok);
      *reinterpret_cast<float2*>(o + g * kTok + 2 * c) = make_float2(acc[m][t][0], acc[m][t][1]);
      *reinterpret_cast<float2*>(o + (g + 8) * kTok + 2 * c) =
          make_float2(acc[m][t][2], acc[m][t][3]);
    }
  __syncthreads();
}

// the warps' sums added in order
template <int MATS, int NT>
__device__ __forceinline__ float sum_warps(const float* red, int m, int row, int tok) {
  const float* o = red + (m * NT + tok / kTok) * (kRows * kTok) + row * kTok + tok % kTok;
  float v = o[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) v += o[w * MATS * NT * kRows * kTok];
  return v;
}

// Rows [r0, r0 + nv) and expert of tile `tau`; false past the last tile.
template <int NT>
__device__ __forceinline__ bool tile_rows(const Params& p, int tau, int& e, int& r0, int& nv) {
  if (!p.row_off) {
    e = 0;
    r0 = tau * NT * kTok;
    nv = min(NT * kTok, p.M - r0);
    return nv > 0;
  }
  if (tau >= __ldg(p.tile_off + p.E)) return false;
  e = expert_of_tile_warp(p.tile_off, p.E, tau);
  r0 = __ldg(p.row_off + e) + (tau - __ldg(p.tile_off + e)) * p.BM;
  nv = min(p.BM, __ldg(p.row_off + e + 1) - r0);
  return true;
}

// Columns n0..n0+15 of y, for the rows of the tiles blockIdx.y, + gridDim.y, ...
template <int NT>
__global__ void __launch_bounds__(kThreads, 2) stream_store_kernel(const Params p) {
  __shared__ __align__(16) float red[kWarps * NT * kRows * kTok];
  pdl_wait();
  pdl_launch();
  const int n0 = blockIdx.x * kRows;
  const int g = (threadIdx.x & 31) >> 2;
  bool over = false;
  for (int tau = blockIdx.y;; tau += gridDim.y) {
    int e, r0, nv;
    if (!tile_rows<NT>(p, tau, e, r0, nv)) break;
    const uint8_t* we = p.w + (size_t)e * p.rows_per_group * p.K;
    // rows past N repeat the last one; their results are not stored
    const uint8_t* const wa[1][2] = {{we + (size_t)min(n0 + g, p.N - 1) * p.K,
                                      we + (size_t)min(n0 + g + 8, p.N - 1) * p.K}};
    const float* const wsc[1] = {p.ws + ((size_t)e * p.scale_rows + n0 / kBlock) * p.KB};
    for (int i = 0; i < nv; i += NT * kTok) {
      tile_products<1, NT>(p, wa, wsc, r0 + i, min(NT * kTok, nv - i), red);
      for (int o = threadIdx.x; o < NT * kTok * kRows; o += kThreads) {
        const int row = o % kRows, tok = o / kRows;
        if (i + tok >= nv || n0 + row >= p.N) continue;
        const float v = sum_warps<1, NT>(red, 0, row, tok);
        const size_t at = (size_t)(r0 + i + tok) * p.N + n0 + row;
        if (p.out_dt == MOE_F16) {
          const __half h = __float2half_rn(v);
          over |= (__half_as_ushort(h) & 0x7FFFu) >= 0x7C00u;
          reinterpret_cast<__half*>(p.out)[at] = h;
        } else if (p.out_dt == MOE_BF16) {
          reinterpret_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(v);
        } else {
          reinterpret_cast<float*>(p.out)[at] = v;
        }
      }
      __syncthreads();
    }
  }
  if (over) report_status(p.status, MOE_ERR_RANGE);
}

// Features f0..f0+15 of h = act(g) * u, quantised over the cluster's 128.
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads, 3)
    stream_glu_kernel(const Params p) {
  __shared__ __align__(16) float red[kWarps * 2 * kRows * kTok];
  __shared__ float s_max[2][kTok];
  pdl_wait();
  pdl_launch();
  cg::cluster_group cluster = cg::this_cluster();
  const int f0 = blockIdx.x * kRows;
  const int g = (threadIdx.x & 31) >> 2;
  const int row = threadIdx.x & 15, tok = threadIdx.x >> 4;      // threads 0..127
  unsigned it = 0;
  for (int tau = blockIdx.y;; tau += gridDim.y) {
    int e, r0, nv;
    if (!tile_rows<1>(p, tau, e, r0, nv)) break;    // the same in all CTAs of the cluster
    const uint8_t* wg = p.w + ((size_t)e * p.rows_per_group + f0 + g) * p.K;
    const uint8_t* wu = wg + (size_t)p.N * p.K;
    const uint8_t* const wa[2][2] = {{wg, wg + (size_t)8 * p.K}, {wu, wu + (size_t)8 * p.K}};
    const float* sg = p.ws + ((size_t)e * p.scale_rows + f0 / kBlock) * p.KB;
    const float* const wsc[2] = {sg, sg + (size_t)(p.N / kBlock) * p.KB};
    for (int i = 0; i < nv; i += kTok, ++it) {
      tile_products<2, 1>(p, wa, wsc, r0 + i, min(kTok, nv - i), red);
      float h = 0.f;
      float(*mx)[kTok] = s_max + (it & 1);
      if (threadIdx.x < kRows * kTok) {
        h = glu_codes(p.act, sum_warps<2, 1>(red, 0, row, tok), sum_warps<2, 1>(red, 1, row, tok));
        float m = finite_abs(h);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (row == 0) (*mx)[tok] = m;
      }
      // the maxima of this pass alternate between two arrays: a CTA passes
      // the next barrier only when every CTA has read this pass's
      cluster.sync();
      if (threadIdx.x < kRows * kTok && i + tok < nv) {
        float m = 0.f;
#pragma unroll
        for (int r = 0; r < kCluster; ++r)
          m = fmaxf(m, *cluster.map_shared_rank(&(*mx)[tok], r));
        const size_t at = (size_t)(r0 + i + tok) * p.N + f0 + row;
        reinterpret_cast<uint8_t*>(p.out)[at] = e4m3x1(code_arg(h, rscale_of(m)));
        if (row == 0 && cluster.block_rank() == 0)
          p.out_s[(size_t)(r0 + i + tok) * (p.N / kBlock) + f0 / kBlock] = scale_of(m);
      }
      __syncthreads();
    }
  }
  cluster.sync();        // no CTA leaves while another may read its maxima
}

}  // namespace fp8s

static unsigned grid_y(long long tiles) { return (unsigned)(tiles < 65535 ? tiles : 65535); }

cudaError_t launch_fp8_matmul_stream(const void* a, const float* sa, const void* b, const float* sb,
                                     int M, int N, int K, int out_dt, void* y, int* status,
                                     cudaStream_t s) {
  using namespace fp8s;
  Params p{};
  p.x = (const uint8_t*)a;
  p.xs = sa;
  p.M = M;
  p.E = 1;
  p.N = N;
  p.K = K;
  p.KB = (K + kBlock - 1) / kBlock;
  p.w = (const uint8_t*)b;
  p.ws = sb;
  p.rows_per_group = N;
  p.scale_rows = (N + kBlock - 1) / kBlock;
  p.out = y;
  p.out_dt = out_dt;
  p.status = status;
  const unsigned gx = (unsigned)((N + kRows - 1) / kRows);
  auto gy = [&](int nt) { return grid_y(((long long)M + nt * kTok - 1) / (nt * kTok)); };
  if (M <= 8)
    launch_pdl(stream_store_kernel<1>, dim3(gx, gy(1)), kThreads, 0, s, p);
  else
    launch_pdl(stream_store_kernel<4>, dim3(gx, gy(4)), kThreads, 0, s, p);
  return cudaGetLastError();
}

cudaError_t launch_swiglu_fp8_stream(const void* xq, const float* xs, const uint32_t* row_map,
                                     const int32_t* row_off, const int32_t* tile_off, int BM, int R,
                                     const moe_experts& ex, void* hq, float* hs, cudaStream_t s) {
  using namespace fp8s;
  if (R <= 0) return cudaSuccess;
  Params p{};
  p.x = (const uint8_t*)xq;
  p.xs = xs;
  p.row_map = row_map;
  p.row_off = row_off;
  p.tile_off = tile_off;
  p.BM = BM;
  p.E = ex.E;
  p.N = ex.F;
  p.K = ex.d;
  p.KB = ex.d / kBlock;
  p.w = (const uint8_t*)ex.w_gu;
  p.ws = (const float*)ex.s_gu;
  p.rows_per_group = 2 * ex.F;
  p.scale_rows = 2 * ex.F / kBlock;
  p.out = hq;
  p.out_s = hs;
  p.act = ex.act;
  const dim3 grid((unsigned)(ex.F / kRows), grid_y(max_tiles(R, ex.E, BM)));
  launch_pdl(stream_glu_kernel, grid, kThreads, 0, s, p);
  return cudaGetLastError();
}

cudaError_t launch_down_fp8_stream(const void* hq, const float* hs, const int32_t* row_off,
                                   const int32_t* tile_off, int BM, int R, const moe_experts& ex,
                                   void* ys, int* status, cudaStream_t s) {
  using namespace fp8s;
  if (R <= 0) return cudaSuccess;
  Params p{};
  p.x = (const uint8_t*)hq;
  p.xs = hs;
  p.row_off = row_off;
  p.tile_off = tile_off;
  p.BM = BM;
  p.E = ex.E;
  p.N = ex.d;
  p.K = ex.F;
  p.KB = ex.F / kBlock;
  p.w = (const uint8_t*)ex.w_dn;
  p.ws = (const float*)ex.s_dn;
  p.rows_per_group = ex.d;
  p.scale_rows = ex.d / kBlock;
  p.out = ys;
  p.out_dt = MOE_F16;
  p.status = status;
  const dim3 grid((unsigned)(ex.d / kRows), grid_y(max_tiles(R, ex.E, BM)));
  launch_pdl(stream_store_kernel<1>, grid, kThreads, 0, s, p);
  return cudaGetLastError();
}

}  // namespace moe
