// Products of e4m3 rows with e4m3 weights on the tensor cores (tcgen05 / TMEM /
// TMA): the dense product and the grouped expert products of many rows.
//
//   y[m][n] = sum_kb xs[m][kb] ws[n / 128][kb] sum_{k in kb} x[m][k] w[n][k]
//
// A unit of work is 128 token rows (the MMA's M, one per TMEM lane) x BN weight
// rows (its N). One k-block is 128 codes, the block that shares a scale, and
// also one 128-byte row of a swizzled tile, so a stage of the TMA ring is one
// k-block. The MMA's accumulator cannot take a factor per row and block, so
// each k-block's products go to a TMEM buffer of their own, and eight warps
// read it back, scale it and add it to fp32 registers while the tensor core
// fills the next buffer. With token rows on the lanes, the factor
// xs[m][kb] ws[.][kb] is one value per thread and 64 columns: one FMA per element.
//
// Warps: 0 loads by TMA (a stage's weight rows in one copy, its token rows in
// another: with the token rows in four copies the product below took 147 instead
// of 123 us, about 65 cycles a copy), 1 issues the
// MMAs, 2 and 3 gather token rows through row_map (16-byte asynchronous copies
// into the same swizzled layout; TMA's four-row gathers were slower), 4..11
// scale, add and store: warp w reads TMEM lanes 32 (w % 4) .., and half (w - 4) / 4 of the
// columns. Register shares: 88 per thread for warps 0..3, 208 for warps 4..11
// (their sums of up to 128 columns live in registers), 168 at launch: 128 x 88 +
// 256 x 208 = 384 x 168. With 72 and 216 the gathering warps spilled more (gate|up of
// 20,480 rows over 512 experts 257 against 238 us sustained); with these the gate|up
// forms spill 24 or 36 bytes a thread and the 16-bit persistent ones 20.
//
// gate|up: the unit's weight rows are 128 gate and the 128 up rows of the same
// features, so a thread holds both for 64 features; the GLU's result is
// quantised in the same epilogue, its block's largest magnitude exchanged
// between the two halves through shared memory.
//
// Two forms:
//   * persistent (one CTA per SM, BN = 256): units enough to go round;
//   * split (BN = 128; gate|up 256): few units. A cluster of up to eight CTAs
//     shares a unit's K blocks; each leaves its sums in its shared memory, and
//     each then adds a share of the rows over the cluster, in rank order, and
//     stores them: all SMs stream weights, and the result stays the same from
//     run to run.
//
// What bounds it, on one B200: many rows, the hand-over of the two accumulator
// buffers and the clock under the power cap (4096 x 4096 x 7168: 116 us in a
// burst, 134 us sustained, 0.63 and 0.54 of twice the measured bf16 rate: 902 cycles
// a k-block; an MMA with its commit, read-back and scaling, operands resident, takes
// 563, the MMAs alone 512, and the 48 KB that a k-block writes to and the 48 KB that
// it reads from shared memory 768 at 128 bytes a cycle); few rows, the weights' bytes
// (down of 256 rows over 128 experts 27.4 us, 0.99 of the measured HBM rate; gate|up of
// 20,480 rows over 512 experts 204 us, 0.81). A pair of CTAs on one tile (cta_group::2) moves a
// third less through shared memory but hands buffers over between SMs: 145 against
// 149 us sustained in an earlier state of the kernel, not kept and not measured
// again since; MMAs of N = 128 with four buffers read the token rows twice: slower.
//
// Every mbarrier wait is bounded, as in the other tensor-core kernels; the
// cluster barriers are reached by every thread, whatever the waits did.
#include <cooperative_groups.h>

#include "fp8.cuh"
#include "launch.h"
#include "tc_ptx.cuh"

namespace moe {
namespace fp8tc {

using namespace fp8;
using namespace tc;

constexpr int BM = 128;                 // token rows per unit (the sort tables' BM)
constexpr int kMaxE = 1024;
constexpr int kThreads = 384;
constexpr int kAccWarp0 = 4;
constexpr int kAccWarps = 8;
constexpr int A_BYTES = BM * kBlock;
// token rows of a tile's copy: the least of these that holds it
constexpr int A_MAPS = 3;
__host__ __device__ constexpr int a_rows(int i) { return 32 << i; }
constexpr int kGatherThreads = 64;      // warps 2 and 3

// a product stored in one of the three types, or gate|up with one of the gate
// activations: fixed at compile time, which keeps the epilogues short
enum { MODE_F32 = MOE_F32, MODE_BF16 = MOE_BF16, MODE_F16 = MOE_F16, MODE_SWIGLU, MODE_GEGLU };
__host__ __device__ constexpr bool is_glu(int mode) { return mode == MODE_SWIGLU || mode == MODE_GEGLU; }
__host__ __device__ constexpr int act_of(int mode) {
  return mode == MODE_GEGLU ? MOE_ACT_GEGLU_TANH : MOE_ACT_SWIGLU;
}

template <int BN, bool SPLIT> struct Cfg {
  static constexpr int B_BYTES = BN * kBlock;
  static constexpr int STAGE = A_BYTES + B_BYTES;
  static constexpr int NS = BN == 256 ? 4 : 6;
  static constexpr int NBUF = 512 / BN;             // accumulator buffers
  static constexpr int COLS = BN / 2;               // columns per scaling warp
  static constexpr int BARS = 256;
  static constexpr int AMAX = 2 * 2 * BM * 4;       // [tile parity][half][row]
  static constexpr int TABLES = 2 * (kMaxE + 1) * 4;
  static constexpr int PATCH_LD = 17;               // 32 rows x 16 columns of one warp
  static constexpr int PATCH = SPLIT ? 0 : kAccWarps * 32 * PATCH_LD * 4;
  static constexpr int SMEM = 1024 + NS * STAGE + BARS + AMAX + TABLES + PATCH + 16;
  // split: the CTA's sums, in the ring once its last MMA is done
  static constexpr int SUM_LD = BN + 4;             // rows 4 banks apart: 16-byte stores
  static_assert(!SPLIT || BM * SUM_LD * 4 <= NS * STAGE, "the sums fit the ring");
  static_assert(SMEM <= 232448, "shared memory per CTA");
};

struct Params {
  CUtensorMap tmA[A_MAPS];   // token rows [.][K]: boxes of 128 x a_rows(i)
  CUtensorMap tmB;           // weight rows: a stage's box (gate|up: 3-D, both blocks)
  CUtensorMap tmB1;          // 128 rows: a last unit of at most 128 columns
  const uint8_t* x;          // token codes, for the gather
  const float* xs;           // [.][KB] scales of the token rows
  const uint32_t* row_map;   // GLU: token row of each sorted row
  const int32_t* row_off;    // null: one dense product of M rows
  const int32_t* tile_off;
  int M, E;
  int N;                     // output columns (GLU: features F)
  int K, KB;
  int n_units;               // units per token tile
  int split;                 // CTAs that share a unit's K blocks (1: persistent form)
  const float* ws;           // [E][scale_rows][KB]
  int rows_per_group, scale_rows;
  void* out;
  float* out_s;              // GLU: [.][N / 128]
  int wide;                  // every output row starts on a 32-byte boundary
  int* status;
  long long wait_limit;
};

// M = 128, N = n, e4m3 x e4m3, fp32 accumulators, both operands K-major
__device__ __forceinline__ uint32_t idesc_e4m3(int n) {
  return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(BM >> 4) << 24);
}

// The four MMAs (K-steps of 32 codes) of one k-block into a fresh accumulator;
// warp-uniform operands, one elected lane issues.
__device__ __forceinline__ void mma_block(uint32_t d, uint32_t alo, uint32_t ahi, uint32_t blo,
                                          uint32_t bhi, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred pf, pt, e;\n\t.reg .b64 a0, a1, a2, a3, b0, b1, b2, b3;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 pf, %5, %5;\n\t"
      "setp.eq.b32 pt, %5, %5;\n\t"
      "mov.b64 a0, {%1, %2};\n\tmov.b64 b0, {%3, %4};\n\t"
      "add.u32 %1, %1, 2;\n\tadd.u32 %3, %3, 2;\n\t"
      "mov.b64 a1, {%1, %2};\n\tmov.b64 b1, {%3, %4};\n\t"
      "add.u32 %1, %1, 2;\n\tadd.u32 %3, %3, 2;\n\t"
      "mov.b64 a2, {%1, %2};\n\tmov.b64 b2, {%3, %4};\n\t"
      "add.u32 %1, %1, 2;\n\tadd.u32 %3, %3, 2;\n\t"
      "mov.b64 a3, {%1, %2};\n\tmov.b64 b3, {%3, %4};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a0, b0, %5, pf;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a1, b1, %5, pt;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a2, b2, %5, pt;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a3, b3, %5, pt;\n\t}\n"
      : "+r"(d), "+r"(alo), "+r"(ahi), "+r"(blo), "+r"(bhi)
      : "r"(idesc)
      : "memory");
}

// a 3-D box: the same rows of consecutive matrices
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* tm, int x, int y, int z,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// arrives on the barrier (one of its count) once this thread's copies have landed
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// 16 columns of this warp's 32 lanes. The registers are written until the
// wait, which takes them as operands, so that nothing reads them before it.
__device__ __forceinline__ void tmem_ld_start(uint32_t ta, uint32_t (&a)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3]), "=r"(a[4]), "=r"(a[5]), "=r"(a[6]), "=r"(a[7]), "=r"(a[8]), "=r"(a[9]), "=r"(a[10]), "=r"(a[11]), "=r"(a[12]), "=r"(a[13]), "=r"(a[14]), "=r"(a[15])
      : "r"(ta)
      : "memory");
}
__device__ __forceinline__ void tmem_ld_wait(uint32_t (&a)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(a[0]), "+r"(a[1]), "+r"(a[2]), "+r"(a[3]), "+r"(a[4]), "+r"(a[5]), "+r"(a[6]), "+r"(a[7]), "+r"(a[8]), "+r"(a[9]), "+r"(a[10]), "+r"(a[11]), "+r"(a[12]), "+r"(a[13]), "+r"(a[14]), "+r"(a[15])
               :
               : "memory");
}

// acc += d * f for two columns at a time
__device__ __forceinline__ void fma2(float& x, float& y, uint32_t d0, uint32_t d1, float f) {
  asm("{\n\t.reg .b64 a, b, c;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %4};\n\tmov.b64 c, {%0, %1};\n\t"
      "fma.rn.f32x2 c, a, b, c;\n\tmov.b64 {%0, %1}, c;\n\t}"
      : "+f"(x), "+f"(y)
      : "r"(d0), "r"(d1), "f"(f));
}

// 32 bytes to a 32-byte-aligned address: one whole sector per lane
__device__ __forceinline__ void st32(void* p, const uint32_t (&v)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

template <int R> __device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R> __device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}

struct Unit {
  int e, r0, nv, unit;       // expert, first row, rows, unit within the tile
};

__device__ __forceinline__ int total_units(const Params& p, const int* s_toff) {
  return (p.row_off ? s_toff[p.E] : (p.M + BM - 1) / BM) * p.n_units;
}

__device__ __forceinline__ Unit decode(const Params& p, const int* s_toff, const int* s_roff,
                                       int u) {
  Unit r;
  const int tile = u / p.n_units;
  r.unit = u - tile * p.n_units;
  if (!p.row_off) {
    r.e = 0;
    r.r0 = tile * BM;
    r.nv = min(BM, p.M - r.r0);
    return r;
  }
  int lo = 0, hi = p.E - 1;              // the largest e with tile_off[e] <= tile
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (s_toff[mid] <= tile) lo = mid; else hi = mid - 1;
  }
  r.e = lo;
  r.r0 = s_roff[lo] + (tile - s_toff[lo]) * BM;
  r.nv = min(BM, s_roff[lo + 1] - r.r0);
  return r;
}

// One value, rounded to the output type.
template <int DT>
__device__ __forceinline__ void store_one(void* out, size_t at, float v, bool& over) {
  if constexpr (DT == MODE_F16) {
    const __half h = __float2half_rn(v);
    over |= (__half_as_ushort(h) & 0x7FFFu) >= 0x7C00u;
    reinterpret_cast<__half*>(out)[at] = h;
  } else if constexpr (DT == MODE_BF16) {
    reinterpret_cast<__nv_bfloat16*>(out)[at] = __float2bfloat16_rn(v);
  } else {
    reinterpret_cast<float*>(out)[at] = v;
  }
}

template <int DT>
__device__ __forceinline__ uint32_t pack_two(float a, float b, uint32_t& hmax) {
  if constexpr (DT == MODE_BF16) return pack_bf16x2(a, b);
  const uint32_t v = pack_f16x2(a, b);
  hmax = max(hmax, max(v & 0x7FFFu, (v >> 16) & 0x7FFFu));
  return v;
}

// four consecutive values to one 8- or 16-byte aligned place (N % 4 == 0)
template <int DT>
__device__ __forceinline__ void store_four(void* out, size_t at, const float* v, bool& over) {
  if constexpr (DT == MODE_F32) {
    *reinterpret_cast<float4*>(reinterpret_cast<float*>(out) + at) =
        make_float4(v[0], v[1], v[2], v[3]);
  } else {
    uint32_t hmax = 0;
    const uint2 o = make_uint2(pack_two<DT>(v[0], v[1], hmax), pack_two<DT>(v[2], v[3], hmax));
    over |= hmax >= 0x7C00u;
    *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(out) + at) = o;
  }
}

// A lane's output row: COLS consecutive columns from column c of N. Where every
// row starts on a 32-byte boundary each lane stores whole sectors of its row;
// elsewhere 16 columns at a time go through shared memory (the warp's patch),
// and half a warp stores those of one row.
template <int DT, int COLS, int LD>
__device__ __forceinline__ void store_rows(const Params& p, int r0, int m0, int nv, int c,
                                           const float (&acc)[COLS], float* patch, bool& over) {
  const int lane = threadIdx.x & 31;
  const int m = m0 + lane;
  if (!p.wide) {
#pragma unroll
    for (int j = 0; j < COLS; j += 16) {
      if (c + j >= p.N) break;                     // the same in the whole warp
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 16; ++i) patch[lane * LD + i] = acc[j + i];
      __syncwarp();
      const int col = c + j + (lane & 15);
      for (int r = lane >> 4; r < 32 && m0 + r < nv; r += 2)
        if (col < p.N)
          store_one<DT>(p.out, ((size_t)r0 + m0 + r) * p.N + col, patch[r * LD + (lane & 15)], over);
    }
    return;
  }
  if (m >= nv) return;
  const size_t at = ((size_t)r0 + m) * p.N + c;
  if constexpr (DT == MODE_F32) {
    float* o = reinterpret_cast<float*>(p.out) + at;
#pragma unroll
    for (int j = 0; j < COLS; j += 8) {
      uint32_t v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = __float_as_uint(acc[j + i]);
      if (c + j < p.N) st32(o + j, v);
    }
  } else {
    uint16_t* o = reinterpret_cast<uint16_t*>(p.out) + at;
    uint32_t hmax = 0;
#pragma unroll
    for (int j = 0; j < COLS; j += 16) {
      if (c + j < p.N) {                           // N % 16 == 0
        uint32_t v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = pack_two<DT>(acc[j + 2 * i], acc[j + 2 * i + 1], hmax);
        st32(o + j, v);
      }
    }
    over |= hmax >= 0x7C00u;
  }
}

// address of a shared-memory place in CTA `rank` of the cluster, and four floats there
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, int rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float4 ld_cluster(uint32_t addr) {
  float4 f;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(f.x), "=f"(f.y), "=f"(f.z), "=f"(f.w)
               : "r"(addr)
               : "memory");
  return f;
}

// Split form: the sums of rows [0, nv) of the unit over the cluster's CTAs, a
// warp for RJ rows at a time (KU of the CTAs' sums of each on their way), and
// their storage. Every CTA takes a share of the rows. The code is kept short:
// it runs once per launch, and a body of several hundred instructions took
// longer to arrive (a thousand cycles for four rows) than to execute. Bound by
// the reads of the other CTAs' sums, about 25 bytes a cycle.
template <int MODE, int BN, int LD, int RJ, int KU>
__device__ __forceinline__ void join_rows(const Params& p, const Unit& t, uint32_t sums, int rank,
                                          bool& over) {
  constexpr int V = BN / 32;               // columns per lane, in runs of 128 columns
  const int warp = (threadIdx.x >> 5) - kAccWarp0, lane = threadIdx.x & 31;
  const bool four = p.N % 4 == 0;
  const int step = p.split * kAccWarps;
#pragma unroll 1
  for (int r0 = rank * kAccWarps + warp; r0 < t.nv; r0 += step * RJ) {
    float v[RJ][V];
#pragma unroll
    for (int j = 0; j < RJ; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) v[j][i] = 0.f;
#pragma unroll 1
    for (int k0 = 0; k0 < p.split; k0 += KU) {
      float4 f[RJ][KU][V / 4];
#pragma unroll
      for (int j = 0; j < RJ; ++j)
#pragma unroll
        for (int k = 0; k < KU; ++k) {
          // (rows past the tile and CTAs past the cluster: the first again)
          const uint32_t s = map_rank(
              sums + (uint32_t)((r0 + j * step < t.nv ? r0 + j * step : r0) * LD + lane * 4) * 4,
              k0 + k < p.split ? k0 + k : rank);
#pragma unroll
          for (int i = 0; i < V / 4; ++i) f[j][k][i] = ld_cluster(s + i * 512);
        }
#pragma unroll
      for (int j = 0; j < RJ; ++j)
#pragma unroll
        for (int k = 0; k < KU; ++k)
          if (k0 + k < p.split) {
#pragma unroll
            for (int i = 0; i < V / 4; ++i) {
              v[j][4 * i] += f[j][k][i].x;
              v[j][4 * i + 1] += f[j][k][i].y;
              v[j][4 * i + 2] += f[j][k][i].z;
              v[j][4 * i + 3] += f[j][k][i].w;
            }
          }
    }
#pragma unroll
    for (int j = 0; j < RJ; ++j) {
      if (r0 + j * step >= t.nv) break;
      const size_t row = (size_t)t.r0 + r0 + j * step;
      if constexpr (is_glu(MODE)) {
        // 4 gate columns and their 4 up columns per lane
        float mx = 0.f, h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          h[i] = glu_codes(act_of(MODE), v[j][i], v[j][4 + i]);
          mx = fmaxf(mx, finite_abs(h[i]));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        const float f = rscale_of(mx);
        const size_t at = row * p.N + t.unit * kBlock + lane * 4;
        *reinterpret_cast<uint32_t*>(reinterpret_cast<uint8_t*>(p.out) + at) =
            e4m3x4(code_arg(h[0], f), code_arg(h[1], f), code_arg(h[2], f), code_arg(h[3], f));
        if (lane == 0) p.out_s[row * (p.N / kBlock) + t.unit] = scale_of(mx);
      } else {
        const int col = t.unit * BN + lane * 4;
        const size_t at = row * p.N + col;
        if (four) {
          if (col < p.N) store_four<MODE>(p.out, at, v[j], over);
        } else {
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (col + c < p.N) store_one<MODE>(p.out, at + c, v[j][c], over);
        }
      }
    }
  }
}

// What a scaling thread needs of a unit: its row's scales, its columns' scales
// (gate|up: those of the gate and of the up half), and the first of each.
struct Lead {
  const float *sa, *w0, *w1;
  float a, b0, b1;
  int r0, nv, unit;
};
template <bool GLU, int BN>
__device__ __forceinline__ Lead lead(const Params& p, const Unit t, int m, int c0, int kb) {
  Lead l;
  l.r0 = t.r0;
  l.nv = t.nv;
  l.unit = t.unit;
  int xrow = t.r0 + min(m, t.nv - 1);
  if (GLU) xrow = (int)__ldg(p.row_map + xrow);
  l.sa = p.xs + (size_t)xrow * p.KB + kb;
  // (columns past N have no scale of their own and are not stored)
  const int n = GLU ? t.unit : min((t.unit * BN + c0) / kBlock, p.scale_rows - 1);
  l.w0 = p.ws + ((size_t)t.e * p.scale_rows + n) * p.KB + kb;
  l.w1 = GLU ? l.w0 + (size_t)(p.N / kBlock) * p.KB : l.w0;
  l.a = __ldg(l.sa);
  l.b0 = __ldg(l.w0);
  l.b1 = GLU ? __ldg(l.w1) : 0.f;
  return l;
}

template <int MODE, int BN, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
    fp8_tc_kernel(const __grid_constant__ Params p) {
  constexpr bool GLU = is_glu(MODE);
  using C = Cfg<BN, SPLIT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~(uintptr_t)1023);
  const uint32_t st_base = smem_u32(smem);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::NS * C::STAGE);   // [NS]
  uint64_t* empty = full + C::NS;                                          // [NS]
  uint64_t* acc_full = empty + C::NS;                                      // [NBUF]
  uint64_t* acc_empty = acc_full + C::NBUF;                                // [NBUF]
  uint64_t* rows_full = acc_empty + C::NBUF;                               // [NS]
  uint64_t* xchg = rows_full + C::NS;                                      // [1]
  uint64_t* drain = xchg + 1;                                              // [1]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  float* s_amax = reinterpret_cast<float*>(smem + C::NS * C::STAGE + C::BARS);
  int* s_toff = reinterpret_cast<int*>(smem + C::NS * C::STAGE + C::BARS + C::AMAX);
  int* s_roff = s_toff + kMaxE + 1;
  float* s_patch = reinterpret_cast<float*>(
      smem + C::NS * C::STAGE + C::BARS + C::AMAX + ((C::TABLES + 15) & ~15));
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::NS; ++i) {
      mbar_init(smem_u32(full + i), 1);                     // TMA
      mbar_init(smem_u32(rows_full + i), kGatherThreads);   // gathered token rows
      mbar_init(smem_u32(empty + i), 1);
    }
    for (int i = 0; i < C::NBUF; ++i) {
      mbar_init(smem_u32(acc_full + i), 1);
      mbar_init(smem_u32(acc_empty + i), kAccWarps);
    }
    mbar_init(smem_u32(xchg), kAccWarps);
    mbar_init(smem_u32(drain), 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&p.tmB)) : "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tmem_slot)),
                 "n"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  pdl_wait();
  pdl_launch();
  if (p.row_off) {
    for (int i = threadIdx.x; i <= p.E; i += kThreads) {
      s_toff[i] = __ldg(p.tile_off + i);
      s_roff[i] = __ldg(p.row_off + i);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int total = total_units(p, s_toff);
  // the CTA's units, and its share of their K blocks
  const int rank = SPLIT ? (int)(blockIdx.x % (unsigned)p.split) : 0;
  const int u0 = SPLIT ? (int)(blockIdx.x / (unsigned)p.split) : (int)blockIdx.x;
  const int u_step = SPLIT ? total : (int)gridDim.x;      // split: one unit
  const int kb_lo = SPLIT ? (int)((long long)p.KB * rank / p.split) : 0;
  const int kb_hi = SPLIT ? (int)((long long)p.KB * (rank + 1) / p.split) : p.KB;

  if (warp < kAccWarp0) {
    regs_dec<88>();
    if (warp == 0) {
      // ---------------------------------------------------------- loads (TMA)
      uint32_t it = 0;
      bool ok = true;
      if (lane == 0) {
        for (int u = u0; u < total && ok; u += u_step) {
          const Unit t = decode(p, s_toff, s_roff, u);
          const int wrow = t.e * p.rows_per_group + t.unit * BN;
          // a last unit of at most 128 columns loads that many weight rows (the
          // rest of the stage keeps old codes, whose columns are not stored)
          const bool narrow = !GLU && BN > kBlock && p.N - t.unit * BN <= kBlock;
          const int am = t.nv <= a_rows(0) ? 0 : t.nv <= a_rows(1) ? 1 : 2;
          const uint32_t bytes = (GLU ? 0u : (uint32_t)(a_rows(am) * kBlock)) +
                                 (narrow ? (uint32_t)(kBlock * kBlock) : (uint32_t)C::B_BYTES);
          for (int kb = kb_lo; kb < kb_hi; ++kb, ++it) {
            const uint32_t s = it % C::NS;
            if (it >= (uint32_t)C::NS) {
              ok = mbar_wait(smem_u32(empty + s), ((it / C::NS) - 1) & 1, abort_flag, p.status,
                             true, p.wait_limit);
              if (!ok) break;
            }
            const uint32_t dst = st_base + s * C::STAGE;
            const uint32_t bar = smem_u32(full + s);
            const int x = kb * kBlock;
            mbar_arrive_tx(bar, bytes);
            if constexpr (GLU) {
              tma_load_3d(dst + A_BYTES, &p.tmB, x, t.unit * kBlock, 2 * t.e, bar);
            } else {
              tma_load_2d(dst + A_BYTES, narrow ? &p.tmB1 : &p.tmB, x, wrow, bar);
              tma_load_2d(dst, &p.tmA[am], x, t.r0, bar);
            }
          }
        }
        for (uint32_t i = 0; i < (uint32_t)C::NS && i < it; ++i) {
          const uint32_t last = it - 1 - i;
          mbar_wait(smem_u32(full + last % C::NS), (last / C::NS) & 1, abort_flag, p.status, false);
        }
      }
      __syncwarp();
    } else if (GLU && warp >= 2) {
      // ---------------------------------------------------------- token rows
      // thread: 16-byte chunk `ch` of rows row0, row0 + 8, ...; chunk c of row r
      // lies at 16 (c ^ r % 8) within its row
      const int tid = threadIdx.x - 2 * 32;
      const int ch = tid & 7, row0 = tid >> 3;
      constexpr int RSTEP = kGatherThreads / 8, NR = BM / RSTEP;
      const uint32_t dst0 = st_base + row0 * kBlock + ((ch ^ row0) << 4);
      uint32_t it = 0;
      bool ok = true;
      for (int u = u0; u < total && ok; u += u_step) {
        const Unit t = decode(p, s_toff, s_roff, u);
        uint32_t rows[NR];
#pragma unroll
        for (int i = 0; i < NR; ++i)
          rows[i] = row0 + i * RSTEP < t.nv ? __ldg(p.row_map + t.r0 + row0 + i * RSTEP) : 0u;
        for (int kb = kb_lo; kb < kb_hi; ++kb, ++it) {
          const uint32_t s = it % C::NS;
          if (it >= (uint32_t)C::NS) {
            ok = mbar_wait_warp(smem_u32(empty + s), ((it / C::NS) - 1) & 1, abort_flag, p.status,
                                true, p.wait_limit);
            if (!ok) break;
          }
          const uint8_t* src = p.x + kb * kBlock + ch * 16;
          const uint32_t dst = dst0 + s * C::STAGE;
#pragma unroll
          for (int i = 0; i < NR; ++i)
            if (row0 + i * RSTEP < t.nv)
              cp_async16(dst + i * (RSTEP * kBlock), src + (size_t)rows[i] * p.K);
          cp_async_arrive(smem_u32(rows_full + s));
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (warp == 1) {
      // ---------------------------------------------------------- MMA issuer
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      const uint64_t da = desc_sw128(st_base), db = desc_sw128(st_base + A_BYTES);
      const uint32_t alo0 = (uint32_t)da, ahi = (uint32_t)(da >> 32);
      const uint32_t blo0 = (uint32_t)db, bhi = (uint32_t)(db >> 32);
      constexpr uint32_t kStage16 = C::STAGE >> 4;
      const uint32_t idesc = idesc_e4m3(BN);
      uint32_t it = 0;
      bool ok = true;
      for (int u = u0; u < total && ok; u += u_step) {
        for (int kb = kb_lo; kb < kb_hi; ++kb, ++it) {
          const uint32_t s = it % C::NS, b = it % C::NBUF;
          // (its first wait is never met at once, so a short bound runs out here)
          ok = mbar_wait_warp<true>(smem_u32(full + s), (it / C::NS) & 1, abort_flag, p.status,
                                    true, p.wait_limit);
          if (ok && GLU)
            ok = mbar_wait_warp(smem_u32(rows_full + s), (it / C::NS) & 1, abort_flag, p.status,
                                true, p.wait_limit);
          // (the gathered rows were written by ordinary copies)
          if (GLU) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          // buffer b was read back NBUF k-blocks ago: waited for last, as the
          // hand-over of the buffers sets the pace
          if (ok && it >= (uint32_t)C::NBUF)
            ok = mbar_wait_warp(smem_u32(acc_empty + b), ((it / C::NBUF) - 1) & 1, abort_flag,
                                p.status, true, p.wait_limit);
          if (!ok) break;
          tc_fence_after();
          const uint32_t off = s * kStage16;
          mma_block(tm + b * BN, alo0 + off, ahi, blo0 + off, bhi, idesc);
          mma_commit_warp(smem_u32(empty + s));
          mma_commit_warp(smem_u32(acc_full + b));
        }
      }
      mma_commit_warp(smem_u32(drain));
      mbar_wait_warp(smem_u32(drain), 0, abort_flag, p.status, false);
    }
    if constexpr (SPLIT) {
      cooperative_groups::this_cluster().sync();     // the two barriers of the joining warps
      cooperative_groups::this_cluster().sync();
    }
  } else {
    // ------------------------------------------------------------ scale, add, store
    regs_inc<208>();
    constexpr int COLS = C::COLS;
    // (warp and, below, row count from lane 0: the compiler then knows that the
    // lanes share them, and the loop runs 5 % faster)
    const int wu = __shfl_sync(0xffffffffu, warp, 0);
    const int q = wu & 3, half = (wu - kAccWarp0) >> 2;
    const uint32_t tl = tmem + ((uint32_t)(q * 32) << 16);
    // the thread's columns: two runs of COLS / 2, one of gate and one of up
    // columns, or one after the other
    const int c0 = GLU ? half * (COLS / 2) : half * COLS;
    const int c1 = GLU ? BN / 2 + c0 : c0 + COLS / 2;
    uint32_t it = 0, tiles = 0;
    bool ok = true, over = false;
    // a unit's rows and scales, their first values loaded: taken for the next
    // unit before the present one is stored
    Lead t{};
    if (u0 < total) t = lead<GLU, BN>(p, decode(p, s_toff, s_roff, u0), q * 32 + lane, c0, kb_lo);
    for (int u = u0; u < total && ok; u += u_step, ++tiles) {
      // some of the warp's lanes are rows
      const bool live = q * 32 < __shfl_sync(0xffffffffu, t.nv, 0);
      const int m = q * 32 + lane;
      float acc[COLS];
#pragma unroll
      for (int j = 0; j < COLS; ++j) acc[j] = 0.f;
      for (int kb = kb_lo; kb < kb_hi; ++kb, ++it) {
        const float f0 = t.a * t.b0, f1 = GLU ? t.a * t.b1 : f0;
        if (kb + 1 < kb_hi) {                     // the next block's, ahead of the wait
          t.a = __ldg(++t.sa);
          t.b0 = __ldg(++t.w0);
          if (GLU) t.b1 = __ldg(++t.w1);
        }
        const uint32_t b = it % C::NBUF;
        ok = mbar_wait_warp(smem_u32(acc_full + b), (it / C::NBUF) & 1, abort_flag, p.status, true,
                            p.wait_limit);
        if (!ok) break;
        tc_fence_after();
        // 16 columns at a time (the two warps of a scheduler hide each other's
        // reads); the buffer is handed back as soon as the last have arrived
        constexpr int NCH = COLS / 16, H = COLS / 2;
        auto hand_back = [&]() {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(acc_empty + b));
        };
        if (live) {
#pragma unroll
          for (int j = 0; j < NCH; ++j) {
            const int c = j * 16;
            uint32_t d[16];
            tmem_ld_start(tl + b * BN + (c < H ? c0 + c : c1 + c - H), d);
            tmem_ld_wait(d);
            if (j + 1 == NCH) hand_back();
            const float f = c < H ? f0 : f1;
#pragma unroll
            for (int i = 0; i < 16; i += 2) fma2(acc[c + i], acc[c + i + 1], d[i], d[i + 1], f);
          }
        } else {
          hand_back();
        }
      }
      if (!ok) break;
      const int r0 = t.r0, nv = t.nv, unit = t.unit;
      if (!SPLIT && u + u_step < total)
        t = lead<GLU, BN>(p, decode(p, s_toff, s_roff, u + u_step), m, c0, kb_lo);
      if constexpr (SPLIT) {
        // every MMA of this CTA is done and every load consumed: the ring is free
        constexpr int H = COLS / 2;
        float* o = reinterpret_cast<float*>(smem) + m * C::SUM_LD;
        if (live) {
#pragma unroll
          for (int j = 0; j < COLS; j += 4)
            *reinterpret_cast<float4*>(o + (j < H ? c0 + j : c1 + j - H)) =
                make_float4(acc[j], acc[j + 1], acc[j + 2], acc[j + 3]);
        }
      } else if constexpr (!GLU) {
        if (live)
          store_rows<MODE, COLS, C::PATCH_LD>(p, r0, q * 32, nv, unit * BN + c0, acc,
                                        s_patch + (warp - kAccWarp0) * 32 * C::PATCH_LD, over);
      } else {
        constexpr int H = COLS / 2;
        float mx = 0.f;
        if (live) {
#pragma unroll
          for (int j = 0; j < H; ++j) {
            acc[j] = glu_codes(act_of(MODE), acc[j], acc[H + j]);
            mx = fmaxf(mx, finite_abs(acc[j]));
          }
        }
        // the block's other 64 features are the other half's warp. The arrays
        // alternate: one is written again only after every warp has passed
        // the next tile's exchange, and so has read this one
        float* am = s_amax + (tiles & 1) * 2 * BM;
        am[half * BM + m] = mx;
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(xchg));
        ok = mbar_wait_warp(smem_u32(xchg), tiles & 1, abort_flag, p.status, true, p.wait_limit);
        if (!ok) break;
        if (m < nv) {
          mx = fmaxf(am[m], am[BM + m]);
          const float r = rscale_of(mx);
          uint8_t* o = reinterpret_cast<uint8_t*>(p.out) + ((size_t)r0 + m) * p.N +
                       unit * kBlock + c0;
#pragma unroll
          for (int j = 0; j < H; j += 32) {
            uint32_t v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
              v[i] = e4m3x4(code_arg(acc[j + 4 * i], r), code_arg(acc[j + 4 * i + 1], r),
                            code_arg(acc[j + 4 * i + 2], r), code_arg(acc[j + 4 * i + 3], r));
            if (p.wide) {
              st32(o + j, v);
            } else {
              *reinterpret_cast<uint4*>(o + j) = make_uint4(v[0], v[1], v[2], v[3]);
              *reinterpret_cast<uint4*>(o + j + 16) = make_uint4(v[4], v[5], v[6], v[7]);
            }
          }
          if (half == 0)
            p.out_s[((size_t)r0 + m) * (p.N / kBlock) + unit] = scale_of(mx);
        }
      }
    }
    if constexpr (SPLIT) {
      cooperative_groups::this_cluster().sync();     // every CTA's sums are in place
      // (a CTA that gave up waiting has left none; the status says so)
      if (u0 < total) {
        if (p.split <= 2)
          join_rows<MODE, BN, C::SUM_LD, GLU ? 1 : 4, 2>(p, decode(p, s_toff, s_roff, u0), st_base,
                                                         rank, over);
        else
          join_rows<MODE, BN, C::SUM_LD, 1, GLU ? 4 : 8>(p, decode(p, s_toff, s_roff, u0), st_base,
                                                         rank, over);
      }
      cooperative_groups::this_cluster().sync();     // no CTA leaves while its sums are read
    }
    if (MODE == MODE_F16 && over) report_status(p.status, MOE_ERR_RANGE);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(512)
                 : "memory");
  }
}

// ------------------------------------------------------------------ host

template <int MODE, int BN, bool SPLIT>
static cudaError_t launch(const Params& p, unsigned grid, cudaStream_t s) {
  auto kern = fp8_tc_kernel<MODE, BN, SPLIT>;
  constexpr int smem = Cfg<BN, SPLIT>::SMEM;
  // (an attribute of the kernel on a device: set once)
  static std::atomic<uint64_t> ready{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (dev >= 64 || !(ready.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    if (dev < 64) ready.fetch_or(bit, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = kThreads;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)p.split;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = SPLIT ? 2 : 1;
  e = cudaLaunchKernelEx(&cfg, kern, p);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

// [2 E][F][K] weight codes: boxes of 128 codes x 128 rows of a gate block and
// the same rows of its up block
static bool gate_up_map(CUtensorMap* m, const void* w, int E, int F, int K) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {(cuuint64_t)K, (cuuint64_t)F, 2 * (cuuint64_t)E};
  cuuint64_t strides[2] = {(cuuint64_t)K, (cuuint64_t)F * K};
  cuuint32_t box[3] = {kBlock, kBlock, 2};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(w), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

static bool row_map2d(CUtensorMap* m, const void* base, long long rows, int K, int box_rows) {
  return make_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, base, K, (uint64_t)rows, K, kBlock, box_rows,
                  CU_TENSOR_MAP_SWIZZLE_128B);
}

// tiles: token tiles at most. The split form is taken where the persistent
// one's units would not fill half of the SMs; its clusters grow while the CTAs
// fit the SMs and each keeps four K blocks or more.
template <int MODE>
static cudaError_t run(Params& p, const void* x, long long x_rows, const void* w, long long tiles,
                       cudaStream_t s) {
  constexpr bool GLU = is_glu(MODE);
  constexpr int BNS = GLU ? 256 : 128;                       // columns of the split form
  p.wait_limit = wait_cycles();
  const int esize = GLU ? 1 : MODE == MODE_F32 ? 4 : 2;
  p.wide = (reinterpret_cast<uintptr_t>(p.out) % 32 == 0) && ((long long)p.N * esize) % 32 == 0;
  // rows are addressed by 32-bit coordinates
  if ((long long)p.E * p.rows_per_group > 0x7fffffffLL) return cudaErrorNotSupported;
  const int sms = num_sms();
  const int per_tile = GLU ? p.N / kBlock : (p.N + 255) / 256;
  const bool split = tiles * per_tile * 2 <= sms;
  const long long w_rows = (long long)p.E * p.rows_per_group;
  p.x = (const uint8_t*)x;
  if (GLU) {
    if (!gate_up_map(&p.tmB, w, p.E, p.N, p.K)) return cudaErrorInvalidValue;
  } else {
    if (!row_map2d(&p.tmB1, w, w_rows, p.K, kBlock)) return cudaErrorInvalidValue;
    if (split)
      p.tmB = p.tmB1;
    else if (!row_map2d(&p.tmB, w, w_rows, p.K, 256))
      return cudaErrorInvalidValue;
    for (int i = 0; i < A_MAPS; ++i)
      if (!row_map2d(&p.tmA[i], x, x_rows, p.K, a_rows(i))) return cudaErrorInvalidValue;
  }
  if (!split) {
    p.n_units = per_tile;
    p.split = 1;
    const long long units = tiles * per_tile;
    if (units > 0x7fffffffLL) return cudaErrorNotSupported;
    return launch<MODE, 256, false>(p, units < sms ? (unsigned)units : (unsigned)sms, s);
  }
  p.n_units = GLU ? p.N / kBlock : (p.N + BNS - 1) / BNS;
  const long long units = tiles * p.n_units;
  p.split = 1;
  while (p.split < 8 && units * p.split * 2 <= sms && p.KB >= p.split * 8) p.split *= 2;
  return launch<MODE, BNS, true>(p, (unsigned)(units * p.split), s);
}

}  // namespace fp8tc

cudaError_t launch_fp8_matmul_tc(const void* a, const float* sa, const void* b, const float* sb,
                                 int M, int N, int K, int out_dt, void* y, int* status,
                                 cudaStream_t s) {
  using namespace fp8tc;
  Params p{};
  p.xs = sa;
  p.M = M;
  p.E = 1;
  p.N = N;
  p.K = K;
  p.KB = (K + kBlock - 1) / kBlock;
  p.ws = sb;
  p.rows_per_group = N;
  p.scale_rows = (N + kBlock - 1) / kBlock;
  p.out = y;
  p.status = status;
  const long long tiles = ((long long)M + BM - 1) / BM;
  if (out_dt == MOE_BF16) return run<MODE_BF16>(p, a, M, b, tiles, s);
  if (out_dt == MOE_F16) return run<MODE_F16>(p, a, M, b, tiles, s);
  return run<MODE_F32>(p, a, M, b, tiles, s);
}

cudaError_t launch_swiglu_fp8_tc(const void* xq, const float* xs, int T, const uint32_t* row_map,
                                 const int32_t* row_off, const int32_t* tile_off, int R,
                                 const moe_experts& ex, void* hq, float* hs, int* status,
                                 cudaStream_t s) {
  using namespace fp8tc;
  if (R <= 0) return cudaSuccess;
  Params p{};
  p.xs = xs;
  p.row_map = row_map;
  p.row_off = row_off;
  p.tile_off = tile_off;
  p.E = ex.E;
  p.N = ex.F;
  p.K = ex.d;
  p.KB = ex.d / kBlock;
  p.ws = (const float*)ex.s_gu;
  p.rows_per_group = 2 * ex.F;
  p.scale_rows = 2 * ex.F / kBlock;
  p.out = hq;
  p.out_s = hs;
  p.status = status;
  const long long tiles = max_tiles(R, ex.E, BM);
  if (ex.act == MOE_ACT_GEGLU_TANH) return run<MODE_GEGLU>(p, xq, T, ex.w_gu, tiles, s);
  return run<MODE_SWIGLU>(p, xq, T, ex.w_gu, tiles, s);
}

cudaError_t launch_down_fp8_tc(const void* hq, const float* hs, const int32_t* row_off,
                               const int32_t* tile_off, int R, const moe_experts& ex, void* ys,
                               int* status, cudaStream_t s) {
  using namespace fp8tc;
  if (R <= 0) return cudaSuccess;
  Params p{};
  p.xs = hs;
  p.row_off = row_off;
  p.tile_off = tile_off;
  p.E = ex.E;
  p.N = ex.d;
  p.K = ex.F;
  p.KB = ex.F / kBlock;
  p.ws = (const float*)ex.s_dn;
  p.rows_per_group = ex.d;
  p.scale_rows = ex.d / kBlock;
  p.out = ys;
  p.status = status;
  return run<MODE_F16>(p, hq, R, ex.w_dn, max_tiles(R, ex.E, BM), s);
}

}  // namespace moe
