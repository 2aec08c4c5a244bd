// The router's balance loss, its per-expert counts and the gradient of the
// logits.
//
// For a sequence b of n_b valid tokens, with p_t = softmax(logits[t]):
//   c[b][e] = valid slots (t, j) with topk_idx[t][j] == e
//   P[b][e] = 1/n_b sum_t p_t[e]
//   L = coef/B sum_b E/(k n_b) sum_e c[b][e] P[b][e]
//   dL/dlogits[t][e] = dloss coef/B E/(k n_b^2) p_t[e] (c[b][e] - sum_e' c[b][e'] p_t[e'])
// (the counts are constants of the gradient).
//
// One warp takes a token: its row stays in registers between the maximum, the
// sum and their use, so each pass reads the logits once, and HBM bounds both.
// The forward pass adds a CTA's tokens in registers and shared memory, writes
// one partial row per (chunk of tokens, sequence) pair, and a second kernel
// adds those in order: no floating-point atomics, so the same inputs give the
// same bits. A sequence's chunks are consecutive, so the pair (chunk c,
// sequence b) can own slot c + b: walking the tokens, each new pair raises c,
// b or both.
#include "common.cuh"
#include "launch.h"

namespace moe {
namespace bal {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
// chunks of tokens at most: three CTAs for each of 148 SMs
constexpr int kMaxChunks = 444;
constexpr int kMinChunk = 16;          // tokens per chunk at least (two per warp)

static int chunk_of(int T) {
  const int c = (int)(((long long)T + kMaxChunks - 1) / kMaxChunks);
  return c < kMinChunk ? kMinChunk : c;
}
static int chunks_of(int T) { return (int)(((long long)T + chunk_of(T) - 1) / chunk_of(T)); }

// VEC consecutive logits per lane and step, NV steps: element
// (i * 32 + lane) * VEC + j of the row is v[i * VEC + j]
template <int NV, int VEC>
struct Row {
  float v[NV * VEC];

  __device__ __forceinline__ void load(const float* p, int E) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = (i * 32 + lane) * VEC;
      if constexpr (VEC == 4) {
        uint4 a = make_uint4(0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u);
        if (e < E) a = ldg_nc_v4(p + e);
        v[4 * i] = __uint_as_float(a.x);
        v[4 * i + 1] = __uint_as_float(a.y);
        v[4 * i + 2] = __uint_as_float(a.z);
        v[4 * i + 3] = __uint_as_float(a.w);
      } else {
        v[i] = e < E ? __ldg(p + e) : -INFINITY;
      }
    }
  }

  // the row's softmax in place; a row of nothing but -inf gives zeros
  __device__ __forceinline__ void softmax() {
    float m = v[0];
#pragma unroll
    for (int i = 1; i < NV * VEC; ++i) m = fmaxf(m, v[i]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    // fmaxf passes over NaN: a row of NaN and -inf alone keeps its NaN below
    float z = 0.f;
    const float base = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int i = 0; i < NV * VEC; ++i) {
      v[i] = __expf(v[i] - base);
      z += v[i];
    }
    z = warp_sum(z);
    const float r = z == 0.f ? 0.f : 1.f / z;
#pragma unroll
    for (int i = 0; i < NV * VEC; ++i) v[i] *= r;
  }
};

// The sequence of token t and where its tokens end: -1 for a token in no
// sequence (end: where that stretch ends). Every result lies inside
// [0, n_seq) and (t, T], whatever the offsets hold.
__device__ __forceinline__ int seq_of(const int32_t* off, int n_seq, int T, int t, int& end) {
  if (!off) {
    end = T;
    return 0;
  }
  if (t < __ldg(off)) {
    end = min(__ldg(off), T);
    return -1;
  }
  int lo = 0, hi = n_seq;               // the largest b in [0, n_seq] with off[b] <= t
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(off + mid) <= t) lo = mid; else hi = mid - 1;
  }
  if (lo == n_seq) {
    end = T;
    return -1;
  }
  end = min(__ldg(off + lo + 1), T);
  return lo;
}

struct FwdParams {
  const float* logits;
  const int32_t* idx;
  const uint8_t* mask;
  const int32_t* off;
  int T, E, k, n_seq, chunk, n_chunks;
  float* part_p;       // [n_chunks + n_seq][E]
  int32_t* part_c;     // [n_chunks + n_seq][E]
  int32_t* part_n;     // [n_chunks + n_seq]
  float* part_loss;    // [n_seq * ceil(E / 32)]
  unsigned* counter;
};

template <int NV, int VEC>
__global__ void __launch_bounds__(kThreads) partial_kernel(const FwdParams p) {
  extern __shared__ float sm[];
  float* s_p = sm;                                             // [kWarps][E]
  int* s_c = reinterpret_cast<int*>(sm + (size_t)kWarps * p.E);  // [E]
  __shared__ int s_n[kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_launch();
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.counter = 0;     // for the kernel behind this one
  const int t1 = (int)min((long long)p.T, (blockIdx.x + 1LL) * p.chunk);
  for (int t0 = blockIdx.x * p.chunk; t0 < t1;) {
    int end;
    const int b = seq_of(p.off, p.n_seq, p.T, t0, end);
    end = min(max(end, t0 + 1), t1);
    if (b < 0) {
      t0 = end;
      continue;
    }
    for (int e = threadIdx.x; e < p.E; e += kThreads) s_c[e] = 0;
    __syncthreads();
    float acc[NV * VEC];
#pragma unroll
    for (int i = 0; i < NV * VEC; ++i) acc[i] = 0.f;
    int n = 0;
    for (int t = t0 + warp; t < end; t += kWarps) {
      if (p.mask && !__ldg(p.mask + t)) continue;
      Row<NV, VEC> r;
      r.load(p.logits + (size_t)t * p.E, p.E);
      if (lane < p.k) {
        const int e = __ldg(p.idx + (size_t)t * p.k + lane);
        if (e >= 0 && e < p.E) atomicAdd(&s_c[e], 1);          // integers: any order
      }
      r.softmax();
#pragma unroll
      for (int i = 0; i < NV * VEC; ++i) acc[i] += r.v[i];
      ++n;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const int e = (i * 32 + lane) * VEC + j;
        if (e < p.E) s_p[warp * p.E + e] = acc[i * VEC + j];
      }
    if (lane == 0) s_n[warp] = n;
    __syncthreads();
    const size_t slot = (size_t)blockIdx.x + b;
    for (int e = threadIdx.x; e < p.E; e += kThreads) {
      float v = s_p[e];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) v += s_p[w * p.E + e];
      p.part_p[slot * p.E + e] = v;
      p.part_c[slot * p.E + e] = s_c[e];
    }
    if (threadIdx.x == 0) {
      int s = 0;
      for (int w = 0; w < kWarps; ++w) s += s_n[w];
      p.part_n[slot] = s;
    }
    __syncthreads();
    t0 = end;
  }
}

// 32 experts of one sequence per CTA: the 8 warps add every 8th chunk's
// partial sums, then those eight in order. The last CTA to finish adds the
// CTAs' parts of the loss, in order.
__global__ void __launch_bounds__(kThreads) finish_kernel(const FwdParams p, float coef,
                                                          float* __restrict__ loss,
                                                          int32_t* __restrict__ counts,
                                                          float* __restrict__ probs,
                                                          int32_t* __restrict__ tokens) {
  __shared__ float s_p[kWarps][32];
  __shared__ int s_c[kWarps][32];
  __shared__ int s_n[kWarps];
  __shared__ float s_l[kWarps];
  __shared__ bool s_last;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_launch();
  const int eb = (p.E + 31) / 32;
  const int b = blockIdx.x / eb, e = (blockIdx.x % eb) * 32 + lane;
  int t0 = 0, t1 = p.T;
  if (p.off) {
    t0 = max(0, min(__ldg(p.off + b), p.T));
    t1 = max(0, min(__ldg(p.off + b + 1), p.T));
  }
  float v = 0.f;
  int c = 0, n = 0;
  if (t0 < t1) {
    const int c1 = (t1 - 1) / p.chunk;
#pragma unroll 4
    for (int i = t0 / p.chunk + warp; i <= c1; i += kWarps) {
      const size_t slot = (size_t)i + b;
      if (e < p.E) {
        v += p.part_p[slot * p.E + e];
        c += p.part_c[slot * p.E + e];
      }
      n += p.part_n[slot];
    }
  }
  s_p[warp][lane] = v;
  s_c[warp][lane] = c;
  if (lane == 0) s_n[warp] = n;
  __syncthreads();
  if (warp == 0) {
    v = 0.f;
    c = 0;
    n = 0;
    for (int w = 0; w < kWarps; ++w) {
      v += s_p[w][lane];
      c += s_c[w][lane];
      n += s_n[w];
    }
    const float inv = n > 0 ? 1.f / (float)n : 0.f;
    v *= inv;
    if (e < p.E) {
      counts[(size_t)b * p.E + e] = c;
      probs[(size_t)b * p.E + e] = v;
    } else {
      v = 0.f;
    }
    const float l = warp_sum((float)c * inv * v);
    if (lane == 0) {
      if (blockIdx.x % eb == 0) tokens[b] = n;
      p.part_loss[blockIdx.x] = l;
      __threadfence();
      s_last = atomicAdd(p.counter, 1u) == gridDim.x - 1;
    }
  }
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  float l = 0.f;
  for (unsigned i = threadIdx.x; i < gridDim.x; i += kThreads) l += __ldcg(p.part_loss + i);
  l = warp_sum(l);
  if (lane == 0) s_l[warp] = l;
  __syncthreads();
  if (threadIdx.x == 0) {
    l = 0.f;
    for (int w = 0; w < kWarps; ++w) l += s_l[w];
    *loss = coef * ((float)p.E / ((float)p.n_seq * (float)p.k)) * l;
  }
}

struct BwdParams {
  const float* logits;
  const uint8_t* mask;
  const int32_t* off;
  const int32_t* counts;
  const int32_t* tokens;
  const float* dloss;
  int T, E, n_seq, chunk;
  float factor;          // coef E / (n_seq k)
  float* dlogits;
};

// A warp takes `chunk` consecutive tokens; the counts of their sequence stay
// in registers.
template <int NV, int VEC>
__global__ void __launch_bounds__(kThreads) backward_kernel(const BwdParams p) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_launch();
  const long long first = ((long long)blockIdx.x * kWarps + warp) * p.chunk;
  const int t1 = (int)min((long long)p.T, first + p.chunk);
  const float up = p.dloss ? __ldg(p.dloss) : 1.f;
  int b = -1, end = 0;
  float a[NV * VEC];
#pragma unroll
  for (int i = 0; i < NV * VEC; ++i) a[i] = 0.f;
  for (int t = (int)min((long long)p.T, first); t < t1; ++t) {
    if (t >= end) {
      b = seq_of(p.off, p.n_seq, p.T, t, end);
      if (b >= 0) {
        const float n = (float)max(__ldg(p.tokens + b), 1);
        const float f = up * p.factor / (n * n);
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            const int e = (i * 32 + lane) * VEC + j;
            a[i * VEC + j] = e < p.E ? f * (float)__ldg(p.counts + (size_t)b * p.E + e) : 0.f;
          }
      }
    }
    float* out = p.dlogits + (size_t)t * p.E;
    Row<NV, VEC> r;
    if (b >= 0 && (!p.mask || __ldg(p.mask + t))) {
      r.load(p.logits + (size_t)t * p.E, p.E);
      r.softmax();
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < NV * VEC; ++i) s = fmaf(a[i], r.v[i], s);
      s = warp_sum(s);
#pragma unroll
      for (int i = 0; i < NV * VEC; ++i) r.v[i] *= a[i] - s;
    } else {
#pragma unroll
      for (int i = 0; i < NV * VEC; ++i) r.v[i] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = (i * 32 + lane) * VEC;
      if (e < p.E) {
        if constexpr (VEC == 4)
          *reinterpret_cast<float4*>(out + e) =
              make_float4(r.v[4 * i], r.v[4 * i + 1], r.v[4 * i + 2], r.v[4 * i + 3]);
        else
          out[e] = r.v[i];
      }
    }
  }
}

struct Ws {
  size_t p, c, n, loss, counter, total;
};
static Ws layout(int T, int E, int n_seq) {
  auto up = [](size_t v) { return (v + 255) & ~(size_t)255; };
  const size_t slots = (size_t)chunks_of(T) + n_seq;
  Ws w;
  w.p = 0;
  w.c = up(slots * E * 4);
  w.n = w.c + up(slots * E * 4);
  w.loss = w.n + up(slots * 4);
  w.counter = w.loss + up((size_t)n_seq * ((E + 31) / 32) * 4);
  w.total = w.counter + 256;
  return w;
}

// f<NV, VEC>() for rows of E logits: 16-byte loads where every row starts on
// a 16-byte boundary (E % 4 == 0)
template <template <int, int> class F, typename P>
static cudaError_t by_width(int E, const P& a) {
  if (E % 4 == 0) {
    if (E <= 128) return F<1, 4>::run(a);
    if (E <= 256) return F<2, 4>::run(a);
    if (E <= 512) return F<4, 4>::run(a);
    return F<8, 4>::run(a);
  }
  if (E <= 32) return F<1, 1>::run(a);
  if (E <= 64) return F<2, 1>::run(a);
  if (E <= 128) return F<4, 1>::run(a);
  if (E <= 256) return F<8, 1>::run(a);
  if (E <= 512) return F<16, 1>::run(a);
  return F<32, 1>::run(a);
}

template <typename P> struct Launch {
  P p;
  unsigned grid;
  cudaStream_t s;
};
template <int NV, int VEC> struct RunFwd {
  static cudaError_t run(const Launch<FwdParams>& l) {
    launch_pdl(partial_kernel<NV, VEC>, l.grid, kThreads, (size_t)(kWarps + 1) * l.p.E * 4, l.s, l.p);
    return cudaGetLastError();
  }
};
template <int NV, int VEC> struct RunBwd {
  static cudaError_t run(const Launch<BwdParams>& l) {
    launch_pdl(backward_kernel<NV, VEC>, l.grid, kThreads, 0, l.s, l.p);
    return cudaGetLastError();
  }
};

}  // namespace bal

size_t balance_workspace_bytes(int T, int E, int n_seq) { return bal::layout(T, E, n_seq).total; }

cudaError_t launch_balance_loss(const float* logits, const int32_t* idx, const uint8_t* mask,
                                const int32_t* seq_off, int T, int E, int k, int n_seq, float coef,
                                float* loss, int32_t* counts, float* probs, int32_t* tokens,
                                void* ws, cudaStream_t s) {
  using namespace bal;
  const Ws w = layout(T, E, n_seq);
  char* base = static_cast<char*>(ws);
  FwdParams p{logits, idx, mask, seq_off, T, E, k, n_seq, chunk_of(T), chunks_of(T),
              (float*)(base + w.p), (int32_t*)(base + w.c), (int32_t*)(base + w.n),
              (float*)(base + w.loss), (unsigned*)(base + w.counter)};
  // at least one CTA, which clears the counter
  const Launch<FwdParams> l{p, (unsigned)(p.n_chunks > 0 ? p.n_chunks : 1), s};
  cudaError_t e = by_width<RunFwd>(E, l);
  if (e != cudaSuccess) return e;
  launch_pdl(finish_kernel, (unsigned)((E + 31) / 32) * (unsigned)n_seq, kThreads, 0, s, p, coef,
             loss, counts, probs, tokens);
  return cudaGetLastError();
}

cudaError_t launch_balance_loss_backward(const float* logits, const uint8_t* mask,
                                         const int32_t* seq_off, int T, int E, int k, int n_seq,
                                         float coef, const int32_t* counts, const int32_t* tokens,
                                         const float* dloss, float* dlogits, cudaStream_t s) {
  using namespace bal;
  // consecutive tokens of one warp: as many as leave four CTAs for each SM
  const int chunk = (int)(((long long)T + 148 * 4 * kWarps - 1) / (148 * 4 * kWarps));
  BwdParams p{logits, mask, seq_off, counts, tokens, dloss, T, E, n_seq, chunk,
              coef * ((float)E / ((float)n_seq * (float)k)), dlogits};
  const long long warps = ((long long)T + chunk - 1) / chunk;
  const Launch<BwdParams> l{p, (unsigned)((warps + kWarps - 1) / kWarps), s};
  return by_width<RunBwd>(E, l);
}

}  // namespace moe
