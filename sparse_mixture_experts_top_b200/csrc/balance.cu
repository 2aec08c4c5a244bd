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
// LPR lanes take a token (fewer than a warp where the row has fewer than 128
// experts): its row stays in registers between the maximum, the sum and their
// use, so each pass reads the logits once. HBM bounds the backward pass, latency
// (the ends of chunks, the second kernel) the forward one. A lane group
// loads the rows of up to four tokens before it looks at the first, since a
// single row's chain (load, maximum, exponentials, sum) is all latency.
// The forward pass adds a CTA's tokens in registers and shared memory, writes
// one partial row per (chunk of tokens, sequence) pair, and a second kernel
// adds those in order: no floating-point atomics, so the same inputs give the
// same bits. A sequence's chunks are consecutive, so the pair (chunk c,
// sequence b) can own slot c + b: walking the tokens, each new pair raises c,
// b or both. A short single sequence is
// one CTA's, with no second kernel. 65521 x 256 logits in 13 masked sequences
// take 24 us forward (0.43 of the measured HBM rate; the second kernel takes 8 us
// when it runs alone, from the latency of its loads) and 28 us backward (0.72) on
// one B200.
#include "common.cuh"
#include "launch.h"

namespace moe {
namespace bal {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxChunks = 592;        // chunks of tokens at most: four CTAs for each of 148 SMs
// the finishing kernel: experts of a CTA, and groups of its threads that share
// out the chunks (a sequence's 592 chunks are nine loads deep)
constexpr int kFinishE = 8;
constexpr int kFinishGroups = 64;
constexpr int kFinishThreads = kFinishE * kFinishGroups;

// How a row of E logits lies in a lane group: LPR lanes, NV steps of VEC
// consecutive logits each (VEC 4 where every row starts on a 16-byte
// boundary, E % 4 == 0): lane l holds elements (i LPR + l) VEC + j.
template <int LPR_, int NV_, int VEC_> struct Shape {
  static constexpr int LPR = LPR_, NV = NV_, VEC = VEC_, N = NV * VEC;
  static constexpr int TPW = 32 / LPR;                           // tokens of a warp at a time
  static constexpr int UN = N <= 8 ? 4 : N <= 16 ? 2 : 1;        // rows in flight per group
  static constexpr int UF = UN > 1 ? UN / 2 : 1;                 // rows of a forward step
  // warps of the CTA that takes a whole short sequence, and the tokens of its
  // at most six steps (a second kernel and its workspace cost more)
  static constexpr int SINGLE_WARPS = N <= 16 ? 16 : 8;
  static constexpr int SINGLE_TOKENS = 6 * SINGLE_WARPS * TPW * UF;
};

// f(Shape) for rows of E logits
template <typename F> static auto by_width(int E, F&& f) {
  if (E % 4 == 0) {
    if (E <= 8) return f(Shape<2, 1, 4>());
    if (E <= 16) return f(Shape<4, 1, 4>());
    if (E <= 32) return f(Shape<8, 1, 4>());
    if (E <= 64) return f(Shape<16, 1, 4>());
    if (E <= 128) return f(Shape<32, 1, 4>());
    if (E <= 256) return f(Shape<32, 2, 4>());
    if (E <= 512) return f(Shape<32, 4, 4>());
    return f(Shape<32, 8, 4>());
  }
  if (E <= 8) return f(Shape<8, 1, 1>());
  if (E <= 32) return f(Shape<32, 1, 1>());
  if (E <= 64) return f(Shape<32, 2, 1>());
  if (E <= 128) return f(Shape<32, 4, 1>());
  if (E <= 256) return f(Shape<32, 8, 1>());
  if (E <= 512) return f(Shape<32, 16, 1>());
  return f(Shape<32, 32, 1>());
}

// Tokens per chunk: as many as four CTAs per SM take, at least what a CTA has
// in flight at a time
static int chunk_of(int T, int E) {
  const int least = by_width(E, [](auto s) { return kWarps * decltype(s)::TPW * decltype(s)::UN; });
  const int c = (int)(((long long)T + kMaxChunks - 1) / kMaxChunks);
  return c < least ? least : c;
}
static int chunks_of(int T, int E) {
  const int c = chunk_of(T, E);
  return (int)(((long long)T + c - 1) / c);
}

template <typename S>
struct Row {
  float v[S::N];

  // element index of value i * VEC + j
  static __device__ __forceinline__ int at(int i, int j) {
    return (i * S::LPR + (int)(threadIdx.x % S::LPR)) * S::VEC + j;
  }

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < S::N; ++i) v[i] = -INFINITY;
  }

  __device__ __forceinline__ void load(const float* p, int E) {
#pragma unroll
    for (int i = 0; i < S::NV; ++i) {
      const int e = at(i, 0);
      if constexpr (S::VEC == 4) {
        if (e < E) {
          const uint4 a = ldg_nc_v4(p + e);
          v[4 * i] = __uint_as_float(a.x);
          v[4 * i + 1] = __uint_as_float(a.y);
          v[4 * i + 2] = __uint_as_float(a.z);
          v[4 * i + 3] = __uint_as_float(a.w);
        }
      } else {
        if (e < E) v[i] = __ldg(p + e);
      }
    }
  }

  // The row's exponentials in place (their largest is 1), and the factor that
  // makes them probabilities; a row of nothing but -inf gives zeros.
  // exp(x) = 2^(x log2 e), results below 2^-126 taken as zero.
  __device__ __forceinline__ float softmax() {
    float m = v[0];
#pragma unroll
    for (int i = 1; i < S::N; ++i) m = fmaxf(m, v[i]);
    if constexpr (S::LPR == 32) {
      asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(m));
    } else {
#pragma unroll
      for (int o = S::LPR / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    }
    // (the maximum passes over NaN, so a row of NaN and -inf alone has m = -inf
    // too; its NaN shows in the exponentials)
    float z = 0.f;
    const float base = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int i = 0; i < S::N; ++i) {
      asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(v[i]) : "f"((v[i] - base) * 1.4426950408889634f));
      z += v[i];
    }
#pragma unroll
    for (int o = S::LPR / 2; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    return z == 0.f ? 0.f : 1.f / z;
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
  float factor;        // coef E / (n_seq k)
  float* part_p;       // [n_chunks + n_seq][E]
  int32_t* part_c;     // [n_chunks + n_seq][E]
  int32_t* part_n;     // [n_chunks + n_seq]
  float* part_loss;    // [n_seq * ceil(E / kFinishE)]
  unsigned* counter;
  float* loss;
  int32_t* counts;
  float* probs;
  int32_t* tokens;
};

// The sum over a CTA of one value per thread, in a fixed order (thread 0 has it)
template <int WARPS>
__device__ __forceinline__ float block_sum(float v, float* s_part) {
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) s_part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.f;
  if (threadIdx.x == 0)
    for (int w = 0; w < WARPS; ++w) v += s_part[w];
  return v;
}

// One chunk of tokens: a partial row for each sequence that it meets. SINGLE:
// all tokens of the only sequence, whose sums are the result.
template <typename S, bool SINGLE>
__global__ void __launch_bounds__(SINGLE ? S::SINGLE_WARPS * 32 : kThreads)
    partial_kernel(const FwdParams p) {
  constexpr int W = SINGLE ? S::SINGLE_WARPS : kWarps, THREADS = W * 32;
  extern __shared__ float sm[];
  float* s_p = sm;                                        // [W][E]
  int* s_c = reinterpret_cast<int*>(sm + (size_t)W * p.E);  // [E]
  __shared__ int s_n[W];
  __shared__ float s_l[W];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int grp = lane / S::LPR, gl = lane % S::LPR;
  constexpr int STEP = W * S::TPW;
  pdl_wait();
  pdl_launch();
  if (!SINGLE && blockIdx.x == 0 && threadIdx.x == 0) *p.counter = 0;   // for the next kernel
  const int t1 = SINGLE ? p.T : (int)min((long long)p.T, (blockIdx.x + 1LL) * p.chunk);
  for (int t0 = blockIdx.x * p.chunk; t0 < t1 || SINGLE;) {
    int end = t1, b = 0;
    if (t0 < t1) {
      b = seq_of(p.off, p.n_seq, p.T, t0, end);
      end = min(max(end, t0 + 1), t1);
      if (b < 0) {
        t0 = end;
        continue;
      }
    }
    for (int e = threadIdx.x; e < p.E; e += THREADS) s_c[e] = 0;
    __syncthreads();
    float acc[S::N];
#pragma unroll
    for (int i = 0; i < S::N; ++i) acc[i] = 0.f;
    int n = 0;
    // The warp's tokens, UF per group and step (the same number of steps in all
    // its groups): while a step's rows are worked on, the next step's rows and
    // ids and the masks of the one behind it are on their way.
    constexpr int UF = S::UF;
    struct Step {
      Row<S> r[UF];
      int id[UF];
      bool ok[UF];
    } cur, next;
    bool ok[UF];
    auto masks = [&](int tw) {
#pragma unroll
      for (int u = 0; u < UF; ++u) {
        const int t = tw + u * STEP + grp;
        ok[u] = t < end && (!p.mask || __ldg(p.mask + t));
      }
    };
    auto rows = [&](int tw, Step& s) {
#pragma unroll
      for (int u = 0; u < UF; ++u) {
        const int t = tw + u * STEP + grp;
        s.ok[u] = ok[u];
        s.r[u].clear();                   // a token that takes no part has no probability
        if (ok[u]) s.r[u].load(p.logits + (size_t)t * p.E, p.E);
        s.id[u] = ok[u] && gl < p.k ? __ldg(p.idx + (size_t)t * p.k + gl) : -1;
      }
    };
    int tw = t0 + warp * S::TPW;
    if (tw < end) {
      masks(tw);
      rows(tw, cur);
      masks(tw + STEP * UF);
    }
    for (; tw < end; tw += STEP * UF) {
      rows(tw + STEP * UF, next);
      masks(tw + 2 * STEP * UF);
#pragma unroll
      for (int u = 0; u < UF; ++u) {
        const int e0 = cur.id[u];
        if (e0 >= 0 && e0 < p.E) atomicAdd(&s_c[e0], 1);       // integers: any order
        if (cur.ok[u] && gl == 0) ++n;
        if (S::LPR < 32 && cur.ok[u]) {   // the slots past one per lane
          const int32_t* ids = p.idx + (size_t)(tw + u * STEP + grp) * p.k;
          for (int j = gl + S::LPR; j < p.k; j += S::LPR) {
            const int e = __ldg(ids + j);
            if (e >= 0 && e < p.E) atomicAdd(&s_c[e], 1);
          }
        }
        __syncwarp();
        const float f = cur.r[u].softmax();
#pragma unroll
        for (int i = 0; i < S::N; ++i) acc[i] = fmaf(cur.r[u].v[i], f, acc[i]);
      }
      cur = next;
    }
#pragma unroll
    for (int o = S::LPR; o < 32; o <<= 1) {                    // the warp's groups
#pragma unroll
      for (int i = 0; i < S::N; ++i) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
    if (grp == 0) {
#pragma unroll
      for (int i = 0; i < S::NV; ++i)
#pragma unroll
        for (int j = 0; j < S::VEC; ++j) {
          const int e = Row<S>::at(i, j);
          if (e < p.E) s_p[warp * p.E + e] = acc[i * S::VEC + j];
        }
    }
    if (lane == 0) s_n[warp] = n;
    __syncthreads();
    n = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) n += s_n[w];
    const size_t slot = SINGLE ? 0 : (size_t)blockIdx.x + b;
    const float inv = n > 0 ? 1.f / (float)n : 0.f;
    float l = 0.f;
    for (int e = threadIdx.x; e < p.E; e += THREADS) {
      float v = s_p[e];
#pragma unroll
      for (int w = 1; w < W; ++w) v += s_p[w * p.E + e];
      if constexpr (SINGLE) {
        p.probs[e] = v * inv;
        p.counts[e] = s_c[e];
        l += (float)s_c[e] * inv * (v * inv);
      } else {
        p.part_p[slot * p.E + e] = v;
        p.part_c[slot * p.E + e] = s_c[e];
      }
    }
    if constexpr (SINGLE) {
      l = block_sum<W>(l, s_l);
      if (threadIdx.x == 0) {
        *p.loss = p.factor * l;
        p.tokens[0] = n;
      }
      return;
    }
    if (threadIdx.x == 0) p.part_n[slot] = n;
    __syncthreads();
    t0 = end;
  }
}

// kFinishE experts of one sequence per CTA: group g of its threads adds the
// partial sums of chunks g, g + kFinishGroups, ..., then the groups' are added
// in order. The last CTA to finish adds the CTAs' parts of the loss, in order.
__global__ void __launch_bounds__(kFinishThreads) finish_kernel(const FwdParams p) {
  __shared__ float s_p[kFinishGroups][kFinishE];
  __shared__ int s_c[kFinishGroups][kFinishE];
  __shared__ int s_n[kFinishGroups];
  __shared__ float s_l[kFinishThreads / 32];
  __shared__ bool s_last;
  const int el = threadIdx.x % kFinishE, grp = threadIdx.x / kFinishE;
  pdl_wait();
  pdl_launch();
  const int eb = (p.E + kFinishE - 1) / kFinishE;
  const int b = blockIdx.x / eb, e = (blockIdx.x % eb) * kFinishE + el;
  int t0 = 0, t1 = p.T;
  if (p.off) {
    t0 = max(0, min(__ldg(p.off + b), p.T));
    t1 = max(0, min(__ldg(p.off + b + 1), p.T));
  }
  float v = 0.f;
  int c = 0, n = 0;
  if (t0 < t1) {
    const int c0 = t0 / p.chunk + grp, c1 = (t1 - 1) / p.chunk;
    // four chunks at a time, whose loads go out together
    for (int i = c0; i <= c1; i += 4 * kFinishGroups) {
      float pv[4];
      int pc[4], pn[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int ch = i + j * kFinishGroups;
        const size_t slot = (size_t)ch + b;
        const bool in = ch <= c1;
        pv[j] = in && e < p.E ? p.part_p[slot * p.E + e] : 0.f;
        pc[j] = in && e < p.E ? p.part_c[slot * p.E + e] : 0;
        pn[j] = in ? p.part_n[slot] : 0;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v += pv[j];
        c += pc[j];
        n += pn[j];
      }
    }
  }
  s_p[grp][el] = v;
  s_c[grp][el] = c;
  if (el == 0) s_n[grp] = n;
  __syncthreads();
  if (threadIdx.x < 32) {
    // lane: expert el of quarter grp of the groups, then the quarters in order
    constexpr int Q = kFinishGroups / 4;
    v = 0.f;
    c = 0;
    n = 0;
#pragma unroll
    for (int g = 0; g < Q; ++g) {
      v += s_p[grp * Q + g][el];
      c += s_c[grp * Q + g][el];
      n += s_n[grp * Q + g];
    }
#pragma unroll
    for (int o = kFinishE; o < 32; o <<= 1) {
      v += __shfl_xor_sync(0xffffffffu, v, o);
      c += __shfl_xor_sync(0xffffffffu, c, o);
      n += __shfl_xor_sync(0xffffffffu, n, o);
    }
    const float inv = n > 0 ? 1.f / (float)n : 0.f;
    v *= inv;
    float l = 0.f;
    if (grp == 0 && e < p.E) {
      p.counts[(size_t)b * p.E + e] = c;
      p.probs[(size_t)b * p.E + e] = v;
      l = (float)c * inv * v;
    }
    l = warp_sum(l);
    if (threadIdx.x == 0) {
      if (blockIdx.x % eb == 0) p.tokens[b] = n;
      p.part_loss[blockIdx.x] = l;
      __threadfence();
      s_last = atomicAdd(p.counter, 1u) == gridDim.x - 1;
    }
  }
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  float l = 0.f;
  for (unsigned i = threadIdx.x; i < gridDim.x; i += kFinishThreads) l += __ldcg(p.part_loss + i);
  l = block_sum<kFinishThreads / 32>(l, s_l);
  if (threadIdx.x == 0) *p.loss = p.factor * l;
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

// A warp takes `chunk` consecutive tokens; the counts of a group's sequence
// stay in registers.
template <typename S>
__global__ void __launch_bounds__(kThreads) backward_kernel(const BwdParams p) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int grp = lane / S::LPR;
  pdl_wait();
  pdl_launch();
  const long long first = ((long long)blockIdx.x * kWarps + warp) * p.chunk;
  const int t1 = (int)min((long long)p.T, first + p.chunk);
  const float up = p.dloss ? __ldg(p.dloss) : 1.f;
  int b = -1, end = 0;
  float a[S::N];
#pragma unroll
  for (int i = 0; i < S::N; ++i) a[i] = 0.f;
  for (int tw = (int)min((long long)p.T, first); tw < t1; tw += S::TPW * S::UN) {
    Row<S> r[S::UN];
    bool ok[S::UN];
#pragma unroll
    for (int u = 0; u < S::UN; ++u) {
      const int t = tw + u * S::TPW + grp;
      ok[u] = t < t1 && (!p.mask || __ldg(p.mask + t));
    }
#pragma unroll
    for (int u = 0; u < S::UN; ++u) {
      r[u].clear();
      if (ok[u]) r[u].load(p.logits + (size_t)(tw + u * S::TPW + grp) * p.E, p.E);
    }
#pragma unroll
    for (int u = 0; u < S::UN; ++u) {
      const int t = tw + u * S::TPW + grp;
      if (t < t1 && t >= end) {
        b = seq_of(p.off, p.n_seq, p.T, t, end);
        const float n = b >= 0 ? (float)max(__ldg(p.tokens + b), 1) : 1.f;
        const float f = up * p.factor / (n * n);
#pragma unroll
        for (int i = 0; i < S::NV; ++i)
#pragma unroll
          for (int j = 0; j < S::VEC; ++j) {
            const int e = Row<S>::at(i, j);
            a[i * S::VEC + j] =
                b >= 0 && e < p.E ? f * (float)__ldg(p.counts + (size_t)b * p.E + e) : 0.f;
          }
      }
      __syncwarp();
      const float z = r[u].softmax();    // zeros for a masked token
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < S::N; ++i) s = fmaf(a[i], r[u].v[i], s);
#pragma unroll
      for (int o = S::LPR / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      s *= z;
      if (t >= t1) continue;
      float* out = p.dlogits + (size_t)t * p.E;
#pragma unroll
      for (int i = 0; i < S::NV; ++i) {
        const int e = Row<S>::at(i, 0);
        if (e >= p.E) continue;
        float d[S::VEC];
#pragma unroll
        for (int j = 0; j < S::VEC; ++j)
          // (a token that takes no part is zero whatever its logits and dloss hold)
          d[j] = b >= 0 && ok[u] ? r[u].v[i * S::VEC + j] * z * (a[i * S::VEC + j] - s) : 0.f;
        if constexpr (S::VEC == 4)
          *reinterpret_cast<float4*>(out + e) = make_float4(d[0], d[1], d[2], d[3]);
        else
          out[e] = d[0];
      }
    }
  }
}

struct Ws {
  size_t p, c, n, loss, counter, total;
};
static Ws layout(int T, int E, int n_seq) {
  auto up = [](size_t v) { return (v + 255) & ~(size_t)255; };
  const size_t slots = (size_t)chunks_of(T, E) + n_seq;
  Ws w;
  w.p = 0;
  w.c = up(slots * E * 4);
  w.n = w.c + up(slots * E * 4);
  w.loss = w.n + up(slots * 4);
  w.counter = w.loss + up((size_t)n_seq * ((E + kFinishE - 1) / kFinishE) * 4);
  w.total = w.counter + 256;
  return w;
}

}  // namespace bal

// one sequence that one CTA takes: no partial sums
static bool single(int T, int E, int n_seq) {
  return n_seq == 1 && T <= bal::by_width(E, [](auto s) { return decltype(s)::SINGLE_TOKENS; });
}

size_t balance_workspace_bytes(int T, int E, int n_seq) {
  return single(T, E, n_seq) ? 0 : bal::layout(T, E, n_seq).total;
}

cudaError_t launch_balance_loss(const float* logits, const int32_t* idx, const uint8_t* mask,
                                const int32_t* seq_off, int T, int E, int k, int n_seq, float coef,
                                float* loss, int32_t* counts, float* probs, int32_t* tokens,
                                void* ws, cudaStream_t s) {
  using namespace bal;
  const Ws w = layout(T, E, n_seq);
  char* base = static_cast<char*>(ws);
  const FwdParams p{logits, idx, mask, seq_off, T, E, k, n_seq, chunk_of(T, E), chunks_of(T, E),
                    coef * ((float)E / ((float)n_seq * (float)k)),
                    (float*)(base + w.p), (int32_t*)(base + w.c), (int32_t*)(base + w.n),
                    (float*)(base + w.loss), (unsigned*)(base + w.counter),
                    loss, counts, probs, tokens};
  const bool one = single(T, E, n_seq);
  // at least one CTA, which clears the counter
  const unsigned grid = (unsigned)(p.n_chunks > 0 ? p.n_chunks : 1);
  const cudaError_t e = by_width(E, [&](auto shape) {
    using S = decltype(shape);
    if (one)
      return launch_pdl(partial_kernel<S, true>, 1, S::SINGLE_WARPS * 32,
                        (size_t)(S::SINGLE_WARPS + 1) * E * 4, s, p);
    return launch_pdl(partial_kernel<S, false>, grid, kThreads, (size_t)(kWarps + 1) * E * 4, s, p);
  });
  if (e != cudaSuccess || one) return e;
  return launch_pdl(finish_kernel, (unsigned)((E + kFinishE - 1) / kFinishE) * (unsigned)n_seq,
                    kFinishThreads, 0, s, p);
}

cudaError_t launch_balance_loss_backward(const float* logits, const uint8_t* mask,
                                         const int32_t* seq_off, int T, int E, int k, int n_seq,
                                         float coef, const int32_t* counts, const int32_t* tokens,
                                         const float* dloss, float* dlogits, cudaStream_t s) {
  using namespace bal;
  return by_width(E, [&](auto shape) {
    using S = decltype(shape);
    // consecutive tokens of one warp: as many as leave eight CTAs for each SM,
    // at least what it has in flight at a time
    constexpr int kCtas = 148 * 8;
    const int c = (int)(((long long)T + kCtas * kWarps - 1) / (kCtas * kWarps));
    const int least = S::TPW * S::UN;
    const int chunk = c < least ? least : c;
    const BwdParams p{logits, mask, seq_off, counts, tokens, dloss, T, E, n_seq, chunk,
                      coef * ((float)E / ((float)n_seq * (float)k)), dlogits};
    const long long warps = ((long long)T + chunk - 1) / chunk;
    return launch_pdl(backward_kernel<S>, (unsigned)((warps + kWarps - 1) / kWarps), kThreads, 0, s,
                      p);
  });
}

}  // namespace moe
