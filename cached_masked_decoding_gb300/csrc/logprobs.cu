// What rows of logits say: log probabilities of given tokens, entropy, the largest alternatives.
//
// With M the largest z of a row, at token a, and sums over the others,
//   S = sum e^(z - M),  W = sum (z - M) e^(z - M):
//   log p_i = (z_i - M) - log1p(S),   entropy = log1p(S) - W / (1 + S).
// The largest term is left out of the sums, so a nearly certain row's S keeps its relative accuracy, and both
// parts of the entropy are of one sign.
//
// Bound by HBM: the logits are read once.  A CTA (or a cluster of up to 8, where rows are few) takes a row and streams
// it; every thread keeps the largest of its elements m and, relative to it, S and W of them all.  What needs the
// elements again is a few threads' worth, which lies in L2 or L1 still:
//   - the thread that holds the row's largest takes its S and W again without it;
//   - the alternatives are among the elements of threads whose m is no less than the top-th largest of 128 group
//     maxima (a lower bound of the top-th largest element): for 20 of 126464 about 22 threads of 512.  Elements above
//     the bound are ranked by counting; its equals join in the order of their ids.
// Rows that would give more than 1024 elements above the bound (one thread's elements are the largest by far) take a
// pass of the row an alternative.
#include <cmath>
#include <type_traits>

#include "ops8.h"
#include "ptx8.cuh"
#include "q8.cuh"

namespace dllm {

struct LogprobsParams {
  const void* logits;
  const int32_t* targets;
  float *logp, *entropy, *top_logp;
  int32_t* top_ids;
  long long rs;
  int vocab, top, cluster;
  float scale;
};

constexpr int kMostTop = 64;
constexpr int kMostAbove = 1024;     // elements above the bound that are ranked
constexpr int kMostEqual = 256;      // and equals that are, before the row is walked for them in order
constexpr int kLogCluster = 8;

struct Best {
  float x;
  int i;    // -1: none
};
// a before b: larger, or of a lower index
__device__ __forceinline__ bool before(const Best& a, const Best& b) {
  return a.i >= 0 && (b.i < 0 || a.x > b.x || (a.x == b.x && a.i < b.i));
}

// 2^x; results below the normal range are 0
__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// The larger, a NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Words of 16 bytes as the element types have them: their largest (a NaN is none), and their pairs.
template <typename E>
struct LogWords {
  template <int n>
  static __device__ __forceinline__ float largest(const uint4 (&r)[n]) {
    using T2 = typename std::conditional<std::is_same<E, ElemBf16>::value, __nv_bfloat162, __half2>::type;
    auto two = [](uint32_t w) { return *reinterpret_cast<const T2*>(&w); };
    T2 m = two(r[0].x);
#pragma unroll
    for (int k = 0; k < n; ++k) {
      if (k) m = __hmax2(m, two(r[k].x));
      m = __hmax2(__hmax2(m, two(r[k].y)), __hmax2(two(r[k].z), two(r[k].w)));
    }
    const float2 f = pair(*reinterpret_cast<const uint32_t*>(&m));
    return fmaxf(f.x, f.y);
  }
  static __device__ __forceinline__ float2 pair(uint32_t w) {
    if constexpr (std::is_same<E, ElemBf16>::value)
      return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    else
      return f16x2_to_f32(w);
  }
  template <typename Fn>
  static __device__ __forceinline__ void pairs(const uint4& r, Fn f) {
    f(pair(r.x));
    f(pair(r.y));
    f(pair(r.z));
    f(pair(r.w));
  }
};
template <>
struct LogWords<ElemF32> {
  template <int n>
  static __device__ __forceinline__ float largest(const uint4 (&r)[n]) {
    float m = __uint_as_float(r[0].x);
#pragma unroll
    for (int k = 0; k < n; ++k) {
      m = fmaxf(fmaxf(m, __uint_as_float(r[k].x)), __uint_as_float(r[k].y));
      m = fmaxf(fmaxf(m, __uint_as_float(r[k].z)), __uint_as_float(r[k].w));
    }
    return m;
  }
  template <typename Fn>
  static __device__ __forceinline__ void pairs(const uint4& r, Fn f) {
    f(make_float2(__uint_as_float(r.x), __uint_as_float(r.y)));
    f(make_float2(__uint_as_float(r.z), __uint_as_float(r.w)));
  }
};

// The largest element m so far (-inf: none yet), and S and W of all elements so far relative to it, W in base 2; kept in
// pairs.  Where m c2 is of ordinary size the reference is m c2 rounded, ref, and a term's exponent x c2 - ref one fused
// rounding (an eighth of the instructions less than (x - m) c2, which rows of the type's lowest value need).
struct LogSums {
  float m = -INFINITY, ref = 0.0f;
  bool plain = false;                  // the reference is ref, not m c2
  uint64_t S = 0, W = 0;

  // the exponent that takes sums from this reference to to_m c2, or to to_ref
  __device__ __forceinline__ float rise(float to_m, float to_ref, bool to_plain, float c2) const {
    return to_plain ? (plain ? ref - to_ref : fmaf(m, c2, -to_ref)) : (plain ? -fmaf(to_m, c2, -ref) : (m - to_m) * c2);
  }
  __device__ __forceinline__ void scale(float d) {
    d = max_nan(d, -200.0f);
    const float f = exp2_fast(d);
    const uint64_t f2 = f32x2(f, f);
    W = mul_f32x2(fma_f32x2(S, f32x2(d, d), W), f2);
    S = mul_f32x2(S, f2);
  }
  __device__ __forceinline__ void raise(float to, float c2) {
    const float to_ref = to * c2;
    const bool to_plain = fabsf(to_ref) <= 32768.0f;
    if (m > -INFINITY) scale(rise(to, to_ref, to_plain, c2));
    m = to;
    ref = to_ref;
    plain = to_plain;
  }
  template <typename E, int n>
  __device__ __forceinline__ void add(const uint4 (&r)[n], float c2) {
    const float top = LogWords<E>::largest(r);
    if (top > m) raise(top, c2);
    const uint64_t S0 = S, W0 = W;
    if (plain) {
      const uint64_t r2 = f32x2(-ref, -ref), s2 = f32x2(c2, c2);
#pragma unroll
      for (int k = 0; k < n; ++k)
        LogWords<E>::pairs(r[k], [&](float2 x) {
          const uint64_t d = fma_f32x2(f32x2(x.x, x.y), s2, r2);
          const float2 v = f32x2_get(d);
          const uint64_t e = f32x2(exp2_fast(v.x), exp2_fast(v.y));
          S = add_f32x2(S, e);
          W = fma_f32x2(d, e, W);
        });
    }
    const float2 w = f32x2_get(W);
    if (!plain || !(w.x + w.y == w.x + w.y)) {
      // an exponent of -inf has to leave W alone (2^-200 is 0)
      S = S0;
      W = W0;
#pragma unroll 1
      for (int k = 0; k < n; ++k) {
        const uint4 x4 = k == 0 ? r[0] : k == 1 ? r[n > 1 ? 1 : 0] : k == 2 ? r[n > 2 ? 2 : 0] : r[n - 1];
        LogWords<E>::pairs(x4, [&](float2 x) { one(x.x, c2), one(x.y, c2); });
      }
    }
  }
  __device__ __forceinline__ void one(float x, float c2) {
    const float d = max_nan(plain ? fmaf(x, c2, -ref) : (x - (m == -INFINITY ? 0.0f : m)) * c2, -200.0f);
    const float e = exp2_fast(d);
    S = add_f32x2(S, f32x2(e, 0.0f));
    W = add_f32x2(W, f32x2(d * e, 0.0f));
  }
};

// A row's (or a part's) largest element, and S and W of the others relative to it.
struct LogRest {
  float m, S, W;
};

// o's joined to t's.
__device__ __forceinline__ void join_sums(LogRest& t, LogRest o, float c2) {
  if (o.m > t.m) {
    const LogRest x = t;
    t = o;
    o = x;
  }
  if (o.m == -INFINITY) {
    t.S += o.S;                        // 0, or a NaN
    return;
  }
  const float d = max_nan((o.m - t.m) * c2, -200.0f), f = exp2_fast(d);
  t.S += (1.0f + o.S) * f;
  t.W += (o.W + (1.0f + o.S) * d) * f;
}

template <int THREADS>
struct LogShared {
  float warp_S[THREADS / 32], warp_W[THREADS / 32];
  int warp_n[THREADS / 32 + 1];
  float group[128];                    // group maxima
  float bound;
  int owner, n_above, n_equal, n_hot;
  int hot[THREADS];
  Best above[kMostAbove];
  int equal[kMostEqual];
  Best top[kLogCluster][kMostTop];     // lists of the cluster's CTAs, in order
  float sums[kLogCluster][3];          // m, S, W
  Best best[THREADS / 32];
};

template <typename E, int THREADS>
struct LogRow {
  using T = typename E::T;
  static constexpr int VE = 16 / (int)sizeof(T);
  const T* x;
  int vocab, head, extra;              // extra: elements before and after the vectors, a thread each
  int nvec, v0, v1;                    // the CTA's vectors
  __device__ __forceinline__ LogRow(const LogprobsParams& p, long long row, int rank, int ranks) {
    x = static_cast<const T*>(p.logits) + row * p.rs;
    vocab = p.vocab;
    head = min(vocab, (int)((16 - (reinterpret_cast<uintptr_t>(x) & 15)) & 15) / (int)sizeof(T));
    nvec = (vocab - head) / VE;
    v0 = (int)((long long)nvec * rank / ranks);
    v1 = (int)((long long)nvec * (rank + 1) / ranks);
    extra = rank == 0 ? vocab - nvec * VE : 0;
  }
  __device__ __forceinline__ int extra_index(int e) const { return e < head ? e : e + nvec * VE; }
  __device__ __forceinline__ int index(int v, int e) const { return head + v * VE + e; }
  __device__ __forceinline__ uint4 load(int v) const { return reinterpret_cast<const uint4*>(x + head)[v]; }
  static __device__ __forceinline__ void floats(const uint4& r, float (&f)[VE]) {
    if constexpr (VE == 8) {
      E::load8(reinterpret_cast<const T*>(&r), f);
    } else {
      f[0] = __uint_as_float(r.x);
      f[1] = __uint_as_float(r.y);
      f[2] = __uint_as_float(r.z);
      f[3] = __uint_as_float(r.w);
    }
  }
  // f(x, index) of every element of thread t, by the lanes of a warp
  template <typename Fn>
  __device__ __forceinline__ void each(int t, int lane, Fn f) const {
    for (int v = v0 + t + lane * THREADS; v < v1; v += 32 * THREADS) {
      float e[VE];
      floats(load(v), e);
#pragma unroll
      for (int i = 0; i < VE; ++i) f(e[i], index(v, i));
    }
    if (lane == 0 && t < extra) f(E::get(x + extra_index(t)), extra_index(t));
  }
};

// The `top` best of the CTA's elements, in order, one pass each.
template <typename E, int THREADS>
__device__ void top_by_passes(const LogRow<E, THREADS>& row, LogShared<THREADS>& sh, int top, Best* out) {
  Best last = {INFINITY, -1};
  for (int k = 0; k < top; ++k) {
    Best b = {0.0f, -1};
    auto look = [&](float x, int i) {
      const Best c = {x, i};
      if (x == x && (k == 0 || before(last, c)) && before(c, b)) b = c;
    };
    for (int v = row.v0 + (int)threadIdx.x; v < row.v1; v += THREADS) {
      float e[LogRow<E, THREADS>::VE];
      row.floats(row.load(v), e);
#pragma unroll
      for (int i = 0; i < LogRow<E, THREADS>::VE; ++i) look(e[i], row.index(v, i));
    }
    if ((int)threadIdx.x < row.extra) look(E::get(row.x + row.extra_index(threadIdx.x)), row.extra_index(threadIdx.x));
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) {
      const Best o = {__shfl_xor_sync(0xffffffffu, b.x, d), __shfl_xor_sync(0xffffffffu, b.i, d)};
      if (before(o, b)) b = o;
    }
    __syncthreads();
    if (threadIdx.x % 32 == 0) sh.best[threadIdx.x / 32] = b;
    __syncthreads();
    b = sh.best[0];
    for (int w = 1; w < THREADS / 32; ++w)
      if (before(sh.best[w], b)) b = sh.best[w];
    if (threadIdx.x == 0) out[k] = b;
    last = b;
    if (b.i < 0) {                     // none left, here and in every further pass
      for (int j = k + 1 + (int)threadIdx.x; j < top; j += THREADS) out[j] = b;
      break;
    }
  }
}

// The first `need` elements equal to `bound` in the order of their ids, and how many there are; the CTA's elements
// lie in the order head, vectors, tail.
template <typename E, int THREADS>
__device__ int equals_in_order(const LogRow<E, THREADS>& row, LogShared<THREADS>& sh, float bound, int need, Best* out) {
  constexpr int VE = LogRow<E, THREADS>::VE;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, heads = row.extra ? row.head : 0;
  int found = 0;
  for (int at = row.v0 - THREADS; at < row.v1 + THREADS && found < need; at += THREADS) {
    // one step for the head, one of THREADS vectors each, one for the tail
    float e[VE];
    int n = 0, first = 0;
    if (at < row.v0) {
      if (tid < heads) {
        e[0] = E::get(row.x + tid);
        n = 1;
        first = tid;
      }
    } else if (at < row.v1) {
      if (at + tid < row.v1) {
        row.floats(row.load(at + tid), e);
        n = VE;
        first = row.index(at + tid, 0);
      }
    } else if (tid < row.extra - heads) {
      first = row.extra_index(heads + tid);
      e[0] = E::get(row.x + first);
      n = 1;
    }
    uint32_t mask = 0;
#pragma unroll
    for (int i = 0; i < VE; ++i)
      if (i < n && e[i] == bound) mask |= 1u << i;
    int upto = __popc(mask);
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, upto, d);
      if (lane >= d) upto += v;
    }
    if (lane == 31) sh.warp_n[warp] = upto;
    __syncthreads();
    int pos = found + upto - __popc(mask);
    int total = 0;
    for (int w = 0; w < THREADS / 32; ++w) {
      if (w < warp) pos += sh.warp_n[w];
      total += sh.warp_n[w];
    }
    for (; mask && pos < need; mask &= mask - 1, ++pos) out[pos] = {bound, first + __ffs(mask) - 1};
    found += total;
    __syncthreads();
  }
  return min(found, need);
}

template <typename E, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) logprobs_kernel(const __grid_constant__ LogprobsParams p) {
  constexpr int QUAD = THREADS / 128, AHEAD = 6;
  __shared__ LogShared<THREADS> sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ranks = p.cluster, rank = ranks > 1 ? (int)cluster_rank() : 0;
  const long long r = ranks > 1 ? blockIdx.x / (unsigned)ranks : blockIdx.x;
  const float c2 = p.scale * 1.4426950408889634f;
  if (tid == 0) {
    sh.owner = THREADS;
    sh.n_above = sh.n_equal = sh.n_hot = 0;
    sh.bound = INFINITY;
  }
  if (ranks > 1) cluster_arrive();     // waited for before the first access of another CTA's memory
  griddep_launch_dependents();
  griddep_wait();
  const LogRow<E, THREADS> row(p, r, rank, ranks);

  // ------------------------------------------------------ one pass
  LogSums mine;
  int v = row.v0 + tid;
  if (v + (AHEAD - 1) * THREADS < row.v1) {
    // a batch in the sums, the next one on its way
    uint4 raw[AHEAD];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) raw[k] = row.load(v + k * THREADS);
    for (v += AHEAD * THREADS; v + (AHEAD - 1) * THREADS < row.v1; v += AHEAD * THREADS) {
      uint4 next[AHEAD];
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) next[k] = row.load(v + k * THREADS);
      mine.template add<E>(raw, c2);
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) raw[k] = next[k];
    }
    mine.template add<E>(raw, c2);
  }
  for (; v < row.v1; v += THREADS) {
    const uint4 raw[1] = {row.load(v)};
    mine.template add<E>(raw, c2);
  }
  if (tid < row.extra) {
    const float x = E::get(row.x + row.extra_index(tid));
    if (x > mine.m) mine.raise(x, c2);
    mine.one(x, c2);
  }

  // ------------------------------------------------------ the largest, and a bound of the alternatives
  float M = mine.m;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
    if (2 * d == QUAD && lane % QUAD == 0) sh.group[tid / QUAD] = M;
  }
  if (QUAD == 1) sh.group[tid] = mine.m;
  if (lane == 0) sh.warp_S[warp] = M;
  __syncthreads();
  for (int w = 0; w < THREADS / 32; ++w) M = fmaxf(M, sh.warp_S[w]);
  if (mine.m == M && M > -INFINITY) atomicMin(&sh.owner, tid);
  if (p.top > 0) {
    // rank of this thread's group among all, a share of the comparisons each
    const int g = tid / QUAD;
    const float x = sh.group[g];
    int n = 0;
#pragma unroll 8
    for (int j = tid % QUAD; j < 128; j += QUAD) {
      const float y = sh.group[j];
      n += y > x || (y == x && j < g) ? 1 : 0;
    }
#pragma unroll
    for (int d = 1; d < QUAD; d <<= 1) n += __shfl_xor_sync(0xffffffffu, n, d);
    if (n == p.top - 1) sh.bound = x;
  }
  __syncthreads();
  const float bound = sh.bound;
  const int owner = sh.owner;
  // (elements of -inf that are alternatives all the same come by the walk in order)
  if (tid == owner || (p.top > 0 && mine.m >= bound && mine.m > -INFINITY))
    sh.hot[atomicAdd(&sh.n_hot, 1)] = tid;
  // everyone's sums relative to M; the owner's come again without the largest
  float S = 0.0f, W = 0.0f;
  if (tid != owner) {
    if (mine.m > -INFINITY) mine.scale(mine.rise(M, 0.0f, false, c2));
    const float2 s = f32x2_get(mine.S), w = f32x2_get(mine.W);
    S = s.x + s.y;
    W = w.x + w.y;
  }
  __syncthreads();
  const int n_hot = sh.n_hot;
  for (int h = warp; h < n_hot; h += THREADS / 32) {
    const int t = sh.hot[h];
    int top_count = 0;
    row.each(t, lane, [&](float x, int i) {
      if (p.top > 0 && x >= bound) {
        // (no more than tells that there are too many)
        if (x > bound) {
          if (*(volatile int*)&sh.n_above <= kMostAbove) {
            const int at = atomicAdd(&sh.n_above, 1);
            if (at < kMostAbove) sh.above[at] = {x, i};
          }
        } else if (bound > -INFINITY && *(volatile int*)&sh.n_equal <= kMostEqual) {
          const int at = atomicAdd(&sh.n_equal, 1);
          if (at < kMostEqual) sh.equal[at] = i;
        }
      }
      if (t == owner) {
        if (x == M) {
          ++top_count;
        } else {
          const float d = max_nan((x - M) * c2, -200.0f), e = exp2_fast(d);
          S += e;
          W += d * e;
        }
      }
    });
    if (t == owner) {
      top_count = __reduce_add_sync(0xffffffffu, top_count);
      if (lane == 0) S += (float)(top_count - 1);
    }
  }
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) {
    S += __shfl_xor_sync(0xffffffffu, S, d);
    W += __shfl_xor_sync(0xffffffffu, W, d);
  }
  if (lane == 0) {
    sh.warp_S[warp] = S;
    sh.warp_W[warp] = W;
  }
  __syncthreads();

  // ------------------------------------------------------ this CTA's alternatives, in order
  Best* list = sh.top[rank];
  if (p.top > 0) {
    const int na = sh.n_above, ne = sh.n_equal;
    if (na > kMostAbove) {
      top_by_passes(row, sh, p.top, list);
    } else {
      for (int i = tid; i < na; i += THREADS) {
        const Best b = sh.above[i];
        int n = 0;
        for (int j = 0; j < na; ++j) n += before(sh.above[j], b) ? 1 : 0;
        if (n < p.top) list[n] = b;
      }
      const int need = p.top - na;
      if (need > 0) {
        int found = min(need, ne);
        if (bound == -INFINITY || ne > kMostEqual) {
          found = equals_in_order(row, sh, bound, need, list + na);
        } else {
          for (int t = tid; t < ne; t += THREADS) {
            const int b = sh.equal[t];
            int n = 0;
            for (int j = 0; j < ne; ++j) n += sh.equal[j] < b ? 1 : 0;
            if (n < need) list[na + n] = {bound, b};
          }
        }
        for (int k = na + found + tid; k < p.top; k += THREADS) list[k] = {-INFINITY, -1};
      }
    }
  }
  LogRest sum = {M, 0.0f, 0.0f};
  for (int w = 0; w < THREADS / 32; ++w) {
    sum.S += sh.warp_S[w];
    sum.W += sh.warp_W[w];
  }
  __syncthreads();

  // ------------------------------------------------------ the cluster's
  if (ranks > 1) {
    cluster_wait();
    if (rank != 0) {
      for (int i = tid; i < 2 * p.top; i += THREADS)
        cluster_store(cluster_addr(smem_u32(reinterpret_cast<float*>(sh.top[rank]) + i), 0),
                      reinterpret_cast<const float*>(list)[i]);
      if (tid < 3)
        cluster_store(cluster_addr(smem_u32(&sh.sums[rank][tid]), 0),
                      tid == 0 ? sum.m : tid == 1 ? sum.S : sum.W);
    }
    cluster_sync();
    if (rank != 0) return;
    for (int k = 1; k < ranks; ++k) join_sums(sum, LogRest{sh.sums[k][0], sh.sums[k][1], sh.sums[k][2]}, c2);
  }
  const bool finite = fabsf(sum.m) != INFINITY && sum.S == sum.S;
  const float nan = __uint_as_float(0x7fffffffu), log_sum = finite ? log1pf(sum.S) : nan;
  if (tid == 0) {
    if (p.logp) {
      const int t = p.targets[r];
      p.logp[r] = t >= 0 && t < p.vocab ? (E::get(row.x + t) - sum.m) * p.scale - log_sum : nan;
    }
    if (p.entropy) p.entropy[r] = log_sum - sum.W * 0.6931471805599453f / (1.0f + sum.S);
  }
  for (int i = tid; i < ranks * p.top; i += THREADS) {
    // an alternative's place: its own in its list, and how many of each other list come before it
    const int k = i / p.top, at = i - k * p.top;
    const Best b = sh.top[k][at];
    int n = at;
    for (int o = 0; o < ranks; ++o) {
      if (o == k) continue;
      int lo = 0, hi = p.top;
      while (lo < hi) {
        const int mid = (lo + hi) / 2;
        // those that are none come last, in the order of the lists
        const Best c = sh.top[o][mid];
        const bool first = b.i < 0 && c.i < 0 ? o < k : before(c, b);
        if (first)
          lo = mid + 1;
        else
          hi = mid;
      }
      n += lo;
    }
    if (n < p.top) {
      p.top_ids[r * p.top + n] = b.i;
      p.top_logp[r * p.top + n] = b.i < 0 ? nan : (b.x - sum.m) * p.scale - log_sum;
    }
  }
}

namespace {

template <typename E>
cudaError_t launch_logprobs(const LogprobsParams& p, int rows, int threads, cudaStream_t st) {
  const dim3 grid((unsigned)rows * (unsigned)p.cluster);
  return threads == 128 ? op_launch(logprobs_kernel<E, 128>, grid, dim3(128), 0, st, p.cluster, p)
                        : op_launch(logprobs_kernel<E, 512>, grid, dim3(512), 0, st, p.cluster, p);
}

}  // namespace
}  // namespace dllm

using namespace dllm;

extern "C" dllm_status dllm_op_token_logprobs(const void* logits, int64_t row_stride, int32_t dtype, int32_t rows,
                                              int32_t vocab, float inv_temperature, const int32_t* targets,
                                              float* logprobs, float* entropy, int32_t top, int32_t* top_ids,
                                              float* top_logprobs, void* stream) {
  const int es = op_dtype_size(dtype);
  if (!logits || rows < 1 || vocab < 1 || vocab > kMostRows || es == 0 || !(inv_temperature > 0.0f) ||
      !std::isfinite(inv_temperature) || top < 0 || top > 64 || top > vocab)
    return op_fail(DLLM_EINVAL,
                   "bad token_logprobs arguments: rows=%d vocab=%d dtype=%d inv_temperature=%g (over 0, finite) top=%d "
                   "(to 64 and vocab)",
                   rows, vocab, dtype, inv_temperature, top);
  if ((logprobs != nullptr) != (targets != nullptr) || (top > 0) != (top_ids != nullptr) ||
      (top > 0) != (top_logprobs != nullptr))
    return op_fail(DLLM_EINVAL,
                   "token_logprobs: targets and logprobs go together, and so do top > 0, top_ids and top_logprobs");
  if (!op_aligned(logits, es) || !op_aligned(targets, 4) || !op_aligned(logprobs, 4) || !op_aligned(entropy, 4) ||
      !op_aligned(top_ids, 4) || !op_aligned(top_logprobs, 4))
    return op_fail(DLLM_EINVAL, "token_logprobs: arrays must be aligned to their elements");
  LogprobsParams p = {};
  p.logits = logits;
  p.rs = row_stride ? row_stride : vocab;
  if (p.rs < vocab || p.rs > (1LL << 40))
    return op_fail(DLLM_EINVAL, "token_logprobs: row stride %lld (0, or at least vocab=%d)", p.rs, vocab);
  p.targets = targets;
  p.logp = logprobs;
  p.entropy = entropy;
  p.top = top;
  p.top_ids = top_ids;
  p.top_logp = top_logprobs;
  p.vocab = vocab;
  p.scale = inv_temperature;
  // Threads of a row, and CTAs: as many as fill the GPU, each with 8192 elements at least.
  const int threads = vocab <= 8192 ? 128 : 512;
  p.cluster = 1;
  while (p.cluster < kLogCluster && (long long)rows * p.cluster * 2 <= 3LL * op_device_sms() &&
         vocab / (p.cluster * 2) >= 8192)
    p.cluster *= 2;
  if ((long long)rows * p.cluster > 0x7fffffff) p.cluster = 1;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  switch (dtype) {
    case DLLM_F32: OP_CK(launch_logprobs<ElemF32>(p, rows, threads, st)); break;
    case DLLM_BF16: OP_CK(launch_logprobs<ElemBf16>(p, rows, threads, st)); break;
    default: OP_CK(launch_logprobs<ElemF16>(p, rows, threads, st)); break;
  }
  return DLLM_OK;
}
