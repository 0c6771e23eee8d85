// What rows of logits say: log probabilities of given tokens, entropy, the largest alternatives.
//
// With M the largest z of a row, at token a, and sums over the others,
//   S = sum e^(z - M),  W = sum (z - M) e^(z - M):
//   log p_i = (z_i - M) - log1p(S),   entropy = log1p(S) - W / (1 + S).
// The largest term is left out of the sums, so a nearly certain row's S keeps its relative accuracy, and both
// parts of the entropy are of one sign.
//
// Bound by HBM: the logits are read once.  A CTA takes row after row (or a cluster of up to 8 one row, where rows are
// few).  One warp copies the rows into a ring in shared memory, past the end of a row too; eight (four for short rows)
// stream them: every thread keeps the largest of its elements m and, relative to it, S and W of them all (in float32
// chains of 256 terms, each joined to those before), leaves them in shared memory and goes on to the next row.  Four
// warps work out a row's results meanwhile (the same threads one after the other took 212 us for the case below, with
// loads into registers and results apart 217).
// What needs elements again is a few threads' worth, which lies in L2 still:
//   - the alternatives are among the elements of units whose largest is no less than the top-th largest of 128 group
//     maxima (a lower bound of the top-th largest element): for 20 of 126464 about 22 units of 32 elements.  Elements
//     above the bound are ranked by counting; its equals join in the order of their ids.
//   - where the others' S is less than the largest's 1, the thread that holds it takes its sums again without it.
// Rows that would give more than 512 elements above the bound (a few threads' are the largest by far) take a pass of the
// row an alternative.
// 4096 rows of 126464 in bf16, 20 alternatives: 172 us, 6.0 TB/s (none: 157, 50: 193; 2048 rows of float32: 156); 32 rows,
// 5 alternatives: 12.4 us, of which a chain of reductions and a cluster's join are the most; 257 rows of 32001 in float32:
// 12.8 us.  Beside HBM the issue slots bound it: the warps that work out results take them from those that stream.  At
// an earlier step (184 us) three CTAs an SM with 56 registers a thread took 212, 384 streaming threads 189.  A second team of
// warps for the results, rows in turn, takes 184 here.
#include <algorithm>
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
  int rows, vocab, top, cluster, slots, units;
  float scale;
};

constexpr int kMostTop = 64;
constexpr int kMostAbove = 512;      // elements above the bound that are ranked
constexpr int kMostEqual = 256;      // and equals that are, before the row is walked for them in order
constexpr int kLogCluster = 8;
constexpr int kLogAhead = 4;         // vectors of a thread in a chunk of the ring (a batch)
constexpr int kLogRest = 128;        // threads that work out a row's results

// MAIN: streaming threads
template <int MAIN>
struct LogCfg {
  static constexpr int THREADS = MAIN + kLogRest + 32;
  static constexpr int CTAS = MAIN == 128 ? 4 : 2;               // an SM
  static constexpr int CHUNK = kLogAhead * MAIN;                 // vectors, a batch of every thread's (two: 212 us)
  static constexpr int SLOTS = 6;                                // of the ring, at most
};
constexpr int kLogGroups = 128;
// alternatives up to which 32 groups give the bound, else 128 (32 / 128 groups, 4096 rows of 126464: 1 alternative 164, 169
// us, 5 167, 172, 20 172.6, 175.4, 24 176.2, 175.8, 32 274, 180; 32 rows, 5 alternatives 12.2, 12.8, 20 18.9, 18.4)
constexpr int kLogFewTop = 24;
constexpr int kLogUnits = 16;        // of a thread's batches at most, each with a largest element of its own (and one for the rest)
constexpr int kMostUnits = 512;      // units that are looked through again, before all are
constexpr int kLogChain = 256;       // additions of a chain of sums at most, before it joins the chains before

static __device__ int g_logprobs_err[1];

struct Best {
  float x;
  int i;    // -1: none
};
// a before b: larger, or of a lower index
__device__ __forceinline__ bool before(const Best& a, const Best& b) {
  return a.i >= 0 && (b.i < 0 || a.x > b.x || (a.x == b.x && a.i < b.i));
}

// A float as a whole number of the same order (-0 as 0), and back.
__device__ __forceinline__ int log_order(float x) {
  const int b = __float_as_int(x + 0.0f);
  return b ^ ((b >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float log_value(int o) { return __int_as_float(o ^ ((o >> 31) & 0x7fffffff)); }
// An element and its id as one number: the larger element, then the lower id, is more.
__device__ __forceinline__ unsigned long long log_key(float x, int i) {
  return (unsigned long long)((uint32_t)log_order(x) ^ 0x80000000u) << 32 | (uint32_t)~i;
}
__device__ __forceinline__ Best log_best(unsigned long long key) {
  return {log_value((int)((uint32_t)(key >> 32) ^ 0x80000000u)), (int)~(uint32_t)key};
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

// (x - M) c, by half the difference: the whole may be more than float32 holds (c: up to 2^126.8).
__device__ __forceinline__ float apart(float x, float M, float c) { return fmaf(x, 0.5f, -0.5f * M) * (2.0f * c); }

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
  __device__ __forceinline__ float add(const uint4 (&r)[n], float c2) {   // their largest
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
    return top;
  }
  // What the sums are relative to m c2 itself, with t's, of no larger an m, joined where there are any; the chain starts
  // anew.
  __device__ __forceinline__ void fold(float& t_m, float& t_S, float& t_W, bool any, float c2) {
    if (plain) scale(rise(m, 0.0f, false, c2));
    const float2 s = f32x2_get(S), w = f32x2_get(W);
    float S_all = s.x + s.y, W_all = w.x + w.y;
    if (any) {
      const float d = t_m == m ? 0.0f : max_nan(apart(t_m, m, c2), -200.0f), f = exp2_fast(d);
      W_all += (t_W + t_S * d) * f;
      S_all += t_S * f;
    }
    t_m = m;
    t_S = S_all;
    t_W = W_all;
    S = W = 0;
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
  const float d = max_nan(apart(o.m, t.m, c2), -200.0f), f = exp2_fast(d);
  t.S += (1.0f + o.S) * f;
  t.W += (o.W + (1.0f + o.S) * d) * f;
}

template <int MAIN>
struct alignas(128) LogShared {
  float m[2][MAIN], S[2][MAIN], W[2][MAIN];      // of the streaming threads, rows in turn
  alignas(8) uint64_t ready[2], done[2], full[LogCfg<MAIN>::SLOTS], empty[LogCfg<MAIN>::SLOTS];
  float own[4];                                  // the owner's S and W, with the largest and taken again without it
  float warp_m[kLogRest / 32], warp_S[kLogRest / 32], warp_W[kLogRest / 32];
  int warp_n[kLogRest / 32], warp_owner[kLogRest / 32];
  alignas(16) int group[kLogGroups];             // group maxima, as whole numbers of their order
  int bound;
  int n_above, n_equal, n_hot;
  int hot[kMostUnits];
  unsigned long long above[kMostAbove];
  int equal[kMostEqual];
  Best top[kLogCluster][kMostTop];               // lists of the cluster's CTAs, in order
  float sums[kLogCluster][3];                    // m, S, W
  Best best[kLogRest / 32];
  int abort;
};

__device__ __forceinline__ void rest_sync() { named_bar_sync(1, kLogRest); }

template <typename E, int MAIN>
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
    v0 = ranks == 1 ? 0 : (int)((long long)nvec * rank / ranks);
    v1 = ranks == 1 ? nvec : (int)((long long)nvec * (rank + 1) / ranks);
    extra = rank == 0 ? vocab - nvec * VE : 0;
  }
  // of a thread: its vectors, and batches that make a unit
  __device__ __forceinline__ int vectors(int t) const { return max(0, (v1 - v0 - t + MAIN - 1) / MAIN); }
  __device__ __forceinline__ int span_log() const {
    const int batches = vectors(0) / kLogAhead;
    return batches <= kLogUnits ? 0 : 32 - __clz((batches - 1) / kLogUnits);
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
};

// The `top` best of the CTA's elements, in order, one pass each.
template <typename E, int MAIN>
__device__ void top_by_passes(const LogRow<E, MAIN>& row, LogShared<MAIN>& sh, int tid, int top, Best* out) {
  Best last = {INFINITY, -1};
  for (int k = 0; k < top; ++k) {
    Best b = {0.0f, -1};
    auto look = [&](float x, int i) {
      const Best c = {x, i};
      if (x == x && (k == 0 || before(last, c)) && before(c, b)) b = c;
    };
    for (int v = row.v0 + tid; v < row.v1; v += kLogRest) {
      float e[LogRow<E, MAIN>::VE];
      row.floats(row.load(v), e);
#pragma unroll
      for (int i = 0; i < LogRow<E, MAIN>::VE; ++i) look(e[i], row.index(v, i));
    }
    if (tid < row.extra) look(E::get(row.x + row.extra_index(tid)), row.extra_index(tid));
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) {
      const Best o = {__shfl_xor_sync(0xffffffffu, b.x, d), __shfl_xor_sync(0xffffffffu, b.i, d)};
      if (before(o, b)) b = o;
    }
    rest_sync();
    if (tid % 32 == 0) sh.best[tid / 32] = b;
    rest_sync();
    b = sh.best[0];
    for (int w = 1; w < kLogRest / 32; ++w)
      if (before(sh.best[w], b)) b = sh.best[w];
    if (tid == 0) out[k] = b;
    last = b;
    if (b.i < 0) {                     // none left, here and in every further pass
      for (int j = k + 1 + tid; j < top; j += kLogRest) out[j] = b;
      break;
    }
  }
}

// The first `need` elements equal to `bound` in the order of their ids, and how many there are; the CTA's elements
// lie in the order head, vectors, tail.
template <typename E, int MAIN>
__device__ int equals_in_order(const LogRow<E, MAIN>& row, LogShared<MAIN>& sh, int tid, float bound, int need, Best* out) {
  constexpr int VE = LogRow<E, MAIN>::VE;
  const int lane = tid & 31, warp = tid >> 5, heads = row.extra ? row.head : 0;
  int found = 0;
  for (int at = row.v0 - kLogRest; at < row.v1 + kLogRest && found < need; at += kLogRest) {
    // one step for the head, one of kLogRest vectors each, one for the tail
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
    rest_sync();
    int pos = found + upto - __popc(mask);
    int total = 0;
    for (int w = 0; w < kLogRest / 32; ++w) {
      if (w < warp) pos += sh.warp_n[w];
      total += sh.warp_n[w];
    }
    for (; mask && pos < need; mask &= mask - 1, ++pos) out[pos] = {bound, first + __ffs(mask) - 1};
    found += total;
    rest_sync();
  }
  return min(found, need);
}

// A row's results from the streaming threads' sums in buffer b; by kLogRest threads.
template <typename E, int MAIN, bool LONG>
__device__ __forceinline__ void row_results(const LogprobsParams& p, LogShared<MAIN>& sh, const LogRow<E, MAIN>& row, int r,
                                            int b, int tid, int rank, int ranks, float c2, const float* unit) {
  constexpr int VE = LogRow<E, MAIN>::VE, EACH = MAIN / kLogRest;
  const int lane = tid & 31, warp = tid >> 5, top = p.top;
  // the given token's logit, on its way from the start: it is due at the end
  const int target = p.logp && tid == 0 && rank == 0 ? p.targets[r] : -1;
  const bool given = target >= 0 && target < p.vocab;
  typename E::T given_x{};
  if (given) given_x = row.x[target];
  float m[EACH], M = -INFINITY;
#pragma unroll
  for (int k = 0; k < EACH; ++k) {
    m[k] = sh.m[b][tid + k * kLogRest];
    M = fmaxf(M, m[k]);
  }
  sh.group[tid] = log_order(M);
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
  if (lane == 0) sh.warp_m[warp] = M;
  if (tid == 0) {
    sh.n_above = sh.n_equal = sh.n_hot = 0;
    sh.bound = 0x7fffffff;
  }
  rest_sync();
#pragma unroll
  for (int w = 0; w < kLogRest / 32; ++w) M = fmaxf(M, sh.warp_m[w]);
  // everyone's sums relative to M; a holder of the largest, the first one, apart
  float S = 0.0f, W = 0.0f, Sown = 0.0f, Wown = 0.0f;
  int owner = MAIN;
#pragma unroll
  for (int k = 0; k < EACH; ++k) {
    const int t = tid + k * kLogRest;
    float s = sh.S[b][t], w = sh.W[b][t];
    if (m[k] > -INFINITY) {
      const float d = max_nan(apart(m[k], M, c2), -200.0f), f = exp2_fast(d);
      w = (w + s * d) * f;
      s *= f;
    }
    if (m[k] == M && M > -INFINITY && owner == MAIN) {
      owner = t;
      Sown = s;
      Wown = w;
    } else {
      S += s;
      W += w;
    }
  }
  // The bound: the least of the group maxima that fewer than `top` others exceed; by every warp for itself from 32 groups
  // where few alternatives are wanted, else from 128.
  int order = 0x7fffffff;
  if (top > kLogFewTop) {
    const int x = sh.group[tid];
    int n = 0;
#pragma unroll 8
    for (int j = 0; j < kLogGroups; j += 4) {
      const int4 y = *reinterpret_cast<const int4*>(&sh.group[j]);
      n += (y.x > x) + (y.y > x) + (y.z > x) + (y.w > x);
    }
    const int least = __reduce_min_sync(0xffffffffu, n < top ? x : 0x7fffffff);
    if (lane == 0) atomicMin(&sh.bound, least);
  } else if (top > 0) {
    const int4 y = *reinterpret_cast<const int4*>(&sh.group[4 * lane]);
    const int x = max(max(y.x, y.y), max(y.z, y.w));
    int n = 0;
#pragma unroll
    for (int j = 0; j < 32; ++j) n += __shfl_sync(0xffffffffu, x, j) > x ? 1 : 0;
    order = __reduce_min_sync(0xffffffffu, n < top ? x : 0x7fffffff);
  }
  const int best_owner = __reduce_min_sync(0xffffffffu, owner);
  if (lane == 0) sh.warp_owner[warp] = best_owner;
  rest_sync();
  owner = MAIN;
#pragma unroll
  for (int w = 0; w < kLogRest / 32; ++w) owner = min(owner, sh.warp_owner[w]);
  if (owner < MAIN && owner % kLogRest == tid) {
    sh.own[0] = Sown;
    sh.own[1] = Wown;
  } else {                             // (another holder's sums are like everyone's)
    S += Sown;
    W += Wown;
  }
  if (top > kLogFewTop) order = sh.bound;
  const float bound = top > 0 ? log_value(order) : INFINITY;
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) {
    S += __shfl_xor_sync(0xffffffffu, S, d);
    W += __shfl_xor_sync(0xffffffffu, W, d);
  }
  if (lane == 0) {
    sh.warp_S[warp] = S;
    sh.warp_W[warp] = W;
  }
  // the units that may hold alternatives (elements of -inf that are some all the same come by the walk in order)
  const int span_log = row.span_log();
  if (top > 0) {
#pragma unroll
    for (int k = 0; k < EACH; ++k) {
      const bool hot = m[k] >= bound && m[k] > -INFINITY;
      if (!__any_sync(0xffffffffu, hot)) continue;
      const int t = tid + k * kLogRest, units = ((row.vectors(t) / kLogAhead + (1 << span_log) - 1) >> span_log) + 1;
      uint32_t mask = 0;
#pragma unroll
      for (int j = 0; j <= kLogUnits; ++j) mask |= j < units && unit[j * MAIN + t] >= bound ? 1u << j : 0;
      if (!hot) mask = 0;
      for (; mask; mask &= mask - 1) {
        const int at = atomicAdd(&sh.n_hot, 1);
        if (at < kMostUnits) sh.hot[at] = (__ffs(mask) - 1) * MAIN + t;
      }
    }
  }
  rest_sync();
  LogRest sum = {M, 0.0f, 0.0f};
#pragma unroll
  for (int w = 0; w < kLogRest / 32; ++w) {
    sum.S += sh.warp_S[w];
    sum.W += sh.warp_W[w];
  }
  // the owner's, without the largest's 1: taken again by the first warp where the subtraction would tell
  const bool owned = owner < MAIN, again = owned && !(sum.S + sh.own[0] >= 2.0f);
  if (owned && !again) {
    sum.S += sh.own[0] - 1.0f;
    sum.W += sh.own[1];
  }
  if (again && warp == 0) {
    float s = 0.0f, w = 0.0f;
    int same = 0;
    auto other = [&](float x) {
      if (x == M) {
        ++same;
        return;
      }
      const float d = max_nan(apart(x, M, c2), -200.0f), e = exp2_fast(d);
      s += e;
      w += d * e;
    };
    float s_all = 0.0f, w_all = 0.0f;  // of the chains before, of 32 vectors each
    int n = 0;
    for (int v = row.v0 + owner + lane * MAIN; v < row.v1; v += 32 * MAIN) {
      float e[VE];
      row.floats(row.load(v), e);
#pragma unroll
      for (int i = 0; i < VE; ++i) other(e[i]);
      if (LONG && (++n & 31) == 0) {
        s_all += s;
        w_all += w;
        s = w = 0.0f;
      }
    }
    if (lane == 0 && owner < row.extra) other(E::get(row.x + row.extra_index(owner)));
    if (LONG) {
      s += s_all;
      w += w_all;
    }
    same = __reduce_add_sync(0xffffffffu, same);
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) {
      s += __shfl_xor_sync(0xffffffffu, s, d);
      w += __shfl_xor_sync(0xffffffffu, w, d);
    }
    if (lane == 0) {
      sh.own[2] = s + (float)(same - 1);
      sh.own[3] = w;
    }
  }
  // ------------------------------------------------------ alternatives: the hot threads' elements
  if (top > 0) {
    // a warp's elements, some of every lane: those above the bound and its equals find places together
    auto look = [&](uint32_t above, uint32_t equal, auto element) {
      if (!__any_sync(0xffffffffu, (above | equal) != 0)) return;
      int upto = __popc(above) | __popc(equal) << 16;
      const int own = upto;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, upto, d);
        if (lane >= d) upto += o;
      }
      int at = 0, ae = 0;
      if (lane == 31) {                // (no more than tells that there are too many)
        at = *(volatile int*)&sh.n_above <= kMostAbove && (upto & 0xffff) ? atomicAdd(&sh.n_above, upto & 0xffff) : kMostAbove;
        ae = *(volatile int*)&sh.n_equal <= kMostEqual && upto >> 16 ? atomicAdd(&sh.n_equal, upto >> 16) : kMostEqual;
      }
      at = __shfl_sync(0xffffffffu, at, 31) + ((upto - own) & 0xffff);
      ae = __shfl_sync(0xffffffffu, ae, 31) + ((upto - own) >> 16);
      for (; above; above &= above - 1, ++at) {
        float x;
        const int i = element(__ffs(above) - 1, x);
        if (at < kMostAbove) sh.above[at] = log_key(x, i);
      }
      for (; equal; equal &= equal - 1, ++ae) {
        float x;
        const int i = element(__ffs(equal) - 1, x);
        if (ae < kMostEqual) sh.equal[ae] = i;
      }
    };
    const int n_hot = sh.n_hot, each = kLogAhead << span_log;   // vectors of a unit, at most
    auto look_vector = [&](int v) {    // (v1: none)
      float e[VE] = {};
      uint32_t above = 0, equal = 0;
      if (v < row.v1) {
        row.floats(row.load(v), e);
#pragma unroll
        for (int i = 0; i < VE; ++i) {
          above |= e[i] > bound ? 1u << i : 0;
          equal |= e[i] == bound && bound > -INFINITY ? 1u << i : 0;
        }
      }
      look(above, equal, [&](int i, float& x) {
        x = E::get(row.x + row.index(v, i));
        return row.index(v, i);
      });
    };
    if (n_hot <= kMostUnits) {
      const int items = n_hot * each;
      for (int i0 = warp * 32; i0 < items; i0 += kLogRest) {
        const int i = i0 + lane, h = i >> (2 + span_log);
        int v = row.v1;
        if (i < items) {
          const int code = sh.hot[h], j = code / MAIN, t = code - j * MAIN;
          const int n = row.vectors(t), batches = n / kLogAhead, units = (batches + (1 << span_log) - 1) >> span_log;
          // the unit's first vector, and the end of its own
          const int first = j < units ? j * each : batches * kLogAhead;
          const int end = j < units ? min(first + each, batches * kLogAhead) : n, at = first + i - h * each;
          if (at < end) v = row.v0 + t + at * MAIN;
        }
        look_vector(v);
      }
    } else {
      for (int v = row.v0 + warp * 32; v < row.v1; v += kLogRest) look_vector(min(v + lane, row.v1));
    }
    if (row.extra > 0 && warp == 0) {
      const float x = lane < row.extra ? E::get(row.x + row.extra_index(lane)) : -INFINITY;
      look(lane < row.extra && x > bound, lane < row.extra && x == bound && bound > -INFINITY, [&](int, float& y) {
        y = x;
        return row.extra_index(lane);
      });
    }
  }
  if (top > 0 || again) rest_sync();   // (again is the same for all)
  if (again) {
    sum.S += sh.own[2];
    sum.W += sh.own[3];
  }
  Best* list = sh.top[rank];
  if (top > 0) {
    const int na = sh.n_above, ne = sh.n_equal;
    if (na > kMostAbove) {
      top_by_passes(row, sh, tid, top, list);
    } else {
      // how many come before an element: eight elements a warp at a time, against 64 in its lanes
      for (int i0 = warp * 8; i0 < na; i0 += 8 * (kLogRest / 32)) {
        int n = 0;                     // lane k: of element i0 + k
        const unsigned long long mine = sh.above[min(i0 + (lane & 7), na - 1)];
        for (int j = 0; j < na; j += 64) {
          const unsigned long long a = j + lane < na ? sh.above[j + lane] : 0;
          const unsigned long long c = j + 32 + lane < na ? sh.above[j + 32 + lane] : 0;
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const unsigned long long x = __shfl_sync(0xffffffffu, mine, k);
            const int more = __popc(__ballot_sync(0xffffffffu, a > x)) + __popc(__ballot_sync(0xffffffffu, c > x));
            n += lane == k ? more : 0;
          }
        }
        if (lane < 8 && i0 + lane < na && n < top) list[n] = log_best(mine);
      }
      const int need = top - na;
      if (need > 0) {
        int found = min(need, ne);
        if (bound == -INFINITY || ne > kMostEqual) {
          found = equals_in_order(row, sh, tid, bound, need, list + na);
        } else {
          for (int t = tid; t < ne; t += kLogRest) {
            const int x = sh.equal[t];
            int n = 0;
            for (int j = 0; j < ne; ++j) n += sh.equal[j] < x ? 1 : 0;
            if (n < need) list[na + n] = {bound, x};
          }
        }
        for (int k = na + found + tid; k < top; k += kLogRest) list[k] = {-INFINITY, -1};
      }
    }
    rest_sync();
  }

  // ------------------------------------------------------ the cluster's
  if (ranks > 1) {
    cluster_wait();
    if (rank != 0) {
      for (int i = tid; i < 2 * top; i += kLogRest)
        cluster_store(cluster_addr(smem_u32(reinterpret_cast<float*>(sh.top[rank]) + i), 0),
                      reinterpret_cast<const float*>(list)[i]);
      if (tid < 3)
        cluster_store(cluster_addr(smem_u32(&sh.sums[rank][tid]), 0), tid == 0 ? sum.m : tid == 1 ? sum.S : sum.W);
    }
    cluster_sync();
    if (rank != 0) return;
    for (int k = 1; k < ranks; ++k) join_sums(sum, LogRest{sh.sums[k][0], sh.sums[k][1], sh.sums[k][2]}, c2);
  }
  const bool finite = fabsf(sum.m) != INFINITY && sum.S == sum.S;
  const float nan = __uint_as_float(0x7fffffffu), log_sum = finite ? log1pf(sum.S) : nan;
  if (tid == 0) {
    if (p.logp) p.logp[r] = given ? apart(E::get(&given_x), sum.m, p.scale) - log_sum : nan;
    if (p.entropy) p.entropy[r] = log_sum - sum.W * 0.6931471805599453f / (1.0f + sum.S);
  }
  for (int i = tid; i < ranks * top; i += kLogRest) {
    // an alternative's place: its own in its list, and how many of each other list come before it
    const int k = ranks == 1 ? 0 : i / top, at = i - k * top;
    const Best x = sh.top[k][at];
    int n = at;
    for (int o = 0; o < ranks; ++o) {
      if (o == k) continue;
      int lo = 0, hi = top;
      while (lo < hi) {
        const int mid = (lo + hi) / 2;
        // those that are none come last, in the order of the lists
        const Best c = sh.top[o][mid];
        const bool first = x.i < 0 && c.i < 0 ? o < k : before(c, x);
        if (first)
          lo = mid + 1;
        else
          hi = mid;
      }
      n += lo;
    }
    if (n < top) {
      p.top_ids[(long long)r * top + n] = x.i;
      p.top_logp[(long long)r * top + n] = x.i < 0 ? nan : apart(x.x, sum.m, p.scale) - log_sum;
    }
  }
}

// Vectors of a CTA whose sums are one chain: two elements of a batch an addition.
template <typename E, int MAIN>
constexpr int kLogChainVectors = kLogChain * 2 / (16 / (int)sizeof(typename E::T)) * MAIN;

// (rows of one chain apart: with the joins in their loop 4096 rows of 126464 in bf16 take 180 us for 173; 256 rows of
// 1048576, which need them, 111 us, 107 with one chain)
template <typename E, int MAIN, bool LONG>
__global__ void __launch_bounds__(LogCfg<MAIN>::THREADS, LogCfg<MAIN>::CTAS)
    logprobs_kernel(const __grid_constant__ LogprobsParams p) {
  using C = LogCfg<MAIN>;
  constexpr int AHEAD = kLogAhead;
  extern __shared__ __align__(128) uint8_t s_raw[];
  LogShared<MAIN>& sh = *reinterpret_cast<LogShared<MAIN>*>(s_raw);
  uint4* ring = reinterpret_cast<uint4*>(s_raw + sizeof(LogShared<MAIN>));   // p.slots chunks
  float* unit0 = reinterpret_cast<float*>(ring + p.slots * C::CHUNK);        // [2][p.units][MAIN] largest elements
  const int tid = threadIdx.x, lane = tid & 31;
  const int ranks = p.cluster, rank = ranks > 1 ? (int)cluster_rank() : 0;
  const float c2 = p.scale * 1.4426950408889634f;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.ready[i], MAIN / 32);
      mbar_init(&sh.done[i], kLogRest / 32);
    }
    for (int i = 0; i < C::SLOTS; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], MAIN / 32);
    }
    sh.abort = 0;
    fence_mbar_init();
  }
  if (ranks > 1) cluster_arrive();     // waited for before the first access of another CTA's memory
  __syncthreads();
  griddep_launch_dependents();
  griddep_wait();
  const int first_row = (int)(blockIdx.x / (unsigned)ranks), row_step = (int)(gridDim.x / (unsigned)ranks);
  int k = 0, slot = 0;                 // rows so far (one where the CTA is of a cluster); the ring's place
  uint32_t phase = 0;
  if (tid < MAIN) {
    for (int r = first_row; r < p.rows; r += row_step, ++k) {
      const LogRow<E, MAIN> row(p, r, rank, ranks);
      const int b = k & 1;
      if (k >= 2) {
        mbar_wait_long(&sh.done[b], (uint32_t)(k / 2 - 1) & 1u, &sh.abort, g_logprobs_err, ERR_LOGPROBS);
        __syncwarp();
      }
      LogSums mine;
      const int span = 1 << row.span_log();
      int left = span;                 // batches until the unit is full
      float largest = -INFINITY;       // the unit's
      float* unit = unit0 + b * p.units * MAIN + tid;
      auto batch = [&](float top) {
        largest = fmaxf(largest, top);
        if (--left == 0) {
          *unit = largest;
          unit += MAIN;
          largest = -INFINITY;
          left = span;
        }
      };
      for (int v0 = row.v0; v0 < row.v1;) {
        constexpr int CHAIN = kLogChainVectors<E, MAIN>;
        static_assert(CHAIN % C::CHUNK == 0, "a chain is whole chunks");
        const int stop = LONG ? min(row.v1, v0 + CHAIN) : row.v1;
        for (; v0 < stop; v0 += C::CHUNK) {
          mbar_wait_long(&sh.full[slot], phase, &sh.abort, g_logprobs_err, ERR_LOGPROBS);
          uint64_t* empty = &sh.empty[slot];
          const uint4* chunk = ring + slot * C::CHUNK + tid;
          if (++slot == p.slots) {
            slot = 0;
            phase ^= 1u;
          }
          if (v0 + C::CHUNK <= row.v1) {
            uint4 raw[AHEAD];
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) raw[i] = chunk[i * MAIN];
            __syncwarp();
            if (lane == 0) mbar_arrive(empty);
            batch(mine.template add<E>(raw, c2));
          } else {                                                     // the row's last chunk
            int v = v0 + tid;
            if (v + (AHEAD - 1) * MAIN < row.v1) {
              uint4 raw[AHEAD];
#pragma unroll
              for (int i = 0; i < AHEAD; ++i) raw[i] = chunk[i * MAIN];
              batch(mine.template add<E>(raw, c2));
              v += AHEAD * MAIN;
            }
            if (left < span) {
              *unit = largest;
              unit += MAIN;
              largest = -INFINITY;
              left = span;
            }
            for (; v < row.v1; v += MAIN, chunk += MAIN) {
              const uint4 raw1[1] = {*chunk};
              largest = fmaxf(largest, mine.template add<E>(raw1, c2));
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(empty);
          }
        }
        if (LONG && v0 < row.v1)       // the chain ends
          mine.fold(sh.m[b][tid], sh.S[b][tid], sh.W[b][tid], stop - row.v0 > CHAIN, c2);
      }
      if (left < span) {
        *unit = largest;
        unit += MAIN;
        largest = -INFINITY;
      }
      *unit = largest;
      if (tid < row.extra) {
        const float x = E::get(row.x + row.extra_index(tid));
        if (x > mine.m) mine.raise(x, c2);
        mine.one(x, c2);
      }
      mine.fold(sh.m[b][tid], sh.S[b][tid], sh.W[b][tid], LONG && row.v1 - row.v0 > kLogChainVectors<E, MAIN>, c2);
      __syncwarp();
      if (tid % 32 == 0) mbar_arrive(&sh.ready[b]);
    }
    __syncwarp();
    if (ranks > 1) {                   // the cluster's barriers count every thread
      cluster_wait();
      cluster_sync();
    }
  } else if (tid >= MAIN + kLogRest) {
    if (lane == 0) {
      bool ok = true;
      int u = 0;                       // chunks so far
      for (int r = first_row; r < p.rows && ok; r += row_step) {
        const LogRow<E, MAIN> row(p, r, rank, ranks);
        for (int v = row.v0; v < row.v1; v += C::CHUNK, ++u) {
          // (the first round over the ring finds it empty)
          if (u >= p.slots &&
              !(ok = mbar_wait_long(&sh.empty[slot], phase ^ 1u, &sh.abort, g_logprobs_err, ERR_LOGPROBS)))
            break;
          const uint32_t bytes = (uint32_t)min(C::CHUNK, row.v1 - v) * 16u;
          mbar_arrive_expect_tx(&sh.full[slot], bytes);
          bulk_load(ring + slot * C::CHUNK, row.x + row.index(v, 0), bytes, &sh.full[slot]);
          if (++slot == p.slots) {
            slot = 0;
            phase ^= 1u;
          }
        }
      }
      if (*(volatile int*)&sh.abort)   // let copies in flight land before the CTA's shared memory goes away
        for (int i = max(u - p.slots, 0); i < u; ++i)
          mbar_wait(&sh.full[i % p.slots], (uint32_t)(i / p.slots) & 1u, nullptr, g_logprobs_err, ERR_LOGPROBS);
    }
    __syncwarp();
    if (ranks > 1) {
      cluster_wait();
      cluster_sync();
    }
  } else {
    for (int r = first_row; r < p.rows; r += row_step, ++k) {
      const LogRow<E, MAIN> row(p, r, rank, ranks);
      const int b = k & 1;
      // (after a wait that gave up the results are invalid, and reported)
      mbar_wait_long(&sh.ready[b], (uint32_t)(k / 2) & 1u, &sh.abort, g_logprobs_err, ERR_LOGPROBS);
      __syncwarp();
      row_results<E, MAIN, LONG>(p, sh, row, r, b, tid - MAIN, rank, ranks, c2, unit0 + b * p.units * MAIN);
      __syncwarp();
      if (tid % 32 == 0) mbar_arrive(&sh.done[b]);
      rest_sync();                     // what the results were made of is read: the next row's may be written
    }
  }
}

namespace {

template <typename E, int MAIN>
cudaError_t launch_logprobs(LogprobsParams& p, cudaStream_t st) {
  using C = LogCfg<MAIN>;
  // a cluster a row, or as many CTAs as fit, which take row after row
  const int sms = op_device_sms(), grid = p.cluster > 1 ? p.rows * p.cluster : std::min(p.rows, C::CTAS * sms);
  // A thread's units; the ring, what an SM's CTAs leave each other, and no more than a CTA has chunks: a small CTA starts
  // beside the kernel before (32 rows of 126464: 12.3 us, with 12 KB more of units 16.4).
  const long long vectors = p.vocab / (16 / (int)sizeof(typename E::T)) / p.cluster + 1;
  p.units = (int)std::min<long long>(kLogUnits, (vectors + MAIN - 1) / MAIN / kLogAhead) + 1;
  const int ctas = std::min(C::CTAS, (grid + sms - 1) / sms);
  const long long chunks = (vectors + C::CHUNK - 1) / C::CHUNK * ((p.rows * (long long)p.cluster + grid - 1) / grid);
  constexpr int chunk = C::CHUNK * 16, shared = (int)sizeof(LogShared<MAIN>), unit = 2 * MAIN * 4;
  const int fixed = shared + p.units * unit, room = (228 * 1024 / ctas - 1024 - fixed) / chunk;
  p.slots = (int)std::min<long long>({room, C::SLOTS, chunks});
  auto kernel = logprobs_kernel<E, MAIN, false>;
  if constexpr (MAIN > 128)            // (128 threads' rows, of 8192 vectors at most, are one chain each)
    if ((p.vocab / (16 / (int)sizeof(typename E::T)) + p.cluster - 1) / p.cluster > kLogChainVectors<E, MAIN>)
      kernel = logprobs_kernel<E, MAIN, true>;
  static_assert(MAIN > 128 || kLogChainVectors<E, MAIN> >= 8192, "a chain a row");
  const cudaError_t e = op_smem_once(reinterpret_cast<const void*>(kernel),
                                     std::min(shared + (kLogUnits + 1) * unit + C::SLOTS * chunk, 227 * 1024));
  if (e != cudaSuccess) return e;
  return op_launch(kernel, dim3((unsigned)grid), dim3(C::THREADS), (size_t)(fixed + p.slots * chunk), st, p.cluster, p);
}

// Streaming threads: few where a row is short (8192 elements are 8 vectors each of 128 threads), or where many rows of no
// more than 128 KB wait for their results: four CTAs an SM work out as many rows at once (4096 rows of bf16, 20
// alternatives: 12000 elements 58 us against 86, 32000 77 against 104, 65536 106 against 115, but 126464 187 against 173;
// 600 rows of 32000 15.4 against 18.3, 257 rows of them in float32 14.8 against 12.8).
template <typename E>
cudaError_t launch_logprobs(LogprobsParams& p, cudaStream_t st) {
  const bool many = p.rows > 2 * op_device_sms() && (long long)p.vocab * (long long)sizeof(typename E::T) <= 128 * 1024;
  return p.vocab <= 8192 || many ? launch_logprobs<E, 128>(p, st) : launch_logprobs<E, 256>(p, st);
}

}  // namespace
cudaError_t logprobs_err_word(int** p) { return cudaGetSymbolAddress(reinterpret_cast<void**>(p), g_logprobs_err); }

}  // namespace dllm

using namespace dllm;

extern "C" dllm_status dllm_op_token_logprobs(const void* logits, int64_t row_stride, int32_t dtype, int32_t rows,
                                              int32_t vocab, float inv_temperature, const int32_t* targets,
                                              float* logprobs, float* entropy, int32_t top, int32_t* top_ids,
                                              float* top_logprobs, void* stream) {
  const int es = op_dtype_size(dtype);
  if (!logits || rows < 1 || rows > kMostRows || vocab < 1 || vocab > kMostRows || es == 0 || !(inv_temperature > 0.0f) ||
      inv_temperature > 1e38f || top < 0 || top > 64 || top > vocab)
    return op_fail(DLLM_EINVAL,
                   "bad token_logprobs arguments: rows=%d vocab=%d dtype=%d inv_temperature=%g (over 0, to 1e38) top=%d "
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
  p.rows = rows;
  // CTAs of a row: as many as fill the GPU, each with 8192 elements at least
  p.cluster = 1;
  while (p.cluster < kLogCluster && (long long)rows * p.cluster * 2 <= 2LL * op_device_sms() &&
         vocab / (p.cluster * 2) >= 8192)
    p.cluster *= 2;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  switch (dtype) {
    case DLLM_F32: OP_CK(launch_logprobs<ElemF32>(p, st)); break;
    case DLLM_BF16: OP_CK(launch_logprobs<ElemBf16>(p, st)); break;
    default: OP_CK(launch_logprobs<ElemF16>(p, st)); break;
  }
  return DLLM_OK;
}
