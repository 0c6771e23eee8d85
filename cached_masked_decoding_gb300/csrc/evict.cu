// Eviction by accumulated weight: which keys of a (sequence, cached head) stay, and their rows' copy.
//
// Weights map to 32-bit whole numbers of the same order.  One CTA takes a (sequence, head) and reads its weights once,
// into shared memory as far as they fit.  The weight of the last key that stays is found from the top: a histogram of
// 12 bits over all keys that compete, then those that agree so far, which are few and kept in a list, are compared one by
// one, or counted by two digits of 10 bits.  A last walk writes the positions that stay in their order: where all of the
// threshold's weight stay, a warp packs its run of positions in place and writes it out; else it counts first.
//
// Latency and issue slots bound the selection (alone 11.8 us for 32768 keys of 8 heads, 5.2 for 4097), HBM the copy: 8 sequences of 16 to 32
// thousand keys of 8 heads of 128 in bf16 to 8192 keys: 104 us in all, 5.3 TB/s; one of 4097 to 1024: 7.6 us.  Clusters
// of four CTAs a head, with histograms added up over distributed shared memory, took 40 us for the selection alone; the
// first histogram in two copies, lanes in turn, nothing less; loops rolled up 107 us.
#include <algorithm>

#include "kv_paged.h"
#include "ptx8.cuh"

namespace dllm {

struct EvictParams {
  PagedKv src, dst;
  const float* mass;
  float* mass_out;
  const int32_t* lens;
  int32_t *kept, *new_lens;
  long long mass_rs, mass_out_rs;
  int keep, sinks, recent;
  int cached;                          // weights held in shared memory
  FastDiv by_chunks;                   // by the CTAs that copy one's rows
};

// Weights as whole numbers of their order; a NaN is the least, -0 is 0.
__device__ __forceinline__ uint32_t weight_order(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f), o = b ^ ((uint32_t)((int)b >> 31) | 0x80000000u);
  return x == x ? o : 0;
}

__device__ __forceinline__ int evict_len(const EvictParams& p, int s) {
  return (int)min((long long)p.src.len(p.lens, s), p.mass_rs);
}

constexpr int kEvictThreads = 1024, kEvictWarps = kEvictThreads / 32;
constexpr int kEvictStep = 8 * kEvictThreads;   // (32 runs of 256 positions)
constexpr int kEvictMost = 6 * kEvictStep;      // positions whose weights stay in shared memory
constexpr int kEvictList = 2048;       // keys that agree with the threshold's first bits, where they are no more
constexpr int kEvictBins = 4096;
// keys of the list that are compared one by one, more by digits (none, 128, 512: 4097 keys of 8 heads 8.15, 7.57, 7.61
// us; 1000 keys 6.74, 5.85, 5.80; 16000 of hd 64 10.5, 10.4, 11.1; the batch above 104, 104, 110)
constexpr int kEvictDirect = 128;
constexpr uint32_t kEvictFixed = 0xffffffffu;   // the weight of what stays in any case

struct EvictShared {
  alignas(16) int hist[kEvictBins];
  alignas(16) uint32_t list[kEvictList];
  int warp[kEvictWarps], equal[kEvictWarps];
  int digit, left, same, n_list;       // of the threshold's digit; how many of its keys stay, of how many
  uint32_t bits;
};

// From a histogram of SIZE bins: the bin from the top in which `left` of its and higher ones' keys are reached (into
// sh.digit), how many of its own that takes (sh.left) and how many it has.  The bins are zeros afterwards.
template <int SIZE>
__device__ __forceinline__ void evict_digit(EvictShared& sh, int left) {
  constexpr int B = SIZE / kEvictThreads;
  static_assert(B == 1 || B == 4, "a thread's bins");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, first = SIZE - B * ((int)threadIdx.x + 1);
  __syncthreads();
  int c[B];                            // from the top
  if constexpr (B == 4) {
    int4* at = reinterpret_cast<int4*>(&sh.hist[first]);
    const int4 h = *at;
    c[0] = h.w;
    c[1] = h.z;
    c[2] = h.y;
    c[3] = h.x;
    *at = make_int4(0, 0, 0, 0);
  } else {
    c[0] = sh.hist[first];
    sh.hist[first] = 0;
  }
  int sum = 0;
#pragma unroll
  for (int k = 0; k < B; ++k) sum += c[k];
  const int total = (int)__reduce_add_sync(0xffffffffu, (uint32_t)sum);
  if (lane == 0) sh.warp[warp] = total;
  __syncthreads();
  int above = (int)__reduce_add_sync(0xffffffffu, lane < warp ? (uint32_t)sh.warp[lane] : 0u);
  if (above < left && above + total >= left) {   // one warp's
    int upto = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, upto, d);
      if (lane >= d) upto += o;
    }
    above += upto - sum;
#pragma unroll
    for (int k = 0; k < B; ++k) {
      if (above < left && above + c[k] >= left) {
        sh.digit = first + B - 1 - k;
        sh.left = left - above;
        sh.same = c[k];
      }
      above += c[k];
    }
  }
  __syncthreads();
}

// What follows the first digit, of the last kept one's weight `bits` and of those that agree `left` that stay: the rest of
// it, and the kept positions.  HELD: all weights are in shared memory, with zeros behind them.
template <bool HELD>
__device__ __forceinline__ void evict_last(const EvictParams& p, EvictShared& sh, uint32_t* s_w, const float* mass,
                                           int32_t* kept, int n, uint32_t bits, int left) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, lo = p.sinks, hi = n - p.recent;
  auto weight = [&](int t) {
    return HELD || t < p.cached ? s_w[t] : t < lo || t >= hi ? kEvictFixed : weight_order(mass[t]);
  };
  // four positions' weights and how many of them there are
  auto four = [&](int f, uint32_t (&w)[4]) {
    if (HELD || f + 4LL <= p.cached) {
      const uint4 v = *reinterpret_cast<const uint4*>(s_w + f);
      w[0] = v.x;
      w[1] = v.y;
      w[2] = v.z;
      w[3] = v.w;
      return 4;
    }
    const int there = max(min(n - f, 4), 0);
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = k < there ? weight(f + k) : 0;
    return there;
  };
  // Those that agree; a list holds them where they are few.  A thread looks at 32 before it asks for places.
  for (long long b0 = 0; b0 < n; b0 += 32 * kEvictThreads) {
    uint32_t mask = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const long long at = b0 + k * 4 * kEvictThreads;
      if (at >= n) break;
      uint32_t w[4];
      const int there = four((int)at + 4 * tid, w);
#pragma unroll
      for (int e = 0; e < 4; ++e) mask |= e < there && (w[e] ^ bits) < 1u << 20 ? 1u << (4 * k + e) : 0;
    }
    if (!__any_sync(0xffffffffu, mask != 0)) continue;
    int upto = __popc(mask);
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, upto, d);
      if (lane >= d) upto += o;
    }
    int to = 0;
    if (lane == 31) to = *(volatile int*)&sh.n_list <= kEvictList ? atomicAdd(&sh.n_list, upto) : kEvictList;
    to = __shfl_sync(0xffffffffu, to, 31) + upto - __popc(mask);
    for (; mask && to < kEvictList; mask &= mask - 1, ++to) {
      const int bit = __ffs(mask) - 1;
      sh.list[to] = weight((int)b0 + (bit >> 2) * 4 * kEvictThreads + 4 * tid + (bit & 3));
    }
  }
  __syncthreads();
  const int n_list = sh.n_list;
  if (n_list <= kEvictDirect) {        // few: the one that fewer than `left` exceed, and no fewer with its equals
    if (tid < n_list) {
      const uint32_t w = sh.list[tid];
      int more = 0, same = 0;
      for (int i = 0; i < n_list; i += 4) {
        const uint4 x = *reinterpret_cast<const uint4*>(&sh.list[i]);
        more += x.x > w;
        same += x.x == w;
        more += i + 1 < n_list && x.y > w;
        same += i + 1 < n_list && x.y == w;
        more += i + 2 < n_list && x.z > w;
        same += i + 2 < n_list && x.z == w;
        more += i + 3 < n_list && x.w > w;
        same += i + 3 < n_list && x.w == w;
      }
      if (more < left && more + same >= left) {
        sh.bits = w;
        sh.left = left - more;
        sh.same = same;
      }
    }
    __syncthreads();
    bits = sh.bits;
    left = sh.left;
  } else {
    const bool listed = n_list <= kEvictList;
#pragma unroll 1
    for (int shift = 10; shift >= 0; shift -= 10) {
      for (int i = tid; i < (listed ? n_list : n); i += kEvictThreads) {
        const uint32_t w = listed ? sh.list[i] : weight(i);
        if ((w >> (shift + 10)) == (bits >> (shift + 10))) atomicAdd(&sh.hist[(w >> shift) & 1023], 1);
      }
      evict_digit<1024>(sh, left);
      bits |= (uint32_t)sh.digit << shift;
      left = sh.left;
    }
  }
  // The kept positions, in order, a run a warp.
  const int run = (int)((n + kEvictStep - 1LL) / kEvictStep * 256), f0 = warp * run, f1 = (int)min((long long)f0 + run, (long long)n);
  int stays = 0, equals = 0;
  if (HELD && sh.same == left && bits != 0) {
    // All of the threshold's weight stay: the run's positions take the place of its weights, then go to theirs.
    uint32_t* own = s_w + f0;
#pragma unroll 2
    for (int f = 0; f < f1 - f0; f += 256) {
      const uint4* at = reinterpret_cast<const uint4*>(own + f + 8 * lane);
      const uint4 a = at[0], c = at[1];
      const uint32_t w[8] = {a.x, a.y, a.z, a.w, c.x, c.y, c.z, c.w};
      int mine = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) mine += w[k] >= bits ? 1 : 0;
      int upto = mine;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, upto, d);
        if (lane >= d) upto += o;
      }
      // (no further than weights that this and the lanes before have read)
      uint32_t* to = own + stays + upto - mine;
      const uint32_t t = (uint32_t)(f0 + f + 8 * lane);
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (w[k] >= bits) *to++ = t + k;
      stays += __shfl_sync(0xffffffffu, upto, 31);
    }
    if (lane == 0) sh.warp[warp] = stays;
    __syncthreads();
    const int base = (int)__reduce_add_sync(0xffffffffu, lane < warp ? (uint32_t)sh.warp[lane] : 0u);
    for (int i = lane; i < stays; i += 32) kept[base + i] = (int32_t)own[i];
    return;
  }
  // Else a warp counts, and with the counts of the warps before writes its own.
#pragma unroll 2
  for (int f = f0; f < f1; f += 128) {
    uint32_t w[4];
    const int there = four(f + 4 * lane, w);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      stays += k < there && w[k] > bits;
      equals += k < there && w[k] == bits;
    }
  }
  stays = (int)__reduce_add_sync(0xffffffffu, (uint32_t)stays);
  equals = (int)__reduce_add_sync(0xffffffffu, (uint32_t)equals);
  if (lane == 0) {
    sh.warp[warp] = stays;
    sh.equal[warp] = equals;
  }
  __syncthreads();
  stays = (int)__reduce_add_sync(0xffffffffu, lane < warp ? (uint32_t)sh.warp[lane] : 0u);
  equals = (int)__reduce_add_sync(0xffffffffu, lane < warp ? (uint32_t)sh.equal[lane] : 0u);
#pragma unroll 2
  for (int f = f0; f < f1; f += 128) {
    uint32_t w[4];
    const int t = f + 4 * lane, there = four(t, w);
    bool stay[4], same[4];
    int own = 0;                       // that stay, and of equals in the upper half
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      stay[k] = k < there && w[k] > bits;
      same[k] = k < there && w[k] == bits;
      own += (stay[k] ? 1 : 0) + (same[k] ? 0x10000 : 0);
    }
    int upto = own;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, upto, d);
      if (lane >= d) upto += o;
    }
    const int total = __shfl_sync(0xffffffffu, upto, 31), own_before = upto - own;
    int eq = equals + (own_before >> 16), at = stays + (own_before & 0xffff) + min(eq, left);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const bool stays_too = stay[k] || (same[k] && eq < left);   // of the equals, those that there is room for
      if (stays_too) kept[at] = t + k;
      at += stays_too ? 1 : 0;
      eq += same[k] ? 1 : 0;
    }
    stays += total & 0xffff;
    equals += total >> 16;
  }
}

__global__ void __launch_bounds__(kEvictThreads) evict_select_kernel(const __grid_constant__ EvictParams p) {
  extern __shared__ __align__(16) uint32_t s_w[];   // weights by position, as far as they fit
  __shared__ EvictShared sh;
  const int tid = threadIdx.x, plane = blockIdx.x, s = plane / p.src.H_kv;
  static_assert(kEvictBins == 4 * kEvictThreads, "four bins a thread");
  reinterpret_cast<int4*>(sh.hist)[tid] = make_int4(0, 0, 0, 0);
  if (tid == 0) sh.n_list = 0;
  griddep_launch_dependents();
  griddep_wait();
  const int n = evict_len(p, s), m = min(n, p.keep);
  const float* mass = p.mass + plane * p.mass_rs;
  int32_t* kept = p.kept + (long long)plane * p.keep;
  if (tid == 0 && plane % p.src.H_kv == 0) p.new_lens[s] = m;
  for (int i = m + tid; i < p.keep; i += kEvictThreads) kept[i] = -1;
  if (n <= p.keep) {
    for (int i = tid; i < n; i += kEvictThreads) kept[i] = i;
    return;
  }
  // Those that stay whatever their weight count as heavier than all others; then keep of n stay.
  const int lo = p.sinks, hi = n - p.recent, held = min(n, p.cached);
  for (int i = tid; i < lo + n - hi; i += kEvictThreads) {
    const int t = i < lo ? i : hi + i - lo;
    if (t < held) s_w[t] = kEvictFixed;
  }
  __syncthreads();
  if (tid == 0) atomicAdd(&sh.hist[kEvictBins - 1], lo + n - hi);
  constexpr int DEEP = 16;
  uint32_t t = lo + tid;
  if (n <= p.cached)
    for (; (int)t + (DEEP - 1) * kEvictThreads < hi; t += DEEP * kEvictThreads) {   // whole batches, all held
      float x[DEEP];
#pragma unroll
      for (int k = 0; k < DEEP; ++k) x[k] = mass[t + k * kEvictThreads];
#pragma unroll
      for (int k = 0; k < DEEP; ++k) {
        const uint32_t w = weight_order(x[k]);
        s_w[t + k * kEvictThreads] = w;
        atomicAdd(&sh.hist[w >> 20], 1);
      }
    }
  for (; t < (uint32_t)hi; t += DEEP * kEvictThreads) {
    const int room = (hi - (int)t + kEvictThreads - 1) / kEvictThreads;   // of the batch, those that there are
    float x[DEEP];
#pragma unroll
    for (int k = 0; k < DEEP; ++k) x[k] = k < room ? mass[t + k * kEvictThreads] : 0.0f;
#pragma unroll
    for (int k = 0; k < DEEP; ++k) {
      if (k >= room) break;
      const uint32_t w = weight_order(x[k]), at = t + k * kEvictThreads;
      if (at < (uint32_t)held) s_w[at] = w;
      atomicAdd(&sh.hist[w >> 20], 1);
    }
  }
  // (what lies behind the last position up to where it is looked at: the least weight, which never finds room)
  for (int t = n + tid; n <= p.cached && t < (n + kEvictStep - 1) / kEvictStep * kEvictStep; t += kEvictThreads) s_w[t] = 0;
  evict_digit<kEvictBins>(sh, p.keep);
  const uint32_t bits = (uint32_t)sh.digit << 20;   // the last kept one's weight
  const int left = sh.left;                         // how many of those that agree stay
  if (n <= p.cached)
    evict_last<true>(p, sh, s_w, mass, kept, n, bits, left);
  else
    evict_last<false>(p, sh, s_w, mass, kept, n, bits, left);
}

// Copies kept positions' K and V: a group of HD / 8 lanes a row of both.  As many warps as fit keep HBM busy, at one row
// a thread: 8 x 8192 rows of 8 heads of 128 with the selection of then 108 us, two rows in flight 113, four 117, eight 132.
template <int HD>
__global__ void __launch_bounds__(256, 8) evict_copy_kernel(const __grid_constant__ EvictParams p) {
  constexpr int L = HD / 8, PER = 256 / L;
  const int l = threadIdx.x % L;
  uint32_t chunk;
  const int plane = (int)p.by_chunks.divmod(blockIdx.x, chunk), s = plane / p.src.H_kv, g = plane - s * p.src.H_kv;
  griddep_launch_dependents();
  griddep_wait();
  const int m = min(evict_len(p, s), p.keep), i = (int)(chunk * PER + threadIdx.x / L);
  if (i >= m) return;
  const int t = p.kept[(long long)plane * p.keep + i];
  const long long from = p.src.row(s, g, t), to = p.dst.row(s, g, i);
  uint4 k = make_uint4(0, 0, 0, 0), v = k;
  if (from >= 0) {
    k = __ldcs(reinterpret_cast<const uint4*>(p.src.k + from) + l);
    v = __ldcs(reinterpret_cast<const uint4*>(p.src.v + from) + l);
  }
  if (p.mass_out && l == 0) p.mass_out[plane * p.mass_out_rs + i] = p.mass[plane * p.mass_rs + t];
  if (to >= 0) {
    __stcs(reinterpret_cast<uint4*>(p.dst.k + to) + l, k);
    __stcs(reinterpret_cast<uint4*>(p.dst.v + to) + l, v);
  }
}

namespace {

template <int HD>
cudaError_t launch_evict_copy(EvictParams& p, long long planes, cudaStream_t st) {
  constexpr int PER = 256 / (HD / 8);
  p.by_chunks = FastDiv((uint32_t)((p.keep + PER - 1) / PER));
  return op_launch(evict_copy_kernel<HD>, dim3((unsigned)(planes * p.by_chunks.d)), dim3(256), 0, st, 1, p);
}

}  // namespace
}  // namespace dllm

using namespace dllm;

extern "C" dllm_status dllm_op_kv_paged_evict(const dllm_kv_paged* src, const dllm_kv_paged* dst, const float* mass,
                                              int64_t mass_stride, const int32_t* lens, int32_t keep, int32_t sinks,
                                              int32_t recent, int32_t* kept, int32_t* new_lens, float* mass_out,
                                              int64_t mass_out_stride, void* stream) {
  if (const dllm_status s = kv_paged_check(src, "kv_paged_evict"); s != DLLM_OK) return s;
  if (const dllm_status s = kv_paged_check(dst, "kv_paged_evict"); s != DLLM_OK) return s;
  if (src->b != dst->b || src->H_kv != dst->H_kv || src->hd != dst->hd || src->dtype != dst->dtype)
    return op_fail(DLLM_EINVAL, "kv_paged_evict: the caches differ in b, H_kv, hd or dtype");
  if (src->k == dst->k && src->table == dst->table)
    return op_fail(DLLM_EINVAL, "kv_paged_evict: dst is src: the kept rows go to pages of their own");
  EvictParams p = {};
  p.src = PagedKv(*src);
  p.dst = PagedKv(*dst);
  if (!mass || !kept || !new_lens || keep < 1 || sinks < 0 || recent < 0 || (int64_t)sinks + recent > keep ||
      keep > p.dst.positions || !op_aligned(mass, 4) || !op_aligned(kept, 4) || !op_aligned(new_lens, 4) ||
      !op_aligned(lens, 4) || !op_aligned(mass_out, 4))
    return op_fail(DLLM_EINVAL, "bad kv_paged_evict arguments: keep=%d (sinks + recent to %lld) sinks=%d recent=%d", keep,
                   p.dst.positions, sinks, recent);
  p.mass_rs = mass_stride ? mass_stride : p.src.positions;
  p.mass_out_rs = mass_out_stride ? mass_out_stride : keep;
  if (p.mass_rs < 1 || p.mass_rs > (1LL << 40) || (mass_out && (p.mass_out_rs < keep || p.mass_out_rs > (1LL << 40))))
    return op_fail(DLLM_EINVAL, "kv_paged_evict: bad strides: mass %lld, mass_out %lld (at least keep=%d)", p.mass_rs,
                   p.mass_out_rs, keep);
  if ((const void*)mass == mass_out) return op_fail(DLLM_EINVAL, "kv_paged_evict: mass_out is mass");
  if (lens && lens == new_lens)   // (CTAs read lens while one writes m)
    return op_fail(DLLM_EINVAL, "kv_paged_evict: new_lens is lens");
  const long long planes = (long long)src->b * src->H_kv;
  if (planes > 0x7fffffff || (double)planes * ((keep + 15) / 16) > 0x7fffffff)
    return op_fail(DLLM_EINVAL, "kv_paged_evict: b=%d H_kv=%d keep=%d are too many for one call", src->b, src->H_kv, keep);
  p.mass = mass;
  p.mass_out = mass_out;
  p.lens = lens;
  p.kept = kept;
  p.new_lens = new_lens;
  p.keep = keep;
  p.sinks = sinks;
  p.recent = recent;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  p.cached = (int)std::min<long long>((std::min(p.src.positions, p.mass_rs) + kEvictStep - 1) / kEvictStep * kEvictStep, kEvictMost);
  OP_CK(op_smem_once(reinterpret_cast<const void*>(evict_select_kernel), kEvictMost * 4));
  OP_CK(op_launch(evict_select_kernel, dim3((unsigned)planes), dim3(kEvictThreads), (size_t)p.cached * 4, st, 1, p));
  OP_CK(src->hd == 64 ? launch_evict_copy<64>(p, planes, st) : launch_evict_copy<128>(p, planes, st));
  return DLLM_OK;
}
