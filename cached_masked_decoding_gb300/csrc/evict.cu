// Eviction by accumulated weight: which keys of a (sequence, cached head) stay, and their rows' copy.
//
// Weights map to 32-bit whole numbers of the same order.  One CTA takes a (sequence, head) and reads its weights once,
// into shared memory as far as they fit.  The weight of the last key that stays is found from the top: a histogram of
// 12 bits over all keys that compete, then two of 10 bits over those that agree so far, which are few and kept in a
// list.  A last walk writes the positions that stay in their order.
//
// Latency and issue slots bound the selection (20 us for 32768 keys, 9 for 4097), HBM the copy: 8 sequences of 16 to 32
// thousand keys of 8 heads of 128 in bf16 to 8192 keys: 110 us in all, 5.0 TB/s; one of 4097 to 1024: 9.5 us.  Clusters
// of four CTAs a head, with histograms added up over distributed shared memory, took 40 us for the selection alone.
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
  if (x != x) return 0;
  const uint32_t b = __float_as_uint(x + 0.0f);
  return (b >> 31) ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ int evict_len(const EvictParams& p, int s) {
  return (int)min((long long)p.src.len(p.lens, s), p.mass_rs);
}

constexpr int kEvictThreads = 1024, kEvictWarps = kEvictThreads / 32;
constexpr int kEvictMost = 49152;      // positions whose weights stay in shared memory
constexpr int kEvictList = 2048;       // keys that agree with the threshold's first bits, where they are no more
constexpr int kEvictBins = 4096;
constexpr uint32_t kEvictFixed = 0xffffffffu;   // the weight of what stays in any case

struct EvictShared {
  int hist[kEvictBins];
  uint32_t list[kEvictList];
  int warp[kEvictWarps];
  int digit, left, n_list;             // of the threshold's digit; how many of its equals stay
};

// Sum over the CTA's threads before this one, and the total.
__device__ __forceinline__ int evict_scan(int v, int* s_warp, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int upto = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, upto, d);
    if (lane >= d) upto += o;
  }
  __syncthreads();                     // (the last scan's sums are read)
  if (lane == 31) s_warp[warp] = upto;
  __syncthreads();
  int sums = s_warp[lane];             // every warp scans the warps' sums
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, sums, d);
    if (lane >= d) sums += o;
  }
  total = __shfl_sync(0xffffffffu, sums, 31);
  const int base = __shfl_sync(0xffffffffu, sums, (warp + 31) & 31);
  return (warp ? base : 0) + upto - v;
}

// From a histogram of SIZE bins: the bin from the top in which `left` of its and higher ones' keys are reached (into
// sh.digit), and how many of its own that takes (sh.left).  The bins are zeros afterwards.
template <int SIZE>
__device__ __forceinline__ void evict_digit(EvictShared& sh, int left) {
  constexpr int B = SIZE / kEvictThreads;
  __syncthreads();
  int c[B], sum = 0;
#pragma unroll
  for (int k = 0; k < B; ++k) sum += c[k] = sh.hist[SIZE - 1 - ((int)threadIdx.x * B + k)];
  int total;
  int above = evict_scan(sum, sh.warp, total);
#pragma unroll
  for (int k = 0; k < B; ++k) {
    const int b = SIZE - 1 - ((int)threadIdx.x * B + k);
    if (above < left && above + c[k] >= left) {
      sh.digit = b;
      sh.left = left - above;
    }
    above += c[k];
    sh.hist[b] = 0;
  }
  __syncthreads();
}

__global__ void __launch_bounds__(kEvictThreads) evict_select_kernel(const __grid_constant__ EvictParams p) {
  extern __shared__ __align__(16) uint32_t s_w[];   // weights by position, as far as they fit
  __shared__ EvictShared sh;
  const int tid = threadIdx.x, plane = blockIdx.x, s = plane / p.src.H_kv;
#pragma unroll
  for (int i = tid; i < kEvictBins; i += kEvictThreads) sh.hist[i] = 0;
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
  auto weight = [&](int t) {
    return t < p.cached ? s_w[t] : t < lo || t >= hi ? kEvictFixed : weight_order(mass[t]);
  };
  for (int i = tid; i < lo + n - hi; i += kEvictThreads) {
    const int t = i < lo ? i : hi + i - lo;
    if (t < held) s_w[t] = kEvictFixed;
  }
  __syncthreads();
  if (tid == 0) atomicAdd(&sh.hist[kEvictBins - 1], lo + n - hi);
  auto count = [&](int t, float x) {
    const uint32_t w = weight_order(x);
    if (t < held) s_w[t] = w;
    atomicAdd(&sh.hist[w >> 20], 1);
  };
  int t = lo + tid;
  for (; hi - t > 7 * kEvictThreads; t += 8 * kEvictThreads) {
    float x[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = mass[t + k * kEvictThreads];
#pragma unroll
    for (int k = 0; k < 8; ++k) count(t + k * kEvictThreads, x[k]);
  }
  for (; t < hi; t += kEvictThreads) count(t, mass[t]);
  int left = p.keep;
  evict_digit<4096>(sh, left);
  uint32_t bits = (uint32_t)sh.digit << 20;         // the last kept one's weight
  left = sh.left;                                   // how many of those that agree stay
  // Those that agree; a list holds them where they are few.
  auto agree = [&](uint32_t w) {
    if ((w >> 20) == (bits >> 20) && *(volatile int*)&sh.n_list <= kEvictList) {
      const int at = atomicAdd(&sh.n_list, 1);
      if (at < kEvictList) sh.list[at] = w;
    }
  };
  for (int f = 4 * tid; f < held; f += 4 * kEvictThreads) {
    const uint4 w = *reinterpret_cast<const uint4*>(s_w + f);   // (past held: of no account)
    agree(w.x);
    if (f + 1 < held) agree(w.y);
    if (f + 2 < held) agree(w.z);
    if (f + 3 < held) agree(w.w);
  }
  for (int f = held + tid; f < n; f += kEvictThreads) agree(weight(f));
  __syncthreads();
  const int n_list = sh.n_list;
  const bool listed = n_list <= kEvictList;
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    const int shift = pass == 0 ? 10 : 0, up = shift + 10;
    for (int i = tid; i < (listed ? n_list : n); i += kEvictThreads) {
      const uint32_t w = listed ? sh.list[i] : weight(i);
      if ((w >> up) == (bits >> up)) atomicAdd(&sh.hist[(w >> shift) & 1023], 1);
    }
    evict_digit<1024>(sh, left);
    bits |= (uint32_t)sh.digit << shift;
    left = sh.left;
  }
  // the kept positions, in order: every thread takes a run of 8
  constexpr int RUN = 8;
  int stays_before = 0, equals_before = 0;
  for (long long b0 = 0; b0 < n; b0 += RUN * kEvictThreads) {
    const int f = (int)b0 + tid * RUN;
    uint32_t above = 0, equal = 0;
    if (f <= held - RUN) {
      const uint4 a = reinterpret_cast<const uint4*>(s_w + f)[0], c = reinterpret_cast<const uint4*>(s_w + f)[1];
      const uint32_t w[RUN] = {a.x, a.y, a.z, a.w, c.x, c.y, c.z, c.w};
#pragma unroll
      for (int k = 0; k < RUN; ++k) {
        above |= w[k] > bits ? 1u << k : 0;
        equal |= w[k] == bits ? 1u << k : 0;
      }
    } else {
      for (int k = 0; k < RUN && k < n - f; ++k) {
        const uint32_t w = weight(f + k);
        above |= w > bits ? 1u << k : 0;
        equal |= w == bits ? 1u << k : 0;
      }
    }
    // both counts in one scan (16 bits each hold RUN * threads)
    int total;
    const int base = evict_scan(__popc(above) | __popc(equal) << 16, sh.warp, total);
    const int eq = equals_before + (base >> 16);
    int at = stays_before + (base & 0xffff) + min(eq, left);
    // of the run's equals, those that there is room for
    uint32_t room = equal;
    for (int over = __popc(equal) - max(left - eq, 0); over > 0 && room; --over) room &= ~(1u << (31 - __clz(room)));
    for (uint32_t stay = above | room; stay; stay &= stay - 1) kept[at++] = f + __ffs(stay) - 1;
    stays_before += total & 0xffff;
    equals_before += total >> 16;
  }
}

// Copies kept positions' K and V: a group of HD / 8 lanes a row of both.  As many warps as fit keep HBM busy, at one row
// a thread: 8 x 8192 rows of 8 heads of 128 with the selection 108 us, two rows in flight 113, four 117, eight 132.
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
  p.cached = (int)std::min<long long>((std::min(p.src.positions, p.mass_rs) + 7) / 8 * 8, kEvictMost);
  OP_CK(op_smem_once(reinterpret_cast<const void*>(evict_select_kernel), kEvictMost * 4));
  OP_CK(op_launch(evict_select_kernel, dim3((unsigned)planes), dim3(kEvictThreads), (size_t)p.cached * 4, st, 1, p));
  OP_CK(src->hd == 64 ? launch_evict_copy<64>(p, planes, st) : launch_evict_copy<128>(p, planes, st));
  return DLLM_OK;
}
