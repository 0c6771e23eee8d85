// Eviction by accumulated weight: which keys of a (sequence, cached head) stay, and their rows' copy.
//
// Weights map to 32-bit whole numbers of the same order.  A cluster takes the positions of a (sequence, head) between
// its CTAs, each reads its share once into shared memory; the weight of the last key that stays is found by three
// histograms of 11, 11 and 10 bits from the top, of the keys that agree in the bits above, added up over the cluster.
// Then every CTA knows how many keys stay, and how many equals, before its share, and writes its part of the kept
// positions in their order.
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
  int cluster, cached;                 // CTAs of a (sequence, head); weights a CTA holds in shared memory
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

constexpr int kEvictThreads = 512, kEvictWarps = kEvictThreads / 32;
constexpr int kEvictMost = 40960;      // positions of a CTA whose weights stay in shared memory
constexpr int kEvictCluster = 8;

struct EvictShared {
  int hist[2048];
  int warp[kEvictWarps];
  int digit, left;                     // of the threshold's digit; how many of its equals stay
  int counts[kEvictCluster][2];        // of every CTA: keys that stay, and equals of the threshold
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
  int base = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kEvictWarps; ++w) {
    const int o = s_warp[w];
    base += w < warp ? o : 0;
    total += o;
  }
  return base + upto - v;
}

__global__ void __launch_bounds__(kEvictThreads) evict_select_kernel(const __grid_constant__ EvictParams p) {
  extern __shared__ uint32_t s_w[];    // the share's weights, as far as they fit
  __shared__ EvictShared sh;
  const int ranks = p.cluster, rank = ranks > 1 ? (int)cluster_rank() : 0, tid = threadIdx.x;
  const int plane = (int)(blockIdx.x / (unsigned)ranks), s = plane / p.src.H_kv;
  griddep_launch_dependents();
  griddep_wait();
  const int n = evict_len(p, s), m = min(n, p.keep);
  const float* mass = p.mass + plane * p.mass_rs;
  int32_t* kept = p.kept + (long long)plane * p.keep;
  if (rank == 0 && tid == 0 && plane % p.src.H_kv == 0) p.new_lens[s] = m;
  for (int i = m + rank * kEvictThreads + tid; i < p.keep; i += ranks * kEvictThreads) kept[i] = -1;
  if (n <= p.keep) {
    for (int i = rank * kEvictThreads + tid; i < n; i += ranks * kEvictThreads) kept[i] = i;
    return;                            // (all of the cluster)
  }
  for (int i = tid; i < 2048; i += kEvictThreads) sh.hist[i] = 0;
  if (ranks > 1) cluster_arrive();     // waited for before the first access of another CTA's memory
  // the positions that compete, and this CTA's share of all
  const int lo = p.sinks, hi = n - p.recent;
  int left = p.keep - p.sinks - p.recent;
  const int t0 = (int)((long long)n * rank / ranks), t1 = (int)((long long)n * (rank + 1) / ranks);
  const int c0 = min(max(t0, lo), t1), c1 = max(min(t1, hi), c0);
  auto weight = [&](int t) {
    const int at = t - c0;
    return at < p.cached ? s_w[at] : weight_order(mass[t]);
  };
  uint32_t bits = 0;                   // the last kept one's weight
  bool waited = ranks == 1;
  __syncthreads();
  if (left > 0) {
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, size = pass == 2 ? 1024 : 2048;
      if (pass == 0) {
        // the share, four loads in flight
        for (int t = c0 + tid; t < c1; t += 4 * kEvictThreads) {
          float x[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) x[k] = t + k * kEvictThreads < c1 ? mass[t + k * kEvictThreads] : 0.0f;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int at = t + k * kEvictThreads - c0;
            if (at >= c1 - c0) break;
            const uint32_t w = weight_order(x[k]);
            if (at < p.cached) s_w[at] = w;
            atomicAdd(&sh.hist[w >> 21], 1);
          }
        }
      } else {
        const int up = pass == 1 ? 21 : 10;
        for (int t = c0 + tid; t < c1; t += kEvictThreads) {
          const uint32_t w = weight(t);
          if ((w >> up) == (bits >> up)) atomicAdd(&sh.hist[(w >> shift) & (size - 1)], 1);
        }
      }
      __syncthreads();
      constexpr int B = 2048 / kEvictThreads;            // bins of a thread, from the top
      int c[B], sum = 0;
      if (ranks > 1) {
        if (!waited) cluster_wait();
        if (!waited) waited = true;
        cluster_sync();                                  // every CTA's histogram is whole
        for (int k = 0; k < B; ++k) c[k] = 0;
        for (int r = 0; r < ranks; ++r)
#pragma unroll
          for (int k = 0; k < B; ++k) {
            const int b = size - 1 - (tid * B + k);
            if (b >= 0) c[k] += cluster_load(cluster_addr(smem_u32(&sh.hist[b]), (uint32_t)r));
          }
      } else {
#pragma unroll
        for (int k = 0; k < B; ++k) {
          const int b = size - 1 - (tid * B + k);
          c[k] = b >= 0 ? sh.hist[b] : 0;
        }
      }
#pragma unroll
      for (int k = 0; k < B; ++k) sum += c[k];
      int total;
      int above = evict_scan(sum, sh.warp, total);       // keys in higher bins
#pragma unroll
      for (int k = 0; k < B; ++k) {
        if (above < left && above + c[k] >= left) {
          sh.digit = size - 1 - (tid * B + k);
          sh.left = left - above;
        }
        above += c[k];
      }
      if (ranks > 1) cluster_sync();                     // the histograms are read
      __syncthreads();
      bits |= (uint32_t)sh.digit << shift;
      left = sh.left;
      for (int i = tid; i < 2048; i += kEvictThreads) sh.hist[i] = 0;
      __syncthreads();
    }
  }
  const bool some = p.keep > p.sinks + p.recent;         // some of those that compete stay
  auto kind = [&](int t) {             // 2: stays, 1: an equal of the last one that does
    if (t < lo || t >= hi) return 2;
    const uint32_t w = some ? weight(t) : 0;
    return !some ? 0 : w > bits ? 2 : w == bits ? 1 : 0;
  };
  // what the CTAs before this one keep
  int stay = 0, equal = 0, stays_before = 0, equals_before = 0;
  if (ranks > 1) {
    for (int t = t0 + tid; t < t1; t += kEvictThreads) {
      const int k = kind(t);
      stay += k >> 1;
      equal += k & 1;
    }
    int stay_all, equal_all;
    evict_scan(stay, sh.warp, stay_all);
    evict_scan(equal, sh.warp, equal_all);
    if (!waited) cluster_wait();
    if (tid < ranks) {
      cluster_store_int(cluster_addr(smem_u32(&sh.counts[rank][0]), (uint32_t)tid), stay_all);
      cluster_store_int(cluster_addr(smem_u32(&sh.counts[rank][1]), (uint32_t)tid), equal_all);
    }
    cluster_sync();
    for (int r = 0; r < rank; ++r) {
      stays_before += sh.counts[r][0];
      equals_before += sh.counts[r][1];
    }
  }
  // the kept positions, in order: every thread takes a run
  constexpr int RUN = 8;
  for (int b0 = t0; b0 < t1; b0 += RUN * kEvictThreads) {
    const int f = b0 + tid * RUN;
    uint32_t two = 0, one = 0;
#pragma unroll
    for (int k = 0; k < RUN; ++k) {
      const int x = f + k < t1 ? kind(f + k) : 0;
      two |= (uint32_t)(x >> 1) << k;
      one |= (uint32_t)(x & 1) << k;
    }
    // equals stay while there is room: both counts in one scan (16 bits each hold RUN * threads)
    int total;
    const int base = evict_scan(__popc(two) | __popc(one) << 16, sh.warp, total);
    int eq = equals_before + (base >> 16);
    int at = stays_before + (base & 0xffff) + min(eq, left);
#pragma unroll
    for (int k = 0; k < RUN; ++k) {
      const bool e = (one >> k) & 1;
      if ((two >> k) & 1 || (e && eq < left)) kept[at++] = f + k;
      eq += e ? 1 : 0;
    }
    stays_before += total & 0xffff;
    equals_before += total >> 16;
  }
}

// Copies kept positions' K and V: a group of HD / 8 lanes a row, ROWS rows in flight.
template <int HD, int ROWS>
__global__ void __launch_bounds__(256) evict_copy_kernel(const __grid_constant__ EvictParams p) {
  constexpr int L = HD / 8, PER = 256 / L;
  const int l = threadIdx.x % L, group = threadIdx.x / L;
  uint32_t chunk;
  const int plane = (int)p.by_chunks.divmod(blockIdx.x, chunk), s = plane / p.src.H_kv, g = plane % p.src.H_kv;
  griddep_launch_dependents();
  griddep_wait();
  const int m = min(evict_len(p, s), p.keep), i0 = (int)chunk * (ROWS * PER) + group;
  if (i0 >= m) return;
  long long from[ROWS], to[ROWS];
  int t[ROWS];
#pragma unroll
  for (int k = 0; k < ROWS; ++k) t[k] = p.kept[(long long)plane * p.keep + min(i0 + k * PER, m - 1)];
#pragma unroll
  for (int k = 0; k < ROWS; ++k) {
    const int i = i0 + k * PER;
    from[k] = p.src.row(s, g, t[k]);
    to[k] = i < m ? p.dst.row(s, g, i) : -1;
  }
  uint4 kv[2][ROWS];
#pragma unroll
  for (int k = 0; k < ROWS; ++k) {
    kv[0][k] = kv[1][k] = make_uint4(0, 0, 0, 0);
    if (from[k] >= 0) {
      kv[0][k] = reinterpret_cast<const uint4*>(p.src.k + from[k])[l];
      kv[1][k] = reinterpret_cast<const uint4*>(p.src.v + from[k])[l];
    }
  }
  if (p.mass_out && l == 0) {
#pragma unroll
    for (int k = 0; k < ROWS; ++k)
      if (i0 + k * PER < m) p.mass_out[plane * p.mass_out_rs + i0 + k * PER] = p.mass[plane * p.mass_rs + t[k]];
  }
#pragma unroll
  for (int k = 0; k < ROWS; ++k)
    if (to[k] >= 0) {
      reinterpret_cast<uint4*>(p.dst.k + to[k])[l] = kv[0][k];
      reinterpret_cast<uint4*>(p.dst.v + to[k])[l] = kv[1][k];
    }
}

namespace {

template <int HD>
cudaError_t launch_evict_copy(EvictParams& p, long long planes, cudaStream_t st) {
  constexpr int ROWS = 4, rows = ROWS * 256 / (HD / 8);
  p.by_chunks = FastDiv((uint32_t)((p.keep + rows - 1) / rows));
  return op_launch(evict_copy_kernel<HD, ROWS>, dim3((unsigned)(planes * p.by_chunks.d)), dim3(256), 0, st, 1, p);
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
  const long long planes = (long long)src->b * src->H_kv;
  if (planes > 0x7fffffff / kEvictCluster || (double)planes * ((keep + 63) / 64) > 0x7fffffff)
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
  // CTAs of a (sequence, head): 4096 positions each, as far as that fills the GPU; more where they do not fit in shared memory
  const long long most = std::min(p.src.positions, p.mass_rs);
  p.cluster = 1;
  while (p.cluster < kEvictCluster && most > 4096LL * p.cluster &&
         (planes * p.cluster * 2 <= 2LL * op_device_sms() || most > (long long)kEvictMost * p.cluster))
    p.cluster *= 2;
  const long long share = (most + p.cluster - 1) / p.cluster;
  p.cached = (int)std::min<long long>(share, kEvictMost);
  const int smem = (p.cached + 3) / 4 * 16;
  OP_CK(op_smem_once(reinterpret_cast<const void*>(evict_select_kernel), kEvictMost * 4));
  OP_CK(op_launch(evict_select_kernel, dim3((unsigned)(planes * p.cluster)), dim3(kEvictThreads), (size_t)smem, st,
                  p.cluster, p));
  OP_CK(src->hd == 64 ? launch_evict_copy<64>(p, planes, st) : launch_evict_copy<128>(p, planes, st));
  return DLLM_OK;
}
