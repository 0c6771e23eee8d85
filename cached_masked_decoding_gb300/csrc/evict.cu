// Eviction by accumulated weight: which keys of a (sequence, cached head) stay, and their rows' copy.
//
// Weights map to 32-bit whole numbers of the same order.  The weight of the last key that stays is found by
// four passes over the positions, eight bits each from the top (a histogram of the keys that agree in the
// bits above); one more pass writes the positions kept in their order.
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

__global__ void __launch_bounds__(1024) evict_select_kernel(const __grid_constant__ EvictParams p) {
  __shared__ int s_hist[256], s_warp[2][32], s_digit, s_left;
  const int plane = blockIdx.x, s = plane / p.src.H_kv, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  griddep_launch_dependents();
  griddep_wait();
  const int n = evict_len(p, s), m = min(n, p.keep);
  if (plane % p.src.H_kv == 0 && tid == 0) p.new_lens[s] = m;
  const float* mass = p.mass + plane * p.mass_rs;
  int32_t* kept = p.kept + (long long)plane * p.keep;
  for (int i = m + tid; i < p.keep; i += 1024) kept[i] = -1;
  const bool all = n <= p.keep;
  const int lo = p.sinks, hi = n - p.recent;      // the positions that compete, unless all stay
  int left = p.keep - p.sinks - p.recent;         // how many of them stay
  uint32_t bits = 0;                              // the last one's weight
  if (!all && left > 0)
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (tid < 256) s_hist[tid] = 0;
      __syncthreads();
      for (int t = lo + tid; t < hi; t += 1024) {
        const uint32_t w = weight_order(mass[t]);
        if (shift == 24 || (w >> (shift + 8)) == (bits >> (shift + 8))) atomicAdd(&s_hist[(w >> shift) & 255], 1);
      }
      __syncthreads();
      if (tid == 0) {
        int d = 255, c = 0;
        while (c + s_hist[d] < left) c += s_hist[d--];
        s_digit = d;
        s_left = left - c;
      }
      __syncthreads();
      bits |= (uint32_t)s_digit << shift;
      left = s_left;
    }
  // in order: those above the last one's weight, and the first `left` of its equals
  int done = 0, equals = 0;
  for (int t0 = 0; t0 < n; t0 += 1024) {
    const int t = t0 + tid;
    const bool fixed = t < n && (all || t < lo || t >= hi);
    const uint32_t w = t < n && !fixed ? weight_order(mass[t]) : 0;
    const bool compete = t < n && !fixed && p.keep > p.sinks + p.recent;
    const bool eq = compete && w == bits;
    const uint32_t be = __ballot_sync(0xffffffffu, eq);
    if (lane == 0) s_warp[0][warp] = __popc(be);
    __syncthreads();
    int before = equals, total = 0;
    for (int i = 0; i < 32; ++i) {
      if (i < warp) before += s_warp[0][i];
      total += s_warp[0][i];
    }
    equals += total;
    const bool stays = fixed || (compete && w > bits) || (eq && before + __popc(be & ((1u << lane) - 1)) < left);
    const uint32_t bs = __ballot_sync(0xffffffffu, stays);
    if (lane == 0) s_warp[1][warp] = __popc(bs);
    __syncthreads();
    int at = done + __popc(bs & ((1u << lane) - 1));
    total = 0;
    for (int i = 0; i < 32; ++i) {
      if (i < warp) at += s_warp[1][i];
      total += s_warp[1][i];
    }
    done += total;
    if (stays) kept[at] = t;
    __syncthreads();
  }
}

// A group of hd / 8 lanes copies a kept position's K and V.
__global__ void __launch_bounds__(256) evict_copy_kernel(const __grid_constant__ EvictParams p) {
  griddep_launch_dependents();
  griddep_wait();
  const int lanes = p.src.hd / 8, l = threadIdx.x % lanes;
  const int plane = blockIdx.y, s = plane / p.src.H_kv, g = plane % p.src.H_kv;
  const int m = min(evict_len(p, s), p.keep), per = 256 / lanes;
  for (int i = blockIdx.x * per + threadIdx.x / lanes; i < m; i += gridDim.x * per) {
    const int t = p.kept[(long long)plane * p.keep + i];
    const long long from = p.src.row(s, g, t), to = p.dst.row(s, g, i);
    uint4 k = make_uint4(0, 0, 0, 0), v = k;
    if (from >= 0) {
      k = reinterpret_cast<const uint4*>(p.src.k + from)[l];
      v = reinterpret_cast<const uint4*>(p.src.v + from)[l];
    }
    if (to >= 0) {
      reinterpret_cast<uint4*>(p.dst.k + to)[l] = k;
      reinterpret_cast<uint4*>(p.dst.v + to)[l] = v;
    }
    if (p.mass_out && l == 0) p.mass_out[plane * p.mass_out_rs + i] = p.mass[plane * p.mass_rs + t];
  }
}

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
  if (planes > 65535)
    return op_fail(DLLM_EINVAL, "kv_paged_evict: b=%d H_kv=%d are too many for one call", src->b, src->H_kv);
  p.mass = mass;
  p.mass_out = mass_out;
  p.lens = lens;
  p.kept = kept;
  p.new_lens = new_lens;
  p.keep = keep;
  p.sinks = sinks;
  p.recent = recent;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  OP_CK(op_launch(evict_select_kernel, dim3((unsigned)planes), dim3(1024), 0, st, 1, p));
  const int per = 256 / (src->hd / 8);
  OP_CK(op_launch(evict_copy_kernel, dim3((unsigned)((keep + per - 1) / per), (unsigned)planes), dim3(256), 0, st, 1, p));
  return DLLM_OK;
}
