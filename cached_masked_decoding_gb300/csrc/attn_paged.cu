// Attention over a paged K/V cache:
//   out[s, i, h] = sum_t p_t V[s, g, t],  p = softmax over t < len[s] of scale * q[s, i, h] . K[s, g, t],
// g = h / (H / H_kv), and the weight that every key received, summed over the rows and heads of g.
//
// One CTA a (sequence, cached head); its rows eight at a time over tiles of 128 keys, a key a thread for the
// scores and a dimension a thread for the values.
#include <algorithm>
#include <cmath>

#include "kv_paged.h"
#include "ptx8.cuh"
#include "q8.cuh"

namespace dllm {

struct AttnPagedParams {
  PagedKv c;
  const uint16_t* q;
  uint16_t* out;
  const int32_t* lens;
  long long q_rs, o_rs, mass_rs;
  float* mass;
  int H, R, group, rows;     // rows: R * group of a cached head
  float scale_log2;
};

template <typename E, int HD>
__global__ void __launch_bounds__(128) attn_paged_simple_kernel(const __grid_constant__ AttnPagedParams p) {
  constexpr int N = 8, KT = 128;
  __shared__ float s_q[N][HD], s_p[N][KT], s_red[N][4], s_m[N], s_l[N], s_up[N];
  const int s = blockIdx.x / p.c.H_kv, g = blockIdx.x % p.c.H_kv, tid = threadIdx.x;
  griddep_wait();
  const int n = p.c.len(p.lens, s);
  using T = typename E::T;
  for (int r0 = 0; r0 < p.rows; r0 += N) {
    const int nr = min(N, p.rows - r0);
    __syncthreads();
    for (int e = tid; e < N * HD; e += 128) {
      const int r = r0 + e / HD;
      s_q[e / HD][e % HD] =
          r < p.rows ? E::get(reinterpret_cast<const T*>(p.q) + ((long long)s * p.R + r / p.group) * p.q_rs +
                              (long long)(g * p.group + r % p.group) * HD + e % HD) : 0.0f;
    }
    if (tid < N) {
      s_m[tid] = -INFINITY;
      s_l[tid] = 0.0f;
    }
    float o[N] = {};
    __syncthreads();
    auto scores = [&](int key, float (&z)[N]) {
      const long long at = key < n ? p.c.row(s, g, key) : -1;
#pragma unroll
      for (int j = 0; j < N; ++j) z[j] = at < 0 ? -INFINITY : 0.0f;
      if (at < 0) return;
      for (int d = 0; d < HD; d += 8) {
        float x[8];
        E::load8(reinterpret_cast<const T*>(p.c.k) + at + d, x);
#pragma unroll
        for (int j = 0; j < N; ++j)
#pragma unroll
          for (int e = 0; e < 8; ++e) z[j] += x[e] * s_q[j][d + e];
      }
#pragma unroll
      for (int j = 0; j < N; ++j) z[j] *= p.scale_log2;
    };
    for (int t0 = 0; t0 < n; t0 += KT) {
      float z[N];
      scores(t0 + tid, z);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        float m = z[j];
        for (int d = 16; d >= 1; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
        if (tid % 32 == 0) s_red[j][tid / 32] = m;
      }
      __syncthreads();
      if (tid < N) {
        const float m = fmaxf(fmaxf(s_red[tid][0], s_red[tid][1]), fmaxf(s_red[tid][2], s_red[tid][3]));
        const float top = fmaxf(m, s_m[tid]);
        s_up[tid] = top == -INFINITY ? 1.0f : exp2f(s_m[tid] - top);
        s_m[tid] = top;
      }
      __syncthreads();
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const float e = z[j] == -INFINITY ? 0.0f : exp2f(z[j] - s_m[j]);
        s_p[j][tid] = e;
        float sum = e;
        for (int d = 16; d >= 1; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        if (tid % 32 == 0) s_red[j][tid / 32] = sum;
        o[j] *= s_up[j];
      }
      __syncthreads();
      if (tid < N) s_l[tid] = s_l[tid] * s_up[tid] + (s_red[tid][0] + s_red[tid][1]) + (s_red[tid][2] + s_red[tid][3]);
      if (tid < HD)
        for (int k = 0; k < min(KT, n - t0); ++k) {
          const long long at = p.c.row(s, g, t0 + k);
          if (at < 0) continue;
          const float v = E::get(reinterpret_cast<const T*>(p.c.v) + at + tid);
#pragma unroll
          for (int j = 0; j < N; ++j) o[j] += s_p[j][k] * v;
        }
      __syncthreads();
    }
    if (tid < HD)
      for (int j = 0; j < nr; ++j) {
        const int r = r0 + j;
        E::put(reinterpret_cast<T*>(p.out) + ((long long)s * p.R + r / p.group) * p.o_rs +
                   (long long)(g * p.group + r % p.group) * HD + tid,
               s_l[j] == 0.0f ? 0.0f : o[j] / s_l[j]);
      }
    if (p.mass)
      for (int t = tid; t < n; t += KT) {
        float z[N], sum = 0.0f;
        scores(t, z);
        for (int j = 0; j < nr; ++j)
          if (z[j] != -INFINITY) sum += exp2f(z[j] - s_m[j]) / s_l[j];
        if (t < p.mass_rs) p.mass[((long long)s * p.c.H_kv + g) * p.mass_rs + t] += sum;
      }
  }
}

}  // namespace dllm

using namespace dllm;

extern "C" dllm_status dllm_op_attention_paged_workspace(int32_t b, int32_t H, int32_t H_kv, int32_t hd, int32_t R,
                                                         int32_t T, int32_t with_mass, int64_t* bytes) {
  if (!bytes || b < 1 || H < 1 || H_kv < 1 || H % H_kv || (hd != 64 && hd != 128) || R < 1 || T < 1 || T > kMostRows)
    return op_fail(DLLM_EINVAL, "bad attention shape: b=%d H=%d H_kv=%d hd=%d R=%d T=%d", b, H, H_kv, hd, R, T);
  if ((__int128)b * R * H > 0x7fffffff)
    return op_fail(DLLM_EINVAL, "attention_paged: b=%d R=%d H=%d are too many rows", b, R, H);
  (void)with_mass;
  *bytes = 0;
  return DLLM_OK;
}

extern "C" dllm_status dllm_op_attention_paged(const void* q, int64_t q_row_stride, const dllm_kv_paged* cache,
                                               const int32_t* lens, float scale, void* out, int64_t out_row_stride,
                                               int32_t H, int32_t R, float* mass, int64_t mass_stride, void* workspace,
                                               int64_t workspace_bytes, void* stream) {
  if (const dllm_status s = kv_paged_check(cache, "attention_paged"); s != DLLM_OK) return s;
  if (!q || !out || H < 1 || H % cache->H_kv || R < 1 || !(scale > 0.0f) || !std::isfinite(scale) ||
      !op_aligned(q, 16) || !op_aligned(out, 16) || !op_aligned(lens, 4) || !op_aligned(mass, 4))
    return op_fail(DLLM_EINVAL,
                   "bad attention_paged arguments: H=%d (a multiple of H_kv=%d) R=%d scale=%g (over 0, finite), q and "
                   "out 16-byte aligned",
                   H, cache->H_kv, R, scale);
  AttnPagedParams p = {};
  p.c = PagedKv(*cache);
  p.q = static_cast<const uint16_t*>(q);
  p.out = static_cast<uint16_t*>(out);
  p.lens = lens;
  const long long width = (long long)H * cache->hd;
  p.q_rs = q_row_stride ? q_row_stride : width;
  p.o_rs = out_row_stride ? out_row_stride : width;
  for (const long long rs : {p.q_rs, p.o_rs})
    if (rs < width || rs > (1LL << 40) || rs % 8)
      return op_fail(DLLM_EINVAL, "attention_paged: row stride %lld (0, or at least H * hd = %lld and a multiple of 8)", rs,
                     width);
  if (mass && (mass_stride < 0 || mass_stride > (1LL << 40)))
    return op_fail(DLLM_EINVAL, "attention_paged: bad mass_stride %lld", (long long)mass_stride);
  p.mass = mass;
  p.mass_rs = mass_stride ? mass_stride : p.c.positions;
  p.H = H;
  p.R = R;
  p.group = H / cache->H_kv;
  p.scale_log2 = scale * 1.4426950408889634f;
  int64_t need = 0;
  if (const dllm_status s = dllm_op_attention_paged_workspace(cache->b, H, cache->H_kv, cache->hd, R,
                                                              (int32_t)p.c.positions, mass != nullptr, &need);
      s != DLLM_OK)
    return s;
  if (need > 0 && (!workspace || workspace_bytes < need || !op_aligned(workspace, 16)))
    return op_fail(DLLM_EINVAL, "attention_paged: a 16-byte aligned workspace of %lld bytes is needed, got %lld",
                   (long long)need, workspace ? (long long)workspace_bytes : 0LL);
  p.rows = R * p.group;
  const dim3 grid((unsigned)(cache->b * cache->H_kv));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool bf = cache->dtype == DLLM_BF16;
  if (cache->hd == 64)
    OP_CK(bf ? op_launch(attn_paged_simple_kernel<ElemBf16, 64>, grid, dim3(128), 0, st, 1, p)
             : op_launch(attn_paged_simple_kernel<ElemF16, 64>, grid, dim3(128), 0, st, 1, p));
  else
    OP_CK(bf ? op_launch(attn_paged_simple_kernel<ElemBf16, 128>, grid, dim3(128), 0, st, 1, p)
             : op_launch(attn_paged_simple_kernel<ElemF16, 128>, grid, dim3(128), 0, st, 1, p));
  return DLLM_OK;
}
