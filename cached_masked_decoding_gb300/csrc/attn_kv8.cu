// Attention over the 8-bit cache:
//   out[s, i, h] = sum_t p_t V[s, g, t],  p = softmax over t < limit[s, i] of
//   scale * q[s, i, h] . K[s, g, t],      g = h / (H / H_kv)
// K = k * 2^ek and V = v * 2^ev with one exponent a row.  A row whose limit is
// 0 or less sees nothing and gives zeros.
//
// One warp per (sequence, row, head) walks its keys with a running maximum and
// sum; the scores, statistics and output are 32-bit.
#include <cmath>

#include "ops8.h"
#include "q8.cuh"

namespace dllm {

dllm_status kv8_check(const dllm_kv8* c, const char* who);

struct AttnKv8Params {
  dllm_kv8 c;
  const uint16_t* q;
  uint16_t* out;
  const int32_t* limits;
  long long q_rs, o_rs;
  int H, R, group;
  float scale_log2;
};

template <int HD>
__global__ void __launch_bounds__(128) attn_kv8_row_kernel(const __grid_constant__ AttnKv8Params p) {
  constexpr int D = HD / 32;
  const long long item = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int h = (int)(item % p.H);
  const long long row = item / p.H;
  if (row >= (long long)p.c.b * p.R) return;
  const int s = (int)(row / p.R);
  const int lim = p.limits ? min(p.limits[row], p.c.T) : p.c.T;
  const long long plane = ((long long)s * p.c.H_kv + h / p.group) * p.c.T;
  float q[D], o[D] = {};
  for (int d = 0; d < D; ++d)
    q[d] = __uint_as_float((uint32_t)p.q[row * p.q_rs + (long long)h * HD + lane * D + d] << 16) * p.scale_log2;
  float m = -INFINITY, l = 0.0f;
  for (int t = 0; t < lim; ++t) {
    const uint8_t* kr = p.c.k + (plane + t) * HD + lane * D;
    const uint8_t* vr = p.c.v + (plane + t) * HD + lane * D;
    const float ks = scale_value(p.c.k_scale[plane + t]), vs = scale_value(p.c.v_scale[plane + t]);
    float z = 0.0f, v[D];
    for (int d = 0; d < D; d += 2) {
      const float2 kf = f16x2_to_f32(cvt_f16x2_e4m3x2((uint16_t)(kr[d] | (kr[d + 1] << 8))));
      const float2 vf = f16x2_to_f32(cvt_f16x2_e4m3x2((uint16_t)(vr[d] | (vr[d + 1] << 8))));
      z += q[d] * kf.x + q[d + 1] * kf.y;
      v[d] = vf.x * vs;
      v[d + 1] = vf.y * vs;
    }
    for (int w = 16; w >= 1; w >>= 1) z += __shfl_xor_sync(0xffffffffu, z, w);
    z *= ks;
    const float mn = z > m ? z : m;
    const float corr = exp2f(m - mn), e = exp2f(z - mn);
    l = l * corr + e;
    for (int d = 0; d < D; ++d) o[d] = o[d] * corr + e * v[d];
    m = mn;
  }
  const float il = lim > 0 ? 1.0f / l : 0.0f;
  for (int d = 0; d < D; ++d) {
    const __nv_bfloat16 r = __float2bfloat16_rn(o[d] * il);
    p.out[row * p.o_rs + (long long)h * HD + lane * D + d] = *reinterpret_cast<const uint16_t*>(&r);
  }
}

}  // namespace dllm

using namespace dllm;

extern "C" dllm_status dllm_op_attention_kv8_workspace(int32_t b, int32_t H, int32_t H_kv, int32_t hd, int32_t R,
                                                       int32_t T, int64_t* bytes) {
  if (!bytes || b < 1 || H < 1 || H_kv < 1 || H % H_kv || (hd != 64 && hd != 128) || R < 1 || T < 1)
    return op_fail(DLLM_EINVAL, "bad attention shape: b=%d H=%d H_kv=%d hd=%d R=%d T=%d", b, H, H_kv, hd, R, T);
  *bytes = 0;
  return DLLM_OK;
}

extern "C" dllm_status dllm_op_attention_kv8(const uint16_t* q, int64_t q_row_stride, const dllm_kv8* cache,
                                             const int32_t* limits, float scale, uint16_t* out,
                                             int64_t out_row_stride, int32_t H, int32_t R, void* workspace,
                                             int64_t workspace_bytes, void* stream) {
  if (const dllm_status s = kv8_check(cache, "attention_kv8"); s != DLLM_OK) return s;
  if (!q || !out || H < 1 || H % cache->H_kv || R < 1 || !(scale > 0.0f) || !std::isfinite(scale) ||
      !op_aligned(q, 16) || !op_aligned(out, 16) || !op_aligned(limits, 4))
    return op_fail(DLLM_EINVAL,
                   "bad attention_kv8 arguments: H=%d (a multiple of H_kv=%d) R=%d scale=%g, q and out 16-byte aligned",
                   H, cache->H_kv, R, scale);
  const long long width = (long long)H * cache->hd;
  AttnKv8Params p = {};
  p.c = *cache;
  p.q = q;
  p.out = out;
  p.limits = limits;
  p.q_rs = q_row_stride ? q_row_stride : width;
  p.o_rs = out_row_stride ? out_row_stride : width;
  for (const long long rs : {p.q_rs, p.o_rs})
    if (rs < width || rs > (1LL << 40) || rs % 8)
      return op_fail(DLLM_EINVAL, "attention_kv8: row stride %lld (0, or at least H * hd = %lld and a multiple of 8)",
                     rs, width);
  p.H = H;
  p.R = R;
  p.group = H / cache->H_kv;
  p.scale_log2 = scale * 1.4426950408889634f;
  const __int128 blocks = ((__int128)cache->b * R * H + 3) / 4;
  if (blocks > 0x7fffffff) return op_fail(DLLM_EINVAL, "attention_kv8: b=%d R=%d H=%d are too many rows", cache->b, R, H);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (cache->hd == 64)
    attn_kv8_row_kernel<64><<<(unsigned)blocks, 128, 0, st>>>(p);
  else
    attn_kv8_row_kernel<128><<<(unsigned)blocks, 128, 0, st>>>(p);
  OP_CK(cudaGetLastError());
  return DLLM_OK;
}
