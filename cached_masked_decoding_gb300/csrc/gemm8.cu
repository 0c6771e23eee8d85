// 8-bit matrix product with a scale for each block of 128 along K, and the
// quantiser of its operands (see q8.cuh):
//   Y[n][m] = sum_B 2^(ex[B][n] + ew[B][m]) * sum_{k in block B} X[n][k] W[m][k]
#include "ops8.h"
#include "q8.cuh"

namespace dllm {

constexpr int kQBlock = 128;

// ---------------------------------------------------------------- quantiser
// A group of 16 lanes owns a block of 128 elements, 8 each.
template <typename E, bool VEC>
__global__ void __launch_bounds__(256) quantise8_kernel(const void* x_, long long rs, int rows, int K, int kb,
                                                        uint8_t* codes, uint8_t* scales) {
  const long long tid = (long long)blockIdx.x * 256 + threadIdx.x;
  const int l = (int)(tid & 15);
  const long long g = tid >> 4;
  const int B = (int)(g % kb);
  const long long row = g / kb;
  const int k0 = B * kQBlock + l * 8;
  const bool on = row < rows && k0 < K;       // K % 16 == 0: a lane's 8 elements are all in or all out
  float x[8] = {};
  if (on) {
    const typename E::T* px = static_cast<const typename E::T*>(x_) + row * rs + k0;
    if constexpr (VEC) {
      E::load8(px, x);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = E::get(px + i);
    }
  }
  uint32_t m = abs_bits8(x);
#pragma unroll
  for (int d = 8; d >= 1; d >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
  const int byte = scale_byte(m);
  if (on) {
    uint2 c = make_uint2(0, 0);
    if (byte != kScaleNan) c = encode8(x, scale_inverse(byte));
    *reinterpret_cast<uint2*>(codes + row * K + k0) = c;
  }
  if (l == 0 && row < rows) scales[(long long)B * rows + row] = (uint8_t)byte;
}

// ---------------------------------------------------------------- product
struct Gemm8Params {
  const uint8_t *w, *ws, *x, *xs;
  void* y;
  int M, N, K, kb, out_bf16;
};

// One 16 x 16 tile of Y a block, a block of 128 along K at a time.
__global__ void __launch_bounds__(256) gemm8_tile_kernel(const __grid_constant__ Gemm8Params p) {
  __shared__ float sw[16][kQBlock + 1], sx[16][kQBlock + 1];
  const int m0 = blockIdx.x * 16, n0 = blockIdx.y * 16;
  const int tm = threadIdx.x & 15, tn = threadIdx.x >> 4;
  float acc = 0.0f;
  for (int B = 0; B < p.kb; ++B) {
    __syncthreads();
    for (int e = threadIdx.x; e < 16 * 64; e += 256) {
      const int r = e >> 6, c = (e & 63) * 2, k = B * kQBlock + c;
      float2 w = make_float2(0.f, 0.f), x = w;
      if (k < p.K && m0 + r < p.M)
        w = f16x2_to_f32(cvt_f16x2_e4m3x2(*reinterpret_cast<const uint16_t*>(p.w + (long long)(m0 + r) * p.K + k)));
      if (k < p.K && n0 + r < p.N)
        x = f16x2_to_f32(cvt_f16x2_e4m3x2(*reinterpret_cast<const uint16_t*>(p.x + (long long)(n0 + r) * p.K + k)));
      sw[r][c] = w.x;
      sw[r][c + 1] = w.y;
      sx[r][c] = x.x;
      sx[r][c + 1] = x.y;
    }
    __syncthreads();
    float d = 0.0f;
    for (int k = 0; k < kQBlock; ++k) d += sw[tm][k] * sx[tn][k];
    if (m0 + tm < p.M && n0 + tn < p.N)
      acc += d * scale_value(p.ws[(long long)B * p.M + m0 + tm]) * scale_value(p.xs[(long long)B * p.N + n0 + tn]);
  }
  if (m0 + tm < p.M && n0 + tn < p.N) {
    const long long o = (long long)(n0 + tn) * p.M + m0 + tm;
    if (p.out_bf16)
      static_cast<__nv_bfloat16*>(p.y)[o] = __float2bfloat16_rn(acc);
    else
      static_cast<float*>(p.y)[o] = acc;
  }
}

namespace {

template <typename E>
cudaError_t launch_quantise8(const void* x, long long rs, int rows, int K, uint8_t* codes, uint8_t* scales, bool vec,
                             unsigned grid, cudaStream_t st) {
  const int kb = (K + kQBlock - 1) / kQBlock;
  if (vec)
    quantise8_kernel<E, true><<<grid, 256, 0, st>>>(x, rs, rows, K, kb, codes, scales);
  else
    quantise8_kernel<E, false><<<grid, 256, 0, st>>>(x, rs, rows, K, kb, codes, scales);
  return cudaGetLastError();
}

}  // namespace
}  // namespace dllm

using namespace dllm;

extern "C" dllm_status dllm_op_quantise8(const void* x, int64_t row_stride, int32_t dtype, int32_t rows, int32_t K,
                                         uint8_t* codes, uint8_t* scales, void* stream) {
  const int es = op_dtype_size(dtype);
  if (!x || !codes || !scales || rows < 1 || K < 16 || K % 16 || es == 0 || !op_aligned(x, es) || !op_aligned(codes, 16))
    return op_fail(DLLM_EINVAL, "bad quantise8 arguments: rows=%d K=%d (K %% 16 == 0) dtype=%d, codes 16-byte aligned",
                   rows, K, dtype);
  const long long rs = row_stride ? row_stride : K;
  if (rs < K || rs > (1LL << 40)) return op_fail(DLLM_EINVAL, "quantise8: row stride %lld (0, or at least K=%d)", rs, K);
  const long long kb = (K + kQBlock - 1) / kQBlock;
  const long long blocks = (rows * kb * 16 + 255) / 256;
  if (blocks > 0x7fffffffLL) return op_fail(DLLM_EINVAL, "quantise8: rows=%d K=%d are too many blocks", rows, K);
  const bool vec = op_aligned(x, 16) && (rs * es) % 16 == 0;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  switch (dtype) {
    case DLLM_F32: OP_CK(launch_quantise8<ElemF32>(x, rs, rows, K, codes, scales, vec, (unsigned)blocks, st)); break;
    case DLLM_BF16: OP_CK(launch_quantise8<ElemBf16>(x, rs, rows, K, codes, scales, vec, (unsigned)blocks, st)); break;
    default: OP_CK(launch_quantise8<ElemF16>(x, rs, rows, K, codes, scales, vec, (unsigned)blocks, st)); break;
  }
  return DLLM_OK;
}

extern "C" dllm_status dllm_op_gemm8(const uint8_t* W, const uint8_t* W_scale, const uint8_t* X,
                                     const uint8_t* X_scale, void* Y, int32_t y_dtype, int32_t M, int32_t N, int32_t K,
                                     void* stream) {
  if (!W || !W_scale || !X || !X_scale || !Y || (y_dtype != DLLM_F32 && y_dtype != DLLM_BF16) || M < 1 || N < 1 ||
      K < 16 || K % 16 || !op_aligned(W, 16) || !op_aligned(X, 16) || !op_aligned(Y, 16))
    return op_fail(DLLM_EINVAL,
                   "bad gemm8 arguments: M=%d N=%d K=%d (K %% 16 == 0) y_dtype=%d (float32 or bf16), W, X and Y "
                   "16-byte aligned",
                   M, N, K, y_dtype);
  if ((N + 15) / 16 > 65535) return op_fail(DLLM_EINVAL, "gemm8: N=%d is too large", N);
  Gemm8Params p = {W, W_scale, X, X_scale, Y, M, N, K, (K + kQBlock - 1) / kQBlock, y_dtype == DLLM_BF16};
  gemm8_tile_kernel<<<dim3((unsigned)((M + 15) / 16), (unsigned)((N + 15) / 16)), 256, 0,
                      static_cast<cudaStream_t>(stream)>>>(p);
  OP_CK(cudaGetLastError());
  return DLLM_OK;
}
