// What rows of logits say: log probabilities of given tokens, entropy, the largest alternatives.
//
// With M the largest z of a row, at token a, and sums over the others,
//   S = sum e^(z - M),  W = sum (z - M) e^(z - M):
//   log p_i = (z_i - M) - log1p(S),   entropy = log1p(S) - W / (1 + S).
// The largest term is left out of the sums, so a nearly certain row's S keeps its relative accuracy, and both
// parts of the entropy are of one sign.
//
// One CTA a row: its maximum, its sums, and one pass for each alternative (the largest that comes after the last).
#include <cmath>

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
  int vocab, top;
  float scale;
};

constexpr int kLogThreads = 512;

struct Best {
  float x;
  int i;    // -1: none
};
// a before b: larger, or of a lower index
__device__ __forceinline__ bool before(const Best& a, const Best& b) {
  return a.i >= 0 && (b.i < 0 || a.x > b.x || (a.x == b.x && a.i < b.i));
}

__device__ Best block_best(Best b, Best* s) {
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) {
    const Best o = {__shfl_xor_sync(0xffffffffu, b.x, d), __shfl_xor_sync(0xffffffffu, b.i, d)};
    if (before(o, b)) b = o;
  }
  __syncthreads();
  if (threadIdx.x % 32 == 0) s[threadIdx.x / 32] = b;
  __syncthreads();
  b = s[0];
  for (int w = 1; w < kLogThreads / 32; ++w)
    if (before(s[w], b)) b = s[w];
  return b;
}

template <typename E>
__global__ void __launch_bounds__(kLogThreads) logprobs_kernel(const __grid_constant__ LogprobsParams p) {
  __shared__ Best s_best[kLogThreads / 32];
  __shared__ float s_sum[2][kLogThreads / 32];
  const int tid = threadIdx.x;
  const long long row = blockIdx.x;
  griddep_launch_dependents();
  griddep_wait();
  const typename E::T* x = static_cast<const typename E::T*>(p.logits) + row * p.rs;
  Best b = {0.0f, -1};
  for (int i = tid; i < p.vocab; i += kLogThreads) {
    const Best c = {E::get(x + i), i};
    if (c.x == c.x && before(c, b)) b = c;
  }
  const Best first = block_best(b, s_best);
  float S = 0.0f, W = 0.0f;
  for (int i = tid; i < p.vocab; i += kLogThreads) {
    if (i == first.i) continue;
    const float v = E::get(x + i), d = (v - first.x) * p.scale;
    const float e = expf(d);
    S += e;
    if (e > 0.0f) W += d * e;      // (a term of 0 may have an infinite d)
  }
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) {
    S += __shfl_xor_sync(0xffffffffu, S, d);
    W += __shfl_xor_sync(0xffffffffu, W, d);
  }
  if (tid % 32 == 0) {
    s_sum[0][tid / 32] = S;
    s_sum[1][tid / 32] = W;
  }
  __syncthreads();
  S = W = 0.0f;
  for (int w = 0; w < kLogThreads / 32; ++w) {
    S += s_sum[0][w];
    W += s_sum[1][w];
  }
  const bool finite = first.i >= 0 && fabsf(first.x) != INFINITY && S == S;
  const float nan = __uint_as_float(0x7fffffffu), log_sum = finite ? log1pf(S) : nan;
  if (tid == 0) {
    if (p.logp) {
      const int t = p.targets[row];
      p.logp[row] = t >= 0 && t < p.vocab ? (E::get(x + t) - first.x) * p.scale - log_sum : nan;
    }
    if (p.entropy) p.entropy[row] = log_sum - W / (1.0f + S);
  }
  Best last = first;
  for (int k = 0; k < p.top; ++k) {
    if (tid == 0) {
      p.top_ids[row * p.top + k] = last.i;
      p.top_logp[row * p.top + k] = last.i < 0 ? nan : (last.x - first.x) * p.scale - log_sum;
    }
    if (k + 1 == p.top || last.i < 0) continue;
    b = {0.0f, -1};
    for (int i = tid; i < p.vocab; i += kLogThreads) {
      const Best c = {E::get(x + i), i};
      if (c.x == c.x && before(last, c) && before(c, b)) b = c;
    }
    last = block_best(b, s_best);
  }
}

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
  const dim3 grid((unsigned)rows), block(kLogThreads);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  switch (dtype) {
    case DLLM_F32: OP_CK(op_launch(logprobs_kernel<ElemF32>, grid, block, 0, st, 1, p)); break;
    case DLLM_BF16: OP_CK(op_launch(logprobs_kernel<ElemBf16>, grid, block, 0, st, 1, p)); break;
    default: OP_CK(op_launch(logprobs_kernel<ElemF16>, grid, block, 0, st, 1, p)); break;
  }
  return DLLM_OK;
}
