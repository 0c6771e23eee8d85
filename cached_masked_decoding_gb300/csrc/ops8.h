// Shared by the translation units of the 8-bit operators: error reporting of
// the C entries, and what each unit gives dllm_op_check.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/dllm.h"

namespace dllm {

// Set this thread's dllm_last_error() message (printf style); returns st.
dllm_status op_fail(dllm_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
dllm_status op_cuda_fail(cudaError_t e, const char* what);

// SMs of the current device.
int op_device_sms();

// 8-bit tensor map over [planes][rows][inner] bytes (rows `row_stride`, planes
// `plane_stride` bytes apart, multiples of 16), box [1][box_rows][box_inner],
// swizzle over box_inner = 64 or 128 bytes.  Out-of-range elements read 0.
dllm_status op_map_u8(CUtensorMap* m, const void* base, uint64_t inner, uint64_t rows, uint64_t planes,
                      uint64_t row_stride, uint64_t plane_stride, uint32_t box_inner, uint32_t box_rows);

// Allow a kernel `bytes` of dynamic shared memory on the current device, once.
cudaError_t op_smem_once(const void* kernel, int bytes);

// Error words of the kernels with bounded waits (device addresses).
cudaError_t gemm8_err_word(int** p);
cudaError_t attn_kv8_err_word(int** p);
cudaError_t attn_paged_err_word(int** p);
cudaError_t heads_err_word(int** p);
cudaError_t logprobs_err_word(int** p);

// Launch with programmatic dependent launch: the kernel's prologue overlaps the
// end of the kernel before it in the stream, and griddepcontrol.wait in the
// kernel orders everything that touches global memory behind that kernel.
// A kernel launched so is resident while the ones before it still write, so its loads are ordinary
// ones: the non-coherent path is for data that nothing writes during the kernel's whole life.
// cluster > 1: that many consecutive CTAs form a cluster.
template <typename Kern, typename... Args>
inline cudaError_t op_launch(Kern kernel, dim3 grid, dim3 block, size_t smem, cudaStream_t st, int cluster,
                             const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Division of n < 2^31 by a launch constant d: a multiply and a shift in place of
// the ~20 instructions of a 32-bit division (m = ceil(2^(31 + s) / d), 2^s >= d, is
// exact for such n).
struct FastDiv {
  uint32_t d, m, s;
  FastDiv() = default;
  explicit FastDiv(uint32_t div) : d(div), m(0), s(0) {
    while ((1ull << s) < d) ++s;
    m = (uint32_t)(((1ull << (31 + s)) + d - 1) / d);
  }
#ifdef __CUDACC__
  __device__ __forceinline__ uint32_t div(uint32_t n) const { return d == 1 ? n : __umulhi(n, m) >> (s - 1); }
  __device__ __forceinline__ uint32_t divmod(uint32_t n, uint32_t& rem) const {
    const uint32_t q = div(n);
    rem = n - q * d;
    return q;
  }
#endif
};

// Most rows of a tiled axis (a cache's positions, a product's sides): tiles past the end and
// the prefetches ahead of them stay in 31 bits.
constexpr int32_t kMostRows = 0x7fffffff - 4095;

inline bool op_aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline int op_dtype_size(int32_t t) { return t == DLLM_F32 ? 4 : (t == DLLM_BF16 || t == DLLM_F16) ? 2 : 0; }

}  // namespace dllm

#define OP_CK(call)                                                  \
  do {                                                               \
    const cudaError_t e_ = (call);                                   \
    if (e_ != cudaSuccess) return ::dllm::op_cuda_fail(e_, #call);   \
  } while (0)
