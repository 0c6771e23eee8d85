// The 8-bit K/V cache: quantising rows as they are written, and reading them
// back.  One scale for each row of hd elements (a token's head), see q8.cuh.
//
// Both directions are bound by HBM (store reads 2 hd elements and writes
// 2 hd + 2 bytes a token and head).  A group of hd / 8 lanes owns a row of K and that of V
// (the slot's arithmetic, a third of the instructions, serves both): each lane
// takes one 16-byte vector of 16-bit elements, the row's largest value
// is a shuffle reduction within the group, and a row's codes are one
// contiguous write of hd bytes.  Consecutive groups take consecutive tokens of a head,
// whose codes and scale bytes lie side by side in the cache (5 % faster than
// consecutive heads of a token, whose elements do: 49 against 51 us for 3 x 5000
// tokens of 16 heads of 64 in float32).  A second row in flight in every thread made it slower
// (64 x 32 tokens of 32 heads of 128 in bf16, store and load, 21.5 us against 20.3, 4.1 TB/s; 4 x 1000
// tokens of 8 heads of 64, 8.9 against 6.9).
#include "ops8.h"
#include "ptx8.cuh"
#include "q8.cuh"

namespace dllm {

struct Kv8Params {
  dllm_kv8 c;
  const void* in[2];     // store: rows of K and V
  void* out[2];          // load: rows of K and V
  long long rs[2];       // their row strides, elements
  const int32_t* starts; // [b] position of a sequence's first row, or null (0)
  const int32_t* counts; // [b] rows of a sequence that take part, or null (R)
  int R;
  uint32_t groups;       // b * R * H_kv row-heads
  FastDiv heads, rows;   // by H_kv and by R
};

// (sequence, row, head) of a thread group's item and its cache slot; false
// where the row takes no part.
struct Kv8Item {
  uint32_t row, h;
  long long elem;        // the head's first element within a row (over 2^32 where heads are many)
  long long slot;        // (sequence * H_kv + head) * T + position
  __device__ __forceinline__ bool init(const Kv8Params& p, uint32_t g) {
    if (g >= p.groups) return false;
    uint32_t i;
    const uint32_t s = p.heads.divmod(p.rows.divmod(g, i), h);
    row = s * (uint32_t)p.R + i;
    const int n = p.counts ? p.counts[s] : p.R;
    if ((int)i >= n) return false;
    const long long pos = (long long)(p.starts ? p.starts[s] : 0) + i;
    if (pos < 0 || pos >= p.c.T) return false;
    elem = (long long)h * p.c.hd;
    slot = ((long long)s * p.c.H_kv + h) * p.c.T + pos;
    return true;
  }
};

template <typename E, int HD>
__global__ void __launch_bounds__(256, 4) kv8_store_kernel(const __grid_constant__ Kv8Params p) {
  constexpr int L = HD / 8;
  const int l = threadIdx.x % L;
  griddep_launch_dependents();
  griddep_wait();
  Kv8Item it;
  const bool on = it.init(p, blockIdx.x * (uint32_t)(256 / L) + threadIdx.x / L);
  Raw8<E> raw[2];
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    raw[w].zero();
    if (on) raw[w].template load<L>(static_cast<const typename E::T*>(p.in[w]) + it.row * p.rs[w] + it.elem, l);
  }
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    float x[8];
    raw[w].floats(x);
    uint32_t m = abs_bits8(x);
#pragma unroll
    for (int d = L / 2; d >= 1; d >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
    if (!on) continue;
    const int byte = scale_byte(m);
    uint2 codes = make_uint2(0, 0);
    if (byte != kScaleNan) codes = encode8(x, scale_inverse(byte));
    Raw8<E>::template store_codes<L>((w ? p.c.v : p.c.k) + it.slot * HD, l, codes);
    if (l == 0) (w ? p.c.v_scale : p.c.k_scale)[it.slot] = (uint8_t)byte;
  }
}

template <typename E, int HD>
__global__ void __launch_bounds__(256, 4) kv8_load_kernel(const __grid_constant__ Kv8Params p) {
  constexpr int L = HD / 8;
  const int l = threadIdx.x % L;
  griddep_launch_dependents();
  griddep_wait();
  Kv8Item it;
  if (!it.init(p, blockIdx.x * (uint32_t)(256 / L) + threadIdx.x / L)) return;
  uint2 codes[2];
  int byte[2];
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    codes[w] = Raw8<E>::template load_codes<L>((w ? p.c.v : p.c.k) + it.slot * HD, l);
    byte[w] = (w ? p.c.v_scale : p.c.k_scale)[it.slot];
  }
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    float x[8];
    decode8(codes[w], scale_value(byte[w]), x);
    Raw8<E> out;
    out.from(x);
    out.template store<L>(static_cast<typename E::T*>(p.out[w]) + it.row * p.rs[w] + it.elem, l);
  }
}

dllm_status kv8_check(const dllm_kv8* c, const char* who) {
  if (!c || !c->k || !c->v || !c->k_scale || !c->v_scale || c->b < 1 || c->H_kv < 1 || c->T < 1 || c->T > kMostRows ||
      (c->hd != 64 && c->hd != 128) || !op_aligned(c->k, 16) || !op_aligned(c->v, 16))
    return op_fail(DLLM_EINVAL, "%s: bad cache (b, H_kv >= 1, T 1..%d, hd 64 or 128, codes 16-byte aligned)%s", who,
                   kMostRows, c ? "" : ": null");
  if ((__int128)c->b * c->H_kv * c->T > ((__int128)1 << 48))
    return op_fail(DLLM_EINVAL, "%s: a cache of b=%d H_kv=%d T=%d is too large", who, c->b, c->H_kv, c->T);
  return DLLM_OK;
}

namespace {

template <typename E, int HD>
cudaError_t launch_kv8(const Kv8Params& p, bool store, cudaStream_t st) {
  constexpr uint32_t per_block = 256 / (HD / 8);
  const dim3 grid((p.groups + per_block - 1) / per_block);
  return store ? op_launch(kv8_store_kernel<E, HD>, grid, dim3(256), 0, st, 1, p)
               : op_launch(kv8_load_kernel<E, HD>, grid, dim3(256), 0, st, 1, p);
}

template <typename E>
cudaError_t launch_kv8(const Kv8Params& p, bool store, cudaStream_t st) {
  return p.c.hd == 64 ? launch_kv8<E, 64>(p, store, st) : launch_kv8<E, 128>(p, store, st);
}

dllm_status kv8_rows(const dllm_kv8* cache, bool store, const void* k, const void* v, int64_t k_rs, int64_t v_rs,
                     int32_t dtype, int32_t R, const int32_t* starts, const int32_t* counts, void* stream) {
  const char* who = store ? "kv8_store" : "kv8_load";
  if (const dllm_status s = kv8_check(cache, who); s != DLLM_OK) return s;
  const int es = op_dtype_size(dtype);
  if (!k || !v || R < 1 || es == 0 || !op_aligned(k, 16) || !op_aligned(v, 16) || !op_aligned(starts, 4) ||
      !op_aligned(counts, 4))
    return op_fail(DLLM_EINVAL, "bad %s arguments: R=%d dtype=%d (k and v 16-byte aligned)", who, R, dtype);
  const long long width = (long long)cache->H_kv * cache->hd;
  Kv8Params p = {};
  p.c = *cache;
  p.rs[0] = k_rs ? k_rs : width;
  p.rs[1] = v_rs ? v_rs : width;
  for (const long long rs : p.rs)
    if (rs < width || rs > (1LL << 40) || (rs * es) % 16)
      return op_fail(DLLM_EINVAL, "%s: row stride %lld (0, or at least H_kv * hd = %lld and a multiple of 16 bytes)",
                     who, rs, width);
  p.in[0] = k;
  p.in[1] = v;
  p.out[0] = const_cast<void*>(k);
  p.out[1] = const_cast<void*>(v);
  p.starts = starts;
  p.counts = counts;
  p.R = R;
  const __int128 groups = (__int128)cache->b * R * cache->H_kv;
  if (groups > 0x7fffff00)
    return op_fail(DLLM_EINVAL, "%s: b=%d R=%d H_kv=%d are too many rows for one call", who, cache->b, R, cache->H_kv);
  p.groups = (uint32_t)groups;
  p.heads = FastDiv((uint32_t)cache->H_kv);
  p.rows = FastDiv((uint32_t)R);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  switch (dtype) {
    case DLLM_F32: OP_CK(launch_kv8<ElemF32>(p, store, st)); break;
    case DLLM_BF16: OP_CK(launch_kv8<ElemBf16>(p, store, st)); break;
    default: OP_CK(launch_kv8<ElemF16>(p, store, st)); break;
  }
  return DLLM_OK;
}

}  // namespace
}  // namespace dllm

using namespace dllm;

extern "C" dllm_status dllm_op_kv8_store(const dllm_kv8* cache, const void* k, const void* v, int64_t k_row_stride,
                                         int64_t v_row_stride, int32_t dtype, int32_t R, const int32_t* starts,
                                         const int32_t* counts, void* stream) {
  return kv8_rows(cache, true, k, v, k_row_stride, v_row_stride, dtype, R, starts, counts, stream);
}

extern "C" dllm_status dllm_op_kv8_load(const dllm_kv8* cache, void* k, void* v, int64_t k_row_stride,
                                        int64_t v_row_stride, int32_t dtype, int32_t R, const int32_t* starts,
                                        const int32_t* counts, void* stream) {
  return kv8_rows(cache, false, k, v, k_row_stride, v_row_stride, dtype, R, starts, counts, stream);
}
