// Attention over a paged K/V cache:
//   out[s, i, h] = sum_t p_t V[s, g, t],  p = softmax over t < len[s] of scale * q[s, i, h] . K[s, g, t],
// g = h / (H / H_kv), and the weight that every key received, summed over the rows and heads of g.  The kernels are
// in attn_paged.cuh; here is what runs, and on what.
#include <algorithm>

#include "attn_paged.cuh"

namespace dllm {

cudaError_t attn_paged_err_word(int** p) { return cudaGetSymbolAddress(reinterpret_cast<void**>(p), g_attn_paged_err); }

namespace {

struct AttnPagedPlan {
  int N, row_tiles, whole, ctas, nz;
  long long items, tiles;     // tiles: of an item, at most
  size_t o, ml, plan, items_at, lse, z, bytes;
};

AttnPagedPlan plan_attn_paged(long long b, long long H_kv, long long rows, int hd, long long T, bool mass) {
  AttnPagedPlan a = {};
  a.N = rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
  a.row_tiles = (int)((rows + a.N - 1) / a.N);
  a.items = b * H_kv * a.row_tiles;
  a.tiles = std::max(1LL, (T + kPagedKeys - 1) / kPagedKeys);
  a.ctas = (a.N <= 16 ? 2 : 1) * op_device_sms();
  // Few keys: items as they are, one kernel.  Whole items and shared runs, us, at 250, 500 and 1000 keys: 32 rows of 32
  // heads 8.2 and 10.9, 11.1 and 11.4, 17.4 and 13.0; of 8 sequences 13.1 and 14.6, 18.6 and 23.2, 30.4 and 33.7; of 16
  // with 32 heads on 8 (500, 1000) 24.6 and 33.3, 38.2 and 45.3; one token of 32 heads 6.9 and 9.3, 10.2 and 9.8, 17.3 and
  // 10.9; of 64 sequences, 32 heads on 8, 16.1 and 17.3, 25.0 and 26.4, 42.1 and 40.4.
  a.whole = a.tiles <= 4;
  a.nz = rows <= 4 ? 4 : a.N;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t from = at;
    at += (bytes + 15) / 16 * 16;
    return from;
  };
  a.o = take(a.whole ? 0 : (size_t)2 * a.ctas * a.N * hd * 4);
  a.ml = take(a.whole ? 0 : (size_t)2 * a.ctas * a.N * 8);
  a.plan = take(a.whole ? 0 : (size_t)a.ctas * 16);
  a.items_at = take(mass && !a.whole ? (size_t)a.items * 8 : 0);
  a.lse = take(mass ? (size_t)a.items * a.N * 4 : 0);
  a.z = take(mass ? (size_t)a.items * a.tiles * kPagedKeys * a.nz * 4 : 0);
  a.bytes = at;
  return a;
}

template <typename F, int HD, int N>
cudaError_t launch_attn_paged(const CUtensorMap& tk, const CUtensorMap& tv, const AttnPagedParams& p,
                              const AttnPagedPlan& a, cudaStream_t st) {
  using C = AttnPagedCfg<HD, N>;
  cudaError_t e = op_smem_once(reinterpret_cast<const void*>(attn_paged_kernel<F, HD, N>), C::SMEM_BYTES);
  if (e != cudaSuccess) return e;
  const long long units = a.whole ? a.items : a.items * (a.tiles + 1);
  const unsigned grid = (unsigned)std::min<long long>(a.ctas, (units + p.min_share - 1) / p.min_share);
  e = op_launch(attn_paged_kernel<F, HD, N>, dim3(grid), dim3(C::THREADS), C::SMEM_BYTES, st, 1, tk, tv, p);
  if (e != cudaSuccess) return e;
  if (a.whole && !p.mass) return cudaSuccess;
  AttnPagedParams f = p;
  f.join_ctas = (int)grid;
  f.joins = a.whole ? 0 : (int)grid * (N > 8 ? (std::min(N, p.rows) + 3) / 4 : p.rows);
  const long long chunks = p.mass ? (long long)p.c.b * p.c.H_kv * p.by_chunks.d : 0;
  const dim3 rest((unsigned)(f.joins + chunks));
  // (the same split of L1 and shared memory as the first kernel's: an SM need not drain to change it)
  const auto finish = p.mass ? attn_paged_finish_kernel<F, HD, true> : attn_paged_finish_kernel<F, HD, false>;
  e = op_smem_once(reinterpret_cast<const void*>(finish), 0);
  if (e != cudaSuccess) return e;
  return op_launch(finish, rest, dim3(128), 0, st, 1, f, N);
}

template <typename F, int HD>
cudaError_t launch_attn_paged(const CUtensorMap& tk, const CUtensorMap& tv, const AttnPagedParams& p,
                              const AttnPagedPlan& a, cudaStream_t st) {
  switch (a.N) {
    case 8: return launch_attn_paged<F, HD, 8>(tk, tv, p, a, st);
    case 16: return launch_attn_paged<F, HD, 16>(tk, tv, p, a, st);
    case 32: return launch_attn_paged<F, HD, 32>(tk, tv, p, a, st);
    default: return launch_attn_paged<F, HD, 64>(tk, tv, p, a, st);
  }
}

}  // namespace
}  // namespace dllm

using namespace dllm;

extern "C" dllm_status dllm_op_attention_paged_workspace(int32_t b, int32_t H, int32_t H_kv, int32_t hd, int32_t R,
                                                         int32_t T, int32_t with_mass, int64_t* bytes) {
  if (!bytes || b < 1 || H < 1 || H_kv < 1 || H % H_kv || (hd != 64 && hd != 128) || R < 1 || T < 1 || T > kMostRows)
    return op_fail(DLLM_EINVAL, "bad attention shape: b=%d H=%d H_kv=%d hd=%d R=%d T=%d", b, H, H_kv, hd, R, T);
  if ((__int128)b * R * H > 0x7fffffff)
    return op_fail(DLLM_EINVAL, "attention_paged: b=%d R=%d H=%d are too many rows", b, R, H);
  const AttnPagedPlan a = plan_attn_paged(b, H_kv, (long long)R * (H / H_kv), hd, T, with_mass != 0);
  if (a.items > 0x7fffffff || (double)a.items * (double)a.tiles > 1e11 || (double)b * a.tiles > 2e9)
    return op_fail(DLLM_EINVAL, "attention_paged: b=%d R=%d H=%d T=%d are too many keys for one call", b, R, H, T);
  *bytes = (int64_t)a.bytes;
  return DLLM_OK;
}

extern "C" dllm_status dllm_op_attention_paged(const void* q, int64_t q_row_stride, const dllm_kv_paged* cache,
                                               const int32_t* lens, float scale, void* out, int64_t out_row_stride,
                                               int32_t H, int32_t R, float* mass, int64_t mass_stride, void* workspace,
                                               int64_t workspace_bytes, void* stream) {
  if (const dllm_status s = kv_paged_check(cache, "attention_paged"); s != DLLM_OK) return s;
  if (!q || !out || H < 1 || H % cache->H_kv || R < 1 || !(scale > 0.0f) || scale > 1e38f ||
      !op_aligned(q, 16) || !op_aligned(out, 16) || !op_aligned(lens, 4) || !op_aligned(mass, 4))
    return op_fail(DLLM_EINVAL,
                   "bad attention_paged arguments: H=%d (a multiple of H_kv=%d) R=%d scale=%g (over 0, to 1e38), q and "
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
  const AttnPagedPlan a = plan_attn_paged(cache->b, cache->H_kv, p.rows, cache->hd, p.c.positions, mass != nullptr);
  p.row_tiles = a.row_tiles;
  p.per_seq = cache->H_kv * a.row_tiles;
  p.whole = a.whole;
  p.min_share = a.whole ? 1 : 2;   // (an item's start and a tile; 3: 13.6 us for 12.7, 32 rows of 32 heads, 768 keys)
  p.by_group = FastDiv((uint32_t)p.group);
  p.by_heads = FastDiv((uint32_t)cache->H_kv);
  p.nz = a.nz;
  p.chunk_keys = a.nz <= 8 ? 256 : 2048 / a.nz;
// (runs that leave every SM 16 CTAs: their rows' log sums are worked out once a run)
  const long long chunks = (p.c.positions + p.chunk_keys - 1) / p.chunk_keys;
  p.chunk_run = (int)std::max(1LL, std::min(32LL, cache->b * (long long)cache->H_kv * chunks / (16LL * op_device_sms())));
  p.by_chunks = FastDiv((uint32_t)((chunks + p.chunk_run - 1) / p.chunk_run));
  p.z_tiles = (int)a.tiles;
  if (mass && (double)cache->b * cache->H_kv * p.by_chunks.d > 0x7fff0000)
    return op_fail(DLLM_EINVAL, "attention_paged: b=%d H_kv=%d of %lld positions are too many weights for one call", cache->b,
                   cache->H_kv, p.c.positions);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.ws_o = reinterpret_cast<float*>(ws + a.o);
  p.ws_ml = reinterpret_cast<float*>(ws + a.ml);
  p.ws_plan = reinterpret_cast<int4*>(ws + a.plan);
  p.ws_items = reinterpret_cast<int2*>(ws + a.items_at);
  p.ws_lse = reinterpret_cast<float*>(ws + a.lse);
  p.ws_z = reinterpret_cast<float*>(ws + a.z);
  // bytes of a page's cached head: rows of hd * 2, in boxes of 128
  const uint64_t row = (uint64_t)cache->hd * 2, plane = row * cache->page_size;
  const uint32_t box = (uint32_t)std::min(cache->page_size, kPagedKeys);
  CUtensorMap tk, tv;
  for (int i = 0; i < 2; ++i)
    if (const dllm_status s = op_map_u8(i ? &tv : &tk, i ? cache->v : cache->k, row, cache->page_size,
                                        (uint64_t)cache->pages * cache->H_kv, row, plane, 128, box);
        s != DLLM_OK)
      return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (cache->dtype == DLLM_BF16)
    OP_CK((cache->hd == 64 ? launch_attn_paged<PairBf16, 64>(tk, tv, p, a, st)
                           : launch_attn_paged<PairBf16, 128>(tk, tv, p, a, st)));
  else
    OP_CK((cache->hd == 64 ? launch_attn_paged<PairF16, 64>(tk, tv, p, a, st)
                           : launch_attn_paged<PairF16, 128>(tk, tv, p, a, st)));
  return DLLM_OK;
}
