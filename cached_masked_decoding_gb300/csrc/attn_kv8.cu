// Attention over the 8-bit cache:
//   out[s, i, h] = sum_t p_t V[s, g, t],  p = softmax over t < limit[s, i] of
//   scale * q[s, i, h] . K[s, g, t],      g = h / (H / H_kv)
// K = k * 2^ek and V = v * 2^ev with one exponent a row.  A row whose limit is
// 0 or less sees nothing and gives zeros.  The kernels are in attn_kv8_rows.cuh
// (up to 64 rows a cached head) and attn_kv8_tiles.cuh (more);
// here is which runs, and on what.
#include <algorithm>
#include <cmath>

#include "attn_kv8_tiles.cuh"

namespace dllm {

dllm_status kv8_check(const dllm_kv8* c, const char* who);

cudaError_t attn_kv8_err_word(int** p) { return cudaGetSymbolAddress(reinterpret_cast<void**>(p), g_attn_kv8_err); }

namespace {

constexpr int kMaxCluster = 8;   // portable cluster size

struct AttnKv8Plan {
  int N, row_tiles, splits, cluster;
  long long items;
  size_t ws_bytes;
};

// Rows of one cached head (R rows of H / H_kv heads) in tiles of N, the keys in
// splits.  256 rows in place of 128 once they are more (192 rows of 64 items, 4096 keys: 54
// us against 66; 8192 causal rows of 8 items, 2048 keys: 50 against 64).  A CTA's time
// is taken as the tiles of keys that it walks; the join of up
// to 8 splits in a cluster as one tile's, that of more (or of 128 rows and up) through the
// workspace as four of 128 keys.  A round of CTAs is two an SM, one with 64 or 256 rows.
AttnKv8Plan plan_attn_kv8(long long b, long long H_kv, long long rows, int hd, int T) {
  AttnKv8Plan a;
  a.N = rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : rows <= 128 ? 128 : 256;
  a.row_tiles = (int)((rows + a.N - 1) / a.N);
  a.items = b * H_kv * a.row_tiles;
  const long long kt = a.N >= 128 ? 64 : 128, tiles = (T + kt - 1) / kt;
  const long long ctas = (a.N == 64 || a.N == 256 ? 1 : 2) * op_device_sms();
  long long best = (a.items + ctas - 1) / ctas * tiles;
  a.splits = 1;
  for (long long s = 2; s <= std::min(tiles, 64LL) && s * a.items <= ctas; ++s) {
    const long long t = (tiles + s - 1) / s + (a.N >= 128 ? 8 : s <= kMaxCluster ? 1 : 4);
    if (t < best) {
      best = t;
      a.splits = (int)s;
    }
  }
  a.cluster = a.N < 128 && a.splits > 1 && a.splits <= kMaxCluster;
  a.ws_bytes = a.splits > 1 && !a.cluster ? (size_t)a.items * a.splits * a.N * (hd + 2) * 4 : 0;
  return a;
}

template <int HD, int N>
cudaError_t launch_attn_rows(const CUtensorMap& tk, const CUtensorMap& tv, const AttnKv8Params& p, unsigned grid,
                             cudaStream_t st) {
  using C = AttnRowsCfg<HD, N>;
  const cudaError_t e = op_smem_once(reinterpret_cast<const void*>(attn_kv8_rows_kernel<HD, N>), C::SMEM_BYTES);
  if (e != cudaSuccess) return e;
  return op_launch(attn_kv8_rows_kernel<HD, N>, dim3(grid), dim3(C::THREADS), C::SMEM_BYTES, st,
                   p.cluster ? p.splits : 1, tk, tv, p);
}

template <int HD, int SUBS>
cudaError_t launch_attn_tiles(const CUtensorMap& tk, const CUtensorMap& tv, const AttnKv8Params& p, unsigned grid,
                              cudaStream_t st) {
  using C = AttnTilesCfg<HD, SUBS>;
  const cudaError_t e = op_smem_once(reinterpret_cast<const void*>(attn_kv8_tiles_kernel<HD, SUBS>), C::SMEM_BYTES);
  if (e != cudaSuccess) return e;
  return op_launch(attn_kv8_tiles_kernel<HD, SUBS>, dim3(grid), dim3(C::THREADS), C::SMEM_BYTES, st, 1, tk, tv, p);
}

template <int HD>
cudaError_t launch_attn(const CUtensorMap& tk, const CUtensorMap& tv, const AttnKv8Params& p, const AttnKv8Plan& a,
                        cudaStream_t st) {
  const unsigned grid = (unsigned)(a.items * a.splits);
  cudaError_t e = a.N == 8    ? launch_attn_rows<HD, 8>(tk, tv, p, grid, st)
                  : a.N == 16 ? launch_attn_rows<HD, 16>(tk, tv, p, grid, st)
                  : a.N == 32 ? launch_attn_rows<HD, 32>(tk, tv, p, grid, st)
                  : a.N == 64 ? launch_attn_rows<HD, 64>(tk, tv, p, grid, st)
                  : a.N == 128 ? launch_attn_tiles<HD, 1>(tk, tv, p, grid, st)
                               : launch_attn_tiles<HD, 2>(tk, tv, p, grid, st);
  if (e != cudaSuccess || a.splits == 1 || a.cluster) return e;
  const long long rows = (long long)p.c.b * p.R * p.H;
  return op_launch(attn_kv8_join_kernel<HD>, dim3((unsigned)((rows + 3) / 4)), dim3(128), 0, st, 1, p, a.N);
}

}  // namespace
}  // namespace dllm

using namespace dllm;

extern "C" dllm_status dllm_op_attention_kv8_workspace(int32_t b, int32_t H, int32_t H_kv, int32_t hd, int32_t R,
                                                       int32_t T, int64_t* bytes) {
  if (!bytes || b < 1 || H < 1 || H_kv < 1 || H % H_kv || (hd != 64 && hd != 128) || R < 1 || T < 1 ||
      T > kMostRows)
    return op_fail(DLLM_EINVAL, "bad attention shape: b=%d H=%d H_kv=%d hd=%d R=%d T=%d", b, H, H_kv, hd, R, T);
  const long long rows = (long long)R * (H / H_kv);
  if (rows > (1LL << 30) || (__int128)b * R * H > 0x7fffffff)
    return op_fail(DLLM_EINVAL, "attention_kv8: b=%d R=%d H=%d are too many rows", b, R, H);
  *bytes = (int64_t)plan_attn_kv8(b, H_kv, rows, hd, T).ws_bytes;
  return DLLM_OK;
}

extern "C" dllm_status dllm_op_attention_kv8(const uint16_t* q, int64_t q_row_stride, const dllm_kv8* cache,
                                             const int32_t* limits, float scale, uint16_t* out,
                                             int64_t out_row_stride, int32_t H, int32_t R, void* workspace,
                                             int64_t workspace_bytes, void* stream) {
  if (const dllm_status s = kv8_check(cache, "attention_kv8"); s != DLLM_OK) return s;
  if (!q || !out || H < 1 || H % cache->H_kv || R < 1 || !(scale > 0.0f) || !(scale <= 1e30f) ||
      !op_aligned(q, 16) || !op_aligned(out, 16) || !op_aligned(limits, 4))
    return op_fail(DLLM_EINVAL,
                   "bad attention_kv8 arguments: H=%d (a multiple of H_kv=%d) R=%d scale=%g (over 0, to 1e30), "
                   "q and out 16-byte aligned",
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
  p.by_group = FastDiv((uint32_t)p.group);
  p.by_heads = FastDiv((uint32_t)cache->H_kv);
  p.scale_log2 = scale * 1.4426950408889634f;
  int64_t need = 0;
  if (const dllm_status s = dllm_op_attention_kv8_workspace(cache->b, H, cache->H_kv, cache->hd, R, cache->T, &need);
      s != DLLM_OK)
    return s;
  if (need > 0 && (!workspace || workspace_bytes < need || !op_aligned(workspace, 16)))
    return op_fail(DLLM_EINVAL, "attention_kv8: a 16-byte aligned workspace of %lld bytes is needed, got %lld",
                   (long long)need, workspace ? (long long)workspace_bytes : 0LL);
  p.rows = R * p.group;
  const AttnKv8Plan a = plan_attn_kv8(cache->b, cache->H_kv, p.rows, cache->hd, cache->T);
  p.row_tiles = a.row_tiles;
  p.splits = a.splits;
  p.by_splits = FastDiv((uint32_t)a.splits);
  p.by_tiles = FastDiv((uint32_t)(a.N < 128 ? a.row_tiles : cache->b * cache->H_kv));
  p.cluster = a.cluster;
  p.ws_o = static_cast<float*>(workspace);
  p.ws_ml = p.ws_o + (a.ws_bytes ? a.items * a.splits * a.N * cache->hd : 0);
  const uint64_t planes = (uint64_t)cache->b * cache->H_kv, plane = (uint64_t)cache->T * cache->hd;
  const uint32_t keys = a.N >= 128 ? 64 : 128;            // of a tile
  CUtensorMap tk, tv;
  if (const dllm_status s = op_map_u8(&tk, cache->k, cache->hd, cache->T, planes, cache->hd, plane, cache->hd, keys);
      s != DLLM_OK)
    return s;
  if (const dllm_status s = op_map_u8(&tv, cache->v, cache->hd, cache->T, planes, cache->hd, plane, cache->hd, keys);
      s != DLLM_OK)
    return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  OP_CK(cache->hd == 64 ? launch_attn<64>(tk, tv, p, a, st) : launch_attn<128>(tk, tv, p, a, st));
  return DLLM_OK;
}
