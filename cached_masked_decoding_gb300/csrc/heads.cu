// Head norms and rotary positions in one pass, with the cache's new rows:
//   y = x / sqrt(mean(x^2) + eps) * weight over each head, then its pairs turn
// by their position (rope.cuh); keys and values go to their pages.
//
// Bound by HBM: every element is read once and written once.  A lane owns 8
// pairs of a head - two 16-byte vectors of 16-bit elements, the members of a pair
// in one thread - so a head of 128 is 8 lanes and its mean three shuffles.  A CTA
// takes whole rows: their cosines and sines are worked out once, by one thread a
// pair, while the first elements are on their way.
#include <algorithm>

#include "kv_paged.h"
#include "ptx8.cuh"
#include "q8.cuh"
#include "rope.cuh"

namespace dllm {

struct HeadsParams {
  const void *q, *k, *v;               // v: paged only
  void *q_out, *k_out;
  long long q_rs, k_rs, v_rs, q_out_rs, k_out_rs;
  const int32_t *pos, *starts, *counts;
  const void *q_w, *k_w;
  float eps, amp, inv_hd;
  int norm, rot, interleaved;
  int rows, H, H_kv, hd, heads;        // heads: of a row, over q, k and (paged) v
  int row_run;                         // rows of a CTA
  FastDiv by_heads, by_R;
  int R;
  PagedKv c;
  uint64_t turns[kMaxPairs];           // turns per position * 2^64
};

constexpr int kHeadsAngles = 1024;     // pairs of a CTA's rows
constexpr int kHeadsRows = 64;         // and most rows

// E, O: element types in and out; L: lanes of a head (8 pairs each, some idle where hd / 16 is no power of two).
template <typename E, typename O, int L, bool PAGED>
__global__ void __launch_bounds__(512, sizeof(typename E::T) == 2 ? 2 : 1)
    heads_kernel(const __grid_constant__ HeadsParams p) {
  using T = typename E::T;
  using TO = typename O::T;
  constexpr int ITEMS = 2;                         // heads of a thread in flight
  __shared__ float2 s_cs[kHeadsAngles];            // [row][pair] cosine and sine
  __shared__ long long s_slot[kHeadsRows];         // row of the cache's head 0, or -1: the row takes no part
  const int row0 = blockIdx.x * p.row_run, n_rows = min(p.row_run, p.rows - row0), pairs = p.rot / 2;
  const int l = threadIdx.x % L, group = threadIdx.x / L, groups = blockDim.x / L;
  const int items = n_rows * p.heads, first = 8 * l;   // first: the lane's first pair
  griddep_launch_dependents();
  griddep_wait();

  struct Item {
    Raw8<E> a, b;
    int r, kind, g;                                // row of the CTA; q, k, v; head
    bool on;
    __device__ __forceinline__ bool turns(int first, int pairs) const { return kind < 2 && first < pairs; }
  };
  // elements a and b: the pairs' members, or 16 in a row
  auto at_a = [&](bool turns) { return turns && !p.interleaved ? first : 2 * first; };
  auto at_b = [&](bool turns) { return turns && !p.interleaved ? first + pairs : 2 * first + 8; };
  auto load = [&](Item& x, int it) {
    x.on = it < items && l * 16 < p.hd;
    uint32_t h = 0;
    x.r = x.on ? (int)p.by_heads.divmod((uint32_t)it, h) : 0;
    x.kind = (int)h < p.H ? 0 : (int)h < p.H + p.H_kv ? 1 : 2;
    x.g = (int)h - (x.kind == 0 ? 0 : x.kind == 1 ? p.H : p.H + p.H_kv);
    if (!x.on) return;
    const long long row = row0 + x.r;
    const T* src = (x.kind == 0   ? static_cast<const T*>(p.q) + row * p.q_rs
                    : x.kind == 1 ? static_cast<const T*>(p.k) + row * p.k_rs
                                  : static_cast<const T*>(p.v) + row * p.v_rs) +
                   (long long)x.g * p.hd;
    const bool t = x.turns(first, pairs);
    x.a.load(src + at_a(t));
    x.b.load(src + at_b(t));
  };
  auto finish = [&](const Item& x) {
    float va[8], vb[8];
    const bool on = x.on && (!PAGED || s_slot[x.r] >= 0), turns = x.turns(first, pairs);
    if (on) {
      x.a.floats(va);
      x.b.floats(vb);
    }
    if (p.norm) {
      float sum = 0.0f;
      if (on) {
#pragma unroll
        for (int e = 0; e < 8; ++e) sum += va[e] * va[e] + vb[e] * vb[e];
      }
#pragma unroll
      for (int d = L / 2; d >= 1; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      if (on && x.kind < 2) {
        const float inv = 1.0f / sqrtf(sum * p.inv_hd + p.eps);
        const T* w = static_cast<const T*>(x.kind == 0 ? p.q_w : p.k_w);
        float wa[8], wb[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) wa[e] = wb[e] = 1.0f;
        if (w) {
          E::load8(w + at_a(turns), wa);
          E::load8(w + at_b(turns), wb);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          va[e] = va[e] * inv * wa[e];
          vb[e] = vb[e] * inv * wb[e];
        }
      }
    }
    if (!on) return;
    if (turns) {
      const float2* cs = s_cs + x.r * pairs + first;
      if (p.interleaved) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float a0 = va[2 * e], a1 = va[2 * e + 1], b0 = vb[2 * e], b1 = vb[2 * e + 1];
          va[2 * e] = a0 * cs[e].x - a1 * cs[e].y;
          va[2 * e + 1] = a1 * cs[e].x + a0 * cs[e].y;
          vb[2 * e] = b0 * cs[e + 4].x - b1 * cs[e + 4].y;
          vb[2 * e + 1] = b1 * cs[e + 4].x + b0 * cs[e + 4].y;
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float x0 = va[e], x1 = vb[e];
          va[e] = x0 * cs[e].x - x1 * cs[e].y;
          vb[e] = x1 * cs[e].x + x0 * cs[e].y;
        }
      }
    }
    const long long row = row0 + x.r;
    TO* out;
    if (x.kind == 0)
      out = static_cast<TO*>(p.q_out) + row * p.q_out_rs + (long long)x.g * p.hd;
    else if constexpr (PAGED)
      out = reinterpret_cast<TO*>(x.kind == 1 ? p.c.k : p.c.v) + (s_slot[x.r] + ((long long)x.g << p.c.page_shift)) * p.hd;
    else
      out = static_cast<TO*>(p.k_out) + row * p.k_out_rs + (long long)x.g * p.hd;
    O::store8(out + at_a(turns), va);
    O::store8(out + at_b(turns), vb);
  };

  // the first heads on their way while the rows' places and angles are worked out
  Item x[ITEMS];
#pragma unroll
  for (int k = 0; k < ITEMS; ++k) load(x[k], group + k * groups);
  for (int r = threadIdx.x; PAGED && r < n_rows; r += blockDim.x) {
    uint32_t i;
    const int s = (int)p.by_R.divmod((uint32_t)(row0 + r), i);
    const int n = p.counts ? p.counts[s] : p.R;
    const long long at = (long long)(p.starts ? p.starts[s] : 0) + i;
    long long slot = -1;
    if ((int)i < n && at >= 0 && at < p.c.positions) {
      const int page = p.c.table[(long long)s * p.c.max_pages + (at >> p.c.page_shift)];
      if ((unsigned)page < (unsigned)p.c.pages)
        slot = (((long long)page * p.H_kv) << p.c.page_shift) + (at & ((1 << p.c.page_shift) - 1));
    }
    s_slot[r] = slot;
  }
  for (int a = threadIdx.x; a < n_rows * pairs; a += blockDim.x) {
    const int r = a / pairs, i = a - r * pairs;
    int pos = 0;
    if (p.pos) {
      pos = p.pos[row0 + r];
    } else if (PAGED) {                             // its place in the cache
      uint32_t k;
      const int s = (int)p.by_R.divmod((uint32_t)(row0 + r), k);
      pos = (int)((p.starts ? p.starts[s] : 0) + (long long)k);
    }
    float c, s;
    turn_cos_sin(p.turns[i], pos, p.amp, c, s);
    s_cs[a] = make_float2(c, s);
  }
  __syncthreads();
  for (int base = 0; base < items; base += ITEMS * groups) {
    if (base > 0) {
#pragma unroll
      for (int k = 0; k < ITEMS; ++k) load(x[k], base + group + k * groups);
    }
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) finish(x[k]);
  }
}

dllm_status kv_paged_check(const dllm_kv_paged* c, const char* who) {
  if (!c || !c->k || !c->v || !c->table || c->b < 1 || c->H_kv < 1 || (c->hd != 64 && c->hd != 128) ||
      (c->dtype != DLLM_BF16 && c->dtype != DLLM_F16) || c->pages < 1 || c->page_size < 16 || c->page_size > 256 ||
      (c->page_size & (c->page_size - 1)) || c->max_pages < 1 || !op_aligned(c->k, 16) || !op_aligned(c->v, 16) ||
      !op_aligned(c->table, 4))
    return op_fail(DLLM_EINVAL,
                   "%s: bad paged cache (b, H_kv, pages, max_pages >= 1, hd 64 or 128, bf16 or f16, page_size a power "
                   "of two, 16..256, k and v 16-byte aligned)%s",
                   who, c ? "" : ": null");
  if ((long long)c->max_pages * c->page_size > kMostRows || (long long)c->pages * c->H_kv > kMostRows ||
      (__int128)c->pages * c->H_kv * c->page_size > ((__int128)1 << 44))
    return op_fail(DLLM_EINVAL, "%s: a cache of %d pages of %d positions, H_kv=%d, %d pages a sequence is too large", who,
                   c->pages, c->page_size, c->H_kv, c->max_pages);
  return DLLM_OK;
}

namespace {

template <typename E, typename O, int L, bool PAGED>
cudaError_t launch_heads(const HeadsParams& p, dim3 grid, dim3 block, cudaStream_t st) {
  return op_launch(heads_kernel<E, O, L, PAGED>, grid, block, 0, st, 1, p);
}

template <typename E, typename O>
cudaError_t launch_heads(const HeadsParams& p, bool paged, int lanes, dim3 grid, dim3 block, cudaStream_t st) {
  if constexpr (sizeof(typename O::T) == 2)
    if (paged)
      return lanes == 4 ? launch_heads<E, O, 4, true>(p, grid, block, st) : launch_heads<E, O, 8, true>(p, grid, block, st);
  switch (lanes) {
    case 1: return launch_heads<E, O, 1, false>(p, grid, block, st);
    case 2: return launch_heads<E, O, 2, false>(p, grid, block, st);
    case 4: return launch_heads<E, O, 4, false>(p, grid, block, st);
    case 8: return launch_heads<E, O, 8, false>(p, grid, block, st);
    default: return launch_heads<E, O, 16, false>(p, grid, block, st);
  }
}

// Checks and launches what both entries share; p has the pointers, strides (0: dense) and sizes.
dllm_status heads(HeadsParams& p, const char* who, bool paged, int dtype, int out_dtype, const dllm_rope* r,
                  void* stream) {
  const int es = op_dtype_size(dtype), os = op_dtype_size(out_dtype);
  if (!p.q || !p.k || !p.q_out || (paged ? !p.v : !p.k_out) || p.rows < 1 || p.H < 1 || p.H_kv < 1 || es == 0 ||
      os == 0 || (dtype != out_dtype && dtype != DLLM_F32) || p.hd < 16 || p.hd > 256 || p.hd % 16)
    return op_fail(DLLM_EINVAL,
                   "bad %s arguments: rows=%d H=%d H_kv=%d hd=%d (a multiple of 16, to 256) dtype=%d out_dtype=%d "
                   "(the same, or 16 bits from float32)",
                   who, p.rows, p.H, p.H_kv, p.hd, dtype, out_dtype);
  for (const void* x : {p.q, p.k, p.v, (const void*)p.q_out, (const void*)p.k_out, p.q_w, p.k_w})
    if (!op_aligned(x, 16)) return op_fail(DLLM_EINVAL, "%s: arrays must be 16-byte aligned", who);
  if (!op_aligned(p.pos, 4) || !op_aligned(p.starts, 4) || !op_aligned(p.counts, 4))
    return op_fail(DLLM_EINVAL, "%s: positions, starts and counts must be 4-byte aligned", who);
  if (!(p.eps < 0.0f) && !(p.eps >= 0.0f && p.eps <= 3e38f))
    return op_fail(DLLM_EINVAL, "%s: bad eps %g", who, p.eps);
  p.norm = p.eps >= 0.0f;
  if (!p.norm && (p.q_w || p.k_w)) return op_fail(DLLM_EINVAL, "%s: weights without a norm (eps=%g < 0)", who, p.eps);
  p.inv_hd = 1.0f / (float)p.hd;
  struct Stride { long long* rs; long long width; int es; const char* name; };
  const long long wq = (long long)p.H * p.hd, wk = (long long)p.H_kv * p.hd;
  for (const Stride& s : {Stride{&p.q_rs, wq, es, "q"}, Stride{&p.k_rs, wk, es, "k"}, Stride{&p.v_rs, wk, es, "v"},
                          Stride{&p.q_out_rs, wq, os, "q_out"}, Stride{&p.k_out_rs, wk, os, "k_out"}}) {
    if (*s.rs == 0) *s.rs = s.width;
    if (*s.rs < s.width || *s.rs > (1LL << 40) || (*s.rs * s.es) % 16)
      return op_fail(DLLM_EINVAL, "%s: %s row stride %lld (0, or at least %lld and a multiple of 16 bytes)", who, s.name,
                     *s.rs, s.width);
  }
  if ((p.q == p.q_out && (dtype != out_dtype || p.q_rs != p.q_out_rs)) ||
      (!paged && p.k == p.k_out && (dtype != out_dtype || p.k_rs != p.k_out_rs)))
    return op_fail(DLLM_EINVAL, "%s: in place needs the same type and stride on both sides", who);
  if (r) {
    if (const dllm_status st = rope_turns(r, p.hd, p.turns, &p.amp); st != DLLM_OK) return st;
    if (r->rot_dim % 16) return op_fail(DLLM_EINVAL, "%s: rot_dim=%d is no multiple of 16", who, r->rot_dim);
    if (!paged && !p.pos) return op_fail(DLLM_EINVAL, "%s: positions are missing", who);
    p.rot = r->rot_dim;
    p.interleaved = r->layout == DLLM_ROPE_INTERLEAVED;
  }
  const long long heads = (long long)p.H + (paged ? 2LL : 1LL) * p.H_kv;
  int lanes = 1;
  while (lanes * 16 < p.hd) lanes *= 2;
  if (heads > (1 << 24)) return op_fail(DLLM_EINVAL, "%s: H=%d H_kv=%d are too many heads", who, p.H, p.H_kv);
  p.heads = (int)heads;
  p.by_heads = FastDiv((uint32_t)heads);
  // rows of a CTA: as many as give 256 threads two heads each, where that leaves the GPU's SMs a CTA each
  p.row_run = 1;
  while (p.row_run < kHeadsRows && 2 * p.row_run * heads * lanes <= 512 && 2 * p.row_run * (p.rot / 2) <= kHeadsAngles &&
         p.rows / (2 * p.row_run) >= op_device_sms())
    p.row_run *= 2;
  const bool few = p.rows <= 2 * op_device_sms();       // a head a thread: its latency counts
  const long long threads = std::min(512LL, (p.row_run * heads * lanes / (few ? 1 : 2) + 31) / 32 * 32);
  const dim3 grid((unsigned)((p.rows + p.row_run - 1) / p.row_run)), block((unsigned)threads);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == DLLM_BF16)
    OP_CK((launch_heads<ElemBf16, ElemBf16>(p, paged, lanes, grid, block, st)));
  else if (dtype == DLLM_F16)
    OP_CK((launch_heads<ElemF16, ElemF16>(p, paged, lanes, grid, block, st)));
  else if (out_dtype == DLLM_BF16)
    OP_CK((launch_heads<ElemF32, ElemBf16>(p, paged, lanes, grid, block, st)));
  else if (out_dtype == DLLM_F16)
    OP_CK((launch_heads<ElemF32, ElemF16>(p, paged, lanes, grid, block, st)));
  else
    OP_CK((launch_heads<ElemF32, ElemF32>(p, paged, lanes, grid, block, st)));
  return DLLM_OK;
}

}  // namespace
}  // namespace dllm

using namespace dllm;

extern "C" dllm_status dllm_op_qk_norm_rope(const void* q, int64_t q_row_stride, const void* k, int64_t k_row_stride,
                                            void* q_out, int64_t q_out_row_stride, void* k_out,
                                            int64_t k_out_row_stride, const int32_t* positions, int32_t rows, int32_t H,
                                            int32_t H_kv, int32_t hd, int32_t dtype, int32_t out_dtype,
                                            const void* q_weight, const void* k_weight, float eps,
                                            const dllm_rope* rope, void* stream) {
  HeadsParams p = {};
  p.q = q;
  p.k = k;
  p.q_out = q_out;
  p.k_out = k_out;
  p.q_rs = q_row_stride;
  p.k_rs = k_row_stride;
  p.q_out_rs = q_out_row_stride;
  p.k_out_rs = k_out_row_stride;
  p.pos = positions;
  p.rows = rows;
  p.H = H;
  p.H_kv = H_kv;
  p.hd = hd;
  p.q_w = q_weight;
  p.k_w = k_weight;
  p.eps = eps;
  return heads(p, "qk_norm_rope", false, dtype, out_dtype, rope, stream);
}

extern "C" dllm_status dllm_op_qk_norm_rope_paged(const dllm_kv_paged* cache, const void* q, int64_t q_row_stride,
                                                  const void* k, int64_t k_row_stride, const void* v,
                                                  int64_t v_row_stride, void* q_out, int64_t q_out_row_stride,
                                                  int32_t H, int32_t R, int32_t dtype, const int32_t* starts,
                                                  const int32_t* counts, const int32_t* positions,
                                                  const void* q_weight, const void* k_weight, float eps,
                                                  const dllm_rope* rope, void* stream) {
  if (const dllm_status s = kv_paged_check(cache, "qk_norm_rope_paged"); s != DLLM_OK) return s;
  if (R < 1 || (long long)cache->b * R > kMostRows)
    return op_fail(DLLM_EINVAL, "qk_norm_rope_paged: bad R=%d for b=%d", R, cache->b);
  HeadsParams p = {};
  p.c = PagedKv(*cache);
  p.q = q;
  p.k = k;
  p.v = v;
  p.q_out = q_out;
  p.q_rs = q_row_stride;
  p.k_rs = k_row_stride;
  p.v_rs = v_row_stride;
  p.q_out_rs = q_out_row_stride;
  p.pos = positions;
  p.starts = starts;
  p.counts = counts;
  p.rows = cache->b * R;
  p.R = R;
  p.by_R = FastDiv((uint32_t)R);
  p.H = H;
  p.H_kv = cache->H_kv;
  p.hd = cache->hd;
  p.q_w = q_weight;
  p.k_w = k_weight;
  p.eps = eps;
  return heads(p, "qk_norm_rope_paged", true, dtype, cache->dtype, rope, stream);
}
