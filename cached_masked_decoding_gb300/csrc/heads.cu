// Head norms and rotary positions in one pass, with the cache's new rows:
//   y = x / sqrt(mean(x^2) + eps) * weight over each head, then its pairs turn
// by their position (rope.cuh); keys and values go to their pages.
//
// Bound by HBM: every element is read once and written once.  A lane owns 8
// pairs of a head - two 16-byte vectors of 16-bit elements, the members of a pair
// in one thread - so a head of 128 is 8 lanes and its mean three shuffles.  A thread
// keeps its head (its weights and addresses) over a run of rows, which come into a ring in shared memory
// by bulk copies, up to 64 KB ahead; the cosines and sines of up to 1024 pairs of rows to come
// are worked out at once, one a thread.
// 8191 rows of 32 + 8 heads of 128 in bf16 with their values to pages: 46.5 us, 4.3 TB/s; the same rows as they are,
// neither normalised nor turned, 35.6 (a plain copy of them 31.6).  Nothing is full there: DRAM 40 % of nominal, half of
// the issue slots, no pipe over a third.  Latency bounds it: 5.4 warps a scheduler, each with one row under way, wait 9
// cycles for every instruction they issue, for shared memory and shuffles, for the instruction before, for global memory
// and at barriers.
// 8 such rows: 3.5 us, a launch's latency.  Loads into registers instead of bulk copies: 56 us; three CTAs of 56
// registers a thread for two of 64: 46.1, but float32 rows of 16 heads 72 us for 66.
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
  int step, batch, run;                // rows of a CTA at once, with angles at hand, in all
  int chunk;                           // heads of a CTA
  int stages, row_bytes;               // of the ring, each `step` rows of a chunk's heads
  FastDiv by_chunk, by_R;
  int R;
  PagedKv c;
  uint64_t turns[kMaxPairs];           // turns per position * 2^64
};

constexpr int kHeadsAngles = 1024;     // pairs of a batch of rows
constexpr int kHeadsRows = 64;         // and most rows
constexpr int kHeadsStages = 8;
constexpr int kHeadsRing = 64 * 1024;

static __device__ int g_heads_err[1];

// E, O: element types in and out; L: lanes of a head (8 pairs each, some idle where hd / 16 is no power of two).
template <typename E, typename O, int L, bool PAGED>
__global__ void __launch_bounds__(512, 2) heads_kernel(const __grid_constant__ HeadsParams p) {
  using T = typename E::T;
  using TO = typename O::T;
  extern __shared__ __align__(16) uint8_t s_ring[];
  // [row][4][lanes]: cosines of a lane's first and last four pairs, then the sines
  __shared__ float4 s_cs[kHeadsAngles / 2];
  __shared__ long long s_slot[kHeadsRows];         // row of the cache's head 0, or -1: the row takes no part
  __shared__ float4 s_w[2][64];                    // q's and k's weights in the order of a lane's four vectors: [4][lanes]
  __shared__ uint64_t s_full[kHeadsStages], s_empty[kHeadsStages];
  __shared__ int s_abort;
  float* s_angle = reinterpret_cast<float*>(s_cs);
  const int row0 = blockIdx.x * p.run, rows = min(p.run, p.rows - row0), pairs = p.rot / 2, turners = pairs / 8;
  const int l = threadIdx.x % L, first = 8 * l;    // first: the lane's first pair
  // this thread's head, and its row of those taken at once
  uint32_t in_chunk;
  const int sub = (int)p.by_chunk.divmod(threadIdx.x / L, in_chunk);
  const int h = (int)(blockIdx.y * p.chunk + in_chunk);
  const bool mine = sub < p.step && h < p.heads && l * 16 < p.hd;
  const int kind = h < p.H ? 0 : h < p.H + p.H_kv ? 1 : 2;                     // q, k, v
  const int g = h - (kind == 0 ? 0 : kind == 1 ? p.H : p.H + p.H_kv);
  const bool turns = kind < 2 && first < pairs, norm = p.norm && kind < 2;
  // elements a and b: the pairs' members, or 16 in a row
  const int a = turns && !p.interleaved ? first : 2 * first, b = turns && !p.interleaved ? first + pairs : a + 8;
  TO* out = kind == 0 ? static_cast<TO*>(p.q_out) + (long long)g * p.hd
            : PAGED   ? reinterpret_cast<TO*>(kind == 1 ? p.c.k : p.c.v) + (((long long)g << p.c.page_shift)) * p.hd
                      : static_cast<TO*>(p.k_out) + (long long)g * p.hd;
  const long long out_rs = kind == 0 ? p.q_out_rs : p.k_out_rs;
  const int steps = (rows + p.step - 1) / p.step;
  if (threadIdx.x == 0) {
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], blockDim.x / 32);
    }
    s_abort = 0;
    fence_mbar_init();
  }
  // step k's rows to their stage, by one thread: the chunk's heads lie in up to three arrays
  auto fetch = [&](int k, int at) {
    const int r0 = k * p.step, n = min(p.step, rows - r0), h0 = blockIdx.y * p.chunk;
    const int h1 = min(h0 + p.chunk, p.heads);
    mbar_arrive_expect_tx(&s_full[at], (uint32_t)(n * (h1 - h0) * p.hd) * (uint32_t)sizeof(T));
    for (int r = 0; r < n; ++r) {
      const long long row = row0 + r0 + r;
      uint8_t* to = s_ring + (at * p.step + r) * p.row_bytes;
#pragma unroll
      for (int i = 0; i < (PAGED ? 3 : 2); ++i) {
        const int lo = i == 0 ? 0 : i == 1 ? p.H : p.H + p.H_kv, hi = lo + (i == 0 ? p.H : p.H_kv);
        const int from = max(lo, h0), until = min(hi, h1);
        if (from >= until) continue;
        const T* src = static_cast<const T*>(i == 0 ? p.q : i == 1 ? p.k : p.v) +
                       row * (i == 0 ? p.q_rs : i == 1 ? p.k_rs : p.v_rs) + (long long)(from - lo) * p.hd;
        bulk_load(to + (from - h0) * p.hd * (int)sizeof(T), src, (uint32_t)((until - from) * p.hd) * (uint32_t)sizeof(T),
                  &s_full[at]);
      }
    }
  };
  griddep_launch_dependents();
  griddep_wait();
  __syncthreads();
  int issued = min(p.stages, steps);               // steps under way or done (thread 0)
  if (threadIdx.x == 0)
    for (int k = 0; k < issued; ++k) fetch(k, k);
  const T* mine_at = reinterpret_cast<const T*>(s_ring) + (long long)sub * (p.row_bytes / (int)sizeof(T)) + in_chunk * p.hd;
  // a lane's elements a, a + 4, b, b + 4 and the three after each
  const bool weighted = p.norm && (p.q_w || p.k_w);
  if (weighted) {
    for (int e = threadIdx.x; e < 2 * p.hd; e += blockDim.x) {
      const int k = e / p.hd, d = e - k * p.hd;
      const T* w = static_cast<const T*>(k ? p.k_w : p.q_w);
      // element d: the lane and the vector that hold it
      int lane, at;
      if (!p.interleaved && d < p.rot) {
        const int i = d < pairs ? d : d - pairs;
        lane = i >> 3;
        at = (d < pairs ? 0 : 8) + (i & 7);
      } else {
        lane = d >> 4;
        at = d & 15;
      }
      reinterpret_cast<float*>(&s_w[k][(at >> 2) * L + lane])[at & 3] = w ? E::get(w + d) : 1.0f;
    }
  }
  const float4* w4 = s_w[kind == 1] + l;
  const int stage_elems = p.step * (p.row_bytes / (int)sizeof(T));
  int stage = 0, last = -1;                        // of the ring: this step's, and the step's before
  uint32_t phase = 0;

  for (int r0 = 0; r0 < rows; r0 += p.batch) {
    const int n = min(p.batch, rows - r0);
    if (r0 > 0) __syncthreads();
    for (int r = threadIdx.x; PAGED && r < n; r += blockDim.x) {
      uint32_t i;
      const int s = (int)p.by_R.divmod((uint32_t)(row0 + r0 + r), i);
      const int count = p.counts ? p.counts[s] : p.R;
      const long long at = (long long)(p.starts ? p.starts[s] : 0) + i;
      long long slot = -1;
      if ((int)i < count && at >= 0 && at < p.c.positions) {
        const int page = p.c.table[(long long)s * p.c.max_pages + (at >> p.c.page_shift)];
        if ((unsigned)page < (unsigned)p.c.pages)
          slot = (((long long)page * p.H_kv) << p.c.page_shift) + (at & ((1 << p.c.page_shift) - 1));
      }
      s_slot[r] = slot;
    }
    for (int e = threadIdx.x; e < n * pairs; e += blockDim.x) {
      const int r = e / pairs, i = e - r * pairs, row = row0 + r0 + r;
      int pos = 0;
      if (p.pos) {
        pos = p.pos[row];
      } else if (PAGED) {                           // its place in the cache
        uint32_t k;
        const int s = (int)p.by_R.divmod((uint32_t)row, k);
        pos = (int)((p.starts ? p.starts[s] : 0) + (long long)k);
      }
      float c, s;
      turn_cos_sin(p.turns[i], pos, p.amp, c, s);
      float* to = s_angle + ((r * 4 + ((i >> 2) & 1)) * turners + (i >> 3)) * 4 + (i & 3);
      to[0] = c;
      to[8 * turners] = s;
    }
    __syncthreads();
    for (int k = 0; k < n; k += p.step) {
      const int r = k + sub;
      mbar_wait(&s_full[stage], phase, &s_abort, g_heads_err, ERR_HEADS);
      // the head's elements in pairs of neighbours
      uint64_t va[4] = {}, vb[4] = {};
      if (mine && r < n) {
        const T* src = mine_at + stage * stage_elems;
        float f[8];
        E::load8(src + a, f);
#pragma unroll
        for (int e = 0; e < 4; ++e) va[e] = f32x2(f[2 * e], f[2 * e + 1]);
        E::load8(src + b, f);
#pragma unroll
        for (int e = 0; e < 4; ++e) vb[e] = f32x2(f[2 * e], f[2 * e + 1]);
      }
      __syncwarp();
      if (threadIdx.x % 32 == 0) mbar_arrive(&s_empty[stage]);
      // the stage of the step before takes the rows that come `stages` behind it
      if (threadIdx.x == 0 && last >= 0 && issued < steps &&
          mbar_wait(&s_empty[last], last < stage ? phase : phase ^ 1u, &s_abort, g_heads_err, ERR_HEADS)) {
        fetch(issued, last);
        ++issued;
      }
      __syncwarp();
      last = stage;
      if (++stage == p.stages) {
        stage = 0;
        phase ^= 1u;
      }
      float inv = 1.0f;
      if (p.norm) {
        uint64_t sq = mul_f32x2(va[0], va[0]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (e > 0) sq = fma_f32x2(va[e], va[e], sq);
          sq = fma_f32x2(vb[e], vb[e], sq);
        }
        const float2 h2 = f32x2_get(sq);
        float sum = h2.x + h2.y;
#pragma unroll
        for (int d = L / 2; d >= 1; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        if (norm) inv = rsqrtf(sum * p.inv_hd + p.eps);
      }
      if (!mine || r >= n) continue;
      const long long slot = PAGED ? s_slot[r] : 0;
      if (PAGED && slot < 0) continue;
      if (norm) {
        const uint64_t inv2 = f32x2(inv, inv);
        if (weighted) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float4 f = w4[e * L], g4 = w4[(2 + e) * L];
            va[2 * e] = mul_f32x2(va[2 * e], f32x2(f.x, f.y));
            va[2 * e + 1] = mul_f32x2(va[2 * e + 1], f32x2(f.z, f.w));
            vb[2 * e] = mul_f32x2(vb[2 * e], f32x2(g4.x, g4.y));
            vb[2 * e + 1] = mul_f32x2(vb[2 * e + 1], f32x2(g4.z, g4.w));
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          va[e] = mul_f32x2(va[e], inv2);
          vb[e] = mul_f32x2(vb[e], inv2);
        }
      }
      if (turns) {
        const float4* cs = s_cs + r * 4 * turners + l;
        if (p.interleaved) {
          const float4 c0 = cs[0], c1 = cs[turners], s0 = cs[2 * turners], s1 = cs[3 * turners];
          const float c[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
          const float s[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 x = f32x2_get(va[e]), y = f32x2_get(vb[e]);
            va[e] = f32x2(x.x * c[e] - x.y * s[e], x.y * c[e] + x.x * s[e]);
            vb[e] = f32x2(y.x * c[e + 4] - y.y * s[e + 4], y.y * c[e + 4] + y.x * s[e + 4]);
          }
        } else {
          const uint64_t minus = f32x2(-1.0f, -1.0f);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int at = (e >> 1) * turners;
            const float4 c4 = cs[at], s4 = cs[2 * turners + at];
            const uint64_t c = e & 1 ? f32x2(c4.z, c4.w) : f32x2(c4.x, c4.y);
            const uint64_t s = e & 1 ? f32x2(s4.z, s4.w) : f32x2(s4.x, s4.y);
            const uint64_t x0 = va[e], x1 = vb[e];
            va[e] = fma_f32x2(x0, c, mul_f32x2(mul_f32x2(x1, s), minus));
            vb[e] = fma_f32x2(x1, c, mul_f32x2(x0, s));
          }
        }
      }
      TO* to = out + (kind == 0 || !PAGED ? (row0 + r0 + r) * out_rs : slot * p.hd);
      float f[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 x = f32x2_get(va[e]);
        f[2 * e] = x.x;
        f[2 * e + 1] = x.y;
      }
      O::store8(to + a, f);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 x = f32x2_get(vb[e]);
        f[2 * e] = x.x;
        f[2 * e + 1] = x.y;
      }
      O::store8(to + b, f);
    }
  }
  if (threadIdx.x == 0 && *(volatile int*)&s_abort)   // let copies in flight land before the CTA's shared memory goes away
    for (int k = max(issued - p.stages, 0); k < issued; ++k)
      mbar_wait(&s_full[k % p.stages], (uint32_t)(k / p.stages) & 1u, nullptr, g_heads_err, ERR_HEADS);
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

cudaError_t heads_err_word(int** p) { return cudaGetSymbolAddress(reinterpret_cast<void**>(p), g_heads_err); }

namespace {

template <typename E, typename O, int L, bool PAGED>
cudaError_t launch_heads(const HeadsParams& p, dim3 grid, dim3 block, cudaStream_t st) {
  const cudaError_t e = op_smem_once(reinterpret_cast<const void*>(heads_kernel<E, O, L, PAGED>), kHeadsRing);
  if (e != cudaSuccess) return e;
  return op_launch(heads_kernel<E, O, L, PAGED>, grid, block, (size_t)p.stages * p.step * p.row_bytes, st, 1, p);
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
  if (!p.q || !p.k || !p.q_out || (paged ? !p.v : !p.k_out) || p.rows < 1 || p.rows > kMostRows || p.H < 1 || p.H_kv < 1 || es == 0 ||
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
  if (heads > (1 << 20)) return op_fail(DLLM_EINVAL, "%s: H=%d H_kv=%d are too many heads", who, p.H, p.H_kv);
  p.heads = (int)heads;
  // heads of a CTA: up to 512 threads' worth, in equal chunks; rows at once: as many as give 256 threads a head each
  const int chunks = (int)((heads * lanes + 511) / 512);
  p.chunk = (int)((heads + chunks - 1) / chunks);
  p.by_chunk = FastDiv((uint32_t)p.chunk);
  const int pairs = p.rot / 2, sms = op_device_sms();
  p.step = 1;
  while (2 * p.step * p.chunk * lanes <= 256 && 2 * p.step * pairs <= kHeadsAngles && 2 * p.step <= kHeadsRows &&
         p.rows / (2 * p.step) >= sms)
    p.step *= 2;
  const int threads = (p.step * p.chunk * lanes + 31) / 32 * 32;
  // rows of a CTA: as few as leave every SM its threads
  const long long ctas = std::max(1LL, (long long)sms * (1024 / threads) / chunks);
  p.run = (int)(((p.rows + ctas - 1) / ctas + p.step - 1) / p.step * p.step);
  p.batch = std::min(p.run, std::min(kHeadsRows, pairs ? kHeadsAngles / pairs : kHeadsRows) / p.step * p.step);
  p.row_bytes = p.chunk * p.hd * es;                    // 32 KB at most
  p.stages = std::min({kHeadsStages, kHeadsRing / (p.step * p.row_bytes), (p.run + p.step - 1) / p.step});
  const dim3 grid((unsigned)(((long long)p.rows + p.run - 1) / p.run), (unsigned)chunks), block((unsigned)threads);
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
