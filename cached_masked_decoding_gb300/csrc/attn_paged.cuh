// Attention over a paged cache for few query rows a cached head (a token, a block, grouped heads).
//
// Keys are the 128-row operand, so K and V go from HBM to the tensor cores as they are.  A tile of 128 keys gives
//   S^T[key][row] = K Q^T,      O^T[dim][row] += V^T P^T        (tcgen05, kind::f16)
// with N = 8, 16, 32 or 64 rows as the narrow operand (8: scores in 16 columns).  V is read MN-major from its
// TMA tile.  A probability is the sum of two values of the cache's type, hi and lo, side by side in 2 N columns of one
// product: one rounding of P to bf16 alone is as large an error as the output's own rounding.  f16 ends at 2^-24 and at
// 65504: there the reference lies 2^8 under the maximum, probabilities go up to 2^15, and lo is 2^12 times what hi left
// (half a step under 2^15 at most, 8: so 2^15 again), which the output's sum of both takes back.  P is then exact to
// 2^-22 of itself, or half of 2^-24 / 2^12 where lo is subnormal: 2^-45 of the maximum.  (lo as it is and a reference at
// the maximum lost what lies 2^24 under it: 8191 keys 17 nats below one with small values gave an output a third off.)
//
// Bound by HBM: 4 hd bytes a key and cached head.  So the work is shared out evenly whatever the lengths: the CTAs, one
// an SM (two for 16 rows and fewer), take equal runs of the tiles of the (sequence, row tile, cached head) items laid
// end to end, and a CTA's ring of TMA tiles runs on across the items' borders.  An item that lies in several CTAs leaves
// its parts - normalised outputs with their reference m and sum l - in the workspace, and a second small kernel joins
// them.
//
// hd 128, bf16: one token of 64 sequences of 4 to 8 thousand keys, 32 heads on 8: 238 us, 6.8 TB/s (the measured copy
// rate); one of 131071 keys: 86 us, 6.2 TB/s; 32 rows of 16 sequences of 32 heads, 2048 keys: 95 us, 5.8 TB/s; of one, 768
// keys: 12.3 us, mostly starts, ends and the join.  hd 64, f16: one token of 15 sequences of 2 to 4 thousand keys, with
// weights: 27 us.  64 rows a cached head are bound by their softmax: 16 rows of 8 sequences, 4096 keys, 32 heads on 8:
// 39 us (21 us of keys).
//
// Softmax runs with one key a thread and RW rows in its registers.  A row's reference is the maximum over the first
// tile of the CTA's part that has a key to see (tiles whose positions all lie on no page have none; f16: 2^8 under it).
// It follows when a probability would exceed 2^20 (f16: 2^15), which one vote a tile finds out; else the warps meet at no
// barrier.  Sums l are kept per key lane and joined once a part.
//
//   warp 0     TMA: the pages of a tile, a lane each, K and V through a ring of 128-key slots
//   warp 1     MMAs, issued by one lane: scores up to two tiles ahead of the products, across items too
//   warps 2..  softmax, one key and RW rows a thread
//   the last four: an item's query tile while the one before is walked, and its output while the next one is (by the
//              softmax warps these took 3.6 us an item)
//
// Positions at or past a sequence's length, or on no page, are not loaded (or come with a page's other rows): their
// scores are taken as -inf and their V rows zeroed in shared memory, so that whatever bytes lie there meet no product.
#pragma once

#include "gemm.cuh"
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
  int H, R, group, rows;      // rows: R * group of a cached head, in row_tiles tiles of N
  int row_tiles, per_seq;     // per_seq: items of a sequence, H_kv * row_tiles
  int min_share, whole;       // units a CTA takes at least; whole: items are not split
  FastDiv by_group, by_heads; // by_heads: by H_kv.  An item of a sequence: row tile * H_kv + cached head, so that the
                              // row tiles of a head's keys run on different SMs at about the same time
  int chunk_keys, chunk_run;  // of the second kernel's CTAs that add up weights: keys at once, and how many times
  FastDiv by_chunks;          // by a table's such CTAs
  float scale_log2;
  int nz, z_tiles;            // scores kept for the weights: [item][z_tiles][128][nz]
  float *ws_o, *ws_ml, *ws_lse, *ws_z;   // [2 * CTAs][N][hd], [2 * CTAs][N][2], [item][N]
  int4* ws_plan;              // [CTA] the split item that starts there, its first and last slots; or -1
  int2* ws_items;             // [item] (for the weights) first and last slots of a split item, or -1
  int joins, join_ctas;       // of the second kernel: CTAs that join; CTAs of the first one
};

static __device__ int g_attn_paged_err[1];

constexpr int kPagedKeys = 128;

struct PairBf16 {
  using E = ElemBf16;
  static constexpr uint32_t kFormat = 1;
  static constexpr float kSlack = 20.0f, kBase = 0.0f;   // log2 of the largest probability, and of one at the maximum
  static constexpr float kLo = 1.0f;                     // what lo is multiplied by
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  static __device__ __forceinline__ float2 unpack(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
};
struct PairF16 {
  using E = ElemF16;
  static constexpr uint32_t kFormat = 0;
  static constexpr float kSlack = 15.0f, kBase = 8.0f;
  static constexpr float kLo = 4096.0f;
  static __device__ __forceinline__ uint32_t pack(float a, float b) { return pack_f16x2(a, b); }
  static __device__ __forceinline__ float2 unpack(uint32_t w) { return f16x2_to_f32(w); }
};

template <int HD, int N>
struct AttnPagedCfg {
  static constexpr int KT = kPagedKeys;
  static constexpr int RW = N <= 16 ? 8 : 16;           // rows of a softmax thread
  static constexpr int WGS = N / RW;                    // groups of four softmax warps
  static constexpr int SOFT = 128 * WGS;                // softmax threads
  static constexpr int HELP = 128;                      // threads of the query tiles and the output
  static constexpr int THREADS = 64 + SOFT + HELP;
  static constexpr int SLOT = KT * HD * 2;              // one K or V tile: HD / 64 parts of 128 keys x 128 bytes
  static constexpr int NP = N < 16 ? 16 : N;            // columns of a product
  static constexpr int Q_BYTES = NP * HD * 2;           // HD / 64 parts of NP rows x 128 bytes
  static constexpr int P_ROW = 4 * N < 128 ? 4 * N : 128;   // a key's probabilities, hi, then lo (64 rows: a part each)
  static constexpr int P_PARTS = N == 64 ? 2 : 1;
  static constexpr int P_BYTES = KT * P_ROW;            // one part
  static constexpr int CTAS = N <= 16 ? 2 : 1;          // an SM
  static constexpr int P_BUFS = N == 16 && HD == 128 ? 1 : 2;
  // places (64 bits), warp maxima (4), m (2 buffers), rise, sums of the warps (4, 2 buffers), their inverse
  static constexpr int STAT_FLOATS = 2 * N + 4 * N + 2 * N + N + 8 * N + N;
  static constexpr int FIXED = 1024 + Q_BYTES + P_BUFS * P_PARTS * P_BYTES + STAT_FLOATS * 4 + 448;
  static constexpr int MOST = (228 * 1024 / CTAS - 1024 - FIXED) / SLOT;
  static constexpr int SLOTS = MOST > 12 ? 12 : MOST;
  static constexpr int SMEM_BYTES = FIXED + SLOTS * SLOT;
  static constexpr int S_COL = 0;                       // two buffers of NP
  static constexpr int O_COL = 2 * NP;                  // two buffers of 2 N, the products of hi and of lo
  static constexpr int TMEM_COLS = N == 8 ? 64 : N == 16 ? 128 : N == 32 ? 256 : 512;
  static_assert(SLOTS >= 3 && SMEM_BYTES <= 232448 && 2 * NP + 4 * N <= TMEM_COLS && CTAS * TMEM_COLS <= 512 && (2 * SLOTS + 17) * 8 + 28 + THREADS / 8 <= 448, "shared and tensor memory");
};

// 2^x; results below the normal range are 0
__device__ __forceinline__ float pow2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// Order-preserving map of a float's bits to a signed integer, and back.
__device__ __forceinline__ int order_of(float x) {
  const int b = __float_as_int(x);
  return b ^ ((b >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float of_order(int o) { return __int_as_float(o ^ ((o >> 31) & 0x7fffffff)); }

__device__ __forceinline__ int paged_tiles(int n) { return (n + kPagedKeys - 1) / kPagedKeys; }

// What an item costs, in the units that are shared out: its tiles, and one for its start and end (about a tile's
// time: two batches of equal keys, one with 8 items of nothing more, took 29 us and 45 us in units of tiles alone).
// whole: items are the units.
__device__ __forceinline__ int paged_units(const AttnPagedParams& p, int n) {
  return p.whole ? 1 : n > 0 ? paged_tiles(n) + 1 : 0;
}

// The parts of a CTA's run of units, one item after the other; every role walks them by itself.
struct PagedWalk {
  int s, item, t0, nt, n, left, next_n, part;   // nt: the part's tiles; part: counts up
  // from unit u0 of an item on, `units` of them
  __device__ __forceinline__ PagedWalk(const AttnPagedParams& p, int s_, int item_, int u0, int units)
      : s(s_), item(item_), left(units), part(0) {
    n = p.c.len(p.lens, s);
    next_n = s + 1 < p.c.b ? p.c.len(p.lens, s + 1) : 0;
    take(p, u0);
  }
  __device__ __forceinline__ void take(const AttnPagedParams& p, int u0) {
    t0 = max(u0 - 1, 0);
    if (p.whole) {
      nt = max(paged_tiles(n), 1);                // (an empty one too: it writes its zeros)
      --left;
    } else {
      const int start = u0 == 0 ? 1 : 0;
      nt = min(paged_tiles(n) - t0, left - start);
      left -= nt + start;
    }
  }
  // false: that was the last one
  __device__ __forceinline__ bool next(const AttnPagedParams& p) {
    if (left <= 0) return false;
    ++part;
    if (++item == p.per_seq) {
      item = 0;
      do {
        ++s;
        n = next_n;
        next_n = s + 1 < p.c.b ? p.c.len(p.lens, s + 1) : 0;
      } while (!p.whole && n == 0 && s + 1 < p.c.b);
    }
    take(p, 0);
    return nt > 0;                                // (no tile: the run ends behind an item's first unit)
  }
  __device__ __forceinline__ bool complete() const { return t0 == 0 && nt >= paged_tiles(n); }
};

template <typename F, int HD, int N>
__global__ void __launch_bounds__(AttnPagedCfg<HD, N>::THREADS, AttnPagedCfg<HD, N>::CTAS)
    attn_paged_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                      const __grid_constant__ AttnPagedParams p) {
  using C = AttnPagedCfg<HD, N>;
  using T = typename F::E::T;
  constexpr int KT = C::KT, RW = C::RW, PARTS = HD / 64;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sKV = smem;
  uint8_t* sQ = sKV + C::SLOTS * C::SLOT;
  uint8_t* sP = sQ + C::Q_BYTES;                        // buffers of hi, lo
  long long* s_to = reinterpret_cast<long long*>(sP + C::P_BUFS * C::P_PARTS * C::P_BYTES);   // [N] where a row goes
  float* s_wmax = reinterpret_cast<float*>(s_to + N);   // [4][N]
  float* s_ref = s_wmax + 4 * N;                        // [2][N] references, of parts in turn
  float* s_up = s_ref + 2 * N;                          // [N] their rise
  float* s_sums = s_up + N;                             // [2][4][N] the warps' sums
  float* s_inv = s_sums + 8 * N;                        // [N] inverse sums
  uint64_t* full = reinterpret_cast<uint64_t*>(s_inv + N);
  uint64_t* empty = full + C::SLOTS;
  uint64_t* qready = empty + C::SLOTS;                  // a part's queries are in place
  uint64_t* qfree = qready + 1;                         // its last scores are there
  uint64_t* sfull = qfree + 1;                          // [2]
  uint64_t* sfree = sfull + 2;                          // [2]
  uint64_t* pready = sfree + 2;                         // [2]
  uint64_t* pvdone = pready + 2;                        // [2]
  uint64_t* lready = pvdone + 2;                        // [2] a part's references and sums are there
  uint64_t* odone = lready + 2;                         // [2] its last product is done
  uint64_t* ofree = odone + 2;                          // [2] its output is out
  uint64_t* mdone = ofree + 2;                          // every MMA is done
  int* s_plan = reinterpret_cast<int*>(mdone + 1);      // first sequence, item, unit; how many units; a CTA's share
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(s_plan + 5);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* s_units = reinterpret_cast<int*>(tmem_slot + 2); // [warps]
  int* err = g_attn_paged_err;

  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::SLOTS; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(qready, C::HELP / 32);
    mbar_init(qfree, 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&lready[s], C::SOFT / 32);
      mbar_init(&odone[s], 1);
      mbar_init(&ofree[s], C::HELP / 32);
      mbar_init(&sfull[s], 1);
      mbar_init(&sfree[s], C::SOFT / 32);
      mbar_init(&pready[s], C::SOFT / 32);
      mbar_init(&pvdone[s], 1);
    }
    mbar_init(mdone, 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tensormap(&tmK);
    prefetch_tensormap(&tmV);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::TMEM_COLS);
    tmem_relinquish();
  }
  if constexpr (N < 16) {   // the columns past the rows: queries of zero
    for (int e = threadIdx.x; e < C::Q_BYTES / 16; e += C::THREADS) reinterpret_cast<uint4*>(sQ)[e] = make_uint4(0, 0, 0, 0);
  }
  griddep_wait();
  // This CTA's run of units: every warp adds up a segment of the sequences, then the first finds the run's start in the
  // segment that holds it.
  constexpr int WARPS = C::THREADS / 32;
  const int segment = (p.c.b + WARPS * 32 - 1) / (WARPS * 32) * 32;
  {
    int sum = 0;
    const int end = min((warp + 1) * segment, p.c.b);
#pragma unroll 4
    for (int s = warp * segment + lane; s < end; s += 32) sum += paged_units(p, p.c.len(p.lens, s));
    // (of a segment's sums the low 32 bits: segments of more units than that are refused)
    sum = (int)__reduce_add_sync(0xffffffffu, (uint32_t)sum);
    if (lane == 0) s_units[warp] = sum;
  }
  __syncthreads();
  if (warp == 0) {
    long long units = 0;
    for (int w = 0; w < WARPS; ++w) units += s_units[w];
    units *= p.per_seq;
    const long long share = max((units + gridDim.x - 1) / gridDim.x, (long long)p.min_share);
    const long long first = min(units, share * blockIdx.x), last = min(units, first + share);
    long long base = 0;
    int s0 = 0, s_at = 0, item = 0, u0 = 0;
    while (s0 + segment < p.c.b && base + (long long)s_units[s0 / segment] * p.per_seq <= first) {
      base += (long long)s_units[s0 / segment] * p.per_seq;
      s0 += segment;
    }
    for (; s0 < p.c.b && first < last; s0 += 32) {
      const int t = s0 + lane < p.c.b ? paged_units(p, p.c.len(p.lens, s0 + lane)) : 0;
      int upto = t;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, upto, d);
        if (lane >= d) upto += v;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, base + (long long)upto * p.per_seq > first);
      if (past) {
        const int l = __ffs(past) - 1;
        const int before = __shfl_sync(0xffffffffu, upto - t, l), tl = __shfl_sync(0xffffffffu, t, l);
        const long long in = first - base - (long long)before * p.per_seq;
        s_at = s0 + l;
        item = (int)(in / tl);
        u0 = (int)(in - (long long)item * tl);
        break;
      }
      base += (long long)__shfl_sync(0xffffffffu, upto, 31) * p.per_seq;
    }
    if (lane == 0) {
      s_plan[0] = s_at;
      s_plan[1] = item;
      s_plan[2] = u0;
      s_plan[3] = (int)(last - first);
      s_plan[4] = (int)min(share, 0x7fffffffLL);
    }
  }
  fence_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  griddep_launch_dependents();                          // not before: a dependent could take the columns awaited

  PagedWalk w(p, s_plan[0], s_plan[1], s_plan[2], s_plan[3]);
  if (s_plan[3] > 0 && w.nt > 0) {
    if (warp == 0) {
      // ------------------------------------------------------ pages to the ring
      const uint64_t pol = p.row_tiles > 1 ? policy_evict_last() : policy_evict_first();
      const int box = min(1 << p.c.page_shift, KT), boxes = KT / box;
      int u = 0;                                          // ring position
      bool ok = true, more = true;
      // this lane's page of a tile, asked for a tile ahead, across parts too
      auto page_of = [&](const PagedWalk& x, int t) {
        const int at = t * KT + lane * box;
        return lane < boxes && at < x.n ? p.c.table[(long long)x.s * p.c.max_pages + (at >> p.c.page_shift)] : -1;
      };
      int page = page_of(w, w.t0);
      while (more && ok) {
        uint32_t g;
        p.by_heads.divmod((uint32_t)w.item, g);
        const int end = w.t0 + w.nt;
        PagedWalk wn = w;
        more = wn.next(p);
        for (int t = w.t0; t < end && ok; ++t) {
          const int next = t + 1 < end ? page_of(w, t + 1) : more ? page_of(wn, wn.t0) : -1;
          const bool there = (unsigned)page < (unsigned)p.c.pages;
          const int y = (t * KT + lane * box) & ((1 << p.c.page_shift) - 1), z = page * p.c.H_kv + (int)g;
          const uint32_t bytes = (uint32_t)(__popc(__ballot_sync(0xffffffffu, there)) * box) * (HD * 2);
#pragma unroll
          for (int v = 0; v < 2; ++v, ++u) {
            const int slot = u % C::SLOTS;
            if (u >= C::SLOTS &&
                !__all_sync(0xffffffffu, mbar_wait_long(&empty[slot], (uint32_t)(u / C::SLOTS - 1) & 1u, abort_flag, err,
                                                        ERR_ATTN_FULL))) {
              ok = false;
              break;
            }
            if (lane == 0) mbar_arrive_expect_tx(&full[slot], bytes);
            __syncwarp();
            if (there) {
#pragma unroll
              for (int h = 0; h < PARTS; ++h)
                tma_load_3d(sKV + slot * C::SLOT + h * (KT * 128) + lane * box * 128, v ? &tmV : &tmK, &full[slot], h * 128,
                            y, z, pol);
            }
          }
          page = next;
        }
        w = wn;
      }
      if (*abort_flag)   // let copies in flight land before the CTA's shared memory goes away
        for (int k = max(u - C::SLOTS, 0); k < u; ++k)
          mbar_wait_long(&full[k % C::SLOTS], (uint32_t)(k / C::SLOTS) & 1u, nullptr, err, ERR_ATTN_FULL);
    } else if (warp == 1) {
      // ------------------------------------------------------ products
      const uint32_t lead = elect_one();
      constexpr uint32_t idesc = (1u << 4) | (F::kFormat << 7) | (F::kFormat << 10) | ((uint32_t)(C::NP >> 3) << 17) |
                                 ((128u >> 4) << 24);
      constexpr uint32_t idesc_o = (1u << 4) | (F::kFormat << 7) | (F::kFormat << 10) | (1u << 15) | (1u << 16) |
                                   ((uint32_t)(2 * N >> 3) << 17) | ((128u >> 4) << 24);     // V and P MN-major
      const uint32_t q0 = smem_u32(sQ), kv0 = smem_u32(sKV), p0 = smem_u32(sP);
      auto wait = [&](uint64_t* bar, int phase) {
        return __all_sync(0xffffffffu, mbar_wait_long(bar, (uint32_t)phase & 1u, abort_flag, err, ERR_ATTN_FULL)) != 0;
      };
      // Scores two tiles ahead of the products: a tile's S and P buffers are those of the tile before the last, and its
      // S is issued behind that one's product.  (Issuing whichever finds its operands first was 5 % slower, hd 64.)
      PagedWalk ws = w;                                   // the scores' part
      int s_left = ws.nt, o_left = w.nt;
      bool s_new = true, o_new = true, s_done = false;
      auto issue_s = [&](int t) {                         // nothing behind the last tile
        if (s_done) return true;
        const int u = 2 * t, slot = u % C::SLOTS, sb = t & 1;
        if ((s_new && !wait(qready, ws.part)) || !wait(&full[slot], u / C::SLOTS) ||
            (t >= 2 && !wait(&sfree[sb], (t >> 1) - 1)))
          return false;
        s_new = false;
        tc_fence_after();
        const uint32_t k = kv0 + slot * C::SLOT, d = tmem + C::S_COL + sb * C::NP;
#pragma unroll
        for (int h = 0; h < PARTS; ++h)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_f16_ss(lead, d, sdesc_rows<128>(k + h * (KT * 128) + kk * 32),
                       sdesc_rows<128>(q0 + h * (C::NP * 128) + kk * 32), idesc, (h > 0 || kk > 0) ? 1u : 0u);
        mma_commit_lead(lead, &empty[slot]);
        mma_commit_lead(lead, &sfull[sb]);
        if (--s_left == 0) {
          mma_commit_lead(lead, qfree);
          s_done = !ws.next(p);
          s_left = ws.nt;
          s_new = true;
        }
        return true;
      };
      bool ok = issue_s(0) && issue_s(1);
      for (int t = 0; ok; ++t) {
        const int u = 2 * t + 1, slot = u % C::SLOTS, b = t & 1, pb = C::P_BUFS == 2 ? b : 0;
        if (!(ok = wait(&pready[b], t >> 1) && wait(&full[slot], u / C::SLOTS))) break;
        tc_fence_after();
        const uint32_t v = kv0 + slot * C::SLOT, pp = p0 + pb * (C::P_PARTS * C::P_BYTES);
#pragma unroll
        for (int kk = 0; kk < KT / 16; ++kk)
          // a 64-wide head fills both halves of the 128 dims: the second repeats the first and is not read
          mma_f16_ss(lead, tmem + C::O_COL + (w.part & 1) * 2 * N, sdesc_rows<128>(v + kk * 2048, HD == 64 ? 0 : KT * 128),
                     sdesc_rows<C::P_ROW>(pp + kk * 16 * C::P_ROW, C::P_PARTS == 2 ? C::P_BYTES : 16), idesc_o,
                     (!o_new || kk > 0) ? 1u : 0u);
        o_new = false;
        mma_commit_lead(lead, &empty[slot]);
        mma_commit_lead(lead, &pvdone[b]);
        if (--o_left == 0) {
          mma_commit_lead(lead, &odone[w.part & 1]);
          if (!w.next(p)) break;
          o_left = w.nt;
          o_new = true;
        }
        ok = issue_s(t + 2);
      }
      mma_commit_lead(lead, mdone);
      mbar_wait_long(mdone, 0u, nullptr, err, ERR_ATTN_FULL);
    } else if (warp < 2 + C::SOFT / 32) {
      // ------------------------------------------------------ softmax
      const int tid = (warp - 2) * 32 + lane, q4 = warp & 3, key_l = q4 * 32 + lane;   // this thread's key of a tile
      const int row0 = ((warp - 2) >> 2) * RW;            // its first row
      const uint32_t trow = tmem + ((uint32_t)(q4 * 32) << 16);
      bool ok = true, more = true;
      // after a wait that gave up (ok false) the loop goes on without waiting, so that every warp meets every
      // barrier; the outputs are invalid and reported
      auto wait = [&](uint64_t* bar, int phase) {
        ok = __all_sync(0xffffffffu, mbar_wait_long(bar, (uint32_t)phase & 1u, abort_flag, err, ERR_ATTN_FULL)) && ok;
      };
      // the page of this thread's key of a tile, asked for a tile ahead, across parts too
      auto page_of = [&](const PagedWalk& x, int t) {
        const int key = t * KT + key_l;
        return key < x.n ? p.c.table[(long long)x.s * p.c.max_pages + (key >> p.c.page_shift)] : -1;
      };
      int page = page_of(w, w.t0);
      int tt = 0;                                         // tiles so far
      while (more) {
        float l_sum[RW];
#pragma unroll
        for (int j = 0; j < RW; ++j) l_sum[j] = 0.0f;
        const long long item = (long long)w.s * p.per_seq + w.item;
        PagedWalk wn = w;
        more = wn.next(p);
        float* m_at = s_ref + (w.part & 1) * N;
        const uint32_t ocol = trow + C::O_COL + (w.part & 1) * 2 * N;
        if (w.part >= 2) wait(&ofree[w.part & 1], (w.part >> 1) - 1);   // the part before the last is out
        bool unset = true;                                // no key of the part seen so far, by any of the threads
        for (int t = 0; t < w.nt; ++t, ++tt) {
          const int b = tt & 1, pb = C::P_BUFS == 2 ? b : 0;
          const bool seen = (unsigned)page < (unsigned)p.c.pages;
          page = t + 1 < w.nt ? page_of(w, w.t0 + t + 1) : more ? page_of(wn, wn.t0) : -1;
          wait(&sfull[b], tt >> 1);
          tc_fence_after();
          float z[RW];
          tmem_ld<RW>(trow + C::S_COL + b * C::NP + row0, z);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sfree[b]);
#pragma unroll
          for (int j = 0; j < RW; ++j) z[j] = seen ? z[j] * p.scale_log2 : -INFINITY;
          if (p.mass) {
            float* zs = p.ws_z + ((item * p.z_tiles + w.t0 + t) * KT + key_l) * p.nz + row0;
#pragma unroll
            for (int j = 0; j < RW; j += 4)
              if (row0 + j < p.nz) *reinterpret_cast<float4*>(zs + j) = make_float4(z[j], z[j + 1], z[j + 2], z[j + 3]);
          }
          float top = -INFINITY;
          if (!unset) {
#pragma unroll
            for (int j = 0; j < RW; j += 4) {
              const float4 m = *reinterpret_cast<const float4*>(m_at + row0 + j);
              z[j] -= m.x;
              z[j + 1] -= m.y;
              z[j + 2] -= m.z;
              z[j + 3] -= m.w;
            }
#pragma unroll
            for (int j = 0; j < RW; ++j) top = fmaxf(top, z[j]);
          }
          if (named_bar_or(2, C::SOFT, unset ? seen : top > F::kSlack)) {
            // references: those of the first tile with a key (until then sums and output are zeros), or higher ones
#pragma unroll
            for (int j = 0; j < RW; ++j) {
              const int r = __reduce_max_sync(0xffffffffu, order_of(z[j]));
              if (lane == j) s_wmax[q4 * N + row0 + j] = of_order(r);
            }
            named_bar_sync(2, C::SOFT);
            if (tid < N) {
              float up = fmaxf(fmaxf(s_wmax[tid], s_wmax[N + tid]), fmaxf(s_wmax[2 * N + tid], s_wmax[3 * N + tid]));
              up = up > -INFINITY ? up - F::kBase : 0.0f;
              if (!unset && up < 0.0f) up = 0.0f;
              s_up[tid] = up;
              m_at[tid] = unset ? up : m_at[tid] + up;
            }
            named_bar_sync(2, C::SOFT);
#pragma unroll
            for (int j = 0; j < RW; ++j) z[j] -= s_up[row0 + j];
            if (!unset) {
              wait(&pvdone[(tt - 1) & 1], (tt - 1) >> 1);
              tc_fence_after();
              float f[RW], o[RW];
#pragma unroll
              for (int j = 0; j < RW; ++j) {
                f[j] = pow2_approx(-s_up[row0 + j]);
                l_sum[j] *= f[j];
              }
#pragma unroll
              for (int part = 0; part < 2; ++part) {
                tmem_ld<RW>(ocol + part * N + row0, o);
#pragma unroll
                for (int j = 0; j < RW; ++j) o[j] *= f[j];
                tmem_st<RW>(ocol + part * N + row0, o);
              }
            }
            unset = false;
            // (the maxima are read again only behind the next vote)
          }
          if (C::P_BUFS == 1 && tt > 0) wait(&pvdone[(tt - 1) & 1], (tt - 1) >> 1);
          // With two buffers this one is free: S of this tile was issued behind the product of the tile before the
          // last, and its commit stands for everything issued before it.
          uint8_t* pp = sP + pb * (C::P_PARTS * C::P_BYTES);
#pragma unroll
          for (int j = 0; j < RW; j += 8) {
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float a = pow2_approx(z[j + 2 * e]), c = pow2_approx(z[j + 2 * e + 1]);
              l_sum[j + 2 * e] += a;
              l_sum[j + 2 * e + 1] += c;
              hi[e] = F::pack(a, c);
              const float2 h = F::unpack(hi[e]);
              lo[e] = F::pack((a - h.x) * F::kLo, (c - h.y) * F::kLo);
            }
            *reinterpret_cast<uint4*>(pp + swizzled<C::P_ROW>(key_l, (row0 + j) >> 3)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4*>(pp + (C::P_PARTS == 1 ? swizzled<C::P_ROW>(key_l, (N + row0 + j) >> 3)
                                                            : C::P_BYTES + swizzled<C::P_ROW>(key_l, (row0 + j) >> 3))) =
                make_uint4(lo[0], lo[1], lo[2], lo[3]);
          }
          if (row0 == 0 && !__all_sync(0xffffffffu, seen)) {
            const int u = 2 * tt + 1, slot = u % C::SLOTS;
            wait(&full[slot], u / C::SLOTS);
            if (!seen) {
#pragma unroll
              for (int h = 0; h < PARTS; ++h)
#pragma unroll
                for (int c = 0; c < 8; ++c)
                  *reinterpret_cast<uint4*>(sKV + slot * C::SLOT + h * (KT * 128) + key_l * 128 + c * 16) =
                      make_uint4(0, 0, 0, 0);
            }
          }
          fence_async_smem();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&pready[b]);
        }
        // sum RW columns over the warp, lane c (modulo RW) ending with column c, while the last product runs
#pragma unroll
        for (int s = RW / 2; s >= 1; s >>= 1) {
          const bool upper = (lane & s) != 0;
#pragma unroll
          for (int i = 0; i < s; ++i) {
            const float send = upper ? l_sum[i] : l_sum[i + s];
            const float keep = upper ? l_sum[i + s] : l_sum[i];
            l_sum[i] = keep + __shfl_xor_sync(0xffffffffu, send, s);
          }
        }
#pragma unroll
        for (int s = RW; s < 32; s <<= 1) l_sum[0] += __shfl_xor_sync(0xffffffffu, l_sum[0], s);
        if (lane < RW) s_sums[(w.part & 1) * 4 * N + q4 * N + row0 + lane] = l_sum[0];
        __syncwarp();
        if (lane == 0) mbar_arrive(&lready[w.part & 1]);
        if (more) w = wn;
      }
    } else {
      // ------------------------------------------------------ query tiles and output
      const int tid = (warp - 2) * 32 + lane - C::SOFT, q4 = warp & 3, dim = q4 * 32 + lane;
      const uint32_t trow = tmem + ((uint32_t)(q4 * 32) << 16);
      constexpr int L = HD / 8, QV = N * L / C::HELP > 0 ? N * L / C::HELP : 1;   // lanes of a row; vectors of a thread
      bool ok = true, more = true;
      auto wait = [&](uint64_t* bar, int phase) {
        ok = __all_sync(0xffffffffu, mbar_wait_long(bar, (uint32_t)phase & 1u, abort_flag, err, ERR_ATTN_FULL)) && ok;
      };
      // a row of a part's tile: where it lies in q, and in out
      auto row_at = [&](const PagedWalk& x, int row, long long stride) {
        uint32_t g, j;
        const int rt = (int)p.by_heads.divmod((uint32_t)x.item, g);
        const uint32_t i = p.by_group.divmod((uint32_t)min(rt * N + row, p.rows - 1), j);
        return ((long long)x.s * p.R + i) * stride + (long long)((int)g * p.group + (int)j) * HD;
      };
      auto rows_of = [&](const PagedWalk& x) {
        return min(N, p.rows - (int)p.by_heads.div((uint32_t)x.item) * N);
      };
      uint4 qv[QV];
      auto q_load = [&](const PagedWalk& x) {
        const int n_rows = rows_of(x);
#pragma unroll
        for (int k = 0; k < QV; ++k) {
          const int e = tid + k * C::HELP, row = e / L;
          qv[k] = make_uint4(0, 0, 0, 0);
          if (row < n_rows) qv[k] = *reinterpret_cast<const uint4*>(p.q + row_at(x, row, p.q_rs) + e % L * 8);
        }
      };
      auto q_store = [&] {
#pragma unroll
        for (int k = 0; k < QV; ++k) {
          const int e = tid + k * C::HELP, row = e / L, c = e % L;
          if (row < N) *reinterpret_cast<uint4*>(sQ + (c >> 3) * (C::NP * 128) + swizzled<128>(row, c & 7)) = qv[k];
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(qready);
      };
      int4 plan = make_int4(-1, 0, 0, 0);                 // (an item that goes on in the next CTA is this one's last)
      q_load(w);
      q_store();
      while (more) {
        PagedWalk wn = w;
        more = wn.next(p);
        if (more) {
          q_load(wn);
          wait(qfree, w.part);
          q_store();
        }
        const int b = w.part & 1, n_rows = rows_of(w), slot = 2 * blockIdx.x + (w.part > 0 ? 1 : 0);
        const long long item = (long long)w.s * p.per_seq + w.item;
        const bool complete = w.complete();
        if (tid < N) s_to[tid] = complete ? row_at(w, tid, p.o_rs) : ((long long)slot * N + tid) * HD;
        if (!complete && w.t0 == 0) {
          // where the item's other parts lie: CTAs that follow, each with `share` units
          const int rest = paged_tiles(w.n) - w.nt, share = s_plan[4];
          plan = make_int4((int)item, slot, 2 * ((int)blockIdx.x + (rest + share - 1) / share), 0);
        }
        if (p.mass && !p.whole && tid == 0 && w.t0 == 0)
          p.ws_items[item] = complete ? make_int2(-1, -1) : make_int2(plan.y, plan.z);
        wait(&lready[b], w.part >> 1);
        if (tid < N) {
          const float* ls = s_sums + b * 4 * N + tid;
          const float l = (ls[0] + ls[N]) + (ls[2 * N] + ls[3 * N]), m = s_ref[b * N + tid];
          if (!complete)
            *reinterpret_cast<float2*>(p.ws_ml + ((long long)slot * N + tid) * 2) = make_float2(m, l);
          else if (p.mass)
            p.ws_lse[item * N + tid] = l == 0.0f ? INFINITY : m + log2f(l);
          s_inv[tid] = l == 0.0f ? 0.0f : 1.0f / l;
        }
        named_bar_sync(3, C::HELP);
        wait(&odone[b], w.part >> 1);
        tc_fence_after();
        const uint32_t ocol = trow + C::O_COL + b * 2 * N;
        // (rolled: code that runs once a part costs its instruction fetches)
        auto put = [&](auto store) {
#pragma unroll 1
          for (int n = 0; n < n_rows; n += 8) {
            float o[8];
            float o2[8];
            tmem_ld8x2(ocol + n, ocol + N + n, o, o2);
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = fmaf(o2[j], 1.0f / F::kLo, o[j]);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float f = s_inv[n + j];
              if (dim < HD && n + j < n_rows) store(s_to[n + j] + dim, f == 0.0f ? 0.0f : o[j] * f);
            }
          }
        };
        if (complete)
          put([&](long long at, float v) { F::E::put(reinterpret_cast<T*>(p.out) + at, v); });
        else
          put([&](long long at, float v) { p.ws_o[at] = v; });
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ofree[b]);
        named_bar_sync(3, C::HELP);                       // the places and sums are read: the next part's may be written
        if (more) w = wn;
      }
      if (tid == 0 && !p.whole) p.ws_plan[blockIdx.x] = plan;
    }
  } else if (threadIdx.x == 0 && !p.whole) {
    p.ws_plan[blockIdx.x] = make_int4(-1, 0, 0, 0);
  }
  // the rows of sequences without keys, which are nobody's items
  if (!p.whole)
    for (int s = blockIdx.x; s < p.c.b; s += gridDim.x)
      if (p.c.len(p.lens, s) == 0)
        for (int r = 0; r < p.R; ++r)
          for (int e = threadIdx.x; e < p.H * (HD / 8); e += C::THREADS)
            reinterpret_cast<uint4*>(p.out + ((long long)s * p.R + r) * p.o_rs)[e] = make_uint4(0, 0, 0, 0);
  // lanes that skipped their role arrive here first: reconverge before the CTA-wide barrier
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

// The slots of a split item's parts: the first CTA's, then every following one's first.
__device__ __forceinline__ int paged_slot(int first, int k) { return k == 0 ? first : ((first >> 1) + k) * 2; }
__device__ __forceinline__ int paged_parts(int first, int last) { return (last >> 1) - (first >> 1) + 1; }

// The second kernel: joins split items, and adds what every key received.  The first p.joins CTAs, rows of the item
// that goes on from one CTA of the kernel before to the next: weights l 2^m over their sum (l is 0 without a key, when
// m means nothing; else 1 at least, 2^51 at most, and m the part's reference: what a weight loses to underflow is nothing
// beside the largest).  The others, runs
// of keys of a cached head: the rows' probabilities from their scores (base 2) and log sums.
template <typename F, int HD, bool MASS>
__global__ void __launch_bounds__(128, MASS ? 8 : 12) attn_paged_finish_kernel(const __grid_constant__ AttnPagedParams p, int N) {
  __shared__ float s_o[4][HD], s_w[4];
  __shared__ __align__(16) float s_lse[64];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  griddep_launch_dependents();
  griddep_wait();
  if (MASS && (int)blockIdx.x >= p.joins) {
    uint32_t chunk;
    const int plane = (int)p.by_chunks.divmod(blockIdx.x - (uint32_t)p.joins, chunk), s = plane / p.c.H_kv, g = plane % p.c.H_kv;
    const int n = (int)min((long long)p.c.len(p.lens, s), p.mass_rs), step = p.chunk_keys;
    const int first = (int)chunk * step * p.chunk_run, end = first + min(n - first, step * p.chunk_run);
    if (first >= n) return;
    const long long item0 = (long long)s * p.per_seq + g;   // the head's first row tile; then H_kv apart
    // a key's scores are nq lanes' 16 bytes; a warp's keys are up to four accesses, all on their way at once
    const int nq = p.nz / 4, q = lane & (nq - 1), keys = 32 / nq, mine = step / 4, k0 = warp * mine + lane / nq;
    float* mass = p.mass + plane * p.mass_rs;
    for (int rt = 0; rt < p.row_tiles; ++rt) {
      const long long item = item0 + (long long)rt * p.c.H_kv;
      const int n_rows = min(N, p.rows - rt * N);
      // the rows' log sums, +inf past the last: as the first kernel left them, or from the parts
      __syncthreads();
      const int2 plan = p.whole ? make_int2(-1, -1) : p.ws_items[item];
      const int parts = plan.x < 0 ? 0 : paged_parts(plan.x, plan.y);
      if (parts <= 4) {
        const int r = threadIdx.x;
        float lse = INFINITY;
        if (r < n_rows) {
          if (parts == 0) {
            lse = p.ws_lse[item * N + r];
          } else {
            float2 ml[4];
            float M = -INFINITY, l = 0.0f;
#pragma unroll
            for (int k = 0; k < 4; ++k)
              ml[k] = *reinterpret_cast<const float2*>(p.ws_ml + ((long long)paged_slot(plan.x, min(k, parts - 1)) * N + r) * 2);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (k < parts && ml[k].y != 0.0f) M = fmaxf(M, ml[k].x);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (k < parts && ml[k].y != 0.0f) l += ml[k].y * exp2f(ml[k].x - M);
            if (l != 0.0f) lse = M + log2f(l);
          }
        }
        if (r < 64) s_lse[r] = lse;
      } else {
        for (int r = warp; r < 64; r += 4) {
          float M = -INFINITY, l = 0.0f;
          for (int k = lane; k < parts && r < n_rows; k += 32) {
            const float2 ml = *reinterpret_cast<const float2*>(p.ws_ml + ((long long)paged_slot(plan.x, k) * N + r) * 2);
            if (ml.y == 0.0f) continue;
            const float top = fmaxf(M, ml.x);
            l = l * exp2f(M - top) + ml.y * exp2f(ml.x - top);
            M = top;
          }
          float top = M;
#pragma unroll
          for (int d = 16; d >= 1; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
          if (M > -INFINITY) l *= exp2f(M - top);
#pragma unroll
          for (int d = 16; d >= 1; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
          if (lane == 0) s_lse[r] = l == 0.0f ? INFINITY : top + log2f(l);
          if (r >= n_rows) break;                         // (of the rows past the last up to three are read)
        }
      }
      __syncthreads();
      const bool rows_here = 4 * q < n_rows;              // (else what lies there is nobody's)
      const float4 l4 = rows_here ? *reinterpret_cast<const float4*>(&s_lse[4 * q]) : make_float4(0.f, 0.f, 0.f, 0.f);
      const float* z = p.ws_z + item * p.z_tiles * kPagedKeys * p.nz + 4 * q;
      for (int at = first; at < end; at += step) {
        float4 v[4];
        float old[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int k = k0 + e * keys;
          const bool there = e * keys < mine && at + k < n;
          v[e] = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
          old[e] = 0.0f;
          if (rows_here && there) v[e] = *reinterpret_cast<const float4*>(z + (long long)(at + k) * p.nz);
          if (q == 0 && there) old[e] = mass[at + k];
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int k = k0 + e * keys;
          float sum = (pow2_approx(v[e].x - l4.x) + pow2_approx(v[e].y - l4.y)) +
                      (pow2_approx(v[e].z - l4.z) + pow2_approx(v[e].w - l4.w));
          for (int d = nq / 2; d >= 1; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
          if (q == 0 && e * keys < mine && at + k < n) mass[at + k] = old[e] + sum;
        }
      }
    }
    return;
  }

  // A row of an item with its parts shared by the warps; or (16 rows of a tile and more) four, a warp each where the parts
  // are few, else one after the other.
  const int r0 = (int)blockIdx.x / p.join_ctas, cta = (int)blockIdx.x - r0 * p.join_ctas;
  const int4 plan = p.ws_plan[cta];
  if (plan.x < 0) return;
  const int s = plan.x / p.per_seq, parts = paged_parts(plan.y, plan.z);
  uint32_t g;
  const int rt = (int)p.by_heads.divmod((uint32_t)(plan.x - s * p.per_seq), g), n_rows = min(N, p.rows - rt * N);
  constexpr int D = HD / 32;
  const int each = N > 8 ? 4 : 1;
  const bool few = N > 8 && parts <= 8;
  for (int k = few ? warp : 0; k < (few ? warp + 1 : each); ++k) {
    const int r = each * r0 + k;
    if (r >= n_rows) break;
    float o[D] = {}, sum = 0.0f, M = -INFINITY;
    for (int k0 = lane; k0 < parts; k0 += 32) {
      const float2 ml = *reinterpret_cast<const float2*>(p.ws_ml + ((long long)paged_slot(plan.y, k0) * N + r) * 2);
      if (ml.y != 0.0f) M = fmaxf(M, ml.x);
    }
    const int step = few ? 1 : 4;
    for (int k0 = few ? 0 : warp; k0 < parts; k0 += 4 * step) {
      // four parts' outputs at once
      float2 ml[4];
      float v[4][D];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const long long at = (long long)paged_slot(plan.y, min(k0 + e * step, parts - 1)) * N + r;
        ml[e] = *reinterpret_cast<const float2*>(p.ws_ml + at * 2);
        const float* src = p.ws_o + at * HD + lane * D;
        if constexpr (D == 4) {
          const float4 f = *reinterpret_cast<const float4*>(src);
          v[e][0] = f.x;
          v[e][1] = f.y;
          v[e][2] = f.z;
          v[e][3] = f.w;
        } else {
          const float2 f = *reinterpret_cast<const float2*>(src);
          v[e][0] = f.x;
          v[e][1] = f.y;
        }
      }
      if (k0 == (few ? 0 : warp)) {
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (k0 + e * step >= parts || ml[e].y == 0.0f) continue;
        const float wk = ml[e].y * exp2f(ml[e].x - M);
        sum += wk;
#pragma unroll
        for (int d = 0; d < D; ++d) o[d] += wk * v[e][d];
      }
    }
    if (!few) {
      __syncthreads();                                    // (the row's before are read)
#pragma unroll
      for (int d = 0; d < D; ++d) s_o[warp][lane * D + d] = o[d];
      if (lane == 0) s_w[warp] = sum;
      __syncthreads();
      if (warp > 0) continue;
      sum = (s_w[0] + s_w[1]) + (s_w[2] + s_w[3]);
#pragma unroll
      for (int d = 0; d < D; ++d)
        o[d] = (s_o[0][lane * D + d] + s_o[1][lane * D + d]) + (s_o[2][lane * D + d] + s_o[3][lane * D + d]);
    }
    uint32_t j;
    const uint32_t i = p.by_group.divmod((uint32_t)(rt * N + r), j);
    const float f = sum == 0.0f ? 0.0f : 1.0f / sum;
    uint32_t word[D / 2];
#pragma unroll
    for (int d = 0; d < D; d += 2) word[d / 2] = F::pack(o[d] * f, o[d + 1] * f);
    uint16_t* out = p.out + ((long long)s * p.R + i) * p.o_rs + (long long)((int)g * p.group + (int)j) * HD + lane * D;
    if constexpr (D == 4)
      *reinterpret_cast<uint2*>(out) = make_uint2(word[0], word[1]);
    else
      *reinterpret_cast<uint32_t*>(out) = word[0];
  }
}

}  // namespace dllm
