// Attention over the 8-bit cache for few query rows a cached head (a token, a
// block, grouped heads): the codes go from HBM to the tensor cores untouched.
//
// Keys are the 128-row operand.  A tile of 128 keys gives
//   S^T[key][row] = K Q^T          (kind::mxf8f6f4, the rows' scales as block scales)
//   O^T[dim][row] += V^T P^T       (kind::mxf8f6f4, V read MN-major from its TMA tile)
// with N = 8, 16, 32 or 64 rows as the narrow operand (8: hi and lo codes side by side in
// one of 16), so the products cost N / 128 of a 128-row tile's and the kernel is bound by the codes it reads: 2 (hd + 1)
// bytes a key and cached head.
//
// 8 bits lose nothing on the query side: a bf16 q scaled by a power of two to at
// most 448 is hi + lo of two e4m3 codes (8 significant bits are 4 + 4; below
// 2^-10 of the row's largest element an error of 2^-18 of that element), two
// products into one accumulator.  A probability is hi + lo as well, each with
// the block scale that the MMA applies to the 32 keys of a warp, so a loud key
// elsewhere does not push the others under e4m3's range.  Its error is 2^-8 of
// itself (a bf16 rounding), or 2^-21 of the block's largest where that is more:
// scaled into [128, 256), hi leaves at most 2^-4 of a value (2^-10 below 2^-6),
// and lo, 2^4 finer, is off by 2^-4 of that or by 2^-14.
// The value scale 2^ev of a key is folded into its probability.
//
// Softmax runs with one key a thread and RW rows in its registers: nothing is
// reduced across threads per tile but the 32-key maximum of each row (one
// redux).  A row's reference is its maximum over the CTA's first 32 keys, and stays:
// float32 sums and block scales hold what exceeds it by up to 2^110 (a probability
// times its value scale by 2^118 over the CTA's number of keys, so that all of them times the
// largest code, 448, add up to less than 2^127), so the
// warps meet at no barrier after the first tile.  A CTA that met more, or
// value scales over 2^60 from the first keys', walks its keys again with references that follow the
// scores, and others that follow the products (score plus value exponent).  Sums l
// are kept per key lane and joined once at the end.  This is the longest of the
// overlapped stages, so the rows of a tile are shared out over N / RW groups of
// four warps (one group of N rows a thread: 1.8 us a tile of 128 keys for N = 16, 2.8 us for
// N = 32).  Now two CTAs of an SM take 1.5 us a tile each for N = 32, about HBM's rate, one
// alone 1.1 us; what a batch loses is starts, ends and the last CTAs alone.  hd 128: one
// token of 32 sequences, 4096 keys, 32 heads on 8: 37 us, 5.5 TB/s; of 8 sequences, up to
// 8193 keys: 24 us, 4.4 TB/s; 32 rows of 16 sequences of 32 heads, up to 2048 keys: 52 us,
// 4.1 TB/s; 32 rows of one sequence, 768 keys: 9.9 us.
//
//   warp 0     TMA: K and V tiles through a ring of 128-key slots
//   warp 1     scale copies and MMAs, issued by one lane
//   warps 2..  softmax, one key and RW rows a thread; the query tile before, the output after
// Keys are split over CTAs when there are few (sequence, head) items.  Up to 8
// splits form a cluster and join through distributed shared memory; more
// leave their normalised outputs and (m, l) in the workspace, and a second small
// kernel joins them.
#pragma once

#include "gemm.cuh"
#include "ops8.h"
#include "ptx8.cuh"
#include "q8.cuh"

namespace dllm {

struct AttnKv8Params {
  dllm_kv8 c;
  const uint16_t* q;
  uint16_t* out;
  const int32_t* limits;
  long long q_rs, o_rs;
  int H, R, group;        // group = H / H_kv query heads share a cached head
  int rows, row_tiles;    // R * group rows of an item, in tiles of N
  int splits, cluster;    // cluster: the splits of an item are one
  FastDiv by_group, by_splits, by_heads;
  FastDiv by_tiles;       // by row_tiles (few rows) or by b * H_kv
  float scale_log2;
  float *ws_o, *ws_ml;    // [item][split][N][hd] and [item][split][N][2]
};

static __device__ int g_attn_kv8_err[1];

template <int HD, int N>
struct AttnRowsCfg {
  static constexpr int KT = 128;
  static constexpr int RW = N <= 16 ? 8 : 16;           // rows of a softmax thread
  static constexpr int WGS = N / RW;                    // groups of four softmax warps
  static constexpr int SOFT = 128 * WGS;                // softmax threads
  static constexpr int THREADS = 64 + SOFT;
  static constexpr int CTAS = N == 64 ? 1 : 2;          // an SM
  static constexpr int SLOT = KT * HD;                  // one K or V tile
  static constexpr int NQ = N < 16 ? 16 : N;            // 8 rows: one operand of 8 hi and 8 lo rows
  static constexpr int Q_BYTES = NQ * HD;               // hi or lo
  static constexpr int Q_PARTS = N < 16 ? 1 : 2;
  static constexpr int P_ROW = N < 16 ? 32 : 2 * N;     // a key's N hi codes, then its N lo codes
  static constexpr int P_BYTES = KT * P_ROW;
  static constexpr int SLOTS = CTAS == 1 ? (HD == 64 ? 16 : 9) : HD == 64 ? 8 : N == 8 ? 6 : 5;
  static constexpr int SF_BYTES = 512;                  // ones, query scales, two buffers of probability scales
  // warp maxima (two), m, d, limits, scales, (m, l) of 8 splits, warps' sums, places (64 and 32 bits)
  static constexpr int STAT_FLOATS = 8 * N + 3 * N + 4 * N + 16 * N + 4 * N + 3 * N;
  static constexpr int SMEM_BYTES = 1024 + SLOTS * SLOT + Q_PARTS * Q_BYTES + 2 * P_BYTES + 4 * SF_BYTES +
                                    STAT_FLOATS * 4 + (2 * SLOTS + 10) * 8 + 24;
  static constexpr int S_COL = 0;                       // two buffers
  static constexpr int O_COL = 2 * NQ;                  // 2 N columns: hi and lo products
  static constexpr int SFA_COL = O_COL + 2 * N;
  static constexpr int SFQ_COL = SFA_COL + 4;
  static constexpr int SFB_COL = SFQ_COL + 4;
  static constexpr int TMEM_COLS = SFB_COL + 8 <= 128 ? 128 : SFB_COL + 8 <= 256 ? 256 : 512;
  static_assert(SFB_COL + 8 <= TMEM_COLS && CTAS * TMEM_COLS <= 512, "tensor memory");
  static_assert(CTAS * (SMEM_BYTES + 1024) <= 228 * 1024, "shared memory");
};

// Order-preserving map of a float's bits to a signed integer (NaN above +inf).
__device__ __forceinline__ int float_order(float x) {
  const int b = __float_as_int(x);
  return b ^ ((b >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float order_float(int o) { return __int_as_float(o ^ ((o >> 31) & 0x7fffffff)); }

// 2^x; results below the normal range are 0
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// A split's sum l of probabilities is up to 2^117 (its reference stays), so that splits weigh by
// l 2^m together: l as a factor in [1, 2) times 2^sum_log, whose exponents join those of m, both less
// the heaviest split's.  (l times 2^(m - M) lost splits of low references to underflow.)
__device__ __forceinline__ int sum_log(float l) { return min((int)(__float_as_uint(l) >> 23), 250) - 127; }
__device__ __forceinline__ float pow2_f32(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

constexpr float kRefSlack = 40.0f;   // log2 a score or a product may exceed a reference by that follows them
constexpr int kRefFixed = 110;       // and a sum one that does not
constexpr int kSumFixed = 118;       // and a product one, plus log2 of the keys that are added up
constexpr int kVRange = 60;          // value exponents' distance from the first tile's that such references allow

// The query tile, rows rt * N .. of the item, by THREADS threads (a multiple of 32):
// load() asks for them, store() puts hi codes to q_hi, lo codes to q_lo from row lo0 on, and a
// word of the row's scale byte to the 512-byte atom sf (prefilled with 1.0) for both.
// Rows from n_rows on are zeros.  All rows are in flight at once, 16 bytes of a row a thread:
// one at a time, 128 rows took 13 us of load latency.
template <int HD, int N, int THREADS>
struct AttnQueryTile {
  static constexpr int L = HD / 8, PASS = THREADS / L;    // lanes of a row, rows a pass
  static constexpr int ROWS = (N + PASS - 1) / PASS;
  Raw8<ElemBf16> raw[ROWS];

  __device__ __forceinline__ void load(const AttnKv8Params& p, int seq, int g, int rt, int n_rows, int tid) {
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
      const int n = tid / L + k * PASS;
      uint32_t j;                                         // a row that there is: a branch would wait for each load
      const uint32_t i = p.by_group.divmod((uint32_t)(rt * N + (n < n_rows ? n : 0)), j);
      raw[k].load(reinterpret_cast<const __nv_bfloat16*>(p.q) + ((long long)seq * p.R + i) * p.q_rs +
                  (long long)(g * p.group + (int)j) * HD + tid % L * 8);
    }
  }
  __device__ __forceinline__ void store(int n_rows, int tid, uint8_t* q_hi, uint8_t* q_lo, int lo0, uint32_t* sf) {
    const int l = tid % L;
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
      const int n = tid / L + k * PASS;
      if (n >= n_rows) raw[k].zero();
      float x[8];
      raw[k].floats(x);
      uint32_t m = abs_bits8(x);
#pragma unroll
      for (int d = L / 2; d >= 1; d >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
      if (n >= N) continue;
      const int byte = scale_byte(m);
      // a row that is not finite becomes NaN
      const float inv = byte == kScaleNan ? __uint_as_float(0x7fffffffu) : scale_inverse(byte);
      uint32_t h[4], w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t xh = pack_f16x2(x[2 * e] * inv, x[2 * e + 1] * inv);   // 8 bits: exact from 2^-14 on
        h[e] = cvt_e4m3x2_f16x2(xh);
        w[e] = cvt_e4m3x2_f16x2(sub_f16x2(xh, cvt_f16x2_e4m3x2((uint16_t)h[e])));
      }
      const uint2 hi = make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
      const uint2 lo = make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
      *reinterpret_cast<uint2*>(q_hi + swizzled<HD>(n, l >> 1) + (l & 1) * 8) = hi;
      *reinterpret_cast<uint2*>(q_lo + swizzled<HD>(n + lo0, l >> 1) + (l & 1) * 8) = lo;
      if (l == 0 && byte != kScaleNan) {
        const uint32_t word = (uint32_t)byte * 0x01010101u;
        sf[(n & 31) * 4 + (n >> 5)] = word;
        if (lo0) sf[((n + lo0) & 31) * 4 + ((n + lo0) >> 5)] = word;
      }
    }
  }
};

template <int HD, int N>
__global__ void __launch_bounds__(AttnRowsCfg<HD, N>::THREADS, AttnRowsCfg<HD, N>::CTAS)
    attn_kv8_rows_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                         const __grid_constant__ AttnKv8Params p) {
  using C = AttnRowsCfg<HD, N>;
  constexpr int KT = C::KT, RW = C::RW;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sKV = smem;
  uint8_t* sQ = sKV + C::SLOTS * C::SLOT;               // hi, lo
  uint8_t* sP = sQ + C::Q_PARTS * C::Q_BYTES;
  uint8_t* sSF = sP + 2 * C::P_BYTES;                   // scale atoms: ones, queries, a P buffer each
  float* s_wmax = reinterpret_cast<float*>(sSF + 4 * C::SF_BYTES);   // [4][N]
  float* s_nmax = s_wmax + 4 * N;                       // [4][N]
  float* s_m = s_nmax + 4 * N;                          // [N] reference maxima
  float* s_d = s_m + N;                                 // [N] O is in units of 2^(m + d)
  int* s_lim = reinterpret_cast<int*>(s_d + N);         // [N]
  float* s_inv = reinterpret_cast<float*>(s_lim + N);   // [softmax warps][RW] inverse block scales
  float* s_cm = s_inv + 4 * N;                          // [8][N] reference maxima of the cluster's splits
  float* s_cl = s_cm + 8 * N;                           // [8][N] and sums
  float* s_ls = s_cl + 8 * N;                           // [4][N] the warps' sums
  long long* s_to = reinterpret_cast<long long*>(s_ls + 4 * N);   // [N] where a row goes
  uint32_t* s_dst = reinterpret_cast<uint32_t*>(s_to + N);        // [N] its place in the cluster
  float* s_part = reinterpret_cast<float*>(sKV);        // [split][own][HD] rows that the cluster joins here
  uint64_t* full = reinterpret_cast<uint64_t*>(s_dst + N);
  uint64_t* empty = full + C::SLOTS;
  uint64_t* qready = empty + C::SLOTS;
  uint64_t* sfull = qready + 1;                         // [2]
  uint64_t* sfree = sfull + 2;                          // [2]
  uint64_t* pready = sfree + 2;                         // [2]
  uint64_t* pvdone = pready + 2;                        // [2]  the product that read a P buffer is done
  uint64_t* mdone = pvdone + 2;                         // every MMA is done (before tensor memory is freed)
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mdone + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* again = abort_flag + 1;                 // the keys have to be walked once more
  int* err = g_attn_kv8_err;

  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  uint32_t split_u, rt_u, g_u;
  const int item = (int)p.by_splits.divmod(blockIdx.x, split_u);
  const int plane = (int)p.by_tiles.divmod((uint32_t)item, rt_u);     // seq * H_kv + cached head
  const int seq = (int)p.by_heads.divmod((uint32_t)plane, g_u);
  const int split = (int)split_u, rt = (int)rt_u, g = (int)g_u;
  const int n_rows = min(N, p.rows - rt * N);

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::SLOTS; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(qready, C::SOFT / 32);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sfull[s], 1);
      mbar_init(&sfree[s], C::SOFT / 32);
      mbar_init(&pready[s], C::SOFT / 32);
      mbar_init(&pvdone[s], 1);
    }
    mbar_init(mdone, 1);
    *abort_flag = 0;
    *again = 0;
    fence_mbar_init();
    prefetch_tensormap(&tmK);
    prefetch_tensormap(&tmV);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::TMEM_COLS);
    tmem_relinquish();
  }
  griddep_wait();
  // rows of a split in a cluster: split, split + splits, ...
  const int own = (int)p.by_splits.div((uint32_t)(N + p.splits - 1));
  // the softmax warps ask for the query tile at once
  const int tid = (warp - 2) * 32 + lane;
  AttnQueryTile<HD, N, C::SOFT> query;
  if (warp >= 2) {
    query.load(p, seq, g, rt, n_rows, tid);
    if (tid < 128) {
#pragma unroll
      for (int f = 0; f < 4; ++f) reinterpret_cast<uint32_t*>(sSF + f * C::SF_BYTES)[tid] = 0x7f7f7f7fu;
    }
    if (tid < N) {
      s_m[tid] = 0.0f;
      uint32_t j;
      const uint32_t i = p.by_group.divmod((uint32_t)(rt * N + tid), j);
      s_to[tid] = p.splits > 1 && !p.cluster
                      ? (((long long)item * p.splits + split) * N + tid) * HD
                      : ((long long)seq * p.R + i) * p.o_rs + (long long)(g * p.group + (int)j) * HD;
      if (p.cluster) {
        uint32_t rank;
        const uint32_t at = p.by_splits.divmod((uint32_t)tid, rank);
        s_dst[tid] = cluster_addr(smem_u32(s_part + (split * own + (int)at) * HD), rank);
      }
    }
  }
  // limits of the tile's rows; rows past the last see what row 0 sees and are not stored
  if (threadIdx.x < N) {
    const int n = (int)threadIdx.x < n_rows ? (int)threadIdx.x : 0;
    const int i = (int)p.by_group.div((uint32_t)(rt * N + n));
    const int lim = p.limits ? p.limits[(long long)seq * p.R + i] : p.c.T;
    s_lim[threadIdx.x] = min(max(lim, 0), p.c.T);
  }
  if (p.cluster) cluster_arrive();                      // waited for before the first access of another CTA's memory
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  griddep_launch_dependents();                          // not before: a dependent could take the columns awaited
  int lim_max, lim_min;
  {
    int hi = s_lim[lane & (N < 32 ? N - 1 : 31)], lo = hi;
    if constexpr (N == 64) {
      hi = max(hi, s_lim[lane + 32]);
      lo = min(lo, s_lim[lane + 32]);
    }
    lim_max = __reduce_max_sync(0xffffffffu, hi);
    lim_min = __reduce_min_sync(0xffffffffu, lo);
  }
  // this split's keys: whole tiles, shared out evenly over the keys some row sees
  const int tiles = (lim_max + KT - 1) / KT;
  const int t0 = (int)p.by_splits.div((uint32_t)(tiles * split));
  const int nt = (int)p.by_splits.div((uint32_t)(tiles * (split + 1))) - t0;

  float l_sum[RW];                                        // softmax: this key lane's sums of its rows
  // tiles count on through the second walk: T of a tile is pass * nt + t
  for (int pass = 0;; ++pass) {
    const int base = pass * nt;
    if (warp == 0) {
      if (lane == 0) {
        const uint64_t pol = p.row_tiles > 1 ? policy_evict_last() : policy_evict_first();
        int issued = 2 * base;
        for (int u = 2 * base; u < 2 * (base + nt); ++u) {
          const int slot = u % C::SLOTS;
          if (u >= C::SLOTS &&
              !mbar_wait_long(&empty[slot], (uint32_t)(u / C::SLOTS - 1) & 1u, abort_flag, err, ERR_ATTN_FULL))
            break;
          mbar_arrive_expect_tx(&full[slot], C::SLOT);
          tma_load_3d(sKV + slot * C::SLOT, (u & 1) ? &tmV : &tmK, &full[slot], 0, (t0 + (u >> 1) - base) * KT, plane,
                      pol);
          issued = u + 1;
        }
        if (*abort_flag)   // let copies in flight land before the CTA's shared memory goes away
          for (int u = max(issued - C::SLOTS, 2 * base); u < issued; ++u)
            mbar_wait_long(&full[u % C::SLOTS], (uint32_t)(u / C::SLOTS) & 1u, nullptr, err, ERR_ATTN_FULL);
      }
    } else if (warp == 1) {
      const uint32_t lead = elect_one();
      auto wait = [&](uint64_t* bar, int phase) {
        return __all_sync(0xffffffffu, mbar_wait_long(bar, (uint32_t)phase & 1u, abort_flag, err, ERR_ATTN_FULL)) != 0;
      };
      if (nt > 0 && (pass > 0 || wait(qready, 0))) {
        tc_fence_after();
        constexpr uint32_t idesc_s = idesc_mxf8(128, C::NQ);
        // V and P MN-major; P's scale byte kk belongs to keys 32 kk .. 32 kk + 31
        constexpr uint32_t idesc_o = idesc_mxf8(128, 2 * N) | (1u << 15) | (1u << 16);
        const uint32_t q0 = smem_u32(sQ), kv0 = smem_u32(sKV), p0 = smem_u32(sP), f0 = smem_u32(sSF);
        const uint32_t sfa = tmem + C::SFA_COL, sfq = tmem + C::SFQ_COL;
        if (pass == 0) {
          tmem_cp_scales(lead, sfa, sdesc_scales(f0));
          tmem_cp_scales(lead, sfq, sdesc_scales(f0 + C::SF_BYTES));
        }
        // Scores two tiles ahead of the products: the order K(t), V(t) of the ring keeps
        // neither waiting on the other for long.
        auto issue_s = [&](int t) {
          const int T = base + t, u = 2 * T, slot = u % C::SLOTS, sb = T & 1;
          if (!wait(&full[slot], u / C::SLOTS) || (T >= 2 && !wait(&sfree[sb], (T >> 1) - 1))) return false;
          tc_fence_after();
          const uint32_t k = kv0 + slot * C::SLOT, d = tmem + C::S_COL + sb * C::NQ;
#pragma unroll
          for (int part = 0; part < C::Q_PARTS; ++part)
#pragma unroll
            for (int kk = 0; kk < HD / 32; ++kk)
              mma_mxf8_ss(lead, d, sdesc_rows<HD>(k + kk * 32), sdesc_rows<HD>(q0 + part * C::Q_BYTES + kk * 32),
                          idesc_s,
                          sfa, sfq, (part > 0 || kk > 0) ? 1u : 0u);
          mma_commit_lead(lead, &empty[slot]);
          mma_commit_lead(lead, &sfull[sb]);
          return true;
        };
        bool ok = issue_s(0) && (nt < 2 || issue_s(1));
        for (int t = 0; t < nt && ok; ++t) {
          const int T = base + t, u = 2 * T + 1, slot = u % C::SLOTS, pb = T & 1;
          if (!(ok = wait(&pready[pb], T >> 1) && wait(&full[slot], u / C::SLOTS))) break;
          tc_fence_after();
          const uint32_t v = kv0 + slot * C::SLOT, pp = p0 + pb * C::P_BYTES, sfb = tmem + C::SFB_COL + 4 * pb;
          tmem_cp_scales(lead, sfb, sdesc_scales(f0 + (2 + pb) * C::SF_BYTES));
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            // a 64-wide head fills both halves of the 128 dims: the second repeats the first and is not read
            mma_mxf8_ss(lead, tmem + C::O_COL, sdesc_rows<HD>(v + kk * 32 * HD, 0),
                        sdesc_rows<C::P_ROW>(pp + kk * 32 * C::P_ROW), idesc_o | ((uint32_t)kk << 4), sfa, sfb,
                        (t > 0 || kk > 0) ? 1u : 0u);
          mma_commit_lead(lead, &empty[slot]);
          mma_commit_lead(lead, &pvdone[pb]);
          if (t + 2 < nt && !(ok = issue_s(t + 2))) break;
        }
        mma_commit_lead(lead, mdone);
        mbar_wait_long(mdone, (uint32_t)pass & 1u, nullptr, err, ERR_ATTN_FULL);
      }
    } else {
      const int q4 = warp & 3, key_l = q4 * 32 + lane;    // this thread's key in a tile, and its tensor-memory lane
      const int row0 = ((warp - 2) >> 2) * RW;            // its first row
      const uint32_t trow = tmem + ((uint32_t)(q4 * 32) << 16);
      // product t of P V is done
      auto pv_wait = [&](int t) {
        const int T = base + t;
        return __all_sync(0xffffffffu, mbar_wait_long(&pvdone[T & 1], (uint32_t)(T >> 1) & 1u, abort_flag, err,
                                                      ERR_ATTN_FULL)) != 0;
      };
      // Scale bytes of this thread's key in four tiles, and of the next four in
      // flight (their latency under load is over a tile's time).  Positions past every
      // limit read the last key's and are of no account.
      const uint8_t* ksc = p.c.k_scale + (long long)plane * p.c.T;
      const uint8_t* vsc = p.c.v_scale + (long long)plane * p.c.T;
      uint32_t kb4 = 0, vb4 = 0;
      int kn[4], vn[4];
      auto fetch = [&](int t) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int key = min((t0 + t + e) * KT + key_l, lim_max - 1);
          kn[e] = ksc[key];
          vn[e] = vsc[key];
        }
      };
      if (nt > 0) fetch(0);
      if (pass > 0) {
        if (tid < N) s_m[tid] = s_d[tid] = 0.0f;
        named_bar_sync(2, C::SOFT);
      } else if (nt > 0) {
        // 8 rows: the lo rows lie behind the hi rows of one operand
        query.store(n_rows, tid, sQ, sQ + (C::Q_PARTS - 1) * C::Q_BYTES, C::Q_PARTS == 1 ? N : 0,
                    reinterpret_cast<uint32_t*>(sSF + C::SF_BYTES));
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(qready);
      }
      // ------------------------------------------------------ the keys
#pragma unroll
      for (int n = 0; n < RW; ++n) l_sum[n] = 0.0f;
      int vref = 0;                                       // the value scales' reference
      uint32_t most = 0;                                  // largest block maximum of this lane's row
      bool far = false;                                   // a value scale far from the first ones
      // After a wait that gave up (ok false) the loop goes on without waiting, so
      // that every warp meets every barrier; the outputs are invalid and reported.
      bool ok = true;
      for (int t = 0; t < nt; ++t) {
        const int T = base + t, b = T & 1;                  // S and P buffer
        const int key = (t0 + t) * KT + key_l;
        if ((t & 3) == 0) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            due(kn[e]);
            due(vn[e]);
          }
          kb4 = (uint32_t)(kn[0] | kn[1] << 8 | kn[2] << 16 | kn[3] << 24);
          vb4 = (uint32_t)(vn[0] | vn[1] << 8 | vn[2] << 16 | vn[3] << 24);
          fetch(t + 4);
        }
        const int kb = (int)(kb4 & 255u), vb = (int)(vb4 & 255u);
        kb4 >>= 8;
        vb4 >>= 8;
        const bool seen = key < lim_max;                  // by some row
        const bool bad = kb == kScaleNan || vb == kScaleNan;
        const float kf = bad ? __uint_as_float(0x7fffffffu) : scale_value(kb) * p.scale_log2;
        const int ev = bad || !seen ? -1000 : vb - 127;   // -1000: no value scale to refer to
        ok = __all_sync(0xffffffffu,
                        mbar_wait_long(&sfull[b], (uint32_t)(T >> 1) & 1u, abort_flag, err, ERR_ATTN_FULL)) &&
             ok;
        tc_fence_after();
        // scores in base 2, relative to their row's reference
        float z[RW];
        if constexpr (C::Q_PARTS == 1) {
          float s[16];
          tmem_ld16(trow + C::S_COL + b * C::NQ, s);
#pragma unroll
          for (int j = 0; j < RW; ++j) z[j] = s[j] + s[j + N];
        } else {
          tmem_ld<RW>(trow + C::S_COL + b * C::NQ + row0, z);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sfree[b]);
        const uint64_t kf2 = f32x2(kf, kf);
        const bool first = t == 0 && pass == 0;           // no references yet: other warps may be writing them
#pragma unroll
        for (int j = 0; j < RW; j += 4) {
          const float4 m =
              first ? make_float4(0.f, 0.f, 0.f, 0.f) : *reinterpret_cast<const float4*>(s_m + row0 + j);
          const float2 za = f32x2_get(fma_f32x2(f32x2(z[j], z[j + 1]), kf2, f32x2(-m.x, -m.y)));
          const float2 zb = f32x2_get(fma_f32x2(f32x2(z[j + 2], z[j + 3]), kf2, f32x2(-m.z, -m.w)));
          z[j] = za.x;
          z[j + 1] = za.y;
          z[j + 2] = zb.x;
          z[j + 3] = zb.y;
        }
        if ((t0 + t + 1) * KT > lim_min) {                  // some row does not see all of the tile
#pragma unroll
          for (int j = 0; j < RW; ++j) z[j] = key < s_lim[row0 + j] ? z[j] : -INFINITY;
        }
        if (first) {
          // the references: over the first quarter's keys (key 0 is seen wherever any is)
          if (q4 == 0) {
            float mine = 0.0f;
#pragma unroll
            for (int j = 0; j < RW; ++j) {
              const float top = order_float(__reduce_max_sync(0xffffffffu, float_order(z[j])));
              if (lane == j) mine = top;
            }
            const int top_ev = max(__reduce_max_sync(0xffffffffu, ev), -127);
            if (lane < RW) {
              s_m[row0 + lane] = mine == -INFINITY ? 0.0f : mine;
              s_d[row0 + lane] = (float)top_ev;
            }
          }
          named_bar_sync(2, C::SOFT);
          vref = (int)s_d[0];
#pragma unroll
          for (int j = 0; j < RW; ++j) z[j] -= s_m[row0 + j];
        } else if (__builtin_expect(pass > 0, 0)) {
          bool need = t == 0;
          float top = -INFINITY;
#pragma unroll
          for (int j = 0; j < RW; ++j) top = fmaxf(top, fmaxf(z[j], z[j] + (float)ev - s_d[row0 + j]));
          need = need || top > kRefSlack;
          if (!ok) need = false;
          if (named_bar_or(2, C::SOFT, need)) {
            // new references: the first tile's, or where scores or products lie far above the last ones
#pragma unroll
            for (int j = 0; j < RW; ++j) {
              const int wt = __reduce_max_sync(0xffffffffu, float_order(z[j]));
              const int nm = __reduce_max_sync(0xffffffffu, float_order(z[j] + (float)ev - s_d[row0 + j]));
              if (lane == j) {
                s_wmax[q4 * N + row0 + j] = order_float(wt);
                s_nmax[q4 * N + row0 + j] = order_float(nm);
              }
            }
            named_bar_sync(2, C::SOFT);
            float up = 0.0f, un = 0.0f;                   // row tid's references rise by these
            if (tid < N) {
              int a = float_order(s_wmax[tid]), c = float_order(s_nmax[tid]);
#pragma unroll
              for (int k = 1; k < 4; ++k) {
                a = max(a, float_order(s_wmax[k * N + tid]));
                c = max(c, float_order(s_nmax[k * N + tid]));
              }
              up = order_float(a);
              un = order_float(c);
              if (up == -INFINITY || (t > 0 && up < 0.0f)) up = 0.0f;
              if (un == -INFINITY || (t > 0 && un < 0.0f)) un = 0.0f;
            }
            named_bar_sync(2, C::SOFT);
            if (tid < N) {
              s_m[tid] += up;
              s_d[tid] += un - up;
              s_wmax[tid] = up;
              s_nmax[tid] = un;
            }
            named_bar_sync(2, C::SOFT);
#pragma unroll
            for (int j = 0; j < RW; ++j) z[j] -= s_wmax[row0 + j];
            if (t > 0) {
              ok = ok && pv_wait(t - 1);
              tc_fence_after();
#pragma unroll
              for (int j = 0; j < RW; ++j) l_sum[j] *= exp2f(-s_wmax[row0 + j]);
#pragma unroll
              for (int part = 0; part < 2; ++part) {
                float o[RW];
                tmem_ld<RW>(trow + C::O_COL + part * N + row0, o);
#pragma unroll
                for (int j = 0; j < RW; ++j) o[j] *= exp2f(-s_nmax[row0 + j]);
                tmem_st<RW>(trow + C::O_COL + part * N + row0, o);
              }
              tc_fence_before();
            }
            named_bar_sync(2, C::SOFT);                   // the maxima are read: the next tile may rewrite them
          }
        }
        // The P buffer is free: S(t) was issued behind the product of tile t - 2, and its
        // commit stands for everything issued before it.
        const int dv = ev - vref;
        far = far || (ev != -1000 && (dv > kVRange || dv < -kVRange));
        const float vf = ev == -1000 ? 0.0f : __uint_as_float((uint32_t)(127 + min(max(dv, -kVRange), kVRange)) << 23);
        uint8_t* prow = sP + b * C::P_BYTES;
        uint8_t* sf = sSF + (2 + b) * C::SF_BYTES;
        // probabilities, and each row's largest of the warp's 32 keys: lane j (modulo RW) keeps row j's
        uint32_t top_me = 0;
        const uint64_t vf2 = f32x2(vf, vf);
#pragma unroll
        for (int j = 0; j < RW; j += 2) {
          const uint64_t pr = f32x2(ex2(z[j]), ex2(z[j + 1]));
          const float2 l = f32x2_get(add_f32x2(f32x2(l_sum[j], l_sum[j + 1]), pr));
          l_sum[j] = l.x;
          l_sum[j + 1] = l.y;
          if (__builtin_expect(pass == 0, 1)) {
            const float2 pv = f32x2_get(mul_f32x2(pr, vf2));
            z[j] = pv.x;
            z[j + 1] = pv.y;
          } else {
            z[j] = ex2(z[j] + (float)ev - s_d[row0 + j]);
            z[j + 1] = ex2(z[j + 1] + (float)ev - s_d[row0 + j + 1]);
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t r = __reduce_max_sync(0xffffffffu, __float_as_uint(z[j + e]));
            if ((lane & (RW - 1)) == j + e) top_me = r;
          }
        }
        most = max(most, top_me);
        // the block's scale puts its largest probability into [128, 256); the lanes work out a row each
        const int byte_me = min(max((int)(top_me >> 23) - 7, 4), 247);
        float* inv = s_inv + (warp - 2) * RW;
        if (lane < RW) inv[lane] = __uint_as_float((uint32_t)(254 - byte_me) << 23);
        if (lane < 2 * RW) {
          // lanes 0 .. RW-1: the scale bytes of the hi rows for this warp's keys, the next RW: of the lo rows
          const int r = row0 + (lane & (RW - 1)) + (lane < RW ? 0 : N);
          sf[(r & 31) * 16 + (r >> 5) * 4 + q4] = (uint8_t)(lane < RW ? byte_me : byte_me - 4);
        }
        __syncwarp();
        uint32_t hi[RW / 4], lo[RW / 4];
#pragma unroll
        for (int j = 0; j < RW; j += 4) {
          const float4 f = *reinterpret_cast<const float4*>(inv + j);
          // hi: the nearest code; lo: what it leaves, at most a 16th of it, in a scale 2^4 smaller
          const float2 a = f32x2_get(mul_f32x2(f32x2(z[j], z[j + 1]), f32x2(f.x, f.y)));
          const float2 c = f32x2_get(mul_f32x2(f32x2(z[j + 2], z[j + 3]), f32x2(f.z, f.w)));
          const uint32_t x0 = pack_f16x2(a.x, a.y), x1 = pack_f16x2(c.x, c.y);
          const uint32_t h0 = cvt_e4m3x2_f16x2(x0), h1 = cvt_e4m3x2_f16x2(x1);
          hi[j >> 2] = h0 | (h1 << 16);
          lo[j >> 2] = cvt_e4m3x2_f16x2(sub_mul16_f16x2(x0, cvt_f16x2_e4m3x2((uint16_t)h0))) |
                       (cvt_e4m3x2_f16x2(sub_mul16_f16x2(x1, cvt_f16x2_e4m3x2((uint16_t)h1))) << 16);
        }
        uint8_t* ph = prow + swizzled<C::P_ROW>(key_l, row0 >> 4) + (row0 & 15);
        uint8_t* pl = prow + swizzled<C::P_ROW>(key_l, (N + row0) >> 4) + ((N + row0) & 15);
        if constexpr (RW == 8) {
          *reinterpret_cast<uint2*>(ph) = make_uint2(hi[0], hi[1]);
          *reinterpret_cast<uint2*>(pl) = make_uint2(lo[0], lo[1]);
        } else {
          *reinterpret_cast<uint4*>(ph) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(pl) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
        if ((t0 + t + 1) * KT > lim_max && row0 == 0) {
          // the last tile runs past every row's limit: whatever bytes lie there
          // (codes of NaN among them) must not meet the zero probabilities
          const int u = 2 * T + 1, slot = u % C::SLOTS;
          ok = __all_sync(0xffffffffu, mbar_wait_long(&full[slot], (uint32_t)(u / C::SLOTS) & 1u, abort_flag, err,
                                                      ERR_ATTN_FULL)) &&
               ok;
          if (!seen) {
#pragma unroll
            for (int c = 0; c < HD / 16; ++c)
              *reinterpret_cast<uint4*>(sKV + slot * C::SLOT + key_l * HD + c * 16) = make_uint4(0, 0, 0, 0);
          }
        }
        fence_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&pready[b]);
      }
      // a product or a sum over what float32 and the block scales hold (a NaN is no reason)
      constexpr uint32_t kOver = (uint32_t)(127 + kRefFixed) << 23;
      const int keys_log = 32 - __clz(max(nt * KT - 1, 1));   // 31 at most
      const uint32_t over_product = (uint32_t)(127 + min(kRefFixed, kSumFixed - keys_log)) << 23;
      bool over = far || (most >= over_product && most <= 0x7f800000u);
#pragma unroll
      for (int j = 0; j < RW; ++j) over = over || l_sum[j] >= __uint_as_float(kOver);
      if (pass == 0 && over) *again = 1;
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
      if (lane < RW) s_ls[q4 * N + row0 + lane] = l_sum[0];
      if (nt > 0) {
        if (ok) ok = pv_wait(nt - 1);
        tc_fence_after();
      }
    }
    // lanes that skipped their role arrive here first: reconverge before the CTA-wide barrier
    __syncwarp();
    __syncthreads();
    if (pass > 0 || *again == 0) break;
  }

  // ------------------------------------------------------ sums and output
  const int q4 = warp & 3, dim = q4 * 32 + lane, row0 = ((warp - 2) >> 2) * RW;
  const uint32_t trow = tmem + ((uint32_t)(q4 * 32) << 16);
  const bool soft = warp >= 2;
  tc_fence_after();
  auto sum_of = [&](int n) { return (s_ls[n] + s_ls[N + n]) + (s_ls[2 * N + n] + s_ls[3 * N + n]); };   // 0 if nt is
  // per row the factors of O (2^d in two steps: it alone may leave the range that the result is in)
  float2* s_f = reinterpret_cast<float2*>(s_nmax);        // [N]
  if (p.cluster) {
    // every split learns the others' (m, l) of its rows
    cluster_wait();
    if (soft)
      for (int e = tid; e < N * p.splits; e += C::SOFT) {
        const int n = e % N;
        const uint32_t r = (uint32_t)(e / N);
        cluster_store(cluster_addr(smem_u32(s_cm + split * N + n), r), s_m[n]);
        cluster_store(cluster_addr(smem_u32(s_cl + split * N + n), r), sum_of(n));
      }
    cluster_sync();   // and every CTA's MMAs and copies are done: the rings are free
  }
  if (soft && tid < N) {
    const float l = sum_of(tid);
    float w = l == 0.0f ? 0.0f : __fdividef(1.0f, l), w2 = 1.0f;
    if (p.cluster) {
      float mr[8], lr[8], M = -INFINITY, top = -INFINITY, sum = 0.0f;
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        lr[r] = r < p.splits ? s_cl[r * N + tid] : 0.0f;
        mr[r] = r < p.splits ? s_cm[r * N + tid] : 0.0f;
      }
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        M = fmaxf(M, lr[r] != 0.0f ? mr[r] : -INFINITY);  // (a NaN comes through the sum)
        top = fmaxf(top, lr[r] != 0.0f ? mr[r] + (float)sum_log(lr[r]) : -INFINITY);
      }
      const int E = (int)(top - M);
      auto weight = [&](float m, float ll) { return ex2((m - M) + (float)(sum_log(ll) - E)); };
#pragma unroll
      for (int r = 0; r < 8; ++r)
        sum += lr[r] != 0.0f ? lr[r] * pow2_f32(-sum_log(lr[r])) * weight(mr[r], lr[r]) : 0.0f;
      w = l == 0.0f ? 0.0f : pow2_f32(-sum_log(l));
      w2 = __fdividef(weight(s_m[tid], l), sum);
    } else if (p.splits > 1 && tid < n_rows) {
      const long long slot = (long long)item * p.splits + split;
      *reinterpret_cast<float2*>(p.ws_ml + (slot * N + tid) * 2) = make_float2(s_m[tid], l);
    }
    const float vs = nt > 0 ? exp2f(0.5f * s_d[tid]) : 0.0f;
    s_f[tid] = w == 0.0f || w2 == 0.0f ? make_float2(0.0f, 0.0f) : make_float2(vs * w, vs * w2);
  }
  if (soft) {
    named_bar_sync(2, C::SOFT);
    // (rolled: code that runs once a CTA costs its instruction fetches; the kinds of output apart, or
    // every row's store would branch)
    auto put = [&](auto store) {
#pragma unroll 1
      for (int n = row0; n < row0 + RW; n += 8) {
        float a[8] = {}, c[8] = {};
        if (nt > 0) tmem_ld8x2(trow + C::O_COL + n, trow + C::O_COL + N + n, a, c);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float2 f = s_f[n + j];
          const float v = f.x == 0.0f ? 0.0f : (a[j] + c[j]) * f.x * f.y;
          if (dim < HD && n + j < n_rows) store(n + j, v);
        }
      }
    };
    if (p.cluster)                                        // zeros from a split that saw no key
      put([&](int r, float v) { cluster_store(s_dst[r] + 4u * (uint32_t)dim, v); });
    else if (p.splits > 1)
      put([&](int r, float v) { p.ws_o[s_to[r] + dim] = v; });
    else
      put([&](int r, float v) { p.out[s_to[r] + dim] = f32_to_bf16_bits(v); });
  }
  if (p.cluster) {
    cluster_sync();
    if (soft)
      for (int e = tid; e < own * (HD / 4); e += C::SOFT) {
        const int i = e / (HD / 4), r = split + i * p.splits, d = e % (HD / 4) * 4;
        if (r >= n_rows) continue;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (k < p.splits) {
            const float4 o = *reinterpret_cast<const float4*>(s_part + (k * own + i) * HD + d);
            v.x += o.x;
            v.y += o.y;
            v.z += o.z;
            v.w += o.w;
          }
        const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), c = __floats2bfloat162_rn(v.z, v.w);
        *reinterpret_cast<uint2*>(p.out + s_to[r] + d) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&c));
      }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

// Join the splits of every row (64 at most): weights l_s 2^m_s over their sum.  A warp
// a row, a lane two splits' weights: they are whole before the first output meets one, since
// a sum times an output may leave float32's range where the row does not.
template <int HD>
__global__ void __launch_bounds__(128) attn_kv8_join_kernel(const __grid_constant__ AttnKv8Params p, int N) {
  const int lane = threadIdx.x & 31;
  const long long idx = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int h = (int)(idx % p.H);
  const long long row = idx / p.H;
  griddep_launch_dependents();
  griddep_wait();
  if (row >= (long long)p.c.b * p.R) return;
  const int seq = (int)(row / p.R), i = (int)(row % p.R), rn = i * p.group + h % p.group;
  const long long item = ((long long)seq * p.c.H_kv + h / p.group) * p.row_tiles + rn / N;
  const long long first = item * p.splits * N + rn % N;   // then N apart
  constexpr int D = HD / 32;
  // eight splits' outputs at once (a dependent load each was a round trip of L2 each), the first
  // eight beside the weights
  float v[8][D];
  auto load = [&](int s0) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float* src = p.ws_o + (first + (long long)min(s0 + k, p.splits - 1) * N) * HD + lane * D;
      if constexpr (D == 4) {
        const float4 f = *reinterpret_cast<const float4*>(src);
        v[k][0] = f.x;
        v[k][1] = f.y;
        v[k][2] = f.z;
        v[k][3] = f.w;
      } else {
        const float2 f = *reinterpret_cast<const float2*>(src);
        v[k][0] = f.x;
        v[k][1] = f.y;
      }
    }
  };
  load(0);
  float2 ml[2];
  float M = -INFINITY, top = -INFINITY;                   // (a NaN comes through the sum)
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int s = lane + 32 * e;
    ml[e] = s < p.splits ? *reinterpret_cast<const float2*>(p.ws_ml + (first + (long long)s * N) * 2)
                         : make_float2(0.0f, 0.0f);
    if (ml[e].y != 0.0f) {                                // 0: the split saw none of the row's keys
      M = fmaxf(M, ml[e].x);
      top = fmaxf(top, ml[e].x + (float)sum_log(ml[e].y));
    }
  }
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) {
    M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
  }
  const int E = (int)(top - M);
  float w[2], sum;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int le = sum_log(ml[e].y);
    w[e] = ml[e].y == 0.0f ? 0.0f : ml[e].y * pow2_f32(-le) * exp2f((ml[e].x - M) + (float)(le - E));
  }
  sum = w[0] + w[1];
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
#pragma unroll
  for (int e = 0; e < 2; ++e) w[e] = w[e] == 0.0f ? 0.0f : w[e] / sum;
  float o[D] = {};
  for (int s0 = 0; s0 < p.splits; s0 += 8) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float wk = __shfl_sync(0xffffffffu, s0 < 32 ? w[0] : w[1], (s0 + k) & 31);   // 0 past the last split
      if (wk == 0.0f) continue;
#pragma unroll
      for (int d = 0; d < D; ++d) o[d] += wk * v[k][d];
    }
    if (s0 + 8 < p.splits) load(s0 + 8);
  }
  uint32_t word[D / 2];
#pragma unroll
  for (int d = 0; d < D; d += 2) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(o[d], o[d + 1]);
    word[d / 2] = *reinterpret_cast<const uint32_t*>(&b);
  }
  uint16_t* out = p.out + row * p.o_rs + (long long)h * HD + lane * D;
  if constexpr (D == 4)
    *reinterpret_cast<uint2*>(out) = make_uint2(word[0], word[1]);
  else
    *reinterpret_cast<uint32_t*>(out) = word[0];
}

}  // namespace dllm
