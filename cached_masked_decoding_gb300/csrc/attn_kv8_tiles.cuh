// Attention over the 8-bit cache for many query rows a cached head (a prefill
// over its own cache, a block of grouped heads): SUBS times 128 rows a CTA, a row in HF
// softmax threads.
//
//   S[row][key] = Q K^T      kind::f8f6f4 on the cache's codes; q as hi + lo codes (two
//                            products, see attn_kv8_rows.cuh), the row's and the key's
//                            scales applied by the softmax
//   O[row][dim] += P V       kind::f16 with bf16; P in tensor memory, V made bf16
// V's codes become bf16 in shared memory with their scale, code * 2^(ev - vsh): four
// significant bits lose nothing.  P is rounded to bf16 (2^-9 of itself; its sum is not).  Both
// have float32's range, so nothing has to follow the scores: a row's reference is its
// maximum over the CTA's first tile of keys and stays, and vsh is the largest value
// exponent there.  A CTA that meets a row whose sum reaches 2^kRowFixed, or value
// exponents more than kVRange above vsh, walks its keys again, with the largest exponent
// it met and references that rise with the scores.
//
// 256 rows (SUBS 2) fill an SM: K and V are fetched, and V converted, once for both
// halves, whose products run under one another's exponentials.  Tensor memory sets the tile:
// 64 keys make the scores of two tiles 128 columns, of which the second tile's are there
// when the first's are used up; P takes the place of its scores; O is 128 more.
// 128 rows are for CTAs that would be half empty, two an SM.
//
// 4096 causal rows of 32 heads on 8, hd 128 (137 GFLOP): 146 us, 0.94 PFLOP/s, 49 % of the
// measured bf16 rate; hd 64: 114 us.  With HF 2 a tile of 256 rows took 2070 cycles, of which the
// products need 1024: shared memory's port is taken by operands (1024 cycles), the walk of scores and
// probabilities through registers (about 770), V's conversion (190) and the key factors
// (256), and what waits for it waits longer.  Tried: 128 keys a tile with one tile's scores
// only, 186 us; 128 rows a CTA throughout, 193; halves in place of bf16 with references that
// follow the scores, 190; e4m3 for P as well, 259.  A CTA's start and end, 19,000 cycles (the
// query tile's conversion 5,000), are the next largest part: nothing else runs on the SM.
//
//   warp 0           TMA: K and V tiles of 64 keys, a ring each
//   warps 1, 3       MMAs of a half, issued by one lane
//   warp 2           scale bytes as factors, fetched four tiles ahead
//   4 HF SUBS warps  softmax, 64 / HF keys of a row a thread; the query tile before, the output after
//   4 SUBS warps     V to bf16; before (HF 1) the query tile with the softmax warps
#pragma once

#include "attn_kv8_rows.cuh"

namespace dllm {

template <int HD, int SUBS>
struct AttnTilesCfg {
  static constexpr int N = 128 * SUBS;                  // rows
  static constexpr int KT = 64;                         // keys of a tile
  static constexpr int SB = 2;                          // buffers of scores
  // Softmax threads of a row: one issues less (hd 128: 146 us against 153 for the rows above),
  // two wait less (256 rows of hd 64: 114 against 127; at 128 rows, two CTAs an SM, one is the faster:
  // 64 sequences of 32 x 4 rows, 2048 keys, 76 us against 83).
  static constexpr int HF = HD == 64 && SUBS == 2 ? 2 : 1;
  static constexpr int SOFT_WARPS = 4 * HF * SUBS, CONV_WARPS = 4 * SUBS;
  static constexpr int THREADS = 32 * (4 + SOFT_WARPS + CONV_WARPS);
  static constexpr int CTAS = SUBS == 1 ? 2 : 1;        // an SM
  // registers, from the launch's a thread shared out anew by warpgroups: 128 + 48 + 56 <= 3 * 80,
  // 2 * 144 + 2 * 56 + 72 <= 5 * 96, 4 * 88 + 2 * 40 + 72 = 7 * 72 (HF 2)
  static constexpr int REGS_SOFT = HF == 2 ? 88 : SUBS == 1 ? 128 : 144;
  static constexpr int REGS_CONV = HF == 2 ? 40 : SUBS == 1 ? 48 : 56;
  static constexpr int REGS_REST = SUBS == 1 ? 56 : 72;
  static constexpr int SLOT = KT * HD;
  static constexpr int VS = SUBS == 1 ? 2 : 3;          // V slots (K has 3)
  static constexpr int VB = SUBS == 1 ? 2 : 3;          // V tiles as bf16
  static constexpr int Q_BYTES = N * HD;                // hi or lo
  static constexpr int V_BYTES = KT * HD * 2;           // V as bf16: 64 dims a 128-byte row
  static constexpr int BARS = 3 + 3 + 2 * VS + SUBS * (1 + SB + 3 + 2) + 3;
  static constexpr int SMEM_BYTES =
      1024 + (3 + VS) * SLOT + 2 * Q_BYTES + VB * V_BYTES + (N + 15 * KT / 2 + N + 2 * N) * 4 + BARS * 8 + 32;
  static constexpr int SUB_COLS = 256;                  // of 128 rows: scores of two tiles, then the output
  static constexpr int O_COL = SB * KT;
  static_assert(O_COL + HD <= SUB_COLS && CTAS * SUBS * SUB_COLS <= 512, "tensor memory");
  static_assert(CTAS * (SMEM_BYTES + 1024) <= 228 * 1024, "shared memory");
};

constexpr float kRowSlack = 8.0f;    // log2 a score may exceed a reference by that rises with the scores
constexpr float kRowFixed = 40.0f;   // and a row's sum one that does not

// A word of four codes to two pairs of bf16, code * 2^-120: the code's exponent and
// mantissa bits in bf16's places.
__device__ __forceinline__ void codes_to_bf16(uint32_t w, uint32_t& a, uint32_t& b) {
  const uint32_t x = __byte_perm(w, 0, 0x1404), y = __byte_perm(w, 0, 0x3424);
  a = ((x >> 4) & 0x07f007f0u) | (x & 0x80008000u);
  b = ((y >> 4) & 0x07f007f0u) | (y & 0x80008000u);
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 d =
      __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&d);
}
// 2^e as a pair of bf16, 0 below the normal range.
__device__ __forceinline__ uint32_t pow2_bf16x2(int e) {
  return e < -126 ? 0u : (uint32_t)(127 + min(e, 127)) * 0x00800080u;
}

template <int HD, int SUBS>
__global__ void __launch_bounds__(AttnTilesCfg<HD, SUBS>::THREADS, AttnTilesCfg<HD, SUBS>::CTAS)
    attn_kv8_tiles_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                          const __grid_constant__ AttnKv8Params p) {
  using C = AttnTilesCfg<HD, SUBS>;
  constexpr int KT = C::KT, N = C::N, HF = C::HF, KH = KT / HF;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sK = smem;
  uint8_t* sV = sK + 3 * C::SLOT;
  uint8_t* sQ = sV + C::VS * C::SLOT;                   // [SUBS] hi, lo of 128 rows
  uint8_t* sH = sQ + 2 * C::Q_BYTES;                    // [VB] V as bf16
  uint32_t* s_q = reinterpret_cast<uint32_t*>(sH + C::VB * C::V_BYTES);   // [SUBS] the rows' scale bytes, an atom
  __nv_bfloat16* s_kf = reinterpret_cast<__nv_bfloat16*>(s_q + N);   // [3][KT] 2^(ek - 9)
  uint32_t* s_vf = reinterpret_cast<uint32_t*>(s_kf + 3 * KT);   // [3][KT] 2^(120 + ev - vsh), bf16 pairs
  uint32_t* s_vg = s_vf + 3 * KT;                       // [3][KT] what of it is over 2^127
  int* s_lim = reinterpret_cast<int*>(s_vg + 3 * KT);   // [N]
  float* s_top = reinterpret_cast<float*>(s_lim + N);   // [2][N] a row's two halves: largest scores, sums
  uint64_t* kfull = reinterpret_cast<uint64_t*>(s_top + 2 * N);   // [3] a tile's K and factors are there
  uint64_t* kempty = kfull + 3;
  uint64_t* vfull = kempty + 3;
  uint64_t* vempty = vfull + C::VS;
  uint64_t* pvdone = vempty + C::VS;                    // [3] a tile's products with V
  uint64_t* qready = pvdone + 3;                        // [SUBS]
  uint64_t* sfull = qready + SUBS;                      // [SUBS][SB] scores
  uint64_t* pready = sfull + C::SB * SUBS;                  // [SUBS][3] probabilities, and V as bf16
  uint64_t* mdone = pready + 3 * SUBS;                  // [SUBS]
  uint64_t* pread = mdone + SUBS;                       // [SUBS] a product has read its probabilities
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(pread + SUBS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* again = abort_flag + 1;                 // the keys have to be walked once more
  volatile int* s_vsh = abort_flag + 2;                 // the value exponents' reference
  volatile int* s_vbig = abort_flag + 3;                // [3] a tile has factors in s_vg
  int* err = g_attn_kv8_err;

  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  uint32_t split_u, plane_u, g_u;
  const int item = (int)p.by_splits.divmod(blockIdx.x, split_u);
  // the last row tiles first: under a causal mask they see the most keys
  const int rt = p.row_tiles - 1 - (int)p.by_tiles.divmod((uint32_t)item, plane_u);
  const int seq = (int)p.by_heads.divmod(plane_u, g_u);
  const int split = (int)split_u, plane = (int)plane_u, g = (int)g_u;
  const int n_rows = min(N, p.rows - rt * N);
  const int subs = SUBS == 1 ? 1 : (n_rows + 127) / 128;   // the last row tile may lack its second half

  if (threadIdx.x == 0) {
    for (int s = 0; s < 3; ++s) {
      mbar_init(&kfull[s], 2);
      mbar_init(&kempty[s], subs);
      mbar_init(&pvdone[s], subs);
    }
    for (int s = 0; s < C::VS; ++s) {
      mbar_init(&vfull[s], 1);
      mbar_init(&vempty[s], C::CONV_WARPS);
    }
    for (int s = 0; s < SUBS; ++s) {
      mbar_init(&qready[s], 8);
      for (int k = 0; k < C::SB; ++k) mbar_init(&sfull[C::SB * s + k], 1);
      for (int k = 0; k < 3; ++k) mbar_init(&pready[3 * s + k], 4 * HF + C::CONV_WARPS);
      mbar_init(&mdone[s], 1);
      mbar_init(&pread[s], 1);
    }
    *abort_flag = 0;
    *again = 0;
    fence_mbar_init();
    prefetch_tensormap(&tmK);
    prefetch_tensormap(&tmV);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, SUBS * C::SUB_COLS);
    tmem_relinquish();
  }
  griddep_wait();
  // The query tile: 128 rows by eight warps, their softmax warps and (HF 1) four that convert V later.
  const bool soft = warp >= 4 && warp < 4 + C::SOFT_WARPS;
  const int sub_w = soft ? (warp - 4) / (4 * HF) : (warp - 4 - C::SOFT_WARPS) / 4;   // of the converting warps, too
  const int tid = (soft ? (warp - 4) % (4 * HF) : 4 + (warp & 3)) * 32 + lane;
  const bool asks = (soft || (HF == 1 && warp >= 4)) && sub_w < subs;
  AttnQueryTile<HD, 128, 256> query;
  if (asks) query.load(p, seq, g, rt * SUBS + sub_w, n_rows - sub_w * 128, tid);
  // the limits by other threads: loads return in order, and the query's are slow
  if (warp < 4) {
#pragma unroll
    for (int k = (int)threadIdx.x; k < N; k += 128) {
      const int i = (int)p.by_group.div((uint32_t)(rt * N + (k < n_rows ? k : 0)));
      const int lim = p.limits ? p.limits[(long long)seq * p.R + i] : p.c.T;
      s_lim[k] = min(max(lim, 0), p.c.T);
      s_q[k] = 0x7f7f7f7fu;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  griddep_launch_dependents();                          // not before: a dependent could take the columns awaited
  int lim_max = 0;
#pragma unroll
  for (int k = 0; k < N / 32; ++k) lim_max = max(lim_max, s_lim[lane + 32 * k]);
  lim_max = __reduce_max_sync(0xffffffffu, lim_max);
  const int tiles = (lim_max + KT - 1) / KT;
  const int t0 = (int)p.by_splits.div((uint32_t)(tiles * split));
  const int nt = (int)p.by_splits.div((uint32_t)(tiles * (split + 1))) - t0;

  auto wait = [&](uint64_t* bar, int phase) {           // decided warp-wide: tensor-memory accesses are collective
    return __all_sync(0xffffffffu, mbar_wait_long(bar, (uint32_t)phase & 1u, abort_flag, err, ERR_ATTN_FULL)) != 0;
  };
  auto query_tile = [&]() {
    if (!asks || nt == 0) return;
    uint8_t* q = sQ + sub_w * (256 * HD);
    query.store(n_rows - sub_w * 128, tid, q, q + 128 * HD, 0, s_q + sub_w * 128);
    fence_async_smem();
    named_bar_sync(2 + sub_w, 256);                       // and the rows' scales are there
    if (lane == 0) mbar_arrive(&qready[sub_w]);
  };
  // Tiles count on through the second walk (T = pass * nt + t); each role walks twice in
  // its own branch, which a register share needs, and meets the others in between.
  auto once_more = [&](int pass) {
    __syncwarp();
    named_bar_sync(1, C::THREADS);
    const bool more = pass == 0 && *again != 0;
    named_bar_sync(1, C::THREADS);
    return more;
  };

  if (warp < 4) {
    setmaxnreg_dec<C::REGS_REST>();   // takes a whole warpgroup
    for (int pass = 0;; ++pass) {
      const int base = pass * nt;
      if (warp == 0) {
        if (lane == 0) {
          const uint64_t pol = policy_evict_last();       // the other row tiles read the same keys
          int k_issued = base, v_issued = base;
          for (int T = base; T < base + nt; ++T) {
            const int ks = T % 3, vs = T % C::VS, row = (t0 + T - base) * KT;
            if (T >= 3 && !mbar_wait_long(&kempty[ks], (uint32_t)(T / 3 - 1) & 1u, abort_flag, err, ERR_ATTN_FULL))
              break;
            mbar_arrive_expect_tx(&kfull[ks], C::SLOT);
            tma_load_3d(sK + ks * C::SLOT, &tmK, &kfull[ks], 0, row, plane, pol);
            k_issued = T + 1;
            if (T >= C::VS &&
                !mbar_wait_long(&vempty[vs], (uint32_t)(T / C::VS - 1) & 1u, abort_flag, err, ERR_ATTN_FULL))
              break;
            mbar_arrive_expect_tx(&vfull[vs], C::SLOT);
            tma_load_3d(sV + vs * C::SLOT, &tmV, &vfull[vs], 0, row, plane, pol);
            v_issued = T + 1;
          }
          if (*abort_flag) {   // let copies in flight land before the CTA's shared memory goes away
            for (int T = max(k_issued - 3, base); T < k_issued; ++T)
              mbar_wait_long(&kfull[T % 3], (uint32_t)(T / 3) & 1u, nullptr, err, ERR_ATTN_FULL);
            for (int T = max(v_issued - C::VS, base); T < v_issued; ++T)
              mbar_wait_long(&vfull[T % C::VS], (uint32_t)(T / C::VS) & 1u, nullptr, err, ERR_ATTN_FULL);
          }
        }
      } else if ((warp & 1) && warp >> 1 < subs) {
        const int sub = warp >> 1;
        const uint32_t lead = elect_one();
        if (nt > 0 && (pass > 0 || wait(&qready[sub], 0))) {
          tc_fence_after();
          constexpr uint32_t idesc_s = idesc_f8(128, KT);
          // bf16 operands (type 1), f32 accumulator, V MN-major
          constexpr uint32_t idesc_o =
              (1u << 4) | (1u << 7) | (1u << 10) | (1u << 16) | ((uint32_t)(HD >> 3) << 17) | (8u << 24);
          const uint32_t q0 = smem_u32(sQ) + sub * (256 * HD), k0 = smem_u32(sK), h0 = smem_u32(sH);
          const uint32_t ts = tmem + sub * C::SUB_COLS, to = ts + C::O_COL;
          auto issue_s = [&](int t) {
            const int T = base + t, b = T % C::SB, slot = T % 3;
            if (!wait(&kfull[slot], T / 3)) return false;
            // Scores come over the probabilities that tile t - SB's product reads: nothing but its
            // completion orders the two.  (Waited for before the keys, 162 us in place of 156.)
            if (t >= C::SB && !wait(&pread[sub], T - C::SB)) return false;
            tc_fence_after();
            const uint32_t k = k0 + slot * C::SLOT;
#pragma unroll
            for (int part = 0; part < 2; ++part)
#pragma unroll
              for (int kk = 0; kk < HD / 32; ++kk)
                mma_f8_ss(lead, ts + b * KT, sdesc_rows<HD>(q0 + part * (128 * HD) + kk * 32),
                          sdesc_rows<HD>(k + kk * 32), idesc_s, (part > 0 || kk > 0) ? 1u : 0u);
            mma_commit_lead(lead, &sfull[C::SB * sub + b]);
            mma_commit_lead(lead, &kempty[slot]);
            return true;
          };
          bool ok = issue_s(0) && (C::SB == 1 || nt < 2 || issue_s(1));
          for (int t = 0; t < nt && ok; ++t) {
            const int T = base + t, r = T % 3;
            if (!wait(&pready[3 * sub + r], T / 3)) break;
            tc_fence_after();
            const uint32_t v = h0 + T % C::VB * C::V_BYTES, pb = ts + T % C::SB * KT;
#pragma unroll
            for (int kk = 0; kk < KT / 16; ++kk)
              mma_f16_ts(lead, to, pb + kk / (KH / 16) * KH + kk % (KH / 16) * 8,
                         sdesc_rows<128>(v + kk * 2048, KT * 128), idesc_o, (t > 0 || kk > 0) ? 1u : 0u);
            mma_commit_lead(lead, &pvdone[r]);
            mma_commit_lead(lead, &pread[sub]);
            if (t + C::SB < nt) ok = issue_s(t + C::SB);
          }
          mma_commit_lead(lead, &mdone[sub]);
          mbar_wait_long(&mdone[sub], (uint32_t)pass & 1u, nullptr, err, ERR_ATTN_FULL);
        }
      } else if (warp == 2) {
        // -------------------------------------------------- factors of keys lane + 32 j of a tile
        constexpr int J = KT / 32, AHEAD = 256 / KT;
        const uint8_t* ksc = p.c.k_scale + (long long)plane * p.c.T;
        const uint8_t* vsc = p.c.v_scale + (long long)plane * p.c.T;
        // bytes of AHEAD tiles, and of the next AHEAD in flight; positions past every limit
        // read the last key's and are of no account
        uint32_t kb4[J] = {}, vb4[J] = {};
        int kn[AHEAD][J], vn[AHEAD][J];
        auto fetch = [&](int t) {
#pragma unroll
          for (int e = 0; e < AHEAD; ++e)
#pragma unroll
            for (int j = 0; j < J; ++j) {
              const int key = min((t0 + t + e) * KT + 32 * j + lane, lim_max - 1);
              kn[e][j] = ksc[key];
              vn[e][j] = vsc[key];
            }
        };
        if (nt > 0) fetch(0);
        int vsh = pass == 0 ? -127 : *s_vsh, most = -127;
        bool far = false;
#pragma unroll 1
        for (int t = 0; t < nt; ++t) {
          const int T = base + t, r = T % 3;
          if (t % AHEAD == 0) {
#pragma unroll
            for (int j = 0; j < J; ++j) {
              kb4[j] = vb4[j] = 0;
#pragma unroll
              for (int e = 0; e < AHEAD; ++e) {
                due(kn[e][j]);
                due(vn[e][j]);
                kb4[j] |= (uint32_t)kn[e][j] << 8 * e;
                vb4[j] |= (uint32_t)vn[e][j] << 8 * e;
              }
            }
            fetch(t + AHEAD);
          }
          int kb[J], ev[J], top = -1000;                  // -1000: no value counts
          bool bad[J];
#pragma unroll
          for (int j = 0; j < J; ++j) {
            kb[j] = (int)(kb4[j] & 255u);
            const int vb = (int)(vb4[j] & 255u);
            kb4[j] >>= 8;
            vb4[j] >>= 8;
            bad[j] = kb[j] == kScaleNan || vb == kScaleNan;
            ev[j] = bad[j] || (t0 + t) * KT + 32 * j + lane >= lim_max ? -1000 : vb - 127;
            top = max(top, ev[j]);
          }
          top = __reduce_max_sync(0xffffffffu, top);
          if (t == 0 && pass == 0) vsh = max(top, -127);
          most = max(most, top);
          far = far || top - vsh > kVRange;
          if (T >= 3 && !wait(&pvdone[r], T / 3 - 1)) break;   // tile T - 3's factors have been read
#pragma unroll
          for (int j = 0; j < J; ++j) {
            const int e = ev[j] == -1000 ? -1000 : min(ev[j] - vsh, 100), at = r * KT + 32 * j + lane;
            // a bad row makes its scores NaN, so that only rows that see it are
            s_kf[at] = __float2bfloat16_rn(scale_value(bad[j] ? kScaleNan : kb[j]) * 0x1p-9f);
            s_vf[at] = pow2_bf16x2(min(120 + e, 127));
            s_vg[at] = pow2_bf16x2(max(e - 7, 0));
          }
          if (lane == 0) s_vbig[r] = top - vsh > 7;
          __syncwarp();
          if (lane == 0) mbar_arrive(&kfull[r]);
        }
        if (lane == 0 && pass == 0 && far) {
          *s_vsh = most;
          *again = 1;
        } else if (lane == 0 && pass == 0) {
          *s_vsh = vsh;
        }
      }
      if (!once_more(pass)) break;
    }
  } else if (warp >= 4 + C::SOFT_WARPS) {
    query_tile();                                         // before registers move: its barrier is for both sides
    setmaxnreg_dec<C::REGS_CONV>();
    // ------------------------------------------------------ V to bf16, KEYS keys of a tile
    constexpr int KEYS = KT / C::CONV_WARPS, ROWS = 512 / HD;   // a warp's keys, of a step
    const int key0 = (warp - 4 - C::SOFT_WARPS) * KEYS;
    for (int pass = 0;; ++pass) {
      const int base = pass * nt;
#pragma unroll 1
      for (int T = base; T < base + nt; ++T) {
        const int r = T % 3, vs = T % C::VS, vb = T % C::VB;
        if (!wait(&kfull[r], T / 3) || !wait(&vfull[vs], T / C::VS) ||
            (T >= C::VB && !wait(&pvdone[(T - C::VB) % 3], (T - C::VB) / 3)))
          break;
        const uint8_t* src = sV + vs * C::SLOT;
        uint8_t* dst = sH + vb * C::V_BYTES;
        const bool big = s_vbig[r] != 0;
#pragma unroll
        for (int i = 0; i < KEYS / ROWS; ++i) {
          // A lane takes 16 codes of a key, into two chunks of 64 dims' 128-byte row.  Eight
          // lanes that access shared memory together touch all banks, loading and storing: two
          // keys of 64 dims one after the other, or half of two keys of 128 dims whose
          // numbers differ in bits 0 and 2, which the swizzles turn into the other banks.
          int key, c;
          if constexpr (HD == 64) {
            key = key0 + i * ROWS + (lane >> 2);
            c = lane & 3;
          } else {
            const int pair = (lane >> 4) + 2 * (i & 1);
            key = key0 + 8 * (i >> 1) + ((lane & 4) ? pair ^ 5 : pair);
            c = (lane & 3) + ((lane >> 1) & 4);
          }
          const uint32_t f = s_vf[r * KT + key];
          const uint4 w = *reinterpret_cast<const uint4*>(src + swizzled<HD>(key, c));
          uint32_t h[8];
          codes_to_bf16(w.x, h[0], h[1]);
          codes_to_bf16(w.y, h[2], h[3]);
          codes_to_bf16(w.z, h[4], h[5]);
          codes_to_bf16(w.w, h[6], h[7]);
          // (past every limit the factor is 0: any code's bits are a finite bf16)
#pragma unroll
          for (int k = 0; k < 8; ++k) h[k] = mul_bf16x2(h[k], f);
          if (__builtin_expect(big, 0)) {
            const uint32_t f2 = s_vg[r * KT + key];
#pragma unroll
            for (int k = 0; k < 8; ++k) h[k] = mul_bf16x2(h[k], f2);
          }
          uint8_t* d = dst + (c >> 2) * (KT * 128);
          *reinterpret_cast<uint4*>(d + swizzled<128>(key, (2 * c) & 7)) = make_uint4(h[0], h[1], h[2], h[3]);
          *reinterpret_cast<uint4*>(d + swizzled<128>(key, (2 * c + 1) & 7)) = make_uint4(h[4], h[5], h[6], h[7]);
        }
        fence_async_smem();
        __syncwarp();
        if (lane < subs) mbar_arrive(&pready[3 * lane + r]);
        if (lane == 0) mbar_arrive(&vempty[vs]);
      }
      if (!once_more(pass)) break;
    }
  } else {
    query_tile();
    setmaxnreg_inc<C::REGS_SOFT>();
    // keys 32 hf .. of a tile, dims HD / 2 * hf ..
    const int sub = sub_w, q4 = warp & 3, hf = ((warp - 4) >> 2) % HF, row = sub * 128 + q4 * 32 + lane;
    const int pair_bar = 4 + sub * 4 + q4;
    const bool part = nt > 0 && sub < subs;
    const uint32_t trow = tmem + sub * C::SUB_COLS + ((uint32_t)(q4 * 32) << 16);
    const int lim_row = s_lim[row], lim = lim_row - hf * KH, lim_min = __reduce_min_sync(0xffffffffu, lim_row);
    // scores to base 2: the row's scale and the softmax's.  The 2^9 comes off the keys'
    // factors, so that neither a query nor a key in bf16 takes its factor out of range (keys
    // under 2^-90 lose bits: they matter to queries over 2^60).
    const float rc = fminf(scale_value((int)(s_q[sub * 128 + lane * 4 + q4] & 255u)) * p.scale_log2 * 0x1p9f, 3e38f);
    const uint64_t rc2 = f32x2(rc, rc);
    float m = 0.0f;                                       // reference (base 2) of this row
    uint64_t l2 = 0;                                      // its sum, in two parts
    for (int pass = 0;; ++pass) {
      const int base = pass * nt;
      m = 0.0f;
      l2 = 0;
      // After a wait that gave up the loop goes on, so that every warp meets every barrier;
      // the outputs are invalid and reported.
      for (int t = 0; t < nt && part; ++t) {
        const int T = base + t, b = T % C::SB, r = T % 3, key0 = (t0 + t) * KT;
        const uint32_t ts = trow + b * KT + hf * KH;
        wait(&sfull[C::SB * sub + b], T / C::SB);
        tc_fence_after();
        // 32 scores, times their keys' factors
        auto scores = [&](int k0, float (&s)[32]) {
          tmem_ld32(ts + k0, s);
          const uint4* kf = reinterpret_cast<const uint4*>(s_kf + r * KT + hf * KH + k0);
#pragma unroll
          for (int c = 0; c < 32; c += 8) {
            const uint4 f = kf[c >> 3];
            const uint32_t w[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint64_t f2 = f32x2(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xffff0000u));
              const float2 a = f32x2_get(mul_f32x2(f32x2(s[c + 2 * e], s[c + 2 * e + 1]), f2));
              s[c + 2 * e] = a.x;
              s[c + 2 * e + 1] = a.y;
            }
          }
          if (__builtin_expect(key0 + KT > lim_min, 0)) {   // some row does not see all of the tile
#pragma unroll
            for (int c = 0; c < 32; ++c) s[c] = key0 + k0 + c < lim ? s[c] : -INFINITY;
          }
        };
        if (__builtin_expect(t == 0 || pass > 0, 0)) {
          float top = -INFINITY;
#pragma unroll 1
          for (int k0 = 0; k0 < KH; k0 += 32) {
            float s[32];
            scores(k0, s);
#pragma unroll
            for (int c = 0; c < 32; ++c) top = fmaxf(top, s[c]);
          }
          if constexpr (HF == 2) {
            s_top[hf * N + row] = top;
            named_bar_sync(pair_bar, 64);
            top = fmaxf(top, s_top[(hf ^ 1) * N + row]);
            named_bar_sync(pair_bar, 64);                 // both are read
          }
          top *= rc;
          const bool up = t == 0 ? top > -INFINITY : top > m + kRowSlack;
          const float corr = t > 0 && up ? exp2f(m - top) : 1.0f;
          if (up) m = top;
          if (t > 0 && __any_sync(0xffffffffu, up)) {
            l2 = mul_f32x2(l2, f32x2(corr, corr));
            wait(&pvdone[(T - 1) % 3], (T - 1) / 3);
            tc_fence_after();
#pragma unroll 1
            for (int c = hf * (HD / HF); c < (hf + 1) * (HD / HF); c += 16) {
              float o[16];
              tmem_ld16(trow + C::O_COL + c, o);
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] *= corr;
              tmem_st16(trow + C::O_COL + c, o);
            }
          }
        }
        const uint64_t m2 = f32x2(-m, -m);
#pragma unroll 1
        for (int k0 = 0; k0 < KH; k0 += 32) {
          float s[32];
          scores(k0, s);
          uint32_t ph[16];
          uint64_t sum[2] = {};
#pragma unroll
          for (int c = 0; c < 32; c += 2) {
            const float2 z = f32x2_get(fma_f32x2(f32x2(s[c], s[c + 1]), rc2, m2));
            const float p0 = ex2(z.x), p1 = ex2(z.y);
            sum[(c >> 1) & 1] = add_f32x2(sum[(c >> 1) & 1], f32x2(p0, p1));
            const __nv_bfloat162 v = __floats2bfloat162_rn(p0, p1);
            ph[c >> 1] = *reinterpret_cast<const uint32_t*>(&v);
          }
          l2 = add_f32x2(l2, add_f32x2(sum[0], sum[1]));
          tmem_st16(ts + k0 / 2, reinterpret_cast<const float*>(ph));   // over scores that have been read
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&pready[3 * sub + r]);
      }
      if (part) {
        wait(&pvdone[(base + nt - 1) % 3], (base + nt - 1) / 3);
        tc_fence_after();
      }
      const float2 l = f32x2_get(l2);
      if (pass == 0 && l.x + l.y >= exp2f(kRowFixed)) *again = 1;   // (a NaN is no reason)
      if (!once_more(pass)) break;
    }
    // ------------------------------------------------------ output
    const float2 lp = f32x2_get(l2);
    float l_sum = lp.x + lp.y;
    if constexpr (HF == 2) {
      s_top[hf * N + row] = l_sum;
      named_bar_sync(pair_bar, 64);
      l_sum = s_top[row] + s_top[N + row];
    }
    // 2^vsh in two steps: it alone may leave the range that the result is in
    const int vsh = nt > 0 ? *s_vsh : 0;
    const float f2 = scale_value(127 + vsh / 2);
    const float f = l_sum == 0.0f ? 0.0f : __fdividef(scale_value(127 + vsh - vsh / 2), l_sum);
    const bool valid = row < n_rows;
    const long long ws_row = ((long long)(plane * p.row_tiles + rt) * p.splits + split) * N + row;
    // Rows leave through the query tile's place, 16 lanes (8) a row's 256 (128) bytes: a row
    // a lane took 4 us of the stores' address cycles.
    uint8_t* stage = sQ + row * (2 * HD);
    constexpr int CHUNKS = HD / 8;
#pragma unroll 1
    for (int c = hf * (HD / HF); c < (hf + 1) * (HD / HF); c += 32) {
      float o[32] = {};
      if (part) tmem_ld32(trow + C::O_COL + c, o);
#pragma unroll
      for (int e = 0; e < 32; ++e) o[e] = l_sum == 0.0f ? 0.0f : o[e] * f * f2;   // a row that sees nothing: 0
      if (p.splits > 1) {
        float4* dst = reinterpret_cast<float4*>(p.ws_o + ws_row * HD + c);
        if (valid) {
#pragma unroll
          for (int e = 0; e < 8; ++e) dst[e] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const __nv_bfloat162 v = __floats2bfloat162_rn(o[8 * e + 2 * k], o[8 * e + 2 * k + 1]);
            w[k] = *reinterpret_cast<const uint32_t*>(&v);
          }
          *reinterpret_cast<uint4*>(stage + ((((c >> 3) + e) ^ (row & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
    }
    if (p.splits == 1) {
      if constexpr (HF == 2) named_bar_sync(pair_bar, 64);
      __syncwarp();
      const int l = lane % CHUNKS;
#pragma unroll 4
      for (int k = 0; k < 32 / HF; k += 32 / CHUNKS) {
        const int n = sub * 128 + q4 * 32 + hf * 16 + k + lane / CHUNKS;
        uint32_t jh;
        const int i = (int)p.by_group.divmod((uint32_t)(rt * N + n), jh), h = g * p.group + (int)jh;
        uint16_t* dst = p.out + ((long long)seq * p.R + i) * p.o_rs + (long long)h * HD + l * 8;
        const uint4 w = *reinterpret_cast<const uint4*>(sQ + n * (2 * HD) + ((l ^ (n & 7)) << 4));
        if (n < n_rows) *reinterpret_cast<uint4*>(dst) = w;
      }
    }
    if (valid && hf == 0 && p.splits > 1) *reinterpret_cast<float2*>(p.ws_ml + ws_row * 2) = make_float2(m, l_sum);
  }
  // lanes that skipped their role arrive here first: reconverge before the CTA-wide barrier
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, SUBS * C::SUB_COLS);
  }
}

}  // namespace dllm
