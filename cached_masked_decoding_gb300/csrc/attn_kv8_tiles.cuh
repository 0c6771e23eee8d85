// Attention over the 8-bit cache for many query rows a cached head (a prefill
// over its own cache): 128 rows a CTA, a row in two softmax threads.
//
//   S[row][key] = Q K^T      kind::mxf8f6f4 on the cache's codes; q as hi + lo codes (two
//                            products, see attn_kv8_rows.cuh), the row's and the
//                            key's scales applied by the MMA
//   O[row][dim] += P V       kind::f16; P in tensor memory, V as halves
// V's codes become halves in shared memory, code * 2^(ev - vref), exact down to
// 2^-24 where the largest row of the tiles so far has values up to 448 (2^-33 of
// it); vref follows the largest exponent.  P is a half too, 2^7 p: 11 bits down to
// 2^-21 of the row's reference.  Where a tile's value exponents reach more than 2^10
// below vref (a loud value may then count although its p is far below 2^-21), the
// codes stay unscaled from there on, P is formed from the score plus the value's
// exponent, and the products get a reference of their own.  With P as two e4m3 codes and V untouched, as
// for few rows, the softmax needed 16 instructions a score and a causal prefill
// of 4096 rows 259 us; converting 64 V rows costs 1.5 a code, shared by 128
// query rows, and leaves the softmax about 4.
//
// A tile of 128 rows by 128 keys takes the tensor cores 1024 cycles (two e4m3
// products cost what one product of halves costs); two CTAs share an SM, so that
// one's products run under the other's exponentials.  Tensor memory sets the
// tile: 64 keys make S 64 columns, P 32, O 128 and the scales 12, just under half.
//
//   warp 0     TMA: K and V tiles of 64 keys, a ring each
//   warp 1     scale copies and MMAs, issued by one lane
//   warp 2     scale bytes: K's for the MMA, V's as factors
//   warps 4-11 softmax, a row in two threads of 32 keys each (with one thread a row the
//              softmax was the longest stage, bound by its latencies: 2600 cycles a
//              tile); the query tile before, the output after
//   warps 12-15 V to halves, 16 keys each
#pragma once

#include "attn_kv8_rows.cuh"

namespace dllm {

template <int HD>
struct AttnTilesCfg {
  static constexpr int N = 128;                         // rows
  static constexpr int KT = 64;
  static constexpr int THREADS = 512;
  // registers: the launch's 64 a thread (4 warpgroups) shared out anew, 80 + 80 + 40 + 56 = 4 * 64
  static constexpr int REGS_SOFT = 80, REGS_CONV = 40, REGS_REST = 56;
  static constexpr int SLOT = KT * HD;
  static constexpr int KS = 3, VS = 2;                  // slots of the two rings
  static constexpr int Q_BYTES = N * HD;                // hi or lo
  static constexpr int V_BYTES = KT * HD * 2;           // V as halves: 64 dims a 128-byte row
  static constexpr int SF_BYTES = 512;                  // query, two of K
  static constexpr int SMEM_BYTES =
      1024 + (KS + VS) * SLOT + 2 * Q_BYTES + 2 * V_BYTES + 3 * SF_BYTES + (4 + 4 * KT + 5 * N) * 4 +
      (2 * (KS + VS) + 12) * 8 + 16;
  static constexpr int S_COL = 0;
  static constexpr int P_COL = KT;                      // two halves a column
  static constexpr int O_COL = P_COL + KT / 2;
  static constexpr int SF_Q = O_COL + HD, SF_K = SF_Q + 4;
  static constexpr int TMEM_COLS = 256;
  static_assert(SF_K + 8 <= TMEM_COLS, "tensor memory");
  static_assert(2 * (SMEM_BYTES + 1024) <= 228 * 1024, "two CTAs an SM");
};

constexpr float kPShift = 7.0f;    // P is held as 2^7 p, p up to 2^kRowSlack: a half has room to 65504
constexpr float kRowSlack = 8.0f;  // log2 a score may exceed its row's reference by
constexpr int kVSpread = 10;       // log2 of the value scales' spread that halves of V and P cover
constexpr int kVSlack = 6;         // and a value exponent the common one: 448 * 2^6 is under 65504

template <int HD>
__global__ void __launch_bounds__(512, 2)
    attn_kv8_tiles_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                          const __grid_constant__ AttnKv8Params p) {
  using C = AttnTilesCfg<HD>;
  constexpr int KT = C::KT, N = C::N;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sK = smem;
  uint8_t* sV = sK + C::KS * C::SLOT;
  uint8_t* sQ = sV + C::VS * C::SLOT;                   // hi, lo
  uint8_t* sH = sQ + 2 * C::Q_BYTES;                    // [2] V as halves
  uint8_t* sSF = sH + 2 * C::V_BYTES;                   // scale atoms: queries, K (two)
  int* s_vref = reinterpret_cast<int*>(sSF + 3 * C::SF_BYTES);   // [2]
  int* s_wide = s_vref + 2;                             // [2] value scales far apart
  float* s_ev = reinterpret_cast<float*>(s_wide + 2);   // [2][KT] their exponents then
  float* s_hf = s_ev + 2 * KT;                          // [2][KT] factors of V's halves
  int* s_lim = reinterpret_cast<int*>(s_hf + 2 * KT);   // [N]
  float* s_top = reinterpret_cast<float*>(s_lim + N);   // [2][N] a row's two halves: largest scores, sums
  float* s_most = s_top + 2 * N;                        // [2][N] largest products
  uint64_t* kfull = reinterpret_cast<uint64_t*>(s_most + 2 * N);
  uint64_t* kempty = kfull + C::KS;
  uint64_t* vfull = kempty + C::KS;
  uint64_t* vempty = vfull + C::VS;
  uint64_t* qready = vempty + C::VS;
  uint64_t* sfull = qready + 1;                         // S of a tile is there
  uint64_t* sfree = sfull + 1;                          // and has been read
  uint64_t* kready = sfree + 1;                         // [2] a tile's scales are there
  uint64_t* vready = kready + 2;                        // [2] its V as halves
  uint64_t* pready = vready + 2;                        // [2] its P
  uint64_t* pvdone = pready + 2;                        // [2] its product
  uint64_t* mdone = pvdone + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mdone + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* err = g_attn_kv8_err;

  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int split = (int)(blockIdx.x % (unsigned)p.splits);
  const int item = (int)(blockIdx.x / (unsigned)p.splits);
  // the last row tiles first: under a causal mask they see the most keys
  const int planes = p.c.b * p.c.H_kv;
  const int rt = p.row_tiles - 1 - item / planes, plane = item % planes;
  const int seq = plane / p.c.H_kv, g = plane % p.c.H_kv;
  const int n_rows = min(N, p.rows - rt * N);

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::KS; ++s) {
      mbar_init(&kfull[s], 1);
      mbar_init(&kempty[s], 1);
    }
    for (int s = 0; s < C::VS; ++s) {
      mbar_init(&vfull[s], 1);
      mbar_init(&vempty[s], 4);
    }
    mbar_init(qready, 8);
    mbar_init(sfull, 1);
    mbar_init(sfree, 8);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&kready[s], 1);
      mbar_init(&vready[s], 4);
      mbar_init(&pready[s], 8);
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
  griddep_launch_dependents();
  griddep_wait();
  if (threadIdx.x < N) {
    const int n = (int)threadIdx.x < n_rows ? (int)threadIdx.x : 0;
    const int i = (int)p.by_group.div((uint32_t)(rt * N + n));
    const int lim = p.limits ? p.limits[(long long)seq * p.R + i] : p.c.T;
    s_lim[threadIdx.x] = min(max(lim, 0), p.c.T);
#pragma unroll
    for (int f = 0; f < 3; ++f) reinterpret_cast<uint32_t*>(sSF + f * C::SF_BYTES)[threadIdx.x] = 0x7f7f7f7fu;   // 1.0
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  int lim_max, lim_min;
  {
    int hi = s_lim[lane], lo = hi;
#pragma unroll
    for (int k = 1; k < 4; ++k) {
      hi = max(hi, s_lim[lane + 32 * k]);
      lo = min(lo, s_lim[lane + 32 * k]);
    }
    lim_max = __reduce_max_sync(0xffffffffu, hi);
    lim_min = __reduce_min_sync(0xffffffffu, lo);
  }
  const int tiles = (lim_max + KT - 1) / KT;
  const int t0 = (int)((long long)tiles * split / p.splits), t1 = (int)((long long)tiles * (split + 1) / p.splits);
  const int nt = t1 - t0;

  // the query tile, by the softmax warps
  auto query_tile = [&](int tid) {
    attn_query_tile<HD, N, 256>(p, seq, g, rt, n_rows, tid, sQ, sQ + C::Q_BYTES, 0, reinterpret_cast<uint32_t*>(sSF));
    fence_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(qready);
  };

  if (warp < 4) {
    setmaxnreg_dec<C::REGS_REST>();   // takes a whole warpgroup: warp 3 has no other part
    if (warp == 0) {
      if (lane == 0) {
        const uint64_t pol = policy_evict_last();           // the other row tiles read the same keys
        RingPos rk{0, 0u}, rv{0, 0u};
        int k_issued = 0, v_issued = 0;
        for (int t = 0; t < nt; ++t) {
          if (t >= C::KS && !mbar_wait_long(&kempty[rk.s], rk.par ^ 1u, abort_flag, err, ERR_ATTN_FULL)) break;
          mbar_arrive_expect_tx(&kfull[rk.s], C::SLOT);
          tma_load_3d(sK + rk.s * C::SLOT, &tmK, &kfull[rk.s], 0, (t0 + t) * KT, plane, pol);
          rk.next(C::KS);
          k_issued = t + 1;
          if (t >= C::VS && !mbar_wait_long(&vempty[rv.s], rv.par ^ 1u, abort_flag, err, ERR_ATTN_FULL)) break;
          mbar_arrive_expect_tx(&vfull[rv.s], C::SLOT);
          tma_load_3d(sV + rv.s * C::SLOT, &tmV, &vfull[rv.s], 0, (t0 + t) * KT, plane, pol);
          rv.next(C::VS);
          v_issued = t + 1;
        }
        if (*abort_flag) {   // let copies in flight land before the CTA's shared memory goes away
          for (int t = max(k_issued - C::KS, 0); t < k_issued; ++t)
            mbar_wait_long(&kfull[t % C::KS], (uint32_t)(t / C::KS) & 1u, nullptr, err, ERR_ATTN_FULL);
          for (int t = max(v_issued - C::VS, 0); t < v_issued; ++t)
            mbar_wait_long(&vfull[t % C::VS], (uint32_t)(t / C::VS) & 1u, nullptr, err, ERR_ATTN_FULL);
        }
      }
    } else if (warp == 1) {
      const uint32_t lead = elect_one();
      auto wait = [&](uint64_t* bar, int phase) {
        return __all_sync(0xffffffffu, mbar_wait_long(bar, (uint32_t)phase & 1u, abort_flag, err, ERR_ATTN_FULL)) != 0;
      };
      if (nt > 0 && wait(qready, 0)) {
        tc_fence_after();
        constexpr uint32_t idesc_s = idesc_mxf8(128, KT);
        // f16 operands (type 0), f32 accumulator, V MN-major
        constexpr uint32_t idesc_o = (1u << 4) | (1u << 16) | ((uint32_t)(HD >> 3) << 17) | (8u << 24);
        const uint32_t q0 = smem_u32(sQ), k0 = smem_u32(sK), h0 = smem_u32(sH), f0 = smem_u32(sSF);
        tmem_cp_scales(lead, tmem + C::SF_Q, sdesc_scales(f0));
        // A tile's key scales go to tensor memory well before its scores' products: an
        // MMA waits for the copy in front of it.
        auto copy_scales = [&](int t) {
          const int b = t & 1;
          if (!wait(&kready[b], t >> 1)) return false;
          tmem_cp_scales(lead, tmem + C::SF_K + 4 * b, sdesc_scales(f0 + (1 + b) * C::SF_BYTES));
          return true;
        };
        auto issue_s = [&](int t) {
          const int slot = t % C::KS;
          if ((t > 0 && !wait(sfree, t - 1)) || !wait(&kfull[slot], t / C::KS)) return false;
          tc_fence_after();
          const uint32_t k = k0 + slot * C::SLOT, sfk = tmem + C::SF_K + 4 * (t & 1);
#pragma unroll
          for (int part = 0; part < 2; ++part)
#pragma unroll
            for (int kk = 0; kk < HD / 32; ++kk)
              mma_mxf8_ss(lead, tmem + C::S_COL, sdesc_rows<HD>(q0 + part * C::Q_BYTES + kk * 32),
                          sdesc_rows<HD>(k + kk * 32), idesc_s, tmem + C::SF_Q, sfk, (part > 0 || kk > 0) ? 1u : 0u);
          mma_commit_lead(lead, &kempty[slot]);
          mma_commit_lead(lead, sfull);
          return true;
        };
        bool ok = copy_scales(0) && issue_s(0) && (nt < 2 || copy_scales(1));
        for (int t = 0; t < nt && ok; ++t) {
          const int b = t & 1;
          // the next tile's scores as soon as these have been read
          if (t + 1 < nt && !(ok = issue_s(t + 1))) break;
          if (!(ok = wait(&vready[b], t >> 1) && wait(&pready[b], t >> 1))) break;
          tc_fence_after();
          const uint32_t v = h0 + b * C::V_BYTES;
#pragma unroll
          for (int kk = 0; kk < KT / 16; ++kk)
            mma_f16_ts(lead, tmem + C::O_COL, tmem + C::P_COL + kk * 8, sdesc_rows<128>(v + kk * 2048, KT * 128), idesc_o,
                        (t > 0 || kk > 0) ? 1u : 0u);
          mma_commit_lead(lead, &pvdone[b]);
          if (t + 2 < nt && !(ok = copy_scales(t + 2))) break;
        }
        mma_commit_lead(lead, mdone);
        mbar_wait_long(mdone, 0u, nullptr, err, ERR_ATTN_FULL);
      }
    } else if (warp == 2) {
      // ------------------------------------------------------ scales, keys lane and lane + 32 of a tile
      const uint8_t* ksc = p.c.k_scale + (long long)plane * p.c.T;
      const uint8_t* vsc = p.c.v_scale + (long long)plane * p.c.T;
      // bytes in four tiles, and of the next four in flight (256: past every limit)
      uint64_t kb4[2] = {}, vb4[2] = {};
      int kn[4][2], vn[4][2];
      auto fetch = [&](int t) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int key = (t0 + t + e) * KT + 32 * j + lane;
            const bool in = t + e < nt && key < lim_max;
            kn[e][j] = in ? __ldg(ksc + key) : 127;
            vn[e][j] = in ? __ldg(vsc + key) : 256;
          }
      };
      if (nt > 0) fetch(0);
      bool ok = true;
      int vref = -127, low = 1000;
      bool wide = false;
      auto wait = [&](uint64_t* bar, int phase) {
        return __all_sync(0xffffffffu, mbar_wait_long(bar, (uint32_t)phase & 1u, abort_flag, err, ERR_ATTN_FULL)) != 0;
      };
#pragma unroll 1
      for (int t = 0; t < nt; ++t) {
        const int b = t & 1;
        if ((t & 3) == 0) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              due(kn[e][j]);
              due(vn[e][j]);
            }
            kb4[j] = (uint64_t)(kn[0][j] | kn[1][j] << 16) | (uint64_t)(kn[2][j] | kn[3][j] << 16) << 32;
            vb4[j] = (uint64_t)(vn[0][j] | vn[1][j] << 16) | (uint64_t)(vn[2][j] | vn[3][j] << 16) << 32;
          }
          fetch(t + 4);
        }
        int kc[2], ev[2], top = -1000;                      // -1000: no value to refer to
        bool bad[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          kc[j] = (int)(kb4[j] & 0xffffu);
          const int vc = (int)(vb4[j] & 0xffffu);
          kb4[j] >>= 16;
          vb4[j] >>= 16;
          bad[j] = kc[j] == kScaleNan || vc == kScaleNan;
          ev[j] = vc > 255 || bad[j] ? -1000 : vc - 127;
          top = max(top, ev[j]);
          low = min(low, ev[j] == -1000 ? 1000 : ev[j]);
        }
        top = __reduce_max_sync(0xffffffffu, top);
        low = __reduce_min_sync(0xffffffffu, low);          // of the tiles so far
        if (top - vref > (t == 0 ? 0 : kVSlack)) vref = top;
        wide = wide || vref - low > kVSpread;
        // tile t - 2's scores are computed and its references and factors read
        if (t >= 2 && !(ok = wait(&pready[b], (t >> 1) - 1) && wait(&vready[b], (t >> 1) - 1))) break;
        // a bad value makes the score NaN, so that only rows that see it are
        *reinterpret_cast<uint2*>(sSF + (1 + b) * C::SF_BYTES + lane * 16) =
            make_uint2((bad[0] ? 255u : (uint32_t)kc[0]) * 0x01010101u, (bad[1] ? 255u : (uint32_t)kc[1]) * 0x01010101u);
        if (lane == 0) {
          s_vref[b] = vref;
          s_wide[b] = wide;
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const bool none = ev[j] == -1000;
          s_ev[b * KT + 32 * j + lane] = none ? 0.0f : (float)ev[j];
          s_hf[b * KT + 32 * j + lane] = none ? 0.0f : wide ? 1.0f : exp2f((float)(ev[j] - vref));
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&kready[b]);
      }
    }
  } else if (warp >= 12) {
    setmaxnreg_dec<C::REGS_CONV>();
    // ------------------------------------------------------ V to halves, keys 16 cw .. 16 cw + 15 of a tile
    const int cw = warp - 12;
    constexpr int CH = HD / 16;                           // 16-code chunks of a row
    auto wait = [&](uint64_t* bar, int phase) {
      return __all_sync(0xffffffffu, mbar_wait_long(bar, (uint32_t)phase & 1u, abort_flag, err, ERR_ATTN_FULL)) != 0;
    };
#pragma unroll 1
    for (int t = 0; t < nt; ++t) {
      const int b = t & 1, slot = t % C::VS;
      if (!wait(&kready[b], t >> 1) || !wait(&vfull[slot], t / C::VS) || (t >= 2 && !wait(&pvdone[b], (t >> 1) - 1)))
        break;
      const uint8_t* src = sV + slot * C::SLOT;
      uint8_t* dst = sH + b * C::V_BYTES;
      // 32 / CH keys a step; 64 dims a 128-byte row of halves
#pragma unroll
      for (int i = 0; i < CH / 2; ++i) {
        const int key_l = 16 * cw + i * (32 / CH) + lane / CH, c = lane % CH;
        const float hf = s_hf[b * KT + key_l];
        const uint32_t f = pack_f16x2(hf, hf);
        uint4 w = *reinterpret_cast<const uint4*>(src + swizzled<HD>(key_l, c));
        if (hf == 0.0f) w = make_uint4(0, 0, 0, 0);       // past every limit: whatever bytes lie there
        uint32_t h[8];
        const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          h[2 * k] = mul_f16x2(cvt_f16x2_e4m3x2((uint16_t)(ww[k] & 0xffffu)), f);
          h[2 * k + 1] = mul_f16x2(cvt_f16x2_e4m3x2((uint16_t)(ww[k] >> 16)), f);
        }
        uint8_t* d = dst + (c >> 2) * (KT * 128);
        *reinterpret_cast<uint4*>(d + swizzled<128>(key_l, (2 * c) & 7)) = make_uint4(h[0], h[1], h[2], h[3]);
        *reinterpret_cast<uint4*>(d + swizzled<128>(key_l, (2 * c + 1) & 7)) = make_uint4(h[4], h[5], h[6], h[7]);
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&vempty[slot]);
        mbar_arrive(&vready[b]);
      }
    }
  } else {
    setmaxnreg_inc<C::REGS_SOFT>();
    const int q4 = warp & 3, row = q4 * 32 + lane, hf = (warp - 4) >> 2;   // keys 32 hf .. of a tile, dims HD / 2 * hf ..
    const uint32_t trow = tmem + ((uint32_t)(q4 * 32) << 16);
    const int lim = s_lim[row];
    if (nt > 0) query_tile((warp - 4) * 32 + lane);
    // ------------------------------------------------------ the keys
    float m = 0.0f;                                       // reference (base 2) of this row
    uint64_t l2 = 0;                                      // its sum, times 2^7, in two parts
    int vref = 0;
    float d = 0.0f;                                       // O is in units of 2^(m + d): d = vref until scales lie far apart
    // After a wait that gave up (ok false) the loop goes on, so that every warp meets
    // every barrier; the outputs are invalid and reported.
    bool ok = true;
    auto wait = [&](uint64_t* bar, int phase) {           // decided warp-wide: tensor-memory accesses are collective
      return __all_sync(0xffffffffu, mbar_wait_long(bar, (uint32_t)phase & 1u, abort_flag, err, ERR_ATTN_FULL)) != 0;
    };
    const uint64_t scale2 = f32x2(p.scale_log2, p.scale_log2);
    for (int t = 0; t < nt; ++t) {
      const int b = t & 1, key0 = (t0 + t) * KT;
      ok = wait(sfull, t) && ok;
      tc_fence_after();
      constexpr int KH = KT / 2;
      float s[KH];
      tmem_ld32(trow + C::S_COL + hf * KH, s);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(sfree);
      if (__builtin_expect(key0 + KT > lim_min, 0)) {     // some row does not see all of the tile
#pragma unroll
        for (int c = 0; c < KH; ++c) s[c] = key0 + hf * KH + c < lim ? s[c] : -INFINITY;
      }
      const int vn = s_vref[b];
      const bool wide = s_wide[b] != 0;
      uint32_t ph[KH / 2];
      // Most tiles: the references stand.  A sum under 2^14 in either half means that no
      // score is over its row's reference by 2^kRowSlack (P holds 2^7 p), so no
      // maximum is taken.
      bool redo = t == 0 || wide || vn != vref;
      uint64_t tile2 = 0;
      if (!redo) {
        const uint64_t off2 = f32x2(kPShift - m, kPShift - m);
        uint64_t sum[4] = {};
#pragma unroll
        for (int c = 0; c < KH; c += 2) {
          const float2 z = f32x2_get(fma_f32x2(f32x2(s[c], s[c + 1]), scale2, off2));
          const float p0 = ex2(z.x), p1 = ex2(z.y);
          sum[(c >> 1) & 3] = add_f32x2(sum[(c >> 1) & 3], f32x2(p0, p1));
          ph[c >> 1] = pack_f16x2(p0, p1);
        }
        tile2 = add_f32x2(add_f32x2(sum[0], sum[1]), add_f32x2(sum[2], sum[3]));
        const float2 both = f32x2_get(tile2);
        redo = both.x + both.y >= 32768.0f;
      }
      if (__builtin_expect(named_bar_or(3 + q4, 64, redo), 0)) {
        float top = s[0];
#pragma unroll
        for (int c = 1; c < KH; ++c) top = fmaxf(top, s[c]);
        s_top[hf * N + row] = top;
        named_bar_sync(3 + q4, 64);
        top = fmaxf(top, s_top[(hf ^ 1) * N + row]) * p.scale_log2;
        const bool up = t == 0 ? top > -INFINITY : top > m + kRowSlack;
        const bool moved = __any_sync(0xffffffffu, up) || (!wide && vn != vref);
        const float mn = up ? top : m;
        const float corr = t > 0 ? exp2f(m - mn) : 1.0f;  // of the row's old sums
        if (moved) l2 = mul_f32x2(l2, f32x2(corr, corr));
        // this half's dims of O times f
        auto rescale = [&](float f) {
          if (!wait(&pvdone[b ^ 1], (t - 1) >> 1)) {
            ok = false;
            return;
          }
          tc_fence_after();
#pragma unroll 1
          for (int c = hf * (HD / 2); c < (hf + 1) * (HD / 2); c += 16) {
            float o[16];
            tmem_ld16(trow + C::O_COL + c, o);
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] *= f;
            tmem_st16(trow + C::O_COL + c, o);
          }
          tc_fence_before();
        };
        tile2 = 0;
        if (!wide) {
          m = mn;
          // exponents below -126 leave nothing of the old sums that counts
          if (moved && t > 0) rescale(vref - vn < -126 ? 0.0f : corr * scale_value(127 + vref - vn));
          vref = vn;
          d = (float)vn;
#pragma unroll
          for (int c = 0; c < KH; c += 2) {
            const float p0 = ex2(fmaf(s[c], p.scale_log2, kPShift - m));
            const float p1 = ex2(fmaf(s[c + 1], p.scale_log2, kPShift - m));
            tile2 = add_f32x2(tile2, f32x2(p0, p1));
            ph[c >> 1] = pack_f16x2(p0, p1);
          }
        } else {
          if (t > 0) d -= mn - m;                         // the products keep their reference m + d
          m = mn;
          float most = -INFINITY;
#pragma unroll
          for (int c = 0; c < KH; ++c) {
            const float z = fmaf(s[c], p.scale_log2, -m);
            tile2 = add_f32x2(tile2, f32x2(ex2(z + kPShift), 0.0f));
            s[c] = z + (s_ev[b * KT + hf * KH + c] - d);
            most = fmaxf(most, s[c]);
          }
          s_most[hf * N + row] = most;
          named_bar_sync(3 + q4, 64);
          most = fmaxf(most, s_most[(hf ^ 1) * N + row]);
          const float un = most > -INFINITY && (t == 0 || most > kRowSlack) ? most : 0.0f;
          d += un;
          if (t > 0 && __any_sync(0xffffffffu, un != 0.0f)) rescale(exp2f(-un));
#pragma unroll
          for (int c = 0; c < KH; c += 2)
            ph[c >> 1] = pack_f16x2(ex2(s[c] - un + kPShift), ex2(s[c + 1] - un + kPShift));
        }
      }
      l2 = add_f32x2(l2, tile2);
      // P is free once the last product is done
      if (t > 0) ok = wait(&pvdone[b ^ 1], (t - 1) >> 1) && ok;
      tc_fence_after();
      tmem_st16(trow + C::P_COL + hf * (KH / 2), reinterpret_cast<const float*>(ph));
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&pready[b]);
    }
    // ------------------------------------------------------ output
    if (nt > 0) ok = wait(&pvdone[(nt - 1) & 1], (nt - 1) >> 1) && ok;
    tc_fence_after();
    const float2 lp = f32x2_get(l2);
    named_bar_sync(3 + q4, 64);
    s_top[hf * N + row] = lp.x + lp.y;
    named_bar_sync(3 + q4, 64);
    const float l_sum = s_top[row] + s_top[N + row];
    // 2^d in two steps: it alone may leave the range that the result is in
    const float f = l_sum == 0.0f ? 0.0f : exp2f(0.5f * d) / l_sum, f2 = exp2f(0.5f * d);
    uint32_t jh;
    const int i = (int)p.by_group.divmod((uint32_t)(rt * N + row), jh), h = g * p.group + (int)jh;
    const bool valid = row < n_rows;
    const long long ws_row = ((long long)(plane * p.row_tiles + rt) * p.splits + split) * N + row;
#pragma unroll 1
    for (int c = hf * (HD / 2); c < (hf + 1) * (HD / 2); c += 16) {
      float o[16] = {};
      if (nt > 0) tmem_ld16(trow + C::O_COL + c, o);
      if (l_sum == 0.0f) {
#pragma unroll
        for (int e = 0; e < 16; ++e) o[e] = 0.0f;         // a row that sees nothing
      }
      if (!valid) {
        // nothing to store; the loads above are the whole warp's
      } else if (p.splits > 1) {
        float4* dst = reinterpret_cast<float4*>(p.ws_o + ws_row * HD + c);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          dst[e] = make_float4(o[4 * e] * f * f2, o[4 * e + 1] * f * f2, o[4 * e + 2] * f * f2, o[4 * e + 3] * f * f2);
      } else {
        uint4* dst = reinterpret_cast<uint4*>(p.out + ((long long)seq * p.R + i) * p.o_rs + (long long)h * HD + c);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          uint32_t w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const __nv_bfloat162 v = __floats2bfloat162_rn(o[8 * e + 2 * k] * f * f2, o[8 * e + 2 * k + 1] * f * f2);
            w[k] = *reinterpret_cast<const uint32_t*>(&v);
          }
          dst[e] = make_uint4(w[0], w[1], w[2], w[3]);
        }
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
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

}  // namespace dllm
