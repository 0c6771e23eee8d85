// Attention over the 8-bit cache for many query rows a cached head (a prefill
// over its own cache): 128 rows a CTA, one a softmax thread.
//
//   S[row][key] = Q K^T      kind::mxf8f6f4; q as hi + lo codes (two products), the
//                            row's and the key's scales applied by the MMA
//   O[row][dim] += P V       kind::mxf8f6f4; P as hi + lo codes in tensor memory, each
//                            with a scale for a row's 32 keys; V MN-major from its TMA tile
// The codes of K and V are used as they lie in the cache; precision of q and P as in
// attn_kv8_rows.cuh.  Two e4m3 products cost what one bf16 product costs, so a
// tile of 128 rows by 128 keys takes the tensor cores 1024 cycles; the softmax
// needs about as many issue slots (10 a score over four schedulers), so two
// CTAs share an SM and one's products run under the other's exponentials.
// Tensor memory sets the tile: 64 keys make S 64 columns, P 32, O 128 and the
// scales 20, just under half of it.
//
//   warp 0     TMA: K and V tiles of 64 keys
//   warp 1     one thread issues scale copies and MMAs
//   warp 2     scale bytes: K's for the MMA, V's as factors of P
//   warps 3-6  softmax, one row a thread; the query tile before, the output after
#pragma once

#include "attn_kv8_rows.cuh"

namespace dllm {

template <int HD>
struct AttnTilesCfg {
  static constexpr int N = 128;                         // rows
  static constexpr int KT = 64;
  static constexpr int SLOT = KT * HD;
  static constexpr int SLOTS = 6;
  static constexpr int Q_BYTES = N * HD;                // hi or lo
  static constexpr int SF_BYTES = 512;                  // ones, query, two of K, P
  static constexpr int STAT_FLOATS = 2 * KT + 4 + N;    // value factors and block exponents (two buffers), limits
  static constexpr int SMEM_BYTES =
      1024 + SLOTS * SLOT + 2 * Q_BYTES + 5 * SF_BYTES + STAT_FLOATS * 4 + (2 * SLOTS + 10) * 8 + 16;
  static constexpr int S_COL = 0;
  static constexpr int P_COL = KT;                      // 16 columns of hi codes, 16 of lo
  static constexpr int O_COL = P_COL + 32;
  static constexpr int SF_ONE = O_COL + HD, SF_Q = SF_ONE + 4, SF_K = SF_Q + 4, SF_P = SF_K + 8;
  static constexpr int TMEM_COLS = 256;
  static_assert(SF_P + 4 <= TMEM_COLS, "tensor memory");
  static_assert(2 * (SMEM_BYTES + 1024) <= 228 * 1024, "two CTAs an SM");
};

template <int HD>
__global__ void __launch_bounds__(224, 2)
    attn_kv8_tiles_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                          const __grid_constant__ AttnKv8Params p) {
  using C = AttnTilesCfg<HD>;
  constexpr int KT = C::KT, N = C::N;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sKV = smem;
  uint8_t* sQ = sKV + C::SLOTS * C::SLOT;               // hi, lo
  uint8_t* sSF = sQ + 2 * C::Q_BYTES;                   // scale atoms: ones, queries, K (two), P
  float* s_vf = reinterpret_cast<float*>(sSF + 5 * C::SF_BYTES);   // [2][KT]
  int* s_eb = reinterpret_cast<int*>(s_vf + 2 * KT);    // [2][2]
  int* s_lim = s_eb + 4;                                // [N]
  uint64_t* full = reinterpret_cast<uint64_t*>(s_lim + N);
  uint64_t* empty = full + C::SLOTS;
  uint64_t* qready = empty + C::SLOTS;
  uint64_t* sfull = qready + 1;                         // S of a tile is there
  uint64_t* sfree = sfull + 1;                          // and has been read
  uint64_t* kready = sfree + 1;                         // [2] a tile's scales are there
  uint64_t* pready = kready + 2;                        // [2] its P
  uint64_t* pvdone = pready + 2;                        // its product
  uint64_t* vfixed = pvdone + 1;                        // the last tile's values past every limit are cleared
  uint64_t* mdone = vfixed + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mdone + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* err = g_attn_kv8_err;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = (int)(blockIdx.x % (unsigned)p.splits);
  const int item = (int)(blockIdx.x / (unsigned)p.splits);
  // the last row tiles first: under a causal mask they see the most keys
  const int planes = p.c.b * p.c.H_kv;
  const int rt = p.row_tiles - 1 - item / planes, plane = item % planes;
  const int seq = plane / p.c.H_kv, g = plane % p.c.H_kv;
  const int n_rows = min(N, p.rows - rt * N);

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::SLOTS; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(qready, 4);
    mbar_init(sfull, 1);
    mbar_init(sfree, 4);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&kready[s], 1);
      mbar_init(&pready[s], 4);
    }
    mbar_init(pvdone, 1);
    mbar_init(vfixed, 1);
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
    const int i = (rt * N + n) / p.group;
    const int lim = p.limits ? p.limits[(long long)seq * p.R + i] : p.c.T;
    s_lim[threadIdx.x] = min(max(lim, 0), p.c.T);
#pragma unroll
    for (int f = 0; f < 5; ++f) reinterpret_cast<uint32_t*>(sSF + f * C::SF_BYTES)[threadIdx.x] = 0x7f7f7f7fu;   // 1.0
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

  if (warp == 0) {
    if (lane == 0) {
      const uint64_t pol = policy_evict_last();           // the other row tiles read the same keys
      RingPos r{0, 0u};
      int issued = 0;
      for (int u = 0; u < 2 * nt; ++u) {
        if (u >= C::SLOTS && !mbar_wait(&empty[r.s], r.par ^ 1u, abort_flag, err, ERR_ATTN_FULL)) break;
        mbar_arrive_expect_tx(&full[r.s], C::SLOT);
        tma_load_3d(sKV + r.s * C::SLOT, (u & 1) ? &tmV : &tmK, &full[r.s], 0, (t0 + (u >> 1)) * KT, plane, pol);
        r.next(C::SLOTS);
        issued = u + 1;
      }
      if (*abort_flag)   // let copies in flight land before the CTA's shared memory goes away
        for (int u = issued > C::SLOTS ? issued - C::SLOTS : 0; u < issued; ++u)
          mbar_wait(&full[u % C::SLOTS], (uint32_t)(u / C::SLOTS) & 1u, nullptr, err, ERR_ATTN_FULL);
    }
  } else if (warp == 1) {
    if (lane == 0 && nt > 0 && mbar_wait(qready, 0u, abort_flag, err, ERR_ATTN_FULL)) {
      tc_fence_after();
      constexpr uint32_t idesc_s = idesc_mxf8(128, KT);
      constexpr uint32_t idesc_o = idesc_mxf8(128, HD) | (1u << 16);   // V MN-major
      const uint32_t q0 = smem_u32(sQ), kv0 = smem_u32(sKV), f0 = smem_u32(sSF);
      tmem_cp_scales(tmem + C::SF_ONE, sdesc_scales(f0));
      tmem_cp_scales(tmem + C::SF_Q, sdesc_scales(f0 + C::SF_BYTES));
      auto wait = [&](uint64_t* bar, uint32_t par) { return mbar_wait(bar, par, abort_flag, err, ERR_ATTN_FULL); };
      auto issue_s = [&](int t) {
        const int u = 2 * t, slot = u % C::SLOTS, b = t & 1;
        if ((t > 0 && !wait(sfree, (uint32_t)(t - 1) & 1u)) || !wait(&full[slot], (uint32_t)(u / C::SLOTS) & 1u) ||
            !wait(&kready[b], (uint32_t)(t >> 1) & 1u))
          return false;
        tc_fence_after();
        const uint32_t k = kv0 + slot * C::SLOT, sfk = tmem + C::SF_K + 4 * b;
        tmem_cp_scales(sfk, sdesc_scales(f0 + (2 + b) * C::SF_BYTES));
#pragma unroll
        for (int part = 0; part < 2; ++part)
#pragma unroll
          for (int kk = 0; kk < HD / 32; ++kk)
            mma_mxf8_ss(tmem + C::S_COL, sdesc_rows<HD>(q0 + part * C::Q_BYTES + kk * 32), sdesc_rows<HD>(k + kk * 32),
                        idesc_s, tmem + C::SF_Q, sfk, (part > 0 || kk > 0) ? 1u : 0u);
        mma_commit(&empty[slot]);
        mma_commit(sfull);
        return true;
      };
      bool ok = issue_s(0);
      for (int t = 0; t < nt && ok; ++t) {
        // the next tile's scores as soon as these have been read
        if (t + 1 < nt && !(ok = issue_s(t + 1))) break;
        const int u = 2 * t + 1, slot = u % C::SLOTS;
        if (!(ok = wait(&pready[t & 1], (uint32_t)(t >> 1) & 1u) && wait(&full[slot], (uint32_t)(u / C::SLOTS) & 1u)))
          break;
        if ((t0 + t + 1) * KT > lim_max && !(ok = wait(vfixed, 0u))) break;
        tc_fence_after();
        const uint32_t v = kv0 + slot * C::SLOT;
        tmem_cp_scales(tmem + C::SF_P, sdesc_scales(f0 + 4 * C::SF_BYTES));
#pragma unroll
        for (int part = 0; part < 2; ++part)
#pragma unroll
          for (int kk = 0; kk < KT / 32; ++kk)
            // P's scale bytes of a row: hi of the first 32 keys, hi of the second, lo, lo
            mma_mxf8_ts(tmem + C::O_COL, tmem + C::P_COL + part * 16 + kk * 8, sdesc_rows<HD>(v + kk * 32 * HD),
                        idesc_o | ((uint32_t)(2 * part + kk) << 29), tmem + C::SF_P, tmem + C::SF_ONE,
                        (t > 0 || part > 0 || kk > 0) ? 1u : 0u);
        mma_commit(&empty[slot]);
        mma_commit(pvdone);
      }
      mma_commit(mdone);
      mbar_wait(mdone, 0u, nullptr, err, ERR_ATTN_FULL);
    }
  } else if (warp == 2) {
    // ------------------------------------------------------ scale bytes, keys lane and lane + 32 of a tile
    const uint8_t* ksc = p.c.k_scale + (long long)plane * p.c.T;
    const uint8_t* vsc = p.c.v_scale + (long long)plane * p.c.T;
    constexpr int AHEAD = 4;
    int kn[AHEAD][2], vn[AHEAD][2];
    auto fetch = [&](int t) {
#pragma unroll
      for (int e = 0; e < AHEAD; ++e)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int key = (t0 + t + e) * KT + 32 * j + lane;
          const bool in = t + e < nt && key < lim_max;
          kn[e][j] = in ? __ldg(ksc + key) : 127;
          vn[e][j] = in ? __ldg(vsc + key) : -1;          // past every limit
        }
    };
    if (nt > 0) fetch(0);
    bool ok = true;
    for (int tb = 0; tb < nt && ok; tb += AHEAD) {
      int kc[AHEAD][2], vc[AHEAD][2];
#pragma unroll
      for (int e = 0; e < AHEAD; ++e)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          kc[e][j] = kn[e][j];
          vc[e][j] = vn[e][j];
        }
      fetch(tb + AHEAD);
#pragma unroll
      for (int e = 0; e < AHEAD; ++e) {
        const int t = tb + e, b = t & 1;
        if (t >= nt || !ok) break;
        // tile t - 2's scores are computed and its factors read once its P is there
        if (t >= 2 && !__all_sync(0xffffffffu, mbar_wait(&pready[b], (uint32_t)((t >> 1) - 1) & 1u, abort_flag, err,
                                                         ERR_ATTN_FULL))) {
          ok = false;
          break;
        }
        uint32_t word[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const bool bad = kc[e][j] == kScaleNan || vc[e][j] == kScaleNan;
          const int ev = vc[e][j] < 0 || bad ? -1000 : vc[e][j] - 127;
          const int top = __reduce_max_sync(0xffffffffu, ev);   // of the 32 keys
          // a bad value makes the score NaN, so that only rows that see it are
          word[j] = (bad ? 255u : (uint32_t)kc[e][j]) * 0x01010101u;
          s_vf[b * KT + 32 * j + lane] = ev == -1000 ? 0.0f : __uint_as_float((uint32_t)(127 + max(ev - top, -126)) << 23);
          if (lane == 0) s_eb[b * 2 + j] = top;
        }
        *reinterpret_cast<uint2*>(sSF + (2 + b) * C::SF_BYTES + lane * 16) = make_uint2(word[0], word[1]);
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&kready[b]);
      }
    }
    if (nt > 0 && ok && (t0 + nt) * KT > lim_max) {
      // whatever bytes lie past every limit (codes of NaN among them) must not meet the zero probabilities
      const int u = 2 * nt - 1, slot = u % C::SLOTS;
      if (__all_sync(0xffffffffu, mbar_wait(&full[slot], (uint32_t)(u / C::SLOTS) & 1u, abort_flag, err, ERR_ATTN_FULL))) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int key_l = 32 * j + lane;
          if ((t0 + nt - 1) * KT + key_l >= lim_max) {
#pragma unroll
            for (int c = 0; c < HD / 16; ++c)
              *reinterpret_cast<uint4*>(sKV + slot * C::SLOT + key_l * HD + c * 16) = make_uint4(0, 0, 0, 0);
          }
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(vfixed);
      }
    }
  } else {
    const int q4 = warp & 3, row = q4 * 32 + lane, tid = (warp - 3) * 32 + lane;
    const uint32_t trow = tmem + ((uint32_t)(q4 * 32) << 16);
    const int lim = s_lim[row];
    if (nt > 0) {
      // ---------------------------------------------------- the query tile
      constexpr int L = HD / 8;                           // lanes of a row
#pragma unroll 4
      for (int n0 = 0; n0 < N; n0 += 128 / L) {
        const int n = n0 + tid / L, l = tid % L;
        float x[8] = {};
        if (n < n_rows) {
          const int rn = rt * N + n, i = rn / p.group, h = g * p.group + rn % p.group;
          ElemBf16::load8(reinterpret_cast<const __nv_bfloat16*>(p.q) + ((long long)seq * p.R + i) * p.q_rs +
                              (long long)h * HD + l * 8,
                          x);
        }
        uint32_t m = abs_bits8(x);
#pragma unroll
        for (int d = L / 2; d >= 1; d >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
        const int byte = scale_byte(m);
        const float inv = byte == kScaleNan ? __uint_as_float(0x7fffffffu) : scale_inverse(byte);
        float r[8], b[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) r[e] = x[e] * inv;    // a row that is not finite becomes NaN
        const uint2 hi = encode8(r, 1.0f);
        decode8(hi, 1.0f, b);
#pragma unroll
        for (int e = 0; e < 8; ++e) b[e] = r[e] - b[e];
        const uint2 lo = encode8(b, 1.0f);
        const uint32_t off = swizzled<HD>(n, l >> 1) + (uint32_t)(l & 1) * 8;
        *reinterpret_cast<uint2*>(sQ + off) = hi;
        *reinterpret_cast<uint2*>(sQ + C::Q_BYTES + off) = lo;
        if (l == 0 && byte != kScaleNan)
          reinterpret_cast<uint32_t*>(sSF + C::SF_BYTES)[(n & 31) * 4 + (n >> 5)] = (uint32_t)byte * 0x01010101u;
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(qready);
    }
    // ------------------------------------------------------ the keys
    float m = 0.0f, l_sum = 0.0f;                         // reference (base 2) and sum of this row
    int vref = 0;
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t par) {        // decided warp-wide: tensor-memory accesses are collective
      return __all_sync(0xffffffffu, mbar_wait(bar, par, abort_flag, err, ERR_ATTN_FULL)) != 0;
    };
    for (int t = 0; t < nt && ok; ++t) {
      const int b = t & 1, key0 = (t0 + t) * KT;
      if (!(ok = wait(sfull, (uint32_t)t & 1u))) break;
      tc_fence_after();
      float s[KT];
      tmem_ld32(trow + C::S_COL, s);
      tmem_ld32(trow + C::S_COL + 32, s + 32);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(sfree);
      if (key0 + KT > lim_min) {                          // some row does not see all of the tile
#pragma unroll
        for (int c = 0; c < KT; ++c) s[c] = key0 + c < lim ? s[c] : -INFINITY;
      }
      float mx = -INFINITY;
#pragma unroll
      for (int c = 0; c < KT; ++c) mx = fmaxf(mx, s[c]);
      mx *= p.scale_log2;
      const int eb0 = s_eb[b * 2], eb1 = s_eb[b * 2 + 1];
      // The row's reference rises when a score exceeds it by 2^8, and the common
      // value reference when a key's exponent exceeds it by 40: float32 sums and
      // the block scales have the range for what lies between.
      const bool up = t == 0 ? mx > -INFINITY : mx > m + 8.0f;
      const bool vup = t == 0 || max(eb0, eb1) - vref > 40;
      if (__any_sync(0xffffffffu, up) || vup) {
        const float mn = up ? mx : m;
        const int vn = vup ? max(max(eb0, eb1), t == 0 ? -127 : vref) : vref;
        if (t > 0) {
          if (!(ok = wait(pvdone, (uint32_t)(t - 1) & 1u))) break;
          tc_fence_after();
          const float corr = exp2f(m - mn);
          const float ocorr = vref - vn < -126 ? 0.0f : corr * scale_value(127 + vref - vn);
          l_sum *= corr;
#pragma unroll 1
          for (int c = 0; c < HD; c += 32) {
            float o[32];
            tmem_ld32(trow + C::O_COL + c, o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] *= ocorr;
            tmem_st32(trow + C::O_COL + c, o);
          }
          tc_fence_before();
        }
        m = mn;
        vref = vn;
      }
      uint32_t hi[16], lo[16], word = 0;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float4* vf = reinterpret_cast<const float4*>(s_vf + b * KT + 32 * j);
        float top = 0.0f;
#pragma unroll
        for (int c = 0; c < 32; c += 4) {
          const float4 f = vf[c >> 2];
          float* x = s + 32 * j + c;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float pr = ex2(fmaf(x[e], p.scale_log2, -m));
            l_sum += pr;
            x[e] = pr * (e == 0 ? f.x : e == 1 ? f.y : e == 2 ? f.z : f.w);
            top = fmaxf(top, x[e]);
          }
        }
        // scaled so that the block's largest lies in [128, 256)
        const int be = max((int)(__float_as_uint(top) >> 23) - 7, 1);
        const float inv = __uint_as_float((uint32_t)(254 - be) << 23);
        const int byte = min(max(be + (j ? eb1 : eb0) - vref, 4), 254);
        word |= (uint32_t)byte << (8 * j) | (uint32_t)(byte - 4) << (16 + 8 * j);
#pragma unroll
        for (int c = 0; c < 32; c += 4) {
          const float* x = s + 32 * j + c;
          const uint32_t x0 = pack_f16x2(x[0] * inv, x[1] * inv), x1 = pack_f16x2(x[2] * inv, x[3] * inv);
          const uint32_t h0 = cvt_e4m3x2_f16x2(x0), h1 = cvt_e4m3x2_f16x2(x1);
          hi[8 * j + (c >> 2)] = h0 | (h1 << 16);
          lo[8 * j + (c >> 2)] = cvt_e4m3x2_f16x2(sub_mul16_f16x2(x0, cvt_f16x2_e4m3x2((uint16_t)h0))) |
                                 (cvt_e4m3x2_f16x2(sub_mul16_f16x2(x1, cvt_f16x2_e4m3x2((uint16_t)h1))) << 16);
        }
      }
      // P is free once the last product is done
      if (t > 0 && !(ok = wait(pvdone, (uint32_t)(t - 1) & 1u))) break;
      tc_fence_after();
      tmem_st16(trow + C::P_COL, reinterpret_cast<const float*>(hi));
      tmem_st16(trow + C::P_COL + 16, reinterpret_cast<const float*>(lo));
      reinterpret_cast<uint32_t*>(sSF + 4 * C::SF_BYTES)[lane * 4 + q4] = word;
      fence_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&pready[b]);
    }
    // ------------------------------------------------------ output
    if (nt > 0 && ok) ok = wait(pvdone, (uint32_t)(nt - 1) & 1u);
    tc_fence_after();
    const float f = l_sum == 0.0f ? 0.0f : scale_value(127 + vref) / l_sum;
    const int rn = rt * N + row, i = rn / p.group, h = g * p.group + rn % p.group;
    const bool valid = row < n_rows;
    const long long ws_row = ((long long)(plane * p.row_tiles + rt) * p.splits + split) * N + row;
#pragma unroll 1
    for (int c = 0; c < HD; c += 32) {
      float o[32];
      if (nt > 0) {
        tmem_ld32(trow + C::O_COL + c, o);
      } else {
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = 0.0f;
      }
      if (l_sum == 0.0f) {
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = 0.0f;         // a row that sees nothing
      }
      if (!valid) {
        // nothing to store; the loads above are the whole warp's
      } else if (p.splits > 1) {
        float4* dst = reinterpret_cast<float4*>(p.ws_o + ws_row * HD + c);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          dst[e] = make_float4(o[4 * e] * f, o[4 * e + 1] * f, o[4 * e + 2] * f, o[4 * e + 3] * f);
      } else {
        uint4* dst = reinterpret_cast<uint4*>(p.out + ((long long)seq * p.R + i) * p.o_rs + (long long)h * HD + c);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const __nv_bfloat162 v = __floats2bfloat162_rn(o[8 * e + 2 * k] * f, o[8 * e + 2 * k + 1] * f);
            w[k] = *reinterpret_cast<const uint32_t*>(&v);
          }
          dst[e] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
    }
    if (valid && p.splits > 1) *reinterpret_cast<float2*>(p.ws_ml + ws_row * 2) = make_float2(m, l_sum);
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
