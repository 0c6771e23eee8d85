// 8-bit matrix product with a scale for each block of 128 along K, and the
// quantiser of its operands (see q8.cuh):
//   Y[n][m] = sum_B 2^(ex[B][n] + ew[B][m]) * sum_{k in block B} X[n][k] W[m][k]
#include <algorithm>

#include "gemm.cuh"
#include "ops8.h"
#include "ptx8.cuh"
#include "q8.cuh"

namespace dllm {

constexpr int kQBlock = 128;

// ---------------------------------------------------------------- quantiser
// Bound by HBM.  A group of 16 lanes owns a block of 128 elements, 8 each; a
// thread group has kQAhead blocks in flight.
constexpr int kQAhead = 4;

struct Quantise8Params {
  const void* x;
  uint8_t *codes, *scales;
  long long rs;
  int rows, K;
  uint32_t groups;     // rows * blocks of a row
  FastDiv blocks;
};

template <typename E, bool VEC>
__global__ void __launch_bounds__(256, 4) quantise8_kernel(const __grid_constant__ Quantise8Params p) {
  const int l = threadIdx.x & 15;
  griddep_launch_dependents();
  griddep_wait();
  const uint32_t g0 = blockIdx.x * (uint32_t)(16 * kQAhead) + (threadIdx.x >> 4);
  Raw8<E> raw[kQAhead];
  uint32_t row[kQAhead], B[kQAhead];
#pragma unroll
  for (int j = 0; j < kQAhead; ++j) {
    const uint32_t g = g0 + 16 * j;
    row[j] = p.blocks.divmod(g, B[j]);
    const int k0 = (int)B[j] * kQBlock + l * 8;
    raw[j].zero();
    if (g < p.groups && k0 < p.K) {            // K % 16 == 0: a lane's 8 elements are all in or all out
      const typename E::T* px = static_cast<const typename E::T*>(p.x) + row[j] * p.rs + k0;
      if constexpr (VEC) {
        raw[j].load(px);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) reinterpret_cast<typename E::T*>(raw[j].w)[e] = px[e];
      }
    }
  }
#pragma unroll
  for (int j = 0; j < kQAhead; ++j) {
    float x[8];
    raw[j].floats(x);
    uint32_t m = abs_bits8(x);
#pragma unroll
    for (int d = 8; d >= 1; d >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
    const int byte = scale_byte(m);
    if (g0 + 16 * j >= p.groups) continue;
    const int k0 = (int)B[j] * kQBlock + l * 8;
    if (k0 < p.K) {
      uint2 c = make_uint2(0, 0);
      if (byte != kScaleNan) c = encode8(x, scale_inverse(byte));
      *reinterpret_cast<uint2*>(p.codes + (long long)row[j] * p.K + k0) = c;
    }
    if (l == 0) p.scales[(long long)B[j] * p.rows + row[j]] = (uint8_t)byte;
  }
}

// ---------------------------------------------------------------- product
struct Gemm8Params {
  const uint8_t *ws, *xs;
  void* y;
  int M, N, K, kb, n_tiles, split_log, out_bf16;
};

// Set by a kernel that gave up a bounded wait; read by dllm_op_check.
static __device__ int g_gemm8_err[1];

template <int BN>
struct Gemm8Cfg {
  static constexpr int A_BYTES = 128 * kQBlock;
  static constexpr int B_BYTES = BN * kQBlock;
  static constexpr int SFB_ATOMS = (BN + 127) / 128;
  static constexpr int SF_BYTES = 512 * (1 + SFB_ATOMS);
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES + SF_BYTES;
  static constexpr int STAGES = BN == 32 ? 5 : BN == 64 ? 4 : 3;   // two CTAs an SM
  static constexpr int SMEM_BYTES = 1024 + STAGES * STAGE_BYTES + (2 * STAGES + 1) * 8 + 16;
  static constexpr int SF_COL = BN;                       // scale columns behind the accumulator
  static constexpr int SF_COLS = 4 * (1 + SFB_ATOMS);     // a stage's
  static constexpr int TMEM_COLS = BN + STAGES * SF_COLS <= 128 ? 128 : 256;
  static_assert(BN + STAGES * SF_COLS <= TMEM_COLS, "tensor memory");
  static_assert(2 * (SMEM_BYTES + 1024) <= 228 * 1024, "two CTAs an SM");
  static_assert(STAGES * STAGE_BYTES >= BN * 128 * 4, "the ring holds the partial tile");
};

// Weights are the 128-row A operand, BN activation rows the B operand, both in
// 128-byte swizzled TMA tiles of one scale block (128 codes) of K.  The
// scales never meet the CUDA cores as numbers: UE8M0 bytes go to tensor
// memory and the block-scaled tcgen05.mma applies them, so blocks accumulate
// in one float32 accumulator.  A CTA computes a share of one tile's K; the
// `split` CTAs of a cluster share a tile and join their partial tiles through
// distributed shared memory in rank order.  Bound by HBM, on the GPU with the quantiser's launch:
// 24576 x 4096 weights, 32 rows, 20 us, 5.3 TB/s; 4096 x 4096, one row, 6.3 us.
//   warp 0     TMA: weight and activation codes
//   warp 1     scale copies and MMAs, issued by one lane
//   warps 2-5  epilogue
//   warp 6     scale bytes: one row's byte replicated over a 32-bit word, in the
//              512-byte layout tcgen05.cp wants (row r at (r % 32) * 16 + (r / 32) * 4)
template <int BN>
__global__ void __launch_bounds__(224, 2)
    gemm8_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                 const __grid_constant__ Gemm8Params p) {
  using C = Gemm8Cfg<BN>;
  constexpr int S = C::STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = smem;
  uint8_t* sB = smem + S * C::A_BYTES;
  uint8_t* sF = sB + S * C::B_BYTES;
  uint64_t* full = reinterpret_cast<uint64_t*>(sF + S * C::SF_BYTES);
  uint64_t* empty = full + S;
  uint64_t* done = empty + S;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* err = g_gemm8_err;

  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int sl = p.split_log, split = 1 << sl, rank = sl ? (int)cluster_rank() : 0;
  const int tile = (int)(blockIdx.x >> sl);
  const int m0 = tile / p.n_tiles * 128, n0 = tile % p.n_tiles * BN;
  const int c0 = (int)((long long)p.kb * rank >> sl), c1 = (int)((long long)p.kb * (rank + 1) >> sl);
  const int nc = c1 - c0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 2);
      mbar_init(&empty[s], 1);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tensormap(&tmW);
    prefetch_tensormap(&tmX);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  griddep_launch_dependents();
  griddep_wait();

  if (warp == 0) {
    if (lane == 0) {
      const uint64_t pol_w = policy_evict_first(), pol_x = policy_evict_last();
      RingPos r{0, 0u};
      int issued = 0;
      for (int i = 0; i < nc; ++i) {
        if (i >= S && !mbar_wait_long(&empty[r.s], r.par ^ 1u, abort_flag, err, ERR_GEMM_EMPTY)) break;
        mbar_arrive_expect_tx(&full[r.s], C::A_BYTES + C::B_BYTES);
        tma_load_3d(sA + r.s * C::A_BYTES, &tmW, &full[r.s], (c0 + i) * kQBlock, m0, 0, pol_w);
        tma_load_3d(sB + r.s * C::B_BYTES, &tmX, &full[r.s], (c0 + i) * kQBlock, n0, 0, pol_x);
        r.next(S);
        issued = i + 1;
      }
      if (*abort_flag)   // let copies in flight land before the CTA's shared memory goes away
        for (int i = issued > S ? issued - S : 0; i < issued; ++i)
          mbar_wait_long(&full[i % S], (uint32_t)(i / S) & 1u, nullptr, err, ERR_GEMM_DRAIN);
    }
  } else if (warp == 1) {
    const uint32_t lead = elect_one();
    constexpr uint32_t idesc = idesc_mxf8(128, BN);
    RingPos r{0, 0u};
    for (int i = 0; i < nc; ++i) {
      if (!__all_sync(0xffffffffu, mbar_wait_long(&full[r.s], r.par, abort_flag, err, ERR_GEMM_FULL))) break;
      tc_fence_after();
      const uint32_t a0 = smem_u32(sA + r.s * C::A_BYTES), b0 = smem_u32(sB + r.s * C::B_BYTES);
      const uint32_t f0 = smem_u32(sF + r.s * C::SF_BYTES);
      // a stage's scale columns are rewritten only once its MMAs are done (the empty barrier)
      const uint32_t sfa = tmem + (uint32_t)(C::SF_COL + r.s * C::SF_COLS), sfb = sfa + 4;
      tmem_cp_scales(lead, sfa, sdesc_scales(f0));
#pragma unroll
      for (int t = 0; t < C::SFB_ATOMS; ++t) tmem_cp_scales(lead, sfb + 4 * t, sdesc_scales(f0 + 512 * (t + 1)));
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
        mma_mxf8_ss(lead, tmem, sdesc_sw128(a0 + kk * 32), sdesc_sw128(b0 + kk * 32), idesc, sfa, sfb,
                    (i > 0 || kk > 0) ? 1u : 0u);
      mma_commit_lead(lead, &empty[r.s]);
      r.next(S);
    }
    mma_commit_lead(lead, done);
  } else if (warp == 6) {
    // Four blocks' bytes in use, the next four's in flight: fetched one at a
    // time, their latency was the block's time (0.7 us, where HBM needs 0.4).
    constexpr int AHEAD = 4, WB = (BN + 31) / 32;
    uint32_t wa[AHEAD][4], wb[AHEAD][WB];
    auto fetch = [&](int i0) {
#pragma unroll
      for (int e = 0; e < AHEAD; ++e) {
        const long long B = c0 + i0 + e;
        const bool in = i0 + e < nc;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int m = m0 + lane + 32 * j;
          wa[e][j] = in && m < p.M ? p.ws[B * p.M + m] : 127u;
        }
#pragma unroll
        for (int j = 0; j < WB; ++j) {
          const int n = n0 + lane + 32 * j;
          wb[e][j] = in && n < p.N ? p.xs[B * p.N + n] : 127u;
        }
      }
    };
    RingPos r{0, 0u};
    fetch(0);
    bool ok = true;
    for (int i0 = 0; i0 < nc && ok; i0 += AHEAD) {
      uint32_t ca[AHEAD][4], cb[AHEAD][WB];
#pragma unroll
      for (int e = 0; e < AHEAD; ++e) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          due(wa[e][j]);
          ca[e][j] = wa[e][j];
        }
#pragma unroll
        for (int j = 0; j < WB; ++j) {
          due(wb[e][j]);
          cb[e][j] = wb[e][j];
        }
      }
      fetch(i0 + AHEAD);
#pragma unroll
      for (int e = 0; e < AHEAD; ++e) {
        if (i0 + e >= nc || !ok) break;
        if (i0 + e >= S &&
            !__all_sync(0xffffffffu, mbar_wait_long(&empty[r.s], r.par ^ 1u, abort_flag, err, ERR_GEMM_EMPTY))) {
          ok = false;
          break;
        }
        uint4* f = reinterpret_cast<uint4*>(sF + r.s * C::SF_BYTES) + lane;
        constexpr uint32_t rep = 0x01010101u;
        f[0] = make_uint4(ca[e][0] * rep, ca[e][1] * rep, ca[e][2] * rep, ca[e][3] * rep);
#pragma unroll
        for (int t = 0; t < C::SFB_ATOMS; ++t) {
          uint32_t w4[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) w4[j] = 4 * t + j < WB ? cb[e][4 * t + j < WB ? 4 * t + j : 0] * rep : 127u * rep;
          f[32 * (t + 1)] = make_uint4(w4[0], w4[1], w4[2], w4[3]);
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[r.s]);
        r.next(S);
      }
    }
  }
  __syncwarp();

  // epilogue: thread = weight row, columns = activation rows
  const int q = warp & 3, l128 = q * 32 + lane, m = m0 + l128;
  const bool epi = warp >= 2 && warp < 6;
  const int cols = min(BN, p.N - n0);
  if (epi) {
    const bool ok = __all_sync(0xffffffffu, mbar_wait_long(done, 0u, abort_flag, err, ERR_GEMM_TFULL));
    (void)ok;   // after a wait that gave up the outputs are invalid and reported as such
    tc_fence_after();
  }
  if (split == 1) {
    if (epi) {
      for (int n = 0; n < cols; n += 32) {
        float v[32];
        tmem_ld32(tmem + ((uint32_t)(q * 32) << 16) + n, v);
        if (m < p.M) {
          long long o = (long long)(n0 + n) * p.M + m;
          if (p.out_bf16) {
            __nv_bfloat16* y = static_cast<__nv_bfloat16*>(p.y);
#pragma unroll
            for (int j = 0; j < 32; ++j, o += p.M)
              if (n + j < cols) y[o] = __float2bfloat16_rn(v[j]);
          } else {
            float* y = static_cast<float*>(p.y);
#pragma unroll
            for (int j = 0; j < 32; ++j, o += p.M)
              if (n + j < cols) y[o] = v[j];
          }
        }
      }
    }
  } else {
    // every CTA's MMAs and copies are done: the rings hold partial tiles now.
    // Rank r owns the columns r, r + split, ... and gets each from every rank.
    float* part = reinterpret_cast<float*>(smem);        // [source rank][owned column][128]
    const int own = (BN + split - 1) >> sl;
    uint32_t to[8];                                      // this thread's place in every rank
#pragma unroll
    for (int k = 0; k < 8; ++k)
      to[k] = cluster_addr(smem_u32(part) + 4u * (uint32_t)(rank * own * 128 + l128), (uint32_t)(k & (split - 1)));
    cluster_sync();
    if (epi) {
#pragma unroll 1
      for (int n = 0; n < cols; n += 8) {
        float v[8];
        tmem_ld8(tmem + ((uint32_t)(q * 32) << 16) + n, v);
#pragma unroll
        for (int j = 0; j < 8; ++j)                      // column n + j: rank (n + j) % split = j % split
          if (n + j < cols) cluster_store(to[j] + 512u * (uint32_t)((n + j) >> sl), v[j]);
      }
    }
    cluster_sync();
    if (epi && m < p.M) {
#pragma unroll 1
      for (int i = 0; (i << sl) + rank < cols; ++i) {
        float v = 0.0f;
#pragma unroll
        for (int s = 0; s < 8; ++s)
          if (s < split) v += part[(s * own + i) * 128 + l128];
        const long long o = (long long)(n0 + (i << sl) + rank) * p.M + m;
        if (p.out_bf16)
          static_cast<__nv_bfloat16*>(p.y)[o] = __float2bfloat16_rn(v);
        else
          static_cast<float*>(p.y)[o] = v;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

// ---------------------------------------------------------------- many rows
// The same product for activations of hundreds of rows, bound by the tensor cores
// and by what L2 delivers to them: at the MMA's full rate a tile of 128 x 128 asks
// for 128 bytes a cycle and SM (measured: about 50 were delivered, 38% of the rate), one of 128 x 192 for
// 107.  A CTA is persistent, one an SM, with two accumulators, so that storing one tile overlaps the next
// one's products.  12288 x 4096 weights, 2048 rows, on the GPU: 80 us with the quantiser, 2.6 PFLOP/s; a block of
// K takes about 650 cycles, in which an SM takes in its 40 KB of operands, for 384 cycles of products.  Tiles of 256 x 192
// (28 KB for the same products, but no accumulator left to store from): 85 us there, 144 against 156 for 24576 x 4096,
// and 22-27 against 15-19 where one round of the smaller tiles is enough.
//   warp 0     TMA: weight and activation codes
//   warp 1     scale copies and MMAs, issued by one lane
//   warp 2     weight scale bytes, warp 3 activation scale bytes
//   warps 4-7  epilogue
struct Gemm8BigCfg {
  static constexpr int BN = 192;
  static constexpr int A_BYTES = 128 * kQBlock;
  static constexpr int B_BYTES = BN * kQBlock;
  static constexpr int SF_BYTES = 3 * 512;
  static constexpr int STAGES = 5;
  static constexpr int SMEM_BYTES = 1024 + STAGES * (A_BYTES + B_BYTES + SF_BYTES) + (2 * STAGES + 5) * 8 + 16;
  static constexpr int SF_COL = 2 * BN, SF_COLS = 12;
  static_assert(SF_COL + STAGES * SF_COLS <= 512, "tensor memory");
  static_assert(SMEM_BYTES <= 232448, "shared memory");
};

__global__ void __launch_bounds__(256, 1)
    gemm8_big_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                     const __grid_constant__ Gemm8Params p) {
  using C = Gemm8BigCfg;
  constexpr int S = C::STAGES, BN = C::BN;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = smem;
  uint8_t* sB = smem + S * C::A_BYTES;
  uint8_t* sF = sB + S * C::B_BYTES;
  uint64_t* full = reinterpret_cast<uint64_t*>(sF + S * C::SF_BYTES);
  uint64_t* empty = full + S;
  uint64_t* tfull = empty + S;    // [2] an accumulator is complete
  uint64_t* tempty = tfull + 2;   // [2] and has been read
  uint64_t* mdone = tempty + 2;   // every MMA is done (before tensor memory is freed)
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mdone + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* err = g_gemm8_err;

  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int total = (p.M + 127) / 128 * p.n_tiles;   // tiles of 128 x BN

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 3);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 4);
    }
    mbar_init(mdone, 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tensormap(&tmW);
    prefetch_tensormap(&tmX);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  griddep_launch_dependents();
  griddep_wait();

  auto wait = [&](uint64_t* bar, uint32_t parity, int site) {
    return __all_sync(0xffffffffu, mbar_wait_long(bar, parity, abort_flag, err, site)) != 0;
  };
  if (warp == 0) {
    const uint32_t lead = elect_one();
    const uint64_t pol_w = policy_evict_first(), pol_x = policy_evict_last();
    RingPos r{0, 0u};
    int issued = 0;
    bool ok = true;
    for (int t = (int)blockIdx.x; t < total && ok; t += (int)gridDim.x) {
      const int m0 = t / p.n_tiles * 128, n0 = t % p.n_tiles * BN;
      for (int i = 0; i < p.kb; ++i) {
        if (issued >= S && !(ok = wait(&empty[r.s], r.par ^ 1u, ERR_GEMM_EMPTY))) break;
        if (lead) {
          mbar_arrive_expect_tx(&full[r.s], C::A_BYTES + C::B_BYTES);
          tma_load_3d(sA + r.s * C::A_BYTES, &tmW, &full[r.s], i * kQBlock, m0, 0, pol_w);
          tma_load_3d(sB + r.s * C::B_BYTES, &tmX, &full[r.s], i * kQBlock, n0, 0, pol_x);
        }
        r.next(S);
        ++issued;
      }
    }
    if (*abort_flag)   // let copies in flight land before the CTA's shared memory goes away
      for (int i = max(issued - S, 0); i < issued; ++i)
        mbar_wait_long(&full[i % S], (uint32_t)(i / S) & 1u, nullptr, err, ERR_GEMM_DRAIN);
  } else if (warp == 1) {
    const uint32_t lead = elect_one();
    constexpr uint32_t idesc = idesc_mxf8(128, BN);
    RingPos r{0, 0u};
    bool ok = true;
    int n = 0;
    for (int t = (int)blockIdx.x; t < total && ok; t += (int)gridDim.x, ++n) {
      const uint32_t d = tmem + (uint32_t)((n & 1) * BN);
      if (n >= 2 && !(ok = wait(&tempty[n & 1], (uint32_t)((n >> 1) - 1) & 1u, ERR_GEMM_TEMPTY))) break;
      tc_fence_after();
      for (int i = 0; i < p.kb; ++i) {
        if (!(ok = wait(&full[r.s], r.par, ERR_GEMM_FULL))) break;
        tc_fence_after();
        const uint32_t a0 = smem_u32(sA + r.s * C::A_BYTES), b0 = smem_u32(sB + r.s * C::B_BYTES);
        const uint32_t f0 = smem_u32(sF + r.s * C::SF_BYTES);
        // a stage's scale columns are rewritten only once its MMAs are done (the empty barrier)
        const uint32_t sfa = tmem + (uint32_t)(C::SF_COL + r.s * C::SF_COLS), sfb = sfa + 4;
        tmem_cp_scales(lead, sfa, sdesc_scales(f0));
        tmem_cp_scales(lead, sfb, sdesc_scales(f0 + 512));
        tmem_cp_scales(lead, sfb + 4, sdesc_scales(f0 + 1024));
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_mxf8_ss(lead, d, sdesc_sw128(a0 + kk * 32), sdesc_sw128(b0 + kk * 32), idesc, sfa, sfb,
                      (i > 0 || kk > 0) ? 1u : 0u);
        mma_commit_lead(lead, &empty[r.s]);
        r.next(S);
      }
      if (ok) mma_commit_lead(lead, &tfull[n & 1]);
    }
    mma_commit_lead(lead, mdone);
    mbar_wait_long(mdone, 0u, nullptr, err, ERR_GEMM_TFULL);
  } else if (warp < 4) {
    // four blocks' bytes in use, the next four's in flight
    constexpr int AHEAD = 4, W = 6;
    const bool is_a = warp == 2;
    const uint8_t* src = is_a ? p.ws : p.xs;
    const int limit = is_a ? p.M : p.N, words = is_a ? 4 : W;
    uint32_t nx[AHEAD][W];
    RingPos r{0, 0u};
    int done = 0;
    bool ok = true;
    for (int t = (int)blockIdx.x; t < total && ok; t += (int)gridDim.x) {
      const int row0 = is_a ? t / p.n_tiles * 128 : t % p.n_tiles * BN;
      auto fetch = [&](int i0) {
#pragma unroll
        for (int e = 0; e < AHEAD; ++e)
#pragma unroll
          for (int j = 0; j < W; ++j) {
            const int row = row0 + lane + 32 * j;
            nx[e][j] = i0 + e < p.kb && j < words && row < limit ? src[(long long)(i0 + e) * limit + row] : 127u;
          }
      };
      fetch(0);
      for (int i0 = 0; i0 < p.kb && ok; i0 += AHEAD) {
        uint32_t cur[AHEAD][W];
#pragma unroll
        for (int e = 0; e < AHEAD; ++e)
#pragma unroll
          for (int j = 0; j < W; ++j) {
            due(nx[e][j]);
            cur[e][j] = nx[e][j];
          }
        fetch(i0 + AHEAD);
#pragma unroll
        for (int e = 0; e < AHEAD; ++e) {
          if (i0 + e >= p.kb || !ok) break;
          if (done >= S && !(ok = wait(&empty[r.s], r.par ^ 1u, ERR_GEMM_EMPTY))) break;
          constexpr uint32_t rep = 0x01010101u;
          uint4* f = reinterpret_cast<uint4*>(sF + r.s * C::SF_BYTES + (is_a ? 0 : 512)) + lane;
          f[0] = make_uint4(cur[e][0] * rep, cur[e][1] * rep, cur[e][2] * rep, cur[e][3] * rep);
          if (!is_a) f[32] = make_uint4(cur[e][4] * rep, cur[e][5] * rep, 127u * rep, 127u * rep);
          fence_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&full[r.s]);
          r.next(S);
          ++done;
        }
      }
    }
  } else {
    // epilogue: thread = weight row, columns = activation rows
    const int q = warp & 3, l128 = q * 32 + lane;
    int n = 0;
    for (int t = (int)blockIdx.x; t < total; t += (int)gridDim.x, ++n) {
      const int m = t / p.n_tiles * 128 + l128, n0 = t % p.n_tiles * BN;
      const int cols = min(BN, p.N - n0);
      if (!wait(&tfull[n & 1], (uint32_t)(n >> 1) & 1u, ERR_GEMM_TFULL)) break;
      tc_fence_after();
      const uint32_t d = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)((n & 1) * BN);
#pragma unroll 1
      for (int c = 0; c < cols; c += 32) {
        float v[32];
        tmem_ld32(d + (uint32_t)c, v);
        if (m < p.M) {
          long long o = (long long)(n0 + c) * p.M + m;
          if (p.out_bf16) {
            __nv_bfloat16* y = static_cast<__nv_bfloat16*>(p.y);
#pragma unroll
            for (int j = 0; j < 32; ++j, o += p.M)
              if (c + j < cols) y[o] = __float2bfloat16_rn(v[j]);
          } else {
            float* y = static_cast<float*>(p.y);
#pragma unroll
            for (int j = 0; j < 32; ++j, o += p.M)
              if (c + j < cols) y[o] = v[j];
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&tempty[n & 1]);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

cudaError_t gemm8_err_word(int** p) { return cudaGetSymbolAddress(reinterpret_cast<void**>(p), g_gemm8_err); }

namespace {

template <typename E>
cudaError_t launch_quantise8(const Quantise8Params& p, bool vec, cudaStream_t st) {
  const dim3 grid((p.groups + 16 * kQAhead - 1) / (16 * kQAhead));
  return vec ? op_launch(quantise8_kernel<E, true>, grid, dim3(256), 0, st, 1, p)
             : op_launch(quantise8_kernel<E, false>, grid, dim3(256), 0, st, 1, p);
}

template <int BN>
cudaError_t launch_gemm8(const CUtensorMap& tw, const CUtensorMap& tx, const Gemm8Params& p, unsigned grid,
                         cudaStream_t st) {
  using C = Gemm8Cfg<BN>;
  const cudaError_t e = op_smem_once(reinterpret_cast<const void*>(gemm8_kernel<BN>), C::SMEM_BYTES);
  if (e != cudaSuccess) return e;
  return op_launch(gemm8_kernel<BN>, dim3(grid), dim3(224), C::SMEM_BYTES, st, 1 << p.split_log, tw, tx, p);
}

cudaError_t launch_gemm8_big(const CUtensorMap& tw, const CUtensorMap& tx, const Gemm8Params& p, unsigned grid,
                             cudaStream_t st) {
  const cudaError_t e = op_smem_once(reinterpret_cast<const void*>(gemm8_big_kernel), Gemm8BigCfg::SMEM_BYTES);
  if (e != cudaSuccess) return e;
  return op_launch(gemm8_big_kernel, dim3(grid), dim3(256), Gemm8BigCfg::SMEM_BYTES, st, 1, tw, tx, p);
}

}  // namespace
}  // namespace dllm

using namespace dllm;

extern "C" dllm_status dllm_op_quantise8(const void* x, int64_t row_stride, int32_t dtype, int32_t rows, int32_t K,
                                         uint8_t* codes, uint8_t* scales, void* stream) {
  const int es = op_dtype_size(dtype);
  if (!x || !codes || !scales || rows < 1 || K < 16 || K % 16 || es == 0 || !op_aligned(x, es) || !op_aligned(codes, 16))
    return op_fail(DLLM_EINVAL, "bad quantise8 arguments: rows=%d K=%d (K %% 16 == 0) dtype=%d, codes 16-byte aligned",
                   rows, K, dtype);
  const long long rs = row_stride ? row_stride : K;
  if (rs < K || rs > (1LL << 40)) return op_fail(DLLM_EINVAL, "quantise8: row stride %lld (0, or at least K=%d)", rs, K);
  const long long kb = ((long long)K + kQBlock - 1) / kQBlock;
  if (rows * kb > 0x7fffff00LL) return op_fail(DLLM_EINVAL, "quantise8: rows=%d K=%d are too many blocks", rows, K);
  const bool vec = op_aligned(x, 16) && (rs * es) % 16 == 0;
  Quantise8Params p = {};
  p.x = x;
  p.codes = codes;
  p.scales = scales;
  p.rs = rs;
  p.rows = rows;
  p.K = K;
  p.groups = (uint32_t)(rows * kb);
  p.blocks = FastDiv((uint32_t)kb);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  switch (dtype) {
    case DLLM_F32: OP_CK(launch_quantise8<ElemF32>(p, vec, st)); break;
    case DLLM_BF16: OP_CK(launch_quantise8<ElemBf16>(p, vec, st)); break;
    default: OP_CK(launch_quantise8<ElemF16>(p, vec, st)); break;
  }
  return DLLM_OK;
}

extern "C" dllm_status dllm_op_gemm8(const uint8_t* W, const uint8_t* W_scale, const uint8_t* X,
                                     const uint8_t* X_scale, void* Y, int32_t y_dtype, int32_t M, int32_t N, int32_t K,
                                     void* stream) {
  if (!W || !W_scale || !X || !X_scale || !Y || (y_dtype != DLLM_F32 && y_dtype != DLLM_BF16) || M < 1 || N < 1 ||
      M > kMostRows || N > kMostRows || K < 16 || K % 16 || !op_aligned(W, 16) || !op_aligned(X, 16) ||
      !op_aligned(Y, 16))
    return op_fail(DLLM_EINVAL,
                   "bad gemm8 arguments: M=%d N=%d K=%d (K %% 16 == 0) y_dtype=%d (float32 or bf16), W, X and Y "
                   "16-byte aligned",
                   M, N, K, y_dtype);
  Gemm8Params p = {};
  p.ws = W_scale;
  p.xs = X_scale;
  p.y = Y;
  p.M = M;
  p.N = N;
  p.K = K;
  p.kb = (int)(((long long)K + kQBlock - 1) / kQBlock);
  p.out_bf16 = y_dtype == DLLM_BF16;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  CUtensorMap tw, tx;
  if (const dllm_status s = op_map_u8(&tw, W, K, M, 1, K, (uint64_t)K * M, 128, 128); s != DLLM_OK) return s;
  const int bn = N <= 32 ? 32 : N <= 64 ? 64 : 128;
  p.n_tiles = (N + bn - 1) / bn;
  const long long tiles = (long long)((M + 127LL) / 128) * p.n_tiles, slots = 2LL * op_device_sms();
  // Split a tile's K over a cluster while all CTAs fit on the GPU at once, two
  // an SM: bound by HBM they then share its bandwidth evenly and finish
  // together.  Each keeps at least two blocks of K.
  while (p.split_log < 3 && (tiles << p.split_log) * 2 <= slots && p.kb >= 4 << p.split_log) ++p.split_log;
  if (N > 64) {
    // Or tiles of 128 x 192 by persistent CTAs.  A block of K takes a round of those 0.36 us and a
    // round of the two CTAs an SM 0.52 us, the join of a split about 15 blocks (measured, us, with
    // the quantiser, persistent / two CTAs: 4096 x 4096 weights, 128 rows 15.0 / 14.4, 400 rows 16.7 / 22.5, 768 rows
    // 18.9 / 21.1, 1024 rows 28.6 / 21.7; 12288 x 4096, 160 rows 17.1 / 20.0, 256 rows 26.9 / 21.7, 512 rows 27.9 / 35.4,
    // 2048 rows 82 / 99; 4096 x 12288, 100 rows 34 / 19, 2048 rows 107 / 99; 688 x 256, 300 rows 6.5 / 5.8).
    const long long sms = op_device_sms(), big = (M + 127LL) / 128 * ((N + Gemm8BigCfg::BN - 1LL) / Gemm8BigCfg::BN);
    const __int128 big_cost = 9 * ((__int128)((big + sms - 1) / sms) * p.kb + 1);
    const __int128 cta_cost = (__int128)13 * (((tiles << p.split_log) + slots - 1) / slots) *
                              (((p.kb + (1 << p.split_log) - 1) >> p.split_log) + (p.split_log ? 15 : 0));
    if (big_cost <= cta_cost && big <= 0x3fffffffLL) {
      p.n_tiles = (N + Gemm8BigCfg::BN - 1) / Gemm8BigCfg::BN;
      if (const dllm_status s = op_map_u8(&tx, X, K, N, 1, K, (uint64_t)K * N, 128, Gemm8BigCfg::BN); s != DLLM_OK)
        return s;
      OP_CK(launch_gemm8_big(tw, tx, p, (unsigned)std::min(sms, big), st));
      return DLLM_OK;
    }
  }
  if ((tiles << p.split_log) > 0x7fffffffLL) return op_fail(DLLM_EINVAL, "gemm8: M=%d N=%d are too large", M, N);
  if (const dllm_status s = op_map_u8(&tx, X, K, N, 1, K, (uint64_t)K * N, 128, bn); s != DLLM_OK) return s;
  const unsigned grid = (unsigned)(tiles << p.split_log);
  switch (bn) {
    case 32: OP_CK(launch_gemm8<32>(tw, tx, p, grid, st)); break;
    case 64: OP_CK(launch_gemm8<64>(tw, tx, p, grid, st)); break;
    default: OP_CK(launch_gemm8<128>(tw, tx, p, grid, st)); break;
  }
  return DLLM_OK;
}
