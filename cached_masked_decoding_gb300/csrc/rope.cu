// Rotary positions: the pairs (x0, x1) of a head turn by the angle pos * f_i,
//   x0' = x0 cos - x1 sin,  x1' = x1 cos + x0 sin,
// f_i = theta^(-2i/rot) and its long-context scalings (see dllm_rope).
//
// The angle of a far position has to be reduced by whole turns before it is
// rounded to 32 bits (position 10^6 in float32 leaves 2^-4 of a radian).  Turns
// are taken in 64-bit fixed point: the host gives each pair's turns per
// position as a fraction of 2^64, and the integer product with the position
// wraps by whole turns exactly - three integer multiplies instead of 64-bit
// floating point, whose rate is a 64th of 32-bit on this chip.
//
// Bound by HBM: one read and one write of x.  A thread owns 8 pairs of a row
// (two 16-byte vectors of 16-bit elements) and walks up to 8 heads with the
// same cosines, four heads' loads in flight.  8191 rows of 40 heads of 128, bf16, half
// of them turned: 28.7 us, 5.8 TB/s; 32 rows of 64 heads: 2.6 us, a launch's latency.
#include <algorithm>
#include <cmath>

#include "ops8.h"
#include "ptx8.cuh"
#include "q8.cuh"

namespace dllm {

constexpr int kMaxPairs = 128;

struct RopeParams {
  const void* x;
  void* out;
  const int32_t* pos;
  long long x_rs, x_hs, o_rs, o_hs;
  uint32_t items;
  FastDiv units, runs;
  int heads, rot, interleaved, head_run;
  float amp;
  uint64_t turns[kMaxPairs];   // turns per position * 2^64
};

__device__ __forceinline__ void turn_cos_sin(uint64_t turns, int pos, float amp, float& c, float& s) {
  const uint64_t t = turns * (uint64_t)(int64_t)pos;          // fraction of a turn, exact modulo 1
  const uint32_t quarter = (uint32_t)((t + (1ull << 61)) >> 62);
  const int64_t r = (int64_t)(t - ((uint64_t)quarter << 62));  // within an eighth of a turn of the quarter
  float cr, sr;
  sincospif((float)r * 0x1p-63f, &sr, &cr);
  c = (quarter & 1) ? sr : cr;
  s = (quarter & 1) ? cr : sr;
  if (quarter == 1 || quarter == 2) c = -c;
  if (quarter >= 2) s = -s;
  c *= amp;
  s *= amp;
}

// VEC: 8 pairs (16 elements) a thread in 16-byte accesses; else one pair.
template <typename E, bool VEC>
__global__ void __launch_bounds__(256) rope_kernel(const __grid_constant__ RopeParams p) {
  using T = typename E::T;
  constexpr int PAIRS = VEC ? 8 : 1;
  constexpr int AHEAD = 4;                     // heads in flight
  griddep_launch_dependents();
  griddep_wait();
  const uint32_t item = blockIdx.x * 256u + threadIdx.x;
  if (item >= p.items) return;
  uint32_t u, run;
  const uint32_t row = p.runs.divmod(p.units.divmod(item, u), run);
  const int h0 = (int)run * p.head_run, h1 = min(p.heads, h0 + p.head_run);
  const T* x = static_cast<const T*>(p.x) + row * p.x_rs;
  T* out = static_cast<T*>(p.out) + row * p.o_rs;
  const int first = (int)u * PAIRS;            // pairs below rot / 2 turn, the rest is copied
  const bool turns = first < p.rot / 2;
  if (!turns && p.x == p.out) return;
  // elements a and b of the unit's first pair
  const int a = !turns || p.interleaved ? 2 * first : first;
  const int b = !turns || p.interleaved ? a + PAIRS : first + p.rot / 2;
  float c[PAIRS], s[PAIRS];
#pragma unroll
  for (int i = 0; i < PAIRS; ++i) {
    c[i] = 1.0f;
    s[i] = 0.0f;
  }
  if (turns) {
    const int pos = p.pos[row];
#pragma unroll
    for (int i = 0; i < PAIRS; ++i) turn_cos_sin(p.turns[first + i], pos, p.amp, c[i], s[i]);
  }
  for (int hb = h0; hb < h1; hb += AHEAD) {
    if constexpr (VEC) {
      constexpr int W = (int)sizeof(T) / 2;    // 16-byte words of 8 elements
      uint4 raw[AHEAD][2][W];
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) {
        if (hb + k >= h1) break;
        const T* xh = x + (hb + k) * p.x_hs;
#pragma unroll
        for (int w = 0; w < W; ++w) {
          raw[k][0][w] = reinterpret_cast<const uint4*>(xh + a)[w];
          raw[k][1][w] = reinterpret_cast<const uint4*>(xh + b)[w];
        }
      }
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) {
        if (hb + k >= h1) break;
        T* oh = out + (hb + k) * p.o_hs;
        if (turns) {
          float v[2][8], r[2][8];
          E::load8(reinterpret_cast<const T*>(raw[k][0]), v[0]);
          E::load8(reinterpret_cast<const T*>(raw[k][1]), v[1]);
          if (p.interleaved) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float x0 = v[i >> 2][2 * (i & 3)], x1 = v[i >> 2][2 * (i & 3) + 1];
              r[i >> 2][2 * (i & 3)] = x0 * c[i] - x1 * s[i];
              r[i >> 2][2 * (i & 3) + 1] = x1 * c[i] + x0 * s[i];
            }
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              r[0][i] = v[0][i] * c[i] - v[1][i] * s[i];
              r[1][i] = v[1][i] * c[i] + v[0][i] * s[i];
            }
          }
          E::store8(reinterpret_cast<T*>(raw[k][0]), r[0]);
          E::store8(reinterpret_cast<T*>(raw[k][1]), r[1]);
        }
#pragma unroll
        for (int w = 0; w < W; ++w) {
          reinterpret_cast<uint4*>(oh + a)[w] = raw[k][0][w];
          reinterpret_cast<uint4*>(oh + b)[w] = raw[k][1][w];
        }
      }
    } else {
      for (int h = hb; h < min(h1, hb + AHEAD); ++h) {
        const T x0 = x[h * p.x_hs + a], x1 = x[h * p.x_hs + b];
        T r0 = x0, r1 = x1;                    // the copied part keeps its bits
        if (turns) {
          const float f0 = E::get(&x0), f1 = E::get(&x1);
          E::put(&r0, f0 * c[0] - f1 * s[0]);
          E::put(&r1, f1 * c[0] + f0 * s[0]);
        }
        out[h * p.o_hs + a] = r0;
        out[h * p.o_hs + b] = r1;
      }
    }
  }
}

namespace {

// Rows and heads of a strided [rows][heads][hd] array do not overlap: heads
// within a row, or rows within a head.
bool strides_ok(long long rows, long long heads, long long hd, long long rs, long long hs) {
  return (hs >= hd && rs >= (heads - 1) * hs + hd) || (rs >= hd && hs >= (rows - 1) * rs + hd);
}

template <typename E>
cudaError_t launch_rope(const RopeParams& p, bool vec, cudaStream_t st) {
  const dim3 grid((p.items + 255) / 256);
  return vec ? op_launch(rope_kernel<E, true>, grid, dim3(256), 0, st, 1, p)
             : op_launch(rope_kernel<E, false>, grid, dim3(256), 0, st, 1, p);
}

}  // namespace
}  // namespace dllm

using namespace dllm;

extern "C" dllm_status dllm_op_rope(const void* x, void* out, const int32_t* positions, int32_t rows, int32_t heads,
                                    int32_t hd, int64_t x_row_stride, int64_t x_head_stride, int64_t out_row_stride,
                                    int64_t out_head_stride, int32_t dtype, const dllm_rope* r, void* stream) {
  const int es = op_dtype_size(dtype);
  if (!x || !out || !positions || !r || rows < 1 || heads < 1 || hd < 2 || hd > 1024 || hd % 2 || es == 0)
    return op_fail(DLLM_EINVAL, "bad rope arguments: rows=%d heads=%d hd=%d (even, 2..1024) dtype=%d", rows, heads, hd,
                   dtype);
  if (!op_aligned(x, es) || !op_aligned(out, es) || !op_aligned(positions, 4))
    return op_fail(DLLM_EINVAL, "rope: x, out and positions must be aligned to their elements");
  if (r->rot_dim < 2 || r->rot_dim % 2 || r->rot_dim > hd || r->rot_dim > 2 * kMaxPairs || r->layout < 0 ||
      r->layout > 1 || r->scaling < 0 || r->scaling > 3 || !(r->theta >= 1.0) || !std::isfinite(r->theta) ||
      !std::isfinite(r->amplitude) || r->amplitude < 0.0)
    return op_fail(DLLM_EINVAL,
                   "bad rope: rot_dim=%d (even, 2..min(hd, 256)) layout=%d scaling=%d theta=%g (>= 1) amplitude=%g",
                   r->rot_dim, r->layout, r->scaling, r->theta, r->amplitude);
  if (r->scaling != DLLM_ROPE_UNSCALED && (!(r->factor >= 1.0) || !std::isfinite(r->factor)))
    return op_fail(DLLM_EINVAL, "bad rope factor %g (>= 1)", r->factor);
  if (r->scaling == DLLM_ROPE_BASE && r->rot_dim < 4)
    return op_fail(DLLM_EINVAL, "rope base scaling needs rot_dim >= 4, got %d", r->rot_dim);
  if (r->scaling == DLLM_ROPE_BY_PARTS &&
      (!(r->orig_len >= 1.0) || !std::isfinite(r->orig_len) || !(r->beta_slow > 0.0) ||
       !(r->beta_fast >= r->beta_slow) || !std::isfinite(r->beta_fast) || !(r->theta > 1.0)))
    return op_fail(DLLM_EINVAL, "bad rope by parts: orig_len=%g beta_fast=%g beta_slow=%g theta=%g", r->orig_len,
                   r->beta_fast, r->beta_slow, r->theta);
  const int64_t most = int64_t(1) << 31;   // rows, heads and strides of 31 bits: offsets stay in 64
  if (x_row_stride < 0 || x_row_stride > most || x_head_stride < 0 || x_head_stride > most || out_row_stride < 0 ||
      out_row_stride > most || out_head_stride < 0 || out_head_stride > most)
    return op_fail(DLLM_EINVAL, "rope strides out of range: x row %lld head %lld, out row %lld head %lld",
                   (long long)x_row_stride, (long long)x_head_stride, (long long)out_row_stride,
                   (long long)out_head_stride);
  RopeParams p = {};
  p.x = x;
  p.out = out;
  p.pos = positions;
  p.heads = heads;
  p.rot = r->rot_dim;
  p.interleaved = r->layout == DLLM_ROPE_INTERLEAVED;
  p.x_hs = x_head_stride ? x_head_stride : hd;
  p.x_rs = x_row_stride ? x_row_stride : (long long)heads * p.x_hs;
  p.o_hs = out_head_stride ? out_head_stride : hd;
  p.o_rs = out_row_stride ? out_row_stride : (long long)heads * p.o_hs;
  if (!strides_ok(rows, heads, hd, p.x_rs, p.x_hs) || !strides_ok(rows, heads, hd, p.o_rs, p.o_hs))
    return op_fail(DLLM_EINVAL, "rope strides overlap: x row %lld head %lld, out row %lld head %lld", p.x_rs, p.x_hs,
                   p.o_rs, p.o_hs);
  if (x == out && (p.x_rs != p.o_rs || p.x_hs != p.o_hs))
    return op_fail(DLLM_EINVAL, "rope in place needs the same strides on both sides");

  // turning rates in 64 bits
  const int pairs = p.rot / 2;
  double theta = r->theta, amp = 1.0, lo = 0.0, hi = 0.0;
  if (r->scaling == DLLM_ROPE_BASE) theta *= std::pow(r->factor, p.rot / (p.rot - 2.0));
  if (r->scaling == DLLM_ROPE_BY_PARTS) {
    const double k = p.rot / (2.0 * std::log(theta)), turn = 2.0 * 3.14159265358979323846;
    // (the ramp may end past the last pair, for long original contexts)
    lo = std::fmax(0.0, std::floor(k * std::log(r->orig_len / (r->beta_fast * turn))));
    hi = std::fmin(p.rot - 1.0, std::ceil(k * std::log(r->orig_len / (r->beta_slow * turn))));
    amp = 0.1 * std::log(r->factor) + 1.0;
  }
  p.amp = (float)(r->amplitude > 0.0 ? r->amplitude : amp);
  // theta^(-2i/rot) as the product of a power for i's upper and one for its lower
  // three bits: 24 powers at most in place of 128 on the calling thread
  double lower[8], upper = 1.0;
  for (int i = 0; i < std::min(pairs, 8); ++i) lower[i] = std::pow(theta, -2.0 * i / p.rot);
  for (int i = 0; i < pairs; ++i) {
    if (i % 8 == 0) upper = std::pow(theta, -2.0 * i / p.rot);
    double f = upper * lower[i % 8];
    if (r->scaling == DLLM_ROPE_LINEAR) f /= r->factor;
    if (r->scaling == DLLM_ROPE_BY_PARTS) {
      const double ramp = std::fmin(1.0, std::fmax(0.0, (i - lo) / std::fmax(hi - lo, 0.001)));
      f = f / r->factor * ramp + f * (1.0 - ramp);
    }
    // f <= 1 (a rounding above it at most), so the turns per position stay under 0.16: 2^64 of them fit
    p.turns[i] = (uint64_t)(f * 0.15915494309189533577 * 0x1p64);
  }

  // 16-byte accesses: units of 8 pairs that do not straddle the turned part,
  // and vectors that start on 16 bytes in every row and head
  const int v16 = 16 / es;
  const bool vec = hd % 16 == 0 && p.rot % 16 == 0 && op_aligned(x, 16) && op_aligned(out, 16) && p.x_rs % v16 == 0 &&
                   p.x_hs % v16 == 0 && p.o_rs % v16 == 0 && p.o_hs % v16 == 0;
  // Heads a thread walks: as many, up to 8, as leave half the GPU's threads an
  // item (8191 rows of 40 heads: 8 heads 29 us, 1 head 68 us; 32 rows of 64 heads
  // take 1).
  const long long units = hd / (vec ? 16 : 2);
  p.head_run = 8;
  while (p.head_run > 1 && (long long)rows * units * ((heads + p.head_run - 1) / p.head_run) < 1024LL * op_device_sms())
    p.head_run /= 2;
  const long long runs = (heads + p.head_run - 1) / p.head_run;
  const __int128 items = (__int128)rows * units * runs;
  if (items > 0x7fffff00) return op_fail(DLLM_EINVAL, "rope: %d rows of %d heads are too many for one call", rows, heads);
  p.items = (uint32_t)items;
  p.units = FastDiv((uint32_t)units);
  p.runs = FastDiv((uint32_t)runs);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  switch (dtype) {
    case DLLM_F32: OP_CK(launch_rope<ElemF32>(p, vec, st)); break;
    case DLLM_BF16: OP_CK(launch_rope<ElemBf16>(p, vec, st)); break;
    default: OP_CK(launch_rope<ElemF16>(p, vec, st)); break;
  }
  return DLLM_OK;
}
