// Rotary positions shared by dllm_op_rope and the head norms' kernel: a pair's turns as a fraction
// of 2^64 (host side), and the cosine and sine of position times that.
#pragma once

#include "ops8.h"

namespace dllm {

constexpr int kMaxPairs = 128;

// Checks *r for heads of hd elements and gives the turns per position * 2^64 of its rot_dim / 2
// pairs, and the amplitude.
dllm_status rope_turns(const dllm_rope* r, int hd, uint64_t* turns, float* amp);

#ifdef __CUDACC__
// turns * pos wraps by whole turns exactly; the rest of the angle is within an eighth of a turn
// of a quarter.
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
#endif

}  // namespace dllm
