// rope.hip -- rotary positions: the table of angles and the rotation of
// heads, forward and backward (gfx950).
//
// A pair (x1, x2) of a head turns by the angle of its position:
//   y1 = x1 cos a - x2 sin a,  y2 = x2 cos a + x1 sin a,
// an orthogonal map, so its gradient is the turn by -a.  The kernel moves 4
// bytes a value (BF16 in and out) for 3 operations: HBM-bound.  The angles
// come from a table made once (they need binary64: at position 10^5 a
// binary32 angle is already off by 2^-8); a row of it serves all heads of a
// token, so the rows' reads stay in the caches.  Measured: the gradient of 16383
// tokens, 40 heads of 128 of which 64 dims turn, 340 MB: 51 us in the kernel, 6.7
// TB/s, 57 a call (65 with plain loads, 61 with non-temporal stores too); 3 tokens
// 2.5 us, a launch.  The table, made once by a program: 131072 positions of 128, 67 MB, 74.5
// us (by parts 80), 0.9 TB/s, bound by `pow` and `sincos` in doubles for every angle.
#include <hip/hip_runtime.h>

#include "fp8bs_internal.h"
#include "rope_device.h"

namespace fp8bs {
namespace {

__global__ __launch_bounds__(256) void rope_table_kernel(float* __restrict__ cs, int64_t n_pos, int half,
                                                         double base, double factor, double orig_len,
                                                         double turns_lo, double turns_hi, double mscale) {
  const int64_t e = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (e >= n_pos * half) return;
  const int64_t p = e / half;
  const int i = static_cast<int>(e - p * half);
  double f = pow(base, -static_cast<double>(i) / half);
  if (orig_len > 0.0) {
    const double turns = orig_len * f * 0.15915494309189535;   // 1 / (2 pi)
    const double w = fmin(fmax((turns - turns_lo) / (turns_hi - turns_lo), 0.0), 1.0);
    f = (1.0 - w) * (f / factor) + w * f;
  } else {
    f = f / factor;
  }
  double s, c;
  sincos(static_cast<double>(p) * f, &s, &c);
  cs[p * 2 * half + i] = static_cast<float>(c * mscale);
  cs[p * 2 * half + half + i] = static_cast<float>(s * mscale);
}

// A wave a token and strip of heads.
template <int UNITS>
__global__ __launch_bounds__(256) void rope_kernel(const uint16_t* x, int64_t ldx, uint16_t* y, int64_t ldy,
                                                   const int32_t* __restrict__ pos, int64_t T, int H, int D,
                                                   RopeShape r, float sign, const float* __restrict__ cs,
                                                   int64_t n_pos, int units, int strip, bool inside) {
  const int64_t e = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
  const int strips = (H + strip - 1) / strip;
  const int64_t t = e / strips;
  if (t >= T) return;
  const int h0 = static_cast<int>(e - t * strips) * strip, heads = H - h0 < strip ? H - h0 : strip;
  int64_t p = pos[t];
  p = p < 0 ? 0 : p >= n_pos ? n_pos - 1 : p;
  rotate_row<UNITS>(x + t * ldx + static_cast<int64_t>(h0) * D, y + t * ldy + static_cast<int64_t>(h0) * D, heads, D, r,
                    sign, cs + p * r.rot, inside, units);
}

}  // namespace

hipError_t launch_rope_table(float* cs, int64_t n_pos, int64_t rot, double base, double factor, double orig_len,
                             double turns_lo, double turns_hi, double mscale, hipStream_t st) {
  const int half = static_cast<int>(rot / 2);
  const int64_t blocks = (n_pos * half + 255) / 256;
  if (blocks > 0x7fffffff) return hipErrorInvalidValue;
  hipLaunchKernelGGL(rope_table_kernel, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, st, cs, n_pos, half,
                     base, factor, orig_len, turns_lo, turns_hi, mscale);
  return hipGetLastError();
}

hipError_t launch_rope(const uint16_t* x, int64_t ldx, uint16_t* y, int64_t ldy, const int32_t* pos, int64_t T,
                       int H, int D, int rot, int rot_off, bool interleaved, bool inverse, const float* cs,
                       int64_t n_pos, hipStream_t st) {
  // in place the other dims stay where they are
  const int units = (x == y ? rot : D) / 16;
  // as many heads a wave as its lanes hold at once: more waves were faster than
  // angles kept over all heads of a token (50.5 us against 52.4 at 16383 x 40 heads of 128)
  const int strip = units >= 64 ? 1 : 64 / units;
  const int64_t waves = T * ((H + strip - 1) / strip), blocks = (waves + 3) / 4;
  if (blocks > 0x7fffffff) return hipErrorInvalidValue;
  const RopeShape r{rot, rot_off, interleaved};
  const dim3 grid(static_cast<unsigned>(blocks)), block(256);
#define FP8BS_ROPE(U) \
  hipLaunchKernelGGL((rope_kernel<U>), grid, block, 0, st, x, ldx, y, ldy, pos, T, H, D, r, inverse ? -1.0f : 1.0f, cs, \
                     n_pos, units, strip, x == y)
  if (units == 8) FP8BS_ROPE(8);
  else if (units == 4) FP8BS_ROPE(4);
  else FP8BS_ROPE(0);
#undef FP8BS_ROPE
  return hipGetLastError();
}

}  // namespace fp8bs
