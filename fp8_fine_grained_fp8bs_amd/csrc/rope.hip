// rope.hip -- rotary positions: the table of angles and the rotation of
// heads, forward and backward (gfx950).
//
// A pair (x1, x2) of a head turns by the angle of its position:
//   y1 = x1 cos a - x2 sin a,  y2 = x2 cos a + x1 sin a,
// an orthogonal map, so its gradient is the turn by -a.  The kernel moves 4
// bytes a value (BF16 in and out) for 3 operations: HBM-bound.  The angles
// come from a table made once (they need binary64: at position 10^5 a
// binary32 angle is already off by 2^-8); a row of it serves all heads of a
// token, so the rows' reads stay in the caches.
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

// One thread a unit of 16 values: a rotated unit (two vectors of 8), or two
// vectors of the head's other dims to copy.
__global__ __launch_bounds__(256) void rope_kernel(const uint16_t* __restrict__ x, int64_t ldx,
                                                   uint16_t* __restrict__ y, int64_t ldy,
                                                   const int32_t* __restrict__ pos, int64_t T, int H, int D,
                                                   RopeShape r, float sign, const float* __restrict__ cs,
                                                   int64_t n_pos, int units) {
  const int per = H * units;
  const int64_t e = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int64_t t = e / per;
  if (t >= T) return;
  const int rest = static_cast<int>(e - t * per);
  const int h = rest / units, c = rest - h * units;
  const uint16_t* xh = x + t * ldx + h * D;
  uint16_t* yh = y + t * ldy + h * D;
  if (8 * c * 2 >= r.rot) {   // copied dims: vectors 2k, 2k+1 of those around the rotated part
    const int k = 2 * (c - r.rot / 16);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      int d = 8 * (k + i);
      if (d >= r.off) d += r.rot;
      *reinterpret_cast<uint4*>(yh + d) = *reinterpret_cast<const uint4*>(xh + d);
    }
    return;
  }
  const int ia = rope_first(r, c), ib = rope_second(r, c);
  const uint4 va = *reinterpret_cast<const uint4*>(xh + ia);
  const uint4 vb = *reinterpret_cast<const uint4*>(xh + ib);
  int64_t p = pos[t];
  p = p < 0 ? 0 : p >= n_pos ? n_pos - 1 : p;
  CosSin k = load_cossin(cs + p * r.rot, r.rot, c);
#pragma unroll
  for (int i = 0; i < 8; ++i) k.s[i] *= sign;
  float a[8], b[8];
  unpack8(va, a);
  unpack8(vb, b);
  rotate8(a, b, k, r.interleaved);
  *reinterpret_cast<uint4*>(yh + ia) = pack8(a);
  *reinterpret_cast<uint4*>(yh + ib) = pack8(b);
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
  const int64_t blocks = (T * H * units + 255) / 256;
  if (blocks > 0x7fffffff) return hipErrorInvalidValue;
  const RopeShape r{rot, rot_off, interleaved};
  hipLaunchKernelGGL(rope_kernel, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, st, x, ldx, y, ldy, pos, T, H,
                     D, r, inverse ? -1.0f : 1.0f, cs, n_pos, units);
  return hipGetLastError();
}

}  // namespace fp8bs
