// rope_device.h -- the rotation of a row's heads, shared by the rotary and cache
// kernels (gfx950).
#pragma once

#include "packed_search.h"

namespace fp8bs {

// The rotated dims of a head: off .. off + rot - 1, in pairs (i, i + rot/2) or,
// interleaved, (2i, 2i + 1).
struct RopeShape {
  int rot;
  int off;
  bool interleaved;
};

struct CosSin {
  float c[8], s[8];
};
// Angles 4j .. 4j + 3 of a table row [cos.. | sin..] into places 4i .. 4i + 3.
__device__ __forceinline__ void load_angles4(CosSin& k, int i, const float* row, int rot, int j) {
  const float4 a = *reinterpret_cast<const float4*>(row + 4 * j);
  const float4 b = *reinterpret_cast<const float4*>(row + (rot >> 1) + 4 * j);
  k.c[4 * i] = a.x; k.c[4 * i + 1] = a.y; k.c[4 * i + 2] = a.z; k.c[4 * i + 3] = a.w;
  k.s[4 * i] = b.x; k.s[4 * i + 1] = b.y; k.s[4 * i + 2] = b.z; k.s[4 * i + 3] = b.w;
}

__device__ __forceinline__ void unpack8(const uint4& w, float v[8]) {
  v[0] = bf16_lo(w.x); v[1] = bf16_hi(w.x);
  v[2] = bf16_lo(w.y); v[3] = bf16_hi(w.y);
  v[4] = bf16_lo(w.z); v[5] = bf16_hi(w.z);
  v[6] = bf16_lo(w.w); v[7] = bf16_hi(w.w);
}
__device__ __forceinline__ uint4 pack8(const float v[8]) {
  return make_uint4(pack_bf16x2_rne(v[0], v[1]), pack_bf16x2_rne(v[2], v[3]), pack_bf16x2_rne(v[4], v[5]),
                    pack_bf16x2_rne(v[6], v[7]));
}

// Rotation of vectors in place.  Every product and sum is rounded by itself
// (the library is built without contraction).
__device__ __forceinline__ void rotate_halves(float a[8], float b[8], const CosSin& k) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float x1 = a[i], x2 = b[i];
    a[i] = x1 * k.c[i] - x2 * k.s[i];
    b[i] = x2 * k.c[i] + x1 * k.s[i];
  }
}
__device__ __forceinline__ void rotate_pairs(float a[8], const CosSin& k, int at) {   // angles at .. at + 3
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float x1 = a[2 * i], x2 = a[2 * i + 1];
    a[2 * i] = x1 * k.c[at + i] - x2 * k.s[at + i];
    a[2 * i + 1] = x2 * k.c[at + i] + x1 * k.s[at + i];
  }
}

// A lane's unit of a head: two vectors of 8 dims at ia and ib.  half: the first
// rot / 16 units are the vectors that pair up, rot / 2 apart, the others two
// of the dims around them; interleaved: vectors c and c + units, each with its
// own pairs.  Either way the lanes' vectors lie side by side.  `inside`: only the
// rotated dims are gone through (in place).
struct RopeUnit {
  int ia, ib;
  bool ra, rb;   // rotated
  CosSin k;
};
__device__ __forceinline__ RopeUnit rope_unit(const RopeShape& r, int c, int units, bool inside, float sign, const float* row) {
  RopeUnit u;
  if (r.interleaved) {
    u.ia = 8 * c + (inside ? r.off : 0);
    u.ib = u.ia + 8 * units;
    u.ra = u.ia >= r.off && u.ia < r.off + r.rot;
    u.rb = u.ib >= r.off && u.ib < r.off + r.rot;
    if (u.ra) load_angles4(u.k, 0, row, r.rot, (u.ia - r.off) >> 3);
    if (u.rb) load_angles4(u.k, 1, row, r.rot, (u.ib - r.off) >> 3);
  } else if (16 * c < r.rot) {
    u.ia = r.off + 8 * c;
    u.ib = u.ia + (r.rot >> 1);
    u.ra = u.rb = true;
    load_angles4(u.k, 0, row, r.rot, 2 * c);
    load_angles4(u.k, 1, row, r.rot, 2 * c + 1);
  } else {
    const int n = units - r.rot / 16, j = c - r.rot / 16;   // of the vectors around the rotated part: j and j + n
    u.ia = 8 * j;
    u.ib = 8 * (j + n);
    u.ia += u.ia >= r.off ? r.rot : 0;
    u.ib += u.ib >= r.off ? r.rot : 0;
    u.ra = u.rb = false;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) u.k.s[i] *= sign;
  return u;
}

// One row's H heads of D values from x to y (may be the same), by one wave:
// lanes over units of 16 values.  Where the units of a head divide the wave
// (UNITS, or 0) a lane keeps its unit, and its angles, from head to head.
template <int UNITS>
__device__ __forceinline__ void rotate_row(const uint16_t* x, uint16_t* y, int H, int D, const RopeShape& r, float sign,
                                           const float* row, bool inside, int units_any = 0) {
  const int lane = static_cast<int>(threadIdx.x) & 63, units = UNITS ? UNITS : units_any;
  RopeUnit u;
  if (UNITS) u = rope_unit(r, lane % units, units, inside, sign, row);
#pragma unroll 4
  for (int e = lane; e < H * units; e += 64) {
    const int h = e / units;
    if (!UNITS) u = rope_unit(r, e - h * units, units, inside, sign, row);
    uint4 va = load16_nt(x + h * D + u.ia), vb = load16_nt(x + h * D + u.ib);
    float a[8], b[8];
    if (r.interleaved) {
      if (u.ra) {
        unpack8(va, a);
        rotate_pairs(a, u.k, 0);
        va = pack8(a);
      }
      if (u.rb) {
        unpack8(vb, b);
        rotate_pairs(b, u.k, 4);
        vb = pack8(b);
      }
    } else if (u.ra) {
      unpack8(va, a);
      unpack8(vb, b);
      rotate_halves(a, b, u.k);
      va = pack8(a);
      vb = pack8(b);
    }
    *reinterpret_cast<uint4*>(y + h * D + u.ia) = va;
    *reinterpret_cast<uint4*>(y + h * D + u.ib) = vb;
  }
}

}  // namespace fp8bs
