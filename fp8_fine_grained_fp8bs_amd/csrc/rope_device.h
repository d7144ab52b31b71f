// rope_device.h -- the rotation of one pair of 8-value vectors, and the
// search for a packed row's sequence, shared by the rotary and cache kernels.
#pragma once

#include "fp8bs_device.h"

namespace fp8bs {

// Where the rotation reads and writes inside a head: unit c rotates eight
// pairs held in two 16-byte vectors.  half: the vectors are rot/2 apart and
// pair up element by element; interleaved: they are adjacent and hold the
// pairs next to each other.
struct RopeShape {
  int rot;
  int off;
  bool interleaved;
};
__device__ __forceinline__ int rope_first(const RopeShape& r, int c) {
  return r.off + (r.interleaved ? 16 * c : 8 * c);
}
__device__ __forceinline__ int rope_second(const RopeShape& r, int c) {
  return r.off + (r.interleaved ? 16 * c + 8 : 8 * c + (r.rot >> 1));
}

struct CosSin {
  float c[8], s[8];
};
// The eight angles of unit c from a table row [cos.. | sin..].
__device__ __forceinline__ CosSin load_cossin(const float* row, int rot, int c) {
  CosSin k;
  const float4* pc = reinterpret_cast<const float4*>(row + 8 * c);
  const float4* ps = reinterpret_cast<const float4*>(row + (rot >> 1) + 8 * c);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float4 a = pc[i], b = ps[i];
    k.c[4 * i] = a.x; k.c[4 * i + 1] = a.y; k.c[4 * i + 2] = a.z; k.c[4 * i + 3] = a.w;
    k.s[4 * i] = b.x; k.s[4 * i + 1] = b.y; k.s[4 * i + 2] = b.z; k.s[4 * i + 3] = b.w;
  }
  return k;
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

// a, b: the unit's two vectors; rotated in place.  Every product and sum is
// rounded by itself (the library is built without contraction).
__device__ __forceinline__ void rotate8(float a[8], float b[8], const CosSin& k, bool interleaved) {
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x1 = a[2 * i], x2 = a[2 * i + 1], y1 = b[2 * i], y2 = b[2 * i + 1];
      a[2 * i] = x1 * k.c[i] - x2 * k.s[i];
      a[2 * i + 1] = x2 * k.c[i] + x1 * k.s[i];
      b[2 * i] = y1 * k.c[4 + i] - y2 * k.s[4 + i];
      b[2 * i + 1] = y2 * k.c[4 + i] + y1 * k.s[4 + i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float x1 = a[i], x2 = b[i];
      a[i] = x1 * k.c[i] - x2 * k.s[i];
      b[i] = x2 * k.c[i] + x1 * k.s[i];
    }
  }
}

// One row's H heads of D values from x to y (may be the same), by one wave:
// lanes over units of 16 values, rotated units first, then the head's other
// dims to copy (units = D / 16, or rot / 16 where they stay in place).  Where
// the units of a head divide the wave (UNITS, or 0) a lane keeps its unit from
// head to head and its angles in registers.
template <int UNITS>
__device__ __forceinline__ void rotate_row(const uint16_t* x, uint16_t* y, int H, int D, const RopeShape& r, float sign,
                                           const float* cs_row, int units_any = 0) {
  const int lane = static_cast<int>(threadIdx.x) & 63, units = UNITS ? UNITS : units_any;
  int h = lane / units, c = lane - h * units;
  CosSin k;
  if (UNITS && 16 * c < r.rot) {
    k = load_cossin(cs_row, r.rot, c);
#pragma unroll
    for (int i = 0; i < 8; ++i) k.s[i] *= sign;
  }
  int ia, ib;
  auto place = [&]() {
    if (16 * c < r.rot) {
      ia = rope_first(r, c);
      ib = rope_second(r, c);
    } else {   // vectors 2j, 2j + 1 of those around the rotated part
      ia = 16 * (c - r.rot / 16);
      ib = ia + 8;
      ia += ia >= r.off ? r.rot : 0;
      ib += ib >= r.off ? r.rot : 0;
    }
  };
  if (UNITS) place();
#pragma unroll 4
  for (int e = lane; e < H * units; e += 64) {
    if (UNITS) {
      h = e / units;
    } else {
      h = e / units;
      c = e - h * units;
      place();
    }
    uint4 va = load16_nt(x + h * D + ia), vb = load16_nt(x + h * D + ib);
    if (16 * c < r.rot) {
      if (!UNITS) {
        k = load_cossin(cs_row, r.rot, c);
#pragma unroll
        for (int i = 0; i < 8; ++i) k.s[i] *= sign;
      }
      float a[8], b[8];
      unpack8(va, a);
      unpack8(vb, b);
      rotate8(a, b, k, r.interleaved);
      va = pack8(a);
      vb = pack8(b);
    }
    *reinterpret_cast<uint4*>(y + h * D + ia) = va;
    *reinterpret_cast<uint4*>(y + h * D + ib) = vb;
  }
}

// Largest b in 0 .. B-1 with key(b) <= t, for a non-decreasing key with
// key(0) <= t: 64 probes at a time, one to a lane of the wave, so 64
// sequences cost one load, 4096 two.  Every lane of the wave must call it.
template <typename Key>
__device__ __forceinline__ int search64(int B, int64_t t, Key key) {
  const int lane = static_cast<int>(threadIdx.x) & 63;
  int lo = 0, n = B;   // the answer lies in lo .. lo + n - 1
  while (n > 1) {
    const int step = (n + 63) >> 6;
    const int p = lane * step;
    const bool le = p < n && key(lo + p) <= t;
    const int cnt = __popcll(__ballot(le));          // le holds for a prefix of the lanes
    const int first = (cnt > 0 ? cnt - 1 : 0) * step;
    lo += first;
    n = n - first < step ? n - first : step;
  }
  return lo;
}

}  // namespace fp8bs
