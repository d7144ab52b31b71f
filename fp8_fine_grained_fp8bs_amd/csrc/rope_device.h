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
