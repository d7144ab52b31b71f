// attn_sched.h -- how the attention kernels share out their work (gfx950).
//
// The rows of a sequence and key/value head are its tokens' queries of that
// head's group, token by token: row r is token r / G, query head r % G of the
// group.  A tile is R consecutive rows; an item is a tile of one key/value
// head; its work is the units of 64 keys that its rows see.  Lengths are known
// on the device only, and differ by orders of magnitude inside a batch, so
// the items' units are laid end to end (heads outermost: neighbouring workers
// read the same head's cache) and every worker, a workgroup, takes an equal
// stretch of that line.  A stretch that starts or ends inside an item leaves
// a partial result (sums, maximum and denominator in FP32) in the workspace;
// a second kernel joins an item's partials in their order, so results do not
// depend on timing.  Every worker computes the line for itself: one load a
// sequence and a scan, about a microsecond, instead of another launch.
#pragma once

#include "fp8bs_internal.h"
#include "fp8bs_device.h"

namespace fp8bs {

constexpr int kUnit = 64;          // keys of a unit
constexpr int kMaxSlots = 2048;    // tiles a head that the line can hold

struct AttnArgs {
  AttnPaged p;
  int G;              // query heads a key/value head
  int pshift;         // log2(page)
  int max_len;        // tokens the table holds
  float scale_log2;   // scale * log2(e)
  int slots;          // tiles a head, some of them empty
  int most;           // tiles a sequence where slots are split directly, else 0
  int workers;        // 0: one item a workgroup, whole
  int min_units;      // least stretch of a worker
  float* part;        // partials: [2 workers][R][D + 2]
  int32_t* rec;       // records: [workers][8]
};

struct Tile {
  int b;
  int n;        // rows of tokens: the call's tokens of the sequence
  int64_t off;  // first packed row
  int row0, rows;
  int len;
  int lo, hi;   // keys seen by any row
  int u0, units;
};

__device__ __forceinline__ Tile tile_of(const AttnArgs& a, int slot, int R) {
  Tile t;
  int rt;
  if (a.most != 0) {
    t.b = slot / a.most;
    rt = slot - t.b * a.most;
  } else {
    // tiles of b <= floor(n_b G / R) + 1: numbered from floor(q_off[b] G / R) + b
    auto key = [&](int i) {
      const int64_t o = a.p.q_off == nullptr ? i : a.p.q_off[i];
      return o * a.G / R + i;
    };
    int lo = 0, hi = a.p.B - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (key(mid) <= slot) lo = mid;
      else hi = mid - 1;
    }
    t.b = lo;
    rt = static_cast<int>(slot - key(lo));
  }
  int64_t o = t.b, e = t.b + 1;
  if (a.p.q_off != nullptr) {
    o = a.p.q_off[t.b];
    e = a.p.q_off[t.b + 1];
    o = o < 0 ? 0 : o > a.p.T ? a.p.T : o;
    e = e < o ? o : e > a.p.T ? a.p.T : e;
  }
  t.off = o;
  t.n = static_cast<int>(e - o);
  const int64_t all = static_cast<int64_t>(t.n) * a.G, first = static_cast<int64_t>(rt) * R;
  if (rt < 0 || first >= all) {
    t.row0 = t.rows = t.len = t.lo = t.hi = t.u0 = t.units = 0;
    return t;
  }
  t.row0 = static_cast<int>(first);
  t.rows = static_cast<int>(all - first < R ? all - first : R);
  int len = a.p.kv_len[t.b];
  len = len < 0 ? 0 : len > a.max_len ? a.max_len : len;
  t.len = len;
  const int64_t p0 = static_cast<int64_t>(len) - t.n + t.row0 / a.G;
  const int64_t p1 = static_cast<int64_t>(len) - t.n + (t.row0 + t.rows - 1) / a.G;
  const int64_t hi = a.p.causal && p1 + 1 < len ? p1 + 1 : len;
  const int64_t lo = a.p.window > 0 && p0 - a.p.window + 1 > 0 ? p0 - a.p.window + 1 : 0;
  const bool some = hi > lo;
  t.lo = some ? static_cast<int>(lo) : 0;
  t.hi = some ? static_cast<int>(hi) : 0;
  t.u0 = t.lo / kUnit;
  t.units = some ? (t.hi + kUnit - 1) / kUnit - t.u0 : 1;   // rows that see nothing still get their zeros
  return t;
}

// Keys that one row sees.
__device__ __forceinline__ void row_keys(const AttnArgs& a, const Tile& t, int row, int& lo, int& hi) {
  const int64_t p = static_cast<int64_t>(t.len) - t.n + row / a.G;
  const int64_t h = a.p.causal && p + 1 < t.len ? p + 1 : t.len;
  const int64_t l = a.p.window > 0 && p - a.p.window + 1 > 0 ? p - a.p.window + 1 : 0;
  hi = h < 0 ? 0 : static_cast<int>(h);
  lo = l > t.len ? t.len : static_cast<int>(l);
}

// Consecutive workgroups run on different XCDs; worker numbers that share an
// XCD's L2 are consecutive.  n is a multiple of 8.
__device__ __forceinline__ int xcd_order(int bid, int n) { return (bid & 7) * (n >> 3) + (bid >> 3); }

// The line of units: prefix sums over one head's slots.
struct Line {
  int64_t* prefix;   // LDS [slots + 1]
  int64_t per_head;
  int64_t total;
  int workers;       // workers with a stretch
};

// Fills the line; every thread of a 256-thread workgroup calls it.
__device__ __forceinline__ Line make_line(const AttnArgs& a, int R, int64_t* prefix, int64_t* wave_sums) {
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 63;
  const int each = (a.slots + 255) >> 8;
  int64_t mine = 0;
  for (int i = 0; i < each; ++i) {
    const int s = tid * each + i;
    const int u = s < a.slots ? tile_of(a, s, R).units : 0;
    if (s < a.slots) prefix[s] = mine;
    mine += u;
  }
  int64_t run = mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int64_t o = __shfl_up(run, d);
    if (lane >= d) run += o;
  }
  if (lane == 63) wave_sums[tid >> 6] = run;
  __syncthreads();
  int64_t before = run - mine, all = 0;
  for (int w = 0; w < 4; ++w) {
    if (w < (tid >> 6)) before += wave_sums[w];
    all += wave_sums[w];
  }
  for (int i = 0; i < each; ++i) {
    const int s = tid * each + i;
    if (s < a.slots) prefix[s] += before;
  }
  if (tid == 0) prefix[a.slots] = all;
  __syncthreads();
  Line l;
  l.prefix = prefix;
  l.per_head = all;
  l.total = all * a.p.Hkv;
  const int64_t useful = (l.total + a.min_units - 1) / a.min_units;
  l.workers = static_cast<int>(useful < a.workers ? useful : a.workers);
  return l;
}
__device__ __forceinline__ int64_t stretch_begin(const Line& l, int w) { return w * l.total / l.workers; }
// The worker whose stretch holds unit x.
__device__ __forceinline__ int worker_of(const Line& l, int64_t x) {
  return static_cast<int>(((x + 1) * l.workers - 1) / l.total);
}
// The slot whose units hold place x of a head's line.
__device__ __forceinline__ int slot_of(const AttnArgs& a, const Line& l, int64_t x) {
  int lo = 0, hi = a.slots - 1;   // last slot with prefix <= x (empty slots share their successor's prefix)
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (l.prefix[mid] <= x) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Where a tile row's query and output live.
__device__ __forceinline__ int64_t row_token(const AttnArgs& a, const Tile& t, int r) { return t.off + (t.row0 + r) / a.G; }
__device__ __forceinline__ int row_head(const AttnArgs& a, const Tile& t, int h, int r) {
  return h * a.G + (t.row0 + r) % a.G;
}

// One finished row's 1/16th (VW = D / 16 values from dim d0) to the output.
template <int VW>
__device__ __forceinline__ void store_out(const AttnArgs& a, int64_t token, int head, int D, int d0, const float* o,
                                          float m, float l) {
  const float inv = l > 0.0f ? 1.0f / l : 0.0f;
  uint32_t w[VW / 2];
#pragma unroll
  for (int i = 0; i < VW / 2; ++i) w[i] = pack_bf16x2_rne(o[2 * i] * inv, o[2 * i + 1] * inv);
  uint16_t* at = a.p.out + token * a.p.ldo + static_cast<int64_t>(head) * D + d0;
  if (VW == 8) *reinterpret_cast<uint4*>(at) = make_uint4(w[0], w[1], w[2 % (VW / 2)], w[3 % (VW / 2)]);
  else *reinterpret_cast<uint2*>(at) = make_uint2(w[0], w[1]);
  if (d0 == 0 && a.p.lse != nullptr)
    a.p.lse[token * a.p.ldl + head] =
        l > 0.0f ? (m + __builtin_amdgcn_logf(l)) * 0.693147180559945f : -__builtin_huge_valf();
}

// One partial row's 1/16th.
template <int VW>
__device__ __forceinline__ void store_part(float* part, int R, int D, int64_t piece, int r, int d0, const float* o,
                                           float m, float l) {
  float* base = part + piece * R * (D + 2);
  float4* at = reinterpret_cast<float4*>(base + r * D + d0);
#pragma unroll
  for (int i = 0; i < VW / 4; ++i) at[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
  if (d0 == 0) {
    base[R * D + 2 * r] = m;
    base[R * D + 2 * r + 1] = l;
  }
}

}  // namespace fp8bs
