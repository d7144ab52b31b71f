// attn_sched.h -- how the attention kernels share out their work (gfx950).
//
// The rows of a sequence and key/value head are its tokens' queries of that
// head's group, token by token: row r is token r / G, query head r % G of the
// group.  A tile is R consecutive rows; an item is a tile of one key/value
// head; its work is the units of 64 keys that its rows see.  Lengths are known
// on the device only, and differ by orders of magnitude inside a batch, so
// the items' units are laid end to end (heads outermost: neighbouring workers
// read the same head's cache) and every worker, a workgroup, takes an equal
// stretch of that line.  An item takes kOpen units of the line more than it has:
// lookups, queries and the first keys' way from memory cost a worker 2 to 6 us, as
// much as some units (a stretch that ends in them has nothing of the item).
// A stretch that starts or ends inside an item leaves
// a partial result (sums, maximum and denominator in FP32) in the workspace;
// a second kernel joins an item's partials in their order, so results do not
// depend on timing.  Every worker computes the line for itself: one load a
// sequence and a scan, about a microsecond, instead of another launch.
#pragma once

#include "fp8bs_internal.h"
#include "packed_search.h"

namespace fp8bs {

constexpr int kUnit = 64;          // keys of a unit
constexpr int kManyRows = 128;     // rows of a tile of the many-rows kernel
constexpr int kMaxSlots = 2048;    // tiles a head that the line can hold
// Opening an item, in units.  With 0, 2, 4, 6 and 8: 96 requests of one token
// 141 133 133 135 137 us, heads of 64 34.1 31.0 29.7 30.3 32.0, drafted tokens
// 46.9 46.2 42.7 42.1 42.5.
constexpr int kOpen = 4;

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
  bool by_item;       // records are numbered by item, else by worker
  float* part;        // partials: [2 workers][R][D + 2]
  int32_t* rec;       // records: [items or workers][8]
};

// The many-rows kernel on `blocks` workgroups (a multiple of 8).
hipError_t launch_attn_prompt(const AttnArgs& a, unsigned blocks, hipStream_t st);

// A value that every lane of the wave has, kept in a scalar register (a load
// gives the compiler no way to know).
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

// A tile's place, and what the device memory says of its sequence.
struct Place {
  int b, rt;      // sequence, tile of the sequence
  int off, n;     // first packed row, rows of tokens
  int len;        // tokens in the cache
};
struct Tile {
  int b;
  int n;          // the call's tokens of the sequence
  int off;        // first packed row
  int row0, rows;
  int len;
  int lo, hi;     // keys seen by any row
  int u0, units;
};

// SAME: every lane asks for the same slot.
template <bool SAME>
__device__ __forceinline__ Place place_of(const AttnArgs& a, int slot, int R) {
  auto same = [](int x) { return SAME ? uniform(x) : x; };
  Place p;
  if (a.most == 1) {
    p.b = slot;
    p.rt = 0;
  } else if (a.most != 0) {
    p.b = static_cast<int>(static_cast<unsigned>(slot) / static_cast<unsigned>(a.most));
    p.rt = slot - p.b * a.most;
  } else {
    // tiles of b <= floor(n_b G / R) + 1: numbered from floor(q_off[b] G / R) + b
    auto key = [&](int i) {
      const int64_t o = a.p.q_off == nullptr ? i : a.p.q_off[i];
      return o * a.G / R + i;
    };
    int lo = 0;
    if (SAME) {
      lo = uniform(search64(a.p.B, slot, key));
    } else {
      int hi = a.p.B - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (key(mid) <= slot) lo = mid;
        else hi = mid - 1;
      }
    }
    p.b = lo;
    p.rt = same(static_cast<int>(slot - key(lo)));
  }
  int o = p.b, e = p.b + 1, len = a.p.kv_len[p.b];
  if (a.p.q_off != nullptr) {
    o = a.p.q_off[p.b];
    e = a.p.q_off[p.b + 1];
  }
  const int T = static_cast<int>(a.p.T);
  o = same(o);
  e = same(e);
  len = same(len);
  p.off = o < 0 ? 0 : o > T ? T : o;
  e = e < p.off ? p.off : e > T ? T : e;
  p.n = e - p.off;
  p.len = len < 0 ? 0 : len > a.max_len ? a.max_len : len;
  return p;
}

__device__ __forceinline__ Tile tile_at(const AttnArgs& a, const Place& p, int R) {
  Tile t;
  t.b = p.b;
  t.off = p.off;
  t.n = p.n;
  const int64_t all = static_cast<int64_t>(p.n) * a.G, first = static_cast<int64_t>(p.rt) * R;
  if (p.rt < 0 || first >= all) {
    t.row0 = t.rows = t.len = t.lo = t.hi = t.u0 = t.units = 0;
    return t;
  }
  t.row0 = static_cast<int>(first);
  t.rows = static_cast<int>(all - first < R ? all - first : R);
  t.len = p.len;
  const unsigned G = static_cast<unsigned>(a.G);
  const int64_t p0 = static_cast<int64_t>(p.len) - p.n + static_cast<unsigned>(t.row0) / G;
  const int64_t p1 = static_cast<int64_t>(p.len) - p.n + static_cast<unsigned>(t.row0 + t.rows - 1) / G;
  const int64_t hi = a.p.causal && p1 + 1 < p.len ? p1 + 1 : p.len;
  const int64_t lo = a.p.window > 0 && p0 - a.p.window + 1 > 0 ? p0 - a.p.window + 1 : 0;
  const bool some = hi > lo;
  t.lo = some ? static_cast<int>(lo) : 0;
  t.hi = some ? static_cast<int>(hi) : 0;
  t.u0 = t.lo / kUnit;
  t.units = some ? (t.hi - 1) / kUnit + 1 - t.u0 : 1;   // rows that see nothing still get their zeros
  return t;
}

// What a tile takes of the line.
__device__ __forceinline__ int line_units(const Tile& t) { return t.units == 0 ? 0 : t.units + kOpen; }

// Keys that one row sees.
__device__ __forceinline__ void row_keys(const AttnArgs& a, const Tile& t, int row, int& lo, int& hi) {
  const int64_t p = static_cast<int64_t>(t.len) - t.n + static_cast<unsigned>(row) / static_cast<unsigned>(a.G);
  const int64_t h = a.p.causal && p + 1 < t.len ? p + 1 : t.len;
  const int64_t l = a.p.window > 0 && p - a.p.window + 1 > 0 ? p - a.p.window + 1 : 0;
  hi = h < 0 ? 0 : static_cast<int>(h);
  lo = l > t.len ? t.len : static_cast<int>(l);
}

// Consecutive workgroups run on different XCDs; worker numbers that share an
// XCD's L2 are consecutive.  n is a multiple of 8.
__device__ __forceinline__ int xcd_order(int bid, int n) { return (bid & 7) * (n >> 3) + (bid >> 3); }

// Inclusive sum over the lanes up to this one (DPP row shifts, then the two
// row broadcasts).
__device__ __forceinline__ int wave_scan(int x) {
  x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xf, 0xf, true);   // row_shr:1
  x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xf, 0xf, true);
  x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xf, 0xf, true);
  x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xf, 0xf, true);
  x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, false);  // row_bcast:15 into rows 1 and 3
  x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, false);  // row_bcast:31 into rows 2 and 3
  return x;
}

// A worker's way along the line.  The first `longer` workers have q + 1
// units, the others q.  All of it fits 32 bits (the host sees to that).
struct Cursor {
  int q, longer;
  int w;              // worker, or item where items are whole
  int slot, h;        // the item
  int cur, stop;      // what is left of the stretch
  int first;          // the item's first unit
  Tile t;             // the item's tile
  int ub, ue;         // the piece: units ub .. ue - 1 of the item
  bool whole;
};

__device__ __forceinline__ int stretch_begin(const Cursor& c, int w) { return w * c.q + (w < c.longer ? w : c.longer); }
// The worker whose stretch holds unit x.
__device__ __forceinline__ int worker_of(const Cursor& c, int x) {
  const int head = c.longer * (c.q + 1);
  return x < head ? static_cast<int>(static_cast<unsigned>(x) / static_cast<unsigned>(c.q + 1))
                  : c.longer + static_cast<int>(static_cast<unsigned>(x - head) / static_cast<unsigned>(c.q));
}

// Shares a line of per_head units a head; false where this worker has none.
__device__ __forceinline__ bool share_line(const AttnArgs& a, int per_head, Cursor& c, int& in_head) {
  const unsigned total = static_cast<unsigned>(per_head) * static_cast<unsigned>(a.p.Hkv);
  const unsigned useful = (total + static_cast<unsigned>(a.min_units) - 1u) / static_cast<unsigned>(a.min_units);
  const unsigned workers = useful < static_cast<unsigned>(a.workers) ? useful : static_cast<unsigned>(a.workers);
  if (static_cast<unsigned>(c.w) >= workers) return false;
  c.q = static_cast<int>(total / workers);
  c.longer = static_cast<int>(total - static_cast<unsigned>(c.q) * workers);
  c.cur = stretch_begin(c, c.w);
  c.stop = stretch_begin(c, c.w + 1);
  c.h = static_cast<int>(static_cast<unsigned>(c.cur) / static_cast<unsigned>(per_head));
  in_head = c.cur - c.h * per_head;
  return true;
}

// Finds the worker's first item; false where it has none.  lds: at least
// kMaxSlots words, free again on return.  backwards: whole items are dealt
// from the last tile (a causal prompt's longest) on.
__device__ __forceinline__ bool begin_work(const AttnArgs& a, int R, bool backwards, void* lds, int* sums, Cursor& c) {
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 63;
  c.w = xcd_order(static_cast<int>(blockIdx.x), static_cast<int>(gridDim.x));
  if (a.workers == 0) {
    c.h = static_cast<int>(static_cast<unsigned>(c.w) / static_cast<unsigned>(a.slots));
    c.slot = c.w - c.h * a.slots;
    if (backwards) c.slot = a.slots - 1 - c.slot;
    if (c.h >= a.p.Hkv) return false;
    c.t = tile_at(a, place_of<true>(a, c.slot, R), R);
    c.cur = c.first = 0;
    c.stop = line_units(c.t);
    return c.t.units != 0;
  }
  if (!a.by_item && tid == 0) a.rec[c.w * 8] = 0;
  int in_head;
  if (a.slots <= 256) {   // up to four slots a lane, every wave for itself
    const int each = (a.slots + 63) >> 6;
    Place p[4];
    int units[4], mine = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int s = lane * each + i;
      p[i] = Place{0, -1, 0, 0, 0};
      if (i < each && s < a.slots) p[i] = place_of<false>(a, s, R);
      units[i] = line_units(tile_at(a, p[i], R));
      mine += units[i];
    }
    const int upto = wave_scan(mine), per_head = __builtin_amdgcn_readlane(upto, 63);
    if (!share_line(a, per_head, c, in_head)) return false;
    const int owner = __popcll(__ballot(upto <= in_head));   // lanes whose slots all end before it
    int left = in_head - (__builtin_amdgcn_readlane(upto, owner) - __builtin_amdgcn_readlane(mine, owner)), k = 0;
    Place s = p[0];
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const int u = __builtin_amdgcn_readlane(units[i], owner);
      if (k == i && left >= u) {   // also past empty slots
        left -= u;
        ++k;
        s = p[i + 1];
      }
    }
    s = Place{__builtin_amdgcn_readlane(s.b, owner), __builtin_amdgcn_readlane(s.rt, owner),
              __builtin_amdgcn_readlane(s.off, owner), __builtin_amdgcn_readlane(s.n, owner),
              __builtin_amdgcn_readlane(s.len, owner)};
    c.slot = owner * each + k;
    c.first = c.cur - left;
    c.t = tile_at(a, s, R);
    return true;
  }
  // prefix sums of every slot in LDS
  int* prefix = static_cast<int*>(lds);
  const int each = tid < 256 ? (a.slots + 255) >> 8 : 0;   // the first four waves add them up
  int mine = 0;
  for (int i = 0; i < each; ++i) {
    const int s = tid * each + i;
    if (s < a.slots) {
      prefix[s] = mine;
      mine += line_units(tile_at(a, place_of<false>(a, s, R), R));
    }
  }
  const int upto = wave_scan(mine);
  if (lane == 63 && tid < 256) sums[tid >> 6] = upto;
  __syncthreads();
  int before = upto - mine, all = 0;
  for (int w = 0; w < 4; ++w) {
    if (w < (tid >> 6)) before += sums[w];
    all += sums[w];
  }
  for (int i = 0; i < each; ++i) {
    const int s = tid * each + i;
    if (s < a.slots) prefix[s] += before;
  }
  __syncthreads();
  const bool some = share_line(a, uniform(all), c, in_head);
  if (!some) return false;
  int lo = 0, hi = a.slots - 1;   // the last slot that begins at or before it (an empty one shares its successor's place)
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (prefix[mid] <= in_head) lo = mid;
    else hi = mid - 1;
  }
  c.slot = uniform(lo);
  c.first = c.cur - in_head + uniform(prefix[lo]);
  c.t = tile_at(a, place_of<true>(a, c.slot, R), R);
  __syncthreads();
  return true;
}

// The part of the stretch that lies in the item at hand; false where it holds none
// of the item's units.
__device__ __forceinline__ bool take_piece(Cursor& c) {
  const int from = c.cur - c.first - kOpen, all = c.t.units, to = c.stop - c.first - kOpen;
  c.ub = from > 0 ? from : 0;
  c.ue = to < all ? to : all;
  c.cur = c.first + kOpen + c.ue;
  c.whole = c.ub == 0 && c.ue == all;
  return c.ue > c.ub;
}
// Whether the stretch goes on into units of another item.
__device__ __forceinline__ bool goes_on(const Cursor& c) { return c.stop - c.cur > kOpen; }

// To another reference, d = old - new (log2): its factor, and a denominator taken there.  That
// goes in two steps, for 2^d may fall below FP32's least where the product does not.
struct Moved {
  float half;
  __device__ __forceinline__ explicit Moved(float d) : half(__builtin_amdgcn_exp2f(0.5f * d)) {}
  __device__ __forceinline__ float factor() const { return half * half; }
  __device__ __forceinline__ float den(float l) const { return l * half * half; }
};

// Where the piece's partial belongs: a worker leaves two at most, of the item
// it ends in the middle of and of the one it begins in the middle of.
__device__ __forceinline__ int64_t piece_of(const Cursor& c) { return 2 * static_cast<int64_t>(c.w) + (c.ub == 0 ? 1 : 0); }

// Records how many pieces the item has, where this worker begins it.
__device__ __forceinline__ void record_piece(const AttnArgs& a, const Cursor& c) {
  if (a.workers != 0 && c.ub == 0 && (a.by_item || !c.whole) && threadIdx.x == 0) {
    int4* rec = reinterpret_cast<int4*>(a.rec + 8 * (a.by_item ? c.h * a.slots + c.slot : c.w));
    const int pieces = c.whole ? 0 : worker_of(c, c.first + kOpen + c.t.units - 1) - c.w + 1;
    rec[0] = make_int4(pieces, c.w, c.h, 0);
    rec[1] = make_int4(c.t.off, c.t.row0, c.t.rows, 0);
  }
}

// Goes on to the next item with rows; only where the stretch holds one.
__device__ __forceinline__ void next_item(const AttnArgs& a, int R, Cursor& c) {
  c.first += line_units(c.t);
  do {
    if (++c.slot == a.slots) {
      c.slot = 0;
      ++c.h;
    }
    c.t = tile_at(a, place_of<true>(a, c.slot, R), R);
  } while (c.t.units == 0);
}

// Where a tile row's query and output live.
__device__ __forceinline__ int64_t row_token(const AttnArgs& a, const Tile& t, int r) {
  return t.off + static_cast<int64_t>(static_cast<unsigned>(t.row0 + r) / static_cast<unsigned>(a.G));
}
__device__ __forceinline__ int row_head(const AttnArgs& a, const Tile& t, int h, int r) {
  return h * a.G + static_cast<int>(static_cast<unsigned>(t.row0 + r) % static_cast<unsigned>(a.G));
}

// One finished row's 1/16th (VW = D / 16 values from dim d0) to the output.
template <int VW>
__device__ __forceinline__ void store_out(const AttnArgs& a, int64_t token, int head, int D, int d0, const float* o,
                                          float m, float l) {
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;   // a NaN goes on
  uint32_t w[VW / 2];
#pragma unroll
  for (int i = 0; i < VW / 2; ++i) w[i] = pack_bf16x2_rne(o[2 * i] * inv, o[2 * i + 1] * inv);
  uint16_t* at = a.p.out + token * a.p.ldo + static_cast<int64_t>(head) * D + d0;
  if (VW == 8) *reinterpret_cast<uint4*>(at) = make_uint4(w[0], w[1], w[2 % (VW / 2)], w[3 % (VW / 2)]);
  else *reinterpret_cast<uint2*>(at) = make_uint2(w[0], w[1]);
  if (d0 == 0 && a.p.lse != nullptr)
    a.p.lse[token * a.p.ldl + head] =
        l == 0.0f ? -__builtin_huge_valf() : (m + __builtin_amdgcn_logf(l)) * 0.693147180559945f;
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
