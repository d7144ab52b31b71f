// kv_append.hip -- keys and values appended to a paged E4M3 cache, the
// rotation of keys and queries on the way (gfx950).
//
// A block of the cache is one page of one key/value head under one FP32
// scale.  One workgroup takes one (page, head): it reads the page's new keys
// and values once, rotates the keys, takes both max-abs, settles both scales
// and writes codes and scales.  No other workgroup touches the block, so a page that fills over
// many calls needs no atomics and the result does not depend on any order:
//   s' = max(s, fl32(amax(new) / 448)); where it grows, the codes already
//   there are encoded again from dec(code) * s.
// Nothing is rounded on the way to a code or a scale: rotated keys are formed as
// doubles, whose products of BF16 and FP32 are exact, held in FP32 for the
// encoder's brackets, and formed again for the values the brackets leave open.
// (Rotated in FP32, about one code in a million fell on the other side of a tie, and a
// third of the scales were an ulp off; the doubles cost 3 us of 90 on prompts.)
// The queries' rotation runs in further workgroups of the same launch: at
// one token a request the call is bound by its launch and its chain of
// dependent loads (offsets, table, cache), for prompts by HBM.  64 requests of one
// token, 32 query and 8 key/value heads of 128: 5.8 us.  Prompts of 20000 tokens
// in all, the same heads: 90 us, 5.1 TB/s of reads and writes.  A block's new tokens are all loaded
// before the first is rotated (92 us one after the other); eight waves a block
// with half the passes each took 102.
//
// Workgroups are laid over pages without knowing lengths on the host: with n_b
// tokens a sequence touches at most floor(n_b / page) + 2 pages, so slot
// numbers floor(q_off[b] / page) + 2 b leave room for each, and a workgroup
// finds its sequence by searching those numbers.  Where max_q gives a tighter
// bound (one token a request: one page each) the slot is split directly.
#include <hip/hip_runtime.h>

#include "fp8bs_internal.h"
#include "rope_device.h"

namespace fp8bs {
namespace {

struct AppendArgs {
  const uint16_t* q;
  int64_t ldq;
  uint16_t* qo;
  int64_t ldqo;
  int Hq;
  const uint16_t* k;
  int64_t ldk;
  const uint16_t* v;
  int64_t ldv;
  int Hkv;
  const float* cs;
  int64_t n_pos;
  RopeShape rope;
  const int32_t* q_off;
  const int32_t* kv_len;
  int B;
  int64_t T;
  const int32_t* table;
  int64_t ldt;
  int64_t max_pages;
  int pshift;
  uint8_t* kc;
  float* ks;
  uint8_t* vc;
  float* vs;
  int64_t n_pages;
  int64_t slots;
  int most;          // pages of a sequence where slots are split directly, else 0
  int64_t page_blocks;
};

// First packed row and row count of sequence b, inside 0 .. T.
__device__ __forceinline__ void rows_of(const int32_t* q_off, int64_t T, int b, int64_t& off, int& n) {
  if (q_off == nullptr) {
    off = b;
    n = 1;
    return;
  }
  int64_t a = q_off[b], e = q_off[b + 1];
  a = a < 0 ? 0 : a > T ? T : a;
  e = e < a ? a : e > T ? T : e;
  off = a;
  n = static_cast<int>(e - a);
}

// fl32(amax / 448) of an amax held as two parts, and the encoder's constants of a
// settled scale.
__device__ __forceinline__ float scale_for(float hi, float lo) {
  return static_cast<float>((static_cast<double>(hi) + lo) * (1.0 / 448.0));
}
__device__ __forceinline__ TileScale scale_of(float s) {
  TileScale t;
  t.s = s;
  t.fast = s >= kFastScaleMin;
  const float r = __builtin_amdgcn_rcpf(t.fast ? s : 1.0f);
  t.rlo = r * kMarginLo;
  t.rhi = r * kMarginHi;
  return t;
}

// Code of y / s for any scale: the magnitudes that bracket it, and where they
// differ the side of their midpoint that |y| is on, ties to even (y is exact to 2^-53,
// the midpoint times s exact).
__device__ __forceinline__ uint32_t code_of(double y, float s) {
  const uint32_t sign = static_cast<uint32_t>(__builtin_bit_cast(uint64_t, y) >> 56) & 0x80u;
  if (s == 0.0f) return sign;
  double a = __builtin_fabs(y);
  if (s < kFastScaleMin) {   // the reciprocal has to be a float
    a *= 0x1p64;
    s *= 0x1p64f;
  }
  const float x = static_cast<float>(a), r = __builtin_amdgcn_rcpf(s);
  const float x_lo = __builtin_fminf(x * (r * kMarginLo), kE4M3Max), x_hi = __builtin_fminf(x * (r * kMarginHi), kE4M3Max);
  const uint32_t lo = cvt4(x_lo, x_lo, x_lo, x_lo) & 0xffu, hi = cvt4(x_hi, x_hi, x_hi, x_hi) & 0xffu;
  const double mid = 0.5 * (static_cast<double>(e4m3_dec(lo)) + e4m3_dec(hi)) * s;
  return sign | (a > mid || (a == mid && (lo & 1u)) ? hi : lo);
}

// Codes of four values rounded to FP32; `open` where one hangs on more than that (one
// value in some 30000) or the scale is small: code_of then settles it.
__device__ __forceinline__ uint32_t encode_or_open(const float v[4], const TileScale& t, bool& open) {
  const uint32_t lo = cvt4(v[0] * t.rlo, v[1] * t.rlo, v[2] * t.rlo, v[3] * t.rlo);
  const uint32_t hi = cvt4(v[0] * t.rhi, v[1] * t.rhi, v[2] * t.rhi, v[3] * t.rhi);
  open |= lo != hi || !t.fast;
  return lo;
}

__device__ __forceinline__ const float* angles(const AppendArgs& a, int64_t p) {
  p = p < 0 ? 0 : p >= a.n_pos ? a.n_pos - 1 : p;
  return a.cs + p * a.rope.rot;
}

// One dim of a rotated key, exact to 2^-53 (products of BF16 and FP32 fit a
// double).
__device__ __forceinline__ double rotated(float x, float partner, float c, float s) {
  return __builtin_fma(static_cast<double>(x), static_cast<double>(c), static_cast<double>(partner) * s);
}

// A key's vector of 8 values at dim d and, where it is rotated by halves, the unit's
// other one (from the cache, another thread owns it).
struct KeyLoad {
  uint4 w, z;
};
__device__ __forceinline__ KeyLoad load_key(const AppendArgs& a, const uint16_t* row, int d) {
  KeyLoad v;
  v.w = v.z = *reinterpret_cast<const uint4*>(row + d);
  const RopeShape& r = a.rope;
  const int o = d - r.off, half = r.rot >> 1;
  if (a.cs != nullptr && !r.interleaved && o >= 0 && o < r.rot)
    v.z = *reinterpret_cast<const uint4*>(row + (o >= half ? d - half : d + half));
  return v;
}

// Its values, rotated where d lies in the rotated part, each given to take(i, value):
// one at a time, a double is two registers.
template <class F>
__device__ __forceinline__ void turn_key(const AppendArgs& a, const KeyLoad& v, int64_t p, int d, F take) {
  const uint4 w = v.w, z = v.z;
  auto value = [](const uint4& v, int i) {
    const uint32_t u = i < 2 ? v.x : i < 4 ? v.y : i < 6 ? v.z : v.w;
    return i & 1 ? bf16_hi(u) : bf16_lo(u);
  };
  const RopeShape& r = a.rope;
  const int o = d - r.off;
  if (a.cs == nullptr || o < 0 || o >= r.rot) {
#pragma unroll
    for (int i = 0; i < 8; ++i) take(i, static_cast<double>(value(w, i)));
    return;
  }
  CosSin k;
  if (r.interleaved) {   // the vector's four pairs are its own
    load_angles4(k, 0, angles(a, p), r.rot, o >> 3);
#pragma unroll
    for (int i = 0; i < 8; ++i) take(i, rotated(value(w, i), value(w, i ^ 1), k.c[i >> 1], i & 1 ? k.s[i >> 1] : -k.s[i >> 1]));
  } else {
    const int half = r.rot >> 1;
    const bool second = o >= half;
    const int j = (second ? o - half : o) >> 2;
    load_angles4(k, 0, angles(a, p), r.rot, j);
    load_angles4(k, 1, angles(a, p), r.rot, j + 1);
#pragma unroll
    for (int i = 0; i < 8; ++i) take(i, rotated(value(w, i), value(z, i), k.c[i], second ? k.s[i] : -k.s[i]));
  }
}

// Encodes the `there` tokens a block already holds for its larger scale, four
// vectors a thread on their way at a time (64 requests whose blocks all grow: 9.8 us
// with the events around them, 10.3 one after the other).
template <int D>
__device__ __forceinline__ void rescale_old(uint8_t* codes, int there, float s_old, const TileScale& ts) {
  constexpr int STEP = 2048 / D;
  const int sub = (static_cast<int>(threadIdx.x) % (D / 8)) * 8;
  for (int r0 = static_cast<int>(threadIdx.x) / (D / 8); r0 < there; r0 += 4 * STEP) {
    uint2 c[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int r = r0 + u * STEP;
      c[u] = *reinterpret_cast<const uint2*>(codes + (r < there ? r : r0) * D + sub);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int r = r0 + u * STEP;
      if (r < there) {
        float f[8];
        auto value = [&](int j) { return e4m3_dec(((j < 4 ? c[u].x : c[u].y) >> (8 * (j & 3))) & 0xffu); };
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = value(j) * s_old;
        bool open = false;
        uint32_t w[2] = {encode_or_open(f, ts, open), encode_or_open(f + 4, ts, open)};
        if (__builtin_expect(open, 0)) {
          w[0] = w[1] = 0;
#pragma unroll
          for (int j = 0; j < 8; ++j) w[j >> 2] |= code_of(static_cast<double>(value(j)) * s_old, ts.s) << (8 * (j & 3));
        }
        *reinterpret_cast<uint2*>(codes + r * D + sub) = make_uint2(w[0], w[1]);
      }
    }
  }
}

// NP: passes of 2048 values over a block's new tokens (256 threads, 8 values each).
template <int D, int NP>
__global__ __launch_bounds__(256) void kv_append_kernel(AppendArgs a) {
  __shared__ float red[3][4];
  poison_lds<sizeof(red)>(red);
  const int tid = static_cast<int>(threadIdx.x);
  int64_t bid = blockIdx.x;
  if (bid >= a.page_blocks) {   // queries: a wave a token, its lanes over units of 16 values
    const int64_t t = (bid - a.page_blocks) * 4 + (tid >> 6);
    if (t >= a.T) return;
    const int b = a.q_off == nullptr ? static_cast<int>(t)
                                     : search64(a.B, t, [&](int i) { return static_cast<int64_t>(a.q_off[i]); });
    int64_t off;
    int n;
    rows_of(a.q_off, a.T, b, off, n);
    const int64_t p = static_cast<int64_t>(a.kv_len[b]) - n + (t - off);
    rotate_row<D / 16>(a.q + t * a.ldq, a.qo + t * a.ldqo, a.Hq, D, a.rope, 1.0f, angles(a, p), false);
    return;
  }
  const int h = static_cast<int>(bid % a.Hkv);
  const int64_t slot = bid / a.Hkv;
  int b, nth;
  if (a.most != 0) {
    b = static_cast<int>(slot / a.most);
    nth = static_cast<int>(slot - static_cast<int64_t>(b) * a.most);
  } else {
    auto key = [&](int i) {
      const int64_t o = a.q_off == nullptr ? i : a.q_off[i];
      return (o >> a.pshift) + 2 * static_cast<int64_t>(i);
    };
    b = search64(a.B, slot, key);
    nth = static_cast<int>(slot - key(b));
  }
  int64_t off;
  int n;
  rows_of(a.q_off, a.T, b, off, n);
  const int64_t len = a.kv_len[b], start = len - n;
  if (n == 0 || start < 0) return;
  const int64_t pg = (start >> a.pshift) + nth;      // the page's place in the sequence
  const int64_t base = pg << a.pshift;
  if (base >= len || pg >= a.max_pages) return;
  const int64_t id = a.table[b * a.ldt + pg];
  if (id < 0 || id >= a.n_pages) return;
  const int there = static_cast<int>(start > base ? start - base : 0);
  const int64_t left = len - base, page = int64_t(1) << a.pshift;
  const int end = static_cast<int>(left < page ? left : page);
  const int64_t blk = id * a.Hkv + h;
  const float sk_old = there > 0 ? a.ks[blk] : 0.0f, sv_old = there > 0 ? a.vs[blk] : 0.0f;

  const int sub = (tid % (D / 8)) * 8, row0 = there + tid / (D / 8);
  KeyLoad kw[NP];
  uint4 vw[NP];
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const int r = i * (2048 / D) + row0;
    if (r < end) {
      const int64_t t = off + (base + r - start);
      kw[i] = load_key(a, a.k + t * a.ldk + h * D, sub);
      vw[i] = load16_nt(a.v + t * a.ldv + h * D + sub);
    }
  }
  float kf[NP][8];
  double top = 0.0;   // of the keys
  float mv = 0.0f;
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const int r = i * (2048 / D) + row0;
    if (r < end) {
      turn_key(a, kw[i], base + r, sub, [&](int j, double y) {
        top = __builtin_fmax(top, __builtin_fabs(y));
        kf[i][j] = static_cast<float>(y);
        __builtin_amdgcn_sched_barrier(0);
      });
      float f[8];
      unpack8(vw[i], f);
#pragma unroll
      for (int j = 0; j < 8; ++j) mv = __builtin_fmaxf(mv, __builtin_fabsf(f[j]));
    }
  }
  // the keys' maximum in two parts, both not negative: the FP32 number at or below
  // it, and what the largest have beyond that
  float mine = static_cast<float>(top);
  if (mine > top) mine = __uint_as_float(__float_as_uint(mine) - 1);
  const float beyond = mine < __builtin_inff() ? static_cast<float>(top - mine) : 0.0f;
  float mk = wave_max(mine), mk_lo = wave_max(mine == mk ? beyond : 0.0f);
  mv = wave_max(mv);
  if ((tid & 63) == 0) {
    red[0][tid >> 6] = mk;
    red[1][tid >> 6] = mv;
    red[2][tid >> 6] = mk_lo;
  }
  __syncthreads();
  mk = __builtin_fmaxf(__builtin_fmaxf(red[0][0], red[0][1]), __builtin_fmaxf(red[0][2], red[0][3]));
  mv = __builtin_fmaxf(__builtin_fmaxf(red[1][0], red[1][1]), __builtin_fmaxf(red[1][2], red[1][3]));
  mk_lo = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) mk_lo = red[0][i] == mk ? __builtin_fmaxf(mk_lo, red[2][i]) : mk_lo;
  const float sk = __builtin_fmaxf(sk_old, scale_for(mk, mk_lo));
  const float sv = __builtin_fmaxf(sv_old, make_tile_scale(mv).s);
  const TileScale tk = scale_of(sk), tv = scale_of(sv);
  uint8_t* kc = a.kc + (blk << a.pshift) * D;
  uint8_t* vc = a.vc + (blk << a.pshift) * D;
  uint32_t open = 0;   // passes with a key's code to settle
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const int r = i * (2048 / D) + row0;
    if (r < end) {
      float f[8];
      unpack8(vw[i], f);
      bool here = false;
      const uint32_t lo = encode_or_open(kf[i], tk, here), hi = encode_or_open(kf[i] + 4, tk, here);
      *reinterpret_cast<uint2*>(kc + r * D + sub) = make_uint2(lo, hi);
      open |= static_cast<uint32_t>(here) << i;
      *reinterpret_cast<uint2*>(vc + r * D + sub) = make_uint2(encode4(f, tv), encode4(f + 4, tv));
    }
  }
#pragma unroll 1
  for (; open != 0; open &= open - 1) {
    const int r = __builtin_ctz(open) * (2048 / D) + row0;
    const uint16_t* row = a.k + (off + (base + r - start)) * a.ldk + h * D;
    uint32_t w[2] = {0, 0};
    turn_key(a, load_key(a, row, sub), base + r, sub, [&](int j, double y) {
      w[j >> 2] |= code_of(y, sk) << (8 * (j & 3));
      __builtin_amdgcn_sched_barrier(0);
    });
    *reinterpret_cast<uint2*>(kc + r * D + sub) = make_uint2(w[0], w[1]);
  }
  if (sk > sk_old) rescale_old<D>(kc, there, sk_old, tk);
  if (sv > sv_old) rescale_old<D>(vc, there, sv_old, tv);
  if (tid == 0) {
    a.ks[blk] = sk;
    a.vs[blk] = sv;
  }
}

}  // namespace

hipError_t launch_kv_append(const KvAppend& p, hipStream_t st) {
  AppendArgs a;
  a.q = p.q; a.ldq = p.ldq; a.qo = p.q_out; a.ldqo = p.ldqo; a.Hq = p.Hq;
  a.k = p.k; a.ldk = p.ldk; a.v = p.v; a.ldv = p.ldv; a.Hkv = p.Hkv;
  a.cs = p.cs; a.n_pos = p.n_pos; a.rope = RopeShape{p.rot, p.rot_off, p.interleaved};
  a.q_off = p.q_off; a.kv_len = p.kv_len; a.B = p.B; a.T = p.T;
  a.table = p.table; a.ldt = p.ldt; a.max_pages = p.max_pages;
  a.pshift = __builtin_ctz(static_cast<unsigned>(p.page));
  a.kc = p.kc; a.ks = p.ks; a.vc = p.vc; a.vs = p.vs; a.n_pages = p.n_pages;
  const int64_t max_q = p.max_q < p.T ? p.max_q : p.T, most = (max_q + p.page - 2) / p.page + 1;
  const int64_t direct = most * p.B, searched = p.T / p.page + 2 * static_cast<int64_t>(p.B);
  a.most = direct <= searched ? static_cast<int>(most) : 0;
  a.slots = direct <= searched ? direct : searched;
  a.page_blocks = a.slots * p.Hkv;
  const int64_t blocks = a.page_blocks + (p.q != nullptr ? (p.T + 3) / 4 : 0);
  if (blocks > 0x7fffffff) return hipErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(blocks)), block(256);
  // passes over the tokens that one call can add to a page
  const int64_t adds = max_q < p.page ? max_q : p.page;
  const int need = static_cast<int>((adds * p.D + 2047) / 2048), np = need <= 2 ? need : need <= 4 ? 4 : 8;
#define FP8BS_APPEND(D_, NP_) \
  if (p.D == D_ && np == NP_) hipLaunchKernelGGL((kv_append_kernel<D_, NP_>), grid, block, 0, st, a)
  FP8BS_APPEND(64, 1);
  FP8BS_APPEND(64, 2);
  FP8BS_APPEND(64, 4);
  FP8BS_APPEND(128, 1);
  FP8BS_APPEND(128, 2);
  FP8BS_APPEND(128, 4);
  FP8BS_APPEND(128, 8);
#undef FP8BS_APPEND
  return hipGetLastError();
}

}  // namespace fp8bs
