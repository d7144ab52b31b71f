// attn.hip -- attention over the paged E4M3 cache: few rows a key/value head
// (decoding), and the joining of partial results (gfx950).
//
// For few rows the call reads len * 2 D bytes of cache a key/value head and
// does 4 D operations a byte pair and row: HBM-bound, so the kernel is built
// around loads in flight.  A wave takes steps of 32 keys, its loads going
// straight from the cache to registers (no LDS, no barrier in the loop), two
// steps in flight, page numbers a further step ahead.  Loads are
// non-temporal: each byte is read once (96 requests of one token: 123 us, with plain
// loads 137.  A cache of 100 MB that is attended again right away, with nothing between,
// stays in the last-level cache with plain loads: 25.0 against 26.7 with heads of 64).
//
// Measured, heads of 128, pages of 64, 32 query heads on 8: 96 requests of 200 to
// 16384 tokens 117 us in this kernel, 6.3 TB/s of the cache's bytes (blocks of 8 KB
// in random order are read at 6.4 by loads alone, a linear copy's reads at 7.1); one
// request of 130000 tokens 45 us, 5.9 TB/s.  Those are bound by HBM.  48 requests with
// heads of 64 take 24 us for 106 MB, 24 requests of 4 drafted tokens and 7 query
// heads a key/value head 35 us for 139 MB: with every page in the caches they would take
// 22 and 33 with the join, so HBM does not bound these.  A wave has 8 steps in the second:
// 393 VALU instructions a step by the counters, 260 in the listing of a step, the rest
// the pieces' starts and joins; VALU is active in 22 % of the wave cycles (two waves a SIMD),
// the matrix units in less.  So it is the chain of each start and join, which few steps
// pay for, and the second launch (5 us) that bound these, with some 58 of a step's
// instructions finding pages and 64-bit addresses by lane.
//
// Mathematics of a step.  S^T = K Q^T on 16x16x32 BF16 MFMAs (every E4M3 code
// is a BF16 value, products are exact), so a lane holds scores of one query row
// (column lane % 16).  With a value block's scale v and key block's scale k
// (both of the lane's 8 keys' page), s' = s * (k scale log2 e) + log2 v is one
// FMA, p' = 2^(s' - m) already carries the value scale, the denominator
// takes p' / v (another FMA), and the values enter the second product as their
// bare codes: O^T += V^T P'^T.  P' goes to FP16 (11 significant bits, where BF16's 8
// would double the output's rounding error) and the codes too, exactly.
// m is a reference, not the exact maximum: it is moved (and O, l rescaled)
// only when a score exceeds it by 2^15; a move sets the largest p' to 2^8, so
// FP16 neither overflows nor loses weights above 2^-33 of the largest.  Keys whose v is
// below 2^-32, blocks of zeros above all, reach the denominator as p / 2^m instead, in a
// second pass over the steps of a piece that has some (kTinyV): p' / v would overflow for a
// long context of them, and vanish beside values 2^43 and larger.
//
// Layouts.  Key rows of the two 16-row MFMA tiles are assigned so that
// lane group g = lane / 16 gets the scores of keys 8g .. 8g+7: those are the
// 8 consecutive k of its P'^T operand, no exchange between lanes.  The
// inner dims are permuted the same way on both sides so that a lane loads 16
// contiguous key bytes.  V^T needs 8 keys of one dim in a lane: it loads 8 keys x
// D/16 dims and transposes bytes in registers (2 v_perm_b32 a dword).
#include <hip/hip_runtime.h>

#include "attn_device.h"

namespace fp8bs {
namespace {

// What a wave holds of one step of 32 keys.
template <int D>
struct Step {
  u32x4 k[2][D / 64];          // two MFMA tiles of 16 keys, 16 bytes a lane and 64 dims
  uint32_t v[8][D / 64];       // 8 keys, D/16 dims a lane
  float ks, vs;                // scales of the lane's 8 keys
};

// Page numbers of a step: of the lane's key row and of its 8 keys.
struct Pages {
  int k, v;
};

template <int D, int NR>
__global__ __launch_bounds__(256, D == 64 && NR == 1 ? 4 : 2) void attn_rows_kernel(AttnArgs a) {
  constexpr int R = 16 * NR, VW = D / 16, NW = D / 64;
  __shared__ __attribute__((aligned(16))) float obuf[4][16][D + 4];
  __shared__ float ml[4][16][2];
  static_assert(sizeof(obuf) >= kMaxSlots * sizeof(int), "the line's prefix sums fit");
  __shared__ int sums[4];
  poison_lds<sizeof(obuf)>(obuf);
  poison_lds<sizeof(ml)>(ml);
  poison_lds<sizeof(sums)>(sums);
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 63, wv = uniform(tid >> 6);
  const int m16 = lane & 15, g = lane >> 4;
  const int page_mask = (1 << a.pshift) - 1;

  Cursor c;
  if (!begin_work(a, R, false, obuf, sums, c) || !take_piece(c)) return;
  const Tile& t = c.t;
  const int& h = c.h;
  // The piece at hand: its queries (B operands, row m16 of each 16-row group),
  // the keys that the lane's rows and all rows see, its steps of 32 keys, and
  // the page numbers of the wave's next step.
  bf16x8 qf[NR][2 * NW];
  int rlo[NR], rhi[NR];
  int all_lo, all_hi, base, steps;
  const int32_t* table;
  Pages pg, pg4;
  const int last_page = static_cast<int>(a.p.max_pages) - 1;
  auto load_pages = [&](int s) {
    Pages p;
    const int t0 = base + 32 * s;
    const int ik = (t0 + 8 * (m16 >> 2)) >> a.pshift, iv = (t0 + 8 * g) >> a.pshift;
    p.k = table[ik < last_page ? ik : last_page];
    p.v = table[iv < last_page ? iv : last_page];
    return p;
  };
  auto open_piece = [&]() {
    table = a.p.table + t.b * a.p.ldt;
    base = (t.u0 + c.ub) * kUnit;
    steps = (c.ue - c.ub) * (kUnit / 32);
    if (base + 32 * steps > t.hi) steps = t.hi > base ? (t.hi - base + 31) / 32 : 0;
    if (wv < steps) {
      pg = load_pages(wv);
      pg4 = load_pages(wv + 4);
    }
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      const int row = 16 * r + m16;
      const bool there = row < t.rows;
      const int rr = there ? row : 0;
      row_keys(a, t, t.row0 + rr, rlo[r], rhi[r]);
      if (!there) rhi[r] = 0;
      const uint16_t* q = a.p.q + row_token(a, t, rr) * a.p.ldq + static_cast<int64_t>(row_head(a, t, h, rr)) * D;
#pragma unroll
      for (int e = 0; e < 2 * NW; ++e)   // a row beyond the last computes row 0 and is not stored
        qf[r][e] = __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4*>(q + 64 * (e >> 1) + 16 * g + 8 * (e & 1)));
    }
    // keys that every row sees need no mask
    int x;
    row_keys(a, t, t.row0, x, all_hi);
    row_keys(a, t, t.row0 + t.rows - 1, all_lo, x);
  };
  open_piece();

  while (true) {
    f32x4 o[NR][4 * NW];
    float mr[NR], lr[NR];
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      mr[r] = kNoKeys;
      lr[r] = 0.0f;
#pragma unroll
      for (int i = 0; i < 4 * NW; ++i) o[r][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }

    auto clamp_page = [&](int id) {
      const unsigned u = static_cast<unsigned>(id), n = static_cast<unsigned>(a.p.n_pages) - 1u;
      return static_cast<int>(u < n ? u : n);
    };
    auto load_step = [&](int s, const Pages& pg) {
      Step<D> x;
      const int t0 = base + 32 * s;
      const int64_t bk = static_cast<int64_t>(clamp_page(pg.k)) * a.p.Hkv + h;
      const int64_t bv = static_cast<int64_t>(clamp_page(pg.v)) * a.p.Hkv + h;
      const int tk = (t0 + 8 * (m16 >> 2) + (m16 & 3)) & page_mask, tv = (t0 + 8 * g) & page_mask;
      const uint8_t* pk = a.p.kc + ((bk << a.pshift) + tk) * D + 16 * g;
      const uint8_t* pv = a.p.vc + ((bv << a.pshift) + tv) * D + m16 * VW;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int c = 0; c < NW; ++c) x.k[i][c] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(pk + 4 * i * D + 64 * c));
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (NW == 2) {
          const u32x2 y = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(pv + j * D));
          x.v[j][0] = y[0];
          x.v[j][NW - 1] = y[1];
        } else {
          x.v[j][0] = __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(pv + j * D));
        }
      }
      x.ks = a.p.ks[bv];
      x.vs = a.p.vs[bv];
      return x;
    };
    auto scores = [&](const Step<D>& x, f32x4 (&sc)[NR][2]) {
#pragma unroll
      for (int r = 0; r < NR; ++r) sc[r][0] = sc[r][1] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int c = 0; c < 2 * NW; ++c) {
          const bf16x8 kf = bf16_of_codes(x.k[i][c >> 1][2 * (c & 1)], x.k[i][c >> 1][2 * (c & 1) + 1]);
#pragma unroll
          for (int r = 0; r < NR; ++r)
            sc[r][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, qf[r][c], sc[r][i], 0, 0, 0);
        }
    };
    auto of_row = [](float x) {   // the largest of a row's four lanes
      x = __builtin_fmaxf(x, __shfl_xor(x, 16));
      return __builtin_fmaxf(x, __shfl_xor(x, 32));
    };
    auto move = [&](int r, float to) {   // the reference
      const Moved by(mr[r] - to);
      lr[r] = by.den(lr[r]);
      mr[r] = to;
#pragma unroll
      for (int i = 0; i < 4 * NW; ++i) o[r][i] *= by.factor();
    };
    bool tiny = false;   // a step had keys with a tiny value scale
    auto compute = [&](int s, Step<D>& x) {
      const int t0 = base + 32 * s, mine = t0 + 8 * g;
      const bool clear = t0 >= all_lo && t0 + 32 <= all_hi;
      float kq = x.ks * a.scale_log2;
      float vs = x.vs > kMinVScale ? x.vs : kMinVScale;
      if (!clear) {
        // keys that no row sees may hold anything: their values become zero
        // codes, the scales of a page that lies wholly outside become harmless
        const bool none = mine >= t.hi || mine + 8 <= t.lo;
        kq = none ? 0.0f : kq;
        vs = none ? 1.0f : vs;
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (mine + j >= t.hi || mine + j < t.lo)
#pragma unroll
            for (int c = 0; c < NW; ++c) x.v[j][c] = 0u;
      }
      const float lv = __builtin_amdgcn_logf(vs);
      const bool few = vs < kTinyV;   // summed apart
      const float iv = few ? 0.0f : __builtin_amdgcn_rcpf(vs);
      tiny |= __ballot(few) != 0;
      f32x4 sc[NR][2];
      scores(x, sc);
      f16x8 pf16[NR];
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        float e[8];
        float top = -__builtin_huge_valf();
#pragma unroll
        for (int j = 0; j < 8; ++j) e[j] = __builtin_fmaf(sc[r][j >> 2][j & 3], kq, lv);
        if (!clear) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            e[j] = mine + j >= rlo[r] && mine + j < rhi[r] ? e[j] : -__builtin_huge_valf();
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) top = __builtin_fmaxf(top, e[j]);
        if (__ballot(top > mr[r] + kHeadroom) != 0) {
          top = of_row(top);
          move(r, top > mr[r] + kHeadroom ? top - kTop : mr[r]);
        }
        u32x4 pw;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          e[j] = __builtin_amdgcn_exp2f(e[j] - mr[r]);
          lr[r] = __builtin_fmaf(e[j], iv, lr[r]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) pw[j] = pack_f16x2(e[2 * j], e[2 * j + 1]);
        pf16[r] = __builtin_bit_cast(f16x8, pw);
      }
#pragma unroll
      for (int c = 0; c < NW; ++c) {
        uint32_t lo4[4], hi4[4];
        transpose4(x.v[0][c], x.v[1][c], x.v[2][c], x.v[3][c], lo4);
        transpose4(x.v[4][c], x.v[5][c], x.v[6][c], x.v[7][c], hi4);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const f16x8 vf = f16_of_codes(lo4[u], hi4[u]);
#pragma unroll
          for (int r = 0; r < NR; ++r)
            o[r][4 * c + u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf, pf16[r], o[r][4 * c + u], 0, 0, 0);
        }
      }
    };

    // The wave's steps: wv, wv + 4, ...  Loads wait for what was issued before them,
    // so page numbers go out a step ahead of the keys that need them, and no load
    // depends on a branch inside the loop: a wait after one would be for both.  The
    // step computed next is not begun before they are out.
    if (wv < steps) {
      int s = wv;
      auto ahead = [&](int s) {
        __builtin_amdgcn_sched_barrier(0);
        const Pages then = load_pages(s + 4);
        const Step<D> x = load_step(s, pg);
        pg = then;
        __builtin_amdgcn_sched_barrier(0);
        return x;
      };
      Step<D> x = load_step(s, pg);
      pg = pg4;
      while (s + 8 < steps) {
        Step<D> y = ahead(s + 4);
        compute(s, x);
        x = ahead(s + 8);
        compute(s + 4, y);
        s += 8;
      }
      if (s + 4 < steps) {
        Step<D> y = ahead(s + 4);
        compute(s, x);
        s += 4;
        x = y;
      }
      compute(s, x);
      // the denominators of keys with a tiny value scale: their scores once more
      if (__builtin_expect(tiny, 0)) {
#pragma unroll 1
        for (s = wv; s < steps; s += 4) {
          const Step<D> y = load_step(s, load_pages(s));
          const int mine = base + 32 * s + 8 * g;
          const bool none = mine >= t.hi || mine + 8 <= t.lo;
          const bool few = !none && !(y.vs >= kTinyV);
          const float kq = none ? 0.0f : y.ks * a.scale_log2;
          f32x4 sc[NR][2];
          scores(y, sc);
#pragma unroll
          for (int r = 0; r < NR; ++r) {
            float e[8];
            float top = -__builtin_huge_valf();
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              e[j] = few && mine + j >= rlo[r] && mine + j < rhi[r] ? sc[r][j >> 2][j & 3] * kq : -__builtin_huge_valf();
              top = __builtin_fmaxf(top, e[j]);
            }
            if (__ballot(top > mr[r] + kDenHeadroom) != 0) {
              top = of_row(top);
              move(r, top > mr[r] + kDenHeadroom ? top - kDenTop : mr[r]);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) lr[r] += __builtin_amdgcn_exp2f(e[j] - mr[r]);
          }
        }
      }
    }

    // The next piece's lookups go out before this one's waves are joined.
    const Tile dt = c.t;
    const int dh = c.h;
    const bool whole = c.whole, more = goes_on(c);
    const int64_t piece = piece_of(c);
    record_piece(a, c);
    if (more) {
      next_item(a, R, c);
      take_piece(c);
      open_piece();
    }

    // join the four waves: row r of the group, D/16 dims a thread
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      float l = lr[r];
      l += __shfl_xor(l, 16);
      l += __shfl_xor(l, 32);
      __syncthreads();
      if (g == 0) {
        ml[wv][m16][0] = mr[r];
        ml[wv][m16][1] = l;
      }
      // lane's values: row m16, dims (4 g + i) * VW + c
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < NW; ++c)
          *reinterpret_cast<f32x4*>(&obuf[wv][m16][(4 * g + i) * VW + 4 * c]) =
              f32x4{o[r][4 * c][i], o[r][4 * c + 1][i], o[r][4 * c + 2][i], o[r][4 * c + 3][i]};
      __syncthreads();
      const int row = tid >> 4, d0 = (tid & 15) * VW;
      float top = kNoKeys;
#pragma unroll
      for (int k = 0; k < 4; ++k) top = __builtin_fmaxf(top, ml[k][row][0]);
      float sum[VW], den = 0.0f;
#pragma unroll
      for (int i = 0; i < VW; ++i) sum[i] = 0.0f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const Moved by(ml[k][row][0] - top);
        const float f = by.factor();
        den += by.den(ml[k][row][1]);
#pragma unroll
        for (int i = 0; i < VW; ++i) sum[i] = __builtin_fmaf(f, obuf[k][row][d0 + i], sum[i]);
      }
      const int tr = 16 * r + row;
      if (tr < dt.rows) {
        if (whole) store_out<VW>(a, row_token(a, dt, tr), row_head(a, dt, dh, tr), D, d0, sum, top, den);
        else store_part<VW>(a.part, R, D, piece, tr, d0, sum, top, den);
      }
    }
    if (!more) break;
  }
}

// Joins the partials of item (or of the item that worker) blockIdx.x began.
// A workgroup takes 16 / PG rows (blockIdx.y): a thread D/16 dims of a row and
// every PG-th piece, all of them in flight at once; the groups' results are
// joined through LDS in their order.  PG = 16 where a few items were shared
// among many workers, PG = 1 where pieces are few.  Bound by its launch and two
// dependent reads: 4 to 5 us for few rows (fetching the first two pieces beside the
// record, not after it, did not shorten it); 16 us and 50 MB read for 256 tiles of
// 128 rows in halves.
template <int D, int PG>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs a, int R) {
  constexpr int VW = D / 16, ROWS = 16 / PG;
  __shared__ float part[PG][ROWS][16][VW + 2];
  poison_lds<sizeof(part)>(part);
  const int tid = static_cast<int>(threadIdx.x);
  const int4* rec = reinterpret_cast<const int4*>(a.rec + static_cast<int64_t>(blockIdx.x) * 8);
  const int4 who = rec[0], what = rec[1];
  if (a.by_item) {   // a slot without rows has no record
    const int slot = static_cast<int>(blockIdx.x % static_cast<unsigned>(a.slots));
    if (tile_at(a, place_of<true>(a, slot, R), R).units == 0) return;
  }
  const int pieces = uniform(who.x), w = uniform(who.y), h = uniform(who.z);
  if (pieces == 0) return;
  Tile t;
  t.off = uniform(what.x);
  t.row0 = uniform(what.y);
  t.rows = uniform(what.z);
  const int c16 = tid & 15, lr = (tid >> 4) % ROWS, grp = (tid >> 4) / ROWS;
  const int r = static_cast<int>(blockIdx.y) * ROWS + lr, d0 = c16 * VW;
  if (static_cast<int>(blockIdx.y) * ROWS >= t.rows) return;
  const int rr = r < t.rows ? r : 0;
  const int64_t size = static_cast<int64_t>(R) * (D + 2);
  float sum[VW], top = kNoKeys, den = 0.0f;
#pragma unroll
  for (int i = 0; i < VW; ++i) sum[i] = 0.0f;
#pragma unroll 4
  for (int k = grp; k < pieces; k += PG) {
    const float* piece = a.part + (2 * static_cast<int64_t>(w + k) + (k == 0 ? 1 : 0)) * size;
    const float m = piece[R * D + 2 * rr], l = piece[R * D + 2 * rr + 1];
    const float to = __builtin_fmaxf(top, m);
    const Moved before(top - to), now(m - to);
    const float f = before.factor(), g = now.factor();
    den = before.den(den) + now.den(l);
#pragma unroll
    for (int i = 0; i < VW / 4; ++i) {
      const float4 x = *reinterpret_cast<const float4*>(piece + rr * D + d0 + 4 * i);
      sum[4 * i] = __builtin_fmaf(g, x.x, sum[4 * i] * f);
      sum[4 * i + 1] = __builtin_fmaf(g, x.y, sum[4 * i + 1] * f);
      sum[4 * i + 2] = __builtin_fmaf(g, x.z, sum[4 * i + 2] * f);
      sum[4 * i + 3] = __builtin_fmaf(g, x.w, sum[4 * i + 3] * f);
    }
    top = to;
  }
  if (PG > 1) {
    float* at = part[grp][lr][c16];
#pragma unroll
    for (int i = 0; i < VW; ++i) at[i] = sum[i];
    at[VW] = top;
    at[VW + 1] = den;
    __syncthreads();
    if (grp != 0) return;
    for (int k = 0; k < PG; ++k) top = __builtin_fmaxf(top, part[k][lr][c16][VW]);
    den = 0.0f;
#pragma unroll
    for (int i = 0; i < VW; ++i) sum[i] = 0.0f;
    for (int k = 0; k < PG; ++k) {
      const float* from = part[k][lr][c16];
      const Moved by(from[VW] - top);
      const float f = by.factor();
      den += by.den(from[VW + 1]);
#pragma unroll
      for (int i = 0; i < VW; ++i) sum[i] = __builtin_fmaf(f, from[i], sum[i]);
    }
  }
  if (r < t.rows) store_out<VW>(a, row_token(a, t, r), row_head(a, t, h, r), D, d0, sum, top, den);
}

// Launch sizes: a function of the call's sizes alone.
struct Plan {
  int R;
  int64_t slots;
  int most;
  int workers;   // 0: one item a workgroup
  int min_units;
  bool by_item;
  int64_t bytes;
};

constexpr int64_t kMaxInt = 0x7fffffff;
// Units of a context that is not worth sharing, of few rows and of many.
constexpr int64_t kBrief = 25, kManyBrief = 17;

// window: keys that a row sees at most, 0 where that is not known.
Plan plan_of(int64_t B, int64_t T, int64_t max_q, int Hq, int Hkv, int D, int64_t max_pages, int page, int64_t window) {
  Plan p;
  const int64_t G = Hq / Hkv, rows = (max_q < T ? max_q : T) * G;
  // 24 requests of 500 to 8000 tokens, heads of 128: 32 rows take 40 us in tiles of 32,
  // 53 in tiles of 16; 64 rows 61 in tiles of 32, 63 in the many-rows kernel; 96 rows
  // 87 in tiles of 32, 66 in the many-rows kernel.
  p.R = rows <= 16 ? 16 : rows <= 64 ? 32 : kManyRows;
  const int64_t most = (rows + p.R - 1) / p.R;
  const int64_t direct = most > kMaxInt / B ? kMaxInt : B * most, searched = T * G / p.R + B;
  p.most = direct <= searched ? static_cast<int>(most) : 0;
  p.slots = direct <= searched ? direct : searched;
  p.min_units = 4;
  // Workers: two a compute unit; with heads of 64 three of many rows where scales are
  // shared by 32 keys or more (7 packed prompts on pages of 32: 73 us against 79 with
  // two).  Four of few rows gave 30.4 us against 28.9 (48 requests of 99 to 4001 tokens).
  const int full = D == 64 && p.R == kManyRows && page >= 32 ? 768 : 512;
  const int64_t units = (max_pages * page + kUnit - 1) / kUnit + 1;   // of an item, at most
  const int64_t line = units + kOpen;
  const int64_t items = p.slots * Hkv;
  // Whole items where sharing them is not worth its joins, and where the line cannot
  // hold them.  Short contexts or windows: 4 requests of 1000 tokens 12.0 us against
  // 16.3 shared, 64 of 100 to 1500 20.4 against 24.3 (4 of 2000 18.9 against 15.9); a
  // prompt of 500 21.3 against 27.3 (2 pieces of 64 over 1500 45.5 against 30.5).
  // Prompts that fill the GPU once, whose tiles' work is graded and dealt from
  // the longest on: two of 2100 tokens 104 us against 129, one of 8192 621 against 660.
  // Pieces of longer contexts are as unequal as those: 80 pieces of 64 over 100 to 9000
  // tokens (1280 items) take 315 us against 269, 160 of them 507 against 511.
  const int64_t seen = window > 0 ? (window + p.R / G) / kUnit + 2 : units;
  const bool brief = (units < seen ? units : seen) <= (p.R == kManyRows ? kManyBrief : kBrief);
  const bool prompts = 2 * max_q >= max_pages * page;
  const bool many = p.R == kManyRows && items >= (prompts ? 1 : 4) * full;
  p.workers = 0;
  p.bytes = 0;
  p.by_item = false;
  if (p.slots <= kMaxSlots && !brief && !many && items <= kMaxInt / line) {
    const int64_t useful = items * ((line + p.min_units - 1) / p.min_units);
    p.workers = static_cast<int>(useful < full ? (useful + 7) / 8 * 8 : full);
    p.bytes = (2 * static_cast<int64_t>(p.workers) * p.R * (D + 2) + 8 * static_cast<int64_t>(p.workers)) * 4;
    // few items in many pieces (one request of 20000 tokens: 16.6 us against 25.4)
    p.by_item = items * 8 <= p.workers;
  }
  return p;
}

}  // namespace

int64_t attn_paged_ws(int64_t B, int64_t T, int64_t max_q, int Hq, int Hkv, int D, int64_t max_pages, int page) {
  return plan_of(B, T, max_q, Hq, Hkv, D, max_pages, page, 0).bytes;
}

hipError_t launch_attn_paged(const AttnPaged& p, hipStream_t st) {
  const Plan plan = plan_of(p.B, p.T, p.max_q, p.Hq, p.Hkv, p.D, p.max_pages, p.page, p.causal ? p.window : 0);
  AttnArgs a;
  a.p = p;
  a.G = p.Hq / p.Hkv;
  a.pshift = __builtin_ctz(static_cast<unsigned>(p.page));
  a.max_len = static_cast<int>(p.max_pages * p.page);
  a.scale_log2 = static_cast<float>(static_cast<double>(p.scale) * 1.4426950408889634);
  const int64_t blocks = plan.workers != 0 ? plan.workers : (plan.slots * p.Hkv + 7) / 8 * 8;
  if (blocks > 0x7fffffff || plan.slots > 0x7fffffff) return hipErrorInvalidValue;
  a.slots = static_cast<int>(plan.slots);
  a.most = plan.most;
  a.workers = plan.workers;
  a.min_units = plan.min_units;
  a.by_item = plan.by_item;
  a.part = static_cast<float*>(p.ws);
  a.rec = reinterpret_cast<int32_t*>(a.part + 2 * static_cast<int64_t>(plan.workers) * plan.R * (p.D + 2));
  const dim3 grid(static_cast<unsigned>(blocks)), block(256);
#define FP8BS_ROWS(D_, NR_) \
  if (p.D == D_ && plan.R == 16 * NR_) hipLaunchKernelGGL((attn_rows_kernel<D_, NR_>), grid, block, 0, st, a)
  FP8BS_ROWS(64, 1);
  FP8BS_ROWS(64, 2);
  FP8BS_ROWS(128, 1);
  FP8BS_ROWS(128, 2);
#undef FP8BS_ROWS
  const hipError_t e = plan.R == kManyRows ? launch_attn_prompt(a, static_cast<unsigned>(blocks), st) : hipGetLastError();
  if (e != hipSuccess || plan.workers == 0) return e;
  // Records are numbered, and joins shared out, by item where a few items lie in
  // many pieces each, else by the worker that began the item.
  const int64_t joins = plan.by_item ? plan.slots * p.Hkv : plan.workers;
  const bool deep = plan.by_item;
  const dim3 jgrid(static_cast<unsigned>(joins), static_cast<unsigned>(deep ? plan.R : plan.R / 16));
#define FP8BS_JOIN(D_, PG_) hipLaunchKernelGGL((attn_join_kernel<D_, PG_>), jgrid, block, 0, st, a, plan.R)
  if (p.D == 64 && deep) FP8BS_JOIN(64, 16);
  else if (p.D == 64) FP8BS_JOIN(64, 1);
  else if (deep) FP8BS_JOIN(128, 16);
  else FP8BS_JOIN(128, 1);
#undef FP8BS_JOIN
  return hipGetLastError();
}

}  // namespace fp8bs
