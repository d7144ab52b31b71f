// attn_prompt.hip -- attention over the paged E4M3 cache: many rows a
// key/value head (prompts and their pieces), on gfx950.
//
// 4 D operations a row and key against 2 D / R bytes of cache: bound by the
// matrix units at R = 128 rows a tile, with as much vector work (softmax,
// decoding) beside them.  A workgroup of four waves takes 128 rows, a wave 32
// of them; the cache goes by in tiles of 64 keys, read once a workgroup,
// decoded once (keys to BF16, values to FP16, both exact) and shared through
// two LDS buffers.  While a tile is multiplied the next one is decoded between
// the products and the one after is on its way from memory, so a tile costs
// one barrier.  Two workgroups live on a compute unit and share no barrier,
// so one's softmax runs under the other's products.
//
// Measured, heads of 128, 32 query heads on 8: a prompt of 8192 tokens 581 us, 947
// TFLOP/s (a large library product of BF16 matrices reaches 1230); two pieces of 512
// tokens 545 us with the join, 916.  Products, LDS reads and barriers alone took 367 us
// of the pieces (in the form with two groups, below): the rest is vector work that does
// not fit under the products, 7 VALU instructions a matrix instruction of 32
// cycles in a tile without a mask, 1 of them an exponential at a quarter rate.  With heads of 64
// it is 12; 7 packed prompts with a window, 74 us, 457 TFLOP/s, issue 20 over the whole
// call: an item has about 12 tiles there, and beside them its start, the filling of all
// groups, a first tile weighed twice, masked tiles at both ends and its output, none
// of it under its own products.  Also built, in us for prompt / pieces: 128 rows with decoding before the
// products 618 / 602; 256 rows on eight waves in two alternating groups 583 / 519, but
// 189 against 143 on packed prompts; one wave a SIMD with 64 rows 756 / 638; codes kept
// in LDS and decoded by each wave 643 / 568; half a tile's weights between the
// products of the other half's scores 620 / 593 (against 581 / 560 in the same run).
//
// Mathematics and number formats are those of the few-rows kernel: S^T = K Q^T
// (32x32x16 BF16 MFMAs), p' = 2^(s k c + log2 v - m) with the value scale v
// inside, O^T += V^T P'^T in FP16 on bare codes, denominator p' / v.  In the
// transposed product a lane holds 16 of 32 keys of one row, which is the order
// the second product takes its operand in, provided the values' keys are laid
// out to match: eight keys of a lane half h are 16s + 4h + 0..3 and 16s + 8 +
// 4h + 0..3.  A lane pair (l, l + 32) holds a row: one exchange a moved reference.
#include <hip/hip_runtime.h>

#include "attn_device.h"

namespace fp8bs {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));

// Instructions stay on their side of this: matrix and other work is laid out
// in the order in which it is written.
#define FP8BS_PIN() __builtin_amdgcn_sched_barrier(0)

// 16-byte chunk c of an LDS row, moved so that lanes reading the same chunk
// of 16 neighbouring rows, and the decoding writes, spread over the banks.
template <int CHUNKS>
__device__ __forceinline__ int swizzle(int row, int c) {
  return CHUNKS == 16 ? c ^ (row & 15) : c ^ ((row >> 1) & 7) ^ ((row >> 4) & 1);
}

// A group of keys that share a block: the factor of its scores, log2 and
// inverse of its value scale, its page.
struct __attribute__((aligned(16))) Group {
  float kq, lv, iv;
  int page;
};
constexpr int kInfo = 256;

// GROUP: keys that surely share a page, hence a pair of scales: a page's, 64 at most.
template <int D, int GROUP>
__global__ __launch_bounds__(256, D == 64 && GROUP >= 32 ? 3 : 2) void attn_prompt_kernel(AttnArgs a) {
  constexpr int KT = kUnit;               // keys of a tile
  constexpr int kAhead = D == 64 && GROUP >= 32 ? 2 : 4;   // LDS reads in flight before their products
  constexpr int NS = D / 16, NX = KT / 32;   // MFMA steps over the inner dim, 32-key tiles
  constexpr int ND = D / 32, NY = KT / 16;   // 32-dim tiles of the output, 16-key steps
  constexpr int NG = KT / GROUP;          // scale groups of a tile
  constexpr int VC = KT / 8;              // 16-byte chunks of a value row
  __shared__ __attribute__((aligned(16))) uint16_t kbuf[2][KT * D];
  __shared__ __attribute__((aligned(16))) uint16_t vbuf[2][D * KT];
  // factors and page of the piece's groups, kInfo at a time: read in the loop
  // by one LDS access each, where memory would cost a chain of three loads
  __shared__ Group info[kInfo];
  __shared__ int sums[4];
  static_assert(sizeof(kbuf) >= kMaxSlots * sizeof(int), "the line's prefix sums fit");
  poison_lds<sizeof(kbuf)>(kbuf);
  poison_lds<sizeof(vbuf)>(vbuf);
  poison_lds<sizeof(info)>(info);
  poison_lds<sizeof(sums)>(sums);
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 63, wv = uniform(tid >> 6);
  const int n32 = lane & 31, h2 = lane >> 5;
  const int page_mask = (1 << a.pshift) - 1;

  Cursor c;
  if (!begin_work(a, kManyRows, true, kbuf, sums, c) || !take_piece(c)) return;
  while (true) {
    const Tile& t = c.t;
    const int h = c.h;

    // the piece's keys
    const int base = (t.u0 + c.ub) * kUnit;
    const int end = base + (c.ue - c.ub) * kUnit;
    const int plo = t.lo > base ? t.lo : base, phi = t.hi < end ? t.hi : end;
    const int tiles = phi > base ? (phi - base + KT - 1) / KT : 0;
    // this wave's rows; a lane's own row is column n32
    const int wrow = 32 * wv, row = wrow + n32;
    const bool live = wrow < t.rows, there = row < t.rows;
    const int last = t.rows - 1 < wrow + 31 ? t.rows - 1 : wrow + 31;
    int rlo = 0, rhi = 0;
    if (there) row_keys(a, t, t.row0 + row, rlo, rhi);
    rhi = rhi < phi ? rhi : phi;
    // tiles b1 .. b2 - 1 hold only keys that all rows of the wave see
    int lo_last = 0, hi_first = 0;
    if (live) {
      int x;
      row_keys(a, t, t.row0 + wrow, x, hi_first);
      row_keys(a, t, t.row0 + last, lo_last, x);
    }
    hi_first = hi_first < phi ? hi_first : phi;
    const int b1 = uniform(lo_last > base ? (lo_last - base + KT - 1) / KT : 0);
    const int b2 = uniform(hi_first > base ? (hi_first - base) / KT : 0);

    bf16x8 qf[NS];
    {
      const int rr = there ? row : 0;
      const uint16_t* q = a.p.q + row_token(a, t, rr) * a.p.ldq + static_cast<int64_t>(row_head(a, t, h, rr)) * D + 8 * h2;
#pragma unroll
      for (int s = 0; s < NS; ++s)   // a row beyond the last computes row 0 and is not stored
        qf[s] = __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4*>(q + 16 * s));
    }
    f32x16 o[ND];
#pragma unroll
    for (int u = 0; u < ND; ++u)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[u][i] = 0.0f;
    float mr = kNoKeys, lr = 0.0f;

    const int32_t* table = a.p.table + t.b * a.p.ldt;
    const int last_page = static_cast<int>(a.p.max_pages) - 1;
    // Group e of the piece.  Scales of groups that no row sees may hold anything.
    auto fill_info = [&](int e) {
      const int key = base + GROUP * e, i = key >> a.pshift;
      const unsigned u = static_cast<unsigned>(table[i < last_page ? i : last_page]);
      const unsigned n = static_cast<unsigned>(a.p.n_pages) - 1u;
      Group g;
      g.page = static_cast<int>(u < n ? u : n);   // never out of range
      const int64_t blk = static_cast<int64_t>(g.page) * a.p.Hkv + h;
      const bool none = key >= phi || key + GROUP <= plo;
      const float f = a.p.ks[blk] * a.scale_log2, vs = a.p.vs[blk];
      const float v = none ? 1.0f : vs > kMinVScale ? vs : kMinVScale;
      g.kq = none ? 1.0f : f > kMinKScale ? f : kMinKScale;
      g.lv = __builtin_amdgcn_logf(v);
      g.iv = v < kTinyV ? 0.0f : __builtin_amdgcn_rcpf(v);   // tiny: summed apart
      info[e % kInfo] = g;
    };
    // Decoding: a thread takes D / 4 codes of one key, and D / 16 keys by 4 dims of
    // the values, in the order of keys that the weights come in.  A wave's keys
    // lie in one sixteen, so in one page.
    const int kkey = tid >> 2, kdim = (tid & 3) * (D / 4);
    constexpr int DQ = D / 4, RV = D / 16;
    const int dq = tid % DQ, vg = tid / DQ;   // D = 128: 8 groups of 8 keys; D = 64: 16 of 4
    const int vkey = D == 128 ? 16 * (vg >> 1) + 4 * (vg & 1) : 16 * (vg >> 2) + 8 * (vg & 1) + 4 * ((vg >> 1) & 1);
    struct Raw {
      u32x4 k[D / 64];
      uint32_t v[RV];
    };
    auto load_tile = [&](int i) {
      Raw x;
      const int page = uniform(info[((KT * i + 16 * wv) / GROUP) % kInfo].page);
      const int64_t at = (static_cast<int64_t>(page) * a.p.Hkv + h) << a.pshift;
      const int t0 = base + KT * i, tk = (t0 + kkey) & page_mask, tv = (t0 + vkey) & page_mask;
      const uint8_t* pk = a.p.kc + at * D + static_cast<unsigned>(tk * D + kdim);
      const uint8_t* pv = a.p.vc + at * D + static_cast<unsigned>(tv * D + 4 * dq);
#pragma unroll
      for (int e = 0; e < D / 64; ++e) x.k[e] = *reinterpret_cast<const u32x4*>(pk + 16 * e);
#pragma unroll
      for (int j = 0; j < RV; ++j) x.v[j] = *reinterpret_cast<const uint32_t*>(pv + (j < 4 ? j : j + 4) * D);
      return x;
    };
    // Decoding of tile i in parts: the keys' 8 codes at a time (0 .. D/32 - 1), the
    // values' bytes turned (4), then four dims (5 .. 8).
    uint32_t lo4[4], hi4[4];
    auto stage = [&](int i, const Raw& x, int part) {
      if (part < D / 32) {
        *reinterpret_cast<bf16x8*>(kbuf[i & 1] + kkey * D + 8 * swizzle<D / 8>(kkey, kdim / 8 + part)) =
            bf16_of_codes(x.k[part >> 1][2 * (part & 1)], x.k[part >> 1][2 * (part & 1) + 1]);
      } else if (part == 4) {
        transpose4(x.v[0], x.v[1], x.v[2], x.v[3], lo4);
        if (D == 128) transpose4(x.v[RV - 4], x.v[RV - 3], x.v[RV - 2], x.v[RV - 1], hi4);
      } else if (part > 4) {
        const int u = part - 5, d = 4 * dq + u;
        uint16_t* vb = vbuf[i & 1] + d * KT;
        if (D == 128) {
          *reinterpret_cast<f16x8*>(vb + 8 * swizzle<VC>(d, vg)) = f16_of_codes(lo4[u], hi4[u]);
        } else {
          const u32x4 y = __builtin_bit_cast(u32x4, f16_of_codes(lo4[u], 0u));
          *reinterpret_cast<u32x2*>(vb + 8 * swizzle<VC>(d, vg >> 1) + 4 * (vg & 1)) = u32x2{y[0], y[1]};
        }
      }
    };
    // values of keys that no row sees may hold anything: they become zeros
    auto clear_values = [&](int i, Raw& x) {
      const int t0 = base + KT * i;
      if (t0 < plo || t0 + KT > phi) {
#pragma unroll
        for (int j = 0; j < RV; ++j) {
          asm volatile("" : "+v"(x.v[j]));   // a branch: two tiles an item come here
          const int key = t0 + vkey + (j < 4 ? j : j + 4);
          if (key < plo || key >= phi) x.v[j] = 0u;
        }
      }
    };

    auto clip = [&](int i) { return i < tiles ? i : tiles - 1; };
    f32x16 sc[NX];
    f16x8 pf[NY];
    Raw x;
    // Operands are read from LDS kAhead products before their use; between the
    // products the next tile is decoded and the loads after it issued.
    constexpr int NV = NY * ND, NK = NX * NS;
    auto scores = [&](int i) {
      auto read = [&](int e) {
        const int key = 32 * (e % NX) + n32;
        return *reinterpret_cast<const bf16x8*>(kbuf[i & 1] + key * D + 8 * swizzle<D / 8>(key, 2 * (e / NX) + h2));
      };
      bf16x8 f[NK];
#pragma unroll
      for (int e = 0; e < kAhead; ++e) f[e] = read(e);
#pragma unroll
      for (int q = 0; q < NX; ++q)
#pragma unroll
        for (int j = 0; j < 16; ++j) sc[q][j] = 0.0f;
#pragma unroll
      for (int e = 0; e < NK; ++e) {
        if (e + kAhead < NK) f[e + kAhead] = read(e + kAhead);
        sc[e % NX] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f[e], qf[e / NX], sc[e % NX], 0, 0, 0);
        if (e % (NK / 4) == NK / 4 - 1) stage(i + 1, x, e / (NK / 4));
        FP8BS_PIN();
      }
    };
    auto output = [&](int i) {
      auto read = [&](int e) {
        const int d = 32 * (e % ND) + n32;
        return *reinterpret_cast<const f16x8*>(vbuf[i & 1] + d * KT + 8 * swizzle<VC>(d, 2 * (e / ND) + h2));
      };
      f16x8 f[NV];
#pragma unroll
      for (int e = 0; e < kAhead; ++e) f[e] = read(e);
#pragma unroll
      for (int e = 0; e < NV; ++e) {
        if (e + kAhead < NV) f[e + kAhead] = read(e + kAhead);
        o[e % ND] = __builtin_amdgcn_mfma_f32_32x32x16_f16(f[e], pf[e / ND], o[e % ND], 0, 0, 0);
        if (e < 5) stage(i + 1, x, 4 + e);
        if (e == 5) x = load_tile(clip(i + 2));
        FP8BS_PIN();
      }
    };
    auto move = [&](float to) {   // the reference
      const Moved by(mr - to);
      lr = by.den(lr);
      mr = to;
#pragma unroll
      for (int u = 0; u < ND; ++u)
#pragma unroll
        for (int j = 0; j < 16; ++j) o[u][j] *= by.factor();
    };
    auto softmax = [&](int i) {
      const int t0 = base + KT * i;
      float kq[NG], lv[NG];
#pragma unroll
      for (int y = 0; y < NG; ++y) {
        const Group g = info[(NG * i + y) % kInfo];
        kq[y] = g.kq;
        lv[y] = g.lv;
      }
      if (i < b1 || i >= b2) {
        const int from = rlo - t0 - 4 * h2, to = rhi - t0 - 4 * h2;
#pragma unroll
        for (int x = 0; x < NX; ++x)
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const int key = 32 * x + 8 * (j >> 2) + (j & 3);
            sc[x][j] = key >= from && key < to ? sc[x][j] : -__builtin_huge_valf();
          }
      }
      bool tiny = false;
#pragma unroll
      for (int y = 0; y < NG; ++y) tiny |= lv[y] < kTinyLog;   // the same in all lanes
      if (__builtin_expect(__ballot(tiny) != 0, 0)) {
        // one score at a time: the registers are full
        auto each = [&](auto take) {
#pragma unroll
          for (int y = 0; y < NY; ++y)
            if (__ballot(lv[16 * y / GROUP] < kTinyLog) != 0)
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                FP8BS_PIN();
                take(sc[y >> 1][8 * (y & 1) + j], kq[16 * y / GROUP]);
              }
        };
        float den;
        auto weigh = [&]() {
          float ref = mr;
          asm volatile("" : "+v"(ref));   // nothing is kept from one sum for the next
          den = 0.0f;
          each([&](float s, float k) { den += __builtin_amdgcn_exp2f(__builtin_fmaf(s, k, -ref)); });
        };
        weigh();
        if (__ballot(den > kMostDen) != 0) {
          float top = -__builtin_huge_valf();
          each([&](float s, float k) { top = __builtin_fmaxf(top, s * k); });
          den = __builtin_fmaxf(den, __shfl_xor(den, 32));   // both halves of a row move together
          top = __builtin_fmaxf(top, __shfl_xor(top, 32));
          move(den > kMostDen ? top - kDenTop : mr);
          weigh();
        }
        lr += den;
      }
      // weights under the reference as it stands; their sum shows whether it
      // still holds (no weight above 2^15), which spares the maximum
      float sum[NG];
      auto weigh = [&]() {
#pragma unroll
        for (int y = 0; y < NY; ++y) {
          const int gr = 16 * y / GROUP;
          const float off = lv[gr] - mr;
          float e[8];
#pragma unroll
          for (int j = 0; j < 8; ++j)
            e[j] = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[y >> 1][8 * (y & 1) + j], kq[gr], off));
          u32x4 pw;
#pragma unroll
          for (int j = 0; j < 4; ++j) pw[j] = pack_f16x2(e[2 * j], e[2 * j + 1]);
          pf[y] = __builtin_bit_cast(f16x8, pw);
          const float s8 = ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
          if (16 * y % GROUP == 0) sum[gr] = s8;
          else sum[gr] += s8;
        }
      };
      weigh();
      float all = sum[0];
#pragma unroll
      for (int y = 1; y < NG; ++y) all += sum[y];
      if (__builtin_expect(__ballot(all > kMostWeight) != 0, 0)) {
        float top = -__builtin_huge_valf();
#pragma unroll
        for (int y = 0; y < NY; ++y) {
          const int gr = 16 * y / GROUP;
          float m = sc[y >> 1][8 * (y & 1)];
#pragma unroll
          for (int j = 1; j < 8; ++j) m = __builtin_fmaxf(m, sc[y >> 1][8 * (y & 1) + j]);
          top = __builtin_fmaxf(top, __builtin_fmaf(m, kq[gr], lv[gr]));
        }
        all = __builtin_fmaxf(all, __shfl_xor(all, 32));   // both halves of a row move together
        top = __builtin_fmaxf(top, __shfl_xor(top, 32));
        move(all > kMostWeight ? top - kTop : mr);
        weigh();
      }
#pragma unroll
      for (int y = 0; y < NG; ++y) lr = __builtin_fmaf(sum[y], info[(NG * i + y) % kInfo].iv, lr);
    };

    if (tiles > 0) {
      // The groups are a ring of two halves; a half is filled again four tiles
      // after the last use of what it held.
      constexpr int HALF = kInfo / 2 / NG;   // tiles of a half
      __syncthreads();   // the piece before is done with the buffers
      fill_info(tid);
      __syncthreads();
      x = load_tile(0);
      {
        Raw first = x;
        x = load_tile(clip(1));
        clear_values(0, first);
#pragma unroll
        for (int e = 0; e < 9; ++e) stage(0, first, e);
      }
      __syncthreads();
      for (int i = 0; i < tiles; ++i) {
        clear_values(i + 1, x);
        // products before the other workgroup's vector work: 554 us against 570
        // (two pieces of 512 tokens)
        __builtin_amdgcn_s_setprio(1);
        scores(i);
        __builtin_amdgcn_s_setprio(0);
        softmax(i);
        __builtin_amdgcn_s_setprio(1);
        output(i);
        __builtin_amdgcn_s_setprio(0);
        if (i > HALF && i % HALF == 4 && tid < kInfo / 2) fill_info(NG * (i - 4 + HALF) + tid);
        __syncthreads();
      }
    }

    // lane pair (l, l + 32) holds row n32: dims 32 u + 8 k + 4 h2 + 0..3
    lr += __shfl_xor(lr, 32);
    int mine = wrow + n32;
    asm volatile("" : "+v"(mine));   // its token and head are found again, not kept through the loop
    if (mine < t.rows) {
      if (c.whole) {
        const float inv = lr == 0.0f ? 0.0f : 1.0f / lr;   // a NaN goes on
        const int64_t token = row_token(a, t, mine);
        const int head = row_head(a, t, h, mine);
        uint16_t* at = a.p.out + token * a.p.ldo + static_cast<int64_t>(head) * D + 4 * h2;
#pragma unroll
        for (int u = 0; u < ND; ++u)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            *reinterpret_cast<uint2*>(at + 32 * u + 8 * k) =
                make_uint2(pack_bf16x2_rne(o[u][4 * k] * inv, o[u][4 * k + 1] * inv),
                           pack_bf16x2_rne(o[u][4 * k + 2] * inv, o[u][4 * k + 3] * inv));
        if (h2 == 0 && a.p.lse != nullptr)
          a.p.lse[token * a.p.ldl + head] =
              lr == 0.0f ? -__builtin_huge_valf() : (mr + __builtin_amdgcn_logf(lr)) * 0.693147180559945f;
      } else {
        float* at = a.part + piece_of(c) * kManyRows * (D + 2);
#pragma unroll
        for (int u = 0; u < ND; ++u)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            *reinterpret_cast<float4*>(at + mine * D + 32 * u + 8 * k + 4 * h2) =
                make_float4(o[u][4 * k], o[u][4 * k + 1], o[u][4 * k + 2], o[u][4 * k + 3]);
        if (h2 == 0) {
          at[kManyRows * D + 2 * mine] = mr;
          at[kManyRows * D + 2 * mine + 1] = lr;
        }
      }
    }
    record_piece(a, c);
    if (!goes_on(c)) break;
    next_item(a, kManyRows, c);
    take_piece(c);
  }
}

}  // namespace

hipError_t launch_attn_prompt(const AttnArgs& a, unsigned blocks, hipStream_t st) {
  const dim3 grid(blocks), block(256);
#define FP8BS_PROMPT(D_, G_) hipLaunchKernelGGL((attn_prompt_kernel<D_, G_>), grid, block, 0, st, a)
  if (a.p.D == 64 && a.p.page >= 64) FP8BS_PROMPT(64, 64);
  else if (a.p.D == 64 && a.p.page == 32) FP8BS_PROMPT(64, 32);
  else if (a.p.D == 64) FP8BS_PROMPT(64, 16);
  else if (a.p.page >= 64) FP8BS_PROMPT(128, 64);
  else if (a.p.page == 32) FP8BS_PROMPT(128, 32);
  else FP8BS_PROMPT(128, 16);
#undef FP8BS_PROMPT
  return hipGetLastError();
}

}  // namespace fp8bs
