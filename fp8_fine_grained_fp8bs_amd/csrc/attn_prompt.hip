// attn_prompt.hip -- attention over the paged E4M3 cache: many rows a
// key/value head (prompts and their pieces), on gfx950.
//
// 4 D operations a row and key against 2 D / R bytes of cache: bound by the
// matrix units at R = 128 rows a tile, with the softmax's vector work beside
// them.  A workgroup of four waves takes 128 rows, a wave 32 of them; the cache
// goes by in tiles of 64 keys, read once a workgroup, decoded once (keys to
// BF16, values to FP16, both exact) and shared through LDS.  Two LDS buffers:
// while a tile is computed the next one is decoded into the other buffer and
// the one after is on its way from memory in registers, so a tile costs one
// barrier.  Two workgroups live on a compute unit; their waves share the SIMDs
// without a common barrier, so one's softmax runs under the other's MFMAs.
//
// Mathematics and number formats are those of the few-rows kernel: S^T = K Q^T
// (32x32x16 BF16 MFMAs), p' = 2^(s k c + log2 v - m) with the value scale v
// inside, O^T += V^T P'^T in FP16 on bare codes, denominator p' / v.  In the
// transposed product a lane holds 16 of 32 keys of one row, which is the order
// the second product takes its operand in, provided the values' keys are laid
// out to match: eight keys of a lane half h are 16s + 4h + 0..3 and 16s + 8 +
// 4h + 0..3.  A lane pair (l, l + 32) holds a row: one exchange a moved reference.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "attn_device.h"

namespace fp8bs {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kRows = 128;

// 16-byte chunk c of an LDS row, moved so that lanes reading the same chunk
// of 16 neighbouring rows, and the decoding writes, spread over the banks.
template <int CHUNKS>
__device__ __forceinline__ int swizzle(int row, int c) {
  return CHUNKS == 16 ? c ^ (row & 15) : c ^ ((row >> 1) & 7) ^ ((row >> 4) & 1);
}

template <int D>
struct Raw {           // a thread's share of a tile on its way
  u32x4 k[D / 64];     // 16 D/64 codes of key tid / 4
  uint32_t v[D / 16];  // D/16 keys by 4 dims
  float ks, vs;        // the tile's scales, or in the first wave those of keys 16 (lane % 4)
};

// PAGE64: a page holds whole tiles (64 or 128 tokens), so a tile has one block,
// one pair of scales, and its addresses are scalar; else a tile's sixteens of
// keys each have their own.
template <int D, bool PAGE64>
__global__ __launch_bounds__(256, 2) void attn_prompt_kernel(AttnArgs a) {
  constexpr int NG = PAGE64 ? 1 : 4;      // scale groups of a tile
  constexpr int kAhead = PAGE64 ? 4 : 2;  // LDS reads in flight before their products (four spill with four groups)
  constexpr int NS = D / 16;   // MFMA steps over the inner dim
  constexpr int ND = D / 32;   // 32-dim tiles of the output
  __shared__ __attribute__((aligned(16))) uint16_t kbuf[2][kUnit * D];
  __shared__ __attribute__((aligned(16))) uint16_t vbuf[2][D * kUnit];
  __shared__ float scales[2][4][4];   // key scale, log2 and inverse of the value scale, of 16 keys
  __shared__ int sums[4];
  static_assert(sizeof(kbuf) >= kMaxSlots * sizeof(int), "the line's prefix sums fit");
  poison_lds<sizeof(kbuf)>(kbuf);
  poison_lds<sizeof(vbuf)>(vbuf);
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 63, wv = uniform(tid >> 6);
  const int n32 = lane & 31, h2 = lane >> 5;
  const int page_mask = (1 << a.pshift) - 1;

  Cursor c;
  if (!begin_work(a, kRows, true, kbuf, sums, c)) return;
  while (c.cur < c.stop) {
    take_piece(c);
    const Tile& t = c.t;
    const int h = c.h;

    // this wave's rows; a lane's own row is column n32
    const int wrow = 32 * wv, row = wrow + n32;
    const bool live = wrow < t.rows, there = row < t.rows;
    const int last = t.rows - 1 < wrow + 31 ? t.rows - 1 : wrow + 31;
    int rlo = 0, rhi = 0;
    if (there) row_keys(a, t, t.row0 + row, rlo, rhi);
    int wlo_first = 0, whi_first = 0, wlo_last = 0, whi_last = 0;   // of the wave's first and last row
    if (live) {
      row_keys(a, t, t.row0 + wrow, wlo_first, whi_first);
      row_keys(a, t, t.row0 + last, wlo_last, whi_last);
    }
    bf16x8 qf[NS];
    {
      const int rr = there ? row : 0;
      const uint16_t* q = a.p.q + row_token(a, t, rr) * a.p.ldq + static_cast<int64_t>(row_head(a, t, h, rr)) * D + 8 * h2;
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        const u32x4 zero = {0u, 0u, 0u, 0u};
        const u32x4 x = *reinterpret_cast<const u32x4*>(q + 16 * s);
        qf[s] = __builtin_bit_cast(bf16x8, there ? x : zero);
      }
    }
    f32x16 o[ND];
#pragma unroll
    for (int u = 0; u < ND; ++u)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[u][i] = 0.0f;
    float mr = kNoKeys, lr = 0.0f;

    const int32_t* table = a.p.table + t.b * a.p.ldt;
    const int last_page = static_cast<int>(a.p.max_pages) - 1;
    const int base = (t.u0 + c.ub) * kUnit;
    const int tiles = t.hi > base ? c.ue - c.ub : 0;
    auto page_at = [&](int key) {   // the table's entry for a key's page, never past the table
      const int i = key >> a.pshift;
      return table[i < last_page ? i : last_page];
    };
    auto block_of = [&](int id) {   // never out of range
      const unsigned u = static_cast<unsigned>(id), n = static_cast<unsigned>(a.p.n_pages) - 1u;
      return static_cast<int64_t>(u < n ? u : n) * a.p.Hkv + h;
    };
    // a thread's keys: one for the key tile; for the value tile those whose
    // products a lane half takes together
    const int kkey = tid >> 2, kdim = (tid & 3) * (D / 4);
    constexpr int DQ = D / 4;                 // groups of 4 dims
    const int dq = tid % DQ, vg = tid / DQ;   // D = 128: 8 groups of 8 keys; D = 64: 16 of 4
    const int vkey = D == 128 ? 16 * (vg >> 1) + 4 * (vg & 1) : 16 * (vg >> 2) + 4 * (vg & 1) + 8 * ((vg >> 1) & 1);
    struct Pages {
      int k, v, s;
    };
    auto load_pages = [&](int i) {
      const int t0 = base + kUnit * i;
      if (PAGE64) {
        const int id = page_at(t0);   // made scalar where it is used: that waits for the load
        return Pages{id, id, id};
      }
      return Pages{page_at(t0 + kkey), page_at(t0 + vkey), page_at(t0 + 16 * (lane & 3))};
    };
    auto load_tile = [&](int i, const Pages& pg) {
      Raw<D> x;
      const int t0 = base + kUnit * i;
      const uint8_t *pk, *pv;
      if (PAGE64) {
        const int64_t blk = block_of(uniform(pg.k)), at = ((blk << a.pshift) + (t0 & page_mask)) * D;
        pk = a.p.kc + at + static_cast<unsigned>(kkey * D + kdim);
        pv = a.p.vc + at + static_cast<unsigned>(vkey * D + 4 * dq);
      } else {
        pk = a.p.kc + ((block_of(pg.k) << a.pshift) + ((t0 + kkey) & page_mask)) * D + kdim;
        pv = a.p.vc + ((block_of(pg.v) << a.pshift) + ((t0 + vkey) & page_mask)) * D + 4 * dq;
      }
#pragma unroll
      for (int c = 0; c < D / 64; ++c) x.k[c] = *reinterpret_cast<const u32x4*>(pk + 16 * c);
#pragma unroll
      for (int j = 0; j < D / 16; ++j) x.v[j] = *reinterpret_cast<const uint32_t*>(pv + (j < 4 ? j : j + 4) * D);
      if (PAGE64 || wv == 0) {
        const int64_t blk = block_of(PAGE64 ? uniform(pg.k) : pg.s);
        x.ks = a.p.ks[blk];
        x.vs = a.p.vs[blk];
      }
      return x;
    };
    // factors of a block: of its scores, log2 and inverse of its value scale;
    // `none`: keys that no row sees, whose scales may hold anything
    auto set_factors = [&](float ks, float vs, bool none, float& kq, float& lv, float& iv) {
      const float f = ks * a.scale_log2, v = none ? 1.0f : vs > kMinVScale ? vs : kMinVScale;
      kq = none ? 1.0f : f > kMinKScale ? f : kMinKScale;
      lv = __builtin_amdgcn_logf(v);
      iv = __builtin_amdgcn_rcpf(v);
    };
    float next_kq = 0.0f, next_lv = 0.0f, next_iv = 0.0f;
    auto stage = [&](int i, Raw<D>& x) {
      const int buf = i & 1, t0 = base + kUnit * i;
      uint16_t* kb = kbuf[buf] + kkey * D;
      constexpr int C = D / 8;
#pragma unroll
      for (int c = 0; c < D / 64; ++c)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          *reinterpret_cast<bf16x8*>(kb + 8 * swizzle<C>(kkey, kdim / 8 + 2 * c + e)) =
              bf16_of_codes(x.k[c][2 * e], x.k[c][2 * e + 1]);
      if (t0 < t.lo || t0 + kUnit > t.hi) {   // keys that no row sees may hold anything
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
          asm volatile("" : "+v"(x.v[j]));    // a branch: two tiles an item come here
          const int key = t0 + vkey + (j < 4 ? j : j + 4);
          if (key < t.lo || key >= t.hi) x.v[j] = 0u;
        }
      }
      uint32_t lo4[4], hi4[4];
      transpose4(x.v[0], x.v[1], x.v[2], x.v[3], lo4);
      if (D == 128) transpose4(x.v[D / 16 - 4], x.v[D / 16 - 3], x.v[D / 16 - 2], x.v[D / 16 - 1], hi4);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int d = 4 * dq + u;
        if (D == 128) {
          *reinterpret_cast<f16x8*>(vbuf[buf] + d * kUnit + 8 * swizzle<8>(d, vg)) = f16_of_codes(lo4[u], hi4[u]);
        } else {
          const f16x8 x8 = f16_of_codes(lo4[u], 0u);
          const u32x4 y = __builtin_bit_cast(u32x4, x8);
          // chunk (16-key step, half), its first or second four keys
          *reinterpret_cast<u32x2*>(vbuf[buf] + d * kUnit + 8 * swizzle<8>(d, 2 * (vg >> 2) + (vg & 1)) +
                                    4 * ((vg >> 1) & 1)) = u32x2{y[0], y[1]};
        }
      }
      if (PAGE64) {   // the tile's factors wait in registers for their turn
        set_factors(x.ks, x.vs, false, next_kq, next_lv, next_iv);
      } else if (tid < 4) {
        const int key = t0 + 16 * tid;
        set_factors(x.ks, x.vs, key >= t.hi || key + 16 <= t.lo, scales[buf][tid][0], scales[buf][tid][1],
                    scales[buf][tid][2]);
      }
    };
    // MASK: some row of the wave does not see all keys of the tile
    auto compute = [&](int i, auto mask, float kq1, float lv1, float iv1) {
      constexpr bool MASK = decltype(mask)::value;
      const int buf = i & 1, t0 = base + kUnit * i;
      f32x16 sc[2];
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int j = 0; j < 16; ++j) sc[x][j] = 0.0f;
      // operands are read from LDS kAhead products before they are used
      {
        bf16x8 kf[2 * NS];
        auto read = [&](int e) {
          const int key = 32 * (e & 1) + n32;
          kf[e] = *reinterpret_cast<const bf16x8*>(kbuf[buf] + key * D + 8 * swizzle<D / 8>(key, 2 * (e >> 1) + h2));
        };
#pragma unroll
        for (int e = 0; e < kAhead; ++e) read(e);
#pragma unroll
        for (int e = 0; e < 2 * NS; ++e) {
          if (e + kAhead < 2 * NS) read(e + kAhead);
          sc[e & 1] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf[e], qf[e >> 1], sc[e & 1], 0, 0, 0);
        }
        __builtin_amdgcn_sched_group_barrier(0x100, kAhead, 0);
#pragma unroll
        for (int e = 0; e < 2 * NS - kAhead; ++e) {
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        }
        __builtin_amdgcn_sched_group_barrier(0x008, kAhead, 0);
      }
      float kq[NG], lv[NG], iv[NG];
      if (PAGE64) {
        kq[0] = kq1;
        lv[0] = lv1;
        iv[0] = iv1;
      } else {
#pragma unroll
        for (int y = 0; y < NG; ++y) {
          kq[y] = scales[buf][y][0];
          lv[y] = scales[buf][y][1];
          iv[y] = scales[buf][y][2];
        }
      }
      if (MASK) {
        const int from = rlo - t0 - 4 * h2, to = rhi - t0 - 4 * h2;
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const int key = 32 * x + 8 * (j >> 2) + (j & 3);
            sc[x][j] = key >= from && key < to ? sc[x][j] : -__builtin_huge_valf();
          }
      }
      // weights under the reference as it stands; their sum shows whether it
      // still holds (no weight above 2^15), which spares the maximum
      f16x8 pf[4];
      float sum[NG];
      auto weigh = [&]() {
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const int gr = PAGE64 ? 0 : y;
          const float c = lv[gr] - mr;
          float e[8];
#pragma unroll
          for (int j = 0; j < 8; ++j)
            e[j] = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[y >> 1][8 * (y & 1) + j], kq[gr], c));
          u32x4 pw;
#pragma unroll
          for (int j = 0; j < 4; ++j) pw[j] = pack_f16x2(e[2 * j], e[2 * j + 1]);
          pf[y] = __builtin_bit_cast(f16x8, pw);
          const float s8 = ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
          if (PAGE64 && y > 0) sum[0] += s8;
          else sum[gr] = s8;
        }
      };
      weigh();
      float all = sum[0];
#pragma unroll
      for (int y = 1; y < NG; ++y) all += sum[y];
      if (__builtin_expect(__ballot(all > kMostWeight) != 0, 0)) {
        float top = -__builtin_huge_valf();
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const int gr = PAGE64 ? 0 : y;
          float m = sc[y >> 1][8 * (y & 1)];
#pragma unroll
          for (int j = 1; j < 8; ++j) m = __builtin_fmaxf(m, sc[y >> 1][8 * (y & 1) + j]);
          top = __builtin_fmaxf(top, __builtin_fmaf(m, kq[gr], lv[gr]));
        }
        all = __builtin_fmaxf(all, __shfl_xor(all, 32));   // both halves of a row move together
        top = __builtin_fmaxf(top, __shfl_xor(top, 32));
        const float to = all > kMostWeight ? top - kTop : mr;
        const float f = __builtin_amdgcn_exp2f(mr - to);
        mr = to;
        lr *= f;
#pragma unroll
        for (int u = 0; u < ND; ++u)
#pragma unroll
          for (int j = 0; j < 16; ++j) o[u][j] *= f;
        weigh();
      }
#pragma unroll
      for (int y = 0; y < NG; ++y) lr = __builtin_fmaf(sum[y], iv[y], lr);
      {
        f16x8 vf[4 * ND];
        auto read = [&](int e) {
          const int d = 32 * (e % ND) + n32;
          vf[e] = *reinterpret_cast<const f16x8*>(vbuf[buf] + d * kUnit + 8 * swizzle<8>(d, 2 * (e / ND) + h2));
        };
#pragma unroll
        for (int e = 0; e < kAhead; ++e) read(e);
#pragma unroll
        for (int e = 0; e < 4 * ND; ++e) {
          if (e + kAhead < 4 * ND) read(e + kAhead);
          o[e % ND] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vf[e], pf[e / ND], o[e % ND], 0, 0, 0);
        }
        __builtin_amdgcn_sched_group_barrier(0x100, kAhead, 1);
#pragma unroll
        for (int e = 0; e < 4 * ND - kAhead; ++e) {
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 1);
          __builtin_amdgcn_sched_group_barrier(0x100, 1, 1);
        }
        __builtin_amdgcn_sched_group_barrier(0x008, kAhead, 1);
      }
    };

    if (tiles > 0) {
      // the wave's way through the tiles: none of its rows sees the first and
      // last ones, all rows see all of the middle ones; masks between
      auto tile_floor = [&](int key) { const int x = (key - base) >> 6; return x < 0 ? 0 : x > tiles ? tiles : x; };
      int b0 = tile_floor(wlo_first), b3 = tile_floor(whi_last + kUnit - 1);
      if (!live || b3 < b0) b0 = b3 = tiles;
      int b1 = tile_floor(wlo_last + kUnit - 1), b2 = tile_floor(whi_first);
      b1 = b1 < b0 ? b0 : b1 > b3 ? b3 : b1;
      b2 = b2 < b1 ? b1 : b2 > b3 ? b3 : b2;
      // on their way: the next tile's codes, and the page numbers of the one after
      Pages pg = load_pages(0), next = load_pages(tiles > 1 ? 1 : 0);
      Raw<D> x = load_tile(0, pg);
      pg = load_pages(tiles > 2 ? 2 : 0);
      __syncthreads();   // the piece before is done with the buffers
      stage(0, x);
      x = load_tile(tiles > 1 ? 1 : 0, next);
      __syncthreads();
      auto run = [&](int from, int to, auto kind) {
        for (int i = from; i < to; ++i) {
          const float kq = next_kq, lv = next_lv, iv = next_iv;
          if (i + 1 < tiles) {
            stage(i + 1, x);
            if (i + 2 < tiles) {
              x = load_tile(i + 2, pg);
              if (i + 3 < tiles) pg = load_pages(i + 3);
            }
          }
          if constexpr (decltype(kind)::value == 1) compute(i, std::true_type{}, kq, lv, iv);
          if constexpr (decltype(kind)::value == 2) compute(i, std::false_type{}, kq, lv, iv);
          __syncthreads();
        }
      };
      run(0, b0, std::integral_constant<int, 0>{});
      run(b0, b1, std::integral_constant<int, 1>{});
      run(b1, b2, std::integral_constant<int, 2>{});
      run(b2, b3, std::integral_constant<int, 1>{});
      run(b3, tiles, std::integral_constant<int, 0>{});
    }

    // lane pair (l, l + 32) holds row n32: dims 32 u + 8 k + 4 h2 + 0..3
    lr += __shfl_xor(lr, 32);
    if (there) {
      if (c.whole) {
        const float inv = lr > 0.0f ? 1.0f / lr : 0.0f;
        const int64_t token = row_token(a, t, row);
        const int head = row_head(a, t, h, row);
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
              lr > 0.0f ? (mr + __builtin_amdgcn_logf(lr)) * 0.693147180559945f : -__builtin_huge_valf();
      } else {
        float* at = a.part + piece_of(c) * kRows * (D + 2);
#pragma unroll
        for (int u = 0; u < ND; ++u)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            *reinterpret_cast<float4*>(at + row * D + 32 * u + 8 * k + 4 * h2) =
                make_float4(o[u][4 * k], o[u][4 * k + 1], o[u][4 * k + 2], o[u][4 * k + 3]);
        if (h2 == 0) {
          at[kRows * D + 2 * row] = mr;
          at[kRows * D + 2 * row + 1] = lr;
        }
      }
    }
    end_piece(a, kRows, c);
  }
}

}  // namespace

hipError_t launch_attn_prompt(const AttnArgs& a, unsigned blocks, hipStream_t st) {
  const dim3 grid(blocks), block(256);
  const bool page64 = a.p.page >= kUnit;
  if (a.p.D == 64 && page64) hipLaunchKernelGGL((attn_prompt_kernel<64, true>), grid, block, 0, st, a);
  else if (a.p.D == 64) hipLaunchKernelGGL((attn_prompt_kernel<64, false>), grid, block, 0, st, a);
  else if (page64) hipLaunchKernelGGL((attn_prompt_kernel<128, true>), grid, block, 0, st, a);
  else hipLaunchKernelGGL((attn_prompt_kernel<128, false>), grid, block, 0, st, a);
  return hipGetLastError();
}

}  // namespace fp8bs
