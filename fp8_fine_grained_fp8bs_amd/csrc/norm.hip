// norm.hip -- the root-mean-square norm with the residual's addition and the
// 1x128 quantization of its output, and its gradient (gfx950).
//
//   h = bf16(x + r), rstd = 1 / sqrt(mean h^2 + eps), n = h rstd gamma
//
// n leaves as E4M3 codes with 1x128 scales, the A operand of the projections
// that follow, and optionally in BF16.  The norm is that of the stored h, so
// that its gradient, which reads h, is the gradient of what was computed.
// With a = gamma dn and u = h rstd the gradient is
//   dx = dres + rstd (a - u mean(a u)),   dgamma = sum over the rows of dn u.
// Both move a few bytes a value for about ten operations: HBM-bound.  A row is
// read once and stays in registers between its sum and its output.
#include <hip/hip_runtime.h>

#include "fp8bs_device.h"
#include "fp8bs_internal.h"

namespace fp8bs {
namespace {

constexpr int kMaxWaves = 16;   // waves of a row

// A row's sum over its waves, each with its lanes' v, in the order of the
// waves.  part: kMaxWaves floats of LDS that no wave still reads.
__device__ __forceinline__ float row_sum(float v, float* part, int waves, int wave) {
  v = wave_sum(v);
  if (waves == 1) return v;
  if ((threadIdx.x & 63) == 0) part[wave] = v;
  __syncthreads();
  float s = part[0];
  for (int w = 1; w < waves; ++w) s += part[w];
  return s;
}

__device__ __forceinline__ void load_gamma(const void* gamma, bool f32, int c, float (&g)[8]) {
  if (f32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(gamma) + c);
    const float4 a = p[0], b = p[1];
    g[0] = a.x; g[1] = a.y; g[2] = a.z; g[3] = a.w;
    g[4] = b.x; g[5] = b.y; g[6] = b.z; g[7] = b.w;
  } else {
    bf16x8_unpack(*reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(gamma) + c), g);
  }
}

__device__ __forceinline__ u32x4 load_nt(const uint16_t* p) {
  return __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
}

// `waves` waves a row, V vectors of 8 values a lane; with one wave a row a
// workgroup has four rows.  x, r and h may be the same buffer: a lane reads
// its own values before it writes them.
template <int V>
__global__ __launch_bounds__(1024) void rmsnorm_kernel(RmsNorm p, int waves) {
  __shared__ float part[kMaxWaves];
  poison_lds<sizeof(part)>(part);
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t row = waves == 1 ? static_cast<int64_t>(blockIdx.x) * 4 + w : blockIdx.x;
  if (row >= p.T) return;
  const int wave = waves == 1 ? 0 : w;
  const int C = p.C;
  u32x4 h[V];
  float ss = 0.0f;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = ((v * waves + wave) * 64 + lane) * 8;
    h[v] = c < C ? load_nt(p.x + row * p.ldx + c) : u32x4{0u, 0u, 0u, 0u};
  }
  if (p.r != nullptr) {
    u32x4 r[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = ((v * waves + wave) * 64 + lane) * 8;
      r[v] = c < C ? load_nt(p.r + row * p.ldr + c) : u32x4{0u, 0u, 0u, 0u};
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = ((v * waves + wave) * 64 + lane) * 8;
      float a[8], b[8];
      bf16x8_unpack(h[v], a);
      bf16x8_unpack(r[v], b);
#pragma unroll
      for (int i = 0; i < 8; ++i) a[i] += b[i];
      h[v] = bf16x8_pack(a);
      if (c < C) *reinterpret_cast<u32x4*>(p.h + row * p.ldh + c) = h[v];
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    float a[8];
    bf16x8_unpack(h[v], a);
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = __builtin_fmaf(a[i], a[i], ss);
  }
  ss = row_sum(ss, part, waves, wave);
  const float rstd = 1.0f / __builtin_sqrtf(ss / static_cast<float>(C) + p.eps);
  if (p.rstd != nullptr && wave == 0 && lane == 0) p.rstd[row] = rstd;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = ((v * waves + wave) * 64 + lane) * 8;
    float n[8], g[8];
    bf16x8_unpack(h[v], n);
    const bool in = c < C;   // the same in all lanes of a tile: C is whole tiles
    load_gamma(p.gamma, p.gamma_f32, in ? c : 0, g);
#pragma unroll
    for (int i = 0; i < 8; ++i) n[i] = (n[i] * rstd) * g[i];
    if (p.q != nullptr) {
      float am = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) am = __builtin_fmaxf(am, __builtin_fabsf(n[i]));
      am = row16_max(am);
      const TileScale ts = make_tile_scale(am);
      const uint2 code = make_uint2(encode4(n, ts), encode4(n + 4, ts));
      if (in) {
        *reinterpret_cast<uint2*>(p.q + row * p.ldq + c) = code;
        if ((lane & 15) == 0) p.s[row * p.lds + (c >> 7)] = ts.s;
      }
    }
    if (p.y != nullptr && in) *reinterpret_cast<u32x4*>(p.y + row * p.ldy + c) = bf16x8_pack(n);
  }
}

// One row's values of a lane.
template <int V>
struct BwdRow {
  u32x4 h[V], dn[V], dres[V];
  float rstd;
};

template <int V>
__device__ __forceinline__ void bwd_load(const RmsNormBwd& p, int64_t row, int waves, int wave, int lane, BwdRow<V>& b) {
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = ((v * waves + wave) * 64 + lane) * 8;
    const bool in = c < p.C;
    b.h[v] = in ? load_nt(p.h + row * p.ldh + c) : u32x4{0u, 0u, 0u, 0u};
    b.dn[v] = in ? load_nt(p.dn + row * p.lddn + c) : u32x4{0u, 0u, 0u, 0u};
    b.dres[v] = in && p.dres != nullptr ? load_nt(p.dres + row * p.lddr + c) : u32x4{0u, 0u, 0u, 0u};
  }
  b.rstd = p.rstd[row];
}

// A worker (a workgroup, or one of its waves with one wave a row) walks the
// rows first, first + workers, ..., loading the next while it computes one
// (AHEAD: where the registers are enough), and keeps its part of dgamma in registers; the parts are summed by
// dgamma_kernel in the order of the workers.  dx may be h, dn or dres.
template <int V, bool AHEAD>
__global__ __launch_bounds__(1024) void rmsnorm_bwd_kernel(RmsNormBwd p, int waves, int64_t workers) {
  __shared__ float part[2][kMaxWaves];
  poison_lds<sizeof(part)>(part);
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t worker = waves == 1 ? static_cast<int64_t>(blockIdx.x) * 4 + w : blockIdx.x;
  if (worker >= workers) return;
  const int wave = waves == 1 ? 0 : w;
  const float inv = 1.0f / static_cast<float>(p.C);
  float held[V][8], acc[V][8];   // gamma's part, kept only with AHEAD
  const auto gamma_of = [&](int v, float (&g)[8]) {
    const int c = ((v * waves + wave) * 64 + lane) * 8;
    load_gamma(p.gamma, p.gamma_f32, c < p.C ? c : 0, g);
  };
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if (AHEAD) gamma_of(v, held[v]);
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[v][i] = 0.0f;
  }
  int turn = 0;
  auto compute = [&](int64_t row, const BwdRow<V>& b) {
    float dot = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float h[8], dn[8], g[8];
      bf16x8_unpack(b.h[v], h);
      bf16x8_unpack(b.dn[v], dn);
      if (!AHEAD) gamma_of(v, g);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float u = h[i] * b.rstd;
        dot = __builtin_fmaf((AHEAD ? held[v][i] : g[i]) * dn[i], u, dot);
        acc[v][i] = __builtin_fmaf(dn[i], u, acc[v][i]);
      }
    }
    const float mean = row_sum(dot, part[turn], waves, wave) * inv;
    turn ^= 1;   // the next row's sum goes elsewhere: one barrier a row
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = ((v * waves + wave) * 64 + lane) * 8;
      float h[8], dn[8], dr[8], g[8];
      if (!AHEAD) gamma_of(v, g);
      bf16x8_unpack(b.h[v], h);
      bf16x8_unpack(b.dn[v], dn);
      bf16x8_unpack(b.dres[v], dr);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float a = (AHEAD ? held[v][i] : g[i]) * dn[i];
        dr[i] = __builtin_fmaf(b.rstd, __builtin_fmaf(-(h[i] * b.rstd), mean, a), dr[i]);
      }
      if (c < p.C) *reinterpret_cast<u32x4*>(p.dx + row * p.lddx + c) = bf16x8_pack(dr);
    }
  };
  BwdRow<V> a, b;
  int64_t row = worker;
  if (!AHEAD) {
    for (; row < p.T; row += workers) {
      bwd_load<V>(p, row, waves, wave, lane, a);
      compute(row, a);
    }
  }
  if (AHEAD) bwd_load<V>(p, row, waves, wave, lane, a);
  for (; AHEAD && row < p.T; row += 2 * workers) {
    const int64_t row2 = row + workers, row3 = row2 + workers;
    if (row2 < p.T) bwd_load<V>(p, row2, waves, wave, lane, b);
    compute(row, a);
    if (row3 < p.T) bwd_load<V>(p, row3, waves, wave, lane, a);
    if (row2 < p.T) compute(row2, b);
  }
  if (p.dgamma != nullptr) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = ((v * waves + wave) * 64 + lane) * 8;
      if (c >= p.C) continue;
      float4* out = reinterpret_cast<float4*>(p.ws + worker * p.C + c);
      out[0] = make_float4(acc[v][0], acc[v][1], acc[v][2], acc[v][3]);
      out[1] = make_float4(acc[v][4], acc[v][5], acc[v][6], acc[v][7]);
    }
  }
}

// dgamma of 32 columns: 32 groups of 8 lanes take every 32nd worker's part,
// joined through LDS in the order of the groups.
__global__ __launch_bounds__(256) void dgamma_kernel(const float* __restrict__ parts, int64_t workers, int C,
                                                     float* __restrict__ dgamma) {
  __shared__ float4 sums[32][8];
  poison_lds<sizeof(sums)>(sums);
  const int sub = threadIdx.x & 7, group = threadIdx.x >> 3;
  const int c = blockIdx.x * 32 + sub * 4;
  float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
  for (int64_t w = group; w < workers; w += 32) {
    const float4 a = *reinterpret_cast<const float4*>(parts + w * C + c);
    s.x += a.x; s.y += a.y; s.z += a.z; s.w += a.w;
  }
  sums[group][sub] = s;
  __syncthreads();
  if (threadIdx.x < 8) {
    s = sums[0][sub];
    for (int k = 1; k < 32; ++k) {
      const float4 a = sums[k][sub];
      s.x += a.x; s.y += a.y; s.z += a.z; s.w += a.w;
    }
    *reinterpret_cast<float4*>(dgamma + c) = s;
  }
}

// Vectors a lane and waves a row.
struct RowShape {
  int V, waves;
};
RowShape row_shape(int C) {
  const int vectors = C / 8;
  const int V = vectors <= 64 * kMaxWaves ? 1 : 2;
  return {V, (vectors + 64 * V - 1) / (64 * V)};
}

// Workers of the gradient: at most as many rows in flight as two workgroups a
// compute unit give.
int64_t bwd_workers(int64_t T, const RowShape& r) {
  const int64_t most = r.waves == 1 ? 4096 : 512;
  return T < most ? T : most;
}

}  // namespace

hipError_t launch_rmsnorm(const RmsNorm& p, hipStream_t st) {
  const RowShape r = row_shape(p.C);
  const int64_t blocks = r.waves == 1 ? (p.T + 3) / 4 : p.T;
  if (blocks > 0x7fffffff) return hipErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(blocks)), block(r.waves == 1 ? 256 : 64 * r.waves);
  if (r.V == 1) hipLaunchKernelGGL((rmsnorm_kernel<1>), grid, block, 0, st, p, r.waves);
  else hipLaunchKernelGGL((rmsnorm_kernel<2>), grid, block, 0, st, p, r.waves);
  return hipGetLastError();
}

int64_t rmsnorm_bwd_ws(int64_t T, int C) {
  return bwd_workers(T, row_shape(C)) * C * static_cast<int64_t>(sizeof(float));
}

hipError_t launch_rmsnorm_bwd(const RmsNormBwd& p, hipStream_t st) {
  const RowShape r = row_shape(p.C);
  const int64_t workers = bwd_workers(p.T, r);
  const dim3 grid(static_cast<unsigned>(r.waves == 1 ? (workers + 3) / 4 : workers));
  const dim3 block(r.waves == 1 ? 256 : 64 * r.waves);
  if (workers == 0) {}   // dgamma alone, a sum of nothing
  else if (r.V == 1) hipLaunchKernelGGL((rmsnorm_bwd_kernel<1, true>), grid, block, 0, st, p, r.waves, workers);
  else hipLaunchKernelGGL((rmsnorm_bwd_kernel<2, false>), grid, block, 0, st, p, r.waves, workers);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.dgamma == nullptr) return e;
  hipLaunchKernelGGL(dgamma_kernel, dim3(static_cast<unsigned>(p.C / 32)), dim3(256), 0, st, p.ws, workers, p.C,
                     p.dgamma);
  return hipGetLastError();
}

}  // namespace fp8bs
