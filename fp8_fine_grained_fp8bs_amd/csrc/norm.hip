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
// read once and stays in registers between its sum and its output.  Measured,
// per call in a stream of calls:
//   4096 x 7168 with residual, codes, BF16 norm and row factors: 265 MB, 43.8 us,
//     6.1 TB/s (a kernel that only moves as many bytes in this mix: 44.5);
//     5 rows 6.5 us, 4.0 in the kernel
//   gradient of 8191 x 7168 with dres: 470 MB, 79.0 us, 76 in the kernel (moving alone:
//     75 to 78) and 4.7 in the sum of dgamma's parts; 131 x 1280 5.5 us, one launch
#include <hip/hip_runtime.h>

#include "fp8bs_device.h"
#include "fp8bs_internal.h"

namespace fp8bs {
namespace {

constexpr int kMaxWaves = 16;   // waves of a row

// A row's values are spread over its workers' lanes, V vectors of 8 a lane.
// Lanes behind the row's end read its first columns, so that loads need no
// branch (a branch around a load makes the compiler wait for all loads in
// flight where the paths meet), and leave the sums and the outputs alone.
struct Lane {
  int waves, wave, lane, C;
  __device__ __forceinline__ int column(int v) const { return ((v * waves + wave) * 64 + lane) * 8; }
  __device__ __forceinline__ bool in(int v) const { return column(v) < C; }
  __device__ __forceinline__ int from(int v) const { return in(v) ? column(v) : lane * 8 & 127; }
};

// A row's sum over its waves, each with its lanes' v.  part: kMaxWaves floats
// of LDS that no wave still reads, zeros behind the waves' own.
__device__ __forceinline__ float row_sum(float v, float4* part, const Lane& at) {
  v = wave_sum(v);
  if (at.waves == 1) return v;
  if (at.lane == 0) reinterpret_cast<float*>(part)[at.wave] = v;
  __syncthreads();
  const float4 a = part[0], b = part[1], c = part[2], d = part[3];
  return (((a.x + a.y) + (a.z + a.w)) + ((b.x + b.y) + (b.z + b.w))) +
         (((c.x + c.y) + (c.z + c.w)) + ((d.x + d.y) + (d.z + d.w)));
}
// Zeros behind the waves' sums (the first row_sum's barrier shows them to all).
__device__ __forceinline__ void clear_tail(float4 (*part)[kMaxWaves / 4], const Lane& at) {
  const int i = threadIdx.x;
  if (i >= at.waves && i < kMaxWaves) {
    reinterpret_cast<float*>(part[0])[i] = 0.0f;
    reinterpret_cast<float*>(part[1])[i] = 0.0f;
  }
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

// A row's workgroup (or one of a workgroup's four waves, a row each).  x, r and
// h may be the same buffer: a lane reads its own values before it writes them.
template <int V, bool RES>
__global__ __launch_bounds__(1024) void rmsnorm_kernel(RmsNorm p, int waves) {
  __shared__ float4 part[2][kMaxWaves / 4];
  poison_lds<sizeof(part)>(part);
  const int w = threadIdx.x >> 6;
  const int64_t group = neighbours_on_an_xcd(), row = waves == 1 ? group * 4 + w : group;
  if (row >= p.T) return;
  const Lane at{waves, waves == 1 ? 0 : w, static_cast<int>(threadIdx.x) & 63, p.C};
  if (waves > 1) clear_tail(part, at);
  u32x4 h[V], r[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    h[v] = load_nt(p.x + row * p.ldx + at.from(v));
    if (RES) r[v] = load_nt(p.r + row * p.ldr + at.from(v));
  }
  float ss = 0.0f;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    float a[8], s = 0.0f;
    bf16x8_unpack(h[v], a);
    if (RES) {
      float b[8];
      bf16x8_unpack(r[v], b);
#pragma unroll
      for (int i = 0; i < 8; ++i) a[i] += b[i];
      h[v] = bf16x8_pack(a);
      bf16x8_unpack(h[v], a);
      if (at.in(v)) *reinterpret_cast<u32x4*>(p.h + row * p.ldh + at.column(v)) = h[v];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) s = __builtin_fmaf(a[i], a[i], s);
    ss += at.in(v) ? s : 0.0f;
  }
  ss = row_sum(ss, part[0], at);
  const float rstd = 1.0f / __builtin_sqrtf(ss / static_cast<float>(p.C) + p.eps);
  if (p.rstd != nullptr && at.wave == 0 && at.lane == 0) p.rstd[row] = rstd;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = at.column(v);
    const bool in = at.in(v);   // the same in all lanes of a tile: C is whole tiles
    float n[8], g[8];
    bf16x8_unpack(h[v], n);
    load_gamma(p.gamma, p.gamma_f32, at.from(v), g);
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
        if ((at.lane & 15) == 0) p.s[row * p.lds + (c >> 7)] = ts.s;
      }
    }
    if (p.y != nullptr && in) *reinterpret_cast<u32x4*>(p.y + row * p.ldy + c) = bf16x8_pack(n);
  }
}

// The gradient.  A worker (a workgroup, or one of its four waves with one wave
// a row) walks the rows first, first + workers, ..., loading the next while it
// computes one, and keeps its part of dgamma in registers; dgamma_kernel sums
// the parts in the order of the workers.  dx may be dres: a lane reads its own
// values before it writes them, and no other row's.
// WIDE: rows of more than 8192 columns, whose lanes have no registers left for
// the next row, for gamma and for dres.
template <int V>
struct BwdRow {
  u32x4 h[V], dn[V], dres[V];
  float rstd;
};

template <bool WIDE, bool RES>
__device__ __forceinline__ void bwd_rows(const RmsNormBwd& p, const Lane& at, int64_t worker, int64_t workers,
                                         float4 (*part)[kMaxWaves / 4]) {
  constexpr int V = WIDE ? 2 : 1;
  const float inv = 1.0f / static_cast<float>(p.C);
  float held[V][8], acc[V][8];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if (!WIDE) load_gamma(p.gamma, p.gamma_f32, at.from(v), held[v]);
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[v][i] = 0.0f;
  }
  int turn = 0;
  const auto load = [&](int64_t row, BwdRow<V>& b) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = at.from(v);
      b.h[v] = load_nt(p.h + row * p.ldh + c);
      b.dn[v] = load_nt(p.dn + row * p.lddn + c);
      if (RES && !WIDE) b.dres[v] = load_nt(p.dres + row * p.lddr + c);
    }
    b.rstd = p.rstd[row];
  };
  const auto compute = [&](int64_t row, const BwdRow<V>& b) {
    float dot = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float h[8], dn[8], g[8], s = 0.0f;
      bf16x8_unpack(b.h[v], h);
      bf16x8_unpack(b.dn[v], dn);
      if (WIDE) load_gamma(p.gamma, p.gamma_f32, at.from(v), g);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float u = h[i] * b.rstd;
        s = __builtin_fmaf((WIDE ? g[i] : held[v][i]) * dn[i], u, s);
        acc[v][i] = __builtin_fmaf(dn[i], u, acc[v][i]);
      }
      dot += at.in(v) ? s : 0.0f;
    }
    const float mean = row_sum(dot, part[turn], at) * inv;
    turn ^= 1;   // the next row's sum goes elsewhere: one barrier a row
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float h[8], dn[8], g[8], dx[8];
      bf16x8_unpack(b.h[v], h);
      bf16x8_unpack(b.dn[v], dn);
      if (WIDE) load_gamma(p.gamma, p.gamma_f32, at.from(v), g);
      if (RES) bf16x8_unpack(WIDE ? load_nt(p.dres + row * p.lddr + at.from(v)) : b.dres[v], dx);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float a = __builtin_fmaf(-(h[i] * b.rstd), mean, (WIDE ? g[i] : held[v][i]) * dn[i]);
        dx[i] = RES ? __builtin_fmaf(b.rstd, a, dx[i]) : b.rstd * a;
      }
      if (at.in(v)) *reinterpret_cast<u32x4*>(p.dx + row * p.lddx + at.column(v)) = bf16x8_pack(dx);
    }
  };
  int64_t row = worker;
  BwdRow<V> now, next;
  load(row, now);
  for (; row + workers < p.T; row += workers) {
    if (!WIDE) load(row + workers, next);
    compute(row, now);
    if (WIDE) load(row + workers, now);
    else now = next;
  }
  compute(row, now);
  if (p.ws != nullptr) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (!at.in(v)) continue;
      float4* out = reinterpret_cast<float4*>(p.ws + worker * p.C + at.column(v));
      out[0] = make_float4(acc[v][0], acc[v][1], acc[v][2], acc[v][3]);
      out[1] = make_float4(acc[v][4], acc[v][5], acc[v][6], acc[v][7]);
    }
  }
}

template <bool WIDE, bool RES>
__global__ __launch_bounds__(1024) void rmsnorm_bwd_kernel(RmsNormBwd p, int waves, int64_t workers) {
  __shared__ float4 part[2][kMaxWaves / 4];
  poison_lds<sizeof(part)>(part);
  const int w = threadIdx.x >> 6;
  const int64_t worker = waves == 1 ? static_cast<int64_t>(blockIdx.x) * 4 + w : blockIdx.x;
  if (worker >= workers) return;
  const Lane at{waves, waves == 1 ? 0 : w, static_cast<int>(threadIdx.x) & 63, p.C};
  if (waves > 1) clear_tail(part, at);
  bwd_rows<WIDE, RES>(p, at, worker, workers, part);
}

// Few rows: one launch.  A workgroup a row as above, and further ones that sum
// 64 columns of dn u over all rows by themselves (8 columns a lane, every
// group of 8 lanes some of the rows, joined through LDS in their order): the
// rows are read once more, from the caches.
template <bool WIDE, bool RES>
__global__ __launch_bounds__(1024) void rmsnorm_bwd_few_kernel(RmsNormBwd p, int waves, int rows) {
  __shared__ float4 part[2][kMaxWaves / 4];
  __shared__ float sums[128][65];
  poison_lds<sizeof(part)>(part);
  poison_lds<sizeof(sums)>(sums);
  const int w = threadIdx.x >> 6;
  if (static_cast<int>(blockIdx.x) < rows) {
    const int64_t worker = waves == 1 ? static_cast<int64_t>(blockIdx.x) * 4 + w : blockIdx.x;
    if (worker >= p.T) return;
    const Lane at{waves, waves == 1 ? 0 : w, static_cast<int>(threadIdx.x) & 63, p.C};
    if (waves > 1) clear_tail(part, at);
    bwd_rows<WIDE, RES>(p, at, worker, p.T, part);
    return;
  }
  const int sub = threadIdx.x & 7, group = threadIdx.x >> 3, groups = blockDim.x >> 3;
  const int c = (blockIdx.x - rows) * 64 + sub * 8;
  float acc[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
  for (int64_t row = group; row < p.T; row += groups) {
    float h[8], dn[8];
    bf16x8_unpack(*reinterpret_cast<const u32x4*>(p.h + row * p.ldh + c), h);
    bf16x8_unpack(*reinterpret_cast<const u32x4*>(p.dn + row * p.lddn + c), dn);
    const float rstd = p.rstd[row];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = __builtin_fmaf(dn[i], h[i] * rstd, acc[i]);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) sums[group][sub * 8 + i] = acc[i];
  __syncthreads();
  if (threadIdx.x < 64) {
    float s = sums[0][threadIdx.x];
    for (int k = 1; k < groups; ++k) s += sums[k][threadIdx.x];
    p.dgamma[(blockIdx.x - rows) * 64 + threadIdx.x] = s;
  }
}

// dgamma of 32 columns: 128 groups of 8 lanes take every 128th worker's part,
// joined through LDS, 16 groups at a time, in their order.
__global__ __launch_bounds__(1024) void dgamma_kernel(const float* __restrict__ parts, int64_t workers, int C,
                                                      float* __restrict__ dgamma) {
  __shared__ float sums[128][33];
  poison_lds<sizeof(sums)>(sums);
  const int sub = threadIdx.x & 7, group = threadIdx.x >> 3;
  const int c = blockIdx.x * 32;
  float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
  for (int64_t w = group; w < workers; w += 128) {
    const float4 a = *reinterpret_cast<const float4*>(parts + w * C + c + sub * 4);
    s.x += a.x; s.y += a.y; s.z += a.z; s.w += a.w;
  }
  float* mine = &sums[group][sub * 4];
  mine[0] = s.x; mine[1] = s.y; mine[2] = s.z; mine[3] = s.w;
  __syncthreads();
  const int column = threadIdx.x & 31, eighth = threadIdx.x >> 5;
  float t = 0.0f;
  if (threadIdx.x < 256) {
#pragma unroll
    for (int k = 0; k < 16; ++k) t += sums[eighth * 16 + k][column];
  }
  __syncthreads();
  if (threadIdx.x < 256) sums[eighth][column] = t;
  __syncthreads();
  if (threadIdx.x < 32) {
    t = sums[0][column];
#pragma unroll
    for (int k = 1; k < 8; ++k) t += sums[k][column];
    dgamma[c + column] = t;
  }
}

// Waves of a row with V vectors a lane.
int row_waves(int C, int V) { return (C / 8 + 64 * V - 1) / (64 * V); }

// Workers of the gradient: as many as are resident, 16 waves a compute unit
// (twice as many, half of which wait for the first, took 85 us against 79 at
// 8191 rows of 7168 columns), but a worker gets eight rows before there are
// more than a compute unit's worth, since each leaves a part of dgamma (4096
// rows of 512: 9.9 us with 1024 workers, 18.0 with 4096).
int64_t bwd_workers(int64_t T, int C) {
  const int waves = row_waves(C, C <= 8192 ? 1 : 2);
  const int64_t resident = 256 * (kMaxWaves / waves), most = T / 8 < 256 ? 256 : T / 8 < resident ? T / 8 : resident;
  return T < most ? T : most;
}

// Rows of a gradient in one launch: at 512 rows of 512, 2048 and 7168 columns 6.4, 6.9
// and 12.8 us against 9.6, 9.4 and 13.3 in two launches; at 1000 rows 8.9, 22.7 and
// 21.4 against 9.6, 12.2 and 17.2.
constexpr int64_t kFewRows = 512;

}  // namespace

hipError_t launch_rmsnorm(const RmsNorm& p, hipStream_t st) {
  // two vectors a lane: level with one and with four at 4096 rows of 7168
  // columns (44.2 us against 44.7 and 44.5)
  const bool narrow = p.C <= 512;
  const int waves = row_waves(p.C, narrow ? 1 : 2);
  const int threads = waves == 1 ? 256 : 64 * waves, together = waves == 1 ? 4 : 1;
  return by_tokens(p, most_blocks(threads) * together, [&](const RmsNorm& p) {
    const dim3 grid(static_cast<unsigned>((p.T + together - 1) / together)), block(threads);
#define FP8BS_NORM(V, RES) hipLaunchKernelGGL((rmsnorm_kernel<V, RES>), grid, block, 0, st, p, waves)
    if (narrow && p.r != nullptr) FP8BS_NORM(1, true);
    else if (narrow) FP8BS_NORM(1, false);
    else if (p.r != nullptr) FP8BS_NORM(2, true);
    else FP8BS_NORM(2, false);
#undef FP8BS_NORM
    return hipGetLastError();
  });
}

int64_t rmsnorm_bwd_ws(int64_t T, int C) {
  return T <= kFewRows ? 0 : bwd_workers(T, C) * C * static_cast<int64_t>(sizeof(float));
}

hipError_t launch_rmsnorm_bwd(const RmsNormBwd& args, hipStream_t st) {
  RmsNormBwd p = args;
  const bool wide = p.C > 8192;
  const int waves = row_waves(p.C, wide ? 2 : 1);
  const dim3 block(waves == 1 ? 256 : 64 * waves);
  if (p.T <= kFewRows) {
    p.ws = nullptr;
    const int rows = static_cast<int>(waves == 1 ? (p.T + 3) / 4 : p.T);
    const dim3 grid(static_cast<unsigned>(rows + (p.dgamma != nullptr ? p.C / 64 : 0)));
#define FP8BS_NORM(WIDE, RES) hipLaunchKernelGGL((rmsnorm_bwd_few_kernel<WIDE, RES>), grid, block, 0, st, p, waves, rows)
    if (wide && p.dres != nullptr) FP8BS_NORM(true, true);
    else if (wide) FP8BS_NORM(true, false);
    else if (p.dres != nullptr) FP8BS_NORM(false, true);
    else FP8BS_NORM(false, false);
#undef FP8BS_NORM
    return hipGetLastError();
  }
  if (p.dgamma == nullptr) p.ws = nullptr;
  const int64_t workers = bwd_workers(p.T, p.C);
  const dim3 grid(static_cast<unsigned>(waves == 1 ? (workers + 3) / 4 : workers));
#define FP8BS_NORM(WIDE, RES) hipLaunchKernelGGL((rmsnorm_bwd_kernel<WIDE, RES>), grid, block, 0, st, p, waves, workers)
  if (wide && p.dres != nullptr) FP8BS_NORM(true, true);
  else if (wide) FP8BS_NORM(true, false);
  else if (p.dres != nullptr) FP8BS_NORM(false, true);
  else FP8BS_NORM(false, false);
#undef FP8BS_NORM
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.dgamma == nullptr) return e;
  hipLaunchKernelGGL(dgamma_kernel, dim3(static_cast<unsigned>(p.C / 32)), dim3(1024), 0, st, p.ws, workers, p.C,
                     p.dgamma);
  return hipGetLastError();
}

}  // namespace fp8bs
