// moe.hip -- tokens sorted by expert and brought back, with their gradients
// (gfx950): what stands before and behind the grouped GEMM.
//
// An assignment (t, j) sends token t to expert ids[t][j].  The assignments to
// the experts held here, ordered by (expert, t, j), are the rows of the
// grouped GEMM's operand; slot[t][j] is an assignment's row, -1 where it has
// none.  Everything else goes by token: a token's row of activations is
// quantized once and written to its k rows, its k rows of outputs are summed
// with their weights, and in the gradient the token's row of dout is
// quantized once and written to k rows.  All of it moves memory: two or three
// operations a byte.  Measured, per call in a stream of calls:
//   8192 tokens of 7168, a tenth of them padding, 8 of 256 experts each, to the 32 held
//     here: 28.7 to 34.6 us, as many as the ids send here; 9.5 of it the sort's two kernels,
//     the rest the rows (19 of 28.7, some 105 MB at 5.5 TB/s); 4096 tokens of 7168 to 8 of
//     64, all held, 71.7 us (301 MB, 4.2 TB/s), from codes 69.0 (273 MB, 4.0);
//     16 tokens to 8 of 64 experts 6.2 us, one launch
//   4099 x 8 rows of 7168 back: 588 MB, 98.3 us, 6.0 TB/s (as many bytes in order, 8
//     reads to a write, move at 6.2)
//   gradient of 8191 x 2 rows of 7168: 474 MB, 89.9 us, 5.3 TB/s: its reads alone take
//     52 us (6.7 TB/s), the scattered rows of codes the rest
#include <hip/hip_runtime.h>

#include "fp8bs_device.h"
#include "fp8bs_internal.h"

namespace fp8bs {
namespace {

// ---------------------------------------------------------------------
// The sort: a stable counting sort by expert.
//
// Workgroups take stretches of the assignments.  An assignment's row is the
// number of those of smaller experts, plus those of its own expert in earlier
// stretches, plus its rank in its stretch.  The first two come from counts by
// stretch and expert, which a kernel of its own writes (large batches) or
// every workgroup counts for itself (small ones: all assignments, from the
// caches).  Within a stretch the order is kept without atomics: a wave
// compares its 64 assignments bit by bit (ballots), which gives an
// assignment's rank among those of its expert, and counts per wave are
// summed over the waves.  Bound by latency: each kernel is a chain of four or
// five dependent loads and barriers (65536 assignments: 4.8 us each).
// ---------------------------------------------------------------------
constexpr int kSortThreads = 512;
constexpr int kSortWaves = kSortThreads / 64;
constexpr int kSteps = 2;                             // assignments of a lane and round
constexpr int kRound = kSortThreads * kSteps;         // of a workgroup and round
constexpr int kPerThread = kMaxExperts / kSortThreads;
// assignments that every workgroup counts for itself (with the rows in a launch of
// their own): 8192 to 64 experts with rows of 128 columns 9.7 us against 12.7 with the
// counting kernel, of 2048 15.0 and 15.6; 16384 with rows of 2048 20.0 against 18.1
constexpr int64_t kCountHere = 8192;

// Expert of assignment i among those held here, or -1.
__device__ __forceinline__ int expert_of(const MoeIds& p, int64_t i) {
  int64_t at = i;
  if (p.ldi != p.k) {
    const int64_t t = static_cast<uint32_t>(i) / static_cast<uint32_t>(p.k);   // T k <= 2^30
    at = t * p.ldi + (i - t * p.k);
  }
  const int64_t id = p.wide ? static_cast<const int64_t*>(p.ids)[at] : static_cast<const int32_t*>(p.ids)[at];
  return id >= p.first && id - p.first < p.E ? static_cast<int>(id - p.first) : -1;
}

__global__ __launch_bounds__(kSortThreads) void moe_count_kernel(MoeIds p, int64_t n, int64_t stretch, int32_t* counts) {
  __shared__ int count[kMaxExperts];
  poison_lds<sizeof(count)>(count);
  for (int e = threadIdx.x; e < p.E; e += kSortThreads) count[e] = 0;
  __syncthreads();
  const int64_t a = blockIdx.x * stretch, b = a + stretch < n ? a + stretch : n;
  for (int64_t i = a + threadIdx.x; i < b; i += kSortThreads) {
    const int e = expert_of(p, i);
    if (e >= 0) atomicAdd(&count[e], 1);   // whole numbers: their order changes nothing
  }
  __syncthreads();
  for (int e = threadIdx.x; e < p.E; e += kSortThreads) counts[static_cast<int64_t>(blockIdx.x) * p.E + e] = count[e];
}

// Exclusive sum of every thread's v over the workgroup's threads, and the
// whole sum in `all`.  sums: one number a wave, which no thread still reads.
__device__ __forceinline__ int exclusive_sum(int v, int* sums, int& all) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  int s = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(s, d);
    if (lane >= d) s += o;
  }
  if (lane == 63) sums[wave] = s;
  __syncthreads();
  int before = 0;
  all = 0;
  for (int k = 0; k < waves; ++k) {
    const int x = sums[k];
    before += k < wave ? x : 0;
    all += x;
  }
  return before + s - v;
}

// All n assignments counted by expert: those before a in `start`, the others in
// `total`.  Bound by the loads' latency: four of a thread are in flight, with
// indices cut to the last assignment in place of branches.  Dispatch of 8192 with rows
// of 2048 10.9 us (12.2 with a branch at each load); of 512 with rows of 7168 6.8, with
// eight in flight 7.3 and with sixteen 8.2, whose surplus loads wait for nothing.
__device__ __forceinline__ void count_all(const MoeIds& p, int n, int a, int* start, int* total) {
  constexpr int kLoads = 4;
  for (int base = threadIdx.x; base < n; base += kLoads * kSortThreads) {
    int e[kLoads];
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      const int i = base + u * kSortThreads;
      e[u] = expert_of(p, i < n ? i : n - 1);
    }
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      const int i = base + u * kSortThreads;
      if (i < n && e[u] >= 0) atomicAdd(i < a ? &start[e[u]] : &total[e[u]], 1);
    }
  }
}

// The stretches' counts summed by expert: of those before stretch `mine` to `start`,
// of all to `total`.  As many threads an expert as there are, each some of the stretches.
__device__ __forceinline__ void add_counts(const int32_t* __restrict__ counts, int E, int stretches, int mine,
                                           int* start, int* total) {
  const int parts = E < kSortThreads ? kSortThreads / E : 1;
  for (int x = threadIdx.x; x < E * parts; x += kSortThreads) {
    const int part = x / E, e = x - part * E;
    int all = 0, earlier = 0;
#pragma unroll 4
    for (int s = part; s < stretches; s += parts) {
      const int c = counts[static_cast<int64_t>(s) * E + e];
      all += c;
      earlier += s < mine ? c : 0;
    }
    atomicAdd(&total[e], all);
    atomicAdd(&start[e], earlier);
  }
}

// counts: of every stretch, or null (counted here).
__global__ __launch_bounds__(kSortThreads) void moe_place_kernel(MoeIds p, int64_t n, int64_t stretch, int stretches,
                                                                 int bits, const int32_t* __restrict__ counts) {
  __shared__ int rows[kSortWaves][kMaxExperts];   // a wave's counts, then what the waves before it have
  __shared__ int total[kMaxExperts];              // assignments of an expert
  __shared__ int start[kMaxExperts];              // those of earlier stretches, then the row of the next
  __shared__ int sums[kSortWaves];
  poison_lds<sizeof(rows)>(rows);
  poison_lds<sizeof(total)>(total);
  poison_lds<sizeof(start)>(start);
  poison_lds<sizeof(sums)>(sums);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const uint64_t below = (uint64_t(1) << lane) - 1;
  const int64_t a = blockIdx.x * stretch, b = a + stretch < n ? a + stretch : n;
  for (int x = tid; x < p.E; x += kSortThreads) {
    total[x] = 0;
    start[x] = 0;
  }
  __syncthreads();
  if (counts != nullptr) {
    add_counts(counts, p.E, stretches, blockIdx.x, start, total);
  } else {
    count_all(p, static_cast<int>(n), static_cast<int>(a), start, total);
    __syncthreads();
    for (int x = tid; x < p.E; x += kSortThreads) total[x] += start[x];
  }
  __syncthreads();
  {
    int mine[kPerThread], sum = 0, all;
#pragma unroll
    for (int x = 0; x < kPerThread; ++x) {
      mine[x] = tid * kPerThread + x < p.E ? total[tid * kPerThread + x] : 0;
      sum += mine[x];
    }
    int first = exclusive_sum(sum, sums, all);
#pragma unroll
    for (int x = 0; x < kPerThread; ++x) {
      const int e = tid * kPerThread + x;
      if (e < p.E) {
        start[e] += first;
        if (blockIdx.x == 0) p.offsets[e] = first < p.M ? first : static_cast<int32_t>(p.M);
      }
      first += mine[x];
    }
    if (blockIdx.x == 0 && tid == 0) p.offsets[p.E] = all < p.M ? all : static_cast<int32_t>(p.M);
  }
  for (int64_t round = a; round < b; round += kRound) {
    int e[kSteps], rank[kSteps];
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int64_t i = round + (wave * kSteps + s) * 64 + lane;
      e[s] = i < b ? expert_of(p, i) : -1;
    }
    for (int x = lane; x < p.E; x += 64) rows[wave][x] = 0;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      uint64_t same = __ballot(e[s] >= 0);
      for (int bit = 0; bit < bits; ++bit) {
        const uint64_t ones = __ballot((e[s] >> bit) & 1);
        same &= (e[s] >> bit) & 1 ? ones : ~ones;
      }
      rank[s] = __popcll(same & below);
      int had = 0;
      if (e[s] >= 0) had = rows[wave][e[s]];
      // all lanes have read before the first of each expert writes: LDS
      // serves a wave's accesses in their order
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      if (e[s] >= 0 && rank[s] == 0) rows[wave][e[s]] = had + __popcll(same);
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      rank[s] += had;
    }
    __syncthreads();
    int mine[kPerThread];
#pragma unroll
    for (int x = 0; x < kPerThread; ++x) {
      const int expert = tid + x * kSortThreads;
      mine[x] = 0;
      if (expert >= p.E) continue;
#pragma unroll
      for (int w = 0; w < kSortWaves; ++w) {
        const int c = rows[w][expert];
        rows[w][expert] = mine[x];
        mine[x] += c;
      }
    }
    __syncthreads();
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int64_t i = round + (wave * kSteps + s) * 64 + lane;
      if (i >= b) continue;
      const int at = e[s] >= 0 ? start[e[s]] + rows[wave][e[s]] + rank[s] : -1;
      p.slot[i] = at < p.M ? at : -1;
    }
    __syncthreads();
#pragma unroll
    for (int x = 0; x < kPerThread; ++x)
      if (tid + x * kSortThreads < p.E) start[tid + x * kSortThreads] += mine[x];
  }
}

// ---------------------------------------------------------------------
// Rows to their places.  A workgroup a token, so that a row's scales, written
// a few at a time, meet in one L2; a lane has V vectors of 8 values at a time.
// ---------------------------------------------------------------------
// A lane's vectors of a row, 512 columns apart.  A lane behind the row's
// end reads the row's first columns and leaves its outputs alone.
struct Columns {
  int c0, N;
  __device__ __forceinline__ int at(int v) const { return c0 + v * 512; }
  __device__ __forceinline__ bool in(int v) const { return at(v) < N; }
  __device__ __forceinline__ int from(int v) const { return in(v) ? at(v) : c0 & 127; }
};

// A token's slots and weights, one a lane.
struct Choices {
  int slot;
  float weight;
  int64_t M;
  __device__ __forceinline__ Choices(const int32_t* s, const float* w, int k, int64_t M, int lane)
      : slot(lane < k ? s[lane] : -1), weight(w != nullptr && lane < k ? w[lane] : 1.0f), M(M) {}
  // assignment j (any number: -1 behind the last), the same in the whole wave
  __device__ __forceinline__ int64_t row(int j) const { return j < 64 ? __builtin_amdgcn_readlane(slot, j) : -1; }
  __device__ __forceinline__ bool there(int64_t row) const { return row >= 0 && row < M; }
  __device__ __forceinline__ bool any() const { return __ballot(there(slot)) != 0; }
  __device__ __forceinline__ float w(int j) const {
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(weight), j & 63));
  }
};

// 8 bf16 values to codes and their tile's scale (all 16 lanes of a tile).
__device__ __forceinline__ uint2 quantize8(const u32x4& v, float& scale) {
  float a[8];
  bf16x8_unpack(v, a);
  float am = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) am = __builtin_fmaxf(am, __builtin_fabsf(a[i]));
  am = row16_max(am);
  const TileScale t = make_tile_scale(am);
  const Bf16Side k = bf16_side(t.s, am);
  scale = t.s;
  return make_uint2(encode4_bf16(a, t, k), encode4_bf16(a + 4, t, k));
}

// A lane's part of a row on its way: values in BF16, or codes with scales.
template <int V>
struct Unit {
  u32x4 x[V];
  uint2 code[V];
  float scale[V];
};

template <bool CODES, int V>
__device__ __forceinline__ void load_unit(const MoeRows& p, int64_t t, const Columns& c, Unit<V>& u) {
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if (CODES) {
      const u32x2 q = __builtin_nontemporal_load(
          reinterpret_cast<const u32x2*>(static_cast<const uint8_t*>(p.x) + t * p.ldx + c.from(v)));
      u.code[v] = make_uint2(q[0], q[1]);
      u.scale[v] = p.s_in[t * p.lds_in + (c.from(v) >> 7)];
    } else {
      u.x[v] = __builtin_nontemporal_load(
          reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(p.x) + t * p.ldx + c.from(v)));
    }
  }
}

// A unit to the rows chosen.  Called by whole waves.
template <bool CODES, int V>
__device__ __forceinline__ void store_unit(const MoeRows& p, const Columns& c, Unit<V>& u, const Choices& chosen, int lane) {
  if (!CODES && p.q != nullptr) {
#pragma unroll
    for (int v = 0; v < V; ++v) u.code[v] = quantize8(u.x[v], u.scale[v]);
  }
  for (int j = 0; j < p.k; ++j) {
    const int64_t row = chosen.row(j);
    if (!chosen.there(row)) continue;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (!c.in(v)) continue;
      if (CODES || p.q != nullptr) {
        // plain stores: past the caches they were 7 us faster by themselves at 8192
        // x 2 rows of 7168, and cost the product that reads them 8
        *reinterpret_cast<uint2*>(p.q + row * p.ldq + c.at(v)) = u.code[v];
        if ((lane & 15) == 0) p.s[row * p.lds + (c.at(v) >> 7)] = u.scale[v];
      }
      if (!CODES && p.y != nullptr) *reinterpret_cast<u32x4*>(p.y + row * p.ldy + c.at(v)) = u.x[v];
    }
  }
}

// Narrow rows (V == 1: up to 512 columns) are a wave's; four such tokens are a
// workgroup (with two vectors a lane, most of them idle, and a workgroup a token the
// gradient of 16384 x 2 rows of 256 took 23.2 us against 13.8, dispatching them 16.5
// against 14.9).
constexpr int kTogether = 4;

// CODES: x holds codes with scales.
template <bool CODES, int V>
__global__ __launch_bounds__(1024) void moe_gather_kernel(MoeRows p) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, wave = V == 1 ? 0 : w, waves = V == 1 ? 1 : blockDim.x >> 6;
  const int64_t t = V == 1 ? neighbours_on_an_xcd() * kTogether + w : neighbours_on_an_xcd();
  if (t >= p.T) return;
  const Choices chosen(p.slot + t * p.k, nullptr, p.k, p.M, lane);
  if (!chosen.any()) return;   // no row: x is not read
  for (int base = wave * (512 * V); base < p.C; base += waves * (512 * V)) {
    const Columns c{base + lane * 8, p.C};
    Unit<V> u;
    load_unit<CODES, V>(p, t, c, u);
    store_unit<CODES, V>(p, c, u, chosen, lane);
  }
}

// Sort and rows in one launch (up to kOneLaunch assignments), or in one behind the
// counting kernel (COUNTED).  A workgroup takes a few tokens, with at most 64
// assignments, and counts those before its own by expert for itself, all of them or
// those of its stretch, which gives its own rows as in the sort above; their ranks
// are one wave's ballots.  A wave's next loads go out before its rows are stored: 1024
// tokens of 7168 to 8 of 64 experts 20.2 us (22.5 without).  Against sort and rows
// in launches of their own: 256 such tokens 8.5 us and 12.1, 512 11.5 and 15.3, 1024 of
// 1024 columns 9.5 and 11.3, of 7168 20.2 and 21.0; 8192 tokens to one expert each 38.1 and
// 37.5.
constexpr int kOneLaunch = 8192;
static_assert(kOneLaunch >= kCountHere, "more assignments have a workspace for their counts");

// Whether a batch of more assignments is COUNTED, or has the sort's two kernels and
// the rows' own.  That kernel has fewer, longer workgroups, which pays as long as the
// launch that it spares is a good part of the whole: 2048 tokens of 2048 to 8 of 64
// experts 14.7 us against 18.0, 4096 to 8 of 8 22.8 and 22.6, 2048 of 7168 38.7
// and 39.5, 4096 of 4096 43.7 and 43.9, 16384 of 1024 to 2 20.0 and 21.9.  Past these
// limits: 16384 of 1024 to 4 28.8 and 28.7, 2048 of 7168 to 16 73.3 and 68.9,
// 8192 of 7168 to 2 59.2 and 54.3 and, held elsewhere for the most part, to 8 of 256 40.8 and
// 28.8; of narrow rows 16384 of 256 to 2 15.8 and 15.0, 32768 of 512 23.8 and 21.3.
inline bool counted_rows(int64_t T, int k, int64_t C) {
  return T <= (C < 1024 ? 8192 : 16384) && T * k <= 32768 && T * C <= 1 << 24 && T * k * C <= 1 << 27;
}

template <bool CODES, bool COUNTED>
__global__ __launch_bounds__(kSortThreads) void moe_dispatch_kernel(MoeIds ids, MoeRows p, int tokens, int bits,
                                                                    int stretch, int stretches,
                                                                    const int32_t* __restrict__ counts) {
  __shared__ int total[kMaxExperts];
  __shared__ int start[kMaxExperts];
  __shared__ int sums[kSortWaves];
  __shared__ int32_t slots[64];
  poison_lds<sizeof(total)>(total);
  poison_lds<sizeof(start)>(start);
  poison_lds<sizeof(sums)>(sums);
  poison_lds<sizeof(slots)>(slots);
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int T = static_cast<int>(ids.T), n = T * ids.k;
  const int t0 = static_cast<int>(neighbours_on_an_xcd()) * tokens, here = T - t0 < tokens ? T - t0 : tokens;
  const int a = t0 * ids.k, b = a + here * ids.k;
  const int chunks = (p.C + 1023) / 1024, items = here * chunks;
  const int step = kSortWaves / chunks, rest = kSortWaves - step * chunks;   // from a wave's item to its next
  int token = wave / chunks, chunk = wave - token * chunks;
  // the first columns are on their way while the rows are counted
  Unit<2> u;
  if (wave < items) load_unit<CODES, 2>(p, t0 + token, Columns{chunk * 1024 + lane * 8, p.C}, u);
  for (int e = tid; e < ids.E; e += kSortThreads) {
    total[e] = 0;
    start[e] = 0;
  }
  __syncthreads();
  if (COUNTED) {
    const int s = a / stretch;
    for (int i = s * stretch + tid; i < a; i += kSortThreads) {
      const int e = expert_of(ids, i);
      if (e >= 0) atomicAdd(&start[e], 1);
    }
    add_counts(counts, ids.E, stretches, s, start, total);
  } else {
    count_all(ids, n, a, start, total);
  }
  __syncthreads();
  {
    int mine[kPerThread], sum = 0, all;
#pragma unroll
    for (int x = 0; x < kPerThread; ++x) {
      const int e = tid * kPerThread + x;
      mine[x] = e >= ids.E ? 0 : COUNTED ? total[e] : total[e] + start[e];
      sum += mine[x];
    }
    int first = exclusive_sum(sum, sums, all);
#pragma unroll
    for (int x = 0; x < kPerThread; ++x) {
      const int e = tid * kPerThread + x;
      if (e < ids.E) {
        start[e] += first;
        if (blockIdx.x == 0) ids.offsets[e] = first < ids.M ? first : static_cast<int32_t>(ids.M);
      }
      first += mine[x];
    }
    if (blockIdx.x == 0 && tid == 0) ids.offsets[ids.E] = all < ids.M ? all : static_cast<int32_t>(ids.M);
  }
  __syncthreads();
  if (wave == 0) {
    const int e = a + lane < b ? expert_of(ids, a + lane) : -1;
    uint64_t same = __ballot(e >= 0);
    for (int bit = 0; bit < bits; ++bit) {
      const uint64_t ones = __ballot((e >> bit) & 1);
      same &= (e >> bit) & 1 ? ones : ~ones;
    }
    const int row = e >= 0 ? start[e] + __popcll(same & ((uint64_t(1) << lane) - 1)) : -1;
    const int at = row < ids.M ? row : -1;
    slots[lane] = at;
    if (a + lane < b) ids.slot[a + lane] = at;
  }
  __syncthreads();
  if (wave >= items) return;
  Choices chosen(slots + token * ids.k, nullptr, ids.k, p.M, lane);
  for (int item = wave; item < items; item += kSortWaves) {
    const Columns c{chunk * 1024 + lane * 8, p.C};
    token += step;
    chunk += rest;
    if (chunk >= chunks) {
      chunk -= chunks;
      ++token;
    }
    Choices next = chosen;
    Unit<2> ahead{};
    if (item + kSortWaves < items) {
      next = Choices(slots + token * ids.k, nullptr, ids.k, p.M, lane);
      if (next.any())   // no row: x is not read
        load_unit<CODES, 2>(p, t0 + token, Columns{chunk * 1024 + lane * 8, p.C}, ahead);
    }
    if (chosen.any()) store_unit<CODES, 2>(p, c, u, chosen, lane);
    u = ahead;
    chosen = next;
  }
}

// ---------------------------------------------------------------------
// Rows back: out[t] = add[t] + sum over j of w[t][j] y[slot[t][j]], j
// ascending, one FMA a row in FP32.  A wave takes 512 V columns of a token, V
// vectors of 8 a lane, with up to kAhead rows' loads in flight.
// ---------------------------------------------------------------------
constexpr int kAhead = 8;

template <bool F32>
struct Values8 {
  u32x4 a, b;   // b: of FP32 rows
};
template <bool F32>
__device__ __forceinline__ Values8<F32> load8(const void* y, int64_t at) {
  Values8<F32> v;
  if (F32) {
    const u32x4* p = reinterpret_cast<const u32x4*>(static_cast<const float*>(y) + at);
    v.a = __builtin_nontemporal_load(p);
    v.b = __builtin_nontemporal_load(p + 1);
  } else {
    v.a = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(y) + at));
  }
  return v;
}
template <bool F32>
__device__ __forceinline__ void values8(const Values8<F32>& v, float (&f)[8]) {
  if (F32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[i] = __uint_as_float(v.a[i]);
      f[4 + i] = __uint_as_float(v.b[i]);
    }
  } else {
    bf16x8_unpack(v.a, f);
  }
}

template <bool F32, int V>
__global__ __launch_bounds__(256) void moe_combine_kernel(MoeCombine p, int chunks) {
  const int64_t item = neighbours_on_an_xcd() * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t = item <= 0xffffffffll ? static_cast<uint32_t>(item) / static_cast<uint32_t>(chunks) : item / chunks;
  if (t >= p.T) return;
  const int lane = threadIdx.x & 63;
  const Columns c{static_cast<int>(item - t * chunks) * (512 * V) + lane * 8, p.N};
  const Choices chosen(p.slot + t * p.k, p.w != nullptr ? p.w + t * p.ldw : nullptr, p.k, p.M, lane);
  float acc[V][8];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    u32x4 add{0u, 0u, 0u, 0u};
    if (p.add != nullptr) add = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p.add + t * p.ldadd + c.from(v)));
    bf16x8_unpack(add, acc[v]);
  }
  for (int j0 = 0; j0 < p.k; j0 += kAhead) {
    Values8<F32> x[kAhead][V];
    bool there[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int64_t row = chosen.row(j0 + j);
      there[j] = chosen.there(row);
      if (!there[j]) continue;
#pragma unroll
      for (int v = 0; v < V; ++v) x[j][v] = load8<F32>(p.y, row * p.ldy + c.from(v));
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (!there[j]) continue;
      const float w = chosen.w(j0 + j);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float f[8];
        values8<F32>(x[j][v], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[v][i] = __builtin_fmaf(w, f[i], acc[v][i]);
      }
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if (!c.in(v)) continue;
    u32x4* out = reinterpret_cast<u32x4*>(p.out + t * p.ldo + c.at(v));
    const u32x4 x = bf16x8_pack(acc[v]);
    // beside rows of FP32 the output is better kept out of their way in the
    // caches (2048 x 8 rows of 7168: 91 us against 100); beside BF16 rows it
    // makes no difference or costs 2% (8192 x 2: 75.1 against 73.4)
    if (F32) __builtin_nontemporal_store(x, out);
    else *out = x;
  }
}

// ---------------------------------------------------------------------
// Gradient of the way back: dy[slot] = w dout[t] as codes (dout's tile is
// quantized once; a row's scales are those of dout times |w|, its signs those
// of w dout) and in BF16, dw[t][j] = dout[t] . y[slot].  A workgroup a token,
// whose waves all have columns in their first turn, or four tokens of a wave
// each, whose row is then one turn.
// ---------------------------------------------------------------------
template <bool F32, int V>
__global__ __launch_bounds__(V == 4 ? 512 : 1024) void moe_combine_bwd_kernel(MoeCombineBwd p) {
  __shared__ float part[kMaxChoices][16];
  poison_lds<sizeof(part)>(part);
  constexpr int kAheadBwd = 8 / V, kStep = 512 * V;   // rows whose loads are in flight, columns of a wave
  const int tid = threadIdx.x, lane = tid & 63, w0 = tid >> 6, wave = V == 1 ? 0 : w0, waves = V == 1 ? 1 : blockDim.x >> 6;
  const int64_t t = V == 1 ? neighbours_on_an_xcd() * kTogether + w0 : neighbours_on_an_xcd();
  if (t >= p.T) return;
  const Choices chosen(p.slot + t * p.k, p.w + t * p.ldw, p.k, p.M, lane);
  const bool any = chosen.any();   // without rows dout is not read
  for (int base = wave * kStep; any && base < p.N; base += waves * kStep) {
    const Columns c{base + lane * 8, p.N};
    u32x4 d[V];
#pragma unroll
    for (int v = 0; v < V; ++v)
      d[v] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p.dout + t * p.lddo + c.from(v)));
    uint2 code[V];
    float scale[V];
    for (int j0 = 0; j0 < p.k; j0 += kAheadBwd) {
      Values8<F32> x[kAheadBwd][V];
      if (p.dw != nullptr) {
#pragma unroll
        for (int j = 0; j < kAheadBwd; ++j) {
          const int64_t row = chosen.row(j0 + j);
          if (!chosen.there(row)) continue;
#pragma unroll
          for (int v = 0; v < V; ++v) x[j][v] = load8<F32>(p.y, row * p.ldy + c.from(v));
        }
      }
      if (j0 == 0 && p.q != nullptr) {
#pragma unroll
        for (int v = 0; v < V; ++v) code[v] = quantize8(d[v], scale[v]);
      }
#pragma unroll
      for (int j = 0; j < kAheadBwd; ++j) {
        const int64_t row = chosen.row(j0 + j);
        if (!chosen.there(row)) continue;
        const float w = chosen.w(j0 + j);
        if (p.dw != nullptr) {
          float dot = 0.0f;
#pragma unroll
          for (int v = 0; v < V; ++v) {
            float f[8], a[8], s = 0.0f;
            values8<F32>(x[j][v], f);
            bf16x8_unpack(d[v], a);
#pragma unroll
            for (int i = 0; i < 8; ++i) s = __builtin_fmaf(a[i], f[i], s);
            dot += c.in(v) ? s : 0.0f;
          }
          dot = wave_sum(dot);
          if (V == 1) {
            if (lane == 0) p.dw[t * p.lddw + j0 + j] = dot;
          } else if (lane == 0) {
            part[j0 + j][wave] = base == wave * kStep ? dot : part[j0 + j][wave] + dot;
          }
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
          if (!c.in(v)) continue;
          if (p.q != nullptr) {
            const uint32_t turn = w < 0.0f ? 0x80808080u : 0u;
            *reinterpret_cast<uint2*>(p.q + row * p.ldq + c.at(v)) = make_uint2(code[v].x ^ turn, code[v].y ^ turn);
            if ((lane & 15) == 0) p.s[row * p.lds + (c.at(v) >> 7)] = __builtin_fabsf(w) * scale[v];
          }
          if (p.dy != nullptr) {
            float a[8];
            bf16x8_unpack(d[v], a);
#pragma unroll
            for (int i = 0; i < 8; ++i) a[i] *= w;
            *reinterpret_cast<u32x4*>(p.dy + row * p.lddy + c.at(v)) = bf16x8_pack(a);
          }
        }
      }
    }
  }
  if (p.dw == nullptr) return;
  if (V == 1) {
    if (lane < p.k && !chosen.there(chosen.slot)) p.dw[t * p.lddw + lane] = 0.0f;
    return;
  }
  __syncthreads();
  for (int j = tid; j < p.k; j += blockDim.x) {
    const int64_t row = p.slot[t * p.k + j];
    float s = 0.0f;
    if (chosen.there(row))
      for (int w = 0; w < waves; ++w) s += part[j][w];
    p.dw[t * p.lddw + j] = s;
  }
}

// Stretches of the sort and their length (whole rounds).  Every workgroup reads
// the counts of all stretches, so many experts get fewer.
struct Stretches {
  int64_t length;
  int count;
};
Stretches stretches_of(int64_t n, int E) {
  const int64_t rounds = (n + kRound - 1) / kRound, most = E <= 64 ? 256 : E <= 128 ? 128 : 64;
  const int64_t each = rounds > most ? (rounds + most - 1) / most : 1;
  // one where there is nothing to place: the offsets are still written
  return {each * kRound, n > 0 ? static_cast<int>((rounds + each - 1) / each) : 1};
}

// Launches by token, V vectors a lane and at most so many waves: a workgroup's threads
// and tokens.
struct Tokens {
  int threads, each;
  int64_t most() const { return most_blocks(threads) * each; }
  dim3 grid(int64_t T) const { return dim3(static_cast<unsigned>((T + each - 1) / each)); }
};
Tokens tokens_of(int columns, int V, int most) {
  if (V == 1) return {64 * kTogether, kTogether};
  const int waves = (columns + 512 * V - 1) / (512 * V);
  return {64 * (waves > most ? most : waves), 1};
}

// Bits of an expert's number.
int id_bits(int E) {
  int bits = 0;
  while ((E - 1) >> bits) ++bits;
  return bits;
}

}  // namespace

int64_t moe_sort_ws(int64_t T, int k, int E) {
  const int64_t n = T * k;
  return n > kCountHere ? stretches_of(n, E).count * E * static_cast<int64_t>(sizeof(int32_t)) : 0;
}

hipError_t launch_moe_sort(const MoeIds& p, hipStream_t st) {
  const int64_t n = p.T * p.k;
  const Stretches s = stretches_of(n, p.E);
  int32_t* counts = nullptr;
  if (n > kCountHere) {
    counts = p.ws;
    hipLaunchKernelGGL(moe_count_kernel, dim3(s.count), dim3(kSortThreads), 0, st, p, n, s.length, counts);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(moe_place_kernel, dim3(s.count), dim3(kSortThreads), 0, st, p, n, s.length, s.count, id_bits(p.E),
                     counts);
  return hipGetLastError();
}

hipError_t launch_moe_gather(const MoeRows& p, hipStream_t st) {
  // four vectors a lane for wide rows in BF16 (8192 tokens of 7168 to 32 of 256 experts
  // 28.9 us against 31.8, all of them to 2 of 8 level), two for narrower ones and for
  // codes, whose lanes have nothing to compute (4096 x 8 rows of 7168: 70.5 us against
  // 73.8); one where a row has no more
  const int V = p.C <= 512 ? 1 : p.codes_in || p.C < 2048 ? 2 : 4;
  const Tokens g = tokens_of(p.C, V, 16);
  return by_tokens(p, g.most(), [&](const MoeRows& p) {
    const dim3 grid = g.grid(p.T), block(g.threads);
    if (p.codes_in && V == 1) hipLaunchKernelGGL((moe_gather_kernel<true, 1>), grid, block, 0, st, p);
    else if (p.codes_in) hipLaunchKernelGGL((moe_gather_kernel<true, 2>), grid, block, 0, st, p);
    else if (V == 1) hipLaunchKernelGGL((moe_gather_kernel<false, 1>), grid, block, 0, st, p);
    else if (V == 2) hipLaunchKernelGGL((moe_gather_kernel<false, 2>), grid, block, 0, st, p);
    else hipLaunchKernelGGL((moe_gather_kernel<false, 4>), grid, block, 0, st, p);
    return hipGetLastError();
  });
}

hipError_t launch_moe_dispatch(const MoeIds& ids, const MoeRows& p, hipStream_t st) {
  const int64_t n = ids.T * ids.k;
  const Stretches s = stretches_of(n, ids.E);
  if (n <= kOneLaunch || counted_rows(ids.T, ids.k, p.C)) {
    const bool counted = n > kOneLaunch;
    if (counted) {
      hipLaunchKernelGGL(moe_count_kernel, dim3(s.count), dim3(kSortThreads), 0, st, ids, n, s.length, ids.ws);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    // enough workgroups for the compute units
    const int T = static_cast<int>(ids.T), most = 64 / ids.k;
    const int each = (T + 511) / 512, tokens = each < most ? each : most;
    const dim3 grid((T + tokens - 1) / tokens), block(kSortThreads);
    const auto kernel = p.codes_in ? counted ? moe_dispatch_kernel<true, true> : moe_dispatch_kernel<true, false>
                        : counted  ? moe_dispatch_kernel<false, true>
                                   : moe_dispatch_kernel<false, false>;
    hipLaunchKernelGGL(kernel, grid, block, 0, st, ids, p, tokens, id_bits(ids.E), static_cast<int>(s.length), s.count,
                       ids.ws);
    return hipGetLastError();
  }
  const hipError_t e = launch_moe_sort(ids, st);
  return e != hipSuccess ? e : launch_moe_gather(p, st);
}

hipError_t launch_moe_combine(const MoeCombine& p, hipStream_t st) {
  // one vector a lane where a row has no more (16384 x 2 rows of 256: 8.9 us against
  // 10.4 with two, 16384 x 8 FP32 rows of 512 53.9 against 63.0)
  const bool narrow = p.N <= 512;
  const int chunks = narrow ? 1 : (p.N + 1023) / 1024;
  return by_tokens(p, most_blocks(256) * 4 / chunks, [&](const MoeCombine& p) {
    const dim3 grid(static_cast<unsigned>((p.T * chunks + 3) / 4)), block(256);
    if (p.y_f32 && narrow) hipLaunchKernelGGL((moe_combine_kernel<true, 1>), grid, block, 0, st, p, chunks);
    else if (p.y_f32) hipLaunchKernelGGL((moe_combine_kernel<true, 2>), grid, block, 0, st, p, chunks);
    else if (narrow) hipLaunchKernelGGL((moe_combine_kernel<false, 1>), grid, block, 0, st, p, chunks);
    else hipLaunchKernelGGL((moe_combine_kernel<false, 2>), grid, block, 0, st, p, chunks);
    return hipGetLastError();
  });
}

hipError_t launch_moe_combine_bwd(const MoeCombineBwd& p, hipStream_t st) {
  // four vectors a lane where there are tokens enough (1024 x 8 rows of 7168: 33.7 us
  // against 37.9, 8191 x 2 90.7 against 91.8), two for few (16 x 8: 8.1 against 9.0);
  // one where a row has no more
  const int V = p.N <= 512 ? 1 : p.T >= 512 && p.N > 1024 ? 4 : 2;
  const Tokens g = tokens_of(p.N, V, V == 4 ? 8 : 16);
  return by_tokens(p, g.most(), [&](const MoeCombineBwd& p) {
    const dim3 grid = g.grid(p.T), block(g.threads);
#define FP8BS_COMBINE(F32, V) hipLaunchKernelGGL((moe_combine_bwd_kernel<F32, V>), grid, block, 0, st, p)
    if (p.y_f32) {
      if (V == 1) FP8BS_COMBINE(true, 1);
      else if (V == 2) FP8BS_COMBINE(true, 2);
      else FP8BS_COMBINE(true, 4);
    } else {
      if (V == 1) FP8BS_COMBINE(false, 1);
      else if (V == 2) FP8BS_COMBINE(false, 2);
      else FP8BS_COMBINE(false, 4);
    }
#undef FP8BS_COMBINE
    return hipGetLastError();
  });
}

}  // namespace fp8bs
