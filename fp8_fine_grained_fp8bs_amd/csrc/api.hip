// api.hip -- the C ABI of libfp8bs: host-side argument checks and dispatch.
//
// Every check runs before the first HIP call, so a rejected call touches no
// device state.  Only after the checks pass is the current device queried
// (once per device, cached) and the kernel enqueued on the caller's stream.
#include <hip/hip_runtime.h>

#include <atomic>
#include <cmath>
#include <cstring>

#include "fp8bs.h"
#include "fp8bs_internal.h"

namespace {

constexpr int kMaxDevices = 64;
// 0 = unknown, 1 = gfx950, 2 = other architecture
std::atomic<int> g_dev_state[kMaxDevices];

// GEMM stride limits: a 256-row tile of codes or scales must span less than
// 4 GiB, so that 32-bit offsets from its first row reach every element.
constexpr int64_t kMaxCodeStride = int64_t(1) << 24;   // bytes per code row
constexpr int64_t kMaxScaleStride = int64_t(1) << 22;  // floats per scale row
constexpr int64_t kMaxRequantStride = int64_t(1) << 25;  // bytes per input row: requant, transpose

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

fp8bs_status check_device() {
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0) {
    (void)hipGetLastError();
    return FP8BS_ERR_NO_DEVICE;
  }
  if (dev >= kMaxDevices) return FP8BS_ERR_NO_DEVICE;
  int st = g_dev_state[dev].load(std::memory_order_acquire);
  if (st == 0) {
    hipDeviceProp_t prop;
    if (hipGetDeviceProperties(&prop, dev) != hipSuccess) {
      (void)hipGetLastError();
      return FP8BS_ERR_NO_DEVICE;
    }
    st = (std::strncmp(prop.gcnArchName, "gfx950", 6) == 0) ? 1 : 2;
    g_dev_state[dev].store(st, std::memory_order_release);
  }
  return st == 1 ? FP8BS_OK : FP8BS_ERR_NO_DEVICE;
}

fp8bs_status launched(hipError_t e) {
  if (e != hipSuccess) {
    (void)hipGetLastError();
    return FP8BS_ERR_LAUNCH;
  }
  return FP8BS_OK;
}

// Common checks of a row-major operand: stride and alignment.
fp8bs_status check_matrix(const void* p, int64_t cols, int64_t ld, int64_t elem_bytes) {
  if (p == nullptr) return FP8BS_ERR_INVALID_ARG;
  if (ld < cols) return FP8BS_ERR_INVALID_ARG;
  if (!aligned(p, 16) || (ld * elem_bytes) % 16 != 0) return FP8BS_ERR_MISALIGNED;
  return FP8BS_OK;
}

fp8bs_status check_scales(const float* p, int64_t cols, int64_t ld) {
  if (p == nullptr) return FP8BS_ERR_INVALID_ARG;
  if (ld < cols) return FP8BS_ERR_INVALID_ARG;
  if (!aligned(p, 4)) return FP8BS_ERR_MISALIGNED;
  return FP8BS_OK;
}

// Attention limits: heads, head dims of the rotation, and what a 32-bit
// position, row or page number reaches.
constexpr int64_t kMaxHeads = int64_t(1) << 16;
constexpr int64_t kMaxHeadDim = 512;
constexpr int64_t kMaxInt32 = 0x7fffffff;
constexpr int64_t kMaxTokens = int64_t(1) << 30;   // of a sequence: positions a little past its end still fit 32 bits

fp8bs_status check_rotation(int64_t rot, int64_t off, fp8bs_rope_layout layout, int64_t D) {
  if (layout != FP8BS_ROPE_HALF && layout != FP8BS_ROPE_INTERLEAVED) return FP8BS_ERR_INVALID_ARG;
  if (rot <= 0 || off < 0) return FP8BS_ERR_INVALID_ARG;
  if (D % 16 != 0 || D > kMaxHeadDim || rot % 16 != 0 || off % 8 != 0 || off > D - rot)
    return FP8BS_ERR_UNSUPPORTED_SHAPE;
  return FP8BS_OK;
}

fp8bs_status check_table(const float* cs, int64_t n_pos) {
  if (cs == nullptr || n_pos <= 0 || n_pos > kMaxInt32) return FP8BS_ERR_INVALID_ARG;
  if (!aligned(cs, 16)) return FP8BS_ERR_MISALIGNED;
  return FP8BS_OK;
}

// Packed rows of a batch.
fp8bs_status check_packing(const int32_t* q_off, int64_t B, int64_t T, int64_t max_q) {
  if (B < 0 || T < 0 || max_q < 0) return FP8BS_ERR_INVALID_ARG;
  if (B > kMaxInt32 || T > kMaxInt32) return FP8BS_ERR_UNSUPPORTED_SHAPE;
  if (T > 0 && B > 0 && max_q == 0) return FP8BS_ERR_INVALID_ARG;
  if (q_off == nullptr && T != B) return FP8BS_ERR_INVALID_ARG;
  return FP8BS_OK;
}

// Rows of a key/value head (tokens times query heads) are numbered in 32 bits.
fp8bs_status check_heads(int64_t Hq, int64_t Hkv, int64_t T) {
  if (Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0) return FP8BS_ERR_INVALID_ARG;
  if (Hq > kMaxHeads || Hq / Hkv > 1024) return FP8BS_ERR_UNSUPPORTED_SHAPE;
  if (T > kMaxInt32 / (Hq / Hkv)) return FP8BS_ERR_UNSUPPORTED_SHAPE;
  return FP8BS_OK;
}

fp8bs_status check_cache_shape(int64_t D, int64_t page, int64_t max_pages, int64_t n_pages) {
  if (D <= 0 || page <= 0 || max_pages <= 0 || n_pages <= 0) return FP8BS_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return FP8BS_ERR_UNSUPPORTED_SHAPE;
  if (page != 16 && page != 32 && page != 64 && page != 128) return FP8BS_ERR_UNSUPPORTED_SHAPE;
  if (max_pages > kMaxTokens / page || n_pages > kMaxInt32) return FP8BS_ERR_UNSUPPORTED_SHAPE;
  return FP8BS_OK;
}

fp8bs_status check_cache(const int32_t* q_off, const int32_t* kv_len, const int32_t* table, int64_t ldt,
                         int64_t max_pages, const uint8_t* kc, const float* ks, const uint8_t* vc,
                         const float* vs) {
  if (kv_len == nullptr || table == nullptr || kc == nullptr || ks == nullptr || vc == nullptr || vs == nullptr)
    return FP8BS_ERR_INVALID_ARG;
  if (ldt < max_pages) return FP8BS_ERR_INVALID_ARG;
  if (!aligned(q_off, 4) || !aligned(kv_len, 4) || !aligned(table, 4) || !aligned(ks, 4) || !aligned(vs, 4) ||
      !aligned(kc, 16) || !aligned(vc, 16))
    return FP8BS_ERR_MISALIGNED;
  return FP8BS_OK;
}

// Rows of the norm live in a workgroup's registers.
constexpr int64_t kMaxNormWidth = 16384;
// Assignments of a sort are numbered in 32 bits, its counts' sums too.
constexpr int64_t kMaxAssignments = int64_t(1) << 30;

fp8bs_status check_type(fp8bs_out_dtype t) {
  return t == FP8BS_OUT_BF16 || t == FP8BS_OUT_F32 ? FP8BS_OK : FP8BS_ERR_INVALID_ARG;
}

fp8bs_status check_norm_sizes(int64_t T, int64_t C) {
  if (T < 0 || C <= 0) return FP8BS_ERR_INVALID_ARG;
  if (C % 128 != 0 || C > kMaxNormWidth || T > kMaxInt32) return FP8BS_ERR_UNSUPPORTED_SHAPE;
  return FP8BS_OK;
}

fp8bs_status check_gamma(const void* gamma, fp8bs_out_dtype gt) {
  if (gamma == nullptr || check_type(gt) != FP8BS_OK) return FP8BS_ERR_INVALID_ARG;
  return aligned(gamma, 16) ? FP8BS_OK : FP8BS_ERR_MISALIGNED;
}

// An output that may be an input itself, but not one with other rows.
fp8bs_status check_in_place(const void* out, int64_t ldo, const void* in, int64_t ldi) {
  return out != nullptr && out == in && ldo != ldi ? FP8BS_ERR_INVALID_ARG : FP8BS_OK;
}

// Codes with their scales, both or neither.
fp8bs_status check_codes(const uint8_t* q, int64_t ldq, const float* s, int64_t lds, int64_t cols) {
  if ((q == nullptr) != (s == nullptr)) return FP8BS_ERR_INVALID_ARG;
  if (q == nullptr) return FP8BS_OK;
  const fp8bs_status st = check_matrix(q, cols, ldq, 1);
  return st != FP8BS_OK ? st : check_scales(s, cols / 128, lds);
}

fp8bs_status check_choices(int64_t T, int64_t k, int64_t M) {
  if (T < 0 || k <= 0 || M < 0) return FP8BS_ERR_INVALID_ARG;
  if (k > fp8bs::kMaxChoices || T > kMaxInt32 || M > kMaxInt32) return FP8BS_ERR_UNSUPPORTED_SHAPE;
  return FP8BS_OK;
}

fp8bs_status check_columns(int64_t C) {
  if (C <= 0) return FP8BS_ERR_INVALID_ARG;
  return C % 128 == 0 && C <= kMaxInt32 - 65536 ? FP8BS_OK : FP8BS_ERR_UNSUPPORTED_SHAPE;   // columns in 32 bits
}

fp8bs_status check_sort_sizes(int64_t T, int64_t k, int64_t E) {
  const fp8bs_status st = check_choices(T, k, 0);
  if (st != FP8BS_OK) return st;
  if (E <= 0) return FP8BS_ERR_INVALID_ARG;
  return E <= fp8bs::kMaxExperts && T <= kMaxAssignments / k ? FP8BS_OK : FP8BS_ERR_UNSUPPORTED_SHAPE;
}

#define FP8BS_TRY(expr)                 \
  do {                                  \
    fp8bs_status _s = (expr);           \
    if (_s != FP8BS_OK) return _s;      \
  } while (0)

// The sort's arguments, checked.
fp8bs_status sort_of(const void* ids, fp8bs_index_type it, int64_t ldi, int64_t T, int64_t k, int64_t first, int64_t E,
                     int64_t M, int32_t* offsets, int32_t* slot, void* ws, int64_t ws_bytes, fp8bs::MoeIds& p) {
  if (it != FP8BS_INDEX_I32 && it != FP8BS_INDEX_I64) return FP8BS_ERR_INVALID_ARG;
  FP8BS_TRY(check_sort_sizes(T, k, E));
  FP8BS_TRY(check_choices(T, k, M));
  if (first < 0 || offsets == nullptr) return FP8BS_ERR_INVALID_ARG;
  if (!aligned(offsets, 4) || !aligned(ws, 4)) return FP8BS_ERR_MISALIGNED;
  if (T > 0) {
    if (ids == nullptr || slot == nullptr || ldi < k) return FP8BS_ERR_INVALID_ARG;
    if (!aligned(ids, it == FP8BS_INDEX_I64 ? 8 : 4) || !aligned(slot, 4)) return FP8BS_ERR_MISALIGNED;
    const int64_t need = fp8bs_moe_sort_ws(T, k, E);
    if (ws_bytes < need || (need > 0 && ws == nullptr)) return FP8BS_ERR_INVALID_ARG;
  }
  p.ids = ids;
  p.wide = it == FP8BS_INDEX_I64;
  p.ldi = ldi;
  p.T = T;
  p.k = static_cast<int>(k);
  p.first = first;
  p.E = static_cast<int>(E);
  p.offsets = offsets;
  p.slot = slot;
  p.M = M;
  p.ws = static_cast<int32_t*>(ws);
  return FP8BS_OK;
}

// The arguments of rows to their places, checked (those of T > 0 tokens).
fp8bs_status rows_of(fp8bs_requant_src src, const void* x, int64_t ldx, const float* s_in, int64_t lds_in, int64_t T,
                     int64_t C, const int32_t* slot, int64_t k, uint8_t* q, int64_t ldq, float* s, int64_t lds, void* y,
                     int64_t ldy, int64_t M, fp8bs::MoeRows& p) {
  if (src != FP8BS_SRC_FP8_1x128 && src != FP8BS_SRC_BF16) return FP8BS_ERR_INVALID_ARG;
  const bool codes = src == FP8BS_SRC_FP8_1x128;
  FP8BS_TRY(check_choices(T, k, M));
  FP8BS_TRY(check_columns(C));
  if ((q == nullptr && y == nullptr) || (codes && y != nullptr)) return FP8BS_ERR_INVALID_ARG;
  FP8BS_TRY(check_codes(q, ldq, s, lds, C));
  if (y != nullptr) FP8BS_TRY(check_matrix(y, C, ldy, 2));
  if (T > 0) {
    FP8BS_TRY(check_matrix(x, C, ldx, codes ? 1 : 2));
    if (codes) FP8BS_TRY(check_scales(s_in, C / 128, lds_in));
    if (slot == nullptr) return FP8BS_ERR_INVALID_ARG;
    if (!aligned(slot, 4)) return FP8BS_ERR_MISALIGNED;
  }
  p.codes_in = codes;
  p.x = x;
  p.ldx = ldx;
  p.s_in = s_in;
  p.lds_in = lds_in;
  p.T = T;
  p.C = static_cast<int>(C);
  p.slot = slot;
  p.k = static_cast<int>(k);
  p.q = q;
  p.ldq = ldq;
  p.s = s;
  p.lds = lds;
  p.y = static_cast<uint16_t*>(y);
  p.ldy = ldy;
  p.M = M;
  return FP8BS_OK;
}

}  // namespace

extern "C" {

const char* fp8bs_status_string(fp8bs_status st) {
  switch (st) {
    case FP8BS_OK: return "FP8BS_OK";
    case FP8BS_ERR_INVALID_ARG: return "FP8BS_ERR_INVALID_ARG";
    case FP8BS_ERR_UNSUPPORTED_SHAPE: return "FP8BS_ERR_UNSUPPORTED_SHAPE";
    case FP8BS_ERR_MISALIGNED: return "FP8BS_ERR_MISALIGNED";
    case FP8BS_ERR_NO_DEVICE: return "FP8BS_ERR_NO_DEVICE";
    case FP8BS_ERR_LAUNCH: return "FP8BS_ERR_LAUNCH";
  }
  return "FP8BS_ERR_UNKNOWN";
}

int fp8bs_version(void) { return 100; }

fp8bs_status fp8bs_quant_act_1x128(const void* x, int64_t M, int64_t K, int64_t ldx,
                                   uint8_t* q, int64_t ldq, float* s, int64_t lds,
                                   void* stream) {
  if (M < 0 || K <= 0) return FP8BS_ERR_INVALID_ARG;
  if (K % 128 != 0) return FP8BS_ERR_UNSUPPORTED_SHAPE;
  if (M == 0) return FP8BS_OK;
  FP8BS_TRY(check_matrix(x, K, ldx, 2));
  FP8BS_TRY(check_matrix(q, K, ldq, 1));
  FP8BS_TRY(check_scales(s, K / 128, lds));
  FP8BS_TRY(check_device());
  return launched(fp8bs::launch_quant_act_1x128(static_cast<const uint16_t*>(x), M, K, ldx, q, ldq,
                                                s, lds, static_cast<hipStream_t>(stream)));
}

fp8bs_status fp8bs_quant_act_w(const void* x, int64_t M, int64_t ldx, uint8_t* qx, int64_t ldqx,
                               float* sx, int64_t ldsx, const void* w, int64_t N, int64_t ldw,
                               uint8_t* qw, int64_t ldqw, float* sw, int64_t ldsw, int64_t K,
                               void* stream) {
  if (M < 0 || N < 0 || K <= 0) return FP8BS_ERR_INVALID_ARG;
  if (K % 128 != 0) return FP8BS_ERR_UNSUPPORTED_SHAPE;
  if (M == 0 && N == 0) return FP8BS_OK;
  if (M > 0) {
    FP8BS_TRY(check_matrix(x, K, ldx, 2));
    FP8BS_TRY(check_matrix(qx, K, ldqx, 1));
    FP8BS_TRY(check_scales(sx, K / 128, ldsx));
  }
  if (N > 0) {
    FP8BS_TRY(check_matrix(w, K, ldw, 2));
    FP8BS_TRY(check_matrix(qw, K, ldqw, 1));
    FP8BS_TRY(check_scales(sw, K / 128, ldsw));
  }
  FP8BS_TRY(check_device());
  return launched(fp8bs::launch_quant_act_w(static_cast<const uint16_t*>(x), M, ldx, qx, ldqx, sx, ldsx,
                                            static_cast<const uint16_t*>(w), N, ldw, qw, ldqw, sw, ldsw,
                                            K, static_cast<hipStream_t>(stream)));
}

fp8bs_status fp8bs_quant_w_128x128(const void* w, int64_t N, int64_t K, int64_t ldw,
                                   uint8_t* q, int64_t ldq, float* s, int64_t lds,
                                   void* stream) {
  if (N < 0 || K <= 0) return FP8BS_ERR_INVALID_ARG;
  if (K % 128 != 0) return FP8BS_ERR_UNSUPPORTED_SHAPE;
  if (N == 0) return FP8BS_OK;
  FP8BS_TRY(check_matrix(w, K, ldw, 2));
  FP8BS_TRY(check_matrix(q, K, ldq, 1));
  FP8BS_TRY(check_scales(s, K / 128, lds));
  FP8BS_TRY(check_device());
  return launched(fp8bs::launch_quant_w_128x128(static_cast<const uint16_t*>(w), N, K, ldw, q, ldq,
                                                s, lds, static_cast<hipStream_t>(stream)));
}

fp8bs_status fp8bs_quant_per_tensor(const void* x, int64_t n, uint8_t* q, float* s, void* stream) {
  if (n < 0) return FP8BS_ERR_INVALID_ARG;
  if (n % 128 != 0) return FP8BS_ERR_UNSUPPORTED_SHAPE;
  if (n == 0) return FP8BS_OK;
  if (x == nullptr || q == nullptr || s == nullptr) return FP8BS_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(q, 16) || !aligned(s, 4)) return FP8BS_ERR_MISALIGNED;
  FP8BS_TRY(check_device());
  return launched(fp8bs::launch_quant_per_tensor(static_cast<const uint16_t*>(x), n, q, s,
                                                 static_cast<hipStream_t>(stream)));
}

fp8bs_status fp8bs_cast_e4m3(const float* x, int64_t n, uint8_t* q, void* stream) {
  if (n < 0) return FP8BS_ERR_INVALID_ARG;
  if (n == 0) return FP8BS_OK;
  if (x == nullptr || q == nullptr) return FP8BS_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(q, 16)) return FP8BS_ERR_MISALIGNED;
  FP8BS_TRY(check_device());
  return launched(fp8bs::launch_cast_e4m3(x, n, q, static_cast<hipStream_t>(stream)));
}

fp8bs_status fp8bs_encode_e5m6(const void* x, int64_t T, int64_t C, int64_t ldx, uint8_t* y,
                               int64_t ldy, void* stream) {
  if (T < 0 || C <= 0) return FP8BS_ERR_INVALID_ARG;
  if (C % 128 != 0) return FP8BS_ERR_UNSUPPORTED_SHAPE;
  if (T == 0) return FP8BS_OK;
  FP8BS_TRY(check_matrix(x, C, ldx, 2));
  FP8BS_TRY(check_matrix(y, C / 2 * 3, ldy, 1));
  FP8BS_TRY(check_device());
  return launched(fp8bs::launch_encode_e5m6(static_cast<const uint16_t*>(x), T, C, ldx, y, ldy,
                                            static_cast<hipStream_t>(stream)));
}

fp8bs_status fp8bs_decode_e5m6(const uint8_t* y, int64_t T, int64_t C, int64_t ldy, void* x,
                               int64_t ldx, void* stream) {
  if (T < 0 || C <= 0) return FP8BS_ERR_INVALID_ARG;
  if (C % 128 != 0) return FP8BS_ERR_UNSUPPORTED_SHAPE;
  if (T == 0) return FP8BS_OK;
  FP8BS_TRY(check_matrix(y, C / 2 * 3, ldy, 1));
  FP8BS_TRY(check_matrix(x, C, ldx, 2));
  FP8BS_TRY(check_device());
  return launched(fp8bs::launch_decode_e5m6(y, T, C, ldy, static_cast<uint16_t*>(x), ldx,
                                            static_cast<hipStream_t>(stream)));
}

fp8bs_status fp8bs_swiglu_quant_1x128(const void* g, int64_t ldg, const void* u, int64_t ldu,
                                      int64_t T, int64_t I, uint8_t* q, int64_t ldq, float* s,
                                      int64_t lds, void* h, int64_t ldh, void* stream) {
  if (T < 0 || I <= 0) return FP8BS_ERR_INVALID_ARG;
  if (I % 128 != 0) return FP8BS_ERR_UNSUPPORTED_SHAPE;
  if ((q == nullptr) != (s == nullptr)) return FP8BS_ERR_INVALID_ARG;
  if (q == nullptr && h == nullptr) return FP8BS_ERR_INVALID_ARG;
  if (T == 0) return FP8BS_OK;
  FP8BS_TRY(check_matrix(g, I, ldg, 2));
  FP8BS_TRY(check_matrix(u, I, ldu, 2));
  if (q != nullptr) {
    FP8BS_TRY(check_matrix(q, I, ldq, 1));
    FP8BS_TRY(check_scales(s, I / 128, lds));
  }
  if (h != nullptr) FP8BS_TRY(check_matrix(h, I, ldh, 2));
  FP8BS_TRY(check_device());
  return launched(fp8bs::launch_swiglu_quant_1x128(static_cast<const uint16_t*>(g), ldg,
                                                   static_cast<const uint16_t*>(u), ldu, T, I, q, ldq, s,
                                                   lds, static_cast<uint16_t*>(h), ldh,
                                                   static_cast<hipStream_t>(stream)));
}

fp8bs_status fp8bs_requant_T_128x1(fp8bs_requant_src src, const void* in, const float* s_in,
                                   int64_t T, int64_t C, int64_t ld_in, int64_t lds_in,
                                   uint8_t* q_out, int64_t ld_out, float* s_out, int64_t lds_out,
                                   void* stream) {
  if (src != FP8BS_SRC_FP8_1x128 && src != FP8BS_SRC_BF16 && src != FP8BS_SRC_E5M6)
    return FP8BS_ERR_INVALID_ARG;
  if (T < 0 || C <= 0) return FP8BS_ERR_INVALID_ARG;
  if (C % 128 != 0) return FP8BS_ERR_UNSUPPORTED_SHAPE;
  if (T == 0) return FP8BS_OK;
  const bool codes = (src == FP8BS_SRC_FP8_1x128);
  // an input row: C codes, C bf16 values, or 1.5 C bytes of E5M6 (ld_in in bytes)
  const int64_t row_bytes = src == FP8BS_SRC_BF16 ? 2 * C : src == FP8BS_SRC_E5M6 ? C / 2 * 3 : C;
  const int64_t elem = src == FP8BS_SRC_BF16 ? 2 : 1;
  FP8BS_TRY(check_matrix(in, row_bytes / elem, ld_in, elem));
  if (codes) FP8BS_TRY(check_scales(s_in, C / 128, lds_in));
  FP8BS_TRY(check_matrix(q_out, T, ld_out, 1));
  FP8BS_TRY(check_scales(s_out, (T + 127) / 128, lds_out));
  // 128-token tiles are addressed with 32-bit offsets from their first row
  if (ld_in * elem >= kMaxRequantStride || (codes && lds_in >= kMaxScaleStride))
    return FP8BS_ERR_UNSUPPORTED_SHAPE;
  FP8BS_TRY(check_device());
  return launched(fp8bs::launch_requant_T_128x1(static_cast<int>(src), in, s_in, T, C, ld_in, lds_in, q_out, ld_out,
                                                s_out, lds_out, static_cast<hipStream_t>(stream)));
}

fp8bs_status fp8bs_transpose_w_128x128(const uint8_t* q, int64_t N, int64_t K, int64_t ldq,
                                       const float* s, int64_t lds, uint8_t* qt, int64_t ldqt,
                                       float* st, int64_t ldst, void* stream) {
  if (N < 0 || K <= 0) return FP8BS_ERR_INVALID_ARG;
  if (N % 128 != 0 || K % 128 != 0) return FP8BS_ERR_UNSUPPORTED_SHAPE;
  if (N == 0) return FP8BS_OK;
  FP8BS_TRY(check_matrix(q, K, ldq, 1));
  FP8BS_TRY(check_scales(s, K / 128, lds));
  FP8BS_TRY(check_matrix(qt, N, ldqt, 1));
  FP8BS_TRY(check_scales(st, N / 128, ldst));
  // 128-row blocks are addressed with 32-bit offsets from their first row
  if (ldq >= kMaxRequantStride) return FP8BS_ERR_UNSUPPORTED_SHAPE;
  FP8BS_TRY(check_device());
  return launched(fp8bs::launch_transpose_w_128x128(q, N, K, ldq, s, lds, qt, ldqt, st, ldst,
                                                    static_cast<hipStream_t>(stream)));
}

fp8bs_status fp8bs_gemm(const uint8_t* a, const float* sa, int64_t lda, int64_t ldsa,
                        const uint8_t* b, const float* sb, int64_t ldb, int64_t ldsb,
                        fp8bs_bscale bmode, void* d, int64_t ldd, fp8bs_out_dtype dt,
                        int64_t M, int64_t N, int64_t K, void* stream) {
  if (bmode != FP8BS_BSCALE_BLOCK_128x128 && bmode != FP8BS_BSCALE_ROW_1x128)
    return FP8BS_ERR_INVALID_ARG;
  if (dt != FP8BS_OUT_BF16 && dt != FP8BS_OUT_F32) return FP8BS_ERR_INVALID_ARG;
  if (M < 0 || N < 0 || K <= 0) return FP8BS_ERR_INVALID_ARG;
  if (K % 128 != 0) return FP8BS_ERR_UNSUPPORTED_SHAPE;
  if (M == 0 || N == 0) return FP8BS_OK;
  FP8BS_TRY(check_matrix(a, K, lda, 1));
  FP8BS_TRY(check_matrix(b, K, ldb, 1));
  FP8BS_TRY(check_scales(sa, K / 128, ldsa));
  FP8BS_TRY(check_scales(sb, K / 128, ldsb));
  FP8BS_TRY(check_matrix(d, N, ldd, dt == FP8BS_OUT_F32 ? 4 : 2));
  // tiles are addressed with 32-bit offsets from their first row
  if (lda >= kMaxCodeStride || ldb >= kMaxCodeStride || ldsa >= kMaxScaleStride ||
      ldsb >= kMaxScaleStride)
    return FP8BS_ERR_UNSUPPORTED_SHAPE;
  FP8BS_TRY(check_device());
  return launched(fp8bs::launch_gemm(a, sa, lda, ldsa, b, sb, ldb, ldsb,
                                     bmode == FP8BS_BSCALE_ROW_1x128, d, ldd, nullptr, 0,
                                     dt == FP8BS_OUT_F32 ? 1 : 0, M, N, K,
                                     static_cast<hipStream_t>(stream)));
}

fp8bs_status fp8bs_gemm_quant_1x128(const uint8_t* a, const float* sa, int64_t lda, int64_t ldsa,
                                    const uint8_t* b, const float* sb, int64_t ldb, int64_t ldsb,
                                    fp8bs_bscale bmode, uint8_t* q, int64_t ldq, float* s,
                                    int64_t lds, int64_t M, int64_t N, int64_t K, void* stream) {
  if (bmode != FP8BS_BSCALE_BLOCK_128x128 && bmode != FP8BS_BSCALE_ROW_1x128)
    return FP8BS_ERR_INVALID_ARG;
  if (M < 0 || N < 0 || K <= 0) return FP8BS_ERR_INVALID_ARG;
  if (K % 128 != 0 || N % 128 != 0) return FP8BS_ERR_UNSUPPORTED_SHAPE;
  if (M == 0 || N == 0) return FP8BS_OK;
  FP8BS_TRY(check_matrix(a, K, lda, 1));
  FP8BS_TRY(check_matrix(b, K, ldb, 1));
  FP8BS_TRY(check_scales(sa, K / 128, ldsa));
  FP8BS_TRY(check_scales(sb, K / 128, ldsb));
  FP8BS_TRY(check_matrix(q, N, ldq, 1));
  FP8BS_TRY(check_scales(s, N / 128, lds));
  if (lda >= kMaxCodeStride || ldb >= kMaxCodeStride || ldsa >= kMaxScaleStride ||
      ldsb >= kMaxScaleStride)
    return FP8BS_ERR_UNSUPPORTED_SHAPE;
  FP8BS_TRY(check_device());
  return launched(fp8bs::launch_gemm(a, sa, lda, ldsa, b, sb, ldb, ldsb,
                                     bmode == FP8BS_BSCALE_ROW_1x128, q, ldq, s, lds, 2, M, N, K,
                                     static_cast<hipStream_t>(stream)));
}

fp8bs_status fp8bs_gemm_bf16a(const void* x, int64_t ldx, uint8_t* qx, int64_t ldqx, float* sx,
                              int64_t ldsx, const uint8_t* b, const float* sb, int64_t ldb, int64_t ldsb,
                              void* d, int64_t ldd, fp8bs_out_dtype dt, int64_t M, int64_t N, int64_t K,
                              void* stream) {
  if (dt != FP8BS_OUT_BF16 && dt != FP8BS_OUT_F32) return FP8BS_ERR_INVALID_ARG;
  if (M < 0 || N < 0 || K <= 0) return FP8BS_ERR_INVALID_ARG;
  if (K % 128 != 0) return FP8BS_ERR_UNSUPPORTED_SHAPE;
  if ((qx == nullptr) != (sx == nullptr)) return FP8BS_ERR_INVALID_ARG;
  if (M == 0 || N == 0) return FP8BS_OK;
  FP8BS_TRY(check_matrix(x, K, ldx, 2));
  FP8BS_TRY(check_matrix(b, K, ldb, 1));
  FP8BS_TRY(check_scales(sb, K / 128, ldsb));
  FP8BS_TRY(check_matrix(d, N, ldd, dt == FP8BS_OUT_F32 ? 4 : 2));
  if (qx != nullptr) {
    FP8BS_TRY(check_matrix(qx, K, ldqx, 1));
    FP8BS_TRY(check_scales(sx, K / 128, ldsx));
  }
  // 64-row tiles of bf16 A and 256-row tiles of codes are addressed with
  // 32-bit offsets from their first row
  if (ldx >= kMaxCodeStride / 2 || ldb >= kMaxCodeStride || ldsb >= kMaxScaleStride)
    return FP8BS_ERR_UNSUPPORTED_SHAPE;
  FP8BS_TRY(check_device());
  return launched(fp8bs::launch_gemm_bf16a(static_cast<const uint16_t*>(x), ldx, qx, ldqx, sx, ldsx, b, sb,
                                           ldb, ldsb, d, ldd, dt == FP8BS_OUT_F32, M, N, K,
                                           static_cast<hipStream_t>(stream)));
}

fp8bs_status fp8bs_grouped_gemm(const uint8_t* a, const float* sa, int64_t ldsa,
                                const uint8_t* b, const float* sb,
                                const int32_t* offsets, int32_t E, int64_t M_total,
                                void* d, fp8bs_out_dtype dt, int64_t N, int64_t K,
                                void* stream) {
  if (dt != FP8BS_OUT_BF16 && dt != FP8BS_OUT_F32) return FP8BS_ERR_INVALID_ARG;
  if (E < 1 || M_total < 0 || N <= 0 || K <= 0) return FP8BS_ERR_INVALID_ARG;
  if (K % 128 != 0) return FP8BS_ERR_UNSUPPORTED_SHAPE;
  if (offsets == nullptr || b == nullptr || sb == nullptr) return FP8BS_ERR_INVALID_ARG;
  if (!aligned(offsets, 4) || !aligned(sb, 4) || !aligned(b, 16)) return FP8BS_ERR_MISALIGNED;
  if (M_total == 0) return FP8BS_OK;
  FP8BS_TRY(check_matrix(a, K, K, 1));
  FP8BS_TRY(check_scales(sa, K / 128, ldsa));
  FP8BS_TRY(check_matrix(d, N, N, dt == FP8BS_OUT_F32 ? 4 : 2));
  if (K >= kMaxCodeStride || ldsa >= kMaxScaleStride) return FP8BS_ERR_UNSUPPORTED_SHAPE;
  FP8BS_TRY(check_device());
  return launched(fp8bs::launch_grouped_gemm(a, sa, ldsa, b, sb, offsets, E, M_total, d,
                                             dt == FP8BS_OUT_F32, N, K,
                                             static_cast<hipStream_t>(stream)));
}

fp8bs_status fp8bs_rope_table(float* cs, int64_t n_pos, int64_t rot, double base, double factor,
                              double orig_len, double turns_lo, double turns_hi, double mscale,
                              void* stream) {
  if (n_pos < 0 || rot <= 0) return FP8BS_ERR_INVALID_ARG;
  if (!(base > 0.0 && factor > 0.0 && orig_len >= 0.0) || !std::isfinite(base) || !std::isfinite(factor) ||
      !std::isfinite(orig_len) || !std::isfinite(mscale))
    return FP8BS_ERR_INVALID_ARG;
  if (orig_len > 0.0 && !(turns_hi > turns_lo && std::isfinite(turns_hi) && std::isfinite(turns_lo)))
    return FP8BS_ERR_INVALID_ARG;
  if (rot % 16 != 0 || rot > kMaxHeadDim) return FP8BS_ERR_UNSUPPORTED_SHAPE;
  if (n_pos > kMaxInt32) return FP8BS_ERR_UNSUPPORTED_SHAPE;
  if (n_pos == 0) return FP8BS_OK;
  if (cs == nullptr) return FP8BS_ERR_INVALID_ARG;
  if (!aligned(cs, 16)) return FP8BS_ERR_MISALIGNED;
  FP8BS_TRY(check_device());
  return launched(fp8bs::launch_rope_table(cs, n_pos, rot, base, factor, orig_len, turns_lo, turns_hi, mscale,
                                           static_cast<hipStream_t>(stream)));
}

fp8bs_status fp8bs_rope(const void* x, int64_t ldx, void* y, int64_t ldy, const int32_t* pos, int64_t T,
                        int64_t H, int64_t D, int64_t rot, int64_t rot_off, fp8bs_rope_layout layout,
                        int inverse, const float* cs, int64_t n_pos, void* stream) {
  if (T < 0 || H <= 0 || D <= 0) return FP8BS_ERR_INVALID_ARG;
  FP8BS_TRY(check_rotation(rot, rot_off, layout, D));
  if (H > kMaxHeads) return FP8BS_ERR_UNSUPPORTED_SHAPE;
  if (T == 0) return FP8BS_OK;
  FP8BS_TRY(check_matrix(x, H * D, ldx, 2));
  FP8BS_TRY(check_matrix(y, H * D, ldy, 2));
  if (x == y && ldx != ldy) return FP8BS_ERR_INVALID_ARG;
  FP8BS_TRY(check_table(cs, n_pos));
  if (pos == nullptr) return FP8BS_ERR_INVALID_ARG;
  if (!aligned(pos, 4)) return FP8BS_ERR_MISALIGNED;
  FP8BS_TRY(check_device());
  return launched(fp8bs::launch_rope(static_cast<const uint16_t*>(x), ldx, static_cast<uint16_t*>(y), ldy, pos, T,
                                     static_cast<int>(H), static_cast<int>(D), static_cast<int>(rot),
                                     static_cast<int>(rot_off), layout == FP8BS_ROPE_INTERLEAVED, inverse != 0, cs,
                                     n_pos, static_cast<hipStream_t>(stream)));
}

fp8bs_status fp8bs_kv_append(const void* q, int64_t ldq, void* q_out, int64_t ldqo, int64_t Hq,
                             const void* k, int64_t ldk, const void* v, int64_t ldv, int64_t Hkv, int64_t D,
                             const float* cs, int64_t n_pos, int64_t rot, int64_t rot_off,
                             fp8bs_rope_layout layout, const int32_t* q_off, const int32_t* kv_len, int64_t B,
                             int64_t T, int64_t max_q, const int32_t* table, int64_t ldt, int64_t max_pages,
                             int64_t page, uint8_t* kc, float* ks, uint8_t* vc, float* vs, int64_t n_pages,
                             void* stream) {
  if (Hkv <= 0 || (q != nullptr && Hq <= 0)) return FP8BS_ERR_INVALID_ARG;
  if (q != nullptr && cs == nullptr) return FP8BS_ERR_INVALID_ARG;
  if (Hkv > kMaxHeads || Hq > kMaxHeads) return FP8BS_ERR_UNSUPPORTED_SHAPE;
  if (cs != nullptr) FP8BS_TRY(check_rotation(rot, rot_off, layout, D));
  FP8BS_TRY(check_packing(q_off, B, T, max_q));
  FP8BS_TRY(check_cache_shape(D, page, max_pages, n_pages));
  if (T == 0 || B == 0) return FP8BS_OK;
  FP8BS_TRY(check_matrix(k, Hkv * D, ldk, 2));
  FP8BS_TRY(check_matrix(v, Hkv * D, ldv, 2));
  if (q != nullptr) {
    FP8BS_TRY(check_matrix(q, Hq * D, ldq, 2));
    FP8BS_TRY(check_matrix(q_out, Hq * D, ldqo, 2));
    if (q == q_out && ldq != ldqo) return FP8BS_ERR_INVALID_ARG;   // rows would overwrite others yet unread
  }
  if (cs != nullptr) FP8BS_TRY(check_table(cs, n_pos));
  FP8BS_TRY(check_cache(q_off, kv_len, table, ldt, max_pages, kc, ks, vc, vs));
  FP8BS_TRY(check_device());
  fp8bs::KvAppend p;
  p.q = static_cast<const uint16_t*>(q);
  p.ldq = ldq;
  p.q_out = static_cast<uint16_t*>(q_out);
  p.ldqo = ldqo;
  p.Hq = static_cast<int>(q != nullptr ? Hq : 0);
  p.k = static_cast<const uint16_t*>(k);
  p.ldk = ldk;
  p.v = static_cast<const uint16_t*>(v);
  p.ldv = ldv;
  p.Hkv = static_cast<int>(Hkv);
  p.D = static_cast<int>(D);
  p.cs = cs;
  p.n_pos = n_pos;
  p.rot = static_cast<int>(cs != nullptr ? rot : 0);
  p.rot_off = static_cast<int>(cs != nullptr ? rot_off : 0);
  p.interleaved = layout == FP8BS_ROPE_INTERLEAVED;
  p.q_off = q_off;
  p.kv_len = kv_len;
  p.B = static_cast<int>(B);
  p.T = T;
  p.max_q = max_q;
  p.table = table;
  p.ldt = ldt;
  p.max_pages = max_pages;
  p.page = static_cast<int>(page);
  p.kc = kc;
  p.ks = ks;
  p.vc = vc;
  p.vs = vs;
  p.n_pages = n_pages;
  return launched(fp8bs::launch_kv_append(p, static_cast<hipStream_t>(stream)));
}

int64_t fp8bs_attn_paged_ws(int64_t B, int64_t T, int64_t max_q, int64_t Hq, int64_t Hkv, int64_t D,
                            int64_t max_pages, int64_t page) {
  if (check_heads(Hq, Hkv, T) != FP8BS_OK || check_packing(nullptr, B, B, max_q) != FP8BS_OK || T < 0 ||
      T > kMaxInt32 || check_cache_shape(D, page, max_pages, 1) != FP8BS_OK)
    return -1;
  if (T == 0 || B == 0) return 0;
  return fp8bs::attn_paged_ws(B, T, max_q, static_cast<int>(Hq), static_cast<int>(Hkv), static_cast<int>(D),
                              max_pages, static_cast<int>(page));
}

fp8bs_status fp8bs_attn_paged(const void* q, int64_t ldq, void* out, int64_t ldo, float* lse, int64_t ldl,
                              const int32_t* q_off, const int32_t* kv_len, int64_t B, int64_t T, int64_t max_q,
                              int64_t Hq, int64_t Hkv, int64_t D, const int32_t* table, int64_t ldt,
                              int64_t max_pages, int64_t page, const uint8_t* kc, const float* ks,
                              const uint8_t* vc, const float* vs, int64_t n_pages, float scale, int causal,
                              int64_t window, void* ws, int64_t ws_bytes, void* stream) {
  FP8BS_TRY(check_heads(Hq, Hkv, T));
  if (!(scale > 0.0f) || !std::isfinite(scale) || window < 0) return FP8BS_ERR_INVALID_ARG;
  FP8BS_TRY(check_packing(q_off, B, T, max_q));
  FP8BS_TRY(check_cache_shape(D, page, max_pages, n_pages));
  if (T == 0 || B == 0) return FP8BS_OK;
  FP8BS_TRY(check_matrix(q, Hq * D, ldq, 2));
  FP8BS_TRY(check_matrix(out, Hq * D, ldo, 2));
  if (lse != nullptr) FP8BS_TRY(check_scales(lse, Hq, ldl));
  FP8BS_TRY(check_cache(q_off, kv_len, table, ldt, max_pages, kc, ks, vc, vs));
  const int64_t need = fp8bs_attn_paged_ws(B, T, max_q, Hq, Hkv, D, max_pages, page);
  if (ws_bytes < need || (need > 0 && ws == nullptr)) return FP8BS_ERR_INVALID_ARG;
  if (!aligned(ws, 16)) return FP8BS_ERR_MISALIGNED;
  FP8BS_TRY(check_device());
  fp8bs::AttnPaged p;
  p.q = static_cast<const uint16_t*>(q);
  p.ldq = ldq;
  p.out = static_cast<uint16_t*>(out);
  p.ldo = ldo;
  p.lse = lse;
  p.ldl = ldl;
  p.q_off = q_off;
  p.kv_len = kv_len;
  p.B = static_cast<int>(B);
  p.T = T;
  p.max_q = max_q;
  p.Hq = static_cast<int>(Hq);
  p.Hkv = static_cast<int>(Hkv);
  p.D = static_cast<int>(D);
  p.table = table;
  p.ldt = ldt;
  p.max_pages = max_pages;
  p.page = static_cast<int>(page);
  p.kc = kc;
  p.ks = ks;
  p.vc = vc;
  p.vs = vs;
  p.n_pages = n_pages;
  p.scale = scale;
  p.causal = causal != 0;
  p.window = window;
  p.ws = ws;
  return launched(fp8bs::launch_attn_paged(p, static_cast<hipStream_t>(stream)));
}

fp8bs_status fp8bs_rmsnorm_quant_1x128(const void* x, int64_t ldx, const void* r, int64_t ldr, const void* gamma,
                                       fp8bs_out_dtype gt, float eps, int64_t T, int64_t C, void* h, int64_t ldh,
                                       uint8_t* q, int64_t ldq, float* s, int64_t lds, void* y, int64_t ldy,
                                       float* rstd, void* stream) {
  FP8BS_TRY(check_norm_sizes(T, C));
  if (!(eps > 0.0f) || !std::isfinite(eps)) return FP8BS_ERR_INVALID_ARG;
  FP8BS_TRY(check_type(gt));
  if (T == 0) return FP8BS_OK;
  if ((r == nullptr) != (h == nullptr)) return FP8BS_ERR_INVALID_ARG;
  if (q == nullptr && y == nullptr) return FP8BS_ERR_INVALID_ARG;
  FP8BS_TRY(check_matrix(x, C, ldx, 2));
  FP8BS_TRY(check_gamma(gamma, gt));
  if (r != nullptr) {
    FP8BS_TRY(check_matrix(r, C, ldr, 2));
    FP8BS_TRY(check_matrix(h, C, ldh, 2));
    FP8BS_TRY(check_in_place(h, ldh, x, ldx));
    FP8BS_TRY(check_in_place(h, ldh, r, ldr));
  }
  FP8BS_TRY(check_codes(q, ldq, s, lds, C));
  if (y != nullptr) FP8BS_TRY(check_matrix(y, C, ldy, 2));
  if (!aligned(rstd, 4)) return FP8BS_ERR_MISALIGNED;
  FP8BS_TRY(check_device());
  fp8bs::RmsNorm p;
  p.x = static_cast<const uint16_t*>(x);
  p.ldx = ldx;
  p.r = static_cast<const uint16_t*>(r);
  p.ldr = ldr;
  p.gamma = gamma;
  p.gamma_f32 = gt == FP8BS_OUT_F32;
  p.eps = eps;
  p.T = T;
  p.C = static_cast<int>(C);
  p.h = static_cast<uint16_t*>(h);
  p.ldh = ldh;
  p.q = q;
  p.ldq = ldq;
  p.s = s;
  p.lds = lds;
  p.y = static_cast<uint16_t*>(y);
  p.ldy = ldy;
  p.rstd = rstd;
  return launched(fp8bs::launch_rmsnorm(p, static_cast<hipStream_t>(stream)));
}

int64_t fp8bs_rmsnorm_bwd_ws(int64_t T, int64_t C) {
  if (check_norm_sizes(T, C) != FP8BS_OK) return -1;
  return fp8bs::rmsnorm_bwd_ws(T, static_cast<int>(C));
}

fp8bs_status fp8bs_rmsnorm_bwd(const void* dn, int64_t lddn, const void* dres, int64_t lddr, const void* h,
                               int64_t ldh, const void* gamma, fp8bs_out_dtype gt, const float* rstd, int64_t T,
                               int64_t C, void* dx, int64_t lddx, float* dgamma, void* ws, int64_t ws_bytes,
                               void* stream) {
  FP8BS_TRY(check_norm_sizes(T, C));
  FP8BS_TRY(check_type(gt));
  if (!aligned(dgamma, 16) || !aligned(ws, 16)) return FP8BS_ERR_MISALIGNED;
  if (T == 0 && dgamma == nullptr) return FP8BS_OK;
  if (T > 0) {
    FP8BS_TRY(check_matrix(dn, C, lddn, 2));
    if (dres != nullptr) FP8BS_TRY(check_matrix(dres, C, lddr, 2));
    FP8BS_TRY(check_matrix(h, C, ldh, 2));
    FP8BS_TRY(check_matrix(dx, C, lddx, 2));
    FP8BS_TRY(check_gamma(gamma, gt));
    FP8BS_TRY(check_in_place(dx, lddx, dres, lddr));
    if (dx == dn || dx == h) return FP8BS_ERR_INVALID_ARG;   // other workgroups may read them for dgamma
    if (rstd == nullptr) return FP8BS_ERR_INVALID_ARG;
    if (!aligned(rstd, 4)) return FP8BS_ERR_MISALIGNED;
    const int64_t need = dgamma != nullptr ? fp8bs_rmsnorm_bwd_ws(T, C) : 0;
    if (ws_bytes < need || (need > 0 && ws == nullptr)) return FP8BS_ERR_INVALID_ARG;
  }
  FP8BS_TRY(check_device());
  fp8bs::RmsNormBwd p;
  p.dn = static_cast<const uint16_t*>(dn);
  p.lddn = lddn;
  p.dres = static_cast<const uint16_t*>(dres);
  p.lddr = lddr;
  p.h = static_cast<const uint16_t*>(h);
  p.ldh = ldh;
  p.gamma = gamma;
  p.gamma_f32 = gt == FP8BS_OUT_F32;
  p.rstd = rstd;
  p.T = T;
  p.C = static_cast<int>(C);
  p.dx = static_cast<uint16_t*>(dx);
  p.lddx = lddx;
  p.dgamma = dgamma;
  p.ws = static_cast<float*>(ws);
  return launched(fp8bs::launch_rmsnorm_bwd(p, static_cast<hipStream_t>(stream)));
}

int64_t fp8bs_moe_sort_ws(int64_t T, int64_t k, int64_t E) {
  if (check_sort_sizes(T, k, E) != FP8BS_OK) return -1;
  return fp8bs::moe_sort_ws(T, static_cast<int>(k), static_cast<int>(E));
}

fp8bs_status fp8bs_moe_sort(const void* ids, fp8bs_index_type it, int64_t ldi, int64_t T, int64_t k, int64_t first,
                            int64_t E, int64_t M, int32_t* offsets, int32_t* slot, void* ws, int64_t ws_bytes,
                            void* stream) {
  fp8bs::MoeIds p;
  FP8BS_TRY(sort_of(ids, it, ldi, T, k, first, E, M, offsets, slot, ws, ws_bytes, p));
  FP8BS_TRY(check_device());
  return launched(fp8bs::launch_moe_sort(p, static_cast<hipStream_t>(stream)));
}

fp8bs_status fp8bs_moe_gather(fp8bs_requant_src src, const void* x, int64_t ldx, const float* s_in, int64_t lds_in,
                              int64_t T, int64_t C, const int32_t* slot, int64_t k, uint8_t* q, int64_t ldq,
                              float* s, int64_t lds, void* y, int64_t ldy, int64_t M, void* stream) {
  fp8bs::MoeRows p;
  if (T == 0 || M == 0) {   // nothing to write: the buffers need not be there
    if (src != FP8BS_SRC_FP8_1x128 && src != FP8BS_SRC_BF16) return FP8BS_ERR_INVALID_ARG;
    FP8BS_TRY(check_choices(T, k, M));
    return check_columns(C);
  }
  FP8BS_TRY(rows_of(src, x, ldx, s_in, lds_in, T, C, slot, k, q, ldq, s, lds, y, ldy, M, p));
  FP8BS_TRY(check_device());
  return launched(fp8bs::launch_moe_gather(p, static_cast<hipStream_t>(stream)));
}

fp8bs_status fp8bs_moe_dispatch(fp8bs_requant_src src, const void* x, int64_t ldx, const float* s_in,
                                int64_t lds_in, int64_t T, int64_t C, const void* ids, fp8bs_index_type it,
                                int64_t ldi, int64_t k, int64_t first, int64_t E, int32_t* offsets, int32_t* slot,
                                uint8_t* q, int64_t ldq, float* s, int64_t lds, void* y, int64_t ldy, int64_t M,
                                void* ws, int64_t ws_bytes, void* stream) {
  fp8bs::MoeIds p;
  fp8bs::MoeRows r;
  FP8BS_TRY(sort_of(ids, it, ldi, T, k, first, E, M, offsets, slot, ws, ws_bytes, p));
  if (T == 0 || M == 0) {   // no rows: the sort alone
    if (src != FP8BS_SRC_FP8_1x128 && src != FP8BS_SRC_BF16) return FP8BS_ERR_INVALID_ARG;
    FP8BS_TRY(check_columns(C));
    FP8BS_TRY(check_device());
    return launched(fp8bs::launch_moe_sort(p, static_cast<hipStream_t>(stream)));
  }
  FP8BS_TRY(rows_of(src, x, ldx, s_in, lds_in, T, C, slot, k, q, ldq, s, lds, y, ldy, M, r));
  FP8BS_TRY(check_device());
  return launched(fp8bs::launch_moe_dispatch(p, r, static_cast<hipStream_t>(stream)));
}

fp8bs_status fp8bs_moe_combine(const void* y, fp8bs_out_dtype yt, int64_t ldy, int64_t M, const int32_t* slot,
                               const float* w, int64_t ldw, int64_t T, int64_t k, int64_t N, const void* add,
                               int64_t ldadd, void* out, int64_t ldo, void* stream) {
  FP8BS_TRY(check_type(yt));
  FP8BS_TRY(check_choices(T, k, M));
  FP8BS_TRY(check_columns(N));
  if (T == 0) return FP8BS_OK;
  if (M > 0) FP8BS_TRY(check_matrix(y, N, ldy, yt == FP8BS_OUT_F32 ? 4 : 2));
  if (slot == nullptr) return FP8BS_ERR_INVALID_ARG;
  if (!aligned(slot, 4)) return FP8BS_ERR_MISALIGNED;
  if (w != nullptr) FP8BS_TRY(check_scales(w, k, ldw));
  if (add != nullptr) FP8BS_TRY(check_matrix(add, N, ldadd, 2));
  FP8BS_TRY(check_matrix(out, N, ldo, 2));
  FP8BS_TRY(check_in_place(out, ldo, add, ldadd));
  if (M > 0 && out == y) return FP8BS_ERR_INVALID_ARG;
  FP8BS_TRY(check_device());
  fp8bs::MoeCombine p;
  p.y = y;
  p.y_f32 = yt == FP8BS_OUT_F32;
  p.ldy = ldy;
  p.M = M;
  p.slot = slot;
  p.w = w;
  p.ldw = ldw;
  p.T = T;
  p.k = static_cast<int>(k);
  p.N = static_cast<int>(N);
  p.add = static_cast<const uint16_t*>(add);
  p.ldadd = ldadd;
  p.out = static_cast<uint16_t*>(out);
  p.ldo = ldo;
  return launched(fp8bs::launch_moe_combine(p, static_cast<hipStream_t>(stream)));
}

fp8bs_status fp8bs_moe_combine_bwd(const void* dout, int64_t lddo, const void* y, fp8bs_out_dtype yt, int64_t ldy,
                                   const int32_t* slot, const float* w, int64_t ldw, int64_t T, int64_t k,
                                   int64_t N, uint8_t* q, int64_t ldq, float* s, int64_t lds, void* dy,
                                   int64_t lddy, int64_t M, float* dw, int64_t lddw, void* stream) {
  FP8BS_TRY(check_type(yt));
  FP8BS_TRY(check_choices(T, k, M));
  FP8BS_TRY(check_columns(N));
  if (T == 0) return FP8BS_OK;
  // without rows there is only dw, all zeros
  if (M == 0) {
    q = nullptr;
    s = nullptr;
    dy = nullptr;
    if (dw == nullptr) return FP8BS_OK;
  }
  if (q == nullptr && dy == nullptr && dw == nullptr) return FP8BS_ERR_INVALID_ARG;
  FP8BS_TRY(check_matrix(dout, N, lddo, 2));
  if (slot == nullptr) return FP8BS_ERR_INVALID_ARG;
  if (!aligned(slot, 4)) return FP8BS_ERR_MISALIGNED;
  FP8BS_TRY(check_scales(w, k, ldw));
  FP8BS_TRY(check_codes(q, ldq, s, lds, N));
  if (dy != nullptr) FP8BS_TRY(check_matrix(dy, N, lddy, 2));
  if (dw != nullptr) {
    FP8BS_TRY(check_scales(dw, k, lddw));
    if (M > 0) FP8BS_TRY(check_matrix(y, N, ldy, yt == FP8BS_OUT_F32 ? 4 : 2));
  }
  if (dy != nullptr && (dy == y || dy == dout)) return FP8BS_ERR_INVALID_ARG;
  FP8BS_TRY(check_device());
  fp8bs::MoeCombineBwd p;
  p.dout = static_cast<const uint16_t*>(dout);
  p.lddo = lddo;
  p.y = y;
  p.y_f32 = yt == FP8BS_OUT_F32;
  p.ldy = ldy;
  p.slot = slot;
  p.w = w;
  p.ldw = ldw;
  p.T = T;
  p.k = static_cast<int>(k);
  p.N = static_cast<int>(N);
  p.q = q;
  p.ldq = ldq;
  p.s = s;
  p.lds = lds;
  p.dy = static_cast<uint16_t*>(dy);
  p.lddy = lddy;
  p.M = M;
  p.dw = dw;
  p.lddw = lddw;
  return launched(fp8bs::launch_moe_combine_bwd(p, static_cast<hipStream_t>(stream)));
}

fp8bs_status fp8bs_swiglu_bwd_quant_1x128(const void* dh, int64_t lddh, const void* g, int64_t ldg, const void* u,
                                          int64_t ldu, int64_t T, int64_t I, uint8_t* q, int64_t ldq, float* s,
                                          int64_t lds, void* d, int64_t ldd, void* h, int64_t ldh, void* stream) {
  if (T < 0 || I <= 0) return FP8BS_ERR_INVALID_ARG;
  if (I % 128 != 0 || I > kMaxInt32 / 4 || T > kMaxInt32) return FP8BS_ERR_UNSUPPORTED_SHAPE;
  if (T == 0) return FP8BS_OK;
  if (q == nullptr && d == nullptr && h == nullptr) return FP8BS_ERR_INVALID_ARG;
  FP8BS_TRY(check_matrix(dh, I, lddh, 2));
  FP8BS_TRY(check_matrix(g, I, ldg, 2));
  FP8BS_TRY(check_matrix(u, I, ldu, 2));
  FP8BS_TRY(check_codes(q, ldq, s, lds, 2 * I));
  if (d != nullptr) FP8BS_TRY(check_matrix(d, 2 * I, ldd, 2));
  if (h != nullptr) FP8BS_TRY(check_matrix(h, I, ldh, 2));
  FP8BS_TRY(check_device());
  fp8bs::SwigluBwd p;
  p.dh = static_cast<const uint16_t*>(dh);
  p.lddh = lddh;
  p.g = static_cast<const uint16_t*>(g);
  p.ldg = ldg;
  p.u = static_cast<const uint16_t*>(u);
  p.ldu = ldu;
  p.T = T;
  p.I = I;
  p.q = q;
  p.ldq = ldq;
  p.s = s;
  p.lds = lds;
  p.d = static_cast<uint16_t*>(d);
  p.ldd = ldd;
  p.h = static_cast<uint16_t*>(h);
  p.ldh = ldh;
  return launched(fp8bs::launch_swiglu_bwd(p, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
