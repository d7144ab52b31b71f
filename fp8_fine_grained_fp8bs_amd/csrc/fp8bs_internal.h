// fp8bs_internal.h -- launchers behind the C ABI (arguments already checked).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp8bs {

hipError_t launch_quant_act_1x128(const uint16_t* x, int64_t M, int64_t K, int64_t ldx,
                                  uint8_t* q, int64_t ldq, float* s, int64_t lds,
                                  hipStream_t st);

hipError_t launch_quant_w_128x128(const uint16_t* w, int64_t N, int64_t K, int64_t ldw,
                                  uint8_t* q, int64_t ldq, float* s, int64_t lds,
                                  hipStream_t st);

hipError_t launch_quant_act_w(const uint16_t* x, int64_t M, int64_t ldx, uint8_t* qx, int64_t ldqx,
                              float* sx, int64_t ldsx, const uint16_t* w, int64_t N, int64_t ldw,
                              uint8_t* qw, int64_t ldqw, float* sw, int64_t ldsw, int64_t K,
                              hipStream_t st);

hipError_t launch_cast_e4m3(const float* x, int64_t n, uint8_t* q, hipStream_t st);

hipError_t launch_swiglu_quant_1x128(const uint16_t* g, int64_t ldg, const uint16_t* u, int64_t ldu,
                                     int64_t T, int64_t I, uint8_t* q, int64_t ldq, float* s,
                                     int64_t lds, uint16_t* h, int64_t ldh, hipStream_t st);

hipError_t launch_quant_per_tensor(const uint16_t* x, int64_t n, uint8_t* q, float* s,
                                   hipStream_t st);

hipError_t launch_encode_e5m6(const uint16_t* x, int64_t T, int64_t C, int64_t ldx, uint8_t* y,
                              int64_t ldy, hipStream_t st);

hipError_t launch_decode_e5m6(const uint8_t* y, int64_t T, int64_t C, int64_t ldy, uint16_t* x,
                              int64_t ldx, hipStream_t st);

// src: 0 E4M3 codes with 1x128 scales, 1 bf16, 2 packed E5M6
hipError_t launch_requant_T_128x1(int src, const void* in, const float* s_in,
                                  int64_t T, int64_t C, int64_t ld_in, int64_t lds_in,
                                  uint8_t* q_out, int64_t ld_out, float* s_out,
                                  int64_t lds_out, hipStream_t st);

hipError_t launch_transpose_w_128x128(const uint8_t* q, int64_t N, int64_t K, int64_t ldq,
                                      const float* s, int64_t lds, uint8_t* qt, int64_t ldqt,
                                      float* st, int64_t ldst, hipStream_t stream);

hipError_t launch_gemm(const uint8_t* a, const float* sa, int64_t lda, int64_t ldsa,
                       const uint8_t* b, const float* sb, int64_t ldb, int64_t ldsb,
                       bool bscale_row, void* d, int64_t ldd, float* s_out, int64_t lds_out,
                       int out, int64_t M, int64_t N, int64_t K, hipStream_t st);

hipError_t launch_gemm_bf16a(const uint16_t* x, int64_t ldx, uint8_t* qx, int64_t ldqx, float* sx,
                             int64_t ldsx, const uint8_t* b, const float* sb, int64_t ldb, int64_t ldsb,
                             void* d, int64_t ldd, bool out_f32, int64_t M, int64_t N, int64_t K,
                             hipStream_t st);

hipError_t launch_grouped_gemm(const uint8_t* a, const float* sa, int64_t ldsa,
                               const uint8_t* b, const float* sb, const int32_t* offsets,
                               int32_t E, int64_t M_total, void* d, bool out_f32,
                               int64_t N, int64_t K, hipStream_t st);

hipError_t launch_rope_table(float* cs, int64_t n_pos, int64_t rot, double base, double factor, double orig_len,
                             double turns_lo, double turns_hi, double mscale, hipStream_t st);

hipError_t launch_rope(const uint16_t* x, int64_t ldx, uint16_t* y, int64_t ldy, const int32_t* pos, int64_t T,
                       int H, int D, int rot, int rot_off, bool interleaved, bool inverse, const float* cs,
                       int64_t n_pos, hipStream_t st);

// Arguments of fp8bs_kv_append (q == nullptr: no queries; cs == nullptr: no rotation).
struct KvAppend {
  const uint16_t* q;
  int64_t ldq;
  uint16_t* q_out;
  int64_t ldqo;
  int Hq;
  const uint16_t* k;
  int64_t ldk;
  const uint16_t* v;
  int64_t ldv;
  int Hkv, D;
  const float* cs;
  int64_t n_pos;
  int rot, rot_off;
  bool interleaved;
  const int32_t* q_off;
  const int32_t* kv_len;
  int B;
  int64_t T, max_q;
  const int32_t* table;
  int64_t ldt, max_pages;
  int page;
  uint8_t* kc;
  float* ks;
  uint8_t* vc;
  float* vs;
  int64_t n_pages;
};
hipError_t launch_kv_append(const KvAppend& p, hipStream_t st);

// Arguments of fp8bs_attn_paged.
struct AttnPaged {
  const uint16_t* q;
  int64_t ldq;
  uint16_t* out;
  int64_t ldo;
  float* lse;
  int64_t ldl;
  const int32_t* q_off;
  const int32_t* kv_len;
  int B;
  int64_t T, max_q;
  int Hq, Hkv, D;
  const int32_t* table;
  int64_t ldt, max_pages;
  int page;
  const uint8_t* kc;
  const float* ks;
  const uint8_t* vc;
  const float* vs;
  int64_t n_pages;
  float scale;
  bool causal;
  int64_t window;
  void* ws;
};
hipError_t launch_attn_paged(const AttnPaged& p, hipStream_t st);
// Working memory of launch_attn_paged: a function of the sizes alone.
int64_t attn_paged_ws(int64_t B, int64_t T, int64_t max_q, int Hq, int Hkv, int D, int64_t max_pages, int page);

}  // namespace fp8bs
