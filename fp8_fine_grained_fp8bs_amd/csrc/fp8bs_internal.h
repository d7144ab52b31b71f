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

// Workgroups of a launch: a grid's threads are numbered in 32 bits.
constexpr int64_t most_blocks(int threads) { return 0xffffffffll / threads; }

// Launches for all of p's tokens, at most so many a launch.  launch(part) takes the
// arguments of some of them; p.part(t, n) gives those of tokens t .. t + n - 1.
template <class P, class Launch>
hipError_t by_tokens(const P& p, int64_t most, Launch launch) {
  if (p.T <= most) return launch(p);
  for (int64_t t = 0; t < p.T; t += most) {
    const hipError_t e = launch(p.part(t, p.T - t < most ? p.T - t : most));
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}
// An optional buffer n elements further.
template <class T>
T* further(T* p, int64_t n) {
  return p != nullptr ? p + n : nullptr;
}

// Arguments of fp8bs_rmsnorm_quant_1x128 (r, q, y, rstd may be null; q with s, r with h).
struct RmsNorm {
  const uint16_t* x;
  int64_t ldx;
  const uint16_t* r;
  int64_t ldr;
  const void* gamma;
  bool gamma_f32;
  float eps;
  int64_t T;
  int C;
  uint16_t* h;
  int64_t ldh;
  uint8_t* q;
  int64_t ldq;
  float* s;
  int64_t lds;
  uint16_t* y;
  int64_t ldy;
  float* rstd;
  RmsNorm part(int64_t t, int64_t n) const {
    RmsNorm p = *this;
    p.T = n;
    p.x += t * ldx;
    p.r = further(r, t * ldr);
    p.h = further(h, t * ldh);
    p.q = further(q, t * ldq);
    p.s = further(s, t * lds);
    p.y = further(y, t * ldy);
    p.rstd = further(rstd, t);
    return p;
  }
};
hipError_t launch_rmsnorm(const RmsNorm& p, hipStream_t st);

// Arguments of fp8bs_rmsnorm_bwd (dres, dgamma may be null; ws with dgamma).
struct RmsNormBwd {
  const uint16_t* dn;
  int64_t lddn;
  const uint16_t* dres;
  int64_t lddr;
  const uint16_t* h;
  int64_t ldh;
  const void* gamma;
  bool gamma_f32;
  const float* rstd;
  int64_t T;
  int C;
  uint16_t* dx;
  int64_t lddx;
  float* dgamma;
  float* ws;
};
hipError_t launch_rmsnorm_bwd(const RmsNormBwd& p, hipStream_t st);
int64_t rmsnorm_bwd_ws(int64_t T, int C);

constexpr int kMaxExperts = 1024;   // held here
constexpr int kMaxChoices = 64;     // experts of a token

// The assignments of a sort, and what it writes.
struct MoeIds {
  const void* ids;
  bool wide;   // int64
  int64_t ldi, T;
  int k;
  int64_t first;
  int E;
  int32_t* offsets;
  int32_t* slot;
  int64_t M;
  int32_t* ws;
};
int64_t moe_sort_ws(int64_t T, int k, int E);
hipError_t launch_moe_sort(const MoeIds& p, hipStream_t st);

// Rows of T tokens and where they go (q with s, y may be null; codes in go out as codes).
struct MoeRows {
  bool codes_in;
  const void* x;
  int64_t ldx;
  const float* s_in;
  int64_t lds_in, T;
  int C;
  const int32_t* slot;
  int k;
  uint8_t* q;
  int64_t ldq;
  float* s;
  int64_t lds;
  uint16_t* y;
  int64_t ldy, M;
  // the outputs' rows go by slot
  MoeRows part(int64_t t, int64_t n) const {
    MoeRows p = *this;
    p.T = n;
    p.x = static_cast<const uint8_t*>(x) + t * ldx * (codes_in ? 1 : 2);
    p.s_in = further(s_in, t * lds_in);
    p.slot += t * k;
    return p;
  }
};
hipError_t launch_moe_gather(const MoeRows& p, hipStream_t st);
hipError_t launch_moe_dispatch(const MoeIds& ids, const MoeRows& p, hipStream_t st);

struct MoeCombine {
  const void* y;
  bool y_f32;
  int64_t ldy, M;
  const int32_t* slot;
  const float* w;   // null: 1
  int64_t ldw, T;
  int k, N;
  const uint16_t* add;   // may be null
  int64_t ldadd;
  uint16_t* out;
  int64_t ldo;
  MoeCombine part(int64_t t, int64_t n) const {
    MoeCombine p = *this;
    p.T = n;
    p.slot += t * k;
    p.w = further(w, t * ldw);
    p.add = further(add, t * ldadd);
    p.out += t * ldo;
    return p;
  }
};
hipError_t launch_moe_combine(const MoeCombine& p, hipStream_t st);

struct MoeCombineBwd {
  const uint16_t* dout;
  int64_t lddo;
  const void* y;   // with dw
  bool y_f32;
  int64_t ldy;
  const int32_t* slot;
  const float* w;
  int64_t ldw, T;
  int k, N;
  uint8_t* q;   // with s; may be null
  int64_t ldq;
  float* s;
  int64_t lds;
  uint16_t* dy;   // may be null
  int64_t lddy, M;
  float* dw;   // may be null
  int64_t lddw;
  MoeCombineBwd part(int64_t t, int64_t n) const {
    MoeCombineBwd p = *this;
    p.T = n;
    p.dout += t * lddo;
    p.slot += t * k;
    p.w += t * ldw;
    p.dw = further(dw, t * lddw);
    return p;
  }
};
hipError_t launch_moe_combine_bwd(const MoeCombineBwd& p, hipStream_t st);

// Arguments of fp8bs_swiglu_bwd_quant_1x128 (q with s, d, h may be null).
struct SwigluBwd {
  const uint16_t* dh;
  int64_t lddh;
  const uint16_t* g;
  int64_t ldg;
  const uint16_t* u;
  int64_t ldu, T, I;
  uint8_t* q;
  int64_t ldq;
  float* s;
  int64_t lds;
  uint16_t* d;
  int64_t ldd;
  uint16_t* h;
  int64_t ldh;
  SwigluBwd part(int64_t t, int64_t n) const {
    SwigluBwd p = *this;
    p.T = n;
    p.dh += t * lddh;
    p.g += t * ldg;
    p.u += t * ldu;
    p.q = further(q, t * ldq);
    p.s = further(s, t * lds);
    p.d = further(d, t * ldd);
    p.h = further(h, t * ldh);
    return p;
  }
};
hipError_t launch_swiglu_bwd(const SwigluBwd& p, hipStream_t st);

}  // namespace fp8bs
