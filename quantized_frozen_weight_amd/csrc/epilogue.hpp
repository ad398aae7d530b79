// The layer's epilogue beyond the adapter, both ways:
//
//   forward:   z = base + s (t B) + bias,  y = act(z) + residual
//   backward:  dx = (base + s (u A^T)) act'(z) + add
//
// (act: QLORA_ACT_*; base as in epilogue_lowrank, ring.hpp), and the 8-bit
// group form of an activation that both sides share.
//
// Activations. relu; gelu = z Phi(z); and two of one family,
// z sigma(z (p + q z^2)): silu has p = 1, q = 0, and the tanh form of gelu
// p = 2 sqrt(2 / pi), q = 0.044715 p, since (1 + tanh(v)) / 2 = sigma(2 v).
// The family shares one code path with two wave-uniform constants, so a
// kernel carries three short branches instead of a variant per activation.
//
// Group form (QLORA_C8G32): 32 consecutive columns of a row share a scale
// 2^e, e the smallest integer with absmax <= 127 2^e, kept as the byte
// e + 127 (1 for an all-zero group, 255 for one with an infinity or a NaN:
// every value of it reads back as NaN). code = round-half-even(v 2^-e), at
// least 1 in size where v is not 0: the sign survives, so relu' taken from
// the code is relu' of the value. A value reads back exactly in bfloat16
// (7 bits times a power of two). The scale being a power of two costs up to
// one of the 8 bits against absmax / 127, and buys a one-byte scale that the
// product's epilogue can form without a division.
#pragma once

#include <type_traits>

#include "ring.hpp"

namespace qlora {

constexpr int kActNone = 0, kActRelu = 1, kActGelu = 2, kActGeluTanh = 3, kActSilu = 4;
constexpr int kGroup = 32;       // columns per scale of the group form

inline __host__ __device__ int group_count(int C) { return C / kGroup + (C % kGroup != 0); }

struct ActParams {
  int kind;      // 0 none, 1 relu, 2 gelu, 3 the sigma family
  float p, q;    // the sigma family's constants
  float p2, q2;  // -log2 e times them
};

inline ActParams act_params(int act) {
  ActParams a{act, 1.f, 0.f, 0.f, 0.f};
  if (act == kActGeluTanh) {
    a.kind = 3;
    a.p = 1.5957691216057308f;               // 2 sqrt(2 / pi)
    a.q = 1.5957691216057308f * 0.044715f;
  } else if (act == kActSilu) {
    a.kind = 3;
  }
  a.p2 = -1.44269504088896341f * a.p;
  a.q2 = -1.44269504088896341f * a.q;
  return a;
}

// max that keeps a NaN (v_max drops it)
__device__ __forceinline__ float at_least(float v, float lo) { return v < lo ? lo : v; }

// e^w for |w| <= 150 as 2^(w log2 e), the product kept in two parts (its
// rounding error, times |w|, would otherwise reach the result): within 3 ulp.
// Overflows to infinity, underflows to 0. For float32 outputs; bfloat16 ones
// take 2^w2 of the rounded exponent w2 = w log2 e (FINE false below), whose
// error, |w| 2^-24 of e^w, they cannot show: e^w only matters where it is not
// far from 1.
__device__ __forceinline__ float exp_fine(float w) {
  constexpr float kL = 1.44269504088896341f, kLlo = 1.925963033500e-8f, kLn2 = 0.693147180559945f;
  const float hi = w * kL;
  const float lo = __builtin_fmaf(w, kLlo, __builtin_fmaf(w, kL, -hi));
  return __builtin_amdgcn_exp2f(hi) * __builtin_fmaf(lo, kLn2, 1.f);
}

// e^(-c^2 / 2), |c| <= 16. FINE: within 4e-7, c^2 in two parts as well (its
// rounding alone is up to 4e-6 of the result at |c| = 12.8).
template <bool FINE>
__device__ __forceinline__ float normal_exp(float c) {
  if constexpr (FINE) {
    const float q = c * c, lo = __builtin_fmaf(c, c, -q);
    return exp_fine(-0.5f * q) * __builtin_fmaf(lo, -0.5f, 1.f);
  } else {
    return __builtin_amdgcn_exp2f(c * c * -0.72134752044448170f);
  }
}

// The smaller tail Phi(-|z|) = erfc(|z| / sqrt 2) / 2 with a relative error
// below 1e-6 where ex has float32 accuracy (1 + erf would cancel there). For x = |z| / sqrt 2 and
// t = 1 / (1 + 0.44 x), e^(x^2) erfc(x) is t times a polynomial of degree 7 in
// t, fitted here to the smallest largest relative error (1.9e-7) on
// 0 <= x <= 15; its coefficients are halved below. a = |z|, ex = e^(-z^2 / 2).
__device__ __forceinline__ float normal_tail(float a, float ex) {
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(a, 0.44f * 0.70710678118654752f, 1.f));
  float c = 0.5f * 0.07150039076805115f;
  c = __builtin_fmaf(c, t, 0.5f * -0.27915504574775696f);
  c = __builtin_fmaf(c, t, 0.5f * 0.29887089133262634f);
  c = __builtin_fmaf(c, t, 0.5f * -0.022297518327832222f);
  c = __builtin_fmaf(c, t, 0.5f * 0.2169952094554901f);
  c = __builtin_fmaf(c, t, 0.5f * 0.2169342190027237f);
  c = __builtin_fmaf(c, t, 0.5f * 0.2489354908466339f);
  c = __builtin_fmaf(c, t, 0.5f * 0.24821652472019196f);
  return t * c * ex;
}

// Arguments are bounded with fminf / fmaxf, which drop a NaN, where z itself
// brings it back or nan_or does.
__device__ __forceinline__ float nan_or(float z, float v) { return z != z ? z : v; }

// act of every v; -inf goes to the limit 0 (not -inf * 0), NaN stays NaN
template <bool FINE, int NV>
__device__ __forceinline__ void act_apply(const ActParams& a, float (&v)[NV]) {
  if (a.kind == 0) return;
  if (a.kind == 1) {
#pragma unroll
    for (int e = 0; e < NV; ++e) v[e] = at_least(v[e], 0.f);
  } else if (a.kind == 2) {
    // z Phi(z) = max(z, 0) - |z| Phi(-|z|); past |z| = 16 the tail is 0
#pragma unroll
    for (int e = 0; e < NV; ++e) {
      const float c = fminf(__builtin_fabsf(v[e]), 16.f);
      v[e] = __builtin_fmaf(-c, normal_tail(c, normal_exp<FINE>(c)), at_least(v[e], 0.f));
    }
  } else {
    // z / (1 + e^-w), w = z (p + q z^2)
#pragma unroll
    for (int e = 0; e < NV; ++e) {
      const float z = at_least(v[e], -1e9f), c = fminf(z, 1e9f), c2 = c * c;
      float x;
      if constexpr (FINE) x = exp_fine(fminf(fmaxf(-c * __builtin_fmaf(a.q, c2, a.p), -150.f), 150.f));
      else x = __builtin_amdgcn_exp2f(c * __builtin_fmaf(a.q2, c2, a.p2));
      v[e] = z * __builtin_amdgcn_rcpf(1.f + x);
    }
  }
}

// v[e] *= act'(z[e]); relu'(0) = 0, relu'(NaN) = NaN
template <bool FINE, int NV>
__device__ __forceinline__ void act_slope_mul(const ActParams& a, const float (&z)[NV], float (&v)[NV]) {
  if (a.kind == 0) return;
  if (a.kind == 1) {
#pragma unroll
    for (int e = 0; e < NV; ++e) v[e] *= nan_or(z[e], z[e] > 0.f ? 1.f : 0.f);
  } else if (a.kind == 2) {
    // Phi + z phi; past |z| = 16 phi is 0 in float32
#pragma unroll
    for (int e = 0; e < NV; ++e) {
      const float c = __builtin_amdgcn_fmed3f(z[e], -16.f, 16.f), ex = normal_exp<FINE>(c);
      const float h = normal_tail(__builtin_fabsf(c), ex);
      v[e] *= nan_or(z[e], __builtin_fmaf(c * 0.3989422804014327f, ex, c < 0.f ? h : 1.f - h));
    }
  } else {
    // sigma + z sigma (1 - sigma) (p + 3 q z^2) with sigma = 1 / (1 + x),
    // 1 - sigma = x sigma, x = e^-w (bounded by 2^115: sigma (1 - sigma) is
    // then below 2^-115 anyway); past |z| = 100 it is 0 or 1
#pragma unroll
    for (int e = 0; e < NV; ++e) {
      const float c = __builtin_amdgcn_fmed3f(z[e], -100.f, 100.f), c2 = c * c;
      float x;
      if constexpr (FINE) x = exp_fine(fminf(fmaxf(-c * __builtin_fmaf(a.q, c2, a.p), -80.f), 80.f));
      else x = __builtin_amdgcn_exp2f(fminf(c * __builtin_fmaf(a.q2, c2, a.p2), 115.f));
      const float s = __builtin_amdgcn_rcpf(1.f + x);
      v[e] *= nan_or(z[e], __builtin_fmaf(c * __builtin_fmaf(3.f * a.q, c2, a.p), s * (x * s), s));
    }
  }
}

// ---- the group form ---------------------------------------------------------
// max over the four lanes 4 i .. 4 i + 3, every lane ending with it
__device__ __forceinline__ uint32_t quad_max_u32(uint32_t v) {
#pragma unroll
  for (int lvl = 2; lvl < 4; ++lvl) {
    const uint32_t w = __float_as_uint(dpp_pair(__uint_as_float(v), lvl));
    v = w > v ? w : v;
  }
  return v;
}

// The scale byte of a group from its abs-max bits: e = p - 6 where the
// abs-max m 2^p (1 <= m < 2) has m <= 127 / 64, else p - 5.
__device__ __forceinline__ int group_byte(uint32_t amax_bits) {
  if (amax_bits >= 0x7f800000u) return 255;
  int b = (int)(amax_bits >> 23) - 6 + ((amax_bits & 0x7fffffu) > 0x7e0000u ? 1 : 0);
  return b < 1 ? 1 : b;
}

// The code of v under scale byte b (not 255) in the low byte; the rest of the
// word is not its sign. v 2^-e, moved out to +-0.75 where it is smaller but v
// is not 0 (so that it rounds to +-1), is rounded to an integer, ties to even,
// by adding 3 2^22: the sum's last 8 bits are the code. (v itself decides, not
// v 2^-e, which underflows to 0 where v is below 2^-149 of the scale.)
__device__ __forceinline__ uint32_t group_code_bits(float v, float inv) {
  const float t = v * inv;
  const float m = __builtin_copysignf(fmaxf(__builtin_fabsf(t), 0.75f), v);
  return __float_as_uint((v == 0.f ? v : m) + 12582912.f);
}
// 2^-e = 2^(127 - b); b in [1, 249]
__device__ __forceinline__ float group_inverse(int b) { return __uint_as_float((uint32_t)(254 - b) << 23); }

__device__ __forceinline__ int8_t group_code(float v, int b) {
  return b == 255 ? 0 : (int8_t)group_code_bits(v, group_inverse(b));
}

// Eight values as codes of scale byte b, packed four to a word.
__device__ __forceinline__ u32x2 group_codes(const float (&v)[8], int b) {
  const float inv = group_inverse(b);
  u32x2 w;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t c[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) c[e] = group_code_bits(v[4 * h + e], inv);
    const uint32_t lo = __builtin_amdgcn_perm(c[1], c[0], 0x0c0c0400u);   // bytes c0, c1, 0, 0
    const uint32_t hi = __builtin_amdgcn_perm(c[3], c[2], 0x04000c0cu);   // bytes 0, 0, c2, c3
    w[h] = b == 255 ? 0u : lo | hi;
  }
  return w;
}

// The scale that byte b stands for; 255: NaN.
__device__ __forceinline__ float group_scale(int b) {
  return __uint_as_float(b == 255 ? 0x7fc00000u : (uint32_t)b << 23);
}

// (Code 64 of byte 249 is an infinity here; every slope has its limit from
// 100 on, so z may stay that.)
__device__ __forceinline__ void group_values(u32x2 c, int b, float (&v)[8]) {
  const float s = group_scale(b);
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = (float)(int8_t)(c[e >> 2] >> (8 * (e & 3))) * s;
}

// ---- eight values of a row in either dtype ------------------------------------
typedef float f32x2v __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2v __attribute__((ext_vector_type(2)));

// two floats to bfloat16, round to nearest even (v_cvt_pk_bf16_f32)
__device__ __forceinline__ uint32_t cvt_bf16x2(float lo, float hi) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2v{lo, hi}, bf16x2v));
}

__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  *reinterpret_cast<f32x4*>(p) = f32x4{v[0], v[1], v[2], v[3]};
  *reinterpret_cast<f32x4*>(p + 4) = f32x4{v[4], v[5], v[6], v[7]};
}
__device__ __forceinline__ void store8(uint16_t* p, const float (&v)[8]) {
  *reinterpret_cast<u32x4*>(p) = u32x4{cvt_bf16x2(v[0], v[1]), cvt_bf16x2(v[2], v[3]),
                                       cvt_bf16x2(v[4], v[5]), cvt_bf16x2(v[6], v[7])};
}

// eight values as loaded: 16 bytes of bf16, 32 of float32
template <typename OutT> struct Raw8;
template <> struct Raw8<uint16_t> {
  u32x4 v;
  __device__ __forceinline__ void load(const void* p, long at) {
    v = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(p) + at);
  }
  // eight bytes of codes in their place
  __device__ __forceinline__ void set2(u32x2 c) { v[0] = c[0]; v[1] = c[1]; }
  __device__ __forceinline__ u32x2 get2() const { return u32x2{v[0], v[1]}; }
  __device__ __forceinline__ void get(float (&o)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o[2 * i] = __uint_as_float(v[i] << 16);
      o[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
    }
  }
};
template <> struct Raw8<float> {
  f32x4 a, b;
  __device__ __forceinline__ void load(const void* p, long at) {
    a = *reinterpret_cast<const f32x4*>(static_cast<const float*>(p) + at);
    b = *reinterpret_cast<const f32x4*>(static_cast<const float*>(p) + at + 4);
  }
  __device__ __forceinline__ void get(float (&o)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) { o[i] = a[i]; o[4 + i] = b[i]; }
  }
};

// The forward epilogue of a call (pointers NULL where unused).
struct FwdEpi {
  ActParams act;
  const float* bias;      // [N]
  const void* res;        // [M, N], may be y
  void* z;                // [M, N]
  int8_t* zc;             // [M, N] codes and [M, zg] scale bytes of z
  uint8_t* zs;
  int zg;
};

// The backward one: z (dense, or group form) and add, [M, K].
struct GradEpi {
  ActParams act;
  const void* z;
  const int8_t* zc;
  const uint8_t* zs;
  int zg;
  const void* add;
};

// LDS bytes of one wave's strip in epilogue_fused: 16 rows of FN * 16 floats,
// each padded by 16 bytes.
template <int FN> constexpr int fused_strip_bytes() { return 16 * (FN * 64 + 16); }

// What a piece of 8 outputs needs besides the product, as loaded.
template <typename OutT> struct Side {
  Raw8<OutT> r;      // residual, or add
  Raw8<OutT> z;      // backward: dense z, or its codes in z's first 8 bytes
  int b;             // scale byte of the codes
};

// Shape of a wave's FM x FN grid of 16 x 16 blocks in epilogue_fused.
template <typename OutT, int FM, int FN> struct EpiShape {
  static constexpr int PITCH = FN * 64 + 16;               // bytes of a strip row
  static constexpr int CPR = 2 * FN;                       // 8-column pieces per strip row
  static constexpr int PN = CPR * 16 / 64;                 // pieces per lane and strip
  static constexpr int AHEAD = sizeof(OutT) == 2 ? FM : FM < 2 ? FM : 2;   // strips whose operands are held
  static constexpr int NB = 64 % CPR == 0 ? 1 : PN;        // distinct column pieces of a lane
  static_assert(CPR % 4 == 0, "four neighbouring lanes hold one 32-column group");
};

// The side operands of a wave's outputs: fetched (start) as early as the
// caller has registers for them, before what is left of its own work.
template <typename OutT, typename Epi, int FM, int FN> struct EpiSide {
  typedef EpiShape<OutT, FM, FN> Sh;
  static constexpr bool GRAD = std::is_same<Epi, GradEpi>::value;
  Side<OutT> side[Sh::AHEAD][Sh::PN];
  float bias[Sh::NB][8];

  // output position of piece p of strip i; N % 16 == 0: 8 columns in or out
  static __device__ __forceinline__ bool place(int i, int p, int M, int N, int row0, int col0, int& m, int& n) {
    const int q = (threadIdx.x & 63) + 64 * p;
    m = row0 + i * 16 + q / Sh::CPR;
    n = col0 + (q % Sh::CPR) * 8;
    return m < M && n < N;
  }

  __device__ __forceinline__ void fetch(const Epi& ep, int i, int M, int N, int row0, int col0) {
#pragma unroll
    for (int p = 0; p < Sh::PN; ++p) {
      int m, n;
      const bool live = place(i, p, M, N, row0, col0, m, n);
      const long at = live ? (long)m * N + n : 0;
      Side<OutT>& sd = side[i % Sh::AHEAD][p];
      if constexpr (GRAD) {
        if (ep.act.kind != 0) {
          if (ep.zc != nullptr) {
            const u32x2 c = *reinterpret_cast<const u32x2*>(ep.zc + at);
            sd.z.set2(c);
            sd.b = ep.zs[live ? (long)m * ep.zg + n / kGroup : 0];
          } else {
            sd.z.load(ep.z, at);
          }
        }
        if (ep.add != nullptr) sd.r.load(ep.add, at);
      } else {
        if (ep.res != nullptr) sd.r.load(ep.res, at);
      }
    }
  }

  __device__ __forceinline__ void start(const Epi& ep, int M, int N, int row0, int col0) {
    if constexpr (!GRAD) {
      if (ep.bias != nullptr) {
#pragma unroll
        for (int p = 0; p < Sh::NB; ++p) {
          const int n = col0 + (((threadIdx.x & 63) + 64 * p) % Sh::CPR) * 8;
          load8(ep.bias + (n < N ? n : 0), bias[p]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < Sh::AHEAD; ++i) fetch(ep, i, M, N, row0, col0);
  }
};

// epilogue_lowrank (ring.hpp) with the rest of the layer behind it. One
// 16-row strip of the wave's outputs at a time goes through LDS in float32,
// so that a lane then holds 8 consecutive columns of a row: every operand
// (residual, saved z, codes) moves in 16- or 8-byte pieces, the activation
// sees the unrounded z, four neighbouring lanes hold one 32-column group,
// and y is rounded once. What bounds it is the latency of the side operands
// (two or three waves per SIMD), hence EpiSide: in bfloat16 all strips' are
// fetched before the first strip is formed, in float32 (twice the registers)
// two strips'.
template <int BM, int BN, int R, bool SCALED, bool AFF = false, typename OutT, typename Epi,
          typename AccT, int FM, int FN>
__device__ __forceinline__ void epilogue_fused(const AccT (&acc)[FM][FN], const float* E, int M,
                                               int N, int m0, int n0, int wr0, int wc0, float s,
                                               OutT* out, const Epi& ep, EpiSide<OutT, Epi, FM, FN>& es,
                                               int8_t* strip) {
  typedef EpiShape<OutT, FM, FN> Sh;
  constexpr bool GRAD = std::is_same<Epi, GradEpi>::value;
  constexpr int PITCH = Sh::PITCH, CPR = Sh::CPR, PN = Sh::PN, AHEAD = Sh::AHEAD, NB = Sh::NB;
  static_assert(!AFF || SCALED, "the affine form uses the row scales");
  const int lane = threadIdx.x & 63;
  const float* ts = E;
  const float* qs = E + BM * R;
  const float* rsv = E + (BM + BN) * R;
  const float* csv = rsv + BM;
  const float* rav = csv + BN;

#pragma unroll
  for (int i = 0; i < FM; ++i) {
    f32x4 low[FN];
#pragma unroll
    for (int jn = 0; jn < FN; ++jn) low[jn] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int kc = 0; kc < R / 4; ++kc) {
      const int j = kc * 4 + (lane >> 4);
      const float ta = ts[(wr0 + i * 16 + (lane & 15)) * R + j];
#pragma unroll
      for (int jn = 0; jn < FN; ++jn)
        low[jn] = __builtin_amdgcn_mfma_f32_16x16x4f32(ta, qs[j * BN + wc0 + jn * 16 + (lane & 15)],
                                                       low[jn], 0, 0, 0);
    }
#pragma unroll
    for (int jn = 0; jn < FN; ++jn) {
      const int nl = wc0 + jn * 16 + (lane & 15);
      const float csn = SCALED ? csv[nl] : 1.f;
#pragma unroll
      for (int ii = 0; ii < 4; ++ii) {
        const int rl = (lane >> 4) * 4 + ii, ml = wr0 + i * 16 + rl;
        float base;
        if constexpr (AFF)
          base = rsv[ml] * ((float)acc[i][jn][ii] + rav[ml]);
        else
          base = SCALED ? (float)acc[i][jn][ii] * (rsv[ml] * csn) : (float)acc[i][jn][ii];
        *reinterpret_cast<float*>(strip + rl * PITCH + (jn * 16 + (lane & 15)) * 4) =
            __builtin_fmaf(s, low[jn][ii], base);
      }
    }
    // (the LDS runs one wave's instructions in order: no wait before the
    // read-back, nor before the next strip's writes)
#pragma unroll
    for (int p = 0; p < PN; ++p) {
      const int q = lane + 64 * p;
      int m, n;
      const bool live = es.place(i, p, M, N, m0 + wr0, n0 + wc0, m, n);
      const long at = (long)m * N + n;
      const Side<OutT>& sd = es.side[i % AHEAD][p];
      float v[8], w[8];
      load8(reinterpret_cast<const float*>(strip + (q / CPR) * PITCH + (q % CPR) * 32), v);
      if constexpr (GRAD) {
        if (ep.act.kind != 0) {
          if (ep.zc != nullptr) group_values(sd.z.get2(), sd.b, w);
          else sd.z.get(w);
          act_slope_mul<sizeof(OutT) == 4>(ep.act, w, v);
        }
        if (ep.add != nullptr) {
          sd.r.get(w);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] += w[e];
        }
      } else {
        if (ep.bias != nullptr) {
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] += es.bias[p % NB][e];
        }
        if (ep.z != nullptr && live) store8(static_cast<OutT*>(ep.z) + at, v);
        if (ep.zc != nullptr) {
          uint32_t t = 0;
#pragma unroll
          for (int e = 0; e < 8; ++e) { const uint32_t b = abs_bits(v[e]); t = b > t ? b : t; }
          const int b = group_byte(quad_max_u32(live ? t : 0u));
          if (live) {
            *reinterpret_cast<u32x2*>(ep.zc + at) = group_codes(v, b);
            if (n % kGroup == 0) ep.zs[(long)m * ep.zg + n / kGroup] = (uint8_t)b;
          }
        }
        act_apply<sizeof(OutT) == 4>(ep.act, v);
        if (ep.res != nullptr) {
          sd.r.get(w);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] += w[e];
        }
      }
      if (live) store8(out + at, v);
    }
    if (i + AHEAD < FM) es.fetch(ep, i + AHEAD, M, N, m0 + wr0, n0 + wc0);
  }
}

}  // namespace qlora
