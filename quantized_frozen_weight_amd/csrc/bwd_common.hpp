// Pieces that the fused backward kernels share: the three-part bf16 split of
// float32 operands, transposing LDS reads, and the x tile from 8-bit codes.
#pragma once
#include "ring.hpp"

namespace qlora {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t pk_bf16(float lo, float hi) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{lo, hi}, bf16x2));
}

// Two float32 values each as a sum of three bf16 values, v = hi + mid + lo:
// hi is the bf16 nearest to v, mid the bf16 nearest to the remainder
// v - hi, lo the bf16 nearest to v - hi - mid (both remainders exact in
// float32). Products with a bf16 operand on the matrix cores then carry v to
// float32 precision (relative error at most 2^-24) instead of 8 significant
// bits, which keeps the float32 adapter's gradients float32-accurate: B (for
// u = dy B^T) and t (for dB = s t^T dy) enter their products as hi, mid and
// lo columns of one operand. A non-finite hi (v infinite or NaN, or past the
// bf16 range) takes mid = lo = 0, so hi alone carries the infinity or NaN.
// Returns the packed hi pair; the mid and lo pairs go to mid2 and lo2.
__device__ __forceinline__ uint32_t pk_bf16_split3(float a, float b, uint32_t& mid2, uint32_t& lo2) {
  const uint32_t h = pk_bf16(a, b);
  const bool fa = (h & 0x7f80u) != 0x7f80u, fb = (h & 0x7f800000u) != 0x7f800000u;
  const float ra = fa ? a - __uint_as_float(h << 16) : 0.f;
  const float rb = fb ? b - __uint_as_float(h & 0xffff0000u) : 0.f;
  mid2 = pk_bf16(ra, rb);
  lo2 = pk_bf16(ra - __uint_as_float(mid2 << 16), rb - __uint_as_float(mid2 & 0xffff0000u));
  return h;
}

// The rank-r products u = dy B^T and dB^T = dy^T t run with 3R operand
// columns: j in [0, R) the hi parts, [R, 2R) the mid parts, [2R, 3R) the lo
// parts. The sum for rank j (j = cb * 16 + lane % 16 < R) of its columns j,
// j + R, j + 2R of the accumulators (column c at block c / 16, lane c % 16 of
// the 16-lane group): R = 4 and 8 put some of them in other lanes of the
// group, read through a lane permute that every lane executes; for R >= 16
// all three are the same lane of blocks cb, cb + R / 16, cb + R / 8.
template <int R, int UCB>
__device__ __forceinline__ float split3_sum(const f32x4 (&v)[UCB], int cb, int ii, int lane) {
  if constexpr (R == 4) {
    static_assert(UCB == 1, "12 columns in one block");
    const int g = lane & ~15;
    return v[0][ii] + __shfl(v[0][ii], g | ((lane + 4) & 15)) + __shfl(v[0][ii], g | ((lane + 8) & 15));
  } else if constexpr (R == 8) {
    static_assert(UCB == 2, "24 columns in two blocks");
    return v[0][ii] + __shfl(v[0][ii], (lane & ~15) | ((lane + 8) & 15)) + v[1][ii];
  } else {
    static_assert(R % 16 == 0 && UCB == 3 * R / 16, "whole blocks per part");
    return v[cb][ii] + v[cb + R / 16][ii] + v[cb + R / 8][ii];
  }
}

// NR transposing LDS reads (ds_read_b64_tr_b16) issued together and completed
// in the same asm block. Written as asm because the builtin form makes the
// compiler wait for every direct-to-LDS load in flight (the ring's later
// stages included) before each read.
template <int NR>
__device__ __forceinline__ void tr16_reads(const uint32_t (&addr)[NR], uint64_t (&out)[NR]) {
  static_assert(NR == 4 || NR == 8, "4 or 8 reads");
  if constexpr (NR == 4) {
    asm volatile(
        "ds_read_b64_tr_b16 %0, %4\n\t"
        "ds_read_b64_tr_b16 %1, %5\n\t"
        "ds_read_b64_tr_b16 %2, %6\n\t"
        "ds_read_b64_tr_b16 %3, %7\n\t"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(out[0]), "=&v"(out[1]), "=&v"(out[2]), "=&v"(out[3])
        : "v"(addr[0]), "v"(addr[1]), "v"(addr[2]), "v"(addr[3])
        : "memory");
  } else {
    asm volatile(
        "ds_read_b64_tr_b16 %0, %8\n\t"
        "ds_read_b64_tr_b16 %1, %9\n\t"
        "ds_read_b64_tr_b16 %2, %10\n\t"
        "ds_read_b64_tr_b16 %3, %11\n\t"
        "ds_read_b64_tr_b16 %4, %12\n\t"
        "ds_read_b64_tr_b16 %5, %13\n\t"
        "ds_read_b64_tr_b16 %6, %14\n\t"
        "ds_read_b64_tr_b16 %7, %15\n\t"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(out[0]), "=&v"(out[1]), "=&v"(out[2]), "=&v"(out[3]),
          "=&v"(out[4]), "=&v"(out[5]), "=&v"(out[6]), "=&v"(out[7])
        : "v"(addr[0]), "v"(addr[1]), "v"(addr[2]), "v"(addr[3]),
          "v"(addr[4]), "v"(addr[5]), "v"(addr[6]), "v"(addr[7])
        : "memory");
  }
}

// a0 or a1 by a wave-uniform flag, as selects rather than a branch (the u
// products take the odd or even row blocks of A by the wave's column half)
__device__ __forceinline__ bf16x8 pick_frag(const bf16x8& a0, const bf16x8& a1, bool second) {
  const u32x4 x = __builtin_bit_cast(u32x4, a0), y = __builtin_bit_cast(u32x4, a1);
  u32x4 r;
#pragma unroll
  for (int e = 0; e < 4; ++e) r[e] = second ? y[e] : x[e];
  return __builtin_bit_cast(bf16x8, r);
}

// 32-bit LDS address of a pointer into a __shared__ array.
__device__ __forceinline__ uint32_t lds_addr(const void* p) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) char*)p;
}

// An x tile from the 8-bit row checkpoint: sixteen codes of one row per
// thread and unit, loaded to registers (fetch) and written (put) as exact
// bfloat16 integers in the layout of the bf16 tile (swizzled 128-byte row
// halves), so that the dA products read either tile alike. Half the bytes of
// bf16 rows; the rows' scales stay out of the rounding (they multiply u or
// the float32 products). thr: the thread among the 256 that share the tile.
// Rows past M are zero, as are columns past K.
template <int BM, int BN>
struct X8Tile {
  static constexpr int NU = BM * BN / 4096, UPR = BN / 16, RH = BN / 64;
  u32x4 v[NU];
  __device__ __forceinline__ void fetch(const int8_t* xq, int M, int K, int m0, int k0, int thr) {
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      const int u = thr + 256 * i, gm = m0 + u / UPR, gk = k0 + 16 * (u % UPR);
      const bool ok = gm < M && gk < K;
      const u32x4 w = *reinterpret_cast<const u32x4*>(xq + (ok ? (long)gm * K + gk : 0));
      v[i] = ok ? w : u32x4{0u, 0u, 0u, 0u};
    }
  }
  __device__ __forceinline__ void put(int8_t* Xs, int thr) const {
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      const int u = thr + 256 * i, row = u / UPR, col = 16 * (u % UPR);
      const int hrow = row * RH + col / 64, c = (col % 64) / 8;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        u32x4 o;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t w = v[i][2 * h + e];
          o[2 * e] = pack_int_bf16x2((int8_t)w, (int8_t)(w >> 8));
          o[2 * e + 1] = pack_int_bf16x2((int8_t)(w >> 16), (int8_t)(w >> 24));
        }
        *reinterpret_cast<u32x4*>(Xs + swz128(hrow, c + h)) = o;
      }
    }
  }
};

// The u operand of the dA products, [UCB][BM / 32][64 lanes][16 B] at UF: u [BM
// rows][R] at E split like B and t into bf16 hi, mid and lo columns, rows past
// `rows` zero. Wave w of four builds fragments w, w + 4, ... With x in 8 bits
// (x8) rows are first multiplied by their scales in float32: rsv[e] is that of
// row 32 (w % (BM / 32)) + 8 (lane / 16) + e, the rows of all its fragments.
template <int BM, int R>
__device__ __forceinline__ void put_u_operand(int8_t* UF, const float* E, int rows, int r, bool x8,
                                              const float (&rsv)[8]) {
  constexpr int UCB = (3 * R + 15) / 16, MC = BM / 32;
  static_assert(4 % MC == 0, "a wave's fragments are all of the same rows");
  const int lane = threadIdx.x & 63, wid = wave_id();
  for (int f = wid; f < UCB * MC; f += 4) {
    const int cb = f / MC, c = f % MC;
    const int j = cb * 16 + (lane & 15), part = j / R, jr = j - part * R;
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int m = 32 * c + 8 * (lane >> 4) + e;
      v[e] = (jr < r && part < 3 && m < rows) ? E[m * R + (jr < r ? jr : 0)] : 0.f;
      if (x8) v[e] = m < rows ? v[e] * rsv[e] : 0.f;      // (a clamped row's scale may be NaN)
    }
    u32x4 hi, mid, lo;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      uint32_t me, le;
      hi[e] = pk_bf16_split3(v[2 * e], v[2 * e + 1], me, le);
      mid[e] = me;
      lo[e] = le;
    }
    *reinterpret_cast<u32x4*>(UF + (f * 64 + lane) * 16) = part == 0 ? hi : part == 1 ? mid : lo;
  }
}

// The dA partial of a block on the matrix cores: dA^T[k][j] = sum_m x[m][k]
// u[m][j] over its rows, u from the operand above and x^T read from the x tile
// through transposing reads (in each 16-lane group lane 4 i + p fetches the 4
// columns at c0 + 4 p of row i, and lane q receives column c0 + q of rows
// 0..3). Wave w of four takes the columns [BN / 4 w, BN / 4 (w + 1)) and writes
// out[j K + k] for the block's columns k0 + k < K. sx (x in 8 bits, else NULL):
// the scales of the block's rows.
template <int BM, int BN, int R>
__device__ __forceinline__ void da_products(const int8_t* Xs, const int8_t* UF, const float* E, const float* sx,
                                            int rows, int r, int k0, int K, float* out) {
  constexpr int UCB = (3 * R + 15) / 16, RCB = (R + 15) / 16, MC = BM / 32;
  constexpr int KB = BN / 64, RH = BN / 64;               // 16-column blocks per wave
  const int lane = threadIdx.x & 63, wid = wave_id();
  f32x4 dacc[KB][UCB];
#pragma unroll
  for (int kb = 0; kb < KB; ++kb)
#pragma unroll
    for (int cb = 0; cb < UCB; ++cb) dacc[kb][cb] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int q = lane & 15, i4 = q >> 2, p4 = q & 3;
#pragma unroll
  for (int c0 = 0; c0 < MC; c0 += 2) {
    uint32_t tra[4 * KB];
    uint64_t trv[4 * KB];
#pragma unroll
    for (int cc = 0; cc < 2; ++cc)
#pragma unroll
      for (int kb = 0; kb < KB; ++kb)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int m = 32 * (c0 + cc) + 8 * (lane >> 4) + 4 * h + i4;
          const int col = (BN / 4) * wid + 16 * kb + 4 * p4;
          tra[(cc * KB + kb) * 2 + h] = lds_addr(Xs + swz128(m * RH + col / 64, (col % 64) >> 3) + (col & 7) * 2);
        }
    tr16_reads<4 * KB>(tra, trv);
#pragma unroll
    for (int cc = 0; cc < 2; ++cc) {
      const int c = c0 + cc;
      bf16x8 uf[UCB];
#pragma unroll
      for (int cb = 0; cb < UCB; ++cb)
        uf[cb] = *reinterpret_cast<const bf16x8*>(UF + ((cb * MC + c) * 64 + lane) * 16);
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
        const int t0 = (cc * KB + kb) * 2;
        const bf16x8 xT = __builtin_bit_cast(bf16x8, u32x4{(uint32_t)trv[t0], (uint32_t)(trv[t0] >> 32),
                                                           (uint32_t)trv[t0 + 1], (uint32_t)(trv[t0 + 1] >> 32)});
#pragma unroll
        for (int cb = 0; cb < UCB; ++cb)
          dacc[kb][cb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xT, uf[cb], dacc[kb][cb], 0, 0, 0);
      }
    }
  }
  float dav[KB][RCB][4];
  bool nan = false;
#pragma unroll
  for (int kb = 0; kb < KB; ++kb)
#pragma unroll
    for (int cb = 0; cb < RCB; ++cb)
#pragma unroll
      for (int ii = 0; ii < 4; ++ii) {
        dav[kb][cb][ii] = split3_sum<R, UCB>(dacc[kb], cb, ii, lane);
        nan |= dav[kb][cb][ii] != dav[kb][cb][ii];
      }
  if (__builtin_amdgcn_ballot_w64(nan) == 0) {
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
      for (int cb = 0; cb < RCB; ++cb) {
        const int j = cb * 16 + (lane & 15);
#pragma unroll
        for (int ii = 0; ii < 4; ++ii) {
          const int kl = (BN / 4) * wid + 16 * kb + 4 * (lane >> 4) + ii;
          if (j < r && k0 + kl < K) out[(long)j * K + k0 + kl] = dav[kb][cb][ii];
        }
      }
  } else {
    // A NaN in the wave's columns: an infinite x times the three parts of
    // u can give inf - inf where the plain product is infinite, so the
    // wave takes its columns again as float32 sums in row order (lane ->
    // column (BN / 4) w + lane % (BN / 4), ranks jb + TPK jj).
    constexpr int CPW = BN / 4, TPK = 64 / CPW, JPT = (R + TPK - 1) / TPK;
    const int kl = CPW * wid + lane % CPW, jb = lane / CPW;
    float da[JPT];
#pragma unroll
    for (int jj = 0; jj < JPT; ++jj) da[jj] = 0.f;
    for (int m = 0; m < rows; ++m) {
      const int e = kl % 64;
      const uint16_t xb = *reinterpret_cast<const uint16_t*>(Xs + swz128(m * RH + kl / 64, e >> 3) + 2 * (e & 7));
      float xv = __uint_as_float((uint32_t)xb << 16);
      if (sx != nullptr) xv *= sx[m];
#pragma unroll
      for (int jj = 0; jj < JPT; ++jj)
        if (jb + TPK * jj < R) da[jj] = __builtin_fmaf(xv, E[m * R + jb + TPK * jj], da[jj]);
    }
#pragma unroll
    for (int jj = 0; jj < JPT; ++jj) {
      const int j = jb + TPK * jj;
      if (j < r && k0 + kl < K) out[(long)j * K + k0 + kl] = da[jj];
    }
  }
}

// The eight codes of a packed 4-bit word (nibble e = k offset e, two's
// complement) times sc: w ^ 0x88888888 turns each code q into q + 8 in
// [0, 15], two masks spread the nibbles over bytes (v_cvt_f32_ubyte takes a
// byte in one instruction), and fma(q + 8, sc, -8 sc) rounds q sc exactly
// once, as q * sc would.
__device__ __forceinline__ void nibble_vals(uint32_t w, float sc, float (&v)[8]) {
  const uint32_t u = w ^ 0x88888888u;
  const uint32_t lo = u & 0x0f0f0f0fu, hi = (u >> 4) & 0x0f0f0f0fu;   // even, odd e
  const float nsc = -8.f * sc;
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    v[2 * b] = __builtin_fmaf((float)((lo >> (8 * b)) & 0xffu), sc, nsc);
    v[2 * b + 1] = __builtin_fmaf((float)((hi >> (8 * b)) & 0xffu), sc, nsc);
  }
}

}  // namespace qlora
