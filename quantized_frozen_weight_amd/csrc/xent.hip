// Softmax cross entropy of the vocabulary layer and its gradient, the logits
// never in memory (formulas: include/qlora.h).
//
// logits kernel  The layer's integer product over tiles of the vocabulary, both
//   operands K-contiguous rows that move from memory to LDS untouched
//   (ring.hpp); 4-bit codes are widened in registers, as 16 q in the upper half
//   of a byte (no sign to extend: the tile took 250 us at 1024 x 4096 x 32000 with
//   it), and their exact sums weighted group by group. What a tile does with its
//   logits:
//   - loss: each row's maximum and sum of exp2 over the tile's columns, lanes by
//     DPP, waves through LDS, 8 bytes a row and tile to the workspace; the
//     target's logit from the tile that holds it. A second, small launch joins
//     the tiles in a fixed order;
//   - gradient: dl = dloss (exp2(l log2e - lse log2e) - [target]) for one piece
//     of the vocabulary, in float16 (int8 weights: times the entry's scale, so that
//     the next product multiplies with the codes, which float16 holds exactly), and
//     with an adapter the tile's parts of u = dl B^T and dB = t^T dl from the
//     float32 dl in three bf16 parts.
// dx kernel      dx += dl W over one piece: dl rows K-contiguous, W as stored,
//   codes [v][d], contracted over v. The 16-bit operand that a matrix
//   instruction wants of W is eight v of one d: a lane reads one dword (4 d) of
//   eight rows v, and takes byte j of each for its j-th column block, so that
//   the transposition costs no instruction beside the conversion, and the four
//   column blocks of a lane are four consecutive d of the output. Float32 dl
//   comes as three bf16 parts, the contraction run over each. The contraction of
//   a piece is split where there are few tiles; every split adds into a float32
//   buffer of its own, piece after piece.
// Pieces are as large as 256 MB of dl allow, and of at least 512 entries. Sums are in a fixed order.
// 2048 x 2048 over 256000 entries: loss 963 us (2.2 POP/s), the gradient's logits 1090,
// dx 1894 (1.13 PFLOP/s; a large library product in bf16 reaches 1.24), all three at
// 40 to 50 % of the matrix units' time with the vector units a third busy. At 768
// features a tile's six stages of products are as long as its exponentials behind them
// (4096 x 768 over 50257: 232 us, 1.36 POP/s). One row: the weight's bytes, 5.9 TB/s.
#include "abi.hpp"
#include "bwd_common.hpp"
#include "launch.hpp"
#include "nibbles.hpp"
#include "rank_sums.hpp"
#include "ring.hpp"
#include "vocab.hpp"

#include <type_traits>

namespace qlora {

namespace {

constexpr int kCUs = 256;
constexpr int kFewTiles = 64;      // of 128 x 128: up to so many are taken as 32 x 256
constexpr int kHalfTiles = 160;    // of 256 x 256: up to so many are taken as 128 x 128
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kNone = -(1 << 30);  // no target: far from every tile (a column is above -2^27)

// Block b of nb as a position in an order that each XCD (every eighth block)
// walks a contiguous part of.
__device__ __forceinline__ int xcd_order(int b, int nb) {
  const int x = b & 7, per = nb >> 3, rest = nb & 7;
  return x * per + (x < rest ? x : rest) + (b >> 3);
}

struct LogitArgs {
  int M, N, K, V, r;
  const int8_t* xq;      // [M, K]
  const float* sx;       // [M]
  const int8_t* codes;   // [N, K], or packed [N, K / 2]
  const void* scales;    // [N], or fp16 [N, K / 128]
  const float* t;        // [M, r]
  const float* B;        // [r, N]
  float s;
  Ids ids;
  int v0, tiles_m, tiles_x;       // first entry, tiles of this launch
  // loss
  float* part;           // [tiles_x][M] pairs (maximum, sum), in powers of two
  float* tl;             // [M] the target's logit
  // gradient
  const float* lse;
  const float* dloss;
  const uint32_t* smax;  // [64] partial maxima of the scales (int8, dl in float16)
  uint16_t* g;           // [parts][M][ldg]
  long ldg, gstride;
  float* up;             // [tiles_x][M][r]
  float* dbp;            // [tiles_m][r][ldg]
};

// Maximum and sum over the four lanes that hold one row of a transposed block
// (lanes l, l + 16, l + 32, l + 48); every one of them ends with the result.
__device__ __forceinline__ float quad_max(float v) {
  const uint32_t b = __float_as_uint(v);
  const auto s32 = __builtin_amdgcn_permlane32_swap(b, b, false, false);
  v = fmaxf(__uint_as_float(s32[0]), __uint_as_float(s32[1]));
  const uint32_t c = __float_as_uint(v);
  const auto s16 = __builtin_amdgcn_permlane16_swap(c, c, false, false);
  return fmaxf(__uint_as_float(s16[0]), __uint_as_float(s16[1]));
}
__device__ __forceinline__ float quad_sum(float v) {
  const uint32_t b = __float_as_uint(v);
  const auto s32 = __builtin_amdgcn_permlane32_swap(b, b, false, false);
  v = __uint_as_float(s32[0]) + __uint_as_float(s32[1]);
  const uint32_t c = __float_as_uint(v);
  const auto s16 = __builtin_amdgcn_permlane16_swap(c, c, false, false);
  return __uint_as_float(s16[0]) + __uint_as_float(s16[1]);
}

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ uint32_t pk_f16(float lo, float hi) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{lo, hi}, f16x2));
}

// Four values as bf16 (packed), and what that leaves of them (0 of an infinity
// or a NaN, whose first part is all).
__device__ __forceinline__ u32x2 bf16_part(float (&v)[4]) {
  u32x2 h;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    h[e] = pk_bf16(v[2 * e], v[2 * e + 1]);
    const bool fa = (h[e] & 0x7f80u) != 0x7f80u, fb = (h[e] & 0x7f800000u) != 0x7f800000u;
    v[2 * e] = fa ? v[2 * e] - __uint_as_float(h[e] << 16) : 0.f;
    v[2 * e + 1] = fb ? v[2 * e + 1] - __uint_as_float(h[e] & 0xffff0000u) : 0.f;
  }
  return h;
}

// The same of values that are no infinities.
__device__ __forceinline__ u32x2 bf16_cut(float (&v)[4]) {
  u32x2 h;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    h[e] = pk_bf16(v[2 * e], v[2 * e + 1]);
    v[2 * e] -= __uint_as_float(h[e] << 16);
    v[2 * e + 1] -= __uint_as_float(h[e] & 0xffff0000u);
  }
  return h;
}

typedef short s16x4 __attribute__((ext_vector_type(4)));

// dl in 16 bits is float16, 11 bits where bf16 has 8 (dx of 2048 x 2048 x 256000 was
// off by 0.26 % from the definition with bf16, where rounding dx alone is 0.17).
// What travels is p - [target] without dloss (the rows' factor, applied where rows
// end), scaled so that the largest is 2^14 and 2^-24 of that still has all bits:
// int8 weights: 2^14 (p - [target]) scale / 2^E, E the smallest (at least -100) with
// every scale below 2^E (a power of two: nothing more is rounded), against the codes;
// 4-bit weights: 2^14 (p - [target]), against q scale 2^(13 - E) in float16, E of
// the same kind: 8 times the largest scale then fits, and a scale keeps its bits
// down to 2^-26 of that (a fixed 1 / 8 lost those of scales under 2^-11, and from
// 2^-22 on all of them: dx of weights of 2e-5 was off by 5 %).
constexpr float kHalfUp = 16384.f;
constexpr int kHalfBits = 14, kHalfBits4 = 14 + 13;      // dx is formed times 2^(this - E)

// The largest of n scales (float32, or 4-bit weights' float16), by 64 partial maxima
// (scales that are no numbers left out: what they enter is none either way).
constexpr int kMaxParts = 64;
template <typename S>
__global__ __launch_bounds__(1024) void xent_scale_max_kernel(const S* scales, int n, uint32_t* part) {
  __shared__ uint32_t red[16];
  uint32_t mx = 0u;
#pragma unroll 4
  for (long i = blockIdx.x * 1024 + threadIdx.x; i < n; i += 1024 * kMaxParts) {
    const uint32_t b = abs_bits((float)scales[i]);
    mx = b < 0x7f800000u && b > mx ? b : mx;
  }
  mx = wave_max_u32(mx);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = mx;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < 16; ++w) mx = red[w] > mx ? red[w] : mx;
    part[blockIdx.x] = mx;
  }
}
// E of the above from a lane's partial maximum; every lane of the wave.
__device__ __forceinline__ int scale_power(uint32_t part) {
  const int e = (int)(wave_max_u32(part) >> 23) - 126;
  return e < -100 ? -100 : e;
}

constexpr int max_int(int a, int b) { return a > b ? a : b; }

// LDS of a logits block, in bytes. Stage: BM + BN rows of 128 bytes (4-bit: 64
// bytes of codes a row), S of them, and the 4-bit scales; after the loop the
// same bytes hold the epilogue's operands, and for the gradient the waves'
// strips and (with an adapter) the tile's sums.
template <bool W4, int BM, int BN, int WM, int WN, int S, int G, int R, bool GRAD>
struct LogitLds {
  static constexpr int NW = WM * WN, FN = BN / WN / 16;
  static constexpr int ASZ = BM * 128, STG = ASZ + BN * (W4 ? 64 : 128);
  static constexpr int SLAB = W4 ? BN * G * 2 : 0;
  static constexpr int QP = BN + 4;                       // pitch of B's rows
  static constexpr int TS = 0, QS = TS + BM * R * 4, RS = QS + R * QP * 4, SW = RS + BM * 4;
  static constexpr int TG = SW + BN * 4, LS = TG + BM * 4, END = LS + BM * 4;
  static constexpr int RED = WN * BM * 8;                 // loss: the waves' maxima and sums
  // gradient: t dloss in three bf16 parts [3][R][TP]; a wave's 16 rows of dl, in
  // three parts for dB, then as they go to memory (afterwards u [BM][R] and dB [R][BN])
  static constexpr int TP = BM + 8, TB = END, PITCH = FN * 32 + 16, PVB = 16 * PITCH;
  static constexpr int ST = TB + (GRAD ? 3 * R * TP * 2 : 0), STRIP = (R > 0 ? 3 : 1) * PVB;
  static constexpr int SUMS = (BM + BN) * R * 4;
  static constexpr int EPI = GRAD ? ST + max_int(NW * STRIP, SUMS) : END + RED;
  static constexpr int BYTES = max_int(S * STG + SLAB, EPI);
  static_assert(BYTES <= 160 * 1024, "LDS of a block");
};

// PARTS: 0 the loss, 1 the gradient with dl in 16 bits, 3 in three bf16 parts.
template <bool W4, int BM, int BN, int WM, int WN, int S, int G, int R, int PARTS>
__global__ __launch_bounds__(64 * WM * WN) void xent_logits_kernel(LogitArgs a) {
  constexpr bool GRAD = PARTS > 0, HALF = PARTS == 1;      // HALF: dl in float16
  using Lds = LogitLds<W4, BM, BN, WM, WN, S, G, R, GRAD>;
  constexpr int NW = WM * WN, NT = 64 * NW, BK = 128;
  constexpr int ASZ = Lds::ASZ, STG = Lds::STG;
  constexpr int FM = BM / WM / 16, FN = BN / WN / 16;
  // loads per wave and stage: 8 rows of 128 bytes (16 of 64) an instruction
  constexpr int AI = BM / 8 / NW, BI = BN / (W4 ? 16 : 8) / NW, LPS = AI + BI;
  static_assert(AI * 8 * NW == BM && BI * (W4 ? 16 : 8) * NW == BN, "whole instructions per wave");
  static_assert(BK == 128, "two steps of 64 a stage");
  __shared__ __attribute__((aligned(1024))) int8_t lds[Lds::BYTES];
  int8_t* ring = lds;
  const _Float16* SC = reinterpret_cast<const _Float16*>(lds + S * STG);

  const int tid = threadIdx.x, lane = tid & 63, wid = wave_id();
  const int l = lane & 15, q = lane >> 4;
  const int wm = wid / WN, wn = wid % WN;
  const int M = a.M, N = a.N, K = a.K;
  const int nk = (K + BK - 1) / BK;
  // an XCD walks whole columns of tiles: the codes come from memory once
  const int order = xcd_order((int)blockIdx.x, a.tiles_m * a.tiles_x);
  const int mt = order % a.tiles_m, ct = order / a.tiles_m;
  const int m0 = mt * BM, c0 = ct * BN, n0 = a.v0 + c0;

  // the epilogue's operands into registers, consumed after the loop
  constexpr int RT = (BM + NT - 1) / NT, CT = (BN + NT - 1) / NT;
  constexpr int NTS = (BM * R + NT - 1) / NT, NQS = (BN * R + NT - 1) / NT;
  constexpr int NTA = NTS > 0 ? NTS : 1;
  float esx[RT], else_[RT], esw[CT], ets[NTA], egm[NTA], eqs[NQS > 0 ? NQS : 1];
  int etg[RT], etr[NTA];                                   // targets, by row and by element of t
  uint32_t emax = 0u;
  if constexpr (HALF && !W4) emax = a.smax[lane];
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    const int row = tid + NT * i, gm = m0 + row < M ? m0 + row : M - 1;
    esx[i] = a.sx[gm];
    etg[i] = row < BM && m0 + row < M ? entry_of(a.ids, gm) : -1;
    if constexpr (GRAD) else_[i] = a.lse[gm];
  }
  if constexpr (!W4) {
#pragma unroll
    for (int i = 0; i < CT; ++i) {
      const int gn = n0 + tid + NT * i;
      esw[i] = static_cast<const float*>(a.scales)[gn < N ? gn : N - 1];
    }
  }
  if constexpr (R > 0) {
#pragma unroll
    for (int i = 0; i < NTS; ++i) {
      const int e = tid + NT * i, j = e % R, gm = m0 + e / R < M ? m0 + e / R : M - 1;
      ets[i] = a.t[(long)gm * a.r + (j < a.r ? j : 0)];
      if constexpr (GRAD) {
        etr[i] = entry_of(a.ids, gm);
        egm[i] = a.dloss[gm];
      }
    }
#pragma unroll
    for (int i = 0; i < NQS; ++i) {
      const int e = tid + NT * i, j = e / BN, gn = n0 + e % BN;
      eqs[i] = a.B[(long)(j < a.r ? j : 0) * N + (gn < N ? gn : N - 1)];
    }
  }
  const int ngrp = K / 128;
  if constexpr (W4) {
    // the tile's scales [BN][ngrp], contiguous in memory
    const int bytes = BN * ngrp * 2;
    const int8_t* src0 = static_cast<const int8_t*>(a.scales) + (long)n0 * ngrp * 2;
    const long valid = ((long)N - n0) * ngrp * 2;
    for (int o = wid * 1024; o < bytes; o += NW * 1024) {
      const int e = o + lane * 16;
      lds_dma16(e < bytes && e < valid ? src0 + e : zero_chunk(lane), lds + S * STG + o);
    }
  }

  // rows past M and entries past N repeat the last one
  uint32_t voA[AI], voB[BI];
#pragma unroll
  for (int i = 0; i < AI; ++i) {
    const int row = (wid * AI + i) * 8 + (lane >> 3), gm = m0 + row;
    voA[i] = (uint32_t)((long)(gm < M ? gm : M - 1) * K + ((lane & 7) ^ ((row >> 1) & 7)) * 16);
  }
#pragma unroll
  for (int i = 0; i < BI; ++i) {
    if constexpr (W4) {
      const int row = (wid * BI + i) * 16 + (lane >> 2), gn = n0 + row;
      voB[i] = (uint32_t)((long)(gn < N ? gn : N - 1) * (K / 2) + ((lane & 3) ^ ((row >> 2) & 3)) * 16);
    } else {
      const int row = (wid * BI + i) * 8 + (lane >> 3), gn = n0 + row;
      voB[i] = (uint32_t)((long)(gn < N ? gn : N - 1) * K + ((lane & 7) ^ ((row >> 1) & 7)) * 16);
    }
  }
  auto issue = [&](int kt, int slot) {
    int8_t* base = ring + slot * STG;
    const int8_t* xb = a.xq + kt * BK;
    const int8_t* cb = a.codes + kt * (W4 ? BK / 2 : BK);
    if (W4 || (kt + 1) * BK <= K) {                        // (4-bit: K % 128 == 0)
#pragma unroll
      for (int i = 0; i < AI; ++i) lds_dma16(xb + voA[i], base + (wid * AI + i) * 1024);
#pragma unroll
      for (int i = 0; i < BI; ++i) lds_dma16(cb + voB[i], base + ASZ + (wid * BI + i) * 1024);
      return;
    }
    // the ragged last stage: chunks past K are zero
#pragma unroll
    for (int i = 0; i < AI; ++i) {
      const int row = (wid * AI + i) * 8 + (lane >> 3), c = (lane & 7) ^ ((row >> 1) & 7);
      lds_dma16(kt * BK + c * 16 < K ? xb + voA[i] : zero_chunk(lane), base + (wid * AI + i) * 1024);
    }
#pragma unroll
    for (int i = 0; i < BI; ++i) {
      const int row = (wid * BI + i) * 8 + (lane >> 3), c = (lane & 7) ^ ((row >> 1) & 7);
      lds_dma16(kt * BK + c * 16 < K ? cb + voB[i] : zero_chunk(lane), base + ASZ + (wid * BI + i) * 1024);
    }
  };

  typedef typename std::conditional<W4, f32x4, i32x4>::type Acc;
  Acc acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = Acc{0, 0, 0, 0};

#pragma unroll
  for (int st = 0; st < S - 1; ++st)
    if (st < nk) issue(st, st);
  int slot = 0;
  for (int kt = 0; kt < nk; ++kt) {
    wait_stages<LPS, 0, S - 2>(nk - 1 - kt);               // stage kt has landed (this wave)
    __builtin_amdgcn_s_barrier();                          // ... for every wave; slot of kt - 1 is free
    if (kt + S - 1 < nk) issue(kt + S - 1, slot == 0 ? S - 1 : slot - 1);
    const int8_t* As = ring + slot * STG;
    const int8_t* Bs = As + ASZ;
    i32x4 part[W4 ? FM : 1][W4 ? FN : 1];
    if constexpr (W4) {
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) part[i][j] = i32x4{0, 0, 0, 0};
    }
    i32x4 af[2][FM], bf[2][FN];
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      const int c = kk * 4 + q;
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const int n = (wn * FN + j) * 16 + l;
        if constexpr (W4)
          bf[kk][j] = widen_nibbles16(*reinterpret_cast<const u32x2*>(Bs + n * 64 + (((c >> 1) ^ ((n >> 2) & 3)) << 4) +
                                                                     (c & 1) * 8));
        else
          bf[kk][j] = *reinterpret_cast<const i32x4*>(Bs + swz128(n, c));
      }
#pragma unroll
      for (int i = 0; i < FM; ++i)
        af[kk][i] = *reinterpret_cast<const i32x4*>(As + swz128((wm * FM + i) * 16 + l, c));
    }
#pragma unroll
    for (int kk = 0; kk < 2; ++kk)
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          // transposed: lane l holds row l of the block, entries 4 q .. 4 q + 3
          if constexpr (W4)
            part[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(bf[kk][j], af[kk][i], part[i][j], 0, 0, 0);
          else
            acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(bf[kk][j], af[kk][i], acc[i][j], 0, 0, 0);
        }
    if constexpr (!W4) {
      // The order of the stage's instructions: the operands of the first products,
      // then two reads behind every FN products until all are under way (left to
      // itself the compiler waits for every pair of reads before the next eight)
      __builtin_amdgcn_sched_group_barrier(0x100, FN + 2, 0);
#pragma unroll
      for (int g = 0; g < (2 * (FM + FN) - FN - 2) / 2; ++g) {
        __builtin_amdgcn_sched_group_barrier(0x008, FN, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
      }
      __builtin_amdgcn_sched_group_barrier(0x008, 2 * FM * FN - FN * ((2 * (FM + FN) - FN - 2) / 2), 0);
    }
    if constexpr (W4) {
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        float sc[4];
#pragma unroll
        for (int ii = 0; ii < 4; ++ii) sc[ii] = (float)SC[((wn * FN + j) * 16 + 4 * q + ii) * ngrp + kt];
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
          for (int ii = 0; ii < 4; ++ii)
            acc[i][j][ii] = __builtin_fmaf((float)part[i][j][ii], sc[ii], acc[i][j][ii]);
      }
    }
    slot = slot == S - 1 ? 0 : slot + 1;
  }

  __syncthreads();                                         // every wave is done with the ring
  float* ts = reinterpret_cast<float*>(lds + Lds::TS);     // s log2e t
  float* qs = reinterpret_cast<float*>(lds + Lds::QS);     // B
  float* rsv = reinterpret_cast<float*>(lds + Lds::RS);    // log2e sx
  float* swv = reinterpret_cast<float*>(lds + Lds::SW);
  int* tgv = reinterpret_cast<int*>(lds + Lds::TG);        // the target's column here, or kNone
  float* lsv = reinterpret_cast<float*>(lds + Lds::LS);    // log2e lse
  uint16_t* tb = reinterpret_cast<uint16_t*>(lds + Lds::TB);
  // int8, dl in float16: the scales times 2^(14 - E), the rows' the other way round
  const int power = HALF && !W4 ? kHalfBits - scale_power(emax) : 0;
  const float up = __builtin_ldexpf(1.f, power), down = __builtin_ldexpf(1.f, -power);
  // Gradient: a row without a target has logits 0 and lse infinite, so that its
  // p is 0 whatever its x is (and is set to 0 below, for weights that are no numbers).
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    const int row = tid + NT * i;
    if (row < BM) {
      const bool none = GRAD && etg[i] < 0;
      rsv[row] = none ? 0.f : esx[i] * (W4 ? kLog2e / 16.f : kLog2e) * down;   // (4-bit: the products are those of 16 q)
      tgv[row] = etg[i] >= 0 ? etg[i] - n0 : kNone;
      if constexpr (GRAD) lsv[row] = none ? INFINITY : else_[i] * kLog2e;
    }
  }
  if constexpr (!W4) {
#pragma unroll
    for (int i = 0; i < CT; ++i)
      if (tid + NT * i < BN) swv[tid + NT * i] = n0 + tid + NT * i < a.V ? esw[i] * up : 0.f;
  }
  if constexpr (R > 0) {
#pragma unroll
    for (int i = 0; i < NTS; ++i) {
      const int e = tid + NT * i, row = e / R, j = e % R;
      if (e < BM * R) {
        const bool in = j < a.r && m0 + row < M && !(GRAD && etr[i] < 0);
        ts[e] = in ? ets[i] * (a.s * kLog2e) : 0.f;
        if constexpr (GRAD) {
          uint32_t mid, low;
          const uint32_t hi = pk_bf16_split3(in ? ets[i] * egm[i] : 0.f, 0.f, mid, low);
          tb[j * Lds::TP + row] = (uint16_t)hi;
          tb[(R + j) * Lds::TP + row] = (uint16_t)mid;
          tb[(2 * R + j) * Lds::TP + row] = (uint16_t)low;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < NQS; ++i) {
      const int e = tid + NT * i, j = e / BN, c = e % BN;
      if (e < BN * R) qs[j * Lds::QP + c] = j < a.r && n0 + c < a.V ? eqs[i] : 0.f;
    }
  }
  __syncthreads();

  const int wr0 = wm * FM * 16, wc0 = wn * FN * 16;
  const bool ragged = n0 + wc0 + FN * 16 > a.V;            // wave-uniform: some columns are no entries
  constexpr int RB = (R + 15) / 16, RBA = RB > 0 ? RB : 1;
  constexpr bool ADAPT = GRAD && R > 0;
  f32x4 sw[FN];
#pragma unroll
  for (int j = 0; j < FN; ++j)
    sw[j] = W4 ? f32x4{1.f, 1.f, 1.f, 1.f} : *reinterpret_cast<const f32x4*>(swv + wc0 + j * 16 + 4 * q);

  // u's operand, B of two column blocks (32 entries in the order in which a lane
  // holds them), in three bf16 parts
  constexpr int NP = FN / 2;
  static_assert(FN % 2 == 0 && FM % 2 == 0, "blocks are taken in pairs");
  u32x4 bp[3][ADAPT ? NP : 1][RBA];
  f32x4 uacc[ADAPT ? FM : 1][RBA], dbacc[ADAPT ? FN : 1][RBA];
  if constexpr (ADAPT) {
#pragma unroll
    for (int jb = 0; jb < RB; ++jb) {
      const int rank = 16 * jb + l;
#pragma unroll
      for (int p = 0; p < NP; ++p)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const f32x4 b4 = *reinterpret_cast<const f32x4*>(qs + (rank < R ? rank : 0) * Lds::QP + wc0 + 32 * p + 16 * h + 4 * q);
          float v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = rank < R ? b4[e] : 0.f;
#pragma unroll
          for (int c = 0; c < 3; ++c) {
            const u32x2 w = bf16_part(v);
            bp[c][p][jb][2 * h] = w.x;
            bp[c][p][jb][2 * h + 1] = w.y;
          }
        }
#pragma unroll
      for (int i = 0; i < FM; ++i) uacc[i][jb] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < FN; ++i) dbacc[i][jb] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
  }
  int8_t* strip = lds + Lds::ST + wid * Lds::STRIP;

#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const int row = wr0 + i * 16 + l;                      // the lane's row of the tile
    const float rs = rsv[row];
    const int tg = tgv[row] - wc0;                         // its target among the wave's columns
    const bool hit = __builtin_amdgcn_ballot_w64(tg >= 0 && tg < FN * 16) != 0;
    const float base = GRAD ? -lsv[row] : 0.f;
    // x: logits in powers of two (gradient: minus lse)
    float x[FN][4];
    f32x4 lo[FN];
    if constexpr (R > 0) {
#pragma unroll
      for (int j = 0; j < FN; ++j) lo[j] = f32x4{base, base, base, base};
#pragma unroll
      for (int kc = 0; kc < R / 4; ++kc) {
        const float tv = ts[row * R + kc * 4 + q];
#pragma unroll
        for (int j = 0; j < FN; ++j)
          lo[j] = __builtin_amdgcn_mfma_f32_16x16x4f32(qs[(kc * 4 + q) * Lds::QP + wc0 + j * 16 + l], tv, lo[j], 0, 0, 0);
      }
    }
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int ii = 0; ii < 4; ++ii) {
        const float t = W4 ? (float)acc[i][j][ii] : (float)acc[i][j][ii] * sw[j][ii];
        x[j][ii] = R > 0 ? __builtin_fmaf(rs, t, lo[j][ii]) : GRAD ? __builtin_fmaf(rs, t, base) : rs * t;
      }
    if constexpr (!GRAD) {
      float* red = reinterpret_cast<float*>(lds + Lds::END);      // [WN][BM] pairs
      if (hit) {
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
          for (int ii = 0; ii < 4; ++ii)
            if (j * 16 + 4 * q + ii == tg) a.tl[m0 + row] = x[j][ii];   // (a row past M has no target)
      }
      if (ragged) {
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
          for (int ii = 0; ii < 4; ++ii)
            if (n0 + wc0 + j * 16 + 4 * q + ii >= a.V) x[j][ii] = -INFINITY;
      }
      float mx = -INFINITY;
#pragma unroll
      for (int j = 0; j < FN; ++j)
        mx = fmaxf(mx, fmaxf(fmaxf(x[j][0], x[j][1]), fmaxf(x[j][2], x[j][3])));
      mx = quad_max(mx);
      const float ref = mx == -INFINITY ? 0.f : mx;        // (no entry here)
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < FN; ++j)
        sum += (__builtin_amdgcn_exp2f(x[j][0] - ref) + __builtin_amdgcn_exp2f(x[j][1] - ref)) +
               (__builtin_amdgcn_exp2f(x[j][2] - ref) + __builtin_amdgcn_exp2f(x[j][3] - ref));
      sum = quad_sum(sum);
      if (q == 0) {
        red[2 * (wn * BM + row)] = mx;
        red[2 * (wn * BM + row) + 1] = sum;
      }
    } else {
      // p - [target], without dloss (the rows' factor, applied where rows end)
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int ii = 0; ii < 4; ++ii) x[j][ii] = __builtin_amdgcn_exp2f(x[j][ii]);
      if (__builtin_amdgcn_ballot_w64(tg < kNone / 2) != 0) {
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
          for (int ii = 0; ii < 4; ++ii) x[j][ii] = tg < kNone / 2 ? 0.f : x[j][ii];
      }
      if (hit) {
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
          for (int ii = 0; ii < 4; ++ii)
            if (j * 16 + 4 * q + ii == tg) x[j][ii] -= 1.f;
      }
      if (ragged) {
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
          for (int ii = 0; ii < 4; ++ii)
            if (n0 + wc0 + j * 16 + 4 * q + ii >= a.V) x[j][ii] = 0.f;
      }
      if constexpr (ADAPT) {
        u32x2 pp[3][FN];
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          float v[4] = {x[j][0], x[j][1], x[j][2], x[j][3]};
#pragma unroll
          for (int c = 0; c < 3; ++c) {
            pp[c][j] = c < 2 ? bf16_cut(v) : u32x2{pk_bf16(v[0], v[1]), pk_bf16(v[2], v[3])};
            *reinterpret_cast<u32x2*>(strip + c * Lds::PVB + l * Lds::PITCH + j * 32 + q * 8) = pp[c][j];
          }
        }
        // u^T [rank][row] += B dl^T: the lane's own values are the operand; the six
        // products of parts that float32 has, the small ones first
#pragma unroll
        for (int p = 0; p < NP; ++p)
#pragma unroll
          for (int o = 2; o >= 0; --o)
#pragma unroll
            for (int c = 0; c <= o; ++c) {
              const u32x2 v0 = pp[o - c][2 * p], v1 = pp[o - c][2 * p + 1];
              const bf16x8 vv = __builtin_bit_cast(bf16x8, u32x4{v0.x, v0.y, v1.x, v1.y});
#pragma unroll
              for (int jb = 0; jb < RB; ++jb)
                uacc[i][jb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, bp[c][p][jb]), vv,
                                                                     uacc[i][jb], 0, 0, 0);
            }
        // dB^T [entry][rank] += dl^T (t dloss) over these 16 rows, dl^T by transposing
        // reads (in each 16-lane group lanes 4 i + p fetch the 4 columns at 4 p of row
        // i, lane k receives column k of rows 0..3)
        asm volatile("" ::: "memory");
        const int i4 = l >> 2, p4 = l & 3;
        s16x4 tp[3][RBA];
#pragma unroll
        for (int jb = 0; jb < RB; ++jb) {
          const int rank = 16 * jb + l;
#pragma unroll
          for (int c = 0; c < 3; ++c) {
            u32x2 w = *reinterpret_cast<const u32x2*>(tb + (c * R + (rank < R ? rank : 0)) * Lds::TP + wr0 + i * 16 + 4 * q);
            if (rank >= R) w = u32x2{0u, 0u};
            tp[c][jb] = __builtin_bit_cast(s16x4, w);
          }
        }
#pragma unroll
        for (int j = 0; j < FN; j += 2) {
          uint32_t ad[8];
          uint64_t v[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {                    // blocks j and j + 1, three parts each (two reads spare)
            const int c = e % 4 < 3 ? e % 4 : 2;
            ad[e] = lds_addr(strip + c * Lds::PVB + (4 * q + i4) * Lds::PITCH + (j + e / 4) * 32 + p4 * 8);
          }
          tr16_reads<8>(ad, v);
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int o = 2; o >= 0; --o)
#pragma unroll
              for (int c = 0; c <= o; ++c)
#pragma unroll
                for (int jb = 0; jb < RB; ++jb)
                  dbacc[j + h][jb] = __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(__builtin_bit_cast(s16x4, v[4 * h + o - c]),
                                                                              tp[c][jb], dbacc[j + h][jb], 0, 0, 0);
        }
      }
      // dl to memory: one 16-row strip at a time through LDS (this wave's own: no
      // wait), float32 dl as bf16 parts, what one leaves to the next
      if constexpr (!W4) {
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
          for (int ii = 0; ii < 4; ++ii) x[j][ii] *= sw[j][ii];
      }
#pragma unroll
      for (int p = 0; p < PARTS; ++p) {
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          u32x2 w;
          if constexpr (W4) w = u32x2{pk_f16(x[j][0] * kHalfUp, x[j][1] * kHalfUp), pk_f16(x[j][2] * kHalfUp, x[j][3] * kHalfUp)};
          else if constexpr (HALF) w = u32x2{pk_f16(x[j][0], x[j][1]), pk_f16(x[j][2], x[j][3])};
          else if (p == PARTS - 1) w = u32x2{pk_bf16(x[j][0], x[j][1]), pk_bf16(x[j][2], x[j][3])};
          else w = bf16_part(x[j]);
          *reinterpret_cast<u32x2*>(strip + l * Lds::PITCH + j * 32 + q * 8) = w;
        }
#pragma unroll
        for (int e = 0; e < FN / 2; ++e) {
          const int u = lane + 64 * e, sr = u / (FN * 2), cq = u % (FN * 2);
          const int m = m0 + wr0 + i * 16 + sr;
          const u32x4 w = *reinterpret_cast<const u32x4*>(strip + sr * Lds::PITCH + cq * 16);
          if (m < M)
            *reinterpret_cast<u32x4*>(a.g + p * a.gstride + m * a.ldg + c0 + wc0 + cq * 8) = w;
        }
      }
    }
  }

  if constexpr (!GRAD) {
    __syncthreads();
    const float* red = reinterpret_cast<const float*>(lds + Lds::END);
    for (int row = tid; row < BM; row += NT) {
      float mx = -INFINITY;
#pragma unroll
      for (int w = 0; w < WN; ++w) mx = fmaxf(mx, red[2 * (w * BM + row)]);
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < WN; ++w) {
        const float m = red[2 * (w * BM + row)], s = red[2 * (w * BM + row) + 1];
        sum += m == -INFINITY ? s : s * __builtin_amdgcn_exp2f(m - mx);       // (s: 0, or NaN)
      }
      if (m0 + row < M) {
        float* out = a.part + 2 * ((long)ct * M + m0 + row);
        out[0] = mx;
        out[1] = sum;
      }
    }
  }
  if constexpr (ADAPT) {
    // the tile's u and dB: the waves' sums added in order
    __syncthreads();                                       // the strips are read
    float* ub = reinterpret_cast<float*>(lds + Lds::ST);
    float* db = ub + BM * R;
    for (int w = 0; w < max_int(WM, WN); ++w) {
      if (wn == w) {
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
          for (int jb = 0; jb < RB; ++jb) {
            const int rank = 16 * jb + 4 * q;
            f32x4* p = reinterpret_cast<f32x4*>(ub + (wr0 + i * 16 + l) * R + rank);
            if (rank < R) *p = w == 0 ? uacc[i][jb] : *p + uacc[i][jb];
          }
      }
      if (wm == w) {
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
          for (int jb = 0; jb < RB; ++jb) {
            const int rank = 16 * jb + l;
            f32x4* p = reinterpret_cast<f32x4*>(db + rank * BN + wc0 + j * 16 + 4 * q);
            if (rank < R) *p = w == 0 ? dbacc[j][jb] : *p + dbacc[j][jb];
          }
      }
      __syncthreads();
    }
    for (int e = tid; e < BM * R; e += NT) {
      const int row = e / R, j = e % R;
      if (j < a.r && m0 + row < M) a.up[((long)ct * M + m0 + row) * a.r + j] = ub[e];
    }
    for (int e = tid; e < R * BN; e += NT) {
      const int j = e / BN;
      if (j < a.r) a.dbp[((long)mt * a.r + j) * a.ldg + c0 + e % BN] = db[e];
    }
  }
}

// Joins the tiles: a block takes `rows` rows (a power of two up to 64), 1024 /
// rows lanes each every so many tiles, then the lanes in a tree: few rows over
// many tiles are as parallel as many rows.
__global__ __launch_bounds__(1024) void xent_join_kernel(const float* part, const float* tl, Ids ids, int tiles, int M,
                                                         int rows, float* loss, float* lse) {
  __shared__ float rm[1024], rsum[1024];
  const int tid = threadIdx.x, row = tid & (rows - 1), lane = tid / rows, lanes = 1024 / rows;
  const int m = blockIdx.x * rows + row, mc = m < M ? m : M - 1;
  float mx = -INFINITY, sum = 0.f;
  auto join = [&](float m2, float s2) {
    const float top = fmaxf(mx, m2);
    const float ref = top == -INFINITY ? 0.f : top;
    sum = sum * __builtin_amdgcn_exp2f(mx - ref) + s2 * __builtin_amdgcn_exp2f(m2 - ref);
    mx = top;
  };
  for (int c = lane; c < tiles; c += 4 * lanes) {
    float pm[4], ps[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const float* p = part + 2 * ((long)(c + u * lanes < tiles ? c + u * lanes : c) * M + mc);
      pm[u] = p[0];
      ps[u] = p[1];
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (c + u * lanes < tiles) join(pm[u], ps[u]);
  }
  rm[tid] = mx;
  rsum[tid] = sum;
  for (int d = 512; d >= rows; d >>= 1) {
    __syncthreads();
    if (tid < d) {
      join(rm[tid + d], rsum[tid + d]);
      rm[tid] = mx;
      rsum[tid] = sum;
    }
  }
  if (lane != 0 || m >= M) return;
  const float rest = logf(sum);
  lse[m] = mx * kLn2 + rest;
  // (the difference first: what the target's logit and the maximum share)
  loss[m] = entry_of(ids, m) >= 0 ? (mx - tl[m]) * kLn2 + rest : 0.f;
}

// ---- dx ---------------------------------------------------------------------------
struct DxArgs {
  int M, N, K, V;
  const uint16_t* g;     // [parts][M][ldg]
  long ldg, gstride;
  int parts;
  const int8_t* codes;
  const _Float16* scales;        // 4-bit
  const uint32_t* smax;          // [64] partial maxima of them
  int v0;                // first entry of the piece
  int tiles_m, tiles_k;
  int splits, nks;       // stages (of all parts) per split
  int first;             // the first piece: the buffer is written, not added to
  float* dxp;            // [splits][M][K]
};

// F: 0 int8 codes and dl in bf16 parts, 1 int8 codes and dl in float16, 2 4-bit.
template <int F, int BM, int WM, int S>
__global__ __launch_bounds__(64 * WM * 4) void xent_dx_kernel(DxArgs a) {
  constexpr bool W4 = F == 2;
  constexpr int WN = 4, NW = WM * WN, BN = 256, KC = 64;
  constexpr int ASZ = BM * 128, RB = W4 ? 128 : 256;         // bytes of a row of codes
  constexpr int BSZ = KC * RB, SSZ = W4 ? NW * 256 : 0, STG = ASZ + BSZ + SSZ;
  constexpr int FM = BM / WM / 16;
  constexpr int AI = BM / 8 / NW, BI = BSZ / 1024 / NW, LPS = AI + BI + (W4 ? 1 : 0);
  static_assert(AI * 8 * NW == BM && BI * 1024 * NW == BSZ, "whole instructions per wave");
  constexpr int SCB = W4 ? NW * 128 : 0;                      // the waves' scales of a stage
  static_assert(S * STG + SCB <= 160 * 1024, "LDS of a block");
  __shared__ __attribute__((aligned(1024))) int8_t ring[S * STG + SCB];

  const int lane = threadIdx.x & 63, wid = wave_id(), l = lane & 15, q = lane >> 4;
  const int wm = wid / WN, wn = wid % WN;
  const int M = a.M, K = a.K;
  const int tiles = a.tiles_m * a.tiles_k;
  const int order = xcd_order((int)blockIdx.x, tiles * a.splits);
  const int split = order / tiles, tile = order % tiles;
  const int mt = tile % a.tiles_m, dt = tile / a.tiles_m;
  const int m0 = mt * BM, d0 = dt * BN;
  const int nkv = (int)(a.ldg / KC), total = nkv * a.parts;  // stages of a part, of all
  const int kt0 = split * a.nks, kt1 = kt0 + a.nks < total ? kt0 + a.nks : total;

  const int8_t* pa[AI];
  uint32_t voB[BI];
  int rB[BI];
#pragma unroll
  for (int i = 0; i < AI; ++i) {
    const int row = (wid * AI + i) * 8 + (lane >> 3), gm = m0 + row;
    pa[i] = reinterpret_cast<const int8_t*>(a.g + (long)(gm < M ? gm : M - 1) * a.ldg) +
            ((lane & 7) ^ ((row >> 1) & 7)) * 16;
  }
  // codes: a row's 64-column quarters (int8: 64 bytes, 4-bit: 32) exchanged by
  // (row / 8) % 4, so that the four rows, 8 apart, of one read lie in different banks
  const long crow = W4 ? K / 2 : K;
#pragma unroll
  for (int i = 0; i < BI; ++i) {
    constexpr int CPR = RB / 16;
    rB[i] = (wid * BI + i) * (64 / CPR) + lane / CPR;
    const int c = (lane % CPR) ^ (((rB[i] >> 3) & 3) << (W4 ? 1 : 2));
    const long b = (W4 ? d0 / 2 : d0) + c * 16;
    voB[i] = b < crow ? (uint32_t)b : 0xffffffffu;
  }
  const int grp = (d0 + wn * 64) / 128, ngrp = K / 128;
  auto issue = [&](int kt, int slot) {
    int8_t* base = ring + slot * STG;
    const int p = a.parts == 1 ? 0 : kt / nkv, kv = kt - p * nkv;
    const long go = ((long)p * a.gstride + (long)kv * KC) * 2;
#pragma unroll
    for (int i = 0; i < AI; ++i) lds_dma16(pa[i] + go, base + (wid * AI + i) * 1024);
#pragma unroll
    for (int i = 0; i < BI; ++i) {
      const int v = a.v0 + kv * KC + rB[i];
      const int8_t* src = a.codes + (long)(v < a.N ? v : a.N - 1) * crow + voB[i];
      lds_dma16(voB[i] != 0xffffffffu ? src : zero_chunk(lane), base + ASZ + (wid * BI + i) * 1024);
    }
    if constexpr (W4) {
      // the 64 entries' scales for this wave's group, as the dwords that hold them
      const int v = a.v0 + kv * KC + lane;
      const long e = (long)(v < a.N ? v : a.N - 1) * ngrp + (grp < ngrp ? grp : 0);
      __builtin_amdgcn_global_load_lds(reinterpret_cast<const uint32_t*>(a.scales) + (e >> 1),
                                       (lds_void*)(base + ASZ + BSZ + wid * 256), 4, 0, 0);
    }
  };

  f32x4 acc[FM][4];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  // 4-bit: the power of two that takes the scales into float16
  const float sf = W4 ? __builtin_ldexpf(1.f, 13 - scale_power(a.smax[lane])) : 0.f;
#pragma unroll
  for (int st = 0; st < S - 1; ++st)
    if (kt0 + st < kt1) issue(kt0 + st, st);
  int slot = 0;
  for (int kt = kt0; kt < kt1; ++kt) {
    wait_stages<LPS, 0, S - 2>(kt1 - 1 - kt);
    __builtin_amdgcn_s_barrier();
    if (kt + S - 1 < kt1) issue(kt + S - 1, slot == 0 ? S - 1 : slot - 1);
    const int8_t* As = ring + slot * STG;
    const int8_t* Bs = As + ASZ;
    int8_t* sch = ring + S * STG + wid * 128;               // this wave's scales times sf of the stage's 64 entries
    if constexpr (W4) {
      // lane: one entry, the half of its dword by the place's parity; entries that
      // are none get 0 (this wave's own bytes: no barrier)
      const int v = a.v0 + kt * KC + lane, vc = v < a.N ? v : a.N - 1;
      const uint32_t two = *reinterpret_cast<const uint32_t*>(Bs + BSZ + wid * 256 + lane * 4);
      const uint16_t hb = (uint16_t)((vc * ngrp + (grp < ngrp ? grp : 0)) & 1 ? two >> 16 : two);
      const float sc = v < a.V ? sf * (float)__builtin_bit_cast(_Float16, hb) : 0.f;
      *reinterpret_cast<_Float16*>(sch + lane * 2) = (_Float16)sc;
      asm volatile("" ::: "memory");
    }
#pragma unroll
    for (int kk = 0; kk < KC / 32; ++kk) {
      bf16x8 af[FM];
#pragma unroll
      for (int i = 0; i < FM; ++i)
        af[i] = *reinterpret_cast<const bf16x8*>(As + swz128((wm * FM + i) * 16 + l, kk * 4 + q));
      // rows 32 kk + 8 q + e, columns 64 wn + 4 l + j (j the column block)
      u32x4 bf[4];
      const int8_t* row = Bs + (32 * kk + 8 * q) * RB;
      if constexpr (!W4) {
        uint32_t w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = *reinterpret_cast<const uint32_t*>(row + e * RB + ((wn ^ q) << 6) + 4 * l);
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if constexpr (F == 0) {
              const float x = (float)(int8_t)(w[2 * e] >> (8 * j)), y = (float)(int8_t)(w[2 * e + 1] >> (8 * j));
              bf[j][e] = __builtin_amdgcn_perm(__float_as_uint(y), __float_as_uint(x), 0x07060302u);
            } else {
              // a byte with its sign bit turned over, under the exponent of 1024, is
              // 1152 + q in float16
              const uint32_t b = __builtin_amdgcn_perm(w[2 * e + 1], w[2 * e], 0x0c040c00u + 0x00010001u * j) ^ 0x64806480u;
              bf[j][e] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, b) -
                                                          f16x2{(_Float16)1152.f, (_Float16)1152.f});
            }
          }
      } else {
        // rows 2 e and 2 e + 1 share a register: nibble j of each, with its sign bit
        // turned over, under the exponent of 1024 is 1032 + q in float16
        const u32x4 s4 = *reinterpret_cast<const u32x4*>(sch + (32 * kk + 8 * q) * 2);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t lo = *reinterpret_cast<const uint16_t*>(row + (2 * e) * RB + ((wn ^ q) << 5) + 2 * l);
          const uint32_t hi = *reinterpret_cast<const uint16_t*>(row + (2 * e + 1) * RB + ((wn ^ q) << 5) + 2 * l);
          const uint32_t w = (lo | (hi << 16)) ^ 0x88888888u;
          const uint32_t s2 = s4[e];                       // (a bit cast of a vector's element takes its first)
          const f16x2 sc = __builtin_bit_cast(f16x2, s2);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const f16x2 x = __builtin_bit_cast(f16x2, ((w >> (4 * j)) & 0x000f000fu) | 0x64006400u);
            bf[j][e] = __builtin_bit_cast(uint32_t, (x - f16x2{(_Float16)1032.f, (_Float16)1032.f}) * sc);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if constexpr (F > 0)
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, af[i]),
                                                              __builtin_bit_cast(f16x8, bf[j]), acc[i][j], 0, 0, 0);
          else
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(af[i], __builtin_bit_cast(bf16x8, bf[j]), acc[i][j], 0, 0, 0);
        }
    }
    slot = slot == S - 1 ? 0 : slot + 1;
  }
  const int d = d0 + wn * 64 + 4 * l;
  if (d >= K || (!a.first && kt0 >= kt1)) return;
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int ii = 0; ii < 4; ++ii) {
      const int m = m0 + (wm * FM + i) * 16 + 4 * q + ii;
      if (m >= M) continue;
      f32x4* p = reinterpret_cast<f32x4*>(a.dxp + ((long)split * M + m) * K + d);
      const f32x4 v{acc[i][0][ii], acc[i][1][ii], acc[i][2][ii], acc[i][3][ii]};
      *p = a.first ? v : *p + v;
    }
}

// After a piece: u += its tiles' parts, dB of its entries = s times the row
// tiles' parts; the last piece also clears dB's padding. The first `ublocks` blocks
// take `ue` elements of u each (a power of two), 256 / ue threads an element that
// share its tiles, few elements where there are few (64 rows of rank 8 over 393
// tiles: 4.8 us, a thread each 30); the others a thread an element, in up to 2^21 blocks.
struct ReduceArgs {
  int M, N, r, tiles_x, tiles_m, v0, vc, first, last, V, ue, ublocks;
  long ldg;
  float s;
  Ids ids;
  const float* dloss;
  const float* up;
  const float* dbp;
  float* u;
  float* dB;
};
// The factor of a row's gradient: dloss, 0 where it has no target.
__device__ __forceinline__ float row_factor(const Ids& ids, const float* dloss, long m) {
  return entry_of(ids, m) >= 0 ? dloss[m] : 0.f;
}

__global__ __launch_bounds__(256) void xent_reduce_kernel(ReduceArgs a) {
  __shared__ float red[256];
  const int tid = threadIdx.x;
  const long nu = (long)a.M * a.r;
  const long ndb = (long)a.r * a.vc, npad = a.last ? (long)a.r * (a.N - a.V) : 0;
  auto sum = [](const float* p, long stride, int n) {
    float s = 0.f;
    for (int i = 0; i < n; i += 8) {
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = p[(i + k < n ? i + k : i) * stride];
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (i + k < n) s += v[k];
    }
    return s;
  };
  if ((int)blockIdx.x < a.ublocks) {
    const int lane = tid / a.ue, lanes = 256 / a.ue;
    const long e = (long)blockIdx.x * a.ue + tid % a.ue, ec = e < nu ? e : 0;
    red[tid] = lane < a.tiles_x ? sum(a.up + lane * nu + ec, lanes * nu, (a.tiles_x - lane + lanes - 1) / lanes) : 0.f;
    for (int d = 128; d >= a.ue; d >>= 1) {
      __syncthreads();
      if (tid < d) red[tid] += red[tid + d];
    }
    if (lane != 0 || e >= nu) return;
    const float u = a.first ? red[tid] : a.u[e] + red[tid];
    a.u[e] = a.last ? u * row_factor(a.ids, a.dloss, e / a.r) : u;     // (u of a row without a target is 0)
    return;
  }
  const long step = (long)((int)gridDim.x - a.ublocks) * 256;
  for (long e = (long)((int)blockIdx.x - a.ublocks) * 256 + tid; e < ndb + npad; e += step) {
    if (e < ndb) {
      const long j = e / a.vc, c = e % a.vc;
      a.dB[j * a.N + a.v0 + c] = a.s * sum(a.dbp + j * a.ldg + c, a.r * a.ldg, a.tiles_m);
    } else {
      const long j = (e - ndb) / (a.N - a.V), c = (e - ndb) % (a.N - a.V);
      a.dB[j * a.N + a.V + c] = 0.f;
    }
  }
}

// dx = factor times the splits' sums + s u A^T, over tiles of 16 rows and 64
// features: lane (l, q) holds the 16 features of quarter q of row l; the adapter's
// part is formed on v_mfma_f32_16x16x4_f32 in that layout (as the lookup's: a thread
// that read its features' rows of A for itself took 49 us for 4096 x 768 at rank 8).
// SW = 1: a wave takes a tile, four a block. SW = 16: the waves of a block share the
// splits of one tile and add through LDS, four of them a quarter of each lane's
// features: where there are at most as many tiles as compute units (64 x 768 in 85
// splits: 15.7 us, one wave a tile 41; 256 x 2048 in 32 splits, 512 tiles, the other
// way round: 25.9 against 19.3).
// dA = s times the row blocks' partial sums (xent_da_kernel) is taken beside it, by the
// blocks with blockIdx.y past the tiles' (its own launch cost 3 to 10 us).
struct DaTotal {
  const float* part;
  int blocks;            // of rows
  float* dA;             // NULL: none
  int y0;                // the first blockIdx.y
};
__device__ __forceinline__ void da_total(const DaTotal& t, long e, int K, int r, float s) {
  const long n = (long)r * K;
  if (e < n) t.dA[e % K * r + e / K] = s * rank_sum_total(t.part, t.blocks, n, e);
}

template <typename OutT, int R, int SW>
__global__ __launch_bounds__(SW == 1 ? 256 : 64 * SW) void xent_dx_join_kernel(const float* dxp, int splits, int M, int K,
                                                                               int r, float s, const float* u,
                                                                               const float* A, Ids ids,
                                                                               const float* dloss, int bits,
                                                                               const uint32_t* smax, OutT* dx,
                                                                               DaTotal total) {
  __shared__ f32x4 red[SW > 1 ? SW * 256 : 1];             // [wave][block of 4 features][lane]
  if constexpr (R > 0) {
    if ((int)blockIdx.y >= total.y0)
      return da_total(total, ((long)((int)blockIdx.y - total.y0) * gridDim.x + blockIdx.x) * blockDim.x + threadIdx.x, K, r, s);
  }
  const int lane = threadIdx.x & 63, l = lane & 15, q = lane >> 4, w = threadIdx.x >> 6;
  const int m = blockIdx.x * 16 + l, mc = m < M ? m : M - 1;
  const int d0 = (SW > 1 ? (int)blockIdx.y : (int)blockIdx.y * 4 + w) * 64, k = d0 + 16 * q, kc = k < K ? k : 0;
  const int first = SW > 1 ? w : 0;
  const long n = (long)M * K;
  const float* p = dxp + (long)mc * K + kc;
  f32x4 v[4];
#pragma unroll
  for (int b = 0; b < 4; ++b)
    v[b] = first < splits ? *reinterpret_cast<const f32x4*>(p + first * n + 4 * b) : f32x4{0.f, 0.f, 0.f, 0.f};
  // (dl in float16: back from 2^(bits - E))
  const float back = smax != nullptr ? __builtin_ldexpf(1.f, scale_power(smax[lane]) - bits) : 1.f;
  const bool live = entry_of(ids, mc) >= 0;
  const float f = dloss[mc] * back;
  f32x4 low[4];
  if constexpr (R > 0) {
#pragma unroll
    for (int b = 0; b < 4; ++b) low[b] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int c = 0; c < R / 4; ++c) {
      const int j = 4 * c + q, jc = j < r ? j : 0;
      const float uv = j < r ? u[(long)mc * r + jc] : 0.f;
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        if (SW > 1 && b != w) continue;                    // (wave-uniform: what this wave writes)
        const int d = d0 + 16 * (l >> 2) + 4 * b + (l & 3);
        const float av = d < K && j < r ? A[(long)(d < K ? d : 0) * r + jc] : 0.f;
        low[b] = __builtin_amdgcn_mfma_f32_16x16x4f32(av, uv, low[b], 0, 0, 0);
      }
    }
  }
  for (int i = first + SW; i < splits; i += 4 * SW) {      // four splits' loads in flight
    f32x4 x[4][4];
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int b = 0; b < 4; ++b)
        x[c][b] = *reinterpret_cast<const f32x4*>(p + (i + c * SW < splits ? i + c * SW : 0) * n + 4 * b);
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int b = 0; b < 4; ++b)
        if (i + c * SW < splits) v[b] += x[c][b];
  }
  OutT* out = dx + (long)m * K + k;
  if constexpr (SW > 1) {
#pragma unroll
    for (int b = 0; b < 4; ++b) red[(w * 4 + b) * 64 + lane] = v[b];
    __syncthreads();
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      if (b != w || m >= M || k >= K) continue;
      f32x4 y = red[b * 64 + lane];
      for (int i = 1; i < SW && i < splits; ++i) y += red[(i * 4 + b) * 64 + lane];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float z = R > 0 ? __builtin_fmaf(s, low[b][c], y[c] * f) : y[c] * f;
        y[c] = live ? z : 0.f;                             // (weights that are no numbers times 0)
      }
      if constexpr (sizeof(OutT) == 4) *reinterpret_cast<f32x4*>(out + 4 * b) = y;
      else *reinterpret_cast<u32x2*>(out + 4 * b) = u32x2{pk_bf16(y[0], y[1]), pk_bf16(y[2], y[3])};
    }
    return;
  }
  if (m >= M || k >= K) return;
#pragma unroll
  for (int b = 0; b < 4; ++b)
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const float y = R > 0 ? __builtin_fmaf(s, low[b][c], v[b][c] * f) : v[b][c] * f;
      v[b][c] = live ? y : 0.f;
    }
  if constexpr (sizeof(OutT) == 4) {
#pragma unroll
    for (int b = 0; b < 4; ++b) *reinterpret_cast<f32x4*>(out + 4 * b) = v[b];
  } else {
#pragma unroll
    for (int b = 0; b < 4; b += 2)
      *reinterpret_cast<u32x4*>(out + 4 * b) = u32x4{pk_bf16(v[b][0], v[b][1]), pk_bf16(v[b][2], v[b][3]),
                                                     pk_bf16(v[b + 1][0], v[b + 1][1]), pk_bf16(v[b + 1][2], v[b + 1][3])};
  }
}

template <typename OutT>
void dx_join(const VocabLayer& L, int M, Ids ids, const float* dloss, const XentPlan& plan, const XentBuffers& buf,
             void* dx, DaTotal total, hipStream_t st) {
  const unsigned rows = (unsigned)((M + 15) / 16), cols = (unsigned)((L.K + 63) / 64);
  const bool shared = plan.splits >= 8 && (long)rows * cols <= kCUs;
  const int bits = L.fmt == 0 ? kHalfBits : kHalfBits4;
  OutT* out = static_cast<OutT*>(dx);
  const auto launch = [&](auto rank) {
    constexpr int R = decltype(rank)::value;
    const uint32_t* smax = plan.parts == 1 ? buf.smax : nullptr;
    const int threads = shared ? 1024 : 256;
    total.y0 = (int)(shared ? cols : (cols + 3) / 4);
    const long per = (long)threads * rows, extra = R > 0 ? ((long)L.r * L.K + per - 1) / per : 0;
    const dim3 grid(rows, (unsigned)(total.y0 + extra));
    if (shared)
      xent_dx_join_kernel<OutT, R, 16><<<grid, 1024, 0, st>>>(buf.dxp, plan.splits, M, L.K, L.r, L.s, buf.u, L.A, ids,
                                                             dloss, bits, smax, out, total);
    else
      xent_dx_join_kernel<OutT, R, 1><<<grid, 256, 0, st>>>(buf.dxp, plan.splits, M, L.K, L.r, L.s, buf.u, L.A, ids,
                                                            dloss, bits, smax, out, total);
  };
  if (L.r == 0) launch(std::integral_constant<int, 0>());
  else if (L.r <= 4) launch(std::integral_constant<int, 4>());
  else if (L.r <= 8) launch(std::integral_constant<int, 8>());
  else if (L.r <= 16) launch(std::integral_constant<int, 16>());
  else launch(std::integral_constant<int, 32>());
}

// dA = s x^T u over the rows that have a target: partial sums, then their total.
template <typename T, int RB>
__global__ __launch_bounds__(256) void xent_da_kernel(const typename Elem<T>::type* x, const float* u, Ids ids, int M,
                                                      int K, int r, int rows, float* part) {
  __shared__ __attribute__((aligned(16))) char lds[rank_sum_lds<RB>()];
  rank_sum_block<T, RB>(blockIdx.x, M, K, r, rows, x, part, lds, [&](int m) { return entry_of(ids, m) >= 0; },
                        [&](int m, int j) { return u[(long)m * r + j]; });
}
__global__ __launch_bounds__(256) void xent_da_total_kernel(DaTotal t, int K, int r, float s) {
  da_total(t, (long)blockIdx.x * 256 + threadIdx.x, K, r, s);
}

// ---- launches ---------------------------------------------------------------------
template <bool W4, int BM, int BN, int WM, int WN, int S, int G, int PARTS>
void logits_ranks(LogitArgs& a, int cols, hipStream_t st) {
  a.tiles_m = (a.M + BM - 1) / BM;
  a.tiles_x = (cols + BN - 1) / BN;
  const dim3 grid((unsigned)(a.tiles_m * a.tiles_x));
  constexpr int NT = 64 * WM * WN;
  if (a.r == 0) xent_logits_kernel<W4, BM, BN, WM, WN, S, G, 0, PARTS><<<grid, NT, 0, st>>>(a);
  else if (a.r <= 4) xent_logits_kernel<W4, BM, BN, WM, WN, S, G, 4, PARTS><<<grid, NT, 0, st>>>(a);
  else if (a.r <= 8) xent_logits_kernel<W4, BM, BN, WM, WN, S, G, 8, PARTS><<<grid, NT, 0, st>>>(a);
  else if (BM * BN > 128 * 128 || a.r <= 16)
    xent_logits_kernel<W4, BM, BN, WM, WN, S, G, 16, PARTS><<<grid, NT, 0, st>>>(a);
  else if constexpr (BM * BN <= 128 * 128)
    xent_logits_kernel<W4, BM, BN, WM, WN, S, G, 32, PARTS><<<grid, NT, 0, st>>>(a);
}

// The tiles of a launch over `cols` entries; fills tiles_m and tiles_x.
template <int PARTS>
void logits(LogitArgs& a, int fmt, int cols, hipStream_t st) {
  if (fmt == 0) {
    const long t128 = (long)((a.M + 127) / 128) * ((cols + 127) / 128);
    const long t256 = (long)((a.M + 255) / 256) * ((cols + 255) / 256);
    // few tiles leave compute units idle: smaller ones then (64 x 768 x 4000 rank 4
    // with gradient 67.5 -> 63.5 us, 128 x 2048 x 4000 64.2 -> 59.4)
    // Large tiles read least from LDS for a product, but take a compute unit each: from
    // 63 to 128 of them smaller ones are faster (256 x 2048 over 32000: loss 41.9 against
    // 34.9 us, 4096 features 58 against 45, 8000 entries of 768 26.6 against 22.1), 189
    // of them not (640 x 2048 over 16000: 42.9 against 44.8)
    if (a.M <= 32 || t128 <= kFewTiles) logits_ranks<false, 32, 256, 1, 4, 4, 1, PARTS>(a, cols, st);
    else if (t256 > kHalfTiles && a.M > 128 && a.r <= 16) logits_ranks<false, 256, 256, 2, 4, 2, 1, PARTS>(a, cols, st);
    else logits_ranks<false, 128, 128, 2, 2, 2, 1, PARTS>(a, cols, st);
  } else if constexpr (PARTS == 3) {
    return;                                                // (float32 has no 4-bit layers)
  } else if (a.M <= 32) {
    if (a.K <= 4096) logits_ranks<true, 32, 128, 1, 4, 3, 32, PARTS>(a, cols, st);
    else logits_ranks<true, 32, 128, 1, 4, 3, 128, PARTS>(a, cols, st);
  } else {
    if (a.K <= 4096) logits_ranks<true, 128, 128, 2, 2, 2, 32, PARTS>(a, cols, st);
    else logits_ranks<true, 128, 128, 2, 2, 2, 128, PARTS>(a, cols, st);
  }
}

LogitArgs logit_args(const VocabLayer& L, int M, Ids ids, const int8_t* xq, const float* sx, const float* t) {
  LogitArgs a{};
  a.M = M; a.N = L.N; a.K = L.K; a.V = ids.vocab; a.r = L.r;
  a.xq = xq; a.sx = sx; a.codes = static_cast<const int8_t*>(L.codes); a.scales = L.scales;
  a.t = t; a.B = L.B; a.s = L.s; a.ids = ids;
  return a;
}

// Rows of a dx tile.
int dx_rows(int M) { return M <= 32 ? 32 : M <= 128 ? 128 : 256; }

template <int F>
void launch_dx(const DxArgs& a, int rows, hipStream_t st) {
  const dim3 grid((unsigned)(a.tiles_m * a.tiles_k * a.splits));
  if (rows == 32) xent_dx_kernel<F, 32, 1, 3><<<grid, 256, 0, st>>>(a);
  else if (rows == 128) xent_dx_kernel<F, 128, 2, 3><<<grid, 512, 0, st>>>(a);
  else xent_dx_kernel<F, 256, 2, 3><<<grid, 512, 0, st>>>(a);
}

}  // namespace

size_t xent_part_floats(int vocab, int M) {
  return ((size_t)((vocab + 127) / 128) * 2 + 1) * (size_t)M;
}

void launch_xent_fwd(const VocabLayer& L, int M, Ids ids, const int8_t* xq, const float* sx,
                     const float* t, float* part, float* loss, float* lse, hipStream_t st) {
  LogitArgs a = logit_args(L, M, ids, xq, sx, t);
  a.tl = part;
  a.part = part + M;
  logits<0>(a, L.fmt, ids.vocab, st);
  int rows = 1;
  while (rows < 64 && rows < M) rows <<= 1;
  xent_join_kernel<<<dim3((unsigned)((M + rows - 1) / rows)), 1024, 0, st>>>(a.part, a.tl, ids, a.tiles_x, M, rows,
                                                                           loss, lse);
}

XentPlan xent_plan(const VocabLayer& L, int vocab, int M, int dtype) {
  XentPlan p{};
  p.parts = dtype == 0 ? 3 : 1;
  // pieces of up to 256 MB of dl, or of 512 entries (the sums of dx are read and written once a
  // piece), of whole rounds of 256 x 256 tiles over the chip where they hold one
  // (4096 x 768 x 50257 at rank 8: 1095 us, 1156 in two equal pieces, 1142 at 128 MB)
  const long most = (128L << 20) / p.parts / M / 256 * 256, tiles_m = (M + 255) / 256;
  const long round = 256 * (kCUs / tiles_m < 1 ? 1 : kCUs / tiles_m), all = ((long)vocab + 255) / 256 * 256;
  const long fit = most >= round ? most / round * round : most < 512 ? 512 : most;
  p.piece = (int)(fit > all ? all : fit);
  const int rows = dx_rows(M);
  const long tiles = (long)((M + rows - 1) / rows) * ((L.K + 255) / 256);
  const int nk = p.parts * (p.piece / 64);
  // as many splits as leave one block a compute unit, each of at least four stages
  p.splits = (int)(kCUs / tiles < 1 ? 1 : kCUs / tiles);
  if (p.splits > nk / 4) p.splits = nk / 4 < 1 ? 1 : nk / 4;
  p.g = (size_t)p.parts * M * p.piece;
  p.dxp = (size_t)p.splits * M * L.K;
  p.smax = kMaxParts;
  if (L.r > 0) {
    p.u = (size_t)M * L.r;
    p.up = (size_t)(p.piece / 128) * M * L.r;
    // row tiles times entries: 128 or 256 rows a tile, or 32 of at most kFewTiles
    // tiles' rows and columns
    const size_t large = (size_t)((M + 127) / 128) * p.piece, few = (size_t)kFewTiles * 4 * 128;
    p.dbp = (large > few ? large : few) * L.r;
    p.pA = rank_sum_floats(M, L.K, L.r);
  }
  return p;
}

void launch_xent_bwd(const VocabLayer& L, int M, int dtype, Ids ids, const void* x, const int8_t* xq, const float* sx,
                     const float* t, const float* lse, const float* dloss, const XentPlan& plan,
                     const XentBuffers& buf, void* dx, float* dA, float* dB, hipStream_t st) {
  const int V = ids.vocab;
  const int rows = dx_rows(M);
  if (L.fmt == 0 && plan.parts == 1)
    xent_scale_max_kernel<<<dim3(kMaxParts), 1024, 0, st>>>(static_cast<const float*>(L.scales), V, buf.smax);
  else if (L.fmt == 1 && dx != nullptr)
    xent_scale_max_kernel<<<dim3(kMaxParts), 1024, 0, st>>>(static_cast<const _Float16*>(L.scales), V * (L.K / 128),
                                                            buf.smax);
  for (int v0 = 0; v0 < V; v0 += plan.piece) {
    const int vc = V - v0 < plan.piece ? V - v0 : plan.piece;
    const long ldg = (vc + 255) / 256 * 256;
    LogitArgs a = logit_args(L, M, ids, xq, sx, t);
    a.v0 = v0; a.lse = lse; a.dloss = dloss; a.g = buf.g; a.ldg = ldg; a.gstride = M * ldg;
    a.up = buf.up; a.dbp = buf.dbp; a.smax = buf.smax;
    if (plan.parts == 1) logits<1>(a, L.fmt, (int)ldg, st);
    else logits<3>(a, L.fmt, (int)ldg, st);
    if (dx != nullptr) {
      DxArgs d{};
      d.M = M; d.N = L.N; d.K = L.K; d.V = V; d.g = buf.g; d.ldg = ldg; d.gstride = a.gstride; d.parts = plan.parts;
      d.codes = a.codes; d.scales = static_cast<const _Float16*>(L.scales); d.smax = buf.smax;
      d.v0 = v0;
      d.tiles_m = (M + rows - 1) / rows; d.tiles_k = (L.K + 255) / 256;
      d.splits = plan.splits;
      d.nks = (plan.parts * (int)(ldg / 64) + plan.splits - 1) / plan.splits;
      d.first = v0 == 0; d.dxp = buf.dxp;
      if (L.fmt == 1) launch_dx<2>(d, rows, st);
      else if (plan.parts == 1) launch_dx<1>(d, rows, st);
      else launch_dx<0>(d, rows, st);
    }
    if (L.r > 0) {
      const long nu = (long)M * L.r;
      // 32: whole lines of every tile's parts; 256 where 8 threads an element and those
      // of dB could be the 2^32 threads that a launch has to stay below (2^24 rows of
      // rank 32 are)
      const int ue = nu > 3L << 27 ? 256 : nu > 8192 ? 32 : 8;
      ReduceArgs r{M, L.N, L.r, a.tiles_x, a.tiles_m, v0, vc, v0 == 0, v0 + vc == V, V, ue, (int)((nu + ue - 1) / ue),
                   ldg, L.s, ids, dloss, buf.up, buf.dbp, buf.u, dB};
      const long n = (long)L.r * vc + (r.last ? (long)L.r * (L.N - V) : 0), nb = (n + 255) / 256;
      xent_reduce_kernel<<<dim3((unsigned)(r.ublocks + (nb < 1L << 21 ? nb : 1L << 21))), 256, 0, st>>>(r);
    }
  }
  DaTotal total{};
  if (L.r > 0) {
    const int rows_a = rank_sum_rows(M, L.K), blocks = rank_sum_blocks(M, L.K);
    const float* xf = static_cast<const float*>(x);
    const uint16_t* xh = static_cast<const uint16_t*>(x);
    if (dtype == 0 && L.r <= 16)
      xent_da_kernel<F32, 1><<<dim3((unsigned)blocks), 256, 0, st>>>(xf, buf.u, ids, M, L.K, L.r, rows_a, buf.pA);
    else if (dtype == 0)
      xent_da_kernel<F32, 2><<<dim3((unsigned)blocks), 256, 0, st>>>(xf, buf.u, ids, M, L.K, L.r, rows_a, buf.pA);
    else if (L.r <= 16)
      xent_da_kernel<BF16, 1><<<dim3((unsigned)blocks), 256, 0, st>>>(xh, buf.u, ids, M, L.K, L.r, rows_a, buf.pA);
    else
      xent_da_kernel<BF16, 2><<<dim3((unsigned)blocks), 256, 0, st>>>(xh, buf.u, ids, M, L.K, L.r, rows_a, buf.pA);
    total = DaTotal{buf.pA, (M + rows_a - 1) / rows_a, dA, 0};
    if (dx == nullptr)
      xent_da_total_kernel<<<dim3((unsigned)(((long)L.r * L.K + 255) / 256)), 256, 0, st>>>(total, L.K, L.r, L.s);
  }
  if (dx == nullptr) return;
  if (dtype == 0) dx_join<float>(L, M, ids, dloss, plan, buf, dx, total, st);
  else dx_join<uint16_t>(L, M, ids, dloss, plan, buf, dx, total, st);
}

}  // namespace qlora
