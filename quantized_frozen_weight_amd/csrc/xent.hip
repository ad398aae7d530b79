// Softmax cross entropy of the vocabulary layer and its gradient, the logits
// never in memory (formulas: include/qlora.h).
//
// logits kernel  The layer's integer product over tiles of the vocabulary, both
//   operands K-contiguous rows that move from memory to LDS untouched
//   (ring.hpp); 4-bit weights are widened in registers and their exact sums
//   weighted group by group (as gemm_a8w4.hip). What a tile does with its
//   logits:
//   - loss: each row's maximum and sum of exp2 over the tile's columns, lanes by
//     DPP, waves through LDS, 8 bytes a row and tile to the workspace; the
//     target's logit from the tile that holds it. A second, small launch joins
//     the tiles in a fixed order;
//   - gradient: dl = dloss (exp2(l log2e - lse log2e) - [target]) for one piece
//     of the vocabulary, in bf16 (int8 weights: times the entry's scale, so that
//     the next product multiplies with the codes, which bf16 holds exactly), and
//     with an adapter the tile's parts of u = dl B^T and dB = t^T dl from the
//     float32 dl.
// dx kernel      dx += dl W over one piece: dl rows K-contiguous, W as stored,
//   codes [v][d], contracted over v. The 16-bit operand that a matrix
//   instruction wants of W is eight v of one d: a lane reads one dword (4 d) of
//   eight rows v, and takes byte j of each for its j-th column block, so that
//   the transposition costs no instruction beside the conversion, and the four
//   column blocks of a lane are four consecutive d of the output. Float32 dl
//   comes as three bf16 parts, the contraction run over each. The contraction of
//   a piece is split where there are few tiles; every split adds into a float32
//   buffer of its own, piece after piece.
// Pieces are as large as 128 MB of dl allow. Sums are in a fixed order.
#include "abi.hpp"
#include "bwd_common.hpp"
#include "launch.hpp"
#include "nibbles.hpp"
#include "ring.hpp"
#include "vocab.hpp"

namespace qlora {

namespace {

constexpr int kCUs = 256;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

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
  uint16_t* g;           // [parts][M][ldg]
  long ldg, gstride;
  int parts;
  float* up;             // [tiles_x][M][r]
  float* dbp;            // [tiles_m][r][ldg]
};

// Maximum and sum over the 16 lanes that hold one row of a 16 x 16 block.
__device__ __forceinline__ float row16_max(float v) {
#pragma unroll
  for (int lvl = 0; lvl < 4; ++lvl) v = fmaxf(v, dpp_pair(v, lvl));
  return v;
}
__device__ __forceinline__ float row16_sum(float v) {
#pragma unroll
  for (int lvl = 0; lvl < 4; ++lvl) v += dpp_pair(v, lvl);
  return v;
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
  static constexpr int TS = 0, QS = TS + BM * R * 4, SX = QS + R * QP * 4, SW = SX + BM * 4;
  static constexpr int TG = SW + BN * 4, LS = TG + BM * 4, GM = LS + BM * 4, END = GM + BM * 4;
  static constexpr int RED = WN * BM * 8;                 // loss: the waves' maxima and sums
  static constexpr int PITCH = FN * 32 + 16, FPITCH = FN * 16 + 4;
  static constexpr int STRIP = R > 0 ? max_int(16 * PITCH, 16 * FPITCH * 4) : 16 * PITCH;
  static constexpr int UB = END + NW * STRIP;             // u [BM][R], dB [R][BN]
  static constexpr int EPI = GRAD ? UB + (BM + BN) * R * 4 : END + RED;
  static constexpr int BYTES = max_int(S * STG + SLAB, EPI);
  static_assert(BYTES <= 160 * 1024, "LDS of a block");
};

template <bool W4, int BM, int BN, int WM, int WN, int S, int G, int R, bool GRAD>
__global__ __launch_bounds__(64 * WM * WN) void xent_logits_kernel(LogitArgs a) {
  using Lds = LogitLds<W4, BM, BN, WM, WN, S, G, R, GRAD>;
  constexpr int NW = WM * WN, NT = 64 * NW, BK = 128;
  constexpr int ASZ = Lds::ASZ, STG = Lds::STG;
  constexpr int FM = BM / WM / 16, FN = BN / WN / 16;
  // loads per wave and stage: 8 rows of 128 bytes (16 of 64) an instruction
  constexpr int AI = BM / 8 / NW, BI = BN / (W4 ? 16 : 8) / NW, LPS = AI + BI;
  static_assert(AI * 8 * NW == BM && BI * (W4 ? 16 : 8) * NW == BN, "whole instructions per wave");
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
  float esx[RT], else_[RT], egm[RT], esw[CT], ets[NTS > 0 ? NTS : 1], eqs[NQS > 0 ? NQS : 1];
  int etg[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    const int row = tid + NT * i, gm = m0 + row < M ? m0 + row : M - 1;
    esx[i] = a.sx[gm];
    etg[i] = row < BM && m0 + row < M ? entry_of(a.ids, gm) : -1;
    if constexpr (GRAD) {
      else_[i] = a.lse[gm];
      egm[i] = a.dloss[gm];
    }
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
      const int e = tid + NT * i, gm = m0 + e / R, j = e % R;
      ets[i] = a.t[(long)(gm < M ? gm : M - 1) * a.r + (j < a.r ? j : 0)];
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
#pragma unroll
    for (int kk = 0; kk < BK / 64; ++kk) {
      const int c = kk * 4 + q;
      i32x4 af[FM], bf[FN];
#pragma unroll
      for (int i = 0; i < FM; ++i)
        af[i] = *reinterpret_cast<const i32x4*>(As + swz128((wm * FM + i) * 16 + l, c));
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const int n = (wn * FN + j) * 16 + l;
        if constexpr (W4)
          bf[j] = widen_nibbles(*reinterpret_cast<const u32x2*>(Bs + n * 64 + (((c >> 1) ^ ((n >> 2) & 3)) << 4) +
                                                               (c & 1) * 8));
        else
          bf[j] = *reinterpret_cast<const i32x4*>(Bs + swz128(n, c));
      }
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          if constexpr (W4) part[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(af[i], bf[j], part[i][j], 0, 0, 0);
          else acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(af[i], bf[j], acc[i][j], 0, 0, 0);
        }
    }
    if constexpr (W4) {
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const float sc = (float)SC[((wn * FN + j) * 16 + l) * ngrp + kt];
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
          for (int ii = 0; ii < 4; ++ii)
            acc[i][j][ii] = __builtin_fmaf((float)part[i][j][ii], sc, acc[i][j][ii]);
      }
    }
    slot = slot == S - 1 ? 0 : slot + 1;
  }

  __syncthreads();                                         // every wave is done with the ring
  float* ts = reinterpret_cast<float*>(lds + Lds::TS);
  float* qs = reinterpret_cast<float*>(lds + Lds::QS);
  float* sxv = reinterpret_cast<float*>(lds + Lds::SX);
  float* swv = reinterpret_cast<float*>(lds + Lds::SW);
  int* tgv = reinterpret_cast<int*>(lds + Lds::TG);
  float* lsv = reinterpret_cast<float*>(lds + Lds::LS);
  float* gmv = reinterpret_cast<float*>(lds + Lds::GM);
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    const int row = tid + NT * i;
    if (row < BM) {
      sxv[row] = esx[i];
      tgv[row] = etg[i] >= 0 ? etg[i] - n0 : INT32_MIN;    // the target's column here; INT32_MIN: none
      if constexpr (GRAD) {
        lsv[row] = else_[i] * kLog2e;
        gmv[row] = egm[i];
      }
    }
  }
  if constexpr (!W4) {
#pragma unroll
    for (int i = 0; i < CT; ++i)
      if (tid + NT * i < BN) swv[tid + NT * i] = esw[i];
  }
  if constexpr (R > 0) {
#pragma unroll
    for (int i = 0; i < NTS; ++i) {
      const int e = tid + NT * i;
      if (e < BM * R) ts[e] = e % R < a.r && m0 + e / R < M ? ets[i] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < NQS; ++i) {
      const int e = tid + NT * i, j = e / BN, c = e % BN;
      if (e < BN * R) qs[j * Lds::QP + c] = j < a.r && n0 + c < a.V ? eqs[i] : 0.f;
    }
  }
  __syncthreads();

  const int wr0 = wm * FM * 16, wc0 = wn * FN * 16;
  constexpr int RB = (R + 15) / 16, RBA = RB > 0 ? RB : 1;
  f32x4 uacc[GRAD && R > 0 ? FM : 1][RBA], dbacc[GRAD && R > 0 ? FN : 1][RBA];
  if constexpr (GRAD && R > 0) {
#pragma unroll
    for (int j = 0; j < RB; ++j) {
#pragma unroll
      for (int i = 0; i < FM; ++i) uacc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < FN; ++i) dbacc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
  }
  int8_t* strip = lds + Lds::END + wid * Lds::STRIP;

#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const int r0 = wr0 + i * 16 + 4 * q;                   // the lane's four rows
    f32x4 lo[FN];
#pragma unroll
    for (int j = 0; j < FN; ++j) lo[j] = f32x4{0.f, 0.f, 0.f, 0.f};
    if constexpr (R > 0) {
#pragma unroll
      for (int kc = 0; kc < R / 4; ++kc) {
        const float ta = ts[(wr0 + i * 16 + l) * R + kc * 4 + q];
#pragma unroll
        for (int j = 0; j < FN; ++j)
          lo[j] = __builtin_amdgcn_mfma_f32_16x16x4f32(ta, qs[(kc * 4 + q) * Lds::QP + wc0 + j * 16 + l], lo[j], 0, 0, 0);
      }
    }
    const f32x4 sx4 = *reinterpret_cast<const f32x4*>(sxv + r0);
    const i32x4 tg4 = *reinterpret_cast<const i32x4*>(tgv + r0);
    f32x4 v[FN];                                           // the logits
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      const float sw = W4 ? 1.f : swv[wc0 + j * 16 + l];
#pragma unroll
      for (int ii = 0; ii < 4; ++ii) {
        const float base = (float)acc[i][j][ii] * (W4 ? sx4[ii] : sx4[ii] * sw);
        v[j][ii] = R > 0 ? __builtin_fmaf(a.s, lo[j][ii], base) : base;
      }
    }
    if constexpr (!GRAD) {
      float* red = reinterpret_cast<float*>(lds + Lds::END);      // [WN][BM] pairs
#pragma unroll
      for (int ii = 0; ii < 4; ++ii) {
        float mx = -INFINITY;
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          const int c = wc0 + j * 16 + l;
          const float x = v[j][ii];
          if (c == tg4[ii]) a.tl[m0 + r0 + ii] = x;        // (a row past M has no target)
          v[j][ii] = n0 + c < a.V ? x * kLog2e : -INFINITY;
          mx = fmaxf(mx, v[j][ii]);
        }
        mx = row16_max(mx);
        const float ref = mx == -INFINITY ? 0.f : mx;      // (no column here)
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < FN; ++j) sum += __builtin_amdgcn_exp2f(v[j][ii] - ref);
        sum = row16_sum(sum);
        if (l == 0) {
          red[2 * (wn * BM + r0 + ii)] = mx;
          red[2 * (wn * BM + r0 + ii) + 1] = sum;
        }
      }
    } else {
      const f32x4 ls4 = *reinterpret_cast<const f32x4*>(lsv + r0);
      const f32x4 gm4 = *reinterpret_cast<const f32x4*>(gmv + r0);
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const int c = wc0 + j * 16 + l;
        const bool in = n0 + c < a.V;
#pragma unroll
        for (int ii = 0; ii < 4; ++ii) {
          const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(v[j][ii], kLog2e, -ls4[ii]));
          const float d = gm4[ii] * (c == tg4[ii] ? p - 1.f : p);
          v[j][ii] = in && tg4[ii] != INT32_MIN ? d : 0.f;
        }
      }
      if constexpr (R > 0) {
        // dB: D[rank][column] += t^T dl, step ii over rows 4 q + ii
#pragma unroll
        for (int ii = 0; ii < 4; ++ii)
#pragma unroll
          for (int jb = 0; jb < RB; ++jb) {
            const float ta = 16 * jb + l < R ? ts[(r0 + ii) * R + (16 * jb + l < R ? 16 * jb + l : 0)] : 0.f;
#pragma unroll
            for (int j = 0; j < FN; ++j)
              dbacc[j][jb] = __builtin_amdgcn_mfma_f32_16x16x4f32(ta, v[j][ii], dbacc[j][jb], 0, 0, 0);
          }
        // u: dl from the strip as the A operand (row l, columns 4 c + q)
        float* fs = reinterpret_cast<float*>(strip);
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
          for (int ii = 0; ii < 4; ++ii) fs[(4 * q + ii) * Lds::FPITCH + j * 16 + l] = v[j][ii];
#pragma unroll
        for (int c = 0; c < FN * 4; ++c) {
          const float da = fs[l * Lds::FPITCH + 4 * c + q];
#pragma unroll
          for (int jb = 0; jb < RB; ++jb) {
            const int j = 16 * jb + l;
            const float bv = j < R ? qs[(j < R ? j : 0) * Lds::QP + wc0 + 4 * c + q] : 0.f;
            uacc[i][jb] = __builtin_amdgcn_mfma_f32_16x16x4f32(da, bv, uacc[i][jb], 0, 0, 0);
          }
        }
      }
      if constexpr (!W4) {
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          const float sw = swv[wc0 + j * 16 + l];
          const bool in = n0 + wc0 + j * 16 + l < a.V;
#pragma unroll
          for (int ii = 0; ii < 4; ++ii) v[j][ii] = in && tg4[ii] != INT32_MIN ? v[j][ii] * sw : 0.f;
        }
      }
      // (the strip is read as float above and written as bf16 below: in this order)
      asm volatile("" ::: "memory");
      for (int p = 0; p < a.parts; ++p) {
        // one 16-row strip in bf16 through LDS (this wave's own: no wait), what
        // is left of the values to the next part
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
          for (int ii = 0; ii < 4; ++ii) {
            const uint32_t h = f32_to_bf16(v[j][ii]);
            reinterpret_cast<uint16_t*>(strip + (4 * q + ii) * Lds::PITCH)[j * 16 + l] = (uint16_t)h;
            // (of an infinity or a NaN the first part is all)
            v[j][ii] = (h & 0x7f80u) == 0x7f80u ? 0.f : v[j][ii] - bf16_to_f32(h);
          }
#pragma unroll
        for (int e = 0; e < FN / 2; ++e) {
          const int u = lane + 64 * e, row = u / (FN * 2), cq = u % (FN * 2);
          const int m = m0 + wr0 + i * 16 + row;
          const u32x4 w = *reinterpret_cast<const u32x4*>(strip + row * Lds::PITCH + cq * 16);
          if (m < M)
            *reinterpret_cast<u32x4*>(a.g + p * a.gstride + m * a.ldg + c0 + wc0 + cq * 8) = w;
        }
        asm volatile("" ::: "memory");
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
  if constexpr (GRAD && R > 0) {
    // the tile's u and dB: the waves' sums added in order
    float* ub = reinterpret_cast<float*>(lds + Lds::UB);
    float* db = ub + BM * R;
    for (int w = 0; w < max_int(WM, WN); ++w) {
      if (wn == w) {
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
          for (int jb = 0; jb < RB; ++jb)
#pragma unroll
            for (int ii = 0; ii < 4; ++ii) {
              const int j = 16 * jb + l;
              float* p = ub + (wr0 + i * 16 + 4 * q + ii) * R + j;
              if (j < R) *p = w == 0 ? uacc[i][jb][ii] : *p + uacc[i][jb][ii];
            }
      }
      if (wm == w) {
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
          for (int jb = 0; jb < RB; ++jb)
#pragma unroll
            for (int ii = 0; ii < 4; ++ii) {
              const int rank = 16 * jb + 4 * q + ii;
              float* p = db + rank * BN + wc0 + j * 16 + l;
              if (rank < R) *p = w == 0 ? dbacc[j][jb][ii] : *p + dbacc[j][jb][ii];
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

// Joins the tiles of 64 rows, sixteen of them side by side, in a fixed order.
__global__ __launch_bounds__(1024) void xent_join_kernel(const float* part, const float* tl, Ids ids, int tiles, int M,
                                                         float* loss, float* lse) {
  __shared__ float red[16][64][2];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, m = blockIdx.x * 64 + lane;
  const int mc = m < M ? m : M - 1;
  float mx = -INFINITY, sum = 0.f;
  auto join = [&](float m2, float s2) {
    const float top = fmaxf(mx, m2);
    const float ref = top == -INFINITY ? 0.f : top;
    sum = sum * __builtin_amdgcn_exp2f(mx - ref) + s2 * __builtin_amdgcn_exp2f(m2 - ref);
    mx = top;
  };
  for (int c = w; c < tiles; c += 64) {
    float pm[4], ps[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const float* p = part + 2 * ((long)(c + 16 * u < tiles ? c + 16 * u : c) * M + mc);
      pm[u] = p[0];
      ps[u] = p[1];
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (c + 16 * u < tiles) join(pm[u], ps[u]);
  }
  red[w][lane][0] = mx;
  red[w][lane][1] = sum;
  __syncthreads();
  if (w != 0 || m >= M) return;
  for (int k = 1; k < 16; ++k) join(red[k][lane][0], red[k][lane][1]);
  const int t = entry_of(ids, m);
  const float top = mx * kLn2, rest = logf(sum);
  lse[m] = top + rest;
  // (the difference first: what the target's logit and the maximum share)
  loss[m] = t >= 0 ? (top - tl[m]) + rest : 0.f;
}

// ---- dx ---------------------------------------------------------------------------
struct DxArgs {
  int M, N, K, V;
  const uint16_t* g;     // [parts][M][ldg]
  long ldg, gstride;
  int parts;
  const int8_t* codes;
  const _Float16* scales;        // 4-bit
  int v0;                // first entry of the piece
  int tiles_m, tiles_k;
  int splits, nks;       // stages (of all parts) per split
  int first;             // the first piece: the buffer is written, not added to
  float* dxp;            // [splits][M][K]
};

template <bool W4, int BM, int WM, int S>
__global__ __launch_bounds__(64 * WM * 4) void xent_dx_kernel(DxArgs a) {
  constexpr int WN = 4, NW = WM * WN, BN = 256, KC = 64;
  constexpr int ASZ = BM * 128, RB = W4 ? 128 : 256;         // bytes of a row of codes
  constexpr int BSZ = KC * RB, SSZ = W4 ? NW * 256 : 0, STG = ASZ + BSZ + SSZ;
  constexpr int FM = BM / WM / 16;
  constexpr int AI = BM / 8 / NW, BI = BSZ / 1024 / NW, LPS = AI + BI + (W4 ? 1 : 0);
  static_assert(AI * 8 * NW == BM && BI * 1024 * NW == BSZ, "whole instructions per wave");
  static_assert(S * STG <= 160 * 1024, "LDS of a block");
  __shared__ __attribute__((aligned(1024))) int8_t ring[S * STG];

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
            const float x = (float)(int8_t)(w[2 * e] >> (8 * j)), y = (float)(int8_t)(w[2 * e + 1] >> (8 * j));
            bf[j][e] = __builtin_amdgcn_perm(__float_as_uint(y), __float_as_uint(x), 0x07060302u);
          }
      } else {
        uint32_t w[8];
        float sc[8];
        const uint32_t* sp = reinterpret_cast<const uint32_t*>(Bs + BSZ + wid * 256) + 32 * kk + 8 * q;
        const int v = a.v0 + (a.parts == 1 ? kt : kt % nkv) * KC + 32 * kk + 8 * q;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          w[e] = *reinterpret_cast<const uint16_t*>(row + e * RB + ((wn ^ q) << 5) + 2 * l);
          const int half = ((v + e) * ngrp + grp) & 1;       // (past N the clamped entry's half: masked)
          const uint16_t hb = (uint16_t)(sp[e] >> (16 * half));
          sc[e] = v + e < a.V ? (float)__builtin_bit_cast(_Float16, hb) : 0.f;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float x = (float)((int)(w[2 * e] << (28 - 4 * j)) >> 28) * sc[2 * e];
            const float y = (float)((int)(w[2 * e + 1] << (28 - 4 * j)) >> 28) * sc[2 * e + 1];
            bf[j][e] = pk_bf16(x, y);
          }
      }
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(af[i], __builtin_bit_cast(bf16x8, bf[j]), acc[i][j], 0, 0, 0);
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
// tiles' parts; the last piece also clears dB's padding. Thread per element.
struct ReduceArgs {
  int M, N, r, tiles_x, tiles_m, v0, vc, first, last, V;
  long ldg;
  float s;
  const float* up;
  const float* dbp;
  float* u;
  float* dB;
};
__global__ __launch_bounds__(256) void xent_reduce_kernel(ReduceArgs a) {
  const long e = (long)blockIdx.x * 256 + threadIdx.x, nu = (long)a.M * a.r;
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
  if (e < nu) {
    const float v = sum(a.up + e, nu, a.tiles_x);
    a.u[e] = a.first ? v : a.u[e] + v;
  } else if (e < nu + ndb) {
    const long j = (e - nu) / a.vc, c = (e - nu) % a.vc;
    a.dB[j * a.N + a.v0 + c] = a.s * sum(a.dbp + j * a.ldg + c, a.r * a.ldg, a.tiles_m);
  } else if (e < nu + ndb + npad) {
    const long j = (e - nu - ndb) / (a.N - a.V), c = (e - nu - ndb) % (a.N - a.V);
    a.dB[j * a.N + a.V + c] = 0.f;
  }
}

// dx = the splits' sums + s u A^T, four features a thread.
template <typename OutT>
__global__ __launch_bounds__(256) void xent_dx_join_kernel(const float* dxp, int splits, int M, int K, int r, float s,
                                                           const float* u, const float* A, OutT* dx) {
  const long e = ((long)blockIdx.x * 256 + threadIdx.x) * 4, n = (long)M * K;
  if (e >= n) return;
  f32x4 v = *reinterpret_cast<const f32x4*>(dxp + e);
  for (int i = 1; i < splits; ++i) v += *reinterpret_cast<const f32x4*>(dxp + i * n + e);
  if (r > 0) {
    const long m = e / K, k = e % K;
    f32x4 low{0.f, 0.f, 0.f, 0.f};
    for (int j = 0; j < r; ++j) {
      const float uj = u[m * r + j];
#pragma unroll
      for (int c = 0; c < 4; ++c) low[c] = __builtin_fmaf(uj, A[(k + c) * r + j], low[c]);
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) v[c] = __builtin_fmaf(s, low[c], v[c]);
  }
  if constexpr (sizeof(OutT) == 4) *reinterpret_cast<f32x4*>(dx + e) = v;
  else *reinterpret_cast<u32x2*>(dx + e) = u32x2{pk_bf16(v[0], v[1]), pk_bf16(v[2], v[3])};
}

// ---- launches ---------------------------------------------------------------------
template <bool W4, int BM, int BN, int WM, int WN, int S, int G, bool GRAD>
void logits_ranks(LogitArgs& a, int cols, hipStream_t st) {
  a.tiles_m = (a.M + BM - 1) / BM;
  a.tiles_x = (cols + BN - 1) / BN;
  const dim3 grid((unsigned)(a.tiles_m * a.tiles_x));
  constexpr int NT = 64 * WM * WN;
  if (a.r == 0) xent_logits_kernel<W4, BM, BN, WM, WN, S, G, 0, GRAD><<<grid, NT, 0, st>>>(a);
  else if (a.r <= 4) xent_logits_kernel<W4, BM, BN, WM, WN, S, G, 4, GRAD><<<grid, NT, 0, st>>>(a);
  else if (a.r <= 8) xent_logits_kernel<W4, BM, BN, WM, WN, S, G, 8, GRAD><<<grid, NT, 0, st>>>(a);
  else if (BM * BN > 128 * 128 || a.r <= 16)
    xent_logits_kernel<W4, BM, BN, WM, WN, S, G, 16, GRAD><<<grid, NT, 0, st>>>(a);
  else if constexpr (BM * BN <= 128 * 128)
    xent_logits_kernel<W4, BM, BN, WM, WN, S, G, 32, GRAD><<<grid, NT, 0, st>>>(a);
}

// The tiles of a launch over `cols` entries; fills tiles_m and tiles_x.
template <bool GRAD>
void logits(LogitArgs& a, int fmt, int cols, hipStream_t st) {
  if (fmt == 0) {
    if (a.M <= 32) logits_ranks<false, 32, 256, 1, 4, 4, 1, GRAD>(a, cols, st);
    else if (a.M > 128 && a.r <= 16) logits_ranks<false, 256, 256, 2, 4, 2, 1, GRAD>(a, cols, st);
    else logits_ranks<false, 128, 128, 2, 2, 2, 1, GRAD>(a, cols, st);
  } else if (a.M <= 32) {
    if (a.K <= 4096) logits_ranks<true, 32, 128, 1, 4, 3, 32, GRAD>(a, cols, st);
    else logits_ranks<true, 32, 128, 1, 4, 3, 128, GRAD>(a, cols, st);
  } else {
    if (a.K <= 4096) logits_ranks<true, 128, 128, 2, 2, 2, 32, GRAD>(a, cols, st);
    else logits_ranks<true, 128, 128, 2, 2, 2, 128, GRAD>(a, cols, st);
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

template <bool W4>
void launch_dx(const DxArgs& a, int rows, hipStream_t st) {
  const dim3 grid((unsigned)(a.tiles_m * a.tiles_k * a.splits));
  if (rows == 32) xent_dx_kernel<W4, 32, 1, 3><<<grid, 256, 0, st>>>(a);
  else if (rows == 128) xent_dx_kernel<W4, 128, 2, 3><<<grid, 512, 0, st>>>(a);
  else xent_dx_kernel<W4, 256, 2, 3><<<grid, 512, 0, st>>>(a);
}

}  // namespace

size_t xent_part_floats(int fmt, int vocab, int M) {
  (void)fmt;
  return ((size_t)((vocab + 127) / 128) * 2 + 1) * (size_t)M;
}

void launch_xent_fwd(const VocabLayer& L, int M, Ids ids, const int8_t* xq, const float* sx,
                     const float* t, float* part, float* loss, float* lse, hipStream_t st) {
  LogitArgs a = logit_args(L, M, ids, xq, sx, t);
  a.tl = part;
  a.part = part + M;
  logits<false>(a, L.fmt, ids.vocab, st);
  xent_join_kernel<<<dim3((unsigned)((M + 63) / 64)), 1024, 0, st>>>(a.part, a.tl, ids, a.tiles_x, M, loss, lse);
}

XentPlan xent_plan(const VocabLayer& L, int vocab, int M, int dtype) {
  XentPlan p{};
  p.parts = dtype == 0 ? 3 : 1;
  const int all = (vocab + 255) / 256 * 256;
  const long most = (64L << 20) / p.parts / M / 256 * 256;      // 128 MB of dl
  p.piece = (int)(most < 512 ? 512 : most > all ? all : most);
  if (p.piece > all) p.piece = all;
  const int rows = dx_rows(M);
  const long tiles = (long)((M + rows - 1) / rows) * ((L.K + 255) / 256);
  const int nk = p.parts * (p.piece / 64);
  p.splits = 1;
  while (tiles * p.splits * 2 <= kCUs && nk / (p.splits * 2) >= 8) p.splits *= 2;
  p.g = (size_t)p.parts * M * p.piece;
  p.dxp = (size_t)p.splits * M * L.K;
  if (L.r > 0) {
    p.u = (size_t)M * L.r;
    p.up = (size_t)(p.piece / 128) * M * L.r;
    p.dbp = (size_t)((M + 127) / 128) * L.r * p.piece;
  }
  return p;
}

void launch_xent_bwd(const VocabLayer& L, int M, int dtype, Ids ids, const int8_t* xq, const float* sx,
                     const float* t, const float* lse, const float* dloss, const XentPlan& plan,
                     const XentBuffers& buf, void* dx, float* dB, hipStream_t st) {
  const int V = ids.vocab;
  const int rows = dx_rows(M);
  for (int v0 = 0; v0 < V; v0 += plan.piece) {
    const int vc = V - v0 < plan.piece ? V - v0 : plan.piece;
    const long ldg = (vc + 255) / 256 * 256;
    LogitArgs a = logit_args(L, M, ids, xq, sx, t);
    a.v0 = v0; a.lse = lse; a.dloss = dloss; a.g = buf.g; a.ldg = ldg; a.gstride = M * ldg; a.parts = plan.parts;
    a.up = buf.up; a.dbp = buf.dbp;
    logits<true>(a, L.fmt, (int)ldg, st);
    if (dx != nullptr) {
      DxArgs d{};
      d.M = M; d.N = L.N; d.K = L.K; d.V = V; d.g = buf.g; d.ldg = ldg; d.gstride = a.gstride; d.parts = plan.parts;
      d.codes = a.codes; d.scales = static_cast<const _Float16*>(L.scales); d.v0 = v0;
      d.tiles_m = (M + rows - 1) / rows; d.tiles_k = (L.K + 255) / 256;
      d.splits = plan.splits;
      d.nks = (plan.parts * (int)(ldg / 64) + plan.splits - 1) / plan.splits;
      d.first = v0 == 0; d.dxp = buf.dxp;
      if (L.fmt == 0) launch_dx<false>(d, rows, st);
      else launch_dx<true>(d, rows, st);
    }
    if (L.r > 0) {
      ReduceArgs r{M, L.N, L.r, a.tiles_x, a.tiles_m, v0, vc, v0 == 0, v0 + vc == V, V, ldg, L.s,
                   buf.up, buf.dbp, buf.u, dB};
      const long n = (long)M * L.r + (long)L.r * vc + (r.last ? (long)L.r * (L.N - V) : 0);
      xent_reduce_kernel<<<dim3((unsigned)((n + 255) / 256)), 256, 0, st>>>(r);
    }
  }
  if (dx == nullptr) return;
  const dim3 grid((unsigned)(((long)M * L.K / 4 + 255) / 256));
  if (dtype == 0)
    xent_dx_join_kernel<float><<<grid, 256, 0, st>>>(buf.dxp, plan.splits, M, L.K, L.r, L.s, buf.u, L.A,
                                                    static_cast<float*>(dx));
  else
    xent_dx_join_kernel<uint16_t><<<grid, 256, 0, st>>>(buf.dxp, plan.splits, M, L.K, L.r, L.s, buf.u, L.A,
                                                       static_cast<uint16_t*>(dx));
}

}  // namespace qlora
