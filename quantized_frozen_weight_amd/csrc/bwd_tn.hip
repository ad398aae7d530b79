// Backward of the layer over a weight laid out for it: a first launch writes
// the dequantized weight once, transposed, as bf16 Wt [K][N] = bf16(deq(W)),
// and the adapter's B as three bf16 parts (bwd_common.hpp) [3 R rows][N]; the
// second is then a plain bf16 product over n,
//
//   [dx0 | u] = dy [Wt | B]^T,   dx = (dx0 + s u A^T) act'(z) + add
//   dB = s t^T dy,   dA = s x^T u      (partial sums per row block)
//
// in which every operand moves from memory to LDS untouched (ring.hpp) and
// nothing is converted between the barriers. gemm_bwd.hip converts the codes
// of a stage once per block and stage instead: it reads a quarter of the
// weight bytes, but at 128 x 128 tiles its vector work and its second barrier
// cost more than the matrix instructions (the measurements are at
// bwd_tn_takes). Counters of the second launch: at 128 x 64 tiles (4096 x 768
// x 2304) the matrix cores are busy 26 % of the time, 40 % of a wave's time
// goes to waiting for its stage's loads and the barrier, 24 % to waiting for
// an issue slot; at 128 x 128 (4096 x 2048 x 16384) 36 % busy and the LDS 23 %:
// a stage's 36 KB in and 72 KB out and its 576 cycles of matrix work a SIMD
// follow one another in each block, and two blocks a compute unit overlap
// them in part (up to rank 8, at 82 KB of LDS a block of 128 x 128; ranks 16
// and 32 take 90 and 115 KB for B's parts, and one block a compute unit).
//
// Around the product it does what gemm_bwd.hip does, with the same operands
// and the same partial-sum layout (so the same combine and, where the
// contraction is split, the same second launch): u on the matrix cores
// beside dx, the dB partial of every tiles_x-th stage from the dy tile, the
// dA partial from an x tile (bf16, or the 8-bit row checkpoint's codes with
// the row scales multiplied into u), and the gradient epilogue.
#include "bwd_common.hpp"
#include "epilogue.hpp"
#include "launch.hpp"
#include "ring.hpp"

namespace qlora {

namespace {

struct TnArgs {
  int M, K, N;
  const uint16_t* dy;      // [M, N] bf16
  const uint16_t* Wt;      // [K, N] bf16
  const uint16_t* BU;      // [16 UCB, N] bf16: B's hi, mid and lo parts, then zeros
  const float* A;          // [K, r]
  const float* t;          // [M, r]
  const uint16_t* x;       // [M, K] bf16, or its row checkpoint (xq not NULL):
  const int8_t* xq;
  const float* sx;
  int r;
  float s;
  uint16_t* dx;            // [M, K]
  float* partA;            // [row blocks, r, K]
  float* partB;            // [row blocks, r, N]
  int tiles_x;
  float* pdx;              // split: as in gemm_bwd.hip
  float* pu;
  int splits, nks;
  GradEpi ge;
};

constexpr int part_blocks(int R) { return (3 * R + 15) / 16; }   // 16-row blocks of BU

// ---- the weight and B laid out ------------------------------------------------
struct PrepArgs {
  int K, N;
  const int8_t* codes;     // [N, K], or packed [N, K / 2]
  const void* scales;
  const float* B;
  int hd, r, R;            // R: the rank the parts are spaced by
  uint16_t* Wt;
  uint16_t* BU;
  int tiles_k, tiles;
};

// Blocks [0, tiles): a tile of 64 n x 64 k (4-bit: 64 n x 128 k), its codes
// read as 16-byte pieces, turned in LDS, and written as 128-byte runs of Wt
// rows. The blocks after them: B's parts, two columns per thread.
template <bool W4>
__global__ __launch_bounds__(256) void bwd_prep_kernel(PrepArgs a) {
  constexpr int TK = W4 ? 128 : 64, RB = 64, PITCH = RB + 16;
  __shared__ __attribute__((aligned(16))) int8_t raw[64 * PITCH];
  const int tid = threadIdx.x, K = a.K, N = a.N;
  if ((int)blockIdx.x >= a.tiles) {
    const long e = ((long)blockIdx.x - a.tiles) * 256 + tid;
    const int half = N / 2, rows = 16 * part_blocks(a.R);
    const int j = (int)(e / half), n = 2 * (int)(e % half);
    if (j >= a.R) {                            // rank rows here; zero rows past the parts
      const int z = 3 * a.R + (j - a.R);
      if (z < rows) *reinterpret_cast<uint32_t*>(a.BU + (long)z * N + n) = 0u;
      return;
    }
    float b0 = 0.f, b1 = 0.f;
    if (j < a.r) {
      const float* p = a.B + head_index(j, n, a.r, a.hd);   // (a pair never straddles a head)
      b0 = p[0];
      b1 = p[1];
    }
    uint32_t mid, lo;
    const uint32_t hi = pk_bf16_split3(b0, b1, mid, lo);
    *reinterpret_cast<uint32_t*>(a.BU + (long)j * N + n) = hi;
    *reinterpret_cast<uint32_t*>(a.BU + (long)(a.R + j) * N + n) = mid;
    *reinterpret_cast<uint32_t*>(a.BU + (long)(2 * a.R + j) * N + n) = lo;
    return;
  }
  const int k0 = (int)(blockIdx.x % a.tiles_k) * TK, n0 = (int)(blockIdx.x / a.tiles_k) * 64;
  const long crs = W4 ? K / 2 : K;
  {
    const int row = tid >> 2, c = 16 * (tid & 3), gn = n0 + row;
    const long gk = (W4 ? k0 / 2 : k0) + c;
    const u32x4 v = *reinterpret_cast<const u32x4*>(a.codes + (long)(gn < N ? gn : N - 1) * crs +
                                                    (gk < crs ? gk : crs - 16));
    *reinterpret_cast<u32x4*>(raw + row * PITCH + c) = v;
  }
  const int nq = tid & 15, kq = tid >> 4, gn = n0 + 4 * nq;
  const bool okn = gn < N;                     // N % 16 == 0: four columns in or out
  float sc[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = okn ? gn + i : N - 1;
    if constexpr (W4) sc[i] = (float)static_cast<const _Float16*>(a.scales)[(long)n * (K / 128) + k0 / 128];
    else sc[i] = static_cast<const float*>(a.scales)[n];
  }
  __syncthreads();
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const uint32_t*>(raw + (4 * nq + i) * PITCH + 4 * kq);
  if constexpr (W4) {
    float v[4][8];
#pragma unroll
    for (int i = 0; i < 4; ++i) nibble_vals(w[i], sc[i], v[i]);
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (okn)                                 // K % 128 == 0
        *reinterpret_cast<u32x2*>(a.Wt + (long)(k0 + 8 * kq + e) * N + gn) =
            u32x2{pk_bf16(v[0][e], v[1][e]), pk_bf16(v[2][e], v[3][e])};
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int k = k0 + 4 * kq + e;
      float v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = (float)(int8_t)(w[i] >> (8 * e)) * sc[i];
      if (okn && k < K)
        *reinterpret_cast<u32x2*>(a.Wt + (long)k * N + gn) = u32x2{pk_bf16(v[0], v[1]), pk_bf16(v[2], v[3])};
    }
  }
}

// ---- the product ----------------------------------------------------------------
// 256 threads, 2 x 2 waves of (BM / 2) x (BN / 2).
template <int BM, int BN, int S, int R, bool SPLIT>
__global__ __launch_bounds__(256, 2) void bwd_tn_kernel(TnArgs a) {
  constexpr int KC = 64;                              // n per stage
  constexpr int UCB = part_blocks(R), RCB = (R + 15) / 16;
  constexpr int ASZ = BM * 128, BSZ = BN * 128, USZ = UCB * 16 * 128, STG = ASZ + BSZ + USZ;
  // loads per wave and stage; the B parts' 2 UCB instructions are dealt to the
  // four waves, some of them twice (same bytes), so that every wave counts alike
  constexpr int AI = BM / 32, BI = BN / 32, UI = (2 * UCB + 3) / 4, LPS = AI + BI + UI;
  constexpr int FM = BM / 32, FN = BN / 32, MC = BM / 32;
  static_assert(FM % 2 == 0, "the u products pair the 16-row blocks by column half");
  constexpr int EFL = (BM + BN) * R;                  // U [BM][R] | A^T [R][BN]
  constexpr int XTSZ = BM * BN * 2, UFSZ = UCB * MC * 1024;
  constexpr int RING = S * STG;
  static_assert(EFL * 4 + XTSZ + UFSZ <= RING, "epilogue operands, x tile and u operand fit in the ring");
  static_assert(4 * fused_strip_bytes<FN>() <= XTSZ + UFSZ, "the strips go over the x tile and the u operand");
  __shared__ __attribute__((aligned(1024))) int8_t ring[RING + UFSZ];
  int8_t* TF = ring + RING;                            // t operand [UCB][MC][64 lanes][16 B]

  const int tid = threadIdx.x, lane = tid & 63, wid = wave_id();
  const int wm = wid >> 1, wn = wid & 1;
  const int M = a.M, K = a.K, N = a.N, r = a.r;
  const int nk = (N + KC - 1) / KC;
  int bid = (int)blockIdx.x, split = 0;
  const int tiles = a.tiles_x * ((M + BM - 1) / BM);
  int mt, kt_blk;
  if constexpr (SPLIT) {
    // split-major, renumbered so that one XCD's blocks share a split's n range
    const int nb = (int)gridDim.x;
    if ((nb & 7) == 0) bid = (bid & 7) * (nb >> 3) + (bid >> 3);
    split = bid / tiles;
    bid -= split * tiles;
    mt = bid / a.tiles_x;
    kt_blk = bid % a.tiles_x;
  } else {
    xcd_tile(bid, (M + BM - 1) / BM, a.tiles_x, mt, kt_blk);
  }
  const int m0 = mt * BM, k0 = kt_blk * BN;
  const int kt0 = SPLIT ? split * a.nks : 0;
  const int kt1 = SPLIT ? (kt0 + a.nks < nk ? kt0 + a.nks : nk) : nk;

  // Stage loads: 128-byte rows swizzled by 16-byte chunk, 8 rows per
  // instruction, as 32-bit offsets from the operand's column nb. Rows past M
  // and K repeat the last one (their products are never stored).
  uint32_t voA[AI], voB[BI], voU[UI];
  int cA[AI], cB[BI], cU[UI], lu[UI];
#pragma unroll
  for (int i = 0; i < AI; ++i) {
    const int row = wid * (BM / 4) + i * 8 + (lane >> 3), gm = m0 + row;
    cA[i] = 8 * ((lane & 7) ^ ((row >> 1) & 7));
    voA[i] = (uint32_t)(((long)(gm < M ? gm : M - 1) * N + cA[i]) * 2);
  }
#pragma unroll
  for (int i = 0; i < BI; ++i) {
    const int row = wid * (BN / 4) + i * 8 + (lane >> 3), gk = k0 + row;
    cB[i] = 8 * ((lane & 7) ^ ((row >> 1) & 7));
    voB[i] = (uint32_t)(((long)(gk < K ? gk : K - 1) * N + cB[i]) * 2);
  }
#pragma unroll
  for (int i = 0; i < UI; ++i) {
    lu[i] = (wid * UI + i) % (2 * UCB);
    const int row = lu[i] * 8 + (lane >> 3);
    cU[i] = 8 * ((lane & 7) ^ ((row >> 1) & 7));
    voU[i] = (uint32_t)(((long)row * N + cU[i]) * 2);
  }
  auto issue = [&](int kt, int slot) {
    int8_t* base = ring + slot * STG;
    const int nb = kt * KC;
    const int8_t* pa = reinterpret_cast<const int8_t*>(a.dy + nb);
    const int8_t* pb = reinterpret_cast<const int8_t*>(a.Wt + nb);
    const int8_t* pu = reinterpret_cast<const int8_t*>(a.BU + nb);
    if (nb + KC <= N) {
#pragma unroll
      for (int i = 0; i < AI; ++i) lds_dma16(pa + voA[i], base + (wid * (BM / 4) + i * 8) * 128);
#pragma unroll
      for (int i = 0; i < BI; ++i) lds_dma16(pb + voB[i], base + ASZ + (wid * (BN / 4) + i * 8) * 128);
#pragma unroll
      for (int i = 0; i < UI; ++i) lds_dma16(pu + voU[i], base + ASZ + BSZ + lu[i] * 1024);
      return;
    }
    // the ragged last stage: chunks past N are zero
#pragma unroll
    for (int i = 0; i < AI; ++i)
      lds_dma16(nb + cA[i] < N ? (const void*)(pa + voA[i]) : (const void*)zero_chunk(lane),
                base + (wid * (BM / 4) + i * 8) * 128);
#pragma unroll
    for (int i = 0; i < BI; ++i)
      lds_dma16(nb + cB[i] < N ? (const void*)(pb + voB[i]) : (const void*)zero_chunk(lane),
                base + ASZ + (wid * (BN / 4) + i * 8) * 128);
#pragma unroll
    for (int i = 0; i < UI; ++i)
      lds_dma16(nb + cU[i] < N ? (const void*)(pu + voU[i]) : (const void*)zero_chunk(lane),
                base + ASZ + BSZ + lu[i] * 1024);
  };

  f32x4 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  f32x4 uacc[FM / 2][UCB];
#pragma unroll
  for (int i = 0; i < FM / 2; ++i)
#pragma unroll
    for (int j = 0; j < UCB; ++j) uacc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  // The dB operand, t in three parts: fragment (cb, c), lane -> column
  // cb 16 + lane % 16 (part j / R of rank j % R), rows 32 c + 8 (lane / 16) + e.
  // Wave w builds fragments w, w + 4, ... (its t values are loaded before the
  // stage loads, which complete behind them).
  constexpr int NF = (UCB * MC + 3) / 4;
  float tv[NF][8];
#pragma unroll
  for (int q = 0; q < NF; ++q) {
    const int f = wid + 4 * q, cb = f / MC, c = f % MC;
    const int j = cb * 16 + (lane & 15), part = j / R, jr = j - part * R;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int gm = m0 + 32 * c + 8 * (lane >> 4) + e;
      tv[q][e] = a.t[(long)(gm < M ? gm : M - 1) * r + (jr < r ? jr : 0)];
      if (!(f < UCB * MC && jr < r && part < 3 && gm < M)) tv[q][e] = 0.f;
    }
  }
#pragma unroll
  for (int st = 0; st < S - 1; ++st)
    if (kt0 + st < kt1) issue(kt0 + st, st);
#pragma unroll
  for (int q = 0; q < NF; ++q) {
    const int f = wid + 4 * q, part = (f / MC * 16 + (lane & 15)) / R;
    u32x4 hi, mid, lo;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      uint32_t me, le;
      hi[e] = pk_bf16_split3(tv[q][2 * e], tv[q][2 * e + 1], me, le);
      mid[e] = me;
      lo[e] = le;
    }
    if (f < UCB * MC)
      *reinterpret_cast<u32x4*>(TF + (f * 64 + lane) * 16) = part == 0 ? hi : part == 1 ? mid : lo;
  }
  __builtin_amdgcn_s_waitcnt(lgkmcnt0_imm());          // before the loop's first barrier

  int slot = 0;
  for (int kt = kt0; kt < kt1; ++kt) {
    wait_stages<LPS, 0, S - 2>(kt1 - 1 - kt);          // stage kt has landed (this wave)
    __builtin_amdgcn_s_barrier();                      // ... for every wave; slot of kt - 1 is free
    if (kt + S - 1 < kt1) issue(kt + S - 1, slot == 0 ? S - 1 : slot - 1);
    const int8_t* As = ring + slot * STG;
    const int8_t* Bs = As + ASZ;
    const int8_t* Us = Bs + BSZ;
#pragma unroll
    for (int kk = 0; kk < KC / 32; ++kk) {
      const int c = kk * 4 + (lane >> 4);
      bf16x8 af[FM], bf[FN];
#pragma unroll
      for (int i = 0; i < FM; ++i)
        af[i] = *reinterpret_cast<const bf16x8*>(As + swz128(wm * (BM / 2) + i * 16 + (lane & 15), c));
#pragma unroll
      for (int j = 0; j < FN; ++j)
        bf[j] = *reinterpret_cast<const bf16x8*>(Bs + swz128(wn * (BN / 2) + j * 16 + (lane & 15), c));
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(af[i], bf[j], acc[i][j], 0, 0, 0);
#pragma unroll
      for (int cb = 0; cb < UCB; ++cb) {
        const bf16x8 bu = *reinterpret_cast<const bf16x8*>(Us + swz128(cb * 16 + (lane & 15), c));
#pragma unroll
        for (int h = 0; h < FM / 2; ++h)
          uacc[h][cb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(pick_frag(af[2 * h], af[2 * h + 1], wn != 0),
                                                               bu, uacc[h][cb], 0, 0, 0);
      }
    }
    // dB partial of this stage's 64 n (one block per row block and stage):
    // wave w takes n in [16 w, 16 w + 16), dy^T through transposing reads (in
    // each 16-lane group lanes 4 i + p fetch the 4 n at 16 w + 4 p of row i,
    // and lane q receives n = 16 w + q of rows 0..3)
    if (kt % a.tiles_x == kt_blk) {
      f32x4 dbacc[UCB];
#pragma unroll
      for (int cb = 0; cb < UCB; ++cb) dbacc[cb] = f32x4{0.f, 0.f, 0.f, 0.f};
      const int q = lane & 15, i4 = q >> 2, p4 = q & 3;
#pragma unroll
      for (int c0 = 0; c0 < MC; c0 += 2) {
        uint32_t tra[4];
        uint64_t trv[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int m = 32 * (c0 + u / 2) + 8 * (lane >> 4) + 4 * (u & 1) + i4;
          const int n = 16 * wid + 4 * p4;
          tra[u] = lds_addr(As + swz128(m, n >> 3) + (n & 7) * 2);
        }
        tr16_reads<4>(tra, trv);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const bf16x8 dyT = __builtin_bit_cast(bf16x8, u32x4{(uint32_t)trv[2 * h], (uint32_t)(trv[2 * h] >> 32),
                                                              (uint32_t)trv[2 * h + 1], (uint32_t)(trv[2 * h + 1] >> 32)});
#pragma unroll
          for (int cb = 0; cb < UCB; ++cb) {
            const bf16x8 tf = *reinterpret_cast<const bf16x8*>(TF + ((cb * MC + c0 + h) * 64 + lane) * 16);
            dbacc[cb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(dyT, tf, dbacc[cb], 0, 0, 0);
          }
        }
      }
#pragma unroll
      for (int cb = 0; cb < RCB; ++cb) {
        const int j = cb * 16 + (lane & 15);
#pragma unroll
        for (int ii = 0; ii < 4; ++ii) {
          const float dbv = split3_sum<R, UCB>(dbacc, cb, ii, lane);
          const int gn = kt * KC + 16 * wid + 4 * (lane >> 4) + ii;
          if (j < r && gn < N) a.partB[((long)mt * r + j) * N + gn] = dbv;
        }
      }
    }
    slot = slot == S - 1 ? 0 : slot + 1;
  }

  if constexpr (SPLIT) {
    // partial products and the column-tile-0 blocks' partial u, as gemm_bwd.hip
    // lays them out
    f32x4* P = reinterpret_cast<f32x4*>(a.pdx) + ((long)(split * tiles + bid) * 4 + wid) * (FM * FN * 64) + lane;
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) P[(i * FN + j) * 64] = acc[i][j];
    if (kt_blk == 0) {
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        if ((i & 1) != wn) continue;
#pragma unroll
        for (int cb = 0; cb < RCB; ++cb) {
          const int j = cb * 16 + (lane & 15);
#pragma unroll
          for (int ii = 0; ii < 4; ++ii) {
            const float uv = split3_sum<R, UCB>(uacc[i >> 1], cb, ii, lane);
            const int gm = m0 + wm * (BM / 2) + i * 16 + (lane >> 4) * 4 + ii;
            if (j < r && gm < M) a.pu[((long)split * M + gm) * r + j] = uv;
          }
        }
      }
    }
    return;
  }

  // ---- after the contraction: u and A^T to LDS, x tile, dA partial, epilogue ----
  float* E = reinterpret_cast<float*>(ring);             // U [BM][R] | A^T [R][BN]
  int8_t* Xs = ring + EFL * 4;                           // x tile [BM][BN] bf16
  int8_t* UF = Xs + XTSZ;                                // u operand
  const int rows_here = M - m0 < BM ? M - m0 : BM;
  const bool x8on = a.xq != nullptr;
  X8Tile<BM, BN> x8;
  float rsv[8];
  __syncthreads();                                        // ring released
  if (x8on) {
    x8.fetch(a.xq, M, K, m0, k0, tid);
    // the scales of the rows whose part of the u operand this wave builds
    static_assert(4 % MC == 0, "wave w's fragments w, w + 4, ... are all of rows 32 (w % MC)");
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int gm = m0 + 32 * (wid % MC) + 8 * (lane >> 4) + e;
      rsv[e] = a.sx[gm < M ? gm : M - 1];
    }
  } else {
    constexpr int RH = BN / 64;                           // 128-byte halves per row
#pragma unroll
    for (int i = 0; i < BM * RH / 32; ++i) {
      const int rb = (wid * (BM * RH / 32) + i) * 8, hrow = rb + (lane >> 3);
      const int row = hrow / RH, half = hrow % RH;
      const int c = (lane & 7) ^ ((hrow >> 1) & 7);
      const int gm = m0 + row, gk = k0 + half * 64 + c * 8;
      lds_dma16(gk < K && gm < M ? (const void*)(a.x + (long)gm * K + gk) : (const void*)zero_chunk(lane),
                Xs + rb * 128);
    }
  }
  constexpr int NQ = (BN * R + 255) / 256;
  float qv[NQ];
#pragma unroll
  for (int i = 0; i < NQ; ++i) {
    const int e = tid + 256 * i, j = e / BN, col = e % BN, gk = k0 + col;
    qv[i] = a.A[(long)(gk < K ? gk : K - 1) * r + (j < r ? j : r - 1)];
  }
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    if ((i & 1) != wn) continue;
#pragma unroll
    for (int cb = 0; cb < RCB; ++cb) {
      const int j = cb * 16 + (lane & 15);
#pragma unroll
      for (int ii = 0; ii < 4; ++ii) {
        const float uv = split3_sum<R, UCB>(uacc[i >> 1], cb, ii, lane);
        const int ml = wm * (BM / 2) + i * 16 + (lane >> 4) * 4 + ii;
        if (j < R) E[ml * R + j] = j < r ? uv : 0.f;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NQ; ++i) {
    const int e = tid + 256 * i, j = e / BN, col = e % BN;
    if (e < BN * R) E[BM * R + e] = (j < r && k0 + col < K) ? qv[i] : 0.f;
  }
  if (x8on) x8.put(Xs, tid);
  __syncthreads();
  put_u_operand<BM, R>(UF, E, rows_here, r, x8on, rsv);
  EpiSide<uint16_t, GradEpi, FM, FN> es;
  __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));              // the x tile
  es.start(a.ge, M, K, m0 + wm * (BM / 2), k0 + wn * (BN / 2));   // (lands behind the dA products)
  __syncthreads();
  da_products<BM, BN, R>(Xs, UF, E, x8on ? a.sx + m0 : nullptr, rows_here, r, k0, K, a.partA + (long)mt * r * K);
  __syncthreads();                                        // every wave is done with the x tile and the u operand
  epilogue_fused<BM, BN, R, false>(acc, E, M, K, m0, k0, wm * (BM / 2), wn * (BN / 2), a.s, a.dx, a.ge, es,
                                   Xs + wid * fused_strip_bytes<FN>());
}

template <int BM, int BN, int S, bool SPLIT>
void tn_launch(TnArgs a, hipStream_t st) {
  a.tiles_x = (a.K + BN - 1) / BN;
  const dim3 grid((unsigned)(a.tiles_x * ((a.M + BM - 1) / BM) * (SPLIT ? a.splits : 1)));
  if (a.r <= 4) bwd_tn_kernel<BM, BN, S, 4, SPLIT><<<grid, 256, 0, st>>>(a);
  else if (a.r <= 8) bwd_tn_kernel<BM, BN, S, 8, SPLIT><<<grid, 256, 0, st>>>(a);
  else if (a.r <= 16) bwd_tn_kernel<BM, BN, S, 16, SPLIT><<<grid, 256, 0, st>>>(a);
  else bwd_tn_kernel<BM, BN, S, 32, SPLIT><<<grid, 256, 0, st>>>(a);
}

inline int rank_width(int r) { return r <= 4 ? 4 : r <= 8 ? 8 : r <= 16 ? 16 : 32; }

}  // namespace

bool bwd_tn_takes(int fmt, int M, int K, int N) {
  // From 1024 rows the second launch's gain pays for the first launch and its
  // 3 bytes a weight (with tanh gelu and z in 8 bits: 1024 x 16384 x 2048 128
  // against 142 us, 4096 x 768 x 2304 46 against 56, 4096 x 2048 x 16384 369
  // against 470); below it does not (512 x 16384 x 2048 80 against 76), nor do
  // layers of so few weights that a launch is what it costs (4096 x 256 x 256
  // 17.8 against 17.5).
  return (fmt == 0 || fmt == 1) && M >= 1024 && (long)K * N >= 1L << 19;
}

size_t bwd_tn_bytes(int K, int N, int r) {
  const size_t w = ((size_t)K * N * 2 + 255) / 256 * 256;
  return w + (size_t)16 * part_blocks(rank_width(r)) * N * 2;
}

void launch_bwd_tn(int fmt, int M, int K, int N, const uint16_t* dy, const void* codes,
                   const void* scales, const float* B, int hd, const float* A, const float* t,
                   const uint16_t* x, const int8_t* xq, const float* sx, int r, float s, uint16_t* dx,
                   float* partA, float* partB, float* pdx, float* pu, void* wt, const GradEpi& ge,
                   hipStream_t st) {
  PrepArgs p{};
  p.K = K; p.N = N; p.codes = static_cast<const int8_t*>(codes); p.scales = scales;
  p.B = B; p.hd = hd; p.r = r; p.R = rank_width(r);
  p.Wt = static_cast<uint16_t*>(wt);
  p.BU = reinterpret_cast<uint16_t*>(static_cast<char*>(wt) + ((size_t)K * N * 2 + 255) / 256 * 256);
  const int tk = fmt == 1 ? 128 : 64;
  p.tiles_k = (K + tk - 1) / tk;
  p.tiles = p.tiles_k * ((N + 63) / 64);
  const int zero_rows = 16 * part_blocks(p.R) - 3 * p.R;
  const long pairs = (long)(p.R + zero_rows) * (N / 2);
  const unsigned blocks = (unsigned)(p.tiles + (pairs + 255) / 256);
  if (fmt == 1) bwd_prep_kernel<true><<<blocks, 256, 0, st>>>(p);
  else bwd_prep_kernel<false><<<blocks, 256, 0, st>>>(p);

  TnArgs a{};
  a.M = M; a.K = K; a.N = N; a.dy = dy; a.Wt = p.Wt; a.BU = p.BU; a.A = A; a.t = t; a.x = x; a.xq = xq;
  a.sx = sx; a.r = r; a.s = s; a.dx = dx; a.partA = partA; a.partB = partB; a.pdx = pdx; a.pu = pu;
  a.ge = ge;
  const int bm = bwd_row_block(fmt, M, K, N, r);
  bwd_split_plan(M, K, N, &a.splits, &a.nks);
  if (a.splits > 1) {
    tn_launch<128, 128, 2, true>(a, st);
    launch_bwd_fixup(M, K, r, s, A, x, xq, sx, pdx, pu, a.splits, dx, partA, ge, st);
  } else if (bm == 64) {
    tn_launch<64, 64, 3, false>(a, st);
  } else if ((long)((M + 127) / 128) * ((K + 127) / 128) <= 256) {
    // one 128 x 128 block per compute unit or fewer (4-bit 1024 x 4096 x 4096,
    // 256 of them: 75 against 90 us; 512 of them: 165 against 160)
    tn_launch<128, 64, 2, false>(a, st);
  } else {
    tn_launch<128, 128, 2, false>(a, st);
  }
}

}  // namespace qlora
