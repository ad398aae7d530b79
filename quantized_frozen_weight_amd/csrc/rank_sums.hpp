// Sums over rows of rank-r outer products, out[j][k] = sum_m P[m][j] Q[m][k], on
// v_mfma_f32_16x16x4_f32 (float32 operands: nothing is rounded), for the
// adapter's gradients of the vocabulary layer. A wave owns 128 columns of Q and
// a range of rows; its partial sums go to [row block][r][C] and are added in
// order by rank_sum_total.
#pragma once
#include "common.hpp"

namespace qlora {

constexpr int kRankCols = 128;       // columns of a wave

// Rows a wave takes: about 2048 waves in all, whole groups of 16, so that the
// partial sums (4 r C bytes each) stay few.
inline int rank_sum_rows(int M, int C) {
  const long waves = ((long)C + kRankCols - 1) / kRankCols;
  const long want = ((long)M * waves / 2048 + 15) / 16 * 16;
  return (int)(want < 32 ? 32 : want > 1024 ? 1024 : want);
}
inline size_t rank_sum_floats(int M, int C, int r) {
  const int rows = rank_sum_rows(M, C);
  return (size_t)((M + rows - 1) / rows) * r * C;
}
// Blocks of 256 threads for all of it (four waves: four column ranges).
inline int rank_sum_blocks(int M, int C) {
  const int rows = rank_sum_rows(M, C), cols = (C + kRankCols - 1) / kRankCols;
  return (M + rows - 1) / rows * ((cols + 3) / 4);
}

// Rows whose loads are under way together, and the LDS that their P takes.
template <typename T> constexpr int rank_sum_chunk() { return sizeof(typename Elem<T>::type) == 2 ? 64 : 32; }
template <int RB> constexpr int rank_sum_lds() { return 64 * (16 * RB + 2) * 4; }

// Block b of rank_sum_blocks, all 256 threads. live(m): whether row m counts
// (what else stands in it is not used); get(m, j): P[m][j]. RB blocks of 16 ranks;
// lds: rank_sum_lds<RB>() bytes.
template <typename T, int RB, typename Live, typename Get>
__device__ __forceinline__ void rank_sum_block(int b, int M, int C, int r, int rows,
                                               const typename Elem<T>::type* Q, float* part, char* lds, Live live,
                                               Get get) {
  constexpr int CH = rank_sum_chunk<T>(), NG = CH / 16, PP = 16 * RB + 1;
  constexpr int QU = sizeof(typename Elem<T>::type) / 2;         // 16-byte pieces of 8 columns
  int* ok = reinterpret_cast<int*>(lds);
  float* ps = reinterpret_cast<float*>(lds) + 64;
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, l = lane & 15, q = lane >> 4;
  const int groups = ((C + kRankCols - 1) / kRankCols + 3) / 4;
  const int rb = b / groups, f = b % groups * 4 + w;
  const int k = f * kRankCols + 8 * l, kc = k < C ? k : 0;
  const int m0 = rb * rows, m1 = m0 + rows < M ? m0 + rows : M;
  f32x4 acc[8][RB];
#pragma unroll
  for (int e = 0; e < 8; ++e)
#pragma unroll
    for (int j = 0; j < RB; ++j) acc[e][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  // A operand: rank l of row c0 + 16 g + 4 h + q; B operand: columns k + e of that
  // row at step e
  for (int c0 = m0; c0 < m1; c0 += CH) {
    u32x4 raw[NG][4][QU];
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const int m = c0 + 16 * g + 4 * h + q;
        const u32x4* p = reinterpret_cast<const u32x4*>(Q + (long)(m < m1 ? m : m0) * C + kc);
#pragma unroll
        for (int u = 0; u < QU; ++u) raw[g][h][u] = p[u];
      }
    __syncthreads();                                   // the last chunk's P is read
    if (tid < CH) ok[tid] = c0 + tid < m1 && live(c0 + tid);
    __syncthreads();
    for (int e = tid; e < CH * 16 * RB; e += 256) {
      const int m = e / (16 * RB), j = e % (16 * RB);
      ps[m * PP + j] = ok[m] && j < r ? get(c0 + m, j) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const int m = 16 * g + 4 * h + q;
        const bool on = ok[m];
        float v[8];
        if constexpr (QU == 1) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            v[2 * e] = __uint_as_float(raw[g][h][0][e] << 16);
            v[2 * e + 1] = __uint_as_float(raw[g][h][0][e] & 0xffff0000u);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(raw[g][h][e / 4][e % 4]);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = on ? v[e] : 0.f;
#pragma unroll
        for (int j = 0; j < RB; ++j) {
          const float p = ps[m * PP + 16 * j + l];
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[e][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(p, v[e], acc[e][j], 0, 0, 0);
        }
      }
  }
  if (k >= C) return;
#pragma unroll
  for (int j = 0; j < RB; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int rank = 16 * j + 4 * q + i;
      if (rank < r) {
        float* out = part + ((long)rb * r + rank) * C + k;
        *reinterpret_cast<f32x4*>(out) = f32x4{acc[0][j][i], acc[1][j][i], acc[2][j][i], acc[3][j][i]};
        *reinterpret_cast<f32x4*>(out + 4) = f32x4{acc[4][j][i], acc[5][j][i], acc[6][j][i], acc[7][j][i]};
      }
    }
}

// Element e = j C + k of the partial sums, added in order.
__device__ __forceinline__ float rank_sum_total(const float* part, int blocks, long stride, long e) {
  constexpr int NB = 32;                               // loads in flight
  const float* p = part + e;
  float sum = 0.f;
  for (int i = 0; i < blocks; i += NB) {
    float v[NB];
#pragma unroll
    for (int k = 0; k < NB; ++k) v[k] = p[(i + k < blocks ? i + k : i) * stride];
#pragma unroll
    for (int k = 0; k < NB; ++k)
      if (i + k < blocks) sum += v[k];
  }
  return sum;
}

}  // namespace qlora
