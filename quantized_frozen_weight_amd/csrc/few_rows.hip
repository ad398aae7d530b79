// The layer with its epilogue for a few rows (serving: one token, or up to
// four at once), in one launch.
//
//   z[m, n] = sx[m] sw[n] (xq[m, :] . q[n, :]) + s (t B)[m, n] + bias[n]     (int8)
//   z[m, n] = sum_g sc[n, g] (x[m, g] . q[n, g]) + s (t B)[m, n] + bias[n]  (4-bit)
//   y = act(z) + residual,   t = x A
//
// (int8: the row quantizer and exact int32 sums of qlora_fwd, so the base
// product is bitwise the same; 4-bit: exact bf16 codes, each 128-wide group's
// float32 sum weighted by its scale in float32.)
//
// With so few rows the weight is all the traffic there is, and the call ends
// when its last byte has arrived: 16384 x 2048 int8 codes are 33.5 MB, 6.5 us
// at the 5.1 TB/s of a large copy. So a block of 16 waves puts its share of
// the weight in flight first (each lane 16 bytes of one output channel per
// load, up to kHold of them held in registers; what a longer share has left
// follows as the first are used), and does everything that the small operands
// need while those loads travel: the rows' abs-max and codes (every block
// quantizes the rows for itself, which costs less than a launch that would do
// it once) and t = x A. Then the codes go from registers straight into the
// matrix instructions: the 16 channels are the columns of a 16 x 16 block, the
// rows sit in the first rows of the other operand (read from LDS; the unused
// rows repeat the last one and their sums are dropped), and the waves' partial
// sums over k are added in LDS in wave order.
//
// A block owns 16 NG columns; its 16 waves are NG groups of 16 columns times
// 16 / NG spans of k. A compute unit holds one block, so NG is the smallest of
// 1, 2, 4 whose blocks all run at once (at least 2 where 32-column groups of z
// are saved); narrow blocks split k further, but a second round costs a whole
// one: 4 rows of 1024 -> 12288 take 8.6 us at 192 blocks of 64 columns, 13.8
// at 384 of 32. Below 4096 outputs some compute units have no block
// (16384 -> 2048: 128 blocks).
//
// Under a wide adapter over long rows (K R past kPreWords) A is the larger
// part of what a block would read (512 KB at 16384 x 8, beside 262 KB of
// codes), so a small launch before takes the abs-max and t in slices of 512 k
// and the blocks add the slices: 14.9 against 22.2 us for 16384 -> 2048 at
// rank 8.
//
// Measured (graph replay, bias and tanh gelu; the tiled product without them
// in brackets): one row of 2048 -> 16384 int8 8.6 us [13.9], 3.9 TB/s; 16384
// -> 2048 14.8 [30.7]; 1024 -> 1024 4.7 [9.7] (rank 8); 4096 -> 4096 4-bit 7.4
// [27.0]; float32 256 -> 256 4.0 [6.5] (rank 4). Four rows: 12.6 [14.0], 20.9
// [30.8], 7.9 [9.7], 9.9 [27.3], 6.7 [6.7]. What is left over the weight's 6.5
// us is the launch and the chain abs-max -> codes -> products -> sums, three
// barriers.
#include "epilogue.hpp"
#include "launch.hpp"

namespace qlora {

namespace {

constexpr int kWaves = 16, kThreads = 64 * kWaves;
constexpr int kHold = 8;                      // code loads a lane holds
constexpr int kFewCUs = 256;
constexpr long kPreWords = 32768;             // K R past which t has a launch of its own

struct FewArgs {
  int M, N, K;
  const void* x;            // [M, K]
  const int8_t* codes;      // [N, K], or packed [N, K / 2]
  const void* scales;       // float [N], or fp16 [N, K / 128]
  const float* A;           // [K, r]
  const float* B;           // [r, N], or [heads, r, hd]
  int hd, r;
  float s;
  void* y;                  // [M, N]
  float* t;                 // [M, r], or NULL
  int8_t* xq;               // x's row checkpoint, or NULL
  float* sx;
  FwdEpi epi;
  uint32_t* pre_max;        // PRE: [slices][MB], [slices][MB][R]
  float* pre_t;
  int slices;
};

// The eight 4-bit codes q of a word (two's complement nibbles) as bf16 values
// q / 16, exact: v_cvt_off_f32_i4 takes the low nibble of a byte in one
// operation, and the upper halves of two results are a bf16 pair. Pair i holds
// nibbles i and i + 4, so the other operand's eight values come in the order
// 0 4 1 5 2 6 3 7 (nibble_order). (Or-ing q + 8 into the last places of 128
// and taking 136 out again by a second product is 8 instead of 14 operations
// and 3 % faster over 1 to 4 rows, but rounds sums at 136 |x|, which drowns the
// other terms where an x far above them meets a zero code.)
__device__ __forceinline__ bf16x8 nibbles_exact(uint32_t w) {
  const uint32_t odd = w >> 4;
  u32x4 o;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t v = i & 1 ? odd : w;
    const float lo = __builtin_amdgcn_cvt_off_f32_i4((int)((v >> (8 * (i / 2))) & 0xffu));
    const float hi = __builtin_amdgcn_cvt_off_f32_i4((int)((v >> (8 * (i / 2) + 16)) & 0xffu));
    o[i] = __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302u);
  }
  return __builtin_bit_cast(bf16x8, o);
}

// The same codes as the tiled product takes them, bf16(q sc), pair i again
// nibbles i and i + 4. A wave whose sums come out non-finite takes its steps
// again with these: sums of x q / 16 pass the float range (from |x| = 2^122
// on) where those of x times the weight do not.
__device__ __forceinline__ bf16x8 nibbles_scaled(uint32_t w, float sc) {
  const uint32_t u = w ^ 0x88888888u;          // q + 8
  const float nsc = -8.f * sc;
  u32x4 o;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    o[i] = cvt_bf16x2(__builtin_fmaf((float)((u >> (4 * i)) & 15u), sc, nsc),
                      __builtin_fmaf((float)((u >> (4 * i + 16)) & 15u), sc, nsc));
  return __builtin_bit_cast(bf16x8, o);
}
__device__ __forceinline__ bool finite(float v) { return abs_bits(v) < 0x7f800000u; }

// eight bf16 values in the order 0 4 1 5 2 6 3 7
__device__ __forceinline__ u32x4 nibble_order(u32x4 v) {
  return u32x4{__builtin_amdgcn_perm(v[2], v[0], 0x05040100u), __builtin_amdgcn_perm(v[2], v[0], 0x07060302u),
               __builtin_amdgcn_perm(v[3], v[1], 0x05040100u), __builtin_amdgcn_perm(v[3], v[1], 0x07060302u)};
}

// acc[4 m + q] += x[m][k] A[k][j0 + q]
template <typename T, int R, int MB>
__device__ __forceinline__ void few_rank_step(const typename Elem<T>::type* x, const float* A, int k, int j0,
                                              int M, int K, int r, float (&acc)[4 * MB]) {
  float av[4];
  if (r == R) {
    const f32x4 v = *reinterpret_cast<const f32x4*>(A + (long)k * R + j0);
    av[0] = v.x; av[1] = v.y; av[2] = v.z; av[3] = v.w;
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q) av[q] = j0 + q < r ? A[(long)k * r + j0 + q] : 0.f;
  }
#pragma unroll
  for (int m = 0; m < MB; ++m) {
    const auto xe = x[(long)(m < M ? m : 0) * K + k];
    float xv;
    if constexpr (std::is_same<T, F32>::value) xv = xe;
    else xv = bf16_to_f32(xe);
#pragma unroll
    for (int q = 0; q < 4; ++q) acc[4 * m + q] = __builtin_fmaf(xv, av[q], acc[4 * m + q]);
  }
}

// The launch before, for long rows under a wide adapter (see launch_fwd_few):
// block b takes the 512 k from 512 b and leaves the rows' abs-max bits [b][MB]
// and sums of x A [b][MB][R].
constexpr int kSlice = 512;
constexpr int kFewMaxK = 32 * kSlice;         // 32 slices: one per lane of half a wave

template <typename T, int R, int MB>
__global__ __launch_bounds__(512) void fwd_few_pre_kernel(FewArgs a) {
  typedef typename Elem<T>::type E;
  constexpr int W = 8, JW = R / 4, KW = W / JW;
  __shared__ uint32_t red_max[MB][W];
  __shared__ float red_t[W][4 * MB];
  const int tid = threadIdx.x, lane = tid & 63, wid = wave_id();
  const int M = a.M, K = a.K, k0 = blockIdx.x * kSlice, k1 = K - k0 < kSlice ? K : k0 + kSlice;
  const E* x = static_cast<const E*>(a.x);
#pragma unroll
  for (int m = 0; m < MB; ++m) {
    uint32_t mx = 0;
    if (m < M && k0 + tid < k1) {
      const E xe = x[(long)m * K + k0 + tid];
      if constexpr (std::is_same<T, F32>::value) mx = abs_bits(xe);
      else mx = abs_bits(bf16_to_f32(xe));
    }
    mx = wave_max_u32(mx);
    if (lane == 0) red_max[m][wid] = mx;
  }
  float acc[4 * MB];
#pragma unroll
  for (int q = 0; q < 4 * MB; ++q) acc[q] = 0.f;
#pragma unroll
  for (int i = 0; i < kSlice / (64 * KW); ++i) {
    const int k = k0 + 64 * (wid / JW + KW * i) + lane;
    if (k < k1) few_rank_step<T, R, MB>(x, a.A, k, 4 * (wid % JW), M, K, a.r, acc);
  }
  const float tot = wave_sum_ranks<4 * MB>(acc);
  if ((lane & (64 / (4 * MB) - 1)) == 0) red_t[wid][rank_of_lane<4 * MB>(lane)] = tot;
  __syncthreads();
  if (tid < MB) {
    uint32_t mx = red_max[tid][0];
#pragma unroll
    for (int w = 1; w < W; ++w) mx = red_max[tid][w] > mx ? red_max[tid][w] : mx;
    a.pre_max[blockIdx.x * MB + tid] = mx;
  }
  if (tid < MB * R) {
    const int m = tid / R, j = tid % R;
    float v = red_t[j / 4][4 * m + j % 4];
#pragma unroll
    for (int w = 1; w < KW; ++w) v += red_t[w * JW + j / 4][4 * m + j % 4];
    a.pre_t[((long)blockIdx.x * MB + m) * R + j] = v;
  }
}

template <typename T, bool W4, int R, int NG, int MB, bool PRE>
__global__ __launch_bounds__(kThreads) void fwd_few_kernel(FewArgs a) {
  typedef typename Elem<T>::type E;
  constexpr int KS = kWaves / NG, BN = 16 * NG;
  constexpr int STEP = W4 ? 128 : 64;          // k per load: 16 bytes of codes a lane, 4 lanes a channel
  extern __shared__ __attribute__((aligned(16))) int8_t xs[];   // [M][K] int8, or [M][K] bf16
  __shared__ f32x4 part[kWaves][16];           // [wave][column] of rows 0..3 (int8: int32 bits)
  __shared__ uint32_t red_max[MB][kWaves];
  __shared__ float red_t[kWaves][4 * MB];
  __shared__ float ts[MB][R];

  const int tid = threadIdx.x, lane = tid & 63, wid = wave_id();
  const int M = a.M, N = a.N, K = a.K, r = a.r;
  const int g = wid / KS, ks = wid % KS;
  const int n0 = blockIdx.x * BN;
  const int S = (K + STEP - 1) / STEP, span = (S + KS - 1) / KS;
  const int s0 = ks * span < S ? ks * span : S, cnt = s0 + span < S ? span : S - s0;

  // ---- the weight: cnt loads of this lane's channel from step s0 ----
  const int n = n0 + 16 * g + (lane & 15), nc = n < N ? n : N - 1;
  const long rowb = W4 ? K / 2 : K;
  const int8_t* cb = a.codes + (long)nc * rowb + 16 * (lane >> 4);
  auto load = [&](int s) {
    // a chunk past the row (int8, K % 64 != 0) reads the row's last one; the
    // rows' codes there are zero in LDS
    const long o = (long)s * 64;
    const long oc = 16 * (lane >> 4) + o < rowb ? o : rowb - 16 - 16 * (lane >> 4);
    return *reinterpret_cast<const u32x4*>(cb + oc);
  };
  const _Float16* scb = W4 ? static_cast<const _Float16*>(a.scales) + (long)nc * S : nullptr;
  u32x4 hold[kHold];
  _Float16 hsc[kHold];
#pragma unroll
  for (int i = 0; i < kHold; ++i)
    if (i < cnt) {
      hold[i] = load(s0 + i);
      if constexpr (W4) hsc[i] = scb[s0 + i];
    }

  // ---- the epilogue's operands: thread v < BN M owns output (v / BN, n0 + v % BN) ----
  const int em = tid / BN, en = n0 + tid % BN;
  const bool mine = em < M && en < N;
  float eb[R], esw = 0.f, ebias = 0.f, eres = 0.f;
  if (mine) {
#pragma unroll
    for (int j = 0; j < R; ++j) eb[j] = j < r ? a.B[head_index(j, en, r, a.hd)] : 0.f;
    if constexpr (!W4) esw = static_cast<const float*>(a.scales)[en];
    if (a.epi.bias != nullptr) ebias = a.epi.bias[en];
    if (a.epi.res != nullptr) {
      const E v = static_cast<const E*>(a.epi.res)[(long)em * N + en];
      if constexpr (std::is_same<T, F32>::value) eres = v;
      else eres = bf16_to_f32(v);
    }
  }

  // ---- the rows: abs-max ----
  const E* x = static_cast<const E*>(a.x);
  const int nchunk = K / 8;
  if (!PRE && (!W4 || a.xq != nullptr)) {
#pragma unroll
    for (int m = 0; m < MB; ++m) {
      uint32_t mx = 0;
      if (m < M)
        for (int c = tid; c < nchunk; c += kThreads) {
          float v[8];
          load8(x + (long)m * K + 8 * c, v);
#pragma unroll
          for (int e = 0; e < 8; ++e) { const uint32_t b = abs_bits(v[e]); mx = b > mx ? b : mx; }
        }
      mx = wave_max_u32(mx);
      if (lane == 0) red_max[m][wid] = mx;
    }
  }
  // ---- t = x A: wave (kw, jw) takes ranks [4 jw, 4 jw + 4) of every KW-th
  // run of 64 k, a lane one k of a run (PRE: summed by the launch before) ----
  constexpr int JW = R / 4, KW = kWaves / JW;
  if constexpr (!PRE) {
    float acc[4 * MB];
#pragma unroll
    for (int q = 0; q < 4 * MB; ++q) acc[q] = 0.f;
    const int j0 = 4 * (wid % JW);
#pragma unroll 4
    for (int k = 64 * (wid / JW) + lane; k < K; k += 64 * KW) few_rank_step<T, R, MB>(x, a.A, k, j0, M, K, r, acc);
    const float tot = wave_sum_ranks<4 * MB>(acc);
    if ((lane & (64 / (4 * MB) - 1)) == 0) red_t[wid][rank_of_lane<4 * MB>(lane)] = tot;
  }
  __syncthreads();                             // the waves' maxima and sums

  // ---- the rows into LDS: codes, or bf16 as it is ----
  QuantParams qp[MB];
#pragma unroll
  for (int m = 0; m < MB; ++m) {
    qp[m] = QuantParams{0.f, 0.f, false};
    if (!W4 || a.xq != nullptr) {
      uint32_t mx;
      if constexpr (PRE) {
        mx = wave_max_u32(lane < a.slices ? a.pre_max[lane * MB + m] : 0u);
      } else {
        mx = red_max[m][0];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) mx = red_max[m][w] > mx ? red_max[m][w] : mx;
      }
      qp[m] = absmax_params(mx, 127.f);
    }
  }
  const int kpad = (K + STEP - 1) / STEP * STEP;     // LDS row length: whole steps
  for (int c = tid; c < kpad / 8; c += kThreads) {
#pragma unroll
    for (int m = 0; m < MB; ++m) {
      if (m >= M) break;
      uint32_t lo = 0, hi = 0;
      float v[8];
      if (c < nchunk) load8(x + (long)m * K + 8 * c, v);
      if (c < nchunk && qp[m].live) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          lo |= (uint32_t)(quant_code(v[e], qp[m].inv, 127.f) & 0xff) << (8 * e);
          hi |= (uint32_t)(quant_code(v[e + 4], qp[m].inv, 127.f) & 0xff) << (8 * e);
        }
      }
      if (blockIdx.x == 0 && a.xq != nullptr && c < nchunk)
        *reinterpret_cast<u32x2*>(a.xq + (long)m * K + 8 * c) = u32x2{lo, hi};
      if constexpr (W4)
        *reinterpret_cast<u32x4*>(xs + ((long)m * kpad + 8 * c) * 2) =
            nibble_order(*reinterpret_cast<const u32x4*>(reinterpret_cast<const uint16_t*>(x) + (long)m * K + 8 * c));
      else
        *reinterpret_cast<u32x2*>(xs + (long)m * kpad + 8 * c) = u32x2{lo, hi};
    }
  }
  if constexpr (PRE) {
    // 32 lanes per (m, j), one slice each (at most 32 of them)
    for (int o = tid / 32; o < MB * R; o += kThreads / 32) {
      float v = (tid & 31) < a.slices ? a.pre_t[(long)(tid & 31) * MB * R + o] : 0.f;
#pragma unroll
      for (int d = 16; d >= 1; d >>= 1) v += __shfl_xor(v, d);
      if ((tid & 31) == 0) {
        const int m = o / R, j = o % R;
        ts[m][j] = j < r ? v : 0.f;            // (an infinite x times the padded ranks' zeros is NaN)
        if (blockIdx.x == 0 && a.t != nullptr && m < M && j < r) a.t[(long)m * r + j] = v;
      }
    }
  } else if (tid < MB * R) {
    const int m = tid / R, j = tid % R;
    float v = red_t[j / 4][4 * m + j % 4];
#pragma unroll
    for (int w = 1; w < KW; ++w) v += red_t[w * JW + j / 4][4 * m + j % 4];
    ts[m][j] = j < r ? v : 0.f;
    if (blockIdx.x == 0 && a.t != nullptr && m < M && j < r) a.t[(long)m * r + j] = v;
  }
  if (blockIdx.x == 0 && a.sx != nullptr && tid < M) {
#pragma unroll
    for (int m = 0; m < MB; ++m)
      if (tid == m) a.sx[m] = qp[m].scale;
  }
  __syncthreads();                             // rows and t

  // ---- the product ----
  const int xm = (lane & 15) < M ? (lane & 15) : M - 1;
  i32x4 acci = i32x4{0, 0, 0, 0};
  f32x4 accf = f32x4{0.f, 0.f, 0.f, 0.f};
  auto step = [&](int s, const u32x4& w, _Float16 sc) {
    if constexpr (W4) {
      const int8_t* xp = xs + ((long)xm * kpad + 128 * s + 32 * (lane >> 4)) * 2;
      f32x4 p = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int q = 0; q < 4; ++q)
        p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(*reinterpret_cast<const bf16x8*>(xp + 16 * q),
                                                    nibbles_exact(w[q]), p, 0, 0, 0);
#pragma unroll
      for (int i = 0; i < 4; ++i) accf[i] = __builtin_fmaf(16.f * (float)sc, p[i], accf[i]);
    } else {
      const i32x4 xv = *reinterpret_cast<const i32x4*>(xs + (long)xm * kpad + 64 * s + 16 * (lane >> 4));
      acci = __builtin_amdgcn_mfma_i32_16x16x64_i8(xv, __builtin_bit_cast(i32x4, w), acci, 0, 0, 0);
    }
  };
  for (int ib = 0; ib < cnt; ib += kHold) {
#pragma unroll
    for (int i = 0; i < kHold; ++i) {
      if (ib + i < cnt) {                      // wave-uniform
        step(s0 + ib + i, hold[i], W4 ? hsc[i] : (_Float16)0.f);
        if (ib + i + kHold < cnt) {
          hold[i] = load(s0 + ib + i + kHold);
          if constexpr (W4) hsc[i] = scb[s0 + ib + i + kHold];
        }
      }
    }
  }
  if constexpr (W4) {
    bool all = true;
#pragma unroll
    for (int i = 0; i < 4; ++i) all &= finite(accf[i]);
    if (__builtin_amdgcn_ballot_w64(!all) != 0) {
      f32x4 again = f32x4{0.f, 0.f, 0.f, 0.f};
      for (int s = s0; s < s0 + cnt; ++s) {
        const u32x4 w = load(s);
        const float sc = (float)scb[s];
        const int8_t* xp = xs + ((long)xm * kpad + 128 * s + 32 * (lane >> 4)) * 2;
#pragma unroll
        for (int q = 0; q < 4; ++q)
          again = __builtin_amdgcn_mfma_f32_16x16x32_bf16(*reinterpret_cast<const bf16x8*>(xp + 16 * q),
                                                          nibbles_scaled(w[q], sc), again, 0, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) accf[i] = finite(accf[i]) ? accf[i] : again[i];   // other rows as they were
    }
  }
  // rows 0..3 of the 16 x 16 block: lanes 0..15
  if (lane < 16) part[wid][lane] = W4 ? accf : __builtin_bit_cast(f32x4, acci);
  __syncthreads();

  // ---- the epilogue, one output per thread ----
  // (all lanes of a wave stay: the group maximum reads its neighbours)
  float z = 0.f;
  if (mine) {
    const int p0 = (tid % BN) / 16 * KS, col = tid & 15;
    float base;
    if constexpr (W4) {
      base = part[p0][col][em];
#pragma unroll
      for (int w = 1; w < KS; ++w) base += part[p0 + w][col][em];
    } else {
      int sum = 0;
#pragma unroll
      for (int w = 0; w < KS; ++w) sum += __float_as_int(part[p0 + w][col][em]);
      float sxm = qp[0].scale;
#pragma unroll
      for (int m = 1; m < MB; ++m) sxm = em == m ? qp[m].scale : sxm;
      base = (float)sum * (sxm * esw);
    }
    float low = 0.f;
#pragma unroll
    for (int j = 0; j < R; ++j) low = __builtin_fmaf(ts[em][j], eb[j], low);
    z = __builtin_fmaf(a.s, low, base);
    if (a.epi.bias != nullptr) z += ebias;
    if (a.epi.z != nullptr) store_out(static_cast<E*>(a.epi.z) + (long)em * N + en, z);
  }
  if constexpr (NG > 1) {
    if (a.epi.zc != nullptr && tid < BN * MB) {        // whole waves: BN MB is a multiple of 32
      uint32_t mx = mine ? abs_bits(z) : 0u;
#pragma unroll
      for (int d = 16; d >= 1; d >>= 1) {
        const uint32_t o = __shfl_xor(mx, d);
        mx = o > mx ? o : mx;
      }
      if (mine) {
        const int b = group_byte(mx);
        a.epi.zc[(long)em * N + en] = group_code(z, b);
        if (en % kGroup == 0) a.epi.zs[(long)em * a.epi.zg + en / kGroup] = (uint8_t)b;
      }
    }
  }
  if (mine) {
    float v[1] = {z};
    act_apply<std::is_same<T, F32>::value>(a.epi.act, v);
    if (a.epi.res != nullptr) v[0] += eres;
    store_out(static_cast<E*>(a.y) + (long)em * N + en, v[0]);
  }
}

template <typename T, bool W4, int R, int NG, int MB>
void few_rows(FewArgs a, hipStream_t st) {
  const int step = W4 ? 128 : 64;
  const size_t lds = (size_t)a.M * ((a.K + step - 1) / step * step) * (W4 ? 2 : 1);
  const unsigned grid = (unsigned)((a.N + 16 * NG - 1) / (16 * NG));
  if ((long)a.K * R > kPreWords) {
    // the slices' maxima and sums, 4 MB (R + 1) bytes each, in the M K bytes of
    // scratch: K is past 2048 here, so a slice stands for 409 k at least, and
    // 68 (one row) or 272 (MB = 4, two rows or more) is below 409 M
    a.slices = (a.K + kSlice - 1) / kSlice;
    a.pre_max = reinterpret_cast<uint32_t*>(a.pre_t + (size_t)a.slices * MB * R);
    fwd_few_pre_kernel<T, R, MB><<<(unsigned)a.slices, 512, 0, st>>>(a);
    fwd_few_kernel<T, W4, R, NG, MB, true><<<grid, kThreads, lds, st>>>(a);
  } else {
    fwd_few_kernel<T, W4, R, NG, MB, false><<<grid, kThreads, lds, st>>>(a);
  }
}

template <typename T, bool W4, int R, int NG>
void few_launch(const FewArgs& a, hipStream_t st) {
  if (a.M == 1) few_rows<T, W4, R, NG, 1>(a, st);
  else few_rows<T, W4, R, NG, 4>(a, st);
}

template <typename T, bool W4, int R>
void few_groups(const FewArgs& a, hipStream_t st) {
  if (a.N > 32 * kFewCUs) few_launch<T, W4, R, 4>(a, st);
  else if (a.N > 16 * kFewCUs || a.epi.zc != nullptr) few_launch<T, W4, R, 2>(a, st);
  else few_launch<T, W4, R, 1>(a, st);
}

template <typename T, bool W4>
void few_ranks(const FewArgs& a, hipStream_t st) {
  if (a.r <= 4) few_groups<T, W4, 4>(a, st);
  else if (a.r <= 8) few_groups<T, W4, 8>(a, st);
  else few_groups<T, W4, 16>(a, st);
}

}  // namespace

// Up to four rows, int8 and 4-bit weights, ranks up to 16, and rows whose bf16
// form fits in LDS four times. Against the tiled product with the same
// epilogue (at five rows): one round of blocks is faster in every case
// measured (int8 4 rows of 256 -> 4096 7.1 against 7.7 us, 4096 -> 4096 r 16
// 13.4 against 30.5); past 16384 outputs one row and 4-bit rows still are, or
// come within a tenth, but 2 to 4 int8 rows are not (2048 -> 32768 24 against
// 19), save where the tiled product's row pass is slow, at ranks past 8 over
// long rows (8192 -> 32768 r 16 59 against 78).
bool fwd_few_takes(int fmt, int M, int N, int K, int r) {
  if (!(fmt == 0 || fmt == 1) || M > 4 || r > 16 || K > kFewMaxK) return false;
  return fmt == 1 || M == 1 || N <= 64 * kFewCUs || (r > 8 && K >= 4096);
}

void launch_fwd_few(int dtype, int fmt, int M, int N, int K, const void* x, const void* codes,
                    const void* scales, const float* A, const float* B, int hd, int r, float s,
                    const FwdEpi& epi, void* y, float* t, int8_t* xq, float* sx, float* scratch,
                    hipStream_t st) {
  FewArgs a{};
  a.M = M; a.N = N; a.K = K; a.x = x; a.codes = static_cast<const int8_t*>(codes); a.scales = scales;
  a.A = A; a.B = B; a.hd = hd; a.r = r; a.s = s; a.y = y; a.t = t; a.xq = xq; a.sx = sx; a.epi = epi;
  a.pre_t = scratch;
  if (fmt == 1) few_ranks<BF16, true>(a, st);
  else if (dtype == 0) few_ranks<F32, false>(a, st);
  else few_ranks<BF16, false>(a, st);
}

}  // namespace qlora
