// 8-bit activation checkpoints (written and read back) and the gradient of an
// activation on its own. All of it is memory-bound: a thread owns one unit of
// 8 consecutive columns of a row (16 bytes of bf16, 8 of codes), and eight
// waves per SIMD cover the latency (two and four units a thread, their loads
// together in flight, are no faster: 512 x 16384 bf16 written in 5.6, 5.8 and
// 6.2 us, read back in 4.9, 5.3 and 5.4).
//
// The group form is described in epilogue.hpp; the row form is the forward's
// own activation quantizer, and its launches (rows.hip) write most of it here.
//
// ("Introduce QLoRA-like technique": activations quantized per row under the
// int8 kernel; keras-llm-light README, "Block-wise gradient checkpointing":
// block inputs are kept and blocks recomputed or differentiated from them.)
#include "epilogue.hpp"
#include "launch.hpp"

namespace qlora {

namespace {

// Units of a row padded to whole groups, so that the four lanes of a quad
// always hold one group: unit u is columns [8 (u % upr), + 8) of row u / upr.
template <typename T>
__global__ __launch_bounds__(256) void ckpt_write_groups_kernel(
    const typename Elem<T>::type* __restrict__ x, int M, int C, int8_t* __restrict__ codes,
    uint8_t* __restrict__ scales) {
  const int zg = group_count(C);
  const uint32_t upr = 4u * zg, n = (uint32_t)M * upr, u = blockIdx.x * 256u + threadIdx.x;
  const uint32_t row = u / upr, col = 8u * (u - row * upr);
  const bool ok = u < n && col < (uint32_t)C;
  const long at = ok ? (long)row * C + col : 0;
  float v[8];
  load8(x + at, v);
  uint32_t m = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) { const uint32_t b = abs_bits(v[e]); m = b > m ? b : m; }
  const int b = group_byte(quad_max_u32(ok ? m : 0u));
  if (ok) {
    *reinterpret_cast<u32x2*>(codes + at) = group_codes(v, b);
    if (col % kGroup == 0) scales[(long)row * zg + col / kGroup] = (uint8_t)b;
  }
}

// The abs-max of a row or group may round up to a product past the largest
// finite value (127 (FLT_MAX / 127); groups from 127 / 64 2^127 on, whose code
// 64 stands for 2^128): such a product reads back as that value, so that
// finite activations stay finite. (The comparisons keep a NaN. Only scales past
// 2^120 can need them: made for every value they cost 0.6 of 5.1 us.)
template <typename T, bool GROUPS>
__global__ __launch_bounds__(256) void ckpt_read_kernel(
    const int8_t* __restrict__ codes, const void* __restrict__ scales, int M, int C,
    typename Elem<T>::type* __restrict__ x) {
  const uint32_t upr = (uint32_t)C / 8u, n = (uint32_t)M * upr, u = blockIdx.x * 256u + threadIdx.x;
  if (u >= n) return;
  const uint32_t row = u / upr, col = 8u * (u - row * upr);
  const u32x2 c = *reinterpret_cast<const u32x2*>(codes + 8L * u);
  float s;
  if constexpr (GROUPS) s = group_scale(static_cast<const uint8_t*>(scales)[(long)row * group_count(C) + col / kGroup]);
  else s = static_cast<const float*>(scales)[row];
  float v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = (float)(int8_t)(c[e >> 2] >> (8 * (e & 3))) * s;
  if (s > 0x1p120f) {
    const float top = __uint_as_float(std::is_same<T, F32>::value ? 0x7f7fffffu : 0x7f7f0000u);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = v[e] > top ? top : v[e] < -top ? -top : v[e];
  }
  store8(x + 8L * u, v);
}

// The row form, a block per row, which reads the row twice, the second time
// from the caches. rows.hip has a wave or half a block per row and holds the
// row in registers up to 16384 entries: better for many rows (bf16, 2048 x
// 16384 18.9 against 19.6 us here, 8192 x 4112 20 against 33), while up to two
// rows per compute unit of more than 4096 entries are quicker here (512 x
// 16384 5.9 against 7.5, 512 x 4112 3.8 against 4.5, one of 16384 3.3 against
// 5.6), and longer ones in any case (64 x 65536 7.4 against 61). The same codes
// and scale: abs-max over the row's bits, then the shared rounding.
bool ckpt_block_per_row(int M, int C) { return C > 16384 || (C > 4096 && M <= 512); }

template <typename T>
__global__ __launch_bounds__(1024) void ckpt_write_rows_kernel(
    const typename Elem<T>::type* __restrict__ x, int C, int8_t* __restrict__ codes,
    float* __restrict__ scales) {
  __shared__ uint32_t red[16];
  const int tid = threadIdx.x;
  const long row = blockIdx.x;
  x += row * C;
  codes += row * C;
  uint32_t m = 0;
#pragma unroll 4
  for (int c = tid; c < C / 8; c += 1024) {
    float v[8];
    load8(x + 8L * c, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) { const uint32_t b = abs_bits(v[e]); m = b > m ? b : m; }
  }
  m = wave_max_u32(m);
  if ((tid & 63) == 0) red[tid >> 6] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 16; ++w) m = red[w] > m ? red[w] : m;
  const QuantParams q = absmax_params(m, 127.f);
  if (tid == 0) scales[row] = q.scale;
#pragma unroll 4
  for (int c = tid; c < C / 8; c += 1024) {
    float v[8];
    load8(x + 8L * c, v);
    uint32_t lo = 0, hi = 0;
    if (q.live) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        lo |= (uint32_t)(quant_code(v[e], q.inv, 127.f) & 0xff) << (8 * e);
        hi |= (uint32_t)(quant_code(v[e + 4], q.inv, 127.f) & 0xff) << (8 * e);
      }
    }
    *reinterpret_cast<u32x2*>(codes + 8L * c) = u32x2{lo, hi};
  }
}

// Row sums of codes, one wave per row (exact in float32: |sum| <= 127 K < 2^24
// up to the longest K that qlora_fwd_ckpt takes, 132096).
__global__ __launch_bounds__(256) void code_sums_kernel(const int8_t* __restrict__ codes, int M,
                                                        int K, float* __restrict__ asum) {
  const int lane = threadIdx.x & 63;
  for (int row = blockIdx.x * 4 + (threadIdx.x >> 6); row < M; row += 4 * (int)gridDim.x) {
    int sum = 0;
    for (int k = 16 * lane; k < K; k += 1024) {
      const i32x4 c = *reinterpret_cast<const i32x4*>(codes + (long)row * K + k);
#pragma unroll
      for (int i = 0; i < 4; ++i) sum = __builtin_amdgcn_sdot4(c[i], 0x01010101, sum, false);
    }
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) sum += __shfl_xor(sum, d);
    if (lane == 0) asum[row] = (float)sum;
  }
}

// ---- dz = dy act'(z), dbias = column sums -----------------------------------
// A block owns 256 columns (32 lanes of 8) and a span of rows, LANES rows at a
// time; a thread keeps the float32 sums of its 8 columns over its rows. The
// row lanes are added in order through LDS, and (more than one span) a second
// launch adds the spans in order. No atomics.
// Up to 128 rows one span of 32 row lanes does: every thread then has one
// group of four rows' loads in flight, and there is no second launch (77 rows
// of 1040 float32: one span of 8 lanes took 12 us). Past that 8 lanes, and a
// thread takes a row at a time: the loads of other waves cover one wave's
// arithmetic better than its own loads of more rows do, which cost registers
// and so waves (gelu, 4096 x 2304: 16.7 us at one row, 18.1 at two, 18.8 at
// four; 8192 x 4096: 35.5, 38.4, 43). The activation's slope is as much work
// as the traffic: 4096 x 2304 bf16 with gelu moves 47 MB (9.3 us at the 5.1
// TB/s of a large copy) and does about 25 vector instructions and two
// transcendental ones per value (8 us).
constexpr int kActCols = 256;
constexpr int act_units(int lanes) { return lanes == 32 ? 4 : 1; }   // rows a thread loads at once

inline int col_blocks(int C) { return C / kActCols + (C % kActCols != 0); }

// Rows per span and row lanes.
void act_bwd_plan(int M, int C, int* spans, int* rows, int* lanes) {
  if (M <= 32 * act_units(32)) {
    // (a launch takes fewer than 2^32 threads: rows past 2^29, at most three
    // of them, get blocks of 8 lanes)
    *spans = 1;
    *rows = M;
    *lanes = col_blocks(C) < 1 << 21 ? 32 : 8;
    return;
  }
  // 4096 blocks where there are that many rows, but 16 rows a span at least,
  // and 32 rather than more than 128 spans: the second launch reads them all
  // (1024 x 1024 6.9 us at 16 rows, 8.4 at 32; 4096 x 768 10.8 and 10.2)
  *lanes = 8;
  int want = 4096 / col_blocks(C);
  if (want < 1) want = 1;
  int r = (M + want - 1) / want;
  const int least = M > 4096 ? 32 : M > 2048 ? (M + 127) / 128 : 16;
  if (r < least) r = least;
  r = (r + 7) / 8 * 8;
  *rows = r;
  *spans = (M + r - 1) / r;
}

template <typename T, bool SUMS, int LANES>
__global__ __launch_bounds__(32 * LANES) void act_bwd_kernel(const typename Elem<T>::type* dy, int M, int C,
                                                      GradEpi ge, typename Elem<T>::type* dz,
                                                      float* __restrict__ out, int rows) {
  constexpr int UNITS = act_units(LANES);
  __shared__ float red[SUMS ? LANES : 1][kActCols + 8];
  const int tid = threadIdx.x, cl = tid & 31, rl = tid >> 5;
  const uint32_t col = blockIdx.x * (uint32_t)kActCols + 8u * cl;   // (may pass 2^31 - 1 in the last block)
  const bool okc = col < (uint32_t)C;
  const uint32_t colc = okc ? col : 0u;
  const int m0 = blockIdx.y * rows, m1 = M - m0 < rows ? M : m0 + rows;
  float sum[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) sum[e] = 0.f;
  for (int mb = m0 + rl; mb < m1; mb += LANES * UNITS) {
    float v[UNITS][8], z[UNITS][8];
    // every load of the group from clamped addresses before the first use
#pragma unroll
    for (int i = 0; i < UNITS; ++i) {
      const int m = mb + LANES * i < m1 ? mb + LANES * i : mb;
      const long at = (long)m * C + colc;
      load8(dy + at, v[i]);
      if (ge.act.kind != 0) {
        if (ge.zc != nullptr)
          group_values(*reinterpret_cast<const u32x2*>(ge.zc + at), ge.zs[(long)m * ge.zg + colc / kGroup], z[i]);
        else
          load8(static_cast<const typename Elem<T>::type*>(ge.z) + at, z[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < UNITS; ++i) {
      const int m = mb + LANES * i;
      if (m < m1) {
        act_slope_mul<std::is_same<T, F32>::value>(ge.act, z[i], v[i]);
        if (dz != nullptr && okc) store8(dz + (long)m * C + col, v[i]);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[e] += v[i][e];
      }
    }
  }
  if constexpr (SUMS) {
#pragma unroll
    for (int e = 0; e < 8; ++e) red[rl][8 * cl + e] = sum[e];
    __syncthreads();
    if (tid >= kActCols) return;
    const uint32_t c = blockIdx.x * (uint32_t)kActCols + tid;
    float s = red[0][tid];
#pragma unroll
    for (int l = 1; l < LANES; ++l) s += red[l][tid];
    if (c < (uint32_t)C) out[(long)blockIdx.y * C + c] = s;
  }
}

// dbias[c] = the spans' sums: 64 columns per block, wave w the spans w, w + 4,
// ... in order, then the four waves in order.
__global__ __launch_bounds__(256) void act_bwd_sum_kernel(const float* __restrict__ part, int spans,
                                                          int C, float* __restrict__ dbias) {
  __shared__ float red[4][64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int c = blockIdx.x * 64 + lane, cc = c < C ? c : 0;
  float s = 0.f;
#pragma unroll 8
  for (int k = w; k < spans; k += 4) s += part[(long)k * C + cc];
  red[w][lane] = s;
  __syncthreads();
  if (w == 0 && c < C) dbias[c] = ((red[0][lane] + red[1][lane]) + red[2][lane]) + red[3][lane];
}

inline unsigned unit_blocks(long units) { return (unsigned)((units + 255) / 256); }

template <typename T>
void act_bwd_launch(int M, int C, const void* dy, const GradEpi& ge, void* dz, float* dbias,
                    float* partial, hipStream_t st) {
  typedef typename Elem<T>::type E;
  int spans, rows, lanes;
  act_bwd_plan(M, C, &spans, &rows, &lanes);
  const dim3 grid((unsigned)col_blocks(C), (unsigned)spans);
  const E* d = static_cast<const E*>(dy);
  E* o = static_cast<E*>(dz);
  if (dbias == nullptr) {
    if (lanes == 32) act_bwd_kernel<T, false, 32><<<grid, 1024, 0, st>>>(d, M, C, ge, o, nullptr, rows);
    else act_bwd_kernel<T, false, 8><<<grid, 256, 0, st>>>(d, M, C, ge, o, nullptr, rows);
    return;
  }
  float* sums = spans == 1 ? dbias : partial;
  if (lanes == 32) act_bwd_kernel<T, true, 32><<<grid, 1024, 0, st>>>(d, M, C, ge, o, sums, rows);
  else act_bwd_kernel<T, true, 8><<<grid, 256, 0, st>>>(d, M, C, ge, o, sums, rows);
  if (spans > 1)
    act_bwd_sum_kernel<<<(unsigned)((C + 63) / 64), 256, 0, st>>>(partial, spans, C, dbias);
}

}  // namespace

void launch_ckpt_write_rows(int dtype, const void* x, int M, int C, int8_t* codes, float* scales,
                            hipStream_t st) {
  if (!ckpt_block_per_row(M, C))
    launch_rowquant(dtype, x, M, C, nullptr, 1, codes, scales, nullptr, st);
  else if (dtype == 0)
    ckpt_write_rows_kernel<F32><<<(unsigned)M, 1024, 0, st>>>(static_cast<const float*>(x), C, codes, scales);
  else
    ckpt_write_rows_kernel<BF16><<<(unsigned)M, 1024, 0, st>>>(static_cast<const uint16_t*>(x), C, codes, scales);
}

void launch_ckpt_write_groups(int dtype, const void* x, int M, int C, int8_t* codes,
                              uint8_t* scales, hipStream_t st) {
  const unsigned nb = unit_blocks(4L * M * group_count(C));
  if (dtype == 0)
    ckpt_write_groups_kernel<F32><<<nb, 256, 0, st>>>(static_cast<const float*>(x), M, C, codes, scales);
  else
    ckpt_write_groups_kernel<BF16><<<nb, 256, 0, st>>>(static_cast<const uint16_t*>(x), M, C, codes, scales);
}

void launch_ckpt_read(int dtype, int cfmt, const int8_t* codes, const void* scales, int M, int C,
                      void* x, hipStream_t st) {
  const unsigned nb = unit_blocks((long)M * (C / 8));
  float* xf = static_cast<float*>(x);
  uint16_t* xb = static_cast<uint16_t*>(x);
  if (cfmt == 0) {
    if (dtype == 0) ckpt_read_kernel<F32, false><<<nb, 256, 0, st>>>(codes, scales, M, C, xf);
    else ckpt_read_kernel<BF16, false><<<nb, 256, 0, st>>>(codes, scales, M, C, xb);
  } else {
    if (dtype == 0) ckpt_read_kernel<F32, true><<<nb, 256, 0, st>>>(codes, scales, M, C, xf);
    else ckpt_read_kernel<BF16, true><<<nb, 256, 0, st>>>(codes, scales, M, C, xb);
  }
}

void launch_code_sums(const int8_t* codes, int M, int K, float* asum, hipStream_t st) {
  const int nb = M / 4 + (M % 4 != 0);
  code_sums_kernel<<<(unsigned)(nb < 1 << 16 ? nb : 1 << 16), 256, 0, st>>>(codes, M, K, asum);
}

size_t act_bwd_floats(int M, int C) {
  int spans, rows, lanes;
  act_bwd_plan(M, C, &spans, &rows, &lanes);
  return spans > 1 ? (size_t)spans * (size_t)C : 0;
}

void launch_act_bwd(int dtype, int M, int C, const void* dy, const GradEpi& ge, void* dz,
                    float* dbias, float* partial, hipStream_t st) {
  if (dtype == 0) act_bwd_launch<F32>(M, C, dy, ge, dz, dbias, partial, st);
  else act_bwd_launch<BF16>(M, C, dy, ge, dz, dbias, partial, st);
}

}  // namespace qlora
