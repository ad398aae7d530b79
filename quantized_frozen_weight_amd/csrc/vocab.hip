// The vocabulary layer at the model's input: the lookup of tokens and its
// gradient (formulas: include/qlora.h).
//
// Lookup. Memory-bound: a row reads K bytes of codes and writes K outputs. A
// thread owns 8 features (4 from rank 9 on, whose rows of A would not fit in
// its registers) for all rows of its block, so A is read once per block; a
// block's tokens, their scales and their columns of B (r scattered floats a
// token) are gathered side by side into LDS first, then the rows' codes stream
// through with four rows in flight.
//
// Gradient. One launch runs four kinds of blocks beside each other, so that the
// serial sort hides behind the products:
//   u      16 rows a block, the four waves a quarter of the features each:
//          u = dy A on v_mfma_f32_16x16x4_f32 (float32 operands: nothing is
//          rounded), the waves added through LDS in order;
//   dA     a wave owns 128 features and a range of rows: dA^T = Bg^T dy with
//          Bg[m] = B[:, token(m)], the same instruction; its sums go to the
//          workspace per block of rows;
//   sort   1024 threads order 2048 tokens by (token, row) in LDS, one slice a
//          block (a bitonic network: 66 steps, no memory traffic);
//   fill   dB cleared (not where the call accumulates).
// A second launch merges the slices where there is more than one (a row's place
// is its place in its slice plus, by binary search, the rows of the others that
// come before it) and adds dA's partial sums; a third adds the rows of u that
// share a token, in order, into dB: short runs by one thread per rank, runs
// past 16 rows by the whole block that holds their first row. No atomics.
#include "abi.hpp"
#include "common.hpp"
#include "vocab.hpp"

namespace qlora {

namespace {

// ---- lookup ---------------------------------------------------------------------
struct EmbedArgs {
  int M, K, N, r;
  const uint8_t* codes;
  const void* scales;
  const float* A;
  const float* B;
  float s, scale;
  Ids ids;
  void* x;
};

constexpr int kEmbedRows = 16;       // rows per block

// The value of code e of a unit's dword(s): int8, or 4-bit (nibble e).
template <bool W4, int F>
__device__ __forceinline__ void unit_codes(const uint32_t (&w)[2], float (&v)[F]) {
#pragma unroll
  for (int e = 0; e < F; ++e) {
    if constexpr (W4) v[e] = (float)((int)(w[0] << (28 - 4 * e)) >> 28);
    else v[e] = (float)(int8_t)(w[e / 4] >> (8 * (e % 4)));
  }
}

// R: the rank rounded up (0: no adapter); F features per thread.
template <typename T, bool W4, int R, int F>
__global__ __launch_bounds__(256) void embed_kernel(EmbedArgs a) {
  typedef typename Elem<T>::type E;
  __shared__ int tok[kEmbedRows];
  __shared__ float bs[kEmbedRows][R > 0 ? R : 1];
  const int tid = threadIdx.x, K = a.K;
  const int units = K / F, wide = units < 256 ? units : 256;      // units a pass covers of a row
  const int lanes = 256 / wide;                                   // rows side by side
  const int m0 = blockIdx.x * kEmbedRows;
  const int unit = (int)blockIdx.y * wide + tid % wide, lane = tid / wide;
  const int rows = a.M - m0 < kEmbedRows ? a.M - m0 : kEmbedRows;
  if (tid < kEmbedRows) tok[tid] = tid < rows ? entry_of(a.ids, m0 + tid) : -1;
  __syncthreads();
  if constexpr (R > 0) {
    for (int e = tid; e < kEmbedRows * R; e += 256) {
      const int row = e / R, j = e % R, t = tok[row];
      bs[row][j] = t >= 0 && j < a.r ? a.B[(long)j * a.N + t] : 0.f;
    }
    __syncthreads();
  }
  if (lane >= lanes || unit >= units) return;
  const int k = unit * F;
  float ar[F][R > 0 ? R : 1];
  if constexpr (R > 0) {
#pragma unroll
    for (int f = 0; f < F; ++f)
#pragma unroll
      for (int j = 0; j < R; ++j) ar[f][j] = a.A[(long)(k + f) * a.r + (j < a.r ? j : 0)];
  }
  for (int i0 = lane; i0 < rows; i0 += 4 * lanes) {
    uint32_t w[4][2];
    float sc[4];
    int t[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int row = i0 + u * lanes;
      t[u] = row < rows ? tok[row] : -1;
      const long at = t[u] >= 0 ? t[u] : 0;
      w[u][1] = 0u;
      if constexpr (W4) {
        const uint8_t* p = a.codes + at * (K / 2) + k / 2;
        w[u][0] = F == 8 ? *reinterpret_cast<const uint32_t*>(p) : (uint32_t)*reinterpret_cast<const uint16_t*>(p);
        sc[u] = (float)static_cast<const _Float16*>(a.scales)[at * (K / 128) + k / 128];
      } else {
        const uint8_t* p = a.codes + at * K + k;
        w[u][0] = *reinterpret_cast<const uint32_t*>(p);
        if constexpr (F == 8) w[u][1] = *reinterpret_cast<const uint32_t*>(p + 4);
        sc[u] = static_cast<const float*>(a.scales)[at];
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int row = i0 + u * lanes;
      if (row >= rows) break;
      float v[F];
      unit_codes<W4, F>(w[u], v);
#pragma unroll
      for (int f = 0; f < F; ++f) {
        float y = v[f] * sc[u];
        if constexpr (R > 0) {
          float low = 0.f;
#pragma unroll
          for (int j = 0; j < R; ++j) low = __builtin_fmaf(ar[f][j], bs[row][j], low);
          y = __builtin_fmaf(a.s, low, y);
        }
        v[f] = t[u] >= 0 ? a.scale * y : 0.f;
      }
      E* out = static_cast<E*>(a.x) + (long)(m0 + row) * K + k;
      if constexpr (sizeof(E) == 4) {
#pragma unroll
        for (int f = 0; f < F; f += 4) *reinterpret_cast<f32x4*>(out + f) = f32x4{v[f], v[f + 1], v[f + 2], v[f + 3]};
      } else if constexpr (F == 8) {
        *reinterpret_cast<u32x4*>(out) = u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                               pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
      } else {
        *reinterpret_cast<u32x2*>(out) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
      }
    }
  }
}

template <typename T, bool W4>
void embed_dispatch(const EmbedArgs& a, hipStream_t st) {
  const auto grid = [&](int F) {
    const int units = a.K / F, wide = units < 256 ? units : 256;
    return dim3((unsigned)((a.M + kEmbedRows - 1) / kEmbedRows), (unsigned)((units + wide - 1) / wide));
  };
  if (a.r == 0) embed_kernel<T, W4, 0, 8><<<grid(8), 256, 0, st>>>(a);
  else if (a.r <= 4) embed_kernel<T, W4, 4, 8><<<grid(8), 256, 0, st>>>(a);
  else if (a.r <= 8) embed_kernel<T, W4, 8, 8><<<grid(8), 256, 0, st>>>(a);
  else if (a.r <= 16) embed_kernel<T, W4, 16, 4><<<grid(4), 256, 0, st>>>(a);
  else embed_kernel<T, W4, 32, 4><<<grid(4), 256, 0, st>>>(a);
}

// ---- gradient ---------------------------------------------------------------------
constexpr int kSlice = 2048;         // tokens one block sorts
constexpr int kURows = 16;           // rows of a u block
constexpr int kFeat = 128;           // features of a dA wave
constexpr int kFill = 16384;         // floats a fill block clears
constexpr int kSegRows = 256;        // sorted rows of a block of the last launch
constexpr int kShort = 16;           // rows of a run that one thread adds

struct EmbedBwdArgs {
  int M, K, N, r;
  const float* A;
  const float* B;
  float c;                           // scale s
  Ids ids;
  const void* dy;
  float* u;                          // [M, r], without c
  float* pA;                         // [row blocks, r, K]
  uint64_t* slices;                  // (token << 32 | row) of every slice, sorted
  int* tok;                          // sorted: token (N for none)
  int* row;                          // and row
  float* dA;                         // [K, r]
  float* dB;                         // [r, N]
  int accumulate;
  int nslices, nsort, nu, nda, nfill, rows_a, blocks_a, feats;
};

// Eight consecutive values of dy as float32, zero where !ok.
template <typename E>
__device__ __forceinline__ void dy8(const E* p, bool ok, float (&v)[8]) {
  load8(p, v);
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = ok ? v[e] : 0.f;
}

// u of 16 rows, ranks in RB blocks of 16. red: 4 x 16 x 16 RB floats.
template <typename T, int RB>
__device__ __forceinline__ void u_block(const EmbedBwdArgs& a, int b, float* red) {
  typedef typename Elem<T>::type E;
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, l = lane & 15, q = lane >> 4;
  const E* dy = static_cast<const E*>(a.dy);
  const int m = b * kURows + l, mc = m < a.M ? m : a.M - 1;
  f32x4 acc[RB];
#pragma unroll
  for (int j = 0; j < RB; ++j) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
  // A operand: row l, features k0 + 8 q + e at step e; B operand: those
  // features of A, rank l (features past K are zero in the A operand)
  for (int k0 = 32 * w; k0 < a.K; k0 += 128) {
    const int k = k0 + 8 * q, kc = k < a.K ? k : 0;
    float v[8];
    dy8(dy + (long)mc * a.K + kc, k < a.K, v);
#pragma unroll
    for (int j = 0; j < RB; ++j) {
      const int rank = 16 * j + l;
      const float* ap = a.A + (long)kc * a.r + (rank < a.r ? rank : 0);
      float av[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) av[e] = k < a.K ? ap[(long)e * a.r] : 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[j] = __builtin_amdgcn_mfma_f32_16x16x4f32(v[e], av[e], acc[j], 0, 0, 0);
    }
  }
#pragma unroll
  for (int j = 0; j < RB; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) red[((w * RB + j) * 16 + 4 * q + i) * 16 + l] = acc[j][i];
  __syncthreads();
  for (int e = tid; e < 256 * RB; e += 256) {
    const int j = e >> 8, mm = (e >> 4) & 15, rank = 16 * j + (e & 15);
    float sum = red[e];
#pragma unroll
    for (int k = 1; k < 4; ++k) sum += red[k * 256 * RB + e];
    if (rank < a.r && b * kURows + mm < a.M) a.u[(long)(b * kURows + mm) * a.r + rank] = sum;
  }
}

// dA partial sums of 4 x 128 features (a wave each) over rows_a rows.
template <typename T, int RB>
__device__ __forceinline__ void da_block(const EmbedBwdArgs& a, int b) {
  typedef typename Elem<T>::type E;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, l = lane & 15, q = lane >> 4;
  const E* dy = static_cast<const E*>(a.dy);
  const int rb = b / ((a.feats + 3) / 4), f = b % ((a.feats + 3) / 4) * 4 + w;
  const int k = f * kFeat + 8 * l, kc = k < a.K ? k : 0;
  const int m0 = rb * a.rows_a, m1 = m0 + a.rows_a < a.M ? m0 + a.rows_a : a.M;
  f32x4 acc[8][RB];
#pragma unroll
  for (int e = 0; e < 8; ++e)
#pragma unroll
    for (int j = 0; j < RB; ++j) acc[e][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  // A operand: rank l of row m0 + 4 g + q; B operand: features k + e of that
  // row at step e (k: 8 per lane of 16)
  for (int g0 = m0; g0 < m1; g0 += 16) {
    float v[4][8], bg[4][RB];
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int m = g0 + 4 * g + q, mc = m < m1 ? m : m0;
      const int t = m < m1 ? entry_of(a.ids, mc) : -1;
      dy8(dy + (long)mc * a.K + kc, t >= 0, v[g]);
#pragma unroll
      for (int j = 0; j < RB; ++j) {
        const int rank = 16 * j + l;
        bg[g][j] = t >= 0 && rank < a.r ? a.B[(long)rank * a.N + t] : 0.f;
      }
    }
#pragma unroll
    for (int g = 0; g < 4; ++g)
#pragma unroll
      for (int e = 0; e < 8; ++e)
#pragma unroll
        for (int j = 0; j < RB; ++j)
          acc[e][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(bg[g][j], v[g][e], acc[e][j], 0, 0, 0);
  }
  if (k >= a.K) return;
#pragma unroll
  for (int j = 0; j < RB; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int rank = 16 * j + 4 * q + i;
      if (rank < a.r) {
        float* out = a.pA + ((long)rb * a.r + rank) * a.K + k;
        *reinterpret_cast<f32x4*>(out) = f32x4{acc[0][j][i], acc[1][j][i], acc[2][j][i], acc[3][j][i]};
        *reinterpret_cast<f32x4*>(out + 4) = f32x4{acc[4][j][i], acc[5][j][i], acc[6][j][i], acc[7][j][i]};
      }
    }
}

// One slice of the tokens sorted by (token, row); 256 threads, 2048 keys in LDS.
__device__ __forceinline__ void sort_block(const EmbedBwdArgs& a, int b, uint64_t* key) {
  const int tid = threadIdx.x;
  for (int i = tid; i < kSlice; i += 256) {
    const int m = b * kSlice + i;
    const int t = m < a.M ? entry_of(a.ids, m) : -1;
    // rows without a token behind all others, what is past the last row behind them
    key[i] = ((uint64_t)(uint32_t)(m < a.M ? (t >= 0 ? t : a.N) : 0x7fffffff) << 32) | (uint32_t)m;
  }
  for (int size = 2; size <= kSlice; size <<= 1)
    for (int d = size >> 1; d >= 1; d >>= 1) {
      __syncthreads();
      for (int p = tid; p < kSlice / 2; p += 256) {
        const int i = 2 * p - (p & (d - 1)), j = i + d;       // i without bit d, and its partner
        const uint64_t x = key[i], y = key[j];
        if ((x > y) == ((i & size) == 0)) { key[i] = y; key[j] = x; }
      }
    }
  __syncthreads();
  for (int i = tid; i < kSlice; i += 256) {
    const int m = b * kSlice + i;
    if (m >= a.M) continue;
    if (a.nslices == 1) {
      a.tok[m] = (int)(key[i] >> 32);
      a.row[m] = (int)(uint32_t)key[i];
    } else {
      a.slices[m] = key[i];
    }
  }
}

// Blocks in this order: sort, u, dA, fill (the slow ones first).
template <typename T, int RB>
__global__ __launch_bounds__(256) void embed_bwd_kernel(EmbedBwdArgs a) {
  __shared__ __attribute__((aligned(16))) char lds[kSlice * 8];
  static_assert(4 * 256 * RB * 4 <= kSlice * 8, "the u blocks' sums fit");
  int b = blockIdx.x;
  if (b < a.nsort) { sort_block(a, b, reinterpret_cast<uint64_t*>(lds)); return; }
  b -= a.nsort;
  if (b < a.nu) { u_block<T, RB>(a, b, reinterpret_cast<float*>(lds)); return; }
  b -= a.nu;
  if (b < a.nda) { da_block<T, RB>(a, b); return; }
  b -= a.nda;
  const long n = (long)a.r * a.N, e1 = (long)(b + 1) * kFill < n ? (long)(b + 1) * kFill : n;
  for (long e = (long)b * kFill + 4 * threadIdx.x; e < e1; e += 1024)     // N % 16 == 0
    *reinterpret_cast<f32x4*>(a.dB + e) = f32x4{0.f, 0.f, 0.f, 0.f};
}

// Rows of slice `sl` (its n sorted keys) before `key`.
__device__ __forceinline__ int before(const uint64_t* p, int n, uint64_t key) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (p[mid] < key) lo = mid + 1;
    else hi = mid;
  }
  return lo;
}

// dA's partial sums added in order; element e = j K + k.
__device__ __forceinline__ void da_sum(const EmbedBwdArgs& a, long e) {
  if (e >= (long)a.r * a.K) return;
  const long stride = (long)a.r * a.K;
  const float* p = a.pA + e;
  float sum = 0.f;
  for (int i = 0; i < a.blocks_a; i += 8) {
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = p[(i + k < a.blocks_a ? i + k : i) * stride];
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (i + k < a.blocks_a) sum += v[k];
  }
  const long k = e % a.K, j = e / a.K;
  float* out = a.dA + k * a.r + j;
  *out = a.accumulate ? *out + a.c * sum : a.c * sum;
}

// Blocks [0, nmerge): the slices merged; the others: dA.
__global__ __launch_bounds__(256) void embed_merge_kernel(EmbedBwdArgs a, int nmerge) {
  const int b = blockIdx.x;
  if (b >= nmerge) {
    da_sum(a, (long)(b - nmerge) * 256 + threadIdx.x);
    return;
  }
  const int m = b * 256 + threadIdx.x;
  if (m >= a.M) return;
  const uint64_t key = a.slices[m];
  const int own = m / kSlice;
  int at = m - own * kSlice;
  for (int s = 0; s < a.nslices; ++s) {
    const int n = a.M - s * kSlice < kSlice ? a.M - s * kSlice : kSlice;
    if (s != own) at += before(a.slices + (long)s * kSlice, n, key);      // (keys differ by their rows)
  }
  a.tok[at] = (int)(key >> 32);
  a.row[at] = (int)(uint32_t)key;
}

// dB: blocks [0, nseg) take 256 sorted rows each and every run of one token
// that begins among them, to its end wherever that is; the others (one slice
// only) dA.
__global__ __launch_bounds__(256) void embed_runs_kernel(EmbedBwdArgs a, int nseg) {
  __shared__ int tok[kSegRows + 1], row[kSegRows], head[kSegRows + 1], heads[4], valid[4];
  __shared__ float red[256];
  const int tid = threadIdx.x, w = tid >> 6, b = blockIdx.x, r = a.r;
  if (b >= nseg) {
    da_sum(a, (long)(b - nseg) * 256 + tid);
    return;
  }
  const int i0 = b * kSegRows, i = i0 + tid;
  const int mine = i < a.M ? a.tok[i] : a.N;                   // N: no token (behind all others)
  const int prev = i > 0 && i < a.M ? a.tok[i - 1] : -1;
  tok[tid] = mine;
  row[tid] = i < a.M ? a.row[i] : 0;
  if (tid == 0) tok[kSegRows] = i0 + kSegRows < a.M ? a.tok[i0 + kSegRows] : a.N;
  // the runs that begin here, in order: head[0 .. nhead), and their end
  const bool first = mine < a.N && mine != prev;
  const uint64_t mask = __builtin_amdgcn_ballot_w64(first), ok = __builtin_amdgcn_ballot_w64(mine < a.N);
  if ((tid & 63) == 0) {
    heads[w] = __builtin_popcountll(mask);
    valid[w] = __builtin_popcountll(ok);
  }
  __syncthreads();
  int at = 0;
  for (int k = 0; k < w; ++k) at += heads[k];
  at += __builtin_popcountll(mask & ((1ull << (tid & 63)) - 1));
  const int nhead = heads[0] + heads[1] + heads[2] + heads[3];
  if (first) head[at] = tid;
  if (tid == 0) head[nhead] = valid[0] + valid[1] + valid[2] + valid[3];
  __syncthreads();

  auto put = [&](int j, int t, float sum) {
    float* out = a.dB + (long)j * a.N + t;
    *out = a.accumulate ? *out + a.c * sum : a.c * sum;
  };
  // short runs that end here: a thread per run and rank, rows in order
  for (int e = tid; e < nhead * r; e += 256) {
    const int k = e / r, j = e - k * r, h = head[k], t = tok[h], len = head[k + 1] - h;
    if (len > kShort || (h + len == kSegRows && tok[kSegRows] == t)) continue;
    float sum = 0.f;
    for (int q = 0; q < len; ++q) sum += a.u[(long)row[h + q] * r + j];
    put(j, t, sum);
  }
  // the others: of `lanes` groups of threads (one thread per rank, rounded up
  // to a power of two), group g adds every lanes-th row, then the groups in order
  int rp = 1;
  while (rp < r) rp <<= 1;
  const int lanes = 256 / rp, j = tid % rp, g = tid / rp;
  for (int k = 0; k < nhead; ++k) {                            // block-uniform
    const int h = head[k], t = tok[h], len = head[k + 1] - h;
    const bool goes_on = h + len == kSegRows && tok[kSegRows] == t;
    if (len <= kShort && !goes_on) continue;
    int s1 = i0 + h + len;
    if (goes_on) {                                             // to where the token ends
      int hi = a.M;
      while (s1 < hi) {
        const int mid = (s1 + hi) >> 1;
        if (a.tok[mid] <= t) s1 = mid + 1;
        else hi = mid;
      }
    }
    float sum = 0.f;
    for (int q = i0 + h + g; q < s1; q += 4 * lanes) {
      float v[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int qq = q + c * lanes < s1 ? q + c * lanes : q;
        v[c] = a.u[(long)a.row[qq] * r + (j < r ? j : 0)];
      }
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (q + c * lanes < s1) sum += v[c];
    }
    __syncthreads();
    red[tid] = sum;
    __syncthreads();
    if (tid < r) {
      float total = red[tid];
      for (int q = 1; q < lanes; ++q) total += red[q * rp + tid];
      put(tid, t, total);
    }
  }
}

struct EmbedBwdLayout {
  size_t u, pA, slices, tok, row, total;
};
// Rows a dA wave takes: about 2048 waves in all, whole groups of 16 rows, so
// that the partial sums (4 r K bytes each) stay few.
int da_rows(int M, int K) {
  const long waves = ((long)K + kFeat - 1) / kFeat;
  const long want = ((long)M * waves / 2048 + 15) / 16 * 16;
  return (int)(want < 32 ? 32 : want > 1024 ? 1024 : want);
}
EmbedBwdLayout embed_bwd_layout(int M, int K, int r) {
  EmbedBwdLayout w{};
  size_t off = 0;
  const int rows = da_rows(M, K);
  w.u = off; off = align_up(off + (size_t)M * r * 4);
  w.pA = off; off = align_up(off + (size_t)((M + rows - 1) / rows) * r * K * 4);
  w.slices = off; off = align_up(off + (M > kSlice ? (size_t)M * 8 : 0));
  w.tok = off; off = align_up(off + (size_t)M * 4);
  w.row = off; off = align_up(off + (size_t)M * 4);
  w.total = off;
  return w;
}

template <typename T>
void embed_bwd_first(const EmbedBwdArgs& a, hipStream_t st) {
  const dim3 grid((unsigned)(a.nsort + a.nu + a.nda + a.nfill));
  if (a.r <= 16) embed_bwd_kernel<T, 1><<<grid, 256, 0, st>>>(a);
  else embed_bwd_kernel<T, 2><<<grid, 256, 0, st>>>(a);
}

}  // namespace

void launch_embed(const VocabLayer& L, int M, int dtype, Ids ids, float scale, void* x, hipStream_t st) {
  EmbedArgs a{M, L.K, L.N, L.r, static_cast<const uint8_t*>(L.codes), L.scales, L.A, L.B, L.s, scale, ids, x};
  if (dtype == 0) embed_dispatch<F32, false>(a, st);
  else if (L.fmt == 0) embed_dispatch<BF16, false>(a, st);
  else embed_dispatch<BF16, true>(a, st);
}

size_t embed_bwd_bytes(int M, int K, int r) { return embed_bwd_layout(M, K, r).total; }

void launch_embed_bwd(const VocabLayer& L, int M, int dtype, Ids ids, float scale, const void* dy,
                      bool accumulate, float* dA, float* dB, void* ws, hipStream_t st) {
  const EmbedBwdLayout w = embed_bwd_layout(M, L.K, L.r);
  EmbedBwdArgs a{};
  a.M = M; a.K = L.K; a.N = L.N; a.r = L.r; a.A = L.A; a.B = L.B; a.c = scale * L.s; a.ids = ids; a.dy = dy;
  a.u = reinterpret_cast<float*>(at(ws, w.u));
  a.pA = reinterpret_cast<float*>(at(ws, w.pA));
  a.slices = reinterpret_cast<uint64_t*>(at(ws, w.slices));
  a.tok = reinterpret_cast<int*>(at(ws, w.tok));
  a.row = reinterpret_cast<int*>(at(ws, w.row));
  a.dA = dA; a.dB = dB; a.accumulate = accumulate;
  a.nslices = a.nsort = (M + kSlice - 1) / kSlice;
  a.nu = (M + kURows - 1) / kURows;
  a.rows_a = da_rows(M, L.K);
  a.blocks_a = (M + a.rows_a - 1) / a.rows_a;
  a.feats = (L.K + kFeat - 1) / kFeat;
  a.nda = a.blocks_a * ((a.feats + 3) / 4);
  a.nfill = accumulate ? 0 : (int)(((long)L.r * L.N + kFill - 1) / kFill);
  if (dtype == 0) embed_bwd_first<F32>(a, st);
  else embed_bwd_first<BF16>(a, st);
  const int nsum = (int)(((long)L.r * L.K + 255) / 256), nseg = (M + kSegRows - 1) / kSegRows;
  if (a.nslices > 1) {
    const int nmerge = (M + 255) / 256;
    embed_merge_kernel<<<dim3((unsigned)(nmerge + nsum)), 256, 0, st>>>(a, nmerge);
    embed_runs_kernel<<<dim3((unsigned)nseg), 256, 0, st>>>(a, nseg);
  } else {
    embed_runs_kernel<<<dim3((unsigned)(nseg + nsum)), 256, 0, st>>>(a, nseg);
  }
}

}  // namespace qlora
