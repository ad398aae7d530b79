// The vocabulary layer at the model's input: the lookup of tokens and its
// gradient (formulas: include/qlora.h).
//
// Lookup. Memory-bound: a row reads K bytes of codes and writes K outputs. A wave
// takes 64 features of up to 64 rows: its lanes' codes (16 a lane, the quarters of
// a row side by side) are all under way while the block gathers the tokens'
// columns of B (r scattered floats each) into LDS, and the adapter's part is
// formed on v_mfma_f32_16x16x4_f32 in the layout of the codes, with A's rows in
// registers (a lane that read its own features' rows of A for vector products
// touched 64 lines an instruction, and took 37 us for 8192 x 2048 at rank 8). That
// case takes 17.2 us now, 50.8 MB, 2.9 TB/s: tokens, codes and stores wait for each
// other, 62 % of the waves' time.
//
// Gradient. One launch runs four kinds of blocks beside each other:
//   place  the tokens sorted by (token, row): a row's place is the number of rows
//          of its slice of 8192 that come before it, counted by comparing it with
//          all of them (2 instructions a pair; 8192 rows: 67 million pairs, 3.4 us
//          of the chip), the tokens in LDS, 32 rows a block.
//          No pass over memory, no rounds that wait for each other;
//   u      16 rows a block, the four waves a quarter of the features each:
//          u = dy A on v_mfma_f32_16x16x4_f32, the waves added through LDS;
//   dA     dy^T B[:, token] by rank_sums.hpp;
//   fill   dB cleared (not where the call accumulates).
// A second launch adds the rows of u that share a token, in order, into dB: a
// thread holds one sorted row, a wave adds runs by six steps of a segmented sum,
// a run that goes on takes the next waves' first runs, and one that leaves the
// block is finished by all of its threads; other blocks of the launch add dA's
// partial sums. (More than one slice: a launch between the two merges them: a
// row's place is its place in its slice plus, by binary search, the rows of the
// other slices that come before it.) No atomics.
// 8192 x 2048, 256000 entries, rank 8: 29 + 8 us (the first launch's kinds alone: place
// 12, u 14, dA 17, fill 3.6); its bytes are 8.3 at a copy's rate.
#include "abi.hpp"
#include "bwd_common.hpp"
#include "rank_sums.hpp"
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

// R: the rank rounded up (0: no adapter); NG groups of 16 rows a block. A wave
// takes 64 features, lane (l, q) the 16 of quarter q for row l of every group.
template <typename T, bool W4, int R, int NG>
__global__ __launch_bounds__(256) void embed_kernel(EmbedArgs a) {
  typedef typename Elem<T>::type E;
  constexpr int RA = R > 0 ? R : 4, KC = RA / 4, RP = RA + 1;     // RP: pitch of a row of bs
  __shared__ int tok[16 * NG];
  __shared__ float bs[16 * NG * RP];
  const int tid = threadIdx.x, lane = tid & 63, l = lane & 15, q = lane >> 4, K = a.K;
  const int m0 = blockIdx.x * (16 * NG), d0 = ((int)blockIdx.y * 4 + (tid >> 6)) * 64;
  if (tid < 16 * NG) tok[tid] = m0 + tid < a.M ? entry_of(a.ids, m0 + tid) : -1;
  __syncthreads();
  const int k = d0 + 16 * q, kc0 = k < K ? k : 0;
  u32x4 w[NG];
  float sc[NG];
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    const int t = tok[16 * g + l];
    const long at = t >= 0 ? t : 0;
    if constexpr (W4) {
      const u32x2 v = *reinterpret_cast<const u32x2*>(a.codes + at * (K / 2) + kc0 / 2);
      w[g] = u32x4{v.x, v.y, 0u, 0u};
      sc[g] = (float)static_cast<const _Float16*>(a.scales)[at * (K / 128) + kc0 / 128];
    } else {
      w[g] = *reinterpret_cast<const u32x4*>(a.codes + at * K + kc0);
      sc[g] = static_cast<const float*>(a.scales)[at];
    }
  }
  // A operand of column block b: row 4 q' + i of it is feature 16 q' + 4 b + i, so
  // that the four blocks of a lane are its 16 features in order
  float ar[4][KC];
  if constexpr (R > 0) {
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const int d = d0 + 16 * (l >> 2) + 4 * b + (l & 3);
#pragma unroll
      for (int c = 0; c < KC; ++c) {
        const int j = 4 * c + q;
        const float v = a.A[(long)(d < K ? d : 0) * a.r + (j < a.r ? j : 0)];
        ar[b][c] = d < K && j < a.r ? v : 0.f;
      }
    }
    for (int e = tid; e < 16 * NG * R; e += 256) {
      const int j = e / (16 * NG), row = e % (16 * NG), t = tok[row];
      bs[row * RP + j] = t >= 0 && j < a.r ? a.B[(long)j * a.N + t] : 0.f;
    }
    __syncthreads();
  }
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    f32x4 low[4];
    if constexpr (R > 0) {
#pragma unroll
      for (int b = 0; b < 4; ++b) low[b] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < KC; ++c) {
        const float bv = bs[(16 * g + l) * RP + 4 * c + q];
#pragma unroll
        for (int b = 0; b < 4; ++b) low[b] = __builtin_amdgcn_mfma_f32_16x16x4f32(ar[b][c], bv, low[b], 0, 0, 0);
      }
    }
    const int m = m0 + 16 * g + l;
    if (m >= a.M || k >= K) continue;
    const bool live = tok[16 * g + l] >= 0;
    float v[16];
#pragma unroll
    for (int f = 0; f < 16; ++f) {
      const float code = W4 ? (float)((int)(w[g][f / 8] << (28 - 4 * (f % 8))) >> 28) : (float)(int8_t)(w[g][f / 4] >> (8 * (f % 4)));
      float y = code * sc[g];
      if constexpr (R > 0) y = __builtin_fmaf(a.s, low[f / 4][f % 4], y);
      v[f] = live ? a.scale * y : 0.f;
    }
    E* out = static_cast<E*>(a.x) + (long)m * K + k;
    if constexpr (sizeof(E) == 4) {
#pragma unroll
      for (int f = 0; f < 16; f += 4) *reinterpret_cast<f32x4*>(out + f) = f32x4{v[f], v[f + 1], v[f + 2], v[f + 3]};
    } else {
#pragma unroll
      for (int f = 0; f < 16; f += 8)
        *reinterpret_cast<u32x4*>(out + f) = u32x4{pk_bf16(v[f], v[f + 1]), pk_bf16(v[f + 2], v[f + 3]),
                                                   pk_bf16(v[f + 4], v[f + 5]), pk_bf16(v[f + 6], v[f + 7])};
    }
  }
}

// Rows a block takes: 64 where that leaves two blocks a compute unit, so that A
// and B are gathered seldom; else 16, for the latency.
template <typename T, bool W4, int R>
void embed_rows(const EmbedArgs& a, hipStream_t st) {
  const unsigned cols = (unsigned)((a.K + 255) / 256);
  if ((long)((a.M + 63) / 64) * cols >= 512)
    embed_kernel<T, W4, R, 4><<<dim3((unsigned)((a.M + 63) / 64), cols), 256, 0, st>>>(a);
  else
    embed_kernel<T, W4, R, 1><<<dim3((unsigned)((a.M + 15) / 16), cols), 256, 0, st>>>(a);
}

template <typename T, bool W4>
void embed_dispatch(const EmbedArgs& a, hipStream_t st) {
  if (a.r == 0) embed_rows<T, W4, 0>(a, st);
  else if (a.r <= 4) embed_rows<T, W4, 4>(a, st);
  else if (a.r <= 8) embed_rows<T, W4, 8>(a, st);
  else if (a.r <= 16) embed_rows<T, W4, 16>(a, st);
  else embed_rows<T, W4, 32>(a, st);
}

// ---- gradient ---------------------------------------------------------------------
constexpr int kSlice = 8192;         // rows sorted together
constexpr int kPlaceRows = 32;       // rows of a place block
constexpr int kURows = 16;           // rows of a u block
constexpr int kFill = 16384;         // floats a fill block clears
constexpr int kSegRows = 256;        // sorted rows of a block of the last launch

struct EmbedBwdArgs {
  int M, K, N, r;
  const float* A;
  const float* B;
  float c;                           // scale s
  Ids ids;
  const void* dy;
  float* u;                          // [M, up], without c; up: r rounded up to 4, 8, 16, 32
  int up;
  float* pA;                         // partial sums of dA
  uint64_t* slices;                  // (token << 32 | row) of every slice, sorted
  int* tok;                          // sorted: token (N for none)
  int* row;                          // and row
  float* dA;                         // [K, r]
  float* dB;                         // [r, N]
  int accumulate;
  int nslices, nplace, nu, nda, rows_a, blocks_a;
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
  constexpr int KU = 4;                                  // steps of 32 features under way together
  for (int k0 = 32 * w; k0 < a.K; k0 += 128 * KU) {
    float v[KU][8], av[KU][RB][8];
#pragma unroll
    for (int s = 0; s < KU; ++s) {
      const int k = k0 + 128 * s + 8 * q, kc = k < a.K ? k : 0;
      dy8(dy + (long)mc * a.K + kc, k < a.K, v[s]);
#pragma unroll
      for (int j = 0; j < RB; ++j) {
        const int rank = 16 * j + l;
        const float* ap = a.A + (long)kc * a.r + (rank < a.r ? rank : 0);
#pragma unroll
        for (int e = 0; e < 8; ++e) av[s][j][e] = k < a.K && rank < a.r ? ap[(long)e * a.r] : 0.f;
      }
    }
#pragma unroll
    for (int s = 0; s < KU; ++s)
#pragma unroll
      for (int j = 0; j < RB; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e)
          acc[j] = __builtin_amdgcn_mfma_f32_16x16x4f32(v[s][e], av[s][j][e], acc[j], 0, 0, 0);
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
    if (rank < a.up && b * kURows + mm < a.M) a.u[(long)(b * kURows + mm) * a.up + rank] = sum;
  }
}

// The places of 32 rows of a slice, four rows a thread and 32 threads a row (four
// tokens read from LDS then serve sixteen comparisons; one row a thread left the
// LDS the bound, 42 us for the launch at 8192 rows). toks: the slice's tokens (N
// for none).
__device__ __forceinline__ void place_block(const EmbedBwdArgs& a, int b, int* toks) {
  constexpr int RT = 4, PT = 256 * RT / kPlaceRows;              // rows a thread, threads a row
  const int tid = threadIdx.x, part = tid % PT;
  const int m0 = b * kPlaceRows, s0 = m0 / kSlice * kSlice;
  const int n = a.M - s0 < kSlice ? a.M - s0 : kSlice;           // rows of the slice
  const int n4 = (n + 4 * PT - 1) / (4 * PT) * (4 * PT);
  auto stage = [&](auto* ids) {
    for (int i0 = tid; i0 < n4; i0 += 8 * 256) {                 // eight loads in flight
      int t[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const auto v = ids[s0 + (i0 + 256 * u < n ? i0 + 256 * u : n - 1)];
        t[u] = v >= 0 && v < a.ids.vocab ? (int)v : a.N;
      }
#pragma unroll
      for (int u = 0; u < 8; ++u)                                // (past the slice: behind every row)
        if (i0 + 256 * u < n4) toks[i0 + 256 * u] = i0 + 256 * u < n ? t[u] : 0x7fffffff;
    }
  };
  if (a.ids.wide) stage(static_cast<const int64_t*>(a.ids.p));
  else stage(static_cast<const int32_t*>(a.ids.p));
  __syncthreads();
  const int mine = m0 - s0 + tid / PT * RT;                      // the first of the thread's rows
  int t[RT], before[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    t[r] = toks[mine + r < n ? mine + r : 0];
    before[r] = 0;
  }
  // rows before one's own come first where their token is not larger, rows behind it
  // where it is smaller; only the block's own rows have to be told apart one by one
  const int own = m0 - s0;
  auto count = [&](int i0, int i1, int more) {                   // tokens below t + more
#pragma unroll 4
    for (int i = i0 + 4 * part; i < i1; i += 4 * PT) {
      const i32x4 v = *reinterpret_cast<const i32x4*>(toks + i);
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int e = 0; e < 4; ++e) before[r] += v[e] < t[r] + more ? 1 : 0;
    }
  };
  count(0, own, 1);
  for (int i = own + part; i < own + kPlaceRows; i += PT) {
#pragma unroll
    for (int r = 0; r < RT; ++r) before[r] += toks[i] < t[r] + (i < mine + r ? 1 : 0) ? 1 : 0;
  }
  count(own + kPlaceRows, n4, 0);
#pragma unroll
  for (int r = 0; r < RT; ++r) {
#pragma unroll
    for (int d = PT / 2; d >= 1; d >>= 1) before[r] += __shfl_xor(before[r], d);
    if (part != r || mine + r >= n) continue;
    const int at = s0 + before[r];
    if (a.nslices == 1) {
      a.tok[at] = t[r];
      a.row[at] = s0 + mine + r;
    } else {
      a.slices[at] = ((uint64_t)(uint32_t)t[r] << 32) | (uint32_t)(s0 + mine + r);
    }
  }
}

// Blocks in this order: place, u, dA, fill.
template <typename T, int RB>
__global__ __launch_bounds__(256) void embed_bwd_kernel(EmbedBwdArgs a) {
  __shared__ __attribute__((aligned(16))) char lds[kSlice * 4];
  static_assert(4 * 256 * RB * 4 <= kSlice * 4 && rank_sum_lds<RB>() <= kSlice * 4, "every kind of block fits");
  int b = blockIdx.x;
  if (b < a.nplace) { place_block(a, b, reinterpret_cast<int*>(lds)); return; }
  b -= a.nplace;
  if (b < a.nu) { u_block<T, RB>(a, b, reinterpret_cast<float*>(lds)); return; }
  b -= a.nu;
  if (b < a.nda) {
    rank_sum_block<T, RB>(b, a.M, a.K, a.r, a.rows_a, static_cast<const typename Elem<T>::type*>(a.dy), a.pA, lds,
                          [&](int m) { return entry_of(a.ids, m) >= 0; },
                          [&](int m, int j) { return a.B[(long)j * a.N + entry_of(a.ids, m)]; });
    return;
  }
  b -= a.nda;
  const long n = (long)a.r * a.N, e1 = (long)(b + 1) * kFill < n ? (long)(b + 1) * kFill : n;
  for (long e = (long)b * kFill + 4 * threadIdx.x; e < e1; e += 1024)     // N % 16 == 0
    *reinterpret_cast<f32x4*>(a.dB + e) = f32x4{0.f, 0.f, 0.f, 0.f};
}

// Keys of a slice's n sorted ones before `key`.
__device__ __forceinline__ int before(const uint64_t* p, int n, uint64_t key) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (p[mid] < key) lo = mid + 1;
    else hi = mid;
  }
  return lo;
}

__global__ __launch_bounds__(256) void embed_merge_kernel(EmbedBwdArgs a) {
  const int m = blockIdx.x * 256 + threadIdx.x;
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

// dB: blocks [0, nseg) take 256 sorted rows each, and every run of one token
// that begins among them to its end wherever that is; the others dA. R: the
// pitch of u.
template <int R>
__global__ __launch_bounds__(256) void embed_runs_kernel(EmbedBwdArgs a, int nseg) {
  __shared__ int first_tok[5];         // the token of each wave's first row, of the next block's
  __shared__ int whole[4];             // a wave that is one run
  __shared__ int found[4];
  __shared__ float first_sum[4][R], rest[4][R];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, b = blockIdx.x;
  if (b >= nseg) {
    const long e = (long)(b - nseg) * 256 + tid, n = (long)a.r * a.K;
    if (e >= n) return;
    const float sum = a.c * rank_sum_total(a.pA, a.blocks_a, n, e);
    float* out = a.dA + e % a.K * a.r + e / a.K;
    *out = a.accumulate ? *out + sum : sum;
    return;
  }
  const int i0 = b * kSegRows, i = i0 + tid;
  const int t = i < a.M ? a.tok[i] : a.N;                      // N: no token (behind all others)
  const int prev = i > 0 && i < a.M ? a.tok[i - 1] : -1;
  float v[R];
  auto load = [&](int at, float (&x)[R]) {
    const float* p = a.u + (long)a.row[at] * R;
#pragma unroll
    for (int j = 0; j < R; j += 4) {
      const f32x4 y = *reinterpret_cast<const f32x4*>(p + j);
#pragma unroll
      for (int c = 0; c < 4; ++c) x[j + c] = y[c];
    }
  };
#pragma unroll
  for (int j = 0; j < R; ++j) v[j] = 0.f;
  if (t < a.N) load(i, v);
  // v of lane k becomes the sum of its run from lane k to the wave's end
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int other = __shfl_down(t, d);
    const bool same = lane + d < 64 && other == t;
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const float x = __shfl_down(v[j], d);
      v[j] += same ? x : 0.f;
    }
  }
  const int last = __shfl(t, 63);
  if (lane == 0) {
    first_tok[w] = t;
    whole[w] = last == t;
#pragma unroll
    for (int j = 0; j < R; ++j) first_sum[w][j] = v[j];
  }
  if (tid == 0) first_tok[4] = i0 + kSegRows < a.M ? a.tok[i0 + kSegRows] : a.N;
  __syncthreads();
  // the run that leaves the block, where it also begins here: what follows, added
  // by all threads (lane by lane, the lanes in a tree, the waves in order)
  const int t3 = __builtin_amdgcn_readfirstlane(first_tok[4]);
  const bool begins = first_tok[0] != t3 || b == 0 || a.tok[i0 - 1] != t3;
  bool leaves = false;
  if (t3 < a.N && begins) {
    // (the block's last row: its wave's last token)
    leaves = a.tok[i0 + kSegRows - 1] == t3;
  }
  if (leaves) {                                                // block-uniform
    // where its token ends: 256 places looked at together, then between two of them
    int lo = i0 + kSegRows, hi = a.M;
    while (lo < hi) {
      const int stride = (hi - lo + 255) / 256, p = lo + tid * stride;
      const int here = __builtin_popcountll(__builtin_amdgcn_ballot_w64(p < hi && a.tok[p < hi ? p : lo] == t3));
      if (lane == 0) found[w] = here;
      __syncthreads();
      const int c = found[0] + found[1] + found[2] + found[3];     // those before the end, in order
      __syncthreads();
      hi = lo + c * stride < hi ? lo + c * stride : hi;
      lo = c > 0 ? lo + (c - 1) * stride + 1 : lo;
    }
    float x[R], y[4][R];
#pragma unroll
    for (int j = 0; j < R; ++j) x[j] = 0.f;
    constexpr int U = R <= 8 ? 4 : 1;                          // rows in flight a thread
    for (int k = i0 + kSegRows + tid; k < lo; k += 256 * U) {
#pragma unroll
      for (int c = 0; c < U; ++c) load(k + 256 * c < lo ? k + 256 * c : k, y[c]);
#pragma unroll
      for (int c = 0; c < U; ++c)
#pragma unroll
        for (int j = 0; j < R; ++j) x[j] += k + 256 * c < lo ? y[c][j] : 0.f;
    }
#pragma unroll
    for (int j = 0; j < R; ++j) {
      x[j] = wave_sum(x[j]);
      if (lane == 0) rest[w][j] = x[j];
    }
    __syncthreads();
  }
  if (t >= a.N || t == prev) return;
  // a run begins at this row: the next waves' first runs where it goes on
  bool on = last == t;
  for (int k = w + 1; k < 4 && on; ++k) {
    if (first_tok[k] != t) { on = false; break; }
#pragma unroll
    for (int j = 0; j < R; ++j) v[j] += first_sum[k][j];
    on = whole[k];
  }
  if (leaves && on && t == t3) {
#pragma unroll
    for (int j = 0; j < R; ++j) v[j] += ((rest[0][j] + rest[1][j]) + rest[2][j]) + rest[3][j];
  }
#pragma unroll
  for (int j = 0; j < R; ++j)
    if (j < a.r) {
      float* out = a.dB + (long)j * a.N + t;
      *out = a.accumulate ? *out + a.c * v[j] : a.c * v[j];
    }
}

struct EmbedBwdLayout {
  size_t u, pA, slices, tok, row, total;
};
int u_pitch(int r) { return r <= 4 ? 4 : r <= 8 ? 8 : r <= 16 ? 16 : 32; }
EmbedBwdLayout embed_bwd_layout(int M, int K, int r) {
  EmbedBwdLayout w{};
  size_t off = 0;
  w.u = off; off = align_up(off + (size_t)M * u_pitch(r) * 4);
  w.pA = off; off = align_up(off + rank_sum_floats(M, K, r) * 4);
  w.slices = off; off = align_up(off + (M > kSlice ? (size_t)M * 8 : 0));
  w.tok = off; off = align_up(off + (size_t)M * 4);
  w.row = off; off = align_up(off + (size_t)M * 4);
  w.total = off;
  return w;
}

template <typename T>
void embed_bwd_first(const EmbedBwdArgs& a, int blocks, hipStream_t st) {
  if (a.r <= 16) embed_bwd_kernel<T, 1><<<dim3((unsigned)blocks), 256, 0, st>>>(a);
  else embed_bwd_kernel<T, 2><<<dim3((unsigned)blocks), 256, 0, st>>>(a);
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
  a.up = u_pitch(L.r);
  a.dA = dA; a.dB = dB; a.accumulate = accumulate;
  a.nslices = (M + kSlice - 1) / kSlice;
  a.nplace = (M + kPlaceRows - 1) / kPlaceRows;
  a.nu = (M + kURows - 1) / kURows;
  a.rows_a = rank_sum_rows(M, L.K);
  a.blocks_a = (M + a.rows_a - 1) / a.rows_a;
  a.nda = rank_sum_blocks(M, L.K);
  const int nfill = accumulate ? 0 : (int)(((long)L.r * L.N + kFill - 1) / kFill);
  const int blocks = a.nplace + a.nu + a.nda + nfill;
  if (dtype == 0) embed_bwd_first<F32>(a, blocks, st);
  else embed_bwd_first<BF16>(a, blocks, st);
  if (a.nslices > 1) embed_merge_kernel<<<dim3((unsigned)((M + 255) / 256)), 256, 0, st>>>(a);
  const int nsum = (int)(((long)L.r * L.K + 255) / 256), nseg = (M + kSegRows - 1) / kSegRows;
  const dim3 grid((unsigned)(nseg + nsum));
  if (a.up == 4) embed_runs_kernel<4><<<grid, 256, 0, st>>>(a, nseg);
  else if (a.up == 8) embed_runs_kernel<8><<<grid, 256, 0, st>>>(a, nseg);
  else if (a.up == 16) embed_runs_kernel<16><<<grid, 256, 0, st>>>(a, nseg);
  else embed_runs_kernel<32><<<grid, 256, 0, st>>>(a, nseg);
}

}  // namespace qlora
