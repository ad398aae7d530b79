// One AdamW step of many float32 tensors, moments in 32 or 8 bits (formulas and
// the 8-bit form: include/qlora.h).
//
// Memory-bound: an element moves 28 bytes with float32 moments, 16.1 with 8-bit
// ones, and 4 more where the norm is taken first (100 million elements in one tensor:
// 527 and 606 us with float32 moments, 5.3 TB/s, 308 and 412 with 8-bit ones, 5.2 and
// 4.9, whose vector work is as long). Two small tensors are one
// block's work in one launch; else two kernels, each launched once per 64
// tensors, their pointers in the kernel's arguments:
//
//   norm    a block sums the squares of one chunk of one tensor in float64 and
//           leaves the sum in the workspace; chunks grow with the total, so
//           that there are up to 512 sums and one more for each tensor, which
//           every block of the update adds (2000 tensors of 1000 elements: 320 us
//           replayed, 32 launches of each kernel, 174 without the norm). Block 0 of the
//           first launch also forms what depends on the step alone (the bias
//           corrections, in float64) and advances the step: nothing else reads
//           it there. Without a norm to take, that block is the whole launch.
//   update  a block takes 4096 elements of one tensor, 16 a thread in four
//           pieces of 16 bytes, all of them in flight before the block adds the
//           sums of the norm (in their order, every block the same).
//
// Eight lanes hold one group of 32 8-bit moments, so its maximum is three DPP
// steps. The operations are written as the formulas have them, each rounded
// (no contraction), so that the float32 results do not depend on how a thread
// holds them.
#include "adamw.hpp"
#include "abi.hpp"
#include "common.hpp"

#pragma clang fp contract(off)

namespace qlora {

namespace {

constexpr int kItems = 64;           // tensors per launch (one a lane; 4 KB of arguments)
constexpr int kChunk = 4096;         // elements per block of the update
constexpr int kNormSums = 512;       // about as many partial sums of the norm
constexpr int kSmall = 8192;         // elements in all that one block steps,
constexpr int kSmallItems = 2;       // in up to so many tensors (a layer's A and B)

// What the norm launch leaves for the update.
struct Hyper {
  float lr, c1, root_c2;             // learning rate, 1 - beta1^k, sqrt(1 - beta2^k)
  int32_t k;
};

__device__ __forceinline__ Hyper hyper_of(int32_t k, double lr, double beta1, double beta2, const float* lr_dev) {
  Hyper h;
  h.lr = lr_dev != nullptr ? *lr_dev : (float)lr;
  h.c1 = (float)(1.0 - pow(beta1, (double)k));
  h.root_c2 = sqrtf((float)(1.0 - pow(beta2, (double)k)));
  h.k = k;
  return h;
}

struct NormArgs {
  const float* g[kItems];
  int n[kItems];
  int bstart[kItems + 1];            // first block of each tensor
  int count, chunk, first;           // first: this launch holds block 0 of the call
  long base;                         // partial sums of earlier launches
  double lr, beta1, beta2;
  const float* lr_dev;
  int32_t* step;
  Hyper* hyper;
  double* sums;
};
static_assert(sizeof(NormArgs) <= 4096, "kernel arguments");

// The tensor of block b: a lane looks at one tensor's first block each.
__device__ __forceinline__ int item_of(const int* bstart, int count, int b) {
  const int lane = threadIdx.x & 63;
  return __builtin_popcountll(__builtin_amdgcn_ballot_w64(lane < count && b >= bstart[lane])) - 1;
}

// Sum over the block's 256 threads, the same in every thread and in a fixed
// order; red: 4 doubles of LDS.
__device__ __forceinline__ double block_sum(double v, double* red) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  return (red[0] + red[1]) + (red[2] + red[3]);
}

__global__ __launch_bounds__(256) void adamw_norm_kernel(NormArgs a) {
  __shared__ double red[4];
  const int tid = threadIdx.x, b = blockIdx.x;
  if (a.first && b == 0 && tid == 0) {
    const Hyper h = hyper_of(*a.step + 1, a.lr, a.beta1, a.beta2, a.lr_dev);
    *a.hyper = h;
    *a.step = h.k;
  }
  if (a.sums == nullptr) return;
  const int i = item_of(a.bstart, a.count, b);
  const long e0 = (long)(b - a.bstart[i]) * a.chunk;
  const long e1 = e0 + a.chunk < a.n[i] ? e0 + a.chunk : a.n[i];
  const float* g = a.g[i];
  double sum = 0.0;
  const long q1 = e0 + ((e1 - e0) & ~3L);
  for (long e = e0 + 4 * tid; e < q1; e += 4096) {          // four pieces in flight
    f32x4 v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      v[u] = *reinterpret_cast<const f32x4*>(g + (e + 1024 * u < q1 ? e + 1024 * u : e));
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (e + 1024 * u < q1)
#pragma unroll
        for (int c = 0; c < 4; ++c) sum += (double)v[u][c] * (double)v[u][c];
  }
  if (q1 + tid < e1) sum += (double)g[q1 + tid] * (double)g[q1 + tid];
  sum = block_sum(sum, red);
  if (tid == 0) a.sums[a.base + b] = sum;
}

struct UpdateItem {
  float* p;
  const float* g;
  void* m;
  void* v;
  uint8_t* ms;
  uint8_t* vs;
  int n;
  float decay;
};
struct UpdateArgs {
  UpdateItem it[kItems];
  int bstart[kItems + 1];
  int count, item0, first;
  int clip, sums_n;                  // clip: the gradient is clipped
  float beta1, rest1, beta2, rest2, eps, clip_norm;
  uint32_t seed;
  int32_t* step;
  const Hyper* hyper;
  const double* sums;                // NULL: no norm
  float* norm;
};
static_assert(sizeof(UpdateArgs) + 32 <= 4096, "kernel arguments");

// 32 bits for one element: two rounds of multiply and shift (odd constants: the
// golden ratio's and the square roots' of 2 and 3 first 32 bits).
__device__ __forceinline__ uint32_t hash32(uint32_t x) {
  x ^= x >> 16;
  x *= 0x6A09E667u;
  x ^= x >> 15;
  x *= 0xBB67AE85u;
  return x ^ (x >> 16);
}

// The largest of the 8 lanes that hold one group.
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
#pragma unroll
  for (int lvl = 1; lvl < 4; ++lvl) {
    const uint32_t w = __float_as_uint(dpp_pair(__uint_as_float(v), lvl));
    v = w > v ? w : v;
  }
  return v;
}

// The exponent e of a group's scale for BITS bits of mantissa, from the bits of
// its largest magnitude (finite): the smallest with top <= (2 - 2^-BITS) 2^e,
// held to [-126, 127].
template <int BITS>
__device__ __forceinline__ int scale_exp(uint32_t top) {
  const int e = (int)(top >> 23) - 127 + ((top & 0x7fffffu) > (0x7fffffu & (~0u << (23 - BITS))) ? 1 : 0);
  return e < -126 ? -126 : e > 127 ? 127 : e;
}

// 2^e, e in [-127, 127]; the factor of a group by its scale byte (255: NaN).
__device__ __forceinline__ float power_of_two(int e) {
  return __uint_as_float(e > -127 ? (uint32_t)(e + 127) << 23 : 0x400000u);
}
__device__ __forceinline__ float group_factor(int byte) {
  return byte == 255 ? __uint_as_float(0x7fc00000u) : power_of_two(byte - 127);
}

// A magnitude under its group's scale as a code: v 2^-(e + 120), `inv` = 2^-e, is a
// float32 whose exponent field is the code's, 0 to 7; the hash's 16 bits are added
// right below the code's last bit.
template <int BITS>
__device__ __forceinline__ uint32_t to_code(float v, float inv, uint32_t rnd) {
  const uint32_t f = __float_as_uint(__builtin_fabsf(v) * inv * 0x1p-120f);
  const uint32_t c = (f + (rnd << (23 - BITS - 16))) >> (23 - BITS);
  constexpr uint32_t most = (8u << BITS) - 1;
  return c < most ? c : most;
}
// A code times its group's factor; bit 31 of `sign` is the value's sign.
template <int BITS>
__device__ __forceinline__ float of_code(uint32_t c, uint32_t sign, float factor) {
  return __uint_as_float((c << (23 - BITS)) | (sign & 0x80000000u)) * 0x1p120f * factor;
}

// What every element of a launch shares.
struct Step {
  float beta1, rest1, beta2, rest2, eps;
  float rate, root_c2, inv_c2;        // lr / (1 - beta1^k); 1 / root_c2
  float coef;                         // of the gradient (1: not clipped)
  uint32_t key;                       // of the hash: step and seed
};

// root / root_c2, the rounded quotient, from the rounded reciprocal: the remainder of
// the first product is exact (roots are 0, or 2^-75 and more), and its share rounds
// once more (a divisor of 24 ones may leave it one step off). A division that knows
// nothing of its divisor is ten instructions, and 8-bit steps are bound by theirs.
__device__ __forceinline__ float over(float root, const Step& s) {
  const float y = root * s.inv_c2, rest = __builtin_fmaf(-y, s.root_c2, root);
  return root <= 3.4028234e38f ? __builtin_fmaf(rest, s.inv_c2, y) : root;
}

// Four elements of one tensor from element e on, in registers.
template <bool S8> struct Piece {
  float p[4], g[4], m[4], v[4];
  uint32_t mc, vc;
  int ms, vs;

  // From clamped places: a piece past the end reads the first one again, a ragged
  // last piece is read by elements.
  __device__ __forceinline__ void load(const UpdateItem& it, int e) {
    const int n = it.n;
    if (e + 4 <= n || e >= n) {
      const long at = e < n ? e : 0;
      const bool whole = n >= 4;                            // (n < 4: nothing is whole, and nothing is used)
      const f32x4 z{0.f, 0.f, 0.f, 0.f};
      const f32x4 pv = whole ? *reinterpret_cast<const f32x4*>(it.p + at) : z;
      const f32x4 gv = whole ? *reinterpret_cast<const f32x4*>(it.g + at) : z;
#pragma unroll
      for (int c = 0; c < 4; ++c) { p[c] = pv[c]; g[c] = gv[c]; }
      if constexpr (S8) {
        mc = whole ? *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(it.m) + at) : 0u;
        vc = whole ? *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(it.v) + at) : 0u;
      } else {
        const f32x4 mv = whole ? *reinterpret_cast<const f32x4*>(static_cast<const float*>(it.m) + at) : z;
        const f32x4 vv = whole ? *reinterpret_cast<const f32x4*>(static_cast<const float*>(it.v) + at) : z;
#pragma unroll
        for (int c = 0; c < 4; ++c) { m[c] = mv[c]; v[c] = vv[c]; }
      }
    } else {
      if constexpr (S8) mc = vc = 0u;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int at = e + c < n ? e + c : e;
        p[c] = it.p[at];
        g[c] = e + c < n ? it.g[at] : 0.f;
        if constexpr (S8) {
          if (e + c < n) {
            mc |= (uint32_t)static_cast<const uint8_t*>(it.m)[at] << (8 * c);
            vc |= (uint32_t)static_cast<const uint8_t*>(it.v)[at] << (8 * c);
          }
        } else {
          m[c] = static_cast<const float*>(it.m)[at];
          v[c] = static_cast<const float*>(it.v)[at];
        }
      }
    }
    if constexpr (S8) {
      ms = it.ms[e < n ? e / 32 : 0];
      vs = it.vs[e < n ? e / 32 : 0];
    }
  }

  // The step, and its results written. All lanes of a wave together (a group's
  // maximum crosses lanes); keep: 1 - lr decay of the tensor, item: its number.
  __device__ __forceinline__ void update(const UpdateItem& it, int e, int item, float keep, const Step& s) {
    const int n = it.n;
    float root[4];
    if constexpr (S8) {
      const float mf = group_factor(ms), vf = group_factor(vs);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint32_t mb = (mc >> (8 * c)) & 0xffu, vb = (vc >> (8 * c)) & 0xffu;
        const float rv = of_code<5>(vb, 0u, vf);
        m[c] = of_code<4>(mb & 127u, mb << 24, mf);
        v[c] = rv * rv;
      }
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const float gc = g[c] * s.coef;
      m[c] = s.beta1 * m[c] + s.rest1 * gc;
      v[c] = s.beta2 * v[c] + s.rest2 * (gc * gc);
      root[c] = sqrtf(v[c]);
      const float moved = p[c] * keep;
      p[c] = moved - s.rate * (m[c] / (over(root[c], s) + s.eps));
    }
    uint32_t mo = 0u, vo = 0u;
    int me = 0, ve = 0;
    if constexpr (S8) {
      // elements past the end are no part of their group
      if (e + 4 > n) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (e + c >= n) m[c] = root[c] = 0.f;
      }
      uint32_t mt = 0u, vt = 0u;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint32_t x = abs_bits(m[c]), y = abs_bits(root[c]);
        mt = x > mt ? x : mt;
        vt = y > vt ? y : vt;
      }
      mt = group_max(mt);
      vt = group_max(vt);
      const bool mbad = mt >= 0x7f800000u, vbad = vt >= 0x7f800000u;
      me = scale_exp<4>(mt);
      ve = scale_exp<5>(vt);
      const float mi = power_of_two(-me), vi = power_of_two(-ve);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint32_t rnd = hash32((uint32_t)(e + c) * 0x9E3779B1u + (uint32_t)item * 0x3C6EF373u + s.key);
        const uint32_t x = to_code<4>(m[c], mi, rnd & 0xffffu) | (m[c] < 0.f ? 128u : 0u);
        const uint32_t y = to_code<5>(root[c], vi, rnd >> 16), bits = __float_as_uint(root[c]);
        const uint32_t least = bits < 1u ? bits : 1u;       // 1 where the root (not negative) is not 0
        mo |= x << (8 * c);
        vo |= (y > least ? y : least) << (8 * c);
      }
      mo = mbad ? 0u : mo;
      vo = vbad ? 0u : vo;
      me = mbad ? 255 : me + 127;
      ve = vbad ? 255 : ve + 127;
    }
    if (e + 4 <= n) {
      *reinterpret_cast<f32x4*>(it.p + e) = f32x4{p[0], p[1], p[2], p[3]};
      if constexpr (S8) {
        *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(it.m) + e) = mo;
        *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(it.v) + e) = vo;
      } else {
        *reinterpret_cast<f32x4*>(static_cast<float*>(it.m) + e) = f32x4{m[0], m[1], m[2], m[3]};
        *reinterpret_cast<f32x4*>(static_cast<float*>(it.v) + e) = f32x4{v[0], v[1], v[2], v[3]};
      }
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (e + c < n) {
          it.p[e + c] = p[c];
          if constexpr (S8) {
            static_cast<uint8_t*>(it.m)[e + c] = (uint8_t)(mo >> (8 * c));
            static_cast<uint8_t*>(it.v)[e + c] = (uint8_t)(vo >> (8 * c));
          } else {
            static_cast<float*>(it.m)[e + c] = m[c];
            static_cast<float*>(it.v)[e + c] = v[c];
          }
        }
    }
    if constexpr (S8) {
      if (e < n && (e & 31) == 0) {
        it.ms[e / 32] = (uint8_t)me;
        it.vs[e / 32] = (uint8_t)ve;
      }
    }
  }
};

// A norm that is infinite or NaN.
__device__ __forceinline__ bool no_norm(float norm) { return !(norm <= 3.4028234e38f); }

__device__ __forceinline__ Step step_of(const UpdateArgs& a, const Hyper& h, float norm) {
  return Step{a.beta1, a.rest1, a.beta2, a.rest2, a.eps, h.lr / h.c1, h.root_c2, 1.f / h.root_c2,
              a.clip ? a.clip_norm / (norm > a.clip_norm ? norm : a.clip_norm) : 1.f,
              (uint32_t)h.k * 0xBB67AE85u + a.seed};
}

template <bool S8>
__global__ __launch_bounds__(256) void adamw_update_kernel(UpdateArgs a) {
  __shared__ double red[4];
  const int tid = threadIdx.x, b = blockIdx.x;
  const int i = item_of(a.bstart, a.count, b);
  const UpdateItem& it = a.it[i];
  const int c0 = (b - a.bstart[i]) * kChunk;
  constexpr int U = kChunk / 1024;
  Piece<S8> x[U];
#pragma unroll
  for (int u = 0; u < U; ++u) x[u].load(it, c0 + 1024 * u + 4 * tid);
  const Hyper h = *a.hyper;
  float norm = 0.f;
  if (a.sums != nullptr) {
    double sum = 0.0;
    for (int q = tid; q < a.sums_n; q += 256) sum += a.sums[q];
    norm = (float)sqrt(block_sum(sum, red));
    const bool skip = a.clip && no_norm(norm);              // nothing is moved
    if (a.first && b == 0 && tid == 0) {
      if (a.norm != nullptr) *a.norm = norm;
      if (skip) *a.step = h.k - 1;
    }
    if (skip) return;
  }
  const Step s = step_of(a, h, norm);
  const float keep = 1.f - h.lr * it.decay;
#pragma unroll
  for (int u = 0; u < U; ++u) x[u].update(it, c0 + 1024 * u + 4 * tid, a.item0 + i, keep, s);
}

// The whole step of few elements in one block and one launch: the norm, then the
// tensors one after the other, 1.8 us each with float32 moments and 3.2 with 8-bit
// ones (replayed: 6.8 and 9.6 us for two tensors, 10.4 and 16 for four; two launches
// take 8.8 and 10.7 for any number). sums_n: whether the norm is wanted.
template <bool S8>
__global__ __launch_bounds__(1024) void adamw_small_kernel(UpdateArgs a, double lr, double beta1, double beta2,
                                                           const float* lr_dev) {
  __shared__ double red[16];
  __shared__ Hyper hyper;
  const int tid = threadIdx.x;
  if (tid == 0) {
    hyper = hyper_of(*a.step + 1, lr, beta1, beta2, lr_dev);
  }
  float norm = 0.f;
  if (a.sums_n) {
    double sum = 0.0;
    for (int i = 0; i < a.count; ++i)
      for (int e = tid; e < a.it[i].n; e += 1024) sum += (double)a.it[i].g[e] * (double)a.it[i].g[e];
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) sum += __shfl_xor(sum, d);
    if ((tid & 63) == 0) red[tid >> 6] = sum;
  }
  __syncthreads();
  const Hyper h = hyper;
  if (a.sums_n) {
    double sum = 0.0;
    for (int w = 0; w < 16; ++w) sum += red[w];
    norm = (float)sqrt(sum);
    if (tid == 0 && a.norm != nullptr) *a.norm = norm;
    if (a.clip && no_norm(norm)) return;                    // nothing is moved
  }
  if (tid == 0) *a.step = h.k;
  const Step s = step_of(a, h, norm);
  for (int i = 0; i < a.count; ++i) {
    const UpdateItem& it = a.it[i];
    const float keep = 1.f - h.lr * it.decay;
    for (int e = 4 * tid; e - 4 * tid < it.n; e += 4096) {  // block-uniform
      Piece<S8> x;
      x.load(it, e);
      x.update(it, e, i, keep, s);
    }
  }
}

// 8-bit moments to float32 or bf16 (exact above 2^-126) and back (to the nearest
// code, halves up): 8 elements a thread, 4 lanes a group. BITS: 4 the first
// moment, 5 the root of the second.
template <typename T, int BITS>
__global__ __launch_bounds__(256) void moment_read_kernel(const uint8_t* codes, const uint8_t* scales, long n,
                                                          typename Elem<T>::type* x) {
  const long e = ((long)blockIdx.x * 256 + threadIdx.x) * 8;
  if (e >= n) return;
  const float factor = group_factor(scales[e / 32]);
  uint32_t w[2] = {0u, 0u};
  if (e + 8 <= n) {
    const u32x2 v = *reinterpret_cast<const u32x2*>(codes + e);
    w[0] = v.x;
    w[1] = v.y;
  } else {
    for (int c = 0; e + c < n; ++c) w[c / 4] |= (uint32_t)codes[e + c] << (8 * (c % 4));
  }
  float v[8];
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    const uint32_t b = (w[c / 4] >> (8 * (c % 4))) & 0xffu;
    v[c] = of_code<BITS>(BITS == 4 ? b & 127u : b, BITS == 4 ? b << 24 : 0u, factor);
  }
  if (e + 8 <= n) {
    if constexpr (sizeof(x[0]) == 4) {
      *reinterpret_cast<f32x4*>(x + e) = f32x4{v[0], v[1], v[2], v[3]};
      *reinterpret_cast<f32x4*>(x + e + 4) = f32x4{v[4], v[5], v[6], v[7]};
    } else {
      *reinterpret_cast<u32x4*>(x + e) = u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                              pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
    }
  } else {
    for (int c = 0; e + c < n; ++c) store_out(x + e + c, v[c]);
  }
}

template <typename T, int BITS>
__global__ __launch_bounds__(256) void moment_write_kernel(const typename Elem<T>::type* x, long n, uint8_t* codes,
                                                           uint8_t* scales) {
  const long e = ((long)blockIdx.x * 256 + threadIdx.x) * 8;
  float v[8];
  if (e + 8 <= n) {
    load8(x + e, v);
  } else {
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      v[c] = 0.f;
      if (e + c < n) {
        if constexpr (sizeof(x[0]) == 4) v[c] = x[e + c];
        else v[c] = bf16_to_f32(x[e + c]);
      }
    }
  }
  uint32_t top = 0u;
#pragma unroll
  for (int c = 0; c < 8; ++c) top = abs_bits(v[c]) > top ? abs_bits(v[c]) : top;
#pragma unroll
  for (int lvl = 2; lvl < 4; ++lvl) {                       // the 4 lanes of the group
    const uint32_t w = __float_as_uint(dpp_pair(__uint_as_float(top), lvl));
    top = w > top ? w : top;
  }
  if (e >= n) return;
  const bool bad = top >= 0x7f800000u;
  const int ex = scale_exp<BITS>(top);
  const float inv = power_of_two(-ex);
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    uint32_t k = to_code<BITS>(v[c], inv, 0x8000u);
    if (BITS == 5) k = k == 0u && v[c] != 0.f ? 1u : k;
    else k |= v[c] < 0.f ? 128u : 0u;
    w[c / 4] |= (bad ? 0u : k) << (8 * (c % 4));
  }
  if (e + 8 <= n) *reinterpret_cast<u32x2*>(codes + e) = u32x2{w[0], w[1]};
  else
    for (int c = 0; e + c < n; ++c) codes[e + c] = (uint8_t)(w[c / 4] >> (8 * (c % 4)));
  if ((e & 31) == 0) scales[e / 32] = (uint8_t)(bad ? 255 : ex + 127);
}

}  // namespace

void launch_moment_read(const uint8_t* codes, const uint8_t* scales, long n, int which, int dtype, void* x,
                        hipStream_t st) {
  const dim3 grid((unsigned)((n + 2047) / 2048));
  float* f = static_cast<float*>(x);
  uint16_t* h = static_cast<uint16_t*>(x);
  if (which == 0 && dtype == 0) moment_read_kernel<F32, 4><<<grid, 256, 0, st>>>(codes, scales, n, f);
  else if (which == 0) moment_read_kernel<BF16, 4><<<grid, 256, 0, st>>>(codes, scales, n, h);
  else if (dtype == 0) moment_read_kernel<F32, 5><<<grid, 256, 0, st>>>(codes, scales, n, f);
  else moment_read_kernel<BF16, 5><<<grid, 256, 0, st>>>(codes, scales, n, h);
}

void launch_moment_write(const void* x, long n, int which, int dtype, uint8_t* codes, uint8_t* scales,
                         hipStream_t st) {
  const dim3 grid((unsigned)((n + 2047) / 2048));
  const float* f = static_cast<const float*>(x);
  const uint16_t* h = static_cast<const uint16_t*>(x);
  if (which == 0 && dtype == 0) moment_write_kernel<F32, 4><<<grid, 256, 0, st>>>(f, n, codes, scales);
  else if (which == 0) moment_write_kernel<BF16, 4><<<grid, 256, 0, st>>>(h, n, codes, scales);
  else if (dtype == 0) moment_write_kernel<F32, 5><<<grid, 256, 0, st>>>(f, n, codes, scales);
  else moment_write_kernel<BF16, 5><<<grid, 256, 0, st>>>(h, n, codes, scales);
}

long adamw_norm_blocks(const qlora_adamw_item* items, int count, long* chunk) {
  long total = 0, blocks = 0;
  for (int i = 0; i < count; ++i) total += items[i].n;
  const long c = (total / kNormSums + kChunk - 1) / kChunk * kChunk;
  *chunk = c < kChunk ? kChunk : c > (1L << 30) ? (1L << 30) : c;
  for (int i = 0; i < count; ++i) blocks += (items[i].n + *chunk - 1) / *chunk;
  return blocks;
}

size_t adamw_bytes(const qlora_adamw_item* items, int count) {
  long chunk;
  return align_up(sizeof(Hyper)) + align_up((size_t)adamw_norm_blocks(items, count, &chunk) * 8);
}

void launch_adamw(const qlora_adamw_config& cfg, const qlora_adamw_item* items, int count, void* ws,
                  hipStream_t st) {
  Hyper* hyper = static_cast<Hyper*>(ws);
  const bool clip = cfg.clip_norm > 0.0, norm = clip || cfg.norm != nullptr;
  double* sums = norm ? reinterpret_cast<double*>(static_cast<char*>(ws) + align_up(sizeof(Hyper))) : nullptr;
  long chunk, total = 0;
  for (int i = 0; i < count; ++i) total += items[i].n;
  const bool small = total <= kSmall && count <= kSmallItems;
  const long nsums = adamw_norm_blocks(items, count, &chunk);
  long base = 0;
  for (int i0 = 0; !small && i0 < (norm ? count : 1); i0 += kItems) {
    NormArgs a{};
    a.count = count - i0 < kItems ? count - i0 : kItems;
    a.chunk = (int)chunk;
    a.first = i0 == 0;
    a.base = base;
    a.lr = cfg.lr; a.beta1 = cfg.beta1; a.beta2 = cfg.beta2; a.lr_dev = cfg.lr_dev;
    a.step = cfg.step; a.hyper = hyper; a.sums = sums;
    for (int i = 0; i < a.count; ++i) {
      a.g[i] = items[i0 + i].g;
      a.n[i] = (int)items[i0 + i].n;
      a.bstart[i + 1] = a.bstart[i] + (int)((items[i0 + i].n + chunk - 1) / chunk);
    }
    base += a.bstart[a.count];
    adamw_norm_kernel<<<dim3(norm ? (unsigned)a.bstart[a.count] : 1u), 256, 0, st>>>(a);
  }
  for (int i0 = 0; i0 < count; i0 += kItems) {
    UpdateArgs a{};
    a.count = count - i0 < kItems ? count - i0 : kItems;
    a.item0 = i0;
    a.first = i0 == 0;
    a.clip = clip;
    a.sums_n = (int)nsums;
    a.beta1 = (float)cfg.beta1; a.rest1 = (float)(1.0 - cfg.beta1);
    a.beta2 = (float)cfg.beta2; a.rest2 = (float)(1.0 - cfg.beta2);
    a.eps = (float)cfg.eps; a.clip_norm = (float)cfg.clip_norm;
    a.seed = cfg.seed; a.step = cfg.step; a.hyper = hyper; a.sums = sums; a.norm = cfg.norm;
    for (int i = 0; i < a.count; ++i) {
      const qlora_adamw_item& s = items[i0 + i];
      a.it[i] = UpdateItem{s.p, s.g, s.m, s.v, s.m_scales, s.v_scales, (int)s.n, (float)s.decay};
      a.bstart[i + 1] = a.bstart[i] + (int)((s.n + kChunk - 1) / kChunk);
    }
    if (small) {
      a.sums_n = norm;
      if (cfg.sfmt == QLORA_S8)
        adamw_small_kernel<true><<<dim3(1), 1024, 0, st>>>(a, cfg.lr, cfg.beta1, cfg.beta2, cfg.lr_dev);
      else
        adamw_small_kernel<false><<<dim3(1), 1024, 0, st>>>(a, cfg.lr, cfg.beta1, cfg.beta2, cfg.lr_dev);
      return;
    }
    const dim3 grid((unsigned)a.bstart[a.count]);
    if (cfg.sfmt == QLORA_S8) adamw_update_kernel<true><<<grid, 256, 0, st>>>(a);
    else adamw_update_kernel<false><<<grid, 256, 0, st>>>(a);
  }
}

}  // namespace qlora
