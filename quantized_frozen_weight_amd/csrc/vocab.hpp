// Internal launchers of the vocabulary layer (vocab.hip, xent.hip). A layer of
// K features and N entries: codes [N, K] (or packed), scales, adapter A [K, r],
// B [r, N] (r may be 0), of which entries [0, vocab) exist.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace qlora {

// A token or target of a row as an entry, -1 where it is none.
struct Ids {
  const void* p;
  int wide;                          // int64
  int vocab;
};

struct VocabLayer {
  int K, N, r, fmt;                  // fmt: 0 int8, 1 4-bit
  const void* codes;
  const void* scales;
  const float* A;
  const float* B;
  float s;
};

// x [M, K] = scale (deq(W)[:, id] + s A B[:, id])
void launch_embed(const VocabLayer& L, int M, int dtype, Ids ids, float scale, void* x, hipStream_t st);

// Its gradient; ws: embed_bwd_bytes.
constexpr int kMaxTokens = 1 << 20;
size_t embed_bwd_bytes(int M, int K, int r);
void launch_embed_bwd(const VocabLayer& L, int M, int dtype, Ids ids, float scale, const void* dy,
                      bool accumulate, float* dA, float* dB, void* ws, hipStream_t st);

// Softmax cross entropy, up to kMaxRows rows and kMaxLogits logits (launches of
// fewer than 2^32 threads). xq, sx: the rows' codes and scales; t [M, r] (NULL at
// r = 0). part: xent_part_floats(...) floats.
constexpr int kMaxRows = 1 << 24;
constexpr long kMaxLogits = 1L << 37;
size_t xent_part_floats(int vocab, int M);
void launch_xent_fwd(const VocabLayer& L, int M, Ids ids, const int8_t* xq, const float* sx,
                     const float* t, float* part, float* loss, float* lse, hipStream_t st);

// The buffers of the gradient: pieces of `piece` entries; floats or bf16 values
// of each buffer (0: not used).
struct XentPlan {
  int piece;                         // entries per piece, a multiple of 256
  int splits;                        // of a piece's contraction for dx
  int parts;                         // dl as 1 float16, or in float32 3 parts in bf16
  size_t g, dxp, u, up, dbp, pA, smax;   // elements: dl (16 bits), partial sums of dx, u, those of u, dB and dA, maxima of scales
};
XentPlan xent_plan(const VocabLayer& L, int vocab, int M, int dtype);
struct XentBuffers {
  uint16_t* g;
  float *dxp, *u, *up, *dbp, *pA;
  uint32_t* smax;
};
// dx (NULL: none), and with an adapter dA and dB.
void launch_xent_bwd(const VocabLayer& L, int M, int dtype, Ids ids, const void* x, const int8_t* xq, const float* sx,
                     const float* t, const float* lse, const float* dloss, const XentPlan& plan,
                     const XentBuffers& buf, void* dx, float* dA, float* dB, hipStream_t st);

#ifdef __HIPCC__
__device__ __forceinline__ int entry_of(const Ids& ids, long m) {
  if (ids.wide) {
    const int64_t v = static_cast<const int64_t*>(ids.p)[m];
    return v >= 0 && v < ids.vocab ? (int)v : -1;
  }
  const int32_t v = static_cast<const int32_t*>(ids.p)[m];
  return v >= 0 && v < ids.vocab ? v : -1;
}
#endif

}  // namespace qlora
