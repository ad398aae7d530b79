// C ABI of the vocabulary layer and the AdamW step: argument validation,
// workspace layout, and the kernel sequence of each call. Contract and
// citations: include/qlora.h.
#include <hip/hip_runtime.h>

#include "abi.hpp"
#include "adamw.hpp"
#include "launch.hpp"
#include "vocab.hpp"

namespace {

using namespace qlora;

// A layer as the vocabulary calls take it (data pointers of the layer included).
int check_vocab(const qlora_linear* L, int vocab, int M, int dtype) {
  if (L == nullptr) return QLORA_EINVAL;
  int st = check_dtype(dtype);
  if (st) return st;
  if (M < 1 || L->K < 16 || L->N < 16 || L->K % 16 || L->N % 16 || L->r < 0 || L->r > 32) return QLORA_EINVAL;
  if (vocab < 1 || vocab > L->N) return QLORA_EINVAL;
  if (!fits_int(M, L->K) || !fits_int(L->K, L->N)) return QLORA_ERANGE;
  if (L->fmt != QLORA_W8 && L->fmt != QLORA_W4G128 && L->fmt != QLORA_W8O) return QLORA_EINVAL;
  if (L->heads < 0) return QLORA_EINVAL;
  if (L->fmt == QLORA_W8O || L->heads > 1) return QLORA_EUNSUPPORTED;
  if (L->fmt == QLORA_W4G128) {
    if (L->K % 128) return QLORA_EINVAL;
    if (dtype != QLORA_BF16 || L->K > 128 * kW4MaxGroups) return QLORA_EUNSUPPORTED;
  }
  const void* ptrs[2] = {L->codes, L->scales};
  for (const void* p : ptrs)
    if (p == nullptr || !aligned16(p)) return QLORA_EINVAL;
  const void* ab[2] = {L->A, L->B};
  for (const void* p : ab)
    if (L->r > 0 ? (p == nullptr || !aligned16(p)) : p != nullptr) return QLORA_EINVAL;
  return QLORA_OK;
}

int check_ids(const void* ids, int itype) {
  if (itype != QLORA_I32 && itype != QLORA_I64) return QLORA_EINVAL;
  return ids != nullptr && aligned16(ids) ? QLORA_OK : QLORA_EINVAL;
}
inline size_t ids_bytes(int M, int itype) { return (size_t)M * (itype == QLORA_I64 ? 8 : 4); }
inline Ids make_ids(const void* p, int itype, int vocab) { return Ids{p, itype == QLORA_I64, vocab}; }

VocabLayer vocab_layer(const qlora_linear* L) {
  return VocabLayer{L->K, L->N, L->r, L->fmt, L->codes, L->scales, L->A, L->B,
                    L->r > 0 ? L->alpha / (float)L->r : 0.f};
}

// The ranges of the layer and of the ids, as inputs.
void add_vocab(Ranges& in, const qlora_linear* L, const void* ids, int M, int itype) {
  size_t cb = 0, sb = 0;
  qlora_weight_bytes(L->K, L->N, L->fmt, &cb, &sb);
  in.add(L->codes, cb);
  in.add(L->scales, sb);
  in.add(L->A, (size_t)L->K * L->r * 4);
  in.add(L->B, (size_t)L->N * L->r * 4);
  in.add(ids, ids_bytes(M, itype));
}

inline bool ws_ok(const void* ws, size_t have, size_t need) {
  return have >= need && (need == 0 || (ws != nullptr && aligned16(ws)));
}

}  // namespace

extern "C" {

int qlora_embed(const qlora_linear* L, int vocab, int M, int dtype, const void* tokens, int itype,
                float scale, void* x, void* stream) {
  int st = check_vocab(L, vocab, M, dtype);
  if (st) return st;
  st = check_ids(tokens, itype);
  if (st) return st;
  if (!x || !aligned16(x)) return QLORA_EINVAL;
  Ranges in, out;
  add_vocab(in, L, tokens, M, itype);
  out.add(x, (size_t)M * L->K * dtype_bytes(dtype));
  if (!disjoint(out, in)) return QLORA_EINVAL;
  if (pending_error()) return QLORA_EHIP;
  launch_embed(vocab_layer(L), M, dtype, make_ids(tokens, itype, vocab), scale, x,
               static_cast<hipStream_t>(stream));
  return launch_status();
}

int qlora_embed_bwd_workspace(const qlora_linear* L, int vocab, int M, int dtype, size_t* bytes) {
  if (bytes == nullptr) return QLORA_EINVAL;
  const int st = check_vocab(L, vocab, M, dtype);
  if (st) return st;
  if (L->r < 1) return QLORA_EINVAL;
  if (M > kMaxTokens) return QLORA_ERANGE;
  *bytes = embed_bwd_bytes(M, L->K, L->r);
  return QLORA_OK;
}

int qlora_embed_bwd(const qlora_linear* L, int vocab, int M, int dtype, const void* tokens, int itype,
                    float scale, const void* dy, int accumulate, float* dA, float* dB, void* ws,
                    size_t ws_bytes, void* stream) {
  size_t need = 0;
  int st = qlora_embed_bwd_workspace(L, vocab, M, dtype, &need);
  if (st) return st;
  st = check_ids(tokens, itype);
  if (st) return st;
  if (!dy || !aligned16(dy) || !dA || !aligned16(dA) || !dB || !aligned16(dB)) return QLORA_EINVAL;
  if (!ws_ok(ws, ws_bytes, need)) return QLORA_EWORKSPACE;
  Ranges in, out;
  add_vocab(in, L, tokens, M, itype);
  in.add(dy, (size_t)M * L->K * dtype_bytes(dtype));
  out.add(dA, (size_t)L->K * L->r * 4);
  out.add(dB, (size_t)L->N * L->r * 4);
  out.add(ws, need);
  if (!disjoint(out, in)) return QLORA_EINVAL;
  if (pending_error()) return QLORA_EHIP;
  launch_embed_bwd(vocab_layer(L), M, dtype, make_ids(tokens, itype, vocab), scale, dy, accumulate != 0, dA,
                   dB, ws, static_cast<hipStream_t>(stream));
  return launch_status();
}

int qlora_adamw_workspace(const qlora_adamw_item* items, int count, size_t* bytes) {
  if (items == nullptr || count < 1 || bytes == nullptr) return QLORA_EINVAL;
  for (int i = 0; i < count; ++i)
    if (items[i].n < 1) return QLORA_EINVAL;
    else if (items[i].n > (1LL << 30)) return QLORA_ERANGE;
  *bytes = adamw_bytes(items, count);
  return QLORA_OK;
}

int qlora_adamw(const qlora_adamw_config* cfg, const qlora_adamw_item* items, int count, void* ws,
                size_t ws_bytes, void* stream) {
  size_t need = 0;
  const int st = qlora_adamw_workspace(items, count, &need);
  if (st) return st;
  if (cfg == nullptr || cfg->step == nullptr) return QLORA_EINVAL;
  // (a comparison with a NaN is false)
  const auto within = [](double v, double lo) { return v >= lo && v <= 3.0e38; };
  if (!within(cfg->lr, 0.0) || !within(cfg->clip_norm, 0.0) || !((float)cfg->eps > 0.f) || !within(cfg->eps, 0.0))
    return QLORA_EINVAL;
  if (!(cfg->beta1 >= 0.0 && cfg->beta1 < 1.0 && cfg->beta2 >= 0.0 && cfg->beta2 < 1.0)) return QLORA_EINVAL;
  if (cfg->clip_norm > 0.0 && !((float)cfg->clip_norm > 0.f)) return QLORA_EINVAL;
  if (cfg->sfmt != QLORA_S32 && cfg->sfmt != QLORA_S8) return QLORA_EINVAL;
  const auto word = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; };
  if (!word(cfg->step) || !word(cfg->lr_dev) || !word(cfg->norm)) return QLORA_EINVAL;
  const bool s8 = cfg->sfmt == QLORA_S8;
  for (int i = 0; i < count; ++i) {
    const qlora_adamw_item& t = items[i];
    const void* ptrs[4] = {t.p, t.g, t.m, t.v};
    for (const void* p : ptrs)
      if (p == nullptr || !aligned16(p)) return QLORA_EINVAL;
    if ((t.m_scales != nullptr) != s8 || (t.v_scales != nullptr) != s8) return QLORA_EINVAL;
    if (!within(t.decay, 0.0)) return QLORA_EINVAL;
    const size_t n = (size_t)t.n, mb = s8 ? n : 4 * n, sb = s8 ? (n + 31) / 32 : 0;
    Ranges in, out;
    in.add(t.g, 4 * n);
    in.add(cfg->lr_dev, 4);
    out.add(t.p, 4 * n);
    out.add(t.m, mb);
    out.add(t.v, mb);
    out.add(t.m_scales, sb);
    out.add(t.v_scales, sb);
    out.add(cfg->step, 4);
    out.add(cfg->norm, 4);
    out.add(ws, need);
    if (!disjoint(out, in)) return QLORA_EINVAL;
  }
  if (!ws_ok(ws, ws_bytes, need)) return QLORA_EWORKSPACE;
  if (pending_error()) return QLORA_EHIP;
  launch_adamw(*cfg, items, count, ws, static_cast<hipStream_t>(stream));
  return launch_status();
}

}  // extern "C"
