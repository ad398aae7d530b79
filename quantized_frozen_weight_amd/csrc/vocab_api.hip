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
  if (!fits_int(M, L->K) || !fits_int(L->K, L->N) || L->K > (1 << 23)) return QLORA_ERANGE;
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
  const uintptr_t off = itype == QLORA_I64 ? 7u : 3u;      // (a slice of a tensor starts anywhere)
  return ids != nullptr && (reinterpret_cast<uintptr_t>(ids) & off) == 0 ? QLORA_OK : QLORA_EINVAL;
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

// Workspace of the loss, and of its gradient.
struct XentFwdLayout {
  size_t xq, sx, t, rs, part, total;
};
XentFwdLayout xent_fwd_layout(const qlora_linear* L, int vocab, int M) {
  XentFwdLayout w{};
  size_t off = 0;
  w.xq = off; off = align_up(off + (size_t)M * L->K);
  w.sx = off; off = align_up(off + (size_t)M * 4);
  w.t = off; off = align_up(off + (size_t)M * L->r * 4);
  w.rs = off; off = align_up(off + row_split_floats(M, L->K, L->r > 0 ? L->r : 1) * 4);
  w.part = off; off = align_up(off + xent_part_floats(vocab, M) * 4);
  w.total = off;
  return w;
}
struct XentBwdLayout {
  XentPlan plan;
  size_t xq, sx, t, rs, g, dxp, u, up, dbp, pA, smax, total;
};
XentBwdLayout xent_bwd_layout(const qlora_linear* L, int vocab, int M, int dtype) {
  XentBwdLayout w{};
  w.plan = xent_plan(vocab_layer(L), vocab, M, dtype);
  size_t off = 0;
  w.xq = off; off = align_up(off + (size_t)M * L->K);
  w.sx = off; off = align_up(off + (size_t)M * 4);
  w.t = off; off = align_up(off + (size_t)M * L->r * 4);
  w.rs = off; off = align_up(off + row_split_floats(M, L->K, L->r > 0 ? L->r : 1) * 4);
  w.g = off; off = align_up(off + w.plan.g * 2);
  w.dxp = off; off = align_up(off + w.plan.dxp * 4);
  w.u = off; off = align_up(off + w.plan.u * 4);
  w.up = off; off = align_up(off + w.plan.up * 4);
  w.dbp = off; off = align_up(off + w.plan.dbp * 4);
  w.pA = off; off = align_up(off + w.plan.pA * 4);
  w.smax = off; off = align_up(off + w.plan.smax * 4);
  w.total = off;
  return w;
}

// The rows' codes and scales, and (t not NULL) t = x A.
void enqueue_rows(const qlora_linear* L, int M, int dtype, const void* x, int8_t* xq, float* sx, float* t,
                  float* rs, hipStream_t s) {
  launch_rowquant(dtype, x, M, L->K, t != nullptr ? L->A : nullptr, t != nullptr ? L->r : 1, xq, sx, t, s, nullptr,
                  rs);
}

// int32 sums of products of codes up to 127 and 128 stay exact; rows and logits
// that one launch covers.
int check_xent(const qlora_linear* L, int vocab, int M, int dtype) {
  const int st = check_vocab(L, vocab, M, dtype);
  if (st) return st;
  if (L->fmt == QLORA_W8 && L->K > 132096) return QLORA_EUNSUPPORTED;
  return M > kMaxRows || (long)M * vocab > kMaxLogits ? QLORA_ERANGE : QLORA_OK;
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

int qlora_xent_fwd_workspace(const qlora_linear* L, int vocab, int M, int dtype, size_t* bytes) {
  if (bytes == nullptr) return QLORA_EINVAL;
  const int st = check_xent(L, vocab, M, dtype);
  if (st) return st;
  *bytes = xent_fwd_layout(L, vocab, M).total;
  return QLORA_OK;
}

int qlora_xent_fwd(const qlora_linear* L, int vocab, int M, int dtype, const void* x,
                   const void* targets, int itype, float* loss, float* lse, float* t_save, void* ws,
                   size_t ws_bytes, void* stream) {
  size_t need = 0;
  int st = qlora_xent_fwd_workspace(L, vocab, M, dtype, &need);
  if (st) return st;
  st = check_ids(targets, itype);
  if (st) return st;
  if (!x || !aligned16(x) || !loss || !aligned16(loss) || !lse || !aligned16(lse) || !opt16(t_save))
    return QLORA_EINVAL;
  if (t_save != nullptr && L->r < 1) return QLORA_EINVAL;
  if (!ws_ok(ws, ws_bytes, need)) return QLORA_EWORKSPACE;
  Ranges in, out;
  add_vocab(in, L, targets, M, itype);
  in.add(x, (size_t)M * L->K * dtype_bytes(dtype));
  out.add(loss, (size_t)M * 4);
  out.add(lse, (size_t)M * 4);
  out.add(t_save, (size_t)M * L->r * 4);
  out.add(ws, need);
  if (!disjoint(out, in)) return QLORA_EINVAL;
  if (pending_error()) return QLORA_EHIP;
  const XentFwdLayout w = xent_fwd_layout(L, vocab, M);
  hipStream_t s = static_cast<hipStream_t>(stream);
  int8_t* xq = reinterpret_cast<int8_t*>(at(ws, w.xq));
  float* sx = reinterpret_cast<float*>(at(ws, w.sx));
  float* t = L->r < 1 ? nullptr : t_save != nullptr ? t_save : reinterpret_cast<float*>(at(ws, w.t));
  enqueue_rows(L, M, dtype, x, xq, sx, t, reinterpret_cast<float*>(at(ws, w.rs)), s);
  launch_xent_fwd(vocab_layer(L), M, make_ids(targets, itype, vocab), xq, sx, t,
                  reinterpret_cast<float*>(at(ws, w.part)), loss, lse, s);
  return launch_status();
}

int qlora_xent_bwd_workspace(const qlora_linear* L, int vocab, int M, int dtype, size_t* bytes) {
  if (bytes == nullptr) return QLORA_EINVAL;
  const int st = check_xent(L, vocab, M, dtype);
  if (st) return st;
  *bytes = xent_bwd_layout(L, vocab, M, dtype).total;
  return QLORA_OK;
}

int qlora_xent_bwd(const qlora_linear* L, int vocab, int M, int dtype, const void* x,
                   const void* targets, int itype, const float* lse, const float* dloss,
                   const float* t_saved, void* dx, float* dA, float* dB, void* ws, size_t ws_bytes,
                   void* stream) {
  size_t need = 0;
  int st = qlora_xent_bwd_workspace(L, vocab, M, dtype, &need);
  if (st) return st;
  st = check_ids(targets, itype);
  if (st) return st;
  if (!x || !aligned16(x) || !lse || !aligned16(lse) || !dloss || !aligned16(dloss) || !opt16(t_saved) || !opt16(dx))
    return QLORA_EINVAL;
  if (L->r > 0 ? (!dA || !aligned16(dA) || !dB || !aligned16(dB)) : (dA || dB || t_saved || !dx)) return QLORA_EINVAL;
  if (!ws_ok(ws, ws_bytes, need)) return QLORA_EWORKSPACE;
  Ranges in, out;
  add_vocab(in, L, targets, M, itype);
  in.add(x, (size_t)M * L->K * dtype_bytes(dtype));
  in.add(lse, (size_t)M * 4);
  in.add(dloss, (size_t)M * 4);
  in.add(t_saved, (size_t)M * L->r * 4);
  out.add(dx, (size_t)M * L->K * dtype_bytes(dtype));
  out.add(dA, (size_t)L->K * L->r * 4);
  out.add(dB, (size_t)L->N * L->r * 4);
  out.add(ws, need);
  if (!disjoint(out, in)) return QLORA_EINVAL;
  if (pending_error()) return QLORA_EHIP;
  const XentBwdLayout w = xent_bwd_layout(L, vocab, M, dtype);
  hipStream_t s = static_cast<hipStream_t>(stream);
  int8_t* xq = reinterpret_cast<int8_t*>(at(ws, w.xq));
  float* sx = reinterpret_cast<float*>(at(ws, w.sx));
  float* tw = L->r < 1 || t_saved != nullptr ? nullptr : reinterpret_cast<float*>(at(ws, w.t));
  enqueue_rows(L, M, dtype, x, xq, sx, tw, reinterpret_cast<float*>(at(ws, w.rs)), s);
  const auto f = [&](size_t off) { return reinterpret_cast<float*>(at(ws, off)); };
  const XentBuffers buf{reinterpret_cast<uint16_t*>(at(ws, w.g)), f(w.dxp), f(w.u), f(w.up), f(w.dbp), f(w.pA),
                        reinterpret_cast<uint32_t*>(at(ws, w.smax))};
  launch_xent_bwd(vocab_layer(L), M, dtype, make_ids(targets, itype, vocab), x, xq, sx,
                  tw != nullptr ? tw : t_saved, lse, dloss, w.plan, buf, dx, dA, dB, s);
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

namespace {
int check_moment(const void* x, const void* codes, const void* scales, int64_t n, int which, int dtype) {
  const int st = check_dtype(dtype);
  if (st) return st;
  if (n < 1 || (which != QLORA_MOMENT1 && which != QLORA_MOMENT2)) return QLORA_EINVAL;
  if (n > (1LL << 30)) return QLORA_ERANGE;
  return x && aligned16(x) && codes && aligned16(codes) && scales ? QLORA_OK : QLORA_EINVAL;
}
}  // namespace

int qlora_moment_read(const uint8_t* codes, const uint8_t* scales, int64_t n, int which, int dtype, void* x,
                      void* stream) {
  const int st = check_moment(x, codes, scales, n, which, dtype);
  if (st) return st;
  Ranges in, out;
  in.add(codes, (size_t)n);
  in.add(scales, (size_t)(n + 31) / 32);
  out.add(x, (size_t)n * dtype_bytes(dtype));
  if (!disjoint(out, in)) return QLORA_EINVAL;
  if (pending_error()) return QLORA_EHIP;
  launch_moment_read(codes, scales, n, which, dtype, x, static_cast<hipStream_t>(stream));
  return launch_status();
}

int qlora_moment_write(const void* x, int64_t n, int which, int dtype, uint8_t* codes, uint8_t* scales,
                       void* stream) {
  const int st = check_moment(x, codes, scales, n, which, dtype);
  if (st) return st;
  Ranges in, out;
  in.add(x, (size_t)n * dtype_bytes(dtype));
  out.add(codes, (size_t)n);
  out.add(scales, (size_t)(n + 31) / 32);
  if (!disjoint(out, in)) return QLORA_EINVAL;
  if (pending_error()) return QLORA_EHIP;
  launch_moment_write(x, n, which, dtype, codes, scales, static_cast<hipStream_t>(stream));
  return launch_status();
}

}  // extern "C"
