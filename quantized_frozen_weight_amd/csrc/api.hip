// C ABI of libqlora: argument validation, workspace layout, and the kernel
// sequence of each call. Contract and citations: include/qlora.h.
#include <hip/hip_runtime.h>

#include <mutex>

#include "abi.hpp"
#include "epilogue.hpp"
#include "launch.hpp"
#include "outlier.hpp"
#include "qlora.h"

namespace {

using namespace qlora;

int check_shape(int M, int K, int N, int r) {
  if (M < 1 || K < 16 || N < 16 || r < 1 || r > 32) return QLORA_EINVAL;
  if (K % 16 || N % 16) return QLORA_EINVAL;
  if (!fits_int(M, K) || !fits_int(M, N) || !fits_int(K, N)) return QLORA_ERANGE;
  return QLORA_OK;
}

// Validate a layer description (weights only; data pointers are checked by
// the individual calls).
int check_linear(const qlora_linear* L, int M, int dtype) {
  if (L == nullptr) return QLORA_EINVAL;
  int st = check_dtype(dtype);
  if (st) return st;
  st = check_shape(M, L->K, L->N, L->r);
  if (st) return st;
  if (L->fmt != QLORA_W8 && L->fmt != QLORA_W4G128 && L->fmt != QLORA_W8O) return QLORA_EINVAL;
  if (L->fmt == QLORA_W8O) {
    if (dtype != QLORA_BF16) return QLORA_EUNSUPPORTED;
    if (L->N >= (1 << 24)) return QLORA_EUNSUPPORTED;
  }
  if (L->fmt == QLORA_W4G128) {
    if (L->K % 128) return QLORA_EINVAL;
    if (dtype != QLORA_BF16) return QLORA_EUNSUPPORTED;
    if (L->K > 128 * kW4MaxGroups) return QLORA_EUNSUPPORTED;
  }
  if (L->heads < 0 || (L->heads > 1 && L->N % L->heads)) return QLORA_EINVAL;
  if (L->heads > 1 && (L->N / L->heads) % 64) return QLORA_EUNSUPPORTED;
  const void* ptrs[4] = {L->codes, L->scales, L->A, L->B};
  for (const void* p : ptrs)
    if (p == nullptr || !aligned16(p)) return QLORA_EINVAL;
  return QLORA_OK;
}

// Head width of B / dB (and of W at quantization): N for a one-head layer.
inline int head_width(const qlora_linear* L) {
  return L->heads > 1 ? L->N / L->heads : L->N;
}

inline float lora_s(const qlora_linear* L) {
  return L->alpha / (float)L->r;   // one float32 divide
}

struct FwdLayout {
  size_t xq, sx, t, asum, pacc, pcorr, rs, total;
};
FwdLayout fwd_layout(const qlora_linear* L, int M) {
  FwdLayout w{};
  size_t off = 0;
  // activation codes and scales: the int8 product, and the integer forward
  // of 4-bit layers (the few-row forward, which keeps its codes in LDS, has
  // its slices of t there)
  w.xq = off; off = align_up(off + (size_t)M * L->K);
  w.sx = off; off = align_up(off + (size_t)M * 4);
  w.t = off; off = align_up(off + (size_t)M * L->r * 4);
  // row sums of the activation codes (affine weights)
  w.asum = off; off = align_up(off + (L->fmt == QLORA_W8O ? (size_t)M * 4 : 0));
  // split contraction of the int8 product (0 bytes when it does not split):
  // int32 partial sums, and the affine weights' partial corrections
  // (4-bit weights: the float32 partial sums of the split 4-bit product)
  const bool w8 = L->fmt == QLORA_W8, w8o = L->fmt == QLORA_W8O;
  const size_t nsplit = (w8 || w8o) ? fwd_split_ints(M, L->N, L->K, w8o)
                                    : fwd_w4_split_floats(M, L->N, L->K);
  w.pacc = off; off = align_up(off + nsplit * 4);
  w.pcorr = off; off = align_up(off + (w8o ? nsplit * 4 : 0));
  // the row pass of long rows split over k (0 bytes for other widths)
  w.rs = off; off = align_up(off + row_split_floats(M, L->K, L->r) * 4);
  w.total = off;
  return w;
}

struct BwdLayout {
  size_t t, u, pB, pA, pdx, pu, rs, total;
};
// Partial sums of dA and dB: one per split of the rows. The fused int8
// backward splits by row block (at least 64 rows), the other paths into at
// most as many splits, so ceil(M / 64) covers both.
inline size_t partial_floats(int M, int r, int C) {
  return (size_t)((M + 63) / 64) * (size_t)r * (size_t)C;
}
BwdLayout bwd_layout(const qlora_linear* L, int M, int dtype) {
  BwdLayout w{};
  size_t off = 0;
  // the partial sums first: they are the only bytes that outlive a call
  // (qlora_bwd_partials_bytes), everything after them is scratch
  w.pB = off; off = align_up(off + partial_floats(M, L->r, L->N) * 4);
  w.pA = off; off = align_up(off + partial_floats(M, L->r, L->K) * 4);
  w.t = off; off = align_up(off + (size_t)M * L->r * 4);
  w.u = off; off = align_up(off + (size_t)M * L->r * 4);
  // split contraction of the bf16 input gradient (0 bytes when it does not split)
  size_t fdx = 0, fu = 0;
  if (dtype == QLORA_BF16) bwd_split_sizes(M, L->K, L->N, L->r, &fdx, &fu);
  w.pdx = off; off = align_up(off + fdx * 4);
  w.pu = off; off = align_up(off + fu * 4);
  // recomputing t over long rows split over k (0 bytes for other widths)
  w.rs = off; off = align_up(off + row_split_floats(M, L->K, L->r) * 4);
  w.total = off;
  return w;
}

// Whether qlora_bwd_epi lays the weight out first, and the workspace it then
// needs after a backward's own.
bool lays_out(const qlora_linear* L, int M, int dtype) {
  return dtype == QLORA_BF16 && bwd_tn_takes(L->fmt, M, L->K, L->N);
}
size_t bwd_epi_bytes(const qlora_linear* L, int M, int dtype) {
  return bwd_layout(L, M, dtype).total + (lays_out(L, M, dtype) ? bwd_tn_bytes(L->K, L->N, L->r) : 0);
}

// Scratch of qlora_bwd_noalloc: a static device array, one copy per GPU the
// library runs on, held until the process ends. In host code `scratch`
// names a host-side stand-in, not device memory: its device address is taken
// once per device with hipGetSymbolAddress (that device current) and only
// that address is passed to kernels.
constexpr size_t kNoAllocScratch = QLORA_NOALLOC_SCRATCH_BYTES;
static __device__ __align__(256) int8_t scratch[kNoAllocScratch];
constexpr int kMaxDevices = 64;
std::mutex g_scratch_mu;
void* g_scratch_dev[kMaxDevices] = {};

// The current device's address of `scratch`, looked up on the first call
// on that device.
int scratch_address(void** out) {
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return QLORA_EHIP;
  std::lock_guard<std::mutex> lock(g_scratch_mu);
  if (g_scratch_dev[dev] == nullptr) {
    void* p = nullptr;
    if (hipGetSymbolAddress(&p, HIP_SYMBOL(scratch)) != hipSuccess || p == nullptr)
      return QLORA_EHIP;
    g_scratch_dev[dev] = p;
  }
  *out = g_scratch_dev[dev];
  return QLORA_OK;
}

// Optional timing marks around a call's main product kernel.
void mark(void* ev, hipStream_t s) {
  if (ev != nullptr) (void)hipEventRecord(static_cast<hipEvent_t>(ev), s);
}

// Row-block count of the adapter-gradient partial sums: the fused bf16
// backward's row tile; the other paths split the rows the same way so that
// the combine needs nothing but (L, M, dtype).
int bwd_splits(const qlora_linear* L, int M) {
  const int bm = bwd_row_block(L->fmt, M, L->K, L->N, L->r);
  return (M + bm - 1) / bm;
}

int bwd_check_ws(const qlora_linear* L, int M, int dtype, void* ws, size_t ws_bytes) {
  const BwdLayout w = bwd_layout(L, M, dtype);
  if (ws_bytes < w.total || !ws || !aligned16(ws)) return QLORA_EWORKSPACE;
  return QLORA_OK;
}

// The launches of a backward's first half, arguments validated: dx (NULL:
// none) and the partial sums of dA and dB in ws. x, or (xq not NULL) its row
// checkpoint; ge (NULL: none) on dx.
void enqueue_bwd_partial(const qlora_linear* L, int M, int dtype, const void* x, const int8_t* xq,
                         const float* sx, const void* dy, const float* t_saved, const GradEpi* ge,
                         void* dx, void* ws, hipStream_t s, int repeats, void* ev_start,
                         void* ev_stop, bool laid_out = false) {
  const BwdLayout w = bwd_layout(L, M, dtype);
  const float sc = lora_s(L);
  float* u = reinterpret_cast<float*>(at(ws, w.u));
  const float* t = t_saved;
  if (t == nullptr) {
    float* tw = reinterpret_cast<float*>(at(ws, w.t));
    launch_lora_down(dtype, x, M, L->K, L->A, L->r, tw, s, reinterpret_cast<float*>(at(ws, w.rs)));
    t = tw;
  }
  float* partB = reinterpret_cast<float*>(at(ws, w.pB));
  float* partA = reinterpret_cast<float*>(at(ws, w.pA));
  if (laid_out) {
    launch_bwd_tn(L->fmt, M, L->K, L->N, static_cast<const uint16_t*>(dy), L->codes, L->scales, L->B,
                  head_width(L), L->A, t, static_cast<const uint16_t*>(x), xq, sx, L->r, sc,
                  static_cast<uint16_t*>(dx), partA, partB, reinterpret_cast<float*>(at(ws, w.pdx)),
                  reinterpret_cast<float*>(at(ws, w.pu)), at(ws, w.total), *ge, s);
    return;
  }
  if (dtype == QLORA_BF16 && dx != nullptr) {
    // one launch: dx, u, and the per-row-block partial sums of dA and dB
    mark(ev_start, s);
    for (int rep = 0; rep < repeats; ++rep)
      launch_bwd_fused(L->fmt, M, L->K, L->N, static_cast<const uint16_t*>(dy),
                       L->codes, L->scales, L->B, head_width(L), L->A, t,
                       static_cast<const uint16_t*>(x), L->r, sc,
                       static_cast<uint16_t*>(dx), partA, partB,
                       reinterpret_cast<float*>(at(ws, w.pdx)),
                       reinterpret_cast<float*>(at(ws, w.pu)), s, xq, sx, ge);
    mark(ev_stop, s);
    return;
  }
  launch_bwd_rows(dtype, dy, M, L->N, L->B, head_width(L), L->r, nullptr, nullptr, u, s);
  SkinnyJobs sk = make_adapter_grad_jobs(M, L->r, sc, t, dy, L->N, nullptr, partB,
                                         u, xq != nullptr ? static_cast<const void*>(xq) : x, L->K,
                                         nullptr, partA);
  sk.sx = sx;
  sk.nsplit = bwd_splits(L, M);
  sk.rows_per_split = (M + sk.nsplit - 1) / sk.nsplit;
  sk.rows_per_split = (sk.rows_per_split + 3) / 4 * 4;
  // float32 compute (int8 weights): the adapter-gradient stage 1, then the
  // float32 input gradient; or no input gradient at all
  launch_skinny_stage1(dtype, sk, s);
  mark(ev_start, s);
  if (dx != nullptr)
    for (int rep = 0; rep < repeats; ++rep)
      launch_gemm_dx_f32(M, L->K, L->N, static_cast<const float*>(dy),
                         static_cast<const int8_t*>(L->codes),
                         static_cast<const float*>(L->scales), u, L->A, L->r,
                         sc, static_cast<float*>(dx), s, ge);
  mark(ev_stop, s);
}

// ---- the epilogue and checkpoint calls -------------------------------------

void add_layer(Ranges& in, const qlora_linear* L) {
  size_t cb = 0, sb = 0;
  qlora_weight_bytes(L->K, L->N, L->fmt, &cb, &sb);
  in.add(L->codes, cb);
  in.add(L->scales, sb);
  in.add(L->A, (size_t)L->K * L->r * 4);
  in.add(L->B, (size_t)L->N * L->r * 4);
}

inline bool pair_ok(const void* codes, const void* scales) {
  return (codes == nullptr) == (scales == nullptr) && opt16(codes) && opt16(scales);
}

// The longest contraction whose int8 sums cannot pass their registers: int32
// products of codes up to 127 and 128 (127 * 128 K < 2^31) and, for the affine
// weights, float32 sums of the row's codes (127 K < 2^24).
constexpr int kI8ExactK = 132096;
inline bool exact_sums(const qlora_linear* L) { return L->fmt == QLORA_W4G128 || L->K <= kI8ExactK; }

inline bool act_ok(int act) { return act >= QLORA_ACT_NONE && act <= QLORA_ACT_SILU; }

// The forward epilogue: pointers checked, and its ranges added. in_y: y given
// as the residual itself.
int check_epilogue(const qlora_epilogue* e, int M, int K, int N, int dtype, const void* y,
                   Ranges& in, Ranges& out) {
  if (e == nullptr || !act_ok(e->act)) return QLORA_EINVAL;
  if (!opt16(e->bias) || !opt16(e->residual) || !opt16(e->z)) return QLORA_EINVAL;
  if (!pair_ok(e->z_codes, e->z_scales) || !pair_ok(e->x_codes, e->x_scales)) return QLORA_EINVAL;
  const size_t mn = (size_t)M * N;
  in.add(e->bias, (size_t)N * 4);
  if (e->residual != y) in.add(e->residual, mn * dtype_bytes(dtype));
  out.add(e->z, mn * dtype_bytes(dtype));
  out.add(e->z_codes, mn);
  out.add(e->z_scales, (size_t)M * group_count(N));
  out.add(e->x_codes, (size_t)M * K);
  out.add(e->x_scales, (size_t)M * 4);
  return QLORA_OK;
}

FwdEpi fwd_epi(const qlora_epilogue* e, int N) {
  FwdEpi f{};
  f.act = act_params(e->act);
  f.bias = e->bias; f.res = e->residual; f.z = e->z;
  f.zc = e->z_codes; f.zs = e->z_scales; f.zg = group_count(N);
  return f;
}

// The int8 and affine products of a call, from x's codes and scales.
void enqueue_fwd_i8(const qlora_linear* L, int M, int dtype, const int8_t* xq, const float* sx,
                    const float* asum, const float* t, const FwdEpi& epi, void* y, void* ws,
                    const FwdLayout& w, hipStream_t s) {
  const int8_t* codes = static_cast<const int8_t*>(L->codes);
  int32_t* pacc = reinterpret_cast<int32_t*>(at(ws, w.pacc));
  if (L->fmt == QLORA_W8)
    launch_gemm_fwd_w8(dtype, M, L->N, L->K, xq, codes, sx, static_cast<const float*>(L->scales), t,
                       L->B, head_width(L), L->r, lora_s(L), y, nullptr, pacc, &epi, s);
  else
    launch_gemm_fwd_w8o(M, L->N, L->K, xq, codes, sx, asum, L->scales, t, L->B, head_width(L), L->r,
                        lora_s(L), static_cast<uint16_t*>(y), pacc,
                        reinterpret_cast<float*>(at(ws, w.pcorr)), &epi, s);
}

// z of a gradient: given in exactly one form where act needs it, else not at
// all.
int check_z(int act, const void* z, const int8_t* zc, const uint8_t* zs) {
  if (!act_ok(act) || !opt16(z) || !pair_ok(zc, zs)) return QLORA_EINVAL;
  const int given = (z != nullptr) + (zc != nullptr);
  return given == (act == QLORA_ACT_NONE ? 0 : 1) ? QLORA_OK : QLORA_EINVAL;
}

GradEpi grad_epi(int act, const void* z, const int8_t* zc, const uint8_t* zs, const void* add, int C) {
  GradEpi g{};
  g.act = act_params(act);
  g.z = z; g.zc = zc; g.zs = zs; g.zg = group_count(C); g.add = add;
  return g;
}

int bwd_epi_check(const qlora_linear* L, int M, int dtype, const void* x, const int8_t* x_codes,
                  const float* x_scales, const void* dy, const float* t_saved,
                  const qlora_grad_epilogue* g, void* dx, float* dA, float* dB, void* ws,
                  size_t ws_bytes) {
  int st = check_linear(L, M, dtype);
  if (st) return st;
  if (!dy || !aligned16(dy) || !opt16(x) || !opt16(t_saved) || !opt16(dx)) return QLORA_EINVAL;
  if (!pair_ok(x_codes, x_scales) || (x != nullptr) == (x_codes != nullptr)) return QLORA_EINVAL;
  if (x_codes != nullptr && t_saved == nullptr) return QLORA_EINVAL;
  const size_t mk = (size_t)M * L->K, es = dtype_bytes(dtype);
  Ranges in, out;
  if (g != nullptr) {
    if (dx == nullptr || !opt16(g->add)) return QLORA_EINVAL;
    st = check_z(g->act, g->z, g->z_codes, g->z_scales);
    if (st) return st;
    in.add(g->z, mk * es);
    in.add(g->z_codes, mk);
    in.add(g->z_scales, (size_t)M * group_count(L->K));
    if (g->add != dx) in.add(g->add, mk * es);
  }
  const size_t need = bwd_epi_bytes(L, M, dtype);
  if (ws_bytes < need || !ws || !aligned16(ws)) return QLORA_EWORKSPACE;
  add_layer(in, L);
  in.add(x, mk * es);
  in.add(x_codes, mk);
  in.add(x_scales, (size_t)M * 4);
  in.add(dy, (size_t)M * L->N * es);
  in.add(t_saved, (size_t)M * L->r * 4);
  out.add(dx, mk * es);
  out.add(dA, (size_t)L->K * L->r * 4);
  out.add(dB, (size_t)L->N * L->r * 4);
  out.add(ws, need);
  return disjoint(out, in) ? QLORA_OK : QLORA_EINVAL;
}

void enqueue_bwd_epi(const qlora_linear* L, int M, int dtype, const void* x, const int8_t* x_codes,
                     const float* x_scales, const void* dy, const float* t_saved,
                     const qlora_grad_epilogue* g, void* dx, void* ws, hipStream_t s) {
  // (x dense and nothing done to dx: qlora_bwd's own kernels)
  const bool plain = x != nullptr && (g == nullptr || (g->act == QLORA_ACT_NONE && g->add == nullptr));
  const GradEpi ge = g != nullptr ? grad_epi(g->act, g->z, g->z_codes, g->z_scales, g->add, L->K) : GradEpi{};
  enqueue_bwd_partial(L, M, dtype, x, x_codes, x_scales, dy, t_saved, plain ? nullptr : &ge, dx, ws, s,
                      1, nullptr, nullptr, !plain && dx != nullptr && lays_out(L, M, dtype));
}


}  // namespace

extern "C" {

const char* qlora_status_str(int status) {
  switch (status) {
    case QLORA_OK: return "ok";
    case QLORA_EINVAL: return "invalid argument";
    case QLORA_EUNSUPPORTED: return "unsupported combination";
    case QLORA_EWORKSPACE: return "workspace too small";
    case QLORA_ERANGE: return "size out of range";
    case QLORA_EHIP: return "HIP launch failure";
    default: return "unknown status";
  }
}

int qlora_weight_bytes(int K, int N, int fmt, size_t* codes_bytes,
                       size_t* scale_bytes) {
  if (codes_bytes == nullptr || scale_bytes == nullptr) return QLORA_EINVAL;
  if (K < 16 || N < 16 || K % 16 || N % 16) return QLORA_EINVAL;
  if (!fits_int(K, N)) return QLORA_ERANGE;
  if (fmt == QLORA_W8) {
    *codes_bytes = (size_t)K * N;
    *scale_bytes = (size_t)N * 4;
    return QLORA_OK;
  }
  if (fmt == QLORA_W4G128) {
    if (K % 128) return QLORA_EINVAL;
    *codes_bytes = (size_t)K * N / 2;
    *scale_bytes = (size_t)N * (K / 128) * 2;
    return QLORA_OK;
  }
  if (fmt == QLORA_W8O) {
    *codes_bytes = (size_t)K * N;
    *scale_bytes = w8o_layout(K, N).total;
    return QLORA_OK;
  }
  return QLORA_EINVAL;
}

int qlora_outlier_layout(int K, int N, size_t* rowptr_off, size_t* col_off,
                         size_t* val_off, int32_t* capacity) {
  if (!rowptr_off || !col_off || !val_off || !capacity) return QLORA_EINVAL;
  if (K < 16 || N < 16 || K % 16 || N % 16) return QLORA_EINVAL;
  if (!fits_int(K, N)) return QLORA_ERANGE;
  const W8OLayout L = w8o_layout(K, N);
  *rowptr_off = L.rowptr;
  *col_off = L.col;
  *val_off = L.val;
  *capacity = L.cap;
  return QLORA_OK;
}

int qlora_quantize(const float* W, int K, int N, int fmt, void* codes,
                   void* scales, void* stream) {
  return qlora_quantize_heads(W, 1, K, N, fmt, codes, scales, stream);
}

int qlora_quantize_heads(const float* W, int heads, int K, int N, int fmt,
                         void* codes, void* scales, void* stream) {
  size_t cb, sb;
  int st = qlora_weight_bytes(K, N, fmt, &cb, &sb);
  if (st) return st;
  if (heads < 1 || N % heads) return QLORA_EINVAL;
  if (heads > 1 && (N / heads) % 64) return QLORA_EUNSUPPORTED;
  if (fmt == QLORA_W8O && (heads > 1 || N >= (1 << 24))) return QLORA_EUNSUPPORTED;
  const int hd = N / heads;
  if (!W || !codes || !scales || !aligned16(W) || !aligned16(codes) || !aligned16(scales))
    return QLORA_EINVAL;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (pending_error()) return QLORA_EHIP;
  if (fmt == QLORA_W8)
    launch_quantize_w8(W, K, N, hd, static_cast<int8_t*>(codes),
                       static_cast<float*>(scales), s);
  else if (fmt == QLORA_W8O)
    launch_quantize_w8o(W, K, N, static_cast<int8_t*>(codes), scales, s);
  else
    launch_quantize_w4(W, K, N, hd, static_cast<uint8_t*>(codes),
                       static_cast<_Float16*>(scales), s);
  return launch_status();
}

int qlora_fwd_workspace(const qlora_linear* L, int M, int dtype, size_t* bytes) {
  if (bytes == nullptr) return QLORA_EINVAL;
  int st = check_linear(L, M, dtype);
  if (st) return st;
  *bytes = fwd_layout(L, M).total;
  return QLORA_OK;
}

int qlora_fwd_timed(const qlora_linear* L, int M, int dtype, const void* x,
                    void* y, float* t_save, void* ws, size_t ws_bytes,
                    void* stream, int repeats, void* ev_start, void* ev_stop) {
  int st = check_linear(L, M, dtype);
  if (st) return st;
  if (repeats < 1) return QLORA_EINVAL;
  if (!x || !y || !aligned16(x) || !aligned16(y)) return QLORA_EINVAL;
  if (t_save && !aligned16(t_save)) return QLORA_EINVAL;
  const FwdLayout w = fwd_layout(L, M);
  if (ws_bytes < w.total || (w.total && (!ws || !aligned16(ws)))) return QLORA_EWORKSPACE;
  hipStream_t s = static_cast<hipStream_t>(stream);
  float* t = t_save ? t_save : reinterpret_cast<float*>(at(ws, w.t));
  if (pending_error()) return QLORA_EHIP;
  if (L->fmt == QLORA_W8) {
    int8_t* xq = reinterpret_cast<int8_t*>(at(ws, w.xq));
    float* sx = reinterpret_cast<float*>(at(ws, w.sx));
    launch_rowquant(dtype, x, M, L->K, L->A, L->r, xq, sx, t, s, nullptr,
                    reinterpret_cast<float*>(at(ws, w.rs)));
    mark(ev_start, s);
    for (int rep = 0; rep < repeats; ++rep)
      launch_gemm_fwd_w8(dtype, M, L->N, L->K, xq,
                         static_cast<const int8_t*>(L->codes), sx,
                         static_cast<const float*>(L->scales), t, L->B, head_width(L), L->r,
                         lora_s(L), y, nullptr, reinterpret_cast<int32_t*>(at(ws, w.pacc)), nullptr, s);
    mark(ev_stop, s);
  } else if (L->fmt == QLORA_W8O) {
    int8_t* xq = reinterpret_cast<int8_t*>(at(ws, w.xq));
    float* sx = reinterpret_cast<float*>(at(ws, w.sx));
    float* asum = reinterpret_cast<float*>(at(ws, w.asum));
    launch_rowquant(dtype, x, M, L->K, L->A, L->r, xq, sx, t, s, asum,
                    reinterpret_cast<float*>(at(ws, w.rs)));
    mark(ev_start, s);
    for (int rep = 0; rep < repeats; ++rep)
      launch_gemm_fwd_w8o(M, L->N, L->K, xq, static_cast<const int8_t*>(L->codes), sx, asum,
                          L->scales, t, L->B, head_width(L), L->r, lora_s(L),
                          static_cast<uint16_t*>(y), reinterpret_cast<int32_t*>(at(ws, w.pacc)),
                          reinterpret_cast<float*>(at(ws, w.pcorr)), nullptr, s);
    mark(ev_stop, s);
  } else {
    launch_lora_down(dtype, x, M, L->K, L->A, L->r, t, s, reinterpret_cast<float*>(at(ws, w.rs)));
    mark(ev_start, s);
    for (int rep = 0; rep < repeats; ++rep)
      launch_gemm_fwd_w4(M, L->N, L->K, static_cast<const uint16_t*>(x),
                         static_cast<const uint8_t*>(L->codes),
                         static_cast<const _Float16*>(L->scales), t, L->B, head_width(L), L->r,
                         lora_s(L), static_cast<uint16_t*>(y),
                         reinterpret_cast<float*>(at(ws, w.pacc)), nullptr, s);
    mark(ev_stop, s);
  }
  return launch_status();
}

int qlora_fwd(const qlora_linear* L, int M, int dtype, const void* x, void* y,
              float* t_save, void* ws, size_t ws_bytes, void* stream) {
  return qlora_fwd_timed(L, M, dtype, x, y, t_save, ws, ws_bytes, stream, 1,
                         nullptr, nullptr);
}

int qlora_fwd_a8w4(const qlora_linear* L, int M, int dtype, const void* x, void* y,
                   float* t_save, void* ws, size_t ws_bytes, void* stream) {
  int st = check_linear(L, M, dtype);
  if (st) return st;
  if (L->fmt != QLORA_W4G128) return QLORA_EUNSUPPORTED;
  if (!x || !y || !aligned16(x) || !aligned16(y)) return QLORA_EINVAL;
  if (t_save && !aligned16(t_save)) return QLORA_EINVAL;
  const FwdLayout w = fwd_layout(L, M);
  if (ws_bytes < w.total || !ws || !aligned16(ws)) return QLORA_EWORKSPACE;
  hipStream_t s = static_cast<hipStream_t>(stream);
  float* t = t_save ? t_save : reinterpret_cast<float*>(at(ws, w.t));
  int8_t* xq = reinterpret_cast<int8_t*>(at(ws, w.xq));
  float* sx = reinterpret_cast<float*>(at(ws, w.sx));
  if (pending_error()) return QLORA_EHIP;
  launch_rowquant(dtype, x, M, L->K, L->A, L->r, xq, sx, t, s, nullptr,
                  reinterpret_cast<float*>(at(ws, w.rs)));
  launch_gemm_fwd_a8w4(M, L->N, L->K, xq, sx, static_cast<const uint8_t*>(L->codes),
                       static_cast<const _Float16*>(L->scales), t, L->B, head_width(L), L->r, lora_s(L),
                       static_cast<uint16_t*>(y), nullptr, s);
  return launch_status();
}

int qlora_bwd_workspace(const qlora_linear* L, int M, int dtype, size_t* bytes) {
  if (bytes == nullptr) return QLORA_EINVAL;
  int st = check_linear(L, M, dtype);
  if (st) return st;
  *bytes = bwd_layout(L, M, dtype).total;
  return QLORA_OK;
}

int qlora_bwd_partial_timed(const qlora_linear* L, int M, int dtype, const void* x,
                            const void* dy, const float* t_saved, void* dx, void* ws,
                            size_t ws_bytes, void* stream, int repeats, void* ev_start,
                            void* ev_stop) {
  int st = check_linear(L, M, dtype);
  if (st) return st;
  if (repeats < 1) return QLORA_EINVAL;
  if (!x || !dy) return QLORA_EINVAL;
  if (!aligned16(x) || !aligned16(dy)) return QLORA_EINVAL;
  if ((t_saved && !aligned16(t_saved)) || (dx && !aligned16(dx))) return QLORA_EINVAL;
  st = bwd_check_ws(L, M, dtype, ws, ws_bytes);
  if (st) return st;
  if (pending_error()) return QLORA_EHIP;
  enqueue_bwd_partial(L, M, dtype, x, nullptr, nullptr, dy, t_saved, nullptr, dx, ws,
                      static_cast<hipStream_t>(stream), repeats, ev_start, ev_stop);
  return launch_status();
}

int qlora_bwd_partial(const qlora_linear* L, int M, int dtype, const void* x,
                      const void* dy, const float* t_saved, void* dx, void* ws,
                      size_t ws_bytes, void* stream) {
  return qlora_bwd_partial_timed(L, M, dtype, x, dy, t_saved, dx, ws, ws_bytes, stream,
                                 1, nullptr, nullptr);
}

namespace {
int finish_check(const qlora_linear* L, int M, int dtype, float* dA, float* dB, void* ws,
                 size_t ws_bytes) {
  int st = check_linear(L, M, dtype);
  if (st) return st;
  if (!dA || !dB || !aligned16(dA) || !aligned16(dB)) return QLORA_EINVAL;
  return bwd_check_ws(L, M, dtype, ws, ws_bytes);
}

// The combine of one layer's partial sums (left in ws by qlora_bwd_partial).
SkinnyJobs finish_jobs(const qlora_linear* L, int M, int dtype, float* dA, float* dB,
                       void* ws) {
  const BwdLayout w = bwd_layout(L, M, dtype);
  SkinnyJobs sk{};
  sk.njobs = 2; sk.M = M; sk.r = L->r; sk.s = lora_s(L);
  sk.nsplit = bwd_splits(L, M);
  sk.partial[0] = reinterpret_cast<float*>(at(ws, w.pB)); sk.C[0] = L->N;
  sk.out[0] = dB; sk.transpose[0] = 0; sk.hd0 = head_width(L);
  sk.partial[1] = reinterpret_cast<float*>(at(ws, w.pA)); sk.C[1] = L->K;
  sk.out[1] = dA; sk.transpose[1] = 1;
  return sk;
}
}  // namespace

int qlora_bwd_finish(const qlora_linear* L, int M, int dtype, float* dA, float* dB,
                     void* ws, size_t ws_bytes, void* stream) {
  const int st = finish_check(L, M, dtype, dA, dB, ws, ws_bytes);
  if (st) return st;
  if (pending_error()) return QLORA_EHIP;
  launch_skinny_stage2(finish_jobs(L, M, dtype, dA, dB, ws), static_cast<hipStream_t>(stream));
  return launch_status();
}

int qlora_bwd_partials_bytes(const qlora_linear* L, int M, int dtype, size_t* bytes) {
  if (!bytes) return QLORA_EINVAL;
  const int st = check_linear(L, M, dtype);
  if (st) return st;
  *bytes = bwd_layout(L, M, dtype).t;
  return QLORA_OK;
}

int qlora_bwd_finish_batch(const qlora_finish_item* items, int count, void* stream) {
  if (!items || count < 1) return QLORA_EINVAL;
  for (int i = 0; i < count; ++i) {
    const qlora_finish_item& it = items[i];
    const int st = finish_check(it.L, it.M, it.dtype, it.dA, it.dB, it.ws, it.ws_bytes);
    if (st) return st;
  }
  if (pending_error()) return QLORA_EHIP;
  SkinnyJobs sk[kFinishBatch];
  for (int i0 = 0; i0 < count; i0 += kFinishBatch) {
    const int n = count - i0 < kFinishBatch ? count - i0 : kFinishBatch;
    for (int i = 0; i < n; ++i) {
      const qlora_finish_item& it = items[i0 + i];
      sk[i] = finish_jobs(it.L, it.M, it.dtype, it.dA, it.dB, it.ws);
    }
    launch_finish_batch(sk, n, static_cast<hipStream_t>(stream));
  }
  return launch_status();
}

int qlora_bwd_timed(const qlora_linear* L, int M, int dtype, const void* x,
                    const void* dy, const float* t_saved, void* dx, float* dA,
                    float* dB, void* ws, size_t ws_bytes, void* stream,
                    int repeats, void* ev_start, void* ev_stop) {
  // both halves are validated before either is enqueued
  int st = check_linear(L, M, dtype);
  if (st) return st;
  if (!dA || !dB || !aligned16(dA) || !aligned16(dB)) return QLORA_EINVAL;
  st = qlora_bwd_partial_timed(L, M, dtype, x, dy, t_saved, dx, ws, ws_bytes, stream,
                               repeats, ev_start, ev_stop);
  if (st) return st;
  return qlora_bwd_finish(L, M, dtype, dA, dB, ws, ws_bytes, stream);
}

int qlora_bwd(const qlora_linear* L, int M, int dtype, const void* x,
              const void* dy, const float* t_saved, void* dx, float* dA,
              float* dB, void* ws, size_t ws_bytes, void* stream) {
  return qlora_bwd_timed(L, M, dtype, x, dy, t_saved, dx, dA, dB, ws, ws_bytes,
                         stream, 1, nullptr, nullptr);
}

const char* qlora_bwd_main_kernel(const qlora_linear* L, int M, int dtype) {
  if (check_linear(L, M, dtype)) return nullptr;
  if (dtype == QLORA_BF16) return bwd_fused_kernel_name(L->fmt, M, L->K, L->N, L->r);
  return "gemm_dx_f32_kernel";
}

int qlora_bwd_noalloc(const qlora_linear* L, int M, int dtype, const void* x,
                      const void* dy, const float* t_saved, void* dx, float* dA,
                      float* dB, void* stream) {
  int st = check_linear(L, M, dtype);
  if (st) return st;
  if (bwd_layout(L, M, dtype).total > kNoAllocScratch) return QLORA_EWORKSPACE;
  if (pending_error()) return QLORA_EHIP;
  void* ws = nullptr;
  st = scratch_address(&ws);
  if (st) return st;
  return qlora_bwd(L, M, dtype, x, dy, t_saved, dx, dA, dB, ws, kNoAllocScratch, stream);
}

int qlora_ckpt_bytes(int M, int C, int cfmt, size_t* codes_bytes, size_t* scale_bytes) {
  if (codes_bytes == nullptr || scale_bytes == nullptr) return QLORA_EINVAL;
  if (M < 1 || C < 16 || C % 16) return QLORA_EINVAL;
  if (!fits_int(M, C)) return QLORA_ERANGE;
  if (cfmt != QLORA_C8ROW && cfmt != QLORA_C8G32) return QLORA_EINVAL;
  *codes_bytes = (size_t)M * C;
  *scale_bytes = cfmt == QLORA_C8ROW ? (size_t)M * 4 : (size_t)M * group_count(C);
  return QLORA_OK;
}

int qlora_ckpt_write(const void* x, int M, int C, int dtype, int cfmt, int8_t* codes,
                     void* scales, void* stream) {
  size_t cb, sb;
  int st = check_dtype(dtype);
  if (st) return st;
  st = qlora_ckpt_bytes(M, C, cfmt, &cb, &sb);
  if (st) return st;
  if (!x || !codes || !scales || !aligned16(x) || !aligned16(codes) || !aligned16(scales))
    return QLORA_EINVAL;
  Ranges in, out;
  in.add(x, cb * dtype_bytes(dtype));
  out.add(codes, cb);
  out.add(scales, sb);
  if (!disjoint(out, in)) return QLORA_EINVAL;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (pending_error()) return QLORA_EHIP;
  if (cfmt == QLORA_C8ROW)
    launch_ckpt_write_rows(dtype, x, M, C, codes, static_cast<float*>(scales), s);
  else
    launch_ckpt_write_groups(dtype, x, M, C, codes, static_cast<uint8_t*>(scales), s);
  return launch_status();
}

int qlora_ckpt_read(const int8_t* codes, const void* scales, int M, int C, int cfmt,
                    int dtype, void* x, void* stream) {
  size_t cb, sb;
  int st = check_dtype(dtype);
  if (st) return st;
  st = qlora_ckpt_bytes(M, C, cfmt, &cb, &sb);
  if (st) return st;
  if (!x || !codes || !scales || !aligned16(x) || !aligned16(codes) || !aligned16(scales))
    return QLORA_EINVAL;
  Ranges in, out;
  in.add(codes, cb);
  in.add(scales, sb);
  out.add(x, cb * dtype_bytes(dtype));
  if (!disjoint(out, in)) return QLORA_EINVAL;
  if (pending_error()) return QLORA_EHIP;
  launch_ckpt_read(dtype, cfmt, codes, scales, M, C, x, static_cast<hipStream_t>(stream));
  return launch_status();
}

int qlora_fwd_epi(const qlora_linear* L, int M, int dtype, const void* x,
                  const qlora_epilogue* e, void* y, float* t_save, void* ws,
                  size_t ws_bytes, void* stream) {
  int st = check_linear(L, M, dtype);
  if (st) return st;
  if (!exact_sums(L)) return QLORA_EUNSUPPORTED;
  if (!x || !y || !aligned16(x) || !aligned16(y) || !opt16(t_save)) return QLORA_EINVAL;
  const int K = L->K, N = L->N;
  Ranges in, out;
  st = check_epilogue(e, M, K, N, dtype, y, in, out);
  if (st) return st;
  const FwdLayout w = fwd_layout(L, M);
  if (ws_bytes < w.total || !ws || !aligned16(ws)) return QLORA_EWORKSPACE;
  add_layer(in, L);
  in.add(x, (size_t)M * K * dtype_bytes(dtype));
  out.add(y, (size_t)M * N * dtype_bytes(dtype));
  out.add(t_save, (size_t)M * L->r * 4);
  out.add(ws, w.total);
  if (!disjoint(out, in)) return QLORA_EINVAL;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const FwdEpi epi = fwd_epi(e, N);
  float* t = t_save ? t_save : reinterpret_cast<float*>(at(ws, w.t));
  int8_t* xq = e->x_codes ? e->x_codes : reinterpret_cast<int8_t*>(at(ws, w.xq));
  float* sx = e->x_scales ? e->x_scales : reinterpret_cast<float*>(at(ws, w.sx));
  float* rs = reinterpret_cast<float*>(at(ws, w.rs));
  if (pending_error()) return QLORA_EHIP;
  if (fwd_few_takes(L->fmt, M, N, K, L->r)) {
    launch_fwd_few(dtype, L->fmt, M, N, K, x, L->codes, L->scales, L->A, L->B, head_width(L), L->r,
                   lora_s(L), epi, y, t_save, e->x_codes, e->x_scales,
                   reinterpret_cast<float*>(at(ws, w.xq)), s);
    return launch_status();
  }
  if (L->fmt == QLORA_W4G128) {
    // the product takes x itself; its codes are made only where they are kept
    if (e->x_codes)
      launch_rowquant(dtype, x, M, K, L->A, L->r, xq, sx, t, s, nullptr, rs);
    else
      launch_lora_down(dtype, x, M, K, L->A, L->r, t, s, rs);
    launch_gemm_fwd_w4(M, N, K, static_cast<const uint16_t*>(x), static_cast<const uint8_t*>(L->codes),
                       static_cast<const _Float16*>(L->scales), t, L->B, head_width(L), L->r, lora_s(L),
                       static_cast<uint16_t*>(y), reinterpret_cast<float*>(at(ws, w.pacc)), &epi, s);
    return launch_status();
  }
  float* asum = L->fmt == QLORA_W8O ? reinterpret_cast<float*>(at(ws, w.asum)) : nullptr;
  launch_rowquant(dtype, x, M, K, L->A, L->r, xq, sx, t, s, asum, rs);
  enqueue_fwd_i8(L, M, dtype, xq, sx, asum, t, epi, y, ws, w, s);
  return launch_status();
}

int qlora_fwd_ckpt(const qlora_linear* L, int M, int dtype, const int8_t* x_codes,
                   const float* x_scales, const float* t, const qlora_epilogue* e,
                   void* y, void* ws, size_t ws_bytes, void* stream) {
  int st = check_linear(L, M, dtype);
  if (st) return st;
  if (!exact_sums(L)) return QLORA_EUNSUPPORTED;
  if (!x_codes || !x_scales || !t || !y || !aligned16(x_codes) || !aligned16(x_scales) ||
      !aligned16(t) || !aligned16(y))
    return QLORA_EINVAL;
  const int K = L->K, N = L->N;
  Ranges in, out;
  st = check_epilogue(e, M, K, N, dtype, y, in, out);
  if (st) return st;
  if (e->x_codes != nullptr) return QLORA_EINVAL;   // x is the checkpoint already
  const FwdLayout w = fwd_layout(L, M);
  if (ws_bytes < w.total || !ws || !aligned16(ws)) return QLORA_EWORKSPACE;
  add_layer(in, L);
  in.add(x_codes, (size_t)M * K);
  in.add(x_scales, (size_t)M * 4);
  in.add(t, (size_t)M * L->r * 4);
  out.add(y, (size_t)M * N * dtype_bytes(dtype));
  out.add(ws, w.total);
  if (!disjoint(out, in)) return QLORA_EINVAL;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const FwdEpi epi = fwd_epi(e, N);
  if (pending_error()) return QLORA_EHIP;
  if (L->fmt == QLORA_W4G128) {
    launch_gemm_fwd_a8w4(M, N, K, x_codes, x_scales, static_cast<const uint8_t*>(L->codes),
                         static_cast<const _Float16*>(L->scales), t, L->B, head_width(L), L->r,
                         lora_s(L), static_cast<uint16_t*>(y), &epi, s);
    return launch_status();
  }
  float* asum = nullptr;
  if (L->fmt == QLORA_W8O) {
    asum = reinterpret_cast<float*>(at(ws, w.asum));
    launch_code_sums(x_codes, M, K, asum, s);
  }
  enqueue_fwd_i8(L, M, dtype, x_codes, x_scales, asum, t, epi, y, ws, w, s);
  return launch_status();
}

int qlora_bwd_epi_workspace(const qlora_linear* L, int M, int dtype, size_t* bytes) {
  if (bytes == nullptr) return QLORA_EINVAL;
  const int st = check_linear(L, M, dtype);
  if (st) return st;
  *bytes = bwd_epi_bytes(L, M, dtype);
  return QLORA_OK;
}

int qlora_bwd_epi_partial(const qlora_linear* L, int M, int dtype, const void* x,
                          const int8_t* x_codes, const float* x_scales, const void* dy,
                          const float* t_saved, const qlora_grad_epilogue* g, void* dx,
                          void* ws, size_t ws_bytes, void* stream) {
  const int st = bwd_epi_check(L, M, dtype, x, x_codes, x_scales, dy, t_saved, g, dx, nullptr, nullptr,
                               ws, ws_bytes);
  if (st) return st;
  if (pending_error()) return QLORA_EHIP;
  enqueue_bwd_epi(L, M, dtype, x, x_codes, x_scales, dy, t_saved, g, dx, ws,
                  static_cast<hipStream_t>(stream));
  return launch_status();
}

int qlora_bwd_epi(const qlora_linear* L, int M, int dtype, const void* x,
                  const int8_t* x_codes, const float* x_scales, const void* dy,
                  const float* t_saved, const qlora_grad_epilogue* g, void* dx,
                  float* dA, float* dB, void* ws, size_t ws_bytes, void* stream) {
  int st = bwd_epi_check(L, M, dtype, x, x_codes, x_scales, dy, t_saved, g, dx, dA, dB, ws, ws_bytes);
  if (st) return st;
  st = finish_check(L, M, dtype, dA, dB, ws, ws_bytes);
  if (st) return st;
  if (pending_error()) return QLORA_EHIP;
  hipStream_t s = static_cast<hipStream_t>(stream);
  enqueue_bwd_epi(L, M, dtype, x, x_codes, x_scales, dy, t_saved, g, dx, ws, s);
  st = launch_status();
  if (st) return st;
  launch_skinny_stage2(finish_jobs(L, M, dtype, dA, dB, ws), s);
  return launch_status();
}

int qlora_act_bwd_workspace(int M, int N, size_t* bytes) {
  if (bytes == nullptr || M < 1 || N < 16 || N % 16) return QLORA_EINVAL;
  if (!fits_int(M, N)) return QLORA_ERANGE;
  *bytes = act_bwd_floats(M, N) * 4;
  return QLORA_OK;
}

int qlora_act_bwd(int act, int M, int N, int dtype, const void* dy, const void* z,
                  const int8_t* z_codes, const uint8_t* z_scales, void* dz, float* dbias,
                  void* ws, size_t ws_bytes, void* stream) {
  size_t need = 0;
  int st = check_dtype(dtype);
  if (st) return st;
  st = qlora_act_bwd_workspace(M, N, &need);
  if (st) return st;
  st = check_z(act, z, z_codes, z_scales);
  if (st) return st;
  if (!dy || !aligned16(dy) || !opt16(dz) || !opt16(dbias) || (!dz && !dbias)) return QLORA_EINVAL;
  if (dbias == nullptr) need = 0;
  if (ws_bytes < need || (need && (!ws || !aligned16(ws)))) return QLORA_EWORKSPACE;
  const size_t mn = (size_t)M * N, es = dtype_bytes(dtype);
  Ranges in, out;
  if (dz != dy) in.add(dy, mn * es);
  in.add(z, mn * es);
  in.add(z_codes, mn);
  in.add(z_scales, (size_t)M * group_count(N));
  out.add(dz, mn * es);
  out.add(dbias, (size_t)N * 4);
  out.add(ws, need);
  if (!disjoint(out, in)) return QLORA_EINVAL;
  if (pending_error()) return QLORA_EHIP;
  launch_act_bwd(dtype, M, N, dy, grad_epi(act, z, z_codes, z_scales, nullptr, N), dz, dbias,
                 static_cast<float*>(ws), static_cast<hipStream_t>(stream));
  return launch_status();
}

int qlora_merge(const qlora_linear* L, void* codes_out, void* scales_out,
                void* stream) {
  int st = check_linear(L, 1, QLORA_BF16);
  if (st) return st;
  if (L->fmt != QLORA_W8) return QLORA_EUNSUPPORTED;
  if (!codes_out || !scales_out || !aligned16(codes_out) || !aligned16(scales_out))
    return QLORA_EINVAL;
  const size_t cb = (size_t)L->N * L->K, sb = (size_t)L->N * 4;
  auto overlaps = [](const void* a, size_t na, const void* b, size_t nb) {
    const char* x = static_cast<const char*>(a);
    const char* y = static_cast<const char*>(b);
    return x < y + nb && y < x + na;
  };
  if (overlaps(codes_out, cb, L->codes, cb) || overlaps(codes_out, cb, L->scales, sb) ||
      overlaps(scales_out, sb, L->codes, cb) || overlaps(scales_out, sb, L->scales, sb) ||
      overlaps(codes_out, cb, scales_out, sb))
    return QLORA_EINVAL;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (pending_error()) return QLORA_EHIP;
  launch_merge_w8(static_cast<const int8_t*>(L->codes), static_cast<const float*>(L->scales),
                  L->A, L->B, head_width(L), L->K, L->N, L->r, lora_s(L),
                  static_cast<int8_t*>(codes_out), static_cast<float*>(scales_out), s);
  return launch_status();
}

int qlora_quantize_rows(const void* x, int M, int K, int dtype, int8_t* xq,
                        float* sx, void* stream) {
  int st = check_dtype(dtype);
  if (st) return st;
  if (M < 1 || K < 16 || K % 16) return QLORA_EINVAL;
  if (!fits_int(M, K)) return QLORA_ERANGE;
  if (!x || !xq || !sx || !aligned16(x) || !aligned16(xq) || !aligned16(sx))
    return QLORA_EINVAL;
  if (pending_error()) return QLORA_EHIP;
  launch_ckpt_write_rows(dtype, x, M, K, xq, sx, static_cast<hipStream_t>(stream));
  return launch_status();
}

int qlora_fwd_acc(const qlora_linear* L, int M, int dtype, const void* x,
                  int32_t* acc, void* ws, size_t ws_bytes, void* stream) {
  int st = check_linear(L, M, dtype);
  if (st) return st;
  if (L->fmt != QLORA_W8 && L->fmt != QLORA_W8O) return QLORA_EUNSUPPORTED;
  if (!x || !acc || !aligned16(x) || !aligned16(acc)) return QLORA_EINVAL;
  const FwdLayout w = fwd_layout(L, M);
  if (ws_bytes < w.total || !ws || !aligned16(ws)) return QLORA_EWORKSPACE;
  hipStream_t s = static_cast<hipStream_t>(stream);
  int8_t* xq = reinterpret_cast<int8_t*>(at(ws, w.xq));
  float* sx = reinterpret_cast<float*>(at(ws, w.sx));
  if (pending_error()) return QLORA_EHIP;
  launch_rowquant(dtype, x, M, L->K, nullptr, 1, xq, sx, nullptr, s);
  // the integer product alone: no scale is read
  launch_gemm_fwd_w8(dtype, M, L->N, L->K, xq,
                     static_cast<const int8_t*>(L->codes), sx, nullptr, nullptr, L->B,
                     head_width(L), L->r, 0.f, nullptr, acc, nullptr, nullptr, s);
  return launch_status();
}

}  // extern "C"
