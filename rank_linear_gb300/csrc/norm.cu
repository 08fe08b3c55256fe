// norm.cu -- the C entry points of the root-mean-square norm with the residual's addition, dropout of the
// branch and an 8-bit output (include/lora_norm.h; ch05 "Acceleration
// principles: Triton kernels and fused LoRA", §5.4: one pass over the row).
//
// A row stays in the registers of the threads that read it: it is read once,
// its sum of squares (and largest magnitude) go through shuffles and shared
// memory, and it is written once.  Bound by memory: what counts is how many bytes
// an SM has on their way.
//
// Two forms.  Wide rows, more than the SMs take at once: blocks stay, and bulk copies
// bring the next rows into a ring in shared memory while one is worked on
// (k_norm_fwd_ring, k_norm_bwd_ring; the backward's narrow rows too where they lie side
// by side, k_norm_bwd_heads).  Narrow rows, several a warp, and few rows, where latency
// counts: straight into registers (k_norm_fwd, k_norm_bwd).
#include <climits>
#include <initializer_list>

#include "host.h"
#include "lora_norm.h"
#include "norm.cuh"

namespace lora {
namespace {

bool aligned(const void *p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

lora_status_t check_shape(const lora_norm_t *sh, lora_dtype_t dtype) {
  if (sh == nullptr) return fail(LORA_ERR_INVALID_ARG, "shape is NULL");
  if (dtype != LORA_BF16 && dtype != LORA_FP32)
    return fail(LORA_ERR_INVALID_ARG, "dtype %d is not LORA_BF16 or LORA_FP32", int(dtype));
  if (sh->outer < 0 || sh->inner < 0) return fail(LORA_ERR_INVALID_ARG, "outer or inner is negative");
  if (sh->dim < 1) return fail(LORA_ERR_INVALID_ARG, "dim = %d", sh->dim);
  if (sh->dim > kMaxDim) return fail(LORA_ERR_UNSUPPORTED, "dim = %d is over %d", sh->dim, kMaxDim);
  if (sh->inner > 0 && sh->outer > INT_MAX / sh->inner)
    return fail(LORA_ERR_UNSUPPORTED, "2^31 rows or more");
  if (sh->inner > INT_MAX) return fail(LORA_ERR_UNSUPPORTED, "2^31 rows or more");
  if ((sh->weight_fp32 | 1) != 1) return fail(LORA_ERR_INVALID_ARG, "weight_fp32 is 0 or 1");
  if (!(sh->eps >= 0.f) || !(sh->eps < 3e38f))
    return fail(LORA_ERR_INVALID_ARG, "eps = %g is not a number >= 0", sh->eps);
  return LORA_OK;
}

// One tensor of the call: checks it and notes its strides and alignment.
struct Tensors {
  const lora_norm_t *sh;
  int es;
  bool vec;
  lora_status_t add(const void *p, const int64_t *s, const char *name, bool out, NormRows &rows,
                    NormSpan *span = nullptr) {
    if (p == nullptr) return fail(LORA_ERR_INVALID_ARG, "%s is NULL", name);
    if (!aligned(p, es)) return fail(LORA_ERR_INVALID_ARG, "%s is not aligned to its type", name);
    rows.outer = sh->outer > 1 ? s[0] : 0;
    rows.inner = sh->inner > 1 ? s[1] : 0;
    if (out) {
      const int64_t r0 = rows.outer < 0 ? -rows.outer : rows.outer;
      const int64_t r1 = rows.inner < 0 ? -rows.inner : rows.inner;
      if ((sh->outer > 1 && r0 < sh->dim) || (sh->inner > 1 && r1 < sh->dim))
        return fail(LORA_ERR_INVALID_ARG, "the rows of %s overlap", name);
    }
    vec = vec && aligned(p, 16) && rows.outer % (16 / es) == 0 && rows.inner % (16 / es) == 0;
    if (span != nullptr) {
      int64_t lo = 0, hi = sh->dim;
      for (const int64_t reach : {rows.outer * (sh->outer - 1), rows.inner * (sh->inner - 1)})
        (reach < 0 ? lo : hi) += reach;
      span->first = reinterpret_cast<uint64_t>(p) + static_cast<uint64_t>(lo * es);
      span->last = reinterpret_cast<uint64_t>(p) + static_cast<uint64_t>(hi * es);
    }
    return LORA_OK;
  }
};
lora_status_t same_place(const void *out, const NormRows &so, const char *out_name, const void *in,
                         const NormRows &si, const char *in_name) {
  if (out == in && (so.outer != si.outer || so.inner != si.inner))
    return fail(LORA_ERR_INVALID_ARG, "%s is %s with other strides", out_name, in_name);
  return LORA_OK;
}
lora_status_t check_weight(const void *w, int es, const char *name, bool &vec) {
  if (w == nullptr) return fail(LORA_ERR_INVALID_ARG, "%s is NULL", name);
  if (!aligned(w, es)) return fail(LORA_ERR_INVALID_ARG, "%s is not aligned to its type", name);
  vec = vec && aligned(w, 16);
  return LORA_OK;
}

// Takes the backward's narrow rows side by side over the ring where they stand so: the shape's inner
// rows, if each tensor has them `dim` apart; or, of plain contiguous rows, as many as
// make some 4096 elements and divide their number.
void use_heads(const lora_norm_t *sh, bool vec, int es, int tensors, NormRows *const *of,
               const bool *given, int n, NormInner &inner, NormSplit &s) {
  if (!vec || s.ring || sh->dim > 256) return;
  int64_t outer = sh->outer, side = sh->inner;
  const bool plain = side == 1;
  if (plain) {
    while (2 * side * sh->dim <= 4096 && sh->outer % (2 * side) == 0) side *= 2;
    outer /= side;
  }
  for (int i = 0; i < n; ++i)
    if (given[i] && (plain ? of[i]->outer : of[i]->inner) != sh->dim) return;
  if (!norm_heads(sh->dim, outer, side, es, tensors, s) || !plain) return;
  inner = norm_inner(side);
  for (int i = 0; i < n; ++i) *of[i] = {side * sh->dim, sh->dim};
}

}  // namespace
}  // namespace lora

using namespace lora;

extern "C" {

lora_status_t lora_norm_fwd(const lora_norm_t *sh, const void *x, const void *residual,
                            const void *w, const lora_dropout_t *dropout, lora_dtype_t dtype,
                            void *h, void *y, float *rstd, void *codes, float *scale,
                            void *stream) {
  clear_error();
  LORA_TRY(check_shape(sh, dtype));
  NormFwdArgs a = {};
  LORA_TRY(drop_args(dropout, a.drop));
  if ((codes == nullptr) != (scale == nullptr))
    return fail(LORA_ERR_INVALID_ARG, "codes and scale are given together");
  const int64_t rows = sh->outer * sh->inner;
  if (rows == 0) return LORA_OK;
  a.dropped = dropout != nullptr && a.drop.threshold != 0;
  if (h != nullptr && residual == nullptr && dropout == nullptr)
    return fail(LORA_ERR_INVALID_ARG, "h is x without residual and dropout: give NULL");
  if (y == nullptr && codes == nullptr && h == nullptr)
    return fail(LORA_ERR_INVALID_ARG, "y, codes and h are NULL");
  Tensors ts = {sh, dtype == LORA_BF16 ? 2 : 4, sh->dim % 8 == 0};
  LORA_TRY(ts.add(x, sh->x, "x", false, a.sx, &a.span_x));
  if (residual != nullptr) LORA_TRY(ts.add(residual, sh->residual, "residual", false, a.sr, &a.span_r));
  if (h != nullptr) {
    LORA_TRY(ts.add(h, sh->h, "h", true, a.sh));
    LORA_TRY(same_place(h, a.sh, "h", x, a.sx, "x"));
    LORA_TRY(same_place(h, a.sh, "h", residual, a.sr, "residual"));
  }
  if (y != nullptr) {
    LORA_TRY(ts.add(y, sh->y, "y", true, a.sy));
    LORA_TRY(same_place(y, a.sy, "y", x, a.sx, "x"));
    LORA_TRY(same_place(y, a.sy, "y", residual, a.sr, "residual"));
    if (y == h) return fail(LORA_ERR_INVALID_ARG, "y and h are the same tensor");
  }
  LORA_TRY(check_weight(w, sh->weight_fp32 ? 4 : ts.es, "w", ts.vec));
  if (!aligned(rstd, 4) || !aligned(scale, 4))
    return fail(LORA_ERR_INVALID_ARG, "rstd or scale is not aligned to its type");
  if (codes != nullptr) ts.vec = ts.vec && aligned(codes, 8);
  a.x = x;
  a.res = residual;
  a.w = w;
  // dropout with p = 0 and no residual copies x
  if (h != nullptr && residual == nullptr) a.dropped = 1;
  a.h = h;
  a.y = y;
  a.rstd = rstd;
  a.codes = static_cast<uint8_t *>(codes);
  a.scale = scale;
  a.rows = rows;
  a.inner = norm_inner(sh->inner > 0 ? sh->inner : 1);
  a.dim = sh->dim;
  a.inv_dim = 1.f / static_cast<float>(sh->dim);
  a.eps = sh->eps;
  a.w32 = dtype == LORA_FP32 ? 0 : sh->weight_fp32;
  const int tensors = residual != nullptr ? 2 : 1;
  NormSplit s = norm_split(sh->dim, rows, ts.es, tensors, ts.vec, false, codes != nullptr);
  if (s.ring && !ts.vec && !a.dropped && sh->inner == 1 && a.w32 == 0) {
    NormShift shift;
    shift.add(x, a.sx.outer, ts.es);
    if (residual != nullptr) shift.add(residual, a.sr.outer, ts.es);
    if (h != nullptr) shift.add(h, a.sh.outer, ts.es);
    if (y != nullptr) shift.add(y, a.sy.outer, ts.es);
    // (a code is a byte: its row lies as far past 8 bytes as a row of bf16 past 16)
    if (codes != nullptr &&
        ((reinterpret_cast<uint64_t>(codes) - reinterpret_cast<uint64_t>(x) / 2) % 8 != 0 || (a.sx.outer - sh->dim) % 8 != 0))
      shift.ok = false;
    const NormSplit t = norm_split(sh->dim, rows, ts.es, tensors, false, false, codes != nullptr, true);
    if (shift.ok && t.ring) s = t;
  }
  a.group = s.group;
  DevInfo di;
  LORA_TRY(device_info(di));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return run(LORA_K_NORM, st, "norm",
             [&] { return launch_norm_fwd(dtype, ts.vec, a, s, tensors, di.status, st); });
}

size_t lora_norm_workspace_bytes(const lora_norm_t *sh, int with_dw) {
  clear_error();
  if (check_shape(sh, LORA_BF16) != LORA_OK || !with_dw) return 0;
  // (the type, the alignment and whether dh is given move the blocks: room for the most)
  const int64_t rows = sh->outer * sh->inner;
  int most = 0;
  for (int es = 2; es <= 4; es += 2)
    for (int tensors = 2; tensors <= 3; ++tensors) {
      for (int vec = 0; vec < 2; ++vec) {
        const int n = norm_bwd_blocks(norm_split(sh->dim, rows, es, tensors, vec != 0, true), rows);
        most = n > most ? n : most;
      }
      const int n = norm_bwd_blocks(norm_split(sh->dim, rows, es, tensors, false, true, false, true), rows);
      most = n > most ? n : most;
    }
  // (narrow rows side by side: twelve blocks an SM at most, of two rows at least)
  if (sh->dim <= 256 && !norm_few_rows(rows / 2)) {
    const int64_t n = rows / 2 < kSms * 12 ? rows / 2 : kSms * 12;
    most = n > most ? static_cast<int>(n) : most;
  }
  return size_t(most) * sh->dim * sizeof(float);
}

lora_status_t lora_norm_bwd(const lora_norm_t *sh, const void *dy, const void *h, const void *w,
                            const float *rstd, const void *dh, const lora_dropout_t *dropout,
                            lora_dtype_t dtype, void *dx, void *dresidual, void *dw,
                            void *workspace, size_t workspace_bytes, void *stream) {
  clear_error();
  LORA_TRY(check_shape(sh, dtype));
  NormBwdArgs a = {};
  LORA_TRY(drop_args(dropout, a.drop));
  const int64_t rows = sh->outer * sh->inner;
  const int ws_es = sh->weight_fp32 || dtype == LORA_FP32 ? 4 : 2;
  if (dw != nullptr && !aligned(dw, ws_es))
    return fail(LORA_ERR_INVALID_ARG, "dw is not aligned to its type");
  const int tensors = dh != nullptr ? 3 : 2;
  bool vec = sh->dim % 8 == 0;
  if (rows > 0) {
    Tensors ts = {sh, dtype == LORA_BF16 ? 2 : 4, vec};
    LORA_TRY(ts.add(dy, sh->dy, "dy", false, a.sdy, &a.span_y));
    LORA_TRY(ts.add(h, sh->h, "h", false, a.sh, &a.span_h));
    if (dh != nullptr) LORA_TRY(ts.add(dh, sh->dh, "dh", false, a.sdh, &a.span_d));
    LORA_TRY(ts.add(dx, sh->dx, "dx", true, a.sdx));
    LORA_TRY(same_place(dx, a.sdx, "dx", dy, a.sdy, "dy"));
    LORA_TRY(same_place(dx, a.sdx, "dx", dh, a.sdh, "dh"));
    LORA_TRY(same_place(dx, a.sdx, "dx", h, a.sh, "h"));
    if (dresidual != nullptr) {
      LORA_TRY(ts.add(dresidual, sh->dresidual, "dresidual", true, a.sdr));
      LORA_TRY(same_place(dresidual, a.sdr, "dresidual", dy, a.sdy, "dy"));
      LORA_TRY(same_place(dresidual, a.sdr, "dresidual", dh, a.sdh, "dh"));
      LORA_TRY(same_place(dresidual, a.sdr, "dresidual", h, a.sh, "h"));
      if (dresidual == dx) return fail(LORA_ERR_INVALID_ARG, "dx and dresidual are the same tensor");
    }
    LORA_TRY(check_weight(w, ws_es, "w", ts.vec));
    if (rstd == nullptr || !aligned(rstd, 4))
      return fail(LORA_ERR_INVALID_ARG, "rstd is NULL or not aligned");
    vec = ts.vec;
  }
  const int es = dtype == LORA_BF16 ? 2 : 4;
  NormSplit s = norm_split(sh->dim, rows, es, tensors, vec, true);
  a.dropped = dropout != nullptr && a.drop.threshold != 0;
  a.w32 = dtype == LORA_FP32 ? 0 : sh->weight_fp32;
  a.inner = norm_inner(sh->inner > 0 ? sh->inner : 1);
  NormRows *of[5] = {&a.sdy, &a.sh, &a.sdx, &a.sdh, &a.sdr};
  const bool given[5] = {true, true, true, dh != nullptr, dresidual != nullptr};
  if (rows > 0) use_heads(sh, vec, es, tensors, of, given, 5, a.inner, s);
  if (rows > 0 && s.ring && !vec && !a.dropped && sh->inner == 1 && a.w32 == 0) {
    NormShift shift;
    shift.add(dy, a.sdy.outer, es);
    shift.add(h, a.sh.outer, es);
    shift.add(dx, a.sdx.outer, es);
    if (dh != nullptr) shift.add(dh, a.sdh.outer, es);
    if (dresidual != nullptr) shift.add(dresidual, a.sdr.outer, es);
    const NormSplit t = norm_split(sh->dim, rows, es, tensors, false, true, false, true);
    if (shift.ok && t.ring) s = t;
  }
  const int blocks = norm_bwd_blocks(s, s.heads ? rows / a.inner.n : rows);
  if (dw != nullptr)
    LORA_TRY(check_ws(workspace, workspace_bytes, size_t(blocks) * sh->dim * sizeof(float)));
  if (rows == 0 && dw == nullptr) return LORA_OK;
  a.dy = dy;
  a.h = h;
  a.w = w;
  a.dh = dh;
  a.rstd = rstd;
  a.dx = dx;
  a.dres = dresidual;
  a.partial = dw != nullptr ? static_cast<float *>(workspace) : nullptr;
  a.rows = rows;
  a.dim = sh->dim;
  a.inv_dim = 1.f / static_cast<float>(sh->dim);
  a.group = s.group;
  DevInfo di;
  LORA_TRY(device_info(di));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (rows > 0)
    LORA_TRY(run(LORA_K_NORM_BWD, st, "norm backward",
                 [&] { return launch_norm_bwd(dtype, vec, a, s, tensors, di.status, st); }));
  if (dw == nullptr) return LORA_OK;
  return run(LORA_K_NORM_BWD, st, "norm dw", [&] {
    return launch_norm_dw(ws_es == 4, static_cast<const float *>(workspace), blocks, sh->dim, dw, st);
  });
}

}  // extern "C"
