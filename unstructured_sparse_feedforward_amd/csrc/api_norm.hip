// C ABI of the residual norm (sffn_rms_norm*): argument validation and
// launches. See include/sffn.h for the contract of every entry point.
#include <cmath>

#include "norm.hpp"
#include "mx.hpp"
#include "place.hpp"
#include "sffn.h"

namespace {

using namespace sffn;

constexpr size_t kAlign = 256;
constexpr int64_t kMaxRows = (int64_t)1 << 27;

bool aligned(const void* p, size_t a) { return p != nullptr && (uintptr_t)p % a == 0; }
bool float_type(int32_t dt) { return dt == SFFN_F32 || dt == SFFN_BF16; }
size_t elem(int32_t dt) { return dt == SFFN_BF16 ? 2 : 4; }
// a matrix or vector of a float type
bool floats(const void* p, int32_t dt) { return float_type(dt) && aligned(p, elem(dt)); }
bool maybe(const void* p, int32_t dt) { return p == nullptr || floats(p, dt); }
sffn_status done(hipError_t e) { return e == hipSuccess ? SFFN_OK : SFFN_E_HIP; }

sffn_status sizes(int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 0) return SFFN_E_ARG;
  return rows > kMaxRows || cols > kNormMaxCols ? SFFN_E_UNSUPPORTED : SFFN_OK;
}

// of a matrix of a float type; of none (p is null), no bytes
Place place(const void* p, int32_t dt, int64_t ld, int64_t rows, int64_t cols) {
  const int e = (int)elem(dt);
  return {p, p ? rows : 0, ld * e, cols * e, e};
}

size_t workspace(int64_t rows, int64_t cols) {
  return ((size_t)norm_grad_parts(rows, cols) * cols * 4 + kAlign - 1) / kAlign * kAlign;
}

}  // namespace

extern "C" {

sffn_status sffn_rms_norm(const sffn_norm* n, int64_t rows, int64_t cols, float eps,
                          const int32_t* n_rows, hipStream_t stream) {
  if (!n) return SFFN_E_ARG;
  const sffn_status st = sizes(rows, cols);
  if (st != SFFN_OK) return st;
  // (a launch has fewer than 2^32 threads)
  if (rows * norm_threads(cols) > (int64_t)1 << 31) return SFFN_E_UNSUPPORTED;
  if (!(eps >= 0.0f) || !std::isfinite(eps)) return SFFN_E_ARG;
  const bool mx8 = n->out_dtype == SFFN_MXFP8;
  if (!mx8 && !float_type(n->out_dtype)) return SFFN_E_ARG;
  if (rows == 0 || cols == 0) return SFFN_OK;
  if (!floats(n->x, n->x_dtype) || n->ldx < cols) return SFFN_E_ARG;
  if ((n->residual == nullptr) != (n->residual_out == nullptr)) return SFFN_E_ARG;
  if (n->residual && (!floats(n->residual, n->residual_dtype) ||
                      !floats(n->residual_out, n->residual_dtype) || n->ldr < cols ||
                      n->ldro < cols))
    return SFFN_E_ARG;
  if (!maybe(n->weight, n->weight_dtype)) return SFFN_E_ARG;
  if (mx8 ? !aligned(n->out, 16) || !aligned(n->out_scales, 4)
          : !aligned(n->out, elem(n->out_dtype)) || n->out_scales != nullptr || n->ldo < cols)
    return SFFN_E_ARG;
  if ((n->rstd && !aligned(n->rstd, 4)) || (n_rows && !aligned(n_rows, 4))) return SFFN_E_ARG;
  // in the place of an operand, or apart from it
  const Place x = place(n->x, n->x_dtype, n->ldx, rows, cols);
  const Place r = place(n->residual, n->residual_dtype, n->ldr, rows, cols);
  const Place ro = place(n->residual_out, n->residual_dtype, n->ldro, rows, cols);
  const int64_t Kp = mx_padded(cols);
  const Place y = mx8 ? Place{n->out, rows, Kp, Kp, 1}
                      : place(n->out, n->out_dtype, n->ldo, rows, cols);
  if (meeting(y, x) == kMixed) return SFFN_E_ARG;
  if (n->residual && (meeting(ro, x) == kMixed || meeting(ro, r) == kMixed ||
                      meeting(y, r) == kMixed || meeting(y, ro) != kApart))
    return SFFN_E_ARG;
  NormArgs a = {};
  a.x = n->x;
  a.res = n->residual;
  a.res_out = n->residual_out;
  a.weight = n->weight;
  a.out = n->out;
  a.out_sc = n->out_scales;
  a.rstd = n->rstd;
  a.n_dev = n_rows;
  a.ldx = n->ldx;
  a.ldr = n->ldr;
  a.ldro = n->ldro;
  a.ldo = n->ldo;
  a.rows = rows;
  a.cols = (int)cols;
  a.eps = eps;
  a.inv_cols = 1.0 / (double)cols;
  a.x_bf = n->x_dtype == SFFN_BF16;
  a.r_bf = n->residual && n->residual_dtype == SFFN_BF16;
  a.w_bf = n->weight && n->weight_dtype == SFFN_BF16;
  a.out_kind = mx8 ? kMx8 : n->out_dtype == SFFN_BF16 ? (int)kBF16 : (int)kF32;
  return done(launch_norm(a, stream));
}

sffn_status sffn_rms_norm_backward_workspace_bytes(int64_t rows, int64_t cols, size_t* bytes) {
  const sffn_status st = sizes(rows, cols);
  if (st != SFFN_OK) return st;
  if (!bytes) return SFFN_E_ARG;
  *bytes = workspace(rows, cols);
  return SFFN_OK;
}

sffn_status sffn_rms_norm_backward(const sffn_norm_grad* n, int64_t rows, int64_t cols, void* ws,
                                   size_t ws_bytes, hipStream_t stream) {
  if (!n) return SFFN_E_ARG;
  const sffn_status st = sizes(rows, cols);
  if (st != SFFN_OK) return st;
  if (n->dweight && (!n->weight || !aligned(n->dweight, 4))) return SFFN_E_ARG;
  if (cols == 0 || (rows == 0 && !n->dweight)) return SFFN_OK;
  if (!maybe(n->weight, n->weight_dtype)) return SFFN_E_ARG;
  if (rows > 0) {
    if (!floats(n->dy, n->dy_dtype) || !floats(n->s, n->s_dtype) || !aligned(n->rstd, 4) ||
        !floats(n->ds, n->ds_dtype) || !maybe(n->dstream, n->dstream_dtype))
      return SFFN_E_ARG;
    if (n->lddy < cols || n->lds < cols || n->ldds < cols || (n->dstream && n->lddstream < cols))
      return SFFN_E_ARG;
    const size_t need = n->dweight ? workspace(rows, cols) : 0;
    if (need > 0 && (!aligned(ws, kAlign) || ws_bytes < need)) return SFFN_E_ARG;
  }
  // ds in the place of an operand, or apart from it
  const Place ds = place(n->ds, n->ds_dtype, n->ldds, rows, cols);
  const Meeting dy_ds = meeting(ds, place(n->dy, n->dy_dtype, n->lddy, rows, cols));
  const Meeting s_ds = meeting(ds, place(n->s, n->s_dtype, n->lds, rows, cols));
  if (dy_ds == kMixed || s_ds == kMixed ||
      meeting(ds, place(n->dstream, n->dstream_dtype, n->lddstream, rows, cols)) == kMixed ||
      meeting(place(n->dweight, SFFN_F32, cols, 1, cols),
              place(n->weight, n->weight_dtype, cols, 1, cols)) != kApart)
    return SFFN_E_ARG;
  NormGradArgs a = {};
  a.dy = n->dy;
  a.s = n->s;
  a.ds_in = n->dstream;
  a.weight = n->weight;
  a.rstd = n->rstd;
  a.ds = n->ds;
  a.dw = n->dweight;
  a.part = (float*)ws;
  a.lddy = n->lddy;
  a.lds = n->lds;
  a.lddi = n->lddstream;
  a.ldds = n->ldds;
  a.rows = rows;
  a.cols = (int)cols;
  a.dy_bf = n->dy_dtype == SFFN_BF16;
  a.s_bf = n->s_dtype == SFFN_BF16;
  a.di_bf = n->dstream && n->dstream_dtype == SFFN_BF16;
  a.w_bf = n->weight && n->weight_dtype == SFFN_BF16;
  a.ds_bf = n->ds_dtype == SFFN_BF16;
  a.parts = norm_grad_parts(rows, cols);
  a.slabs = a.parts == 0 && n->dweight ? norm_grad_slabs(cols) : 0;
  a.in_place = dy_ds == kSame || s_ds == kSame;
  return done(launch_norm_grad(a, stream));
}

}  // extern "C"
