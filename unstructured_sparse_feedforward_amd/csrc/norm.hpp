// The residual's addition and the root-mean-square norm (norm.hip), as
// api_norm.hip launches them.
#pragma once

#include "sffn_internal.hpp"

namespace sffn {

constexpr int64_t kNormMaxCols = 16384;

// what a norm is stored as: kF32, kBF16 or kMx8
constexpr int kMx8 = 2;

struct NormArgs {
  const void* x;            // [rows, cols]
  const void* res;          // nullable
  void* res_out;            // the sum, of res's type (may be res)
  const void* weight;       // nullable
  void* out;                // [rows, cols], or MXFP8 codes
  uint8_t* out_sc;          // their scales
  float* rstd;              // nullable
  const int32_t* n_dev;     // nullable: the number of valid rows
  int64_t ldx, ldr, ldro, ldo;
  int64_t rows;
  int cols;
  float eps;
  double inv_cols;          // 1 / cols
  int x_bf, r_bf, w_bf;     // bf16, else float32
  int out_kind;
};
hipError_t launch_norm(const NormArgs& a, hipStream_t s);

struct NormGradArgs {
  const void* dy;           // [rows, cols]
  const void* s;            // the normalised rows
  const void* ds_in;        // nullable: the gradient that reaches s beside the norm's
  const void* weight;       // nullable
  const float* rstd;        // [rows]
  void* ds;                 // [rows, cols]
  float* dw;                // [cols], nullable
  float* part;              // workspace [parts, cols], nullable iff dw is
  int64_t lddy, lds, lddi, ldds;
  int64_t rows;
  int cols;
  int dy_bf, s_bf, di_bf, w_bf, ds_bf;
  int parts;                // rows of the workspace
  int slabs;                // of columns, where dw needs no workspace (else 0)
  int in_place;             // ds is in the place of dy or s
};
// rows of the workspace, and workgroups of the first kernel; 0: one launch does
// without
int norm_grad_parts(int64_t rows, int64_t cols);
int norm_grad_slabs(int64_t cols);
// threads for a row of the norm
int norm_threads(int64_t cols);
hipError_t launch_norm_grad(const NormGradArgs& a, hipStream_t s);

}  // namespace sffn
