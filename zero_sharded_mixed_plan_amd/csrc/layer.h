// Declarations shared by the C ABI of the pre-norm feed-forward sub-layer
// (layer_abi.cpp) and its kernels: RMS norm and its gradient (norm.hip,
// norm_grad.hip), matrices held in 8 bits and the gated activation's gradient
// (held.hip), the gated projections and their products (gated.hip).
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "input.h"
#include "zero_internal.h"

namespace zk {

constexpr int kBlock = 32;      // columns that share a scale
constexpr int64_t kMaxNormCols = 8192;  // a row waits in one workgroup's registers

// A matrix held in 8 bits: e4m3 codes and one scale 2^(byte - 127) per block.
struct Held {
  char* codes;            // or null
  char* scales;
  const char* codes_end;
  int64_t ld_codes, ld_scales;  // bytes
};

struct RmsLaunch {
  const char* x;
  const char* res;        // or null
  const char* weight;     // or null
  char* total;            // or null
  char* y;                // or null
  float* rstd;            // or null
  Held held;
  const char* x_end;
  const char* res_end;
  const char* weight_end;
  int64_t ld_x, ld_res, ld_total, ld_y;  // bytes
  int64_t rows;
  uint32_t cols;
  int32_t weight_type, y_type;
  double eps, per_col;    // per_col: 1 / cols
};

struct RmsGradLaunch {
  const char* dy;
  const char* h;          // or null: held
  Held held;
  const float* rstd;
  const char* weight;     // or null
  const char* dres;       // or null
  char* dh;
  char* dweight;          // or null
  float* partial;         // [partials, cols] sums over a workgroup's rows
  const char* dy_end;
  const char* h_end;
  const char* dres_end;
  const char* weight_end;
  int64_t ld_dy, ld_h, ld_dres, ld_dh;  // bytes
  int64_t rows;
  uint32_t cols;
  uint32_t partials;
  int32_t weight_type, dweight_type, accumulate;
};
// Workgroups, and rows of partial sums, of a gradient, and a bound of theirs for any width.
uint32_t rms_grad_partials(int64_t rows, int64_t cols);
int64_t rms_grad_partials_most(int64_t rows);

struct HoldLaunch {
  char* x;                // the matrix: read when packing, else written
  const char* x_end;
  Held held;
  int64_t ld_x;           // bytes
  uint32_t rows, cols;
  uint32_t units;         // rows * groups
  FastDiv groups;         // 4 * ceil(cols / 32)
};

enum Act : int32_t { kSilu = 0, kGelu = 1 };

struct GatedGradLaunch {
  const char* da;
  const char* g;          // or null: held
  const char* u;
  Held hg, hu;
  char* dg;
  char* du;
  char* a;                // or null
  const char* da_end;
  const char* g_end;
  const char* u_end;
  int64_t ld_da, ld_g, ld_u, ld_dg, ld_du, ld_a;  // bytes
  uint32_t rows, cols;
  uint32_t units;
  FastDiv groups;
};

// The products of the gated projections and of their gradients, all
//   out[r, c] = sum over k of Q(r, k) P(c, k)
// with two of Q, P or out:
//   kForward  Q = x [rows, k]; P = w_gate and w_up [cols, k]; act(first) * second
//   kInput    the sum of two: Q = dg, du [rows, k]; P = w_gate, w_up [k, cols]
//   kWeight   two results: Q = dg, du [k, rows]; P = x [k, cols]
enum Product : int32_t { kForward = 0, kInput = 1, kWeight = 2 };

struct ProductLaunch {
  const char* q[2];
  const char* p[2];
  const char* q_end[2];
  const char* p_end[2];
  char* out[2];           // kForward, kInput: the first
  char* kept[2];          // kForward: gate and up as they are, or null
  Held held[2];           // kForward: held in 8 bits, or null codes
  int64_t ld_q[2], ld_p[2], ld_out[2], ld_kept[2];  // bytes
  int64_t rows, cols, k;
  int32_t act;            // kForward
  int32_t out_type;       // kWeight
  int32_t accumulate;     // kWeight
  float* ws;              // kInput, kWeight: product_ws_bytes()
};
// Bytes that the products of the backward pass need; never fall as an argument grows.
int64_t product_ws_bytes(int64_t tokens, int64_t dim, int64_t hidden);

int launch_rms(const RmsLaunch& a, zero_dtype_t xt, zero_dtype_t rt, void* stream);
int launch_rms_grad(const RmsGradLaunch& a, zero_dtype_t at, zero_dtype_t st, void* stream);
int launch_pack(const HoldLaunch& a, zero_dtype_t t, void* stream);
int launch_unpack(const HoldLaunch& a, zero_dtype_t t, void* stream);
int launch_product(Product kind, const ProductLaunch& a, zero_dtype_t t, void* stream);
int launch_gated_grad(const GatedGradLaunch& a, zero_dtype_t t, int32_t act, void* stream);

}  // namespace zk
