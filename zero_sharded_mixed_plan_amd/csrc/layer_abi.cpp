// C ABI of the pre-norm gated feed-forward sub-layer: argument validation (before
// anything is enqueued) and the launches.
#include <algorithm>
#include <cmath>
#include <string>

#include "abi_checks.h"
#include "layer.h"

namespace {

constexpr int64_t kMaxRows = int64_t(1) << 31;

int error(const char* fn, const char* what) { return fail(ZERO_EINVAL, std::string(fn) + ": " + what); }

int64_t blocks_of(int64_t cols) { return (cols + zk::kBlock - 1) / zk::kBlock; }

// A vector of `n` elements.
int vector(const char* fn, const char* what, const void* p, int64_t n, zero_dtype_t t) {
  return matrix(fn, what, p, n > 0 ? 1 : 0, n, n, t);
}

Span vector_span(const void* p, int64_t n, zero_dtype_t t) { return span(p, n * bytes_of(t)); }

int held_matrix(const char* fn, const char* what, const zero_held_t* h, int64_t rows, int64_t cols) {
  if (rows == 0) return ZERO_OK;
  const std::string name = std::string(fn) + ": " + what;
  if (!h->codes || !h->scales) return fail(ZERO_EINVAL, name + ": codes or scales are NULL");
  if (rows > 1 && (h->ld_codes < cols || h->ld_scales < blocks_of(cols)))
    return fail(ZERO_EINVAL, name + ": rows of codes or scales overlap");
  for (int64_t ld : {h->ld_codes, h->ld_scales})
    if (ld < 0 || ld > kMaxLd || (rows > 1 && ld > (int64_t(1) << 60) / rows))
      return fail(ZERO_EINVAL, name + ": a stride is out of range");
  return ZERO_OK;
}
Span codes_span(const zero_held_t* h, int64_t rows, int64_t cols) { return span(h->codes, rows, cols, h->ld_codes, 1); }
Span scales_span(const zero_held_t* h, int64_t rows, int64_t cols) {
  return span(h->scales, rows, blocks_of(cols), h->ld_scales, 1);
}
zk::Held held_launch(const zero_held_t* h, int64_t rows, int64_t cols) {
  zk::Held k{};
  if (!h) return k;
  k.codes = static_cast<char*>(h->codes);
  k.scales = static_cast<char*>(h->scales);
  k.ld_codes = h->ld_codes;
  k.ld_scales = h->ld_scales;
  k.codes_end = end_of(codes_span(h, rows, cols));
  return k;
}
void advance(zk::Held& k, int64_t rows) {
  if (!k.codes) return;
  k.codes += rows * k.ld_codes;
  k.scales += rows * k.ld_scales;
}

// What a call reads and writes: no written range may meet another one, but for the pairs
// that allow() names.  Matrices with one stride may lie side by side, as column ranges of one buffer do.
struct Ranges {
  static constexpr int kMost = 24;
  Span s[kMost];
  uintptr_t ld[kMost], width[kMost];  // bytes; 0: not a matrix
  bool written[kMost];
  int n = 0;
  int add(const Span& x, bool w, int64_t ld_bytes = 0, int64_t row_bytes = 0) {
    s[n] = x;
    ld[n] = (uintptr_t)ld_bytes;
    width[n] = (uintptr_t)row_bytes;
    written[n] = w;
    return n++;
  }
  int add(const void* p, int64_t rows, int64_t cols, int64_t ld_elements, int eb, bool w) {
    return add(span(p, rows, cols, ld_elements, eb), w, ld_elements * eb, cols * eb);
  }
  int add_codes(const zero_held_t* h, int64_t rows, int64_t cols, bool w) {
    return add(codes_span(h, rows, cols), w, h->ld_codes, cols);
  }
  int add_scales(const zero_held_t* h, int64_t rows, int64_t cols, bool w) {
    return add(scales_span(h, rows, cols), w, h->ld_scales, blocks_of(cols));
  }
  uint32_t allowed[kMost] = {};
  void allow(int i, int j) {
    allowed[i] |= 1u << j;
    allowed[j] |= 1u << i;
  }
  bool beside(int i, int j) const {
    if (ld[i] == 0 || ld[i] != ld[j]) return false;
    const uintptr_t d = s[j].lo >= s[i].lo ? (s[j].lo - s[i].lo) % ld[i] : (ld[i] - (s[i].lo - s[j].lo) % ld[i]) % ld[i];
    return d >= width[i] && d + width[j] <= ld[i];
  }
  bool clash() const {
    for (int i = 0; i < n; ++i)
      for (int j = 0; j < i; ++j)
        if ((written[i] || written[j]) && !(allowed[i] >> j & 1) && overlap(s[i], s[j]) && !beside(i, j)) return true;
    return false;
  }
};

// Whether a result may lie on an operand: one matrix, read and written element by element.
bool in_place(const void* a, int64_t ld_a, zero_dtype_t ta, const void* b, int64_t ld_b, zero_dtype_t tb, int64_t rows) {
  return a == b && ta == tb && (ld_a == ld_b || rows == 1);
}

zk::HoldLaunch hold_launch(void* x, int64_t ld_x, zero_dtype_t t, const zero_held_t* held, int64_t rows, int64_t cols) {
  zk::HoldLaunch a{};
  a.x = static_cast<char*>(x);
  a.x_end = end_of(span(x, rows, cols, ld_x, bytes_of(t)));
  a.held = held_launch(held, rows, cols);
  a.ld_x = ld_x * bytes_of(t);
  a.cols = (uint32_t)cols;
  a.groups = zk::fast_div((uint32_t)(4 * blocks_of(cols)));
  return a;
}

int hold(const char* fn, bool pack, void* x, int64_t ld_x, zero_dtype_t t, const zero_held_t* held, int64_t rows,
         int64_t cols, void* stream) {
  if (rows < 0 || rows >= kMaxLd) return error(fn, "rows out of range");
  if (cols < 1 || cols >= kMax31) return error(fn, "cols must lie in [1, 2^31)");
  int rc;
  if ((rc = matrix(fn, pack ? "x" : "out", x, rows, cols, ld_x, t))) return rc;
  if (!held) return error(fn, "held is NULL");
  if ((rc = held_matrix(fn, "held", held, rows, cols))) return rc;
  if (rows == 0) return ZERO_OK;
  Ranges r;
  r.add(x, rows, cols, ld_x, bytes_of(t), !pack);
  r.add_codes(held, rows, cols, pack);
  r.add_scales(held, rows, cols, pack);
  if (r.clash()) return error(fn, "what is written overlaps something else");
  zk::HoldLaunch a = hold_launch(x, ld_x, t, held, rows, cols);
  const int64_t per_launch = std::max<int64_t>(1, zk::kMaxUnits / a.groups.d);
  for (int64_t i = 0; i < rows; i += per_launch) {
    a.rows = (uint32_t)std::min(per_launch, rows - i);
    a.units = a.rows * a.groups.d;
    if ((rc = pack ? zk::launch_pack(a, t, stream) : zk::launch_unpack(a, t, stream))) return rc;
    a.x += per_launch * a.ld_x;
    advance(a.held, per_launch);
  }
  return ZERO_OK;
}

// The stream's type beside another tensor's.
bool stream_types(zero_dtype_t other, zero_dtype_t stream) { return other == stream || stream == ZERO_F32; }

int rms(const zero_rms_args_t* args, void* stream) {
  const char* const fn = "zero_rms_norm";
  if (!args) return error(fn, "args is NULL");
  const zero_rms_args_t& A = *args;
  if (A.rows < 0 || A.rows >= kMaxLd) return error(fn, "rows out of range");
  if (A.cols < 1 || A.cols > zk::kMaxNormCols) return error(fn, "cols must lie in [1, 8192]");
  if (!(A.eps >= 0.0) || !std::isfinite(A.eps)) return error(fn, "eps must be finite and at least 0");
  int rc;
  if ((rc = matrix(fn, "x", A.x, A.rows, A.cols, A.ld_x, A.x_dtype))) return rc;
  const bool res = A.residual != nullptr;
  if (A.rows > 0 && res != (A.total != nullptr)) return error(fn, "residual and total go together");
  if (res) {
    if ((rc = matrix(fn, "the residual", A.residual, A.rows, A.cols, A.ld_res, A.res_dtype))) return rc;
    if ((rc = matrix(fn, "total", A.total, A.rows, A.cols, A.ld_total, A.res_dtype))) return rc;
    if (!stream_types(A.x_dtype, A.res_dtype)) return error(fn, "the residual must be of x's type or fp32");
  }
  if (A.weight && (rc = vector(fn, "the weight", A.weight, A.cols, A.weight_dtype))) return rc;
  if (A.out && (rc = matrix(fn, "out", A.out, A.rows, A.cols, A.ld_out, A.out_dtype))) return rc;
  if (A.held && (rc = held_matrix(fn, "held", A.held, A.rows, A.cols))) return rc;
  if (A.rstd && !aligned(A.rstd, 4)) return fail(ZERO_EALIGN, std::string(fn) + ": rstd is not element aligned");
  if (A.rows == 0) return ZERO_OK;
  if (!A.out && !A.held) return error(fn, "neither out nor held is given");
  const int xb = bytes_of(A.x_dtype), rb = res ? bytes_of(A.res_dtype) : 0;
  Ranges r;
  const int x = r.add(A.x, A.rows, A.cols, A.ld_x, xb, false);
  if (A.weight) r.add(vector_span(A.weight, A.cols, A.weight_dtype), false);
  if (res) {
    const int d = r.add(A.residual, A.rows, A.cols, A.ld_res, rb, false);
    const int h = r.add(A.total, A.rows, A.cols, A.ld_total, rb, true);
    if (in_place(A.total, A.ld_total, A.res_dtype, A.x, A.ld_x, A.x_dtype, A.rows)) r.allow(h, x);
    if (in_place(A.total, A.ld_total, A.res_dtype, A.residual, A.ld_res, A.res_dtype, A.rows)) r.allow(h, d);
  }
  if (A.out) r.add(A.out, A.rows, A.cols, A.ld_out, bytes_of(A.out_dtype), true);
  if (A.held) {
    r.add_codes(A.held, A.rows, A.cols, true);
    r.add_scales(A.held, A.rows, A.cols, true);
  }
  if (A.rstd) r.add(span(A.rstd, A.rows * 4), true);
  if (r.clash()) return error(fn, "what is written overlaps something else");

  zk::RmsLaunch a{};
  a.x = static_cast<const char*>(A.x);
  a.x_end = end_of(r.s[x]);
  a.ld_x = A.ld_x * xb;
  if (res) {
    a.res = static_cast<const char*>(A.residual);
    a.res_end = end_of(span(A.residual, A.rows, A.cols, A.ld_res, rb));
    a.total = static_cast<char*>(A.total);
    a.ld_res = A.ld_res * rb;
    a.ld_total = A.ld_total * rb;
  }
  if (A.weight) {
    a.weight = static_cast<const char*>(A.weight);
    a.weight_end = end_of(vector_span(A.weight, A.cols, A.weight_dtype));
    a.weight_type = A.weight_dtype;
  }
  if (A.out) {
    a.y = static_cast<char*>(A.out);
    a.ld_y = A.ld_out * bytes_of(A.out_dtype);
    a.y_type = A.out_dtype;
  }
  a.held = held_launch(A.held, A.rows, A.cols);
  a.rstd = A.rstd;
  a.rows = A.rows;
  a.cols = (uint32_t)A.cols;
  a.eps = A.eps;
  a.per_col = 1.0 / (double)A.cols;
  return zk::launch_rms(a, A.x_dtype, res ? A.res_dtype : A.x_dtype, stream);
}

bool rms_grad_sizes_ok(int64_t rows, int64_t cols) {
  return rows >= 0 && rows < kMaxLd && cols >= 1 && cols <= zk::kMaxNormCols;
}

int rms_grad(const zero_rms_grad_args_t* args, void* stream) {
  const char* const fn = "zero_rms_norm_grad";
  if (!args) return error(fn, "args is NULL");
  const zero_rms_grad_args_t& A = *args;
  if (A.rows < 0 || A.rows >= kMaxLd) return error(fn, "rows out of range");
  if (A.cols < 1 || A.cols > zk::kMaxNormCols) return error(fn, "cols must lie in [1, 8192]");
  if (A.reserved != 0) return error(fn, "reserved must be 0");
  if (bytes_of(A.dy_dtype) == 0 || bytes_of(A.h_dtype) == 0) return error(fn, "unsupported dtype");
  if (!stream_types(A.dy_dtype, A.h_dtype)) return error(fn, "h must be of dy's type or fp32");
  int rc;
  if ((rc = matrix(fn, "dy", A.dy, A.rows, A.cols, A.ld_dy, A.dy_dtype))) return rc;
  if (A.rows > 0 && (A.h != nullptr) == (A.held != nullptr)) return error(fn, "exactly one of h and held is given");
  if (A.h && (rc = matrix(fn, "h", A.h, A.rows, A.cols, A.ld_h, A.h_dtype))) return rc;
  if (A.held && (rc = held_matrix(fn, "held", A.held, A.rows, A.cols))) return rc;
  if ((rc = vector(fn, "rstd", A.rstd, A.rows, ZERO_F32))) return rc;
  if (A.weight && (rc = vector(fn, "the weight", A.weight, A.cols, A.weight_dtype))) return rc;
  if (A.dres && (rc = matrix(fn, "dres", A.dres, A.rows, A.cols, A.ld_dres, A.h_dtype))) return rc;
  if ((rc = matrix(fn, "dh", A.dh, A.rows, A.cols, A.ld_dh, A.h_dtype))) return rc;
  const int64_t need = zero_rms_grad_ws_bytes(A.rows, A.cols);
  if (A.dweight) {
    if ((rc = vector(fn, "dweight", A.dweight, A.cols, A.dweight_dtype))) return rc;
    if (!A.ws || A.ws_bytes < need)
      return fail(ZERO_EINVAL, std::string(fn) + ": the workspace needs " + std::to_string(need) + " bytes");
    if (!aligned(A.ws, 16)) return fail(ZERO_EALIGN, std::string(fn) + ": the workspace must be 16-byte aligned");
  }
  const int yb = bytes_of(A.dy_dtype), hb = bytes_of(A.h_dtype);
  Ranges r;
  const int dy = r.add(A.dy, A.rows, A.cols, A.ld_dy, yb, false);
  const int dh = r.add(A.dh, A.rows, A.cols, A.ld_dh, hb, true);
  if (in_place(A.dh, A.ld_dh, A.h_dtype, A.dy, A.ld_dy, A.dy_dtype, A.rows)) r.allow(dh, dy);
  if (A.h) {
    const int h = r.add(A.h, A.rows, A.cols, A.ld_h, hb, false);
    if (in_place(A.dh, A.ld_dh, A.h_dtype, A.h, A.ld_h, A.h_dtype, A.rows)) r.allow(dh, h);
  }
  if (A.dres) {
    const int d = r.add(A.dres, A.rows, A.cols, A.ld_dres, hb, false);
    if (in_place(A.dh, A.ld_dh, A.h_dtype, A.dres, A.ld_dres, A.h_dtype, A.rows)) r.allow(dh, d);
  }
  if (A.held && A.rows > 0) {
    r.add_codes(A.held, A.rows, A.cols, false);
    r.add_scales(A.held, A.rows, A.cols, false);
  }
  if (A.rows > 0) r.add(vector_span(A.rstd, A.rows, ZERO_F32), false);
  if (A.weight) r.add(vector_span(A.weight, A.cols, A.weight_dtype), false);
  if (A.dweight) {
    r.add(vector_span(A.dweight, A.cols, A.dweight_dtype), true);
    r.add(span(A.ws, need), true);
  }
  if (r.clash()) return error(fn, "what is written overlaps something else");

  zk::RmsGradLaunch a{};
  a.dy = static_cast<const char*>(A.dy);
  a.dy_end = end_of(span(A.dy, A.rows, A.cols, A.ld_dy, yb));
  a.ld_dy = A.ld_dy * yb;
  if (A.h) {
    a.h = static_cast<const char*>(A.h);
    a.h_end = end_of(span(A.h, A.rows, A.cols, A.ld_h, hb));
    a.ld_h = A.ld_h * hb;
  }
  if (A.rows > 0) a.held = held_launch(A.held, A.rows, A.cols);
  a.rstd = A.rstd;
  if (A.weight) {
    a.weight = static_cast<const char*>(A.weight);
    a.weight_end = end_of(vector_span(A.weight, A.cols, A.weight_dtype));
    a.weight_type = A.weight_dtype;
  }
  if (A.dres) {
    a.dres = static_cast<const char*>(A.dres);
    a.dres_end = end_of(span(A.dres, A.rows, A.cols, A.ld_dres, hb));
    a.ld_dres = A.ld_dres * hb;
  }
  a.dh = static_cast<char*>(A.dh);
  a.ld_dh = A.ld_dh * hb;
  a.dweight = static_cast<char*>(A.dweight);
  a.dweight_type = A.dweight_dtype;
  a.accumulate = A.accumulate != 0;
  a.partial = static_cast<float*>(A.ws);
  a.rows = A.rows;
  a.cols = (uint32_t)A.cols;
  a.partials = A.rows > 0 ? zk::rms_grad_partials(A.rows, A.cols) : 0;
  return zk::launch_rms_grad(a, A.dy_dtype, A.h_dtype, stream);
}

// --- the gated projections -------------------------------------------------------

int gated_sizes(const char* fn, const zero_gated_args_t* A, bool with_dim) {
  if (!A) return error(fn, "args is NULL");
  if (A->tokens < 0 || A->tokens >= kMaxRows) return error(fn, "tokens must lie in [0, 2^31)");
  if (A->hidden < 1 || A->hidden >= kMaxRows) return error(fn, "hidden must lie in [1, 2^31)");
  if (with_dim && (A->dim < 1 || A->dim >= kMaxRows)) return error(fn, "dim must lie in [1, 2^31)");
  if (bytes_of(A->dtype) == 0) return error(fn, "unsupported dtype");
  return ZERO_OK;
}

int known_act(const char* fn, int32_t act) {
  return act == ZERO_SILU || act == ZERO_GELU ? ZERO_OK : error(fn, "unknown activation");
}

int gated(const zero_gated_args_t* args, void* stream) {
  const char* const fn = "zero_gated";
  int rc;
  if ((rc = gated_sizes(fn, args, true))) return rc;
  const zero_gated_args_t& A = *args;
  if ((rc = known_act(fn, A.act))) return rc;
  const int eb = bytes_of(A.dtype);
  if ((rc = matrix(fn, "x", A.x, A.tokens, A.dim, A.ld_x, A.dtype))) return rc;
  if ((rc = matrix(fn, "w_gate", A.w_gate, A.hidden, A.dim, A.ld_w_gate, A.dtype))) return rc;
  if ((rc = matrix(fn, "w_up", A.w_up, A.hidden, A.dim, A.ld_w_up, A.dtype))) return rc;
  if ((rc = matrix(fn, "a", A.a, A.tokens, A.hidden, A.ld_a, A.dtype))) return rc;
  if ((A.g != nullptr) != (A.u != nullptr) || (A.g8 != nullptr) != (A.u8 != nullptr) || (A.g && A.g8))
    return error(fn, "g and u are kept both or neither, as tensors or in 8 bits");
  if (A.g && (rc = matrix(fn, "g", A.g, A.tokens, A.hidden, A.ld_g, A.dtype))) return rc;
  if (A.u && (rc = matrix(fn, "u", A.u, A.tokens, A.hidden, A.ld_u, A.dtype))) return rc;
  if (A.g8 && (rc = held_matrix(fn, "g8", A.g8, A.tokens, A.hidden))) return rc;
  if (A.u8 && (rc = held_matrix(fn, "u8", A.u8, A.tokens, A.hidden))) return rc;
  if (A.tokens == 0) return ZERO_OK;
  Ranges r;
  r.add(A.x, A.tokens, A.dim, A.ld_x, eb, false);
  r.add(A.w_gate, A.hidden, A.dim, A.ld_w_gate, eb, false);
  r.add(A.w_up, A.hidden, A.dim, A.ld_w_up, eb, false);
  r.add(A.a, A.tokens, A.hidden, A.ld_a, eb, true);
  if (A.g) {
    r.add(A.g, A.tokens, A.hidden, A.ld_g, eb, true);
    r.add(A.u, A.tokens, A.hidden, A.ld_u, eb, true);
  }
  if (A.g8)
    for (const zero_held_t* h : {A.g8, A.u8}) {
      r.add_codes(h, A.tokens, A.hidden, true);
      r.add_scales(h, A.tokens, A.hidden, true);
    }
  if (r.clash()) return error(fn, "what is written overlaps something else");

  zk::ProductLaunch a{};
  a.q[0] = static_cast<const char*>(A.x);
  a.q_end[0] = end_of(r.s[0]);
  a.ld_q[0] = A.ld_x * eb;
  a.p[0] = static_cast<const char*>(A.w_gate);
  a.p_end[0] = end_of(r.s[1]);
  a.ld_p[0] = A.ld_w_gate * eb;
  a.p[1] = static_cast<const char*>(A.w_up);
  a.p_end[1] = end_of(r.s[2]);
  a.ld_p[1] = A.ld_w_up * eb;
  a.out[0] = static_cast<char*>(A.a);
  a.ld_out[0] = A.ld_a * eb;
  a.kept[0] = static_cast<char*>(A.g);
  a.kept[1] = static_cast<char*>(A.u);
  a.ld_kept[0] = A.ld_g * eb;
  a.ld_kept[1] = A.ld_u * eb;
  a.held[0] = held_launch(A.g8, A.tokens, A.hidden);
  a.held[1] = held_launch(A.u8, A.tokens, A.hidden);
  a.rows = A.tokens;
  a.cols = A.hidden;
  a.k = A.dim;
  a.act = A.act;
  return zk::launch_product(zk::kForward, a, A.dtype, stream);
}

int gated_grad(const zero_gated_args_t* args, void* stream) {
  const char* const fn = "zero_gated_grad";
  int rc;
  if ((rc = gated_sizes(fn, args, false))) return rc;
  const zero_gated_args_t& A = *args;
  if ((rc = known_act(fn, A.act))) return rc;
  const int eb = bytes_of(A.dtype);
  const int64_t n = A.tokens, h = A.hidden;
  if ((rc = matrix(fn, "da", A.da, n, h, A.ld_da, A.dtype))) return rc;
  if ((rc = matrix(fn, "dg", A.dg, n, h, A.ld_dg, A.dtype))) return rc;
  if ((rc = matrix(fn, "du", A.du, n, h, A.ld_du, A.dtype))) return rc;
  if (A.a && (rc = matrix(fn, "a", A.a, n, h, A.ld_a, A.dtype))) return rc;
  if (n > 0 && ((A.g != nullptr) != (A.u != nullptr) || (A.g8 != nullptr) != (A.u8 != nullptr) ||
                (A.g != nullptr) == (A.g8 != nullptr)))
    return error(fn, "g and u are given as tensors or in 8 bits");
  if (A.g && (rc = matrix(fn, "g", A.g, n, h, A.ld_g, A.dtype))) return rc;
  if (A.u && (rc = matrix(fn, "u", A.u, n, h, A.ld_u, A.dtype))) return rc;
  if (A.g8 && (rc = held_matrix(fn, "g8", A.g8, n, h))) return rc;
  if (A.u8 && (rc = held_matrix(fn, "u8", A.u8, n, h))) return rc;
  if (n == 0) return ZERO_OK;
  Ranges r;
  struct In {
    const void* p;
    int64_t ld;
    int at;
  } in[3] = {{A.da, A.ld_da, 0}, {A.g, A.ld_g, 0}, {A.u, A.ld_u, 0}};
  for (In& i : in) i.at = i.p ? r.add(i.p, n, h, i.ld, eb, false) : -1;
  if (A.g8)
    for (const zero_held_t* k : {A.g8, A.u8}) {
      r.add_codes(k, n, h, false);
      r.add_scales(k, n, h, false);
    }
  const struct {
    void* p;
    int64_t ld;
  } out[3] = {{A.dg, A.ld_dg}, {A.du, A.ld_du}, {A.a, A.ld_a}};
  for (const auto& o : out) {
    if (!o.p) continue;
    const int at = r.add(o.p, n, h, o.ld, eb, true);
    for (const In& i : in)
      if (i.p && in_place(o.p, o.ld, A.dtype, i.p, i.ld, A.dtype, n)) r.allow(at, i.at);
  }
  if (r.clash()) return error(fn, "what is written overlaps something else");

  zk::GatedGradLaunch a{};
  a.da = static_cast<const char*>(A.da);
  a.g = static_cast<const char*>(A.g);
  a.u = static_cast<const char*>(A.u);
  a.hg = held_launch(A.g8, n, h);
  a.hu = held_launch(A.u8, n, h);
  a.dg = static_cast<char*>(A.dg);
  a.du = static_cast<char*>(A.du);
  a.a = static_cast<char*>(A.a);
  a.da_end = end_of(r.s[0]);
  if (A.g) {
    a.g_end = end_of(r.s[1]);
    a.u_end = end_of(r.s[2]);
  }
  a.ld_da = A.ld_da * eb;
  a.ld_g = A.ld_g * eb;
  a.ld_u = A.ld_u * eb;
  a.ld_dg = A.ld_dg * eb;
  a.ld_du = A.ld_du * eb;
  a.ld_a = A.ld_a * eb;
  a.cols = (uint32_t)h;
  a.groups = zk::fast_div((uint32_t)(4 * blocks_of(h)));
  const int64_t per_launch = std::max<int64_t>(1, zk::kMaxUnits / a.groups.d);
  for (int64_t i = 0; i < n; i += per_launch) {
    a.rows = (uint32_t)std::min(per_launch, n - i);
    a.units = a.rows * a.groups.d;
    if ((rc = zk::launch_gated_grad(a, A.dtype, A.act, stream))) return rc;
    a.da += per_launch * a.ld_da;
    if (a.g) {
      a.g += per_launch * a.ld_g;
      a.u += per_launch * a.ld_u;
    }
    advance(a.hg, per_launch);
    advance(a.hu, per_launch);
    a.dg += per_launch * a.ld_dg;
    a.du += per_launch * a.ld_du;
    if (a.a) a.a += per_launch * a.ld_a;
  }
  return ZERO_OK;
}

bool gated_sizes_ok(int64_t tokens, int64_t dim, int64_t hidden) {
  return tokens >= 0 && tokens < kMaxRows && dim >= 1 && dim < kMaxRows && hidden >= 1 && hidden < kMaxRows;
}

int workspace(const char* fn, const zero_gated_args_t& A, int64_t need) {
  if (!A.ws || A.ws_bytes < need)
    return fail(ZERO_EINVAL, std::string(fn) + ": the workspace needs " + std::to_string(need) + " bytes");
  if (!aligned(A.ws, 16)) return fail(ZERO_EALIGN, std::string(fn) + ": the workspace must be 16-byte aligned");
  return ZERO_OK;
}

int input_grad(const zero_gated_args_t* args, void* stream) {
  const char* const fn = "zero_gated_input_grad";
  int rc;
  if ((rc = gated_sizes(fn, args, true))) return rc;
  const zero_gated_args_t& A = *args;
  const int eb = bytes_of(A.dtype);
  if ((rc = matrix(fn, "dg", A.dg, A.tokens, A.hidden, A.ld_dg, A.dtype))) return rc;
  if ((rc = matrix(fn, "du", A.du, A.tokens, A.hidden, A.ld_du, A.dtype))) return rc;
  if ((rc = matrix(fn, "w_gate", A.w_gate, A.hidden, A.dim, A.ld_w_gate, A.dtype))) return rc;
  if ((rc = matrix(fn, "w_up", A.w_up, A.hidden, A.dim, A.ld_w_up, A.dtype))) return rc;
  if ((rc = matrix(fn, "dx", A.dx, A.tokens, A.dim, A.ld_dx, A.dtype))) return rc;
  if (A.tokens == 0) return ZERO_OK;
  const int64_t need = zero_gated_ws_bytes(A.tokens, A.dim, A.hidden);
  if ((rc = workspace(fn, A, need))) return rc;
  Ranges r;
  r.add(A.dg, A.tokens, A.hidden, A.ld_dg, eb, false);
  r.add(A.du, A.tokens, A.hidden, A.ld_du, eb, false);
  r.add(A.w_gate, A.hidden, A.dim, A.ld_w_gate, eb, false);
  r.add(A.w_up, A.hidden, A.dim, A.ld_w_up, eb, false);
  r.add(A.dx, A.tokens, A.dim, A.ld_dx, eb, true);
  r.add(span(A.ws, need), true);
  if (r.clash()) return error(fn, "what is written overlaps something else");
  zk::ProductLaunch a{};
  a.q[0] = static_cast<const char*>(A.dg);
  a.q[1] = static_cast<const char*>(A.du);
  a.p[0] = static_cast<const char*>(A.w_gate);
  a.p[1] = static_cast<const char*>(A.w_up);
  for (int i = 0; i < 2; ++i) {
    a.q_end[i] = end_of(r.s[i]);
    a.p_end[i] = end_of(r.s[2 + i]);
  }
  a.ld_q[0] = A.ld_dg * eb;
  a.ld_q[1] = A.ld_du * eb;
  a.ld_p[0] = A.ld_w_gate * eb;
  a.ld_p[1] = A.ld_w_up * eb;
  a.out[0] = static_cast<char*>(A.dx);
  a.ld_out[0] = A.ld_dx * eb;
  a.rows = A.tokens;
  a.cols = A.dim;
  a.k = A.hidden;
  a.ws = static_cast<float*>(A.ws);
  return zk::launch_product(zk::kInput, a, A.dtype, stream);
}

int weight_grad(const zero_gated_args_t* args, void* stream) {
  const char* const fn = "zero_gated_weight_grad";
  int rc;
  if ((rc = gated_sizes(fn, args, true))) return rc;
  const zero_gated_args_t& A = *args;
  const int eb = bytes_of(A.dtype);
  if ((rc = matrix(fn, "dg", A.dg, A.tokens, A.hidden, A.ld_dg, A.dtype))) return rc;
  if ((rc = matrix(fn, "du", A.du, A.tokens, A.hidden, A.ld_du, A.dtype))) return rc;
  if ((rc = matrix(fn, "x", A.x, A.tokens, A.dim, A.ld_x, A.dtype))) return rc;
  if ((rc = matrix(fn, "dw_gate", A.dw_gate, A.hidden, A.dim, A.ld_dw_gate, A.dw_dtype))) return rc;
  if ((rc = matrix(fn, "dw_up", A.dw_up, A.hidden, A.dim, A.ld_dw_up, A.dw_dtype))) return rc;
  const int64_t need = zero_gated_ws_bytes(A.tokens, A.dim, A.hidden);
  if ((rc = workspace(fn, A, need))) return rc;
  const int wb = bytes_of(A.dw_dtype);
  Ranges r;
  r.add(A.dg, A.tokens, A.hidden, A.ld_dg, eb, false);
  r.add(A.du, A.tokens, A.hidden, A.ld_du, eb, false);
  r.add(A.x, A.tokens, A.dim, A.ld_x, eb, false);
  r.add(A.dw_gate, A.hidden, A.dim, A.ld_dw_gate, wb, true);
  r.add(A.dw_up, A.hidden, A.dim, A.ld_dw_up, wb, true);
  r.add(span(A.ws, need), true);
  if (r.clash()) return error(fn, "what is written overlaps something else");
  zk::ProductLaunch a{};
  a.q[0] = static_cast<const char*>(A.dg);
  a.q[1] = static_cast<const char*>(A.du);
  a.q_end[0] = end_of(r.s[0]);
  a.q_end[1] = end_of(r.s[1]);
  a.ld_q[0] = A.ld_dg * eb;
  a.ld_q[1] = A.ld_du * eb;
  a.p[0] = static_cast<const char*>(A.x);
  a.p_end[0] = end_of(r.s[2]);
  a.ld_p[0] = A.ld_x * eb;
  a.out[0] = static_cast<char*>(A.dw_gate);
  a.out[1] = static_cast<char*>(A.dw_up);
  a.ld_out[0] = A.ld_dw_gate * wb;
  a.ld_out[1] = A.ld_dw_up * wb;
  a.rows = A.hidden;
  a.cols = A.dim;
  a.k = A.tokens;
  a.out_type = A.dw_dtype;
  a.accumulate = A.accumulate != 0;
  a.ws = static_cast<float*>(A.ws);
  return zk::launch_product(zk::kWeight, a, A.dtype, stream);
}

}  // namespace

extern "C" int zero_pack8(const void* x, int64_t ld_x, zero_dtype_t x_dtype, int64_t rows, int64_t cols,
                          const zero_held_t* held, void* stream) {
  return guarded([&] { return hold("zero_pack8", true, const_cast<void*>(x), ld_x, x_dtype, held, rows, cols, stream); });
}

extern "C" int zero_unpack8(const zero_held_t* held, int64_t rows, int64_t cols, void* out, int64_t ld_out,
                            zero_dtype_t out_dtype, void* stream) {
  return guarded([&] { return hold("zero_unpack8", false, out, ld_out, out_dtype, held, rows, cols, stream); });
}

extern "C" int zero_rms_norm(const zero_rms_args_t* args, void* stream) {
  return guarded([&] { return rms(args, stream); });
}

extern "C" int64_t zero_rms_grad_ws_bytes(int64_t rows, int64_t cols) {
  return rms_grad_sizes_ok(rows, cols) ? 256 + zk::rms_grad_partials_most(rows) * cols * 4 : 0;
}

extern "C" int zero_rms_norm_grad(const zero_rms_grad_args_t* args, void* stream) {
  return guarded([&] { return rms_grad(args, stream); });
}

extern "C" int64_t zero_gated_ws_bytes(int64_t tokens, int64_t dim, int64_t hidden) {
  return gated_sizes_ok(tokens, dim, hidden) ? 256 + zk::product_ws_bytes(tokens, dim, hidden) : 0;
}

extern "C" int zero_gated(const zero_gated_args_t* args, void* stream) {
  return guarded([&] { return gated(args, stream); });
}
extern "C" int zero_gated_grad(const zero_gated_args_t* args, void* stream) {
  return guarded([&] { return gated_grad(args, stream); });
}
extern "C" int zero_gated_input_grad(const zero_gated_args_t* args, void* stream) {
  return guarded([&] { return input_grad(args, stream); });
}
extern "C" int zero_gated_weight_grad(const zero_gated_args_t* args, void* stream) {
  return guarded([&] { return weight_grad(args, stream); });
}
