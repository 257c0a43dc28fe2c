// C ABI of the input layer: argument validation (before anything is enqueued)
// and the launches of embedding lookup, embedding gradient and dropout.
#include <algorithm>
#include <cmath>
#include <string>

#include "abi_checks.h"
#include "input.h"

namespace {

// the drop of `rows` rows, as the kernels take it
int make_drop(const char* fn, const zero_drop_t* d, int64_t rows, zk::DropK* k, double* ks) {
  *k = zk::DropK{};
  k->ks = 1.0f;
  *ks = 1.0;
  if (!d) return ZERO_OK;
  if (!(d->p >= 0.0 && d->p <= 1.0)) return fail(ZERO_EINVAL, std::string(fn) + ": p must lie in [0, 1]");
  if (d->reserved != 0) return fail(ZERO_EINVAL, std::string(fn) + ": drop.reserved must be 0");
  if (!d->step_dev && (d->step < 0 || d->step >= (int64_t(1) << 32)))
    return fail(ZERO_EINVAL, std::string(fn) + ": the step must lie in [0, 2^32)");
  if (d->step_dev && !aligned(d->step_dev, 8)) return fail(ZERO_EALIGN, std::string(fn) + ": step_dev must be 8-byte aligned");
  if (d->row0 < 0 || d->row0 > (int64_t(1) << 32) - rows)
    return fail(ZERO_EINVAL, std::string(fn) + ": row0 + rows must lie in [0, 2^32]");
  const double t = std::nearbyint(d->p * 65536.0);
  k->thr = (uint32_t)t;
  *ks = t < 65536.0 ? 65536.0 / (65536.0 - t) : 0.0;
  k->ks = (float)*ks;
  k->key0 = (uint32_t)d->seed;
  k->key1 = (uint32_t)(d->seed >> 32);
  k->step = (uint32_t)(d->step_dev ? 0 : d->step);
  k->site = d->site;
  k->step_dev = d->step_dev;
  k->row0 = (uint32_t)d->row0;
  return ZERO_OK;
}

bool drop_overlaps(const zero_drop_t* d, const Span& out) {
  return d && d->step_dev && overlap(span(d->step_dev, 8), out);
}

// --- gradient workspace: n_valid, order, has, partial rows ---------------------
constexpr int64_t kHead = 256;

int64_t round_up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }
int64_t slabs_of(int64_t dim) { return (dim + 511) / 512; }
int64_t has_offset(int64_t n) { return kHead + round_up(n * 16, 256); }
int64_t partial_offset(int64_t n, int64_t rows) { return has_offset(n) + round_up(rows, 256); }
// Pairs of partial rows (512 columns of a chunk and of a tail): ceil(n / chunk) * slabs
// are used.  The chunk halves as a batch shrinks, so that number rises again below
// each such step; what is set aside must not, or a workspace of the largest batch would
// be too small for others.  Chunks under the longest leave fewer than kGradWaves whole
// ones and one begun in each slab, and no more than the shortest chunks do; either bound
// and the longest chunks' own number grow with n and dim.
int64_t partial_pairs(int64_t n, int64_t dim) {
  const int64_t slabs = slabs_of(dim), longest = int64_t(1) << zk::kMaxLgChunk;
  return std::max(std::min((n + zk::kMinChunk - 1) / zk::kMinChunk * slabs, zk::kGradWaves + slabs),
                  (n + longest - 1) / longest * slabs);
}
int64_t ws_need(int64_t n, int64_t rows, int64_t dim) {
  return partial_offset(n, rows) + partial_pairs(n, dim) * 2 * 512 * 4;
}

// The waves that sum, at most two a pair, and all workgroups are counted in 32 bits.
bool grad_sizes_ok(int64_t n, int64_t rows, int64_t dim) {
  return n >= 0 && n < kMax31 && rows >= 0 && rows < kMax31 && dim >= 1 && dim < kMax31 &&
         partial_pairs(n, dim) < kMax31 - 4;
}

int dropout(const void* x, int64_t ld_x, zero_dtype_t xt, const void* res, int64_t ld_res, void* out,
            int64_t ld_out, zero_dtype_t ot, int64_t rows, int64_t cols, const zero_drop_t* drop, void* stream) {
  const char* const fn = "zero_dropout";
  if (rows < 0 || rows >= kMaxLd) return fail(ZERO_EINVAL, std::string(fn) + ": rows out of range");
  if (cols < 1 || cols >= kMax31) return fail(ZERO_EINVAL, std::string(fn) + ": cols must lie in [1, 2^31)");
  int rc;
  if ((rc = matrix(fn, "x", x, rows, cols, ld_x, xt))) return rc;
  if (res && (rc = matrix(fn, "the residual", res, rows, cols, ld_res, ot))) return rc;
  if ((rc = matrix(fn, "out", out, rows, cols, ld_out, ot))) return rc;
  zk::DropK k;
  double ks;
  if ((rc = make_drop(fn, drop, rows, &k, &ks))) return rc;
  if (rows == 0) return ZERO_OK;
  const Span so = span(out, rows, cols, ld_out, bytes_of(ot));
  const bool same_x = out == x && xt == ot && (ld_out == ld_x || rows == 1);
  if (!same_x && overlap(so, span(x, rows, cols, ld_x, bytes_of(xt))))
    return fail(ZERO_EINVAL, std::string(fn) + ": out overlaps x");
  const bool same_res = out == res && (ld_out == ld_res || rows == 1);
  if (res && !same_res && overlap(so, span(res, rows, cols, ld_res, bytes_of(ot))))
    return fail(ZERO_EINVAL, std::string(fn) + ": out overlaps the residual");
  if (drop_overlaps(drop, so)) return fail(ZERO_EINVAL, std::string(fn) + ": out overlaps step_dev");

  const int64_t groups = (cols + zk::kGroup - 1) / zk::kGroup;
  const int64_t per_launch = std::max<int64_t>(1, zk::kMaxUnits / groups);
  for (int64_t r = 0; r < rows; r += per_launch) {
    zk::DropoutLaunch a{};
    a.ld_x = ld_x * bytes_of(xt);
    a.ld_res = ld_res * bytes_of(ot);
    a.ld_out = ld_out * bytes_of(ot);
    a.x = static_cast<const char*>(x) + r * a.ld_x;
    a.res = res ? static_cast<const char*>(res) + r * a.ld_res : nullptr;
    a.out = static_cast<char*>(out) + r * a.ld_out;
    a.x_end = end_of(span(x, rows, cols, ld_x, bytes_of(xt)));
    a.res_end = res ? end_of(span(res, rows, cols, ld_res, bytes_of(ot))) : nullptr;
    a.rows = (uint32_t)std::min(per_launch, rows - r);
    a.cols = (uint32_t)cols;
    a.units = (uint32_t)(a.rows * groups);
    a.groups = zk::fast_div((uint32_t)groups);
    a.drop = k;
    a.drop.row0 += (uint32_t)r;
    if ((rc = zk::launch_dropout(a, xt, ot, stream))) return rc;
  }
  return ZERO_OK;
}

int lookup(const zero_embed_args_t* args, void* stream) {
  const char* const fn = "zero_embed_lookup";
  if (!args) return fail(ZERO_EINVAL, std::string(fn) + ": args is NULL");
  const zero_embed_args_t& A = *args;
  if (A.n_ids < 0 || A.n_ids >= kMax31) return fail(ZERO_EINVAL, std::string(fn) + ": n_ids must lie in [0, 2^31)");
  if (A.dim < 1 || A.dim >= kMax31) return fail(ZERO_EINVAL, std::string(fn) + ": dim must lie in [1, 2^31)");
  if (A.rows < 0 || A.pos_rows < 0) return fail(ZERO_EINVAL, std::string(fn) + ": a table has a negative number of rows");
  if (A.id_bytes != 4 && A.id_bytes != 8) return fail(ZERO_EINVAL, std::string(fn) + ": id_bytes must be 4 or 8");
  if (!std::isfinite(A.scale)) return fail(ZERO_EINVAL, std::string(fn) + ": scale is not finite");
  int rc;
  if ((rc = matrix(fn, "the table", A.table, A.rows, A.dim, A.ld_table, A.table_dtype))) return rc;
  const bool with_pos = A.pos_table != nullptr;
  if (with_pos) {
    if ((rc = matrix(fn, "the position table", A.pos_table, A.pos_rows, A.dim, A.ld_pos, A.table_dtype))) return rc;
    if (!A.pos && A.pos_period < 1) return fail(ZERO_EINVAL, std::string(fn) + ": pos_period must be at least 1");
    if (A.pos && !aligned(A.pos, A.id_bytes)) return fail(ZERO_EALIGN, std::string(fn) + ": pos is not element aligned");
  } else if (A.pos) {
    return fail(ZERO_EINVAL, std::string(fn) + ": pos without a position table");
  }
  if ((rc = matrix(fn, "out", A.out, A.n_ids, A.dim, A.ld_out, A.out_dtype))) return rc;
  zk::DropK k;
  double ks;
  if ((rc = make_drop(fn, A.drop, A.n_ids, &k, &ks))) return rc;
  if (A.n_ids == 0) return ZERO_OK;
  if (!A.ids) return fail(ZERO_EINVAL, std::string(fn) + ": ids is NULL");
  if (!aligned(A.ids, A.id_bytes)) return fail(ZERO_EALIGN, std::string(fn) + ": ids is not element aligned");
  const int tb = bytes_of(A.table_dtype), ob = bytes_of(A.out_dtype);
  const Span so = span(A.out, A.n_ids, A.dim, A.ld_out, ob);
  if (overlap(so, span(A.table, A.rows, A.dim, A.ld_table, tb)) ||
      overlap(so, span(A.ids, A.n_ids * A.id_bytes)) ||
      (with_pos && overlap(so, span(A.pos_table, A.pos_rows, A.dim, A.ld_pos, tb))) ||
      (A.pos && overlap(so, span(A.pos, A.n_ids * A.id_bytes))) || drop_overlaps(A.drop, so))
    return fail(ZERO_EINVAL, std::string(fn) + ": out overlaps an input");

  const int64_t groups = (A.dim + zk::kGroup - 1) / zk::kGroup;
  const int64_t per_launch = std::max<int64_t>(1, zk::kMaxUnits / groups);
  for (int64_t t = 0; t < A.n_ids; t += per_launch) {
    zk::LookupLaunch a{};
    a.table = static_cast<const char*>(A.table);
    a.pos_table = static_cast<const char*>(A.pos_table);
    a.table_end = end_of(span(A.table, A.rows, A.dim, A.ld_table, tb));
    a.pos_end = with_pos ? end_of(span(A.pos_table, A.pos_rows, A.dim, A.ld_pos, tb)) : nullptr;
    a.ids = static_cast<const char*>(A.ids) + t * A.id_bytes;
    a.pos = A.pos ? static_cast<const char*>(A.pos) + t * A.id_bytes : nullptr;
    a.ld_table = A.ld_table * tb;
    a.ld_pos = A.ld_pos * tb;
    a.ld_out = A.ld_out * ob;
    a.out = static_cast<char*>(A.out) + t * a.ld_out;
    a.rows = A.rows;
    a.id0 = A.id0;
    a.pos_rows = A.pos_rows;
    a.id64 = A.id_bytes == 8;
    a.n = (uint32_t)std::min(per_launch, A.n_ids - t);
    a.dim = (uint32_t)A.dim;
    a.units = (uint32_t)(a.n * groups);
    a.groups = zk::fast_div((uint32_t)groups);
    a.t0 = (uint32_t)t;
    // t < 2^31, so a longer period is none
    a.period = zk::fast_div((uint32_t)(with_pos && !A.pos ? std::min<int64_t>(A.pos_period, kMax31 - 1) : 1));
    a.scale = A.scale;
    a.drop = k;
    if ((rc = zk::launch_lookup(a, A.table_dtype, A.out_dtype, stream))) return rc;
  }
  return ZERO_OK;
}

int gradient(const zero_embed_grad_args_t* args, void* stream) {
  const char* const fn = "zero_embed_grad";
  if (!args) return fail(ZERO_EINVAL, std::string(fn) + ": args is NULL");
  const zero_embed_grad_args_t& A = *args;
  if (A.n_ids < 0 || A.n_ids >= kMax31) return fail(ZERO_EINVAL, std::string(fn) + ": n_ids must lie in [0, 2^31)");
  if (A.rows < 0 || A.rows >= kMax31) return fail(ZERO_EINVAL, std::string(fn) + ": rows must lie in [0, 2^31)");
  if (A.dim < 1 || A.dim >= kMax31) return fail(ZERO_EINVAL, std::string(fn) + ": dim must lie in [1, 2^31)");
  if (!grad_sizes_ok(A.n_ids, A.rows, A.dim)) return fail(ZERO_EINVAL, std::string(fn) + ": n_ids, rows and dim are out of range together");
  if (A.id_bytes != 4 && A.id_bytes != 8) return fail(ZERO_EINVAL, std::string(fn) + ": id_bytes must be 4 or 8");
  if (!A.ids && A.n_ids > 0 && A.period < 1)
    return fail(ZERO_EINVAL, std::string(fn) + ": ids is NULL and the period is not at least 1");
  if (!std::isfinite(A.scale)) return fail(ZERO_EINVAL, std::string(fn) + ": scale is not finite");
  int rc;
  if ((rc = matrix(fn, "dy", A.dy, A.n_ids, A.dim, A.ld_dy, A.dy_dtype))) return rc;
  if ((rc = matrix(fn, "grad", A.grad, A.rows, A.dim, A.ld_grad, A.grad_dtype))) return rc;
  if (A.ids && !aligned(A.ids, A.id_bytes)) return fail(ZERO_EALIGN, std::string(fn) + ": ids is not element aligned");
  zk::DropK k;
  double ks;
  if ((rc = make_drop(fn, A.drop, A.n_ids, &k, &ks))) return rc;
  const double factor = (double)A.scale * ks;
  if (!std::isfinite((float)factor)) return fail(ZERO_EINVAL, std::string(fn) + ": scale / (1 - p) is not finite in fp32");
  if (A.rows == 0) return ZERO_OK;
  const int64_t need = ws_need(A.n_ids, A.rows, A.dim);
  if (!A.ws || A.ws_bytes < need)
    return fail(ZERO_EINVAL, std::string(fn) + ": the workspace needs " + std::to_string(need) + " bytes");
  if (!aligned(A.ws, 16)) return fail(ZERO_EALIGN, std::string(fn) + ": the workspace must be 16-byte aligned");
  const Span sg = span(A.grad, A.rows, A.dim, A.ld_grad, bytes_of(A.grad_dtype)), sw = span(A.ws, need);
  const Span sd = span(A.dy, A.n_ids, A.dim, A.ld_dy, bytes_of(A.dy_dtype));
  const Span si = span(A.ids, A.n_ids * A.id_bytes);
  if (overlap(sg, sw)) return fail(ZERO_EINVAL, std::string(fn) + ": grad overlaps the workspace");
  for (const Span& o : {sg, sw})
    if (overlap(o, sd) || overlap(o, si) || drop_overlaps(A.drop, o))
      return fail(ZERO_EINVAL, std::string(fn) + ": grad or the workspace overlaps an input");

  zk::GradLaunch a{};
  a.dy = static_cast<const char*>(A.dy);
  a.dy_end = end_of(sd);
  a.ids = A.ids;
  a.grad = static_cast<char*>(A.grad);
  a.ld_dy = A.ld_dy * bytes_of(A.dy_dtype);
  a.ld_grad = A.ld_grad * bytes_of(A.grad_dtype);
  a.id0 = A.id0;
  a.rows = A.rows;
  a.id64 = A.id_bytes == 8;
  a.accumulate = A.accumulate != 0;
  a.n = (uint32_t)A.n_ids;
  a.dim = (uint32_t)A.dim;
  a.factor = (float)factor;
  a.drop = k;
  char* const ws = static_cast<char*>(A.ws);
  a.n_valid = reinterpret_cast<uint32_t*>(ws);
  a.order = reinterpret_cast<uint4*>(ws + kHead);
  a.has = reinterpret_cast<uint8_t*>(ws + has_offset(A.n_ids));
  a.partial = reinterpret_cast<float*>(ws + partial_offset(A.n_ids, A.rows));
  a.longest = (uint32_t)A.n_ids;
  int64_t positions = A.n_ids;
  if (A.ids) {
    uint32_t lg = 0;
    while ((1 << lg) < zk::kSortMinClasses || (A.rows + (int64_t(1) << lg) - 1) >> lg > zk::kSortKeys) ++lg;
    a.lg_classes = lg;
    a.keys = (uint32_t)((A.rows + (int64_t(1) << lg) - 1) >> lg);
  } else if (A.n_ids > 0) {
    // ids run 0 .. period - 1 over and over; id < n % period has one more
    const int64_t period = std::min(A.period, A.n_ids);
    const int64_t occ = A.n_ids / period, more = A.n_ids % period;
    auto start = [&](int64_t id) { return id * occ + std::min(id, more); };
    // the ids among the rows, 0 <= id < period
    const int64_t hi = std::min<int64_t>(period, A.id0 > kMax31 ? 0 : std::max<int64_t>(A.id0 + A.rows, 0));
    const int64_t lo = std::min<int64_t>(std::max<int64_t>(A.id0, 0), hi);
    a.row_lo = hi > lo ? (uint32_t)(lo - A.id0) : 0;
    a.row_hi = hi > lo ? (uint32_t)(hi - A.id0) : 0;
    a.start_lo = (uint32_t)start(lo);
    positions = start(hi) - start(lo);
    a.long_ids = (uint32_t)more;
    a.split = (uint32_t)(more * (occ + 1));
    a.total = (uint32_t)positions;
    a.period = (uint32_t)period;
    a.div_long = zk::fast_div((uint32_t)(occ + 1));
    a.div_short = zk::fast_div((uint32_t)occ);
    a.longest = (uint32_t)(occ + (more > 0 ? 1 : 0));
  }
  a.places = (uint32_t)positions;
  a.lg_chunk = zk::grad_lg_chunk(A.n_ids, A.dim);
  a.window = 1u << (a.lg_chunk - 1);
  a.windows = (uint32_t)((positions + a.window - 1) / a.window);
  a.slabs = (uint32_t)slabs_of(A.dim);
  // with an array of ids the sorted form, by period without one; either zeroes every
  // row of an empty batch's gradient
  return zk::launch_embed_grad(a, A.dy_dtype, A.grad_dtype, stream);
}

}  // namespace

extern "C" int zero_dropout(const void* x, int64_t ld_x, zero_dtype_t x_dtype, const void* residual, int64_t ld_res,
                            void* out, int64_t ld_out, zero_dtype_t out_dtype, int64_t rows, int64_t cols,
                            const zero_drop_t* drop, void* stream) {
  return guarded([&] {
    return dropout(x, ld_x, x_dtype, residual, ld_res, out, ld_out, out_dtype, rows, cols, drop, stream);
  });
}

extern "C" int zero_embed_lookup(const zero_embed_args_t* args, void* stream) {
  return guarded([&] { return lookup(args, stream); });
}

extern "C" int64_t zero_embed_grad_ws_bytes(int64_t n_ids, int64_t rows, int64_t dim) {
  return grad_sizes_ok(n_ids, rows, dim) ? ws_need(n_ids, rows, dim) : 0;
}

extern "C" int zero_embed_grad(const zero_embed_grad_args_t* args, void* stream) {
  return guarded([&] { return gradient(args, stream); });
}
