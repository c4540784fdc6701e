// C ABI entry points of the mixture-of-experts block: validation, kernel argument
// marshalling and launch. Every step runs in the HIP kernels.
#include <hip/hip_runtime_api.h>

#include <algorithm>

#include "moe.h"

using namespace plr;

namespace {

bool a16(const void* p) { return ((uintptr_t)p & 15) == 0; }
bool a4(const void* p) { return ((uintptr_t)p & 3) == 0; }
bool a8(const void* p) { return ((uintptr_t)p & 7) == 0; }

uint64_t elem(int dtype) { return dtype == PLR_F8 ? 1 : dtype == PLR_F32 ? 4 : 2; }
bool is_float(int dtype) { return dtype == PLR_BF16 || dtype == PLR_F16 || dtype == PLR_F32; }

constexpr int64_t kMaxRows = 0x7FFFFFFF;  // row numbers are int32
constexpr int64_t kMaxTokens = 1 << 24;
constexpr int64_t kMaxCols = 1 << 24;
constexpr uint64_t kMaxPitch = 0x7FFFFFF0;  // a row's address is a 32 by 32 bit product away from the first

// Rows of `len` bytes, `pitch` bytes apart.
struct Rows {
  uintptr_t at;
  uint64_t len, pitch;
  int64_t rows;
};
Rows rows_of(const void* p, uint64_t len, uint64_t pitch, int64_t rows) {
  return Rows{(uintptr_t)p, p ? len : 0, pitch, rows};
}
Rows block_of(const void* p, uint64_t bytes) { return rows_of(p, bytes, bytes, 1); }

// Whether two sets of rows share a byte. Sets whose ranges cross are told apart only when
// they interleave at one pitch (columns of one matrix); otherwise they count as sharing.
bool meets(const Rows& a, const Rows& b) {
  if (!a.len || !b.len || a.rows <= 0 || b.rows <= 0) return false;
  const uint64_t alen = (uint64_t)(a.rows - 1) * a.pitch + a.len, blen = (uint64_t)(b.rows - 1) * b.pitch + b.len;
  if (!(a.at < b.at + blen && b.at < a.at + alen)) return false;
  if (a.pitch == b.pitch && a.rows > 1 && b.rows > 1) {
    const uint64_t d = b.at >= a.at ? (b.at - a.at) % a.pitch : (a.pitch - (a.at - b.at) % a.pitch) % a.pitch;
    return d < a.len || d + b.len > a.pitch;
  }
  return true;
}
bool same(const Rows& a, const Rows& b) {
  return a.at == b.at && a.len == b.len && (a.pitch == b.pitch || a.rows <= 1);
}

// A pitch holds a row and keeps its vectors aligned, and the rows end below 2^63.
int check_pitch(uint64_t pitch, uint64_t len, int64_t rows) {
  if (pitch % 16) return PLR_EALIGN;
  if (pitch > kMaxPitch) return PLR_EUNSUPPORTED;
  if (rows > 1 && pitch < len) return PLR_EINVAL;
  if (rows > 0 && pitch > (uint64_t)INT64_MAX / (uint64_t)rows) return PLR_EINVAL;
  return PLR_OK;
}

#define PLR_TRY(expr)          \
  do {                         \
    const int rc_ = (expr);    \
    if (rc_) return rc_;       \
  } while (0)

int status(hipError_t e) { return e == hipSuccess ? PLR_OK : record_hip_error(e); }

// cols: whole 16-byte vectors in the type, and few enough for one workgroup's registers.
int check_norm(int dtype, int64_t rows, int64_t cols) {
  if (!is_float(dtype)) return PLR_EINVAL;
  if (rows < 0 || cols < 1) return PLR_EINVAL;
  if (rows > kMaxRows) return PLR_EUNSUPPORTED;
  if (cols > kMaxCols) return PLR_EUNSUPPORTED;
  if (cols * elem(dtype) % 16) return PLR_EALIGN;
  if (cols * elem(dtype) / 16 > (uint64_t)kNormMaxThreads * kNormMaxVecs) return PLR_EUNSUPPORTED;
  return PLR_OK;
}

}  // namespace

extern "C" int plr_rmsnorm(int dtype, int out_dtype, int world, int64_t rows, int64_t cols, const void* const* srcs,
                           size_t src_pitch, const void* residual, size_t residual_pitch, const void* gamma,
                           float eps, void* sum_out, size_t sum_pitch, void* out, size_t out_pitch, float* out_scale,
                           float* rstd, void* stream) {
  PLR_TRY(check_norm(dtype, rows, cols));
  if (out_dtype != dtype && out_dtype != PLR_F8) return PLR_EINVAL;
  if (world < 1) return PLR_EINVAL;
  if (world > PLR_MAX_WORLD) return PLR_EUNSUPPORTED;
  if (!(eps >= 0)) return PLR_EINVAL;
  const bool f8 = out_dtype == PLR_F8;
  if (!srcs || !gamma) return PLR_EINVAL;
  if (f8 && cols % 16) return PLR_EALIGN;
  if (rows == 0) return PLR_OK;  // without rows no output has an entry: their addresses may be NULL
  if (!out || (f8 && !out_scale)) return PLR_EINVAL;
  const uint64_t len = cols * elem(dtype), out_len = cols * elem(out_dtype);
  if (!a16(gamma) || !a16(residual) || !a16(sum_out) || !a16(out) || !a4(out_scale) || !a4(rstd)) return PLR_EALIGN;
  PLR_TRY(check_pitch(src_pitch, len, rows));
  if (residual) PLR_TRY(check_pitch(residual_pitch, len, rows));
  if (sum_out) PLR_TRY(check_pitch(sum_pitch, len, rows));
  PLR_TRY(check_pitch(out_pitch, out_len, rows));
  NormArgs a{};
  const Rows o = rows_of(out, out_len, out_pitch, rows), sum = rows_of(sum_out, len, sum_pitch, rows);
  const Rows scale = block_of(f8 ? out_scale : nullptr, rows * 4), rs = block_of(rstd, rows * 4);
  const Rows outs[4] = {o, sum, scale, rs};
  for (int i = 0; i < 4; ++i) {
    if (meets(outs[i], block_of(gamma, len))) return PLR_EINVAL;
    for (int j = i + 1; j < 4; ++j)
      if (meets(outs[i], outs[j])) return PLR_EINVAL;
  }
  for (int w = 0; w <= world; ++w) {  // an output may be an input's own rows: a thread reads before it writes
    const void* p = w < world ? srcs[w] : residual;
    if (w < world && !p) return PLR_EINVAL;
    if (!a16(p)) return PLR_EALIGN;
    const Rows in = rows_of(p, len, w < world ? src_pitch : residual_pitch, rows);
    for (int i = 0; i < 4; ++i)
      if (meets(outs[i], in) && !(i < 2 && same(outs[i], in))) return PLR_EINVAL;
    if (w < world) a.src[w] = static_cast<const char*>(p);
  }
  a.src_pitch = src_pitch;
  a.residual = static_cast<const char*>(residual);
  a.residual_pitch = residual_pitch;
  a.gamma = static_cast<const char*>(gamma);
  a.sum_out = static_cast<char*>(sum_out);
  a.sum_pitch = sum_pitch;
  a.out = static_cast<char*>(out);
  a.out_pitch = out_pitch;
  a.out_scale = out_scale;
  a.rstd = rstd;
  a.rows = rows;
  a.nvec = (uint32_t)(len / 16);
  a.world = (uint32_t)world;
  a.inv_cols = 1.0f / (float)cols;
  a.eps = eps;
  return status(launch_norm(a, dtype, out_dtype, static_cast<hipStream_t>(stream)));
}

extern "C" size_t plr_rmsnorm_backward_workspace_bytes(int dtype, int64_t rows, int64_t cols) {
  if (check_norm(dtype, rows, cols) != PLR_OK) return 0;
  return (size_t)(norm_back_blocks(rows) * cols * 4);
}

extern "C" int plr_rmsnorm_backward(int dtype, int64_t rows, int64_t cols, const void* dout, size_t dout_pitch,
                                    const void* h, size_t h_pitch, const void* gamma, const float* rstd,
                                    const void* dsum, size_t dsum_pitch, void* dx, size_t dx_pitch, float* dgamma,
                                    void* workspace, void* stream) {
  PLR_TRY(check_norm(dtype, rows, cols));
  if (!gamma || !dgamma || !workspace) return PLR_EINVAL;
  if (!a16(gamma) || !a16(dgamma) || !a16(workspace)) return PLR_EALIGN;
  if (rows > 0 && (!dout || !h || !rstd || !dx)) return PLR_EINVAL;
  if (!a16(dout) || !a16(h) || !a16(dsum) || !a16(dx) || !a4(rstd)) return PLR_EALIGN;
  const uint64_t len = cols * elem(dtype);
  PLR_TRY(check_pitch(dout_pitch, len, rows));
  PLR_TRY(check_pitch(h_pitch, len, rows));
  if (dsum) PLR_TRY(check_pitch(dsum_pitch, len, rows));
  PLR_TRY(check_pitch(dx_pitch, len, rows));
  const int64_t blocks = norm_back_blocks(rows);
  const Rows o = rows_of(dx, len, dx_pitch, rows), g = block_of(dgamma, cols * 4);
  const Rows ws = block_of(workspace, blocks * cols * 4);
  const Rows ins[3] = {rows_of(dout, len, dout_pitch, rows), rows_of(h, len, h_pitch, rows),
                       rows_of(dsum, len, dsum_pitch, rows)};
  for (const Rows& in : ins) {
    if (meets(o, in) && !same(o, in)) return PLR_EINVAL;
    if (meets(g, in) || meets(ws, in)) return PLR_EINVAL;
  }
  const Rows fixed[2] = {block_of(gamma, len), block_of(rstd, rows * 4)};
  for (const Rows& in : fixed)
    if (meets(o, in) || meets(g, in) || meets(ws, in)) return PLR_EINVAL;
  if (meets(o, g) || meets(o, ws) || meets(g, ws)) return PLR_EINVAL;
  NormBackArgs a{};
  a.dout = static_cast<const char*>(dout);
  a.h = static_cast<const char*>(h);
  a.gamma = static_cast<const char*>(gamma);
  a.rstd = rstd;
  a.dsum = static_cast<const char*>(dsum);
  a.dx = static_cast<char*>(dx);
  a.partial = blocks == 1 ? dgamma : static_cast<float*>(workspace);
  a.dout_pitch = dout_pitch;
  a.h_pitch = h_pitch;
  a.dsum_pitch = dsum_pitch;
  a.dx_pitch = dx_pitch;
  a.rows = rows;
  a.nvec = (uint32_t)(len / 16);
  a.inv_cols = 1.0f / (float)cols;
  return status(launch_norm_back(a, dtype, blocks, dgamma, static_cast<hipStream_t>(stream)));
}

static int check_route(int dtype, int64_t tokens, int experts, int k) {
  if (!is_float(dtype)) return PLR_EINVAL;
  if (tokens < 0 || experts < 1 || k < 1) return PLR_EINVAL;
  if (tokens > kMaxTokens || experts > kRouteMaxExperts || k > kRouteMaxK) return PLR_EUNSUPPORTED;
  return PLR_OK;
}

static int64_t route_blocks(int64_t tokens) { return std::max<int64_t>(1, (tokens + kRouteTokens - 1) / kRouteTokens); }

extern "C" size_t plr_route_workspace_bytes(int64_t tokens, int experts) {
  if (check_route(PLR_F32, tokens, experts, 1) != PLR_OK) return 0;
  return (size_t)((route_blocks(tokens) + 1) * experts * 4 + 15) / 16 * 16;
}

extern "C" int plr_route(int dtype, int64_t tokens, int experts, int k, const void* logits, size_t logits_pitch,
                         int32_t* ids, float* weights, int32_t* positions, int32_t* row_token, int64_t* offsets,
                         void* workspace, void* stream) {
  PLR_TRY(check_route(dtype, tokens, experts, k));
  const uint64_t e = elem(dtype), len = experts * e;
  if (!offsets || !workspace) return PLR_EINVAL;
  if (tokens > 0 && (!logits || !ids || !weights || !positions || !row_token)) return PLR_EINVAL;
  if (((uintptr_t)logits % e) || logits_pitch % e || !a4(ids) || !a4(weights) || !a4(positions) || !a4(row_token) ||
      !a8(offsets) || !a16(workspace))
    return PLR_EALIGN;
  if (tokens > 1 && logits_pitch < len) return PLR_EINVAL;
  if (tokens > 0 && logits_pitch > (uint64_t)INT64_MAX / (uint64_t)tokens) return PLR_EINVAL;
  const uint64_t pairs = (uint64_t)tokens * k * 4;
  const Rows outs[6] = {block_of(ids, pairs), block_of(weights, pairs), block_of(positions, pairs),
                        block_of(row_token, pairs), block_of(offsets, 8ull * (experts + 1)),
                        block_of(workspace, plr_route_workspace_bytes(tokens, experts))};
  const Rows in = rows_of(logits, len, logits_pitch, tokens);
  for (int i = 0; i < 6; ++i) {
    if (meets(outs[i], in)) return PLR_EINVAL;
    for (int j = i + 1; j < 6; ++j)
      if (meets(outs[i], outs[j])) return PLR_EINVAL;
  }
  RouteArgs a{};
  a.logits = static_cast<const char*>(logits);
  a.pitch = logits_pitch;
  a.ids = ids;
  a.weights = weights;
  a.positions = positions;
  a.row_token = row_token;
  a.offsets = offsets;
  a.totals = static_cast<int32_t*>(workspace);
  a.counts = a.totals + experts;
  a.tokens = tokens;
  a.blocks = (uint32_t)route_blocks(tokens);
  a.experts = (uint32_t)experts;
  a.k = (uint32_t)k;
  return status(launch_route(a, dtype, static_cast<hipStream_t>(stream)));
}

extern "C" int plr_route_backward(int dtype, int64_t tokens, int experts, int k, const int32_t* ids,
                                  const float* weights, const float* dweights, void* dlogits, size_t dlogits_pitch,
                                  void* stream) {
  PLR_TRY(check_route(dtype, tokens, experts, k));
  if (tokens == 0) return PLR_OK;
  if (!ids || !weights || !dweights || !dlogits) return PLR_EINVAL;
  const uint64_t e = elem(dtype), len = experts * e;
  if (!a4(ids) || !a4(weights) || !a4(dweights) || !a16(dlogits) || dlogits_pitch % e) return PLR_EALIGN;
  if (tokens > 1 && dlogits_pitch < len) return PLR_EINVAL;
  if (dlogits_pitch > (uint64_t)INT64_MAX / (uint64_t)tokens) return PLR_EINVAL;
  const Rows o = rows_of(dlogits, len, dlogits_pitch, tokens);
  const uint64_t pairs = (uint64_t)tokens * k * 4;
  if (meets(o, block_of(ids, pairs)) || meets(o, block_of(weights, pairs)) || meets(o, block_of(dweights, pairs)))
    return PLR_EINVAL;
  RouteBackArgs a{};
  a.ids = ids;
  a.weights = weights;
  a.dweights = dweights;
  a.dlogits = static_cast<char*>(dlogits);
  a.pitch = dlogits_pitch;
  a.tokens = tokens;
  a.experts = (uint32_t)experts;
  a.k = (uint32_t)k;
  return status(launch_route_back(a, dtype, static_cast<hipStream_t>(stream)));
}

// Common checks of the three grouped products.
static int check_group(int dtype, int out_dtype, bool f8_allowed, int groups, int64_t rows, int64_t n, int64_t k,
                       const int64_t* offsets) {
  if (dtype == PLR_F32) return PLR_EUNSUPPORTED;
  if (dtype != PLR_BF16 && dtype != PLR_F16 && dtype != PLR_F8) return PLR_EINVAL;
  if (dtype == PLR_F8 && !f8_allowed) return PLR_EUNSUPPORTED;
  if (!is_float(out_dtype)) return PLR_EINVAL;
  if (dtype != PLR_F8 && out_dtype != dtype && out_dtype != PLR_F32) return PLR_EINVAL;
  if (groups < 1 || rows < 0 || n < 1 || k < 1 || !offsets) return PLR_EINVAL;
  if (groups > PLR_GROUP_MAX || rows > kMaxRows || n > PLR_GROUP_MAX_COLS || k > PLR_GROUP_MAX_COLS)
    return PLR_EUNSUPPORTED;
  if (n % 8 || k % (16 / elem(dtype)) || !a8(offsets)) return PLR_EALIGN;
  return PLR_OK;
}

// Output tiles of 256 x 256: `rows` of the ragged axis (each group may end in part of a
// tile), or of every group (dw).
static bool tiles_fit(int64_t row_tiles, int64_t cols) { return row_tiles * ((cols + 255) / 256) <= kGroupMaxTiles; }
static int64_t ragged_tiles(int64_t rows, int groups) { return rows / 256 + std::min<int64_t>(rows, groups); }

extern "C" int plr_group_matmul(int dtype, int out_dtype, int groups, int64_t rows, int64_t n, int64_t k,
                                const void* x, size_t x_pitch, int64_t x_rows, const int32_t* row_of, const void* w,
                                const int64_t* offsets, const float* x_scale, const float* w_scale, void* y,
                                size_t y_pitch, void* stream) {
  PLR_TRY(check_group(dtype, out_dtype, true, groups, rows, n, k, offsets));
  const bool f8 = dtype == PLR_F8;
  if (f8 ? !w_scale || (!x_scale && x_rows > 0) : x_scale || w_scale) return PLR_EINVAL;
  if (x_rows < 0 || (!row_of && x_rows < rows)) return PLR_EINVAL;
  if (x_rows > kMaxRows) return PLR_EUNSUPPORTED;
  if (rows == 0) return PLR_OK;
  if (!w || !y || (x_rows > 0 && !x)) return PLR_EINVAL;
  if (!a16(x) || !a16(w) || !a16(y) || !a4(row_of) || !a4(x_scale) || !a4(w_scale)) return PLR_EALIGN;
  if (!tiles_fit(ragged_tiles(rows, groups), n)) return PLR_EUNSUPPORTED;
  const uint64_t e = elem(dtype), out_len = n * elem(out_dtype);
  PLR_TRY(check_pitch(x_pitch, k * e, x_rows));
  PLR_TRY(check_pitch(y_pitch, out_len, rows));
  const Rows o = rows_of(y, out_len, y_pitch, rows);
  if (meets(o, rows_of(x, k * e, x_pitch, x_rows)) || meets(o, block_of(w, (uint64_t)groups * n * k * e)) ||
      meets(o, block_of(row_of, rows * 4)) || meets(o, block_of(offsets, 8ull * (groups + 1))) ||
      meets(o, block_of(x_scale, x_rows * 4)) || meets(o, block_of(w_scale, (uint64_t)groups * n * 4)))
    return PLR_EINVAL;
  GroupArgs a{};
  a.a = static_cast<const char*>(x);
  a.b = static_cast<const char*>(w);
  a.out = static_cast<char*>(y);
  a.row_of = row_of;
  a.offsets = offsets;
  a.a_scale = x_scale;
  a.b_scale = w_scale;
  a.a_pitch = x_pitch;
  a.b_pitch = k * e;
  a.out_pitch = y_pitch;
  a.rows = rows;
  a.src_rows = x_rows;
  a.n = n;
  a.k = k;
  a.groups = groups;
  a.out_dtype = out_dtype;
  return status(launch_group(a, kGroupY, dtype, static_cast<hipStream_t>(stream)));
}

extern "C" int plr_group_matmul_dx(int dtype, int out_dtype, int groups, int64_t rows, int64_t n, int64_t k,
                                   const void* dy, size_t dy_pitch, const void* w, const int64_t* offsets, void* dx,
                                   size_t dx_pitch, void* stream) {
  PLR_TRY(check_group(dtype, out_dtype, false, groups, rows, n, k, offsets));
  if (rows == 0) return PLR_OK;
  if (!dy || !w || !dx) return PLR_EINVAL;
  if (!a16(dy) || !a16(w) || !a16(dx)) return PLR_EALIGN;
  if (!tiles_fit(ragged_tiles(rows, groups), k)) return PLR_EUNSUPPORTED;
  const uint64_t e = elem(dtype), out_len = k * elem(out_dtype);
  PLR_TRY(check_pitch(dy_pitch, n * e, rows));
  PLR_TRY(check_pitch(dx_pitch, out_len, rows));
  const Rows o = rows_of(dx, out_len, dx_pitch, rows);
  if (meets(o, rows_of(dy, n * e, dy_pitch, rows)) || meets(o, block_of(w, (uint64_t)groups * n * k * e)) ||
      meets(o, block_of(offsets, 8ull * (groups + 1))))
    return PLR_EINVAL;
  GroupArgs a{};
  a.a = static_cast<const char*>(dy);
  a.b = static_cast<const char*>(w);
  a.out = static_cast<char*>(dx);
  a.offsets = offsets;
  a.a_pitch = dy_pitch;
  a.b_pitch = k * e;
  a.out_pitch = dx_pitch;
  a.rows = a.src_rows = rows;
  a.n = n;
  a.k = k;
  a.groups = groups;
  a.out_dtype = out_dtype;
  return status(launch_group(a, kGroupDx, dtype, static_cast<hipStream_t>(stream)));
}

extern "C" int plr_group_matmul_dw(int dtype, int out_dtype, int groups, int64_t rows, int64_t n, int64_t k,
                                   const void* dy, size_t dy_pitch, const void* x, size_t x_pitch, int64_t x_rows,
                                   const int32_t* row_of, const int64_t* offsets, void* dw, void* stream) {
  PLR_TRY(check_group(dtype, out_dtype, false, groups, rows, n, k, offsets));
  if (x_rows < 0 || (!row_of && x_rows < rows)) return PLR_EINVAL;
  if (x_rows > kMaxRows) return PLR_EUNSUPPORTED;
  if (!dw || (rows > 0 && !dy) || (rows > 0 && x_rows > 0 && !x)) return PLR_EINVAL;
  if (!a16(dy) || !a16(x) || !a16(dw) || !a4(row_of)) return PLR_EALIGN;
  if (!tiles_fit(groups * ((n + 255) / 256), k)) return PLR_EUNSUPPORTED;
  const uint64_t e = elem(dtype), out_len = k * elem(out_dtype);
  PLR_TRY(check_pitch(dy_pitch, n * e, rows));
  PLR_TRY(check_pitch(x_pitch, k * e, x_rows));
  const Rows o = block_of(dw, (uint64_t)groups * n * out_len);
  if (meets(o, rows_of(dy, n * e, dy_pitch, rows)) || meets(o, rows_of(x, k * e, x_pitch, x_rows)) ||
      meets(o, block_of(row_of, rows * 4)) || meets(o, block_of(offsets, 8ull * (groups + 1))))
    return PLR_EINVAL;
  GroupArgs a{};
  a.a = static_cast<const char*>(dy);
  a.b = static_cast<const char*>(x);
  a.out = static_cast<char*>(dw);
  a.row_of = row_of;
  a.offsets = offsets;
  a.a_pitch = dy_pitch;
  a.b_pitch = x_pitch;
  a.out_pitch = out_len;
  a.rows = rows;
  a.src_rows = x_rows;
  a.n = n;
  a.k = k;
  a.groups = groups;
  a.out_dtype = out_dtype;
  return status(launch_group(a, kGroupDw, dtype, static_cast<hipStream_t>(stream)));
}

static int check_combine(int dtype, int64_t tokens, int k, int64_t cols, int64_t y_rows) {
  if (!is_float(dtype)) return PLR_EINVAL;
  if (tokens < 0 || k < 1 || cols < 1 || y_rows < 0) return PLR_EINVAL;
  if (tokens > kMaxTokens || k > kCombineMaxK || cols > kMaxCols || y_rows > kMaxRows) return PLR_EUNSUPPORTED;
  if (cols * elem(dtype) % 16) return PLR_EALIGN;
  return PLR_OK;
}

extern "C" int plr_combine(int dtype, int64_t tokens, int k, int64_t cols, const void* y, size_t y_pitch,
                           int64_t y_rows, const int32_t* positions, const float* weights, void* out,
                           size_t out_pitch, void* stream) {
  PLR_TRY(check_combine(dtype, tokens, k, cols, y_rows));
  if (tokens == 0) return PLR_OK;
  if (!positions || !out || (y_rows > 0 && !y)) return PLR_EINVAL;
  if (!a16(y) || !a16(out) || !a4(positions) || !a4(weights)) return PLR_EALIGN;
  const uint64_t len = cols * elem(dtype), pairs = (uint64_t)tokens * k * 4;
  PLR_TRY(check_pitch(y_pitch, len, y_rows));
  PLR_TRY(check_pitch(out_pitch, len, tokens));
  const Rows o = rows_of(out, len, out_pitch, tokens);
  if (meets(o, rows_of(y, len, y_pitch, y_rows)) || meets(o, block_of(positions, pairs)) ||
      meets(o, block_of(weights, pairs)))
    return PLR_EINVAL;
  CombineArgs a{};
  a.y = static_cast<const char*>(y);
  a.positions = positions;
  a.weights = weights;
  a.out = static_cast<char*>(out);
  a.y_pitch = y_pitch;
  a.out_pitch = out_pitch;
  a.tokens = tokens;
  a.rows = y_rows;
  a.k = (uint32_t)k;
  a.nvec = (uint32_t)(len / 16);
  return status(launch_combine(a, dtype, static_cast<hipStream_t>(stream)));
}

extern "C" int plr_combine_backward(int dtype, int64_t tokens, int k, int64_t cols, const void* dout,
                                    size_t dout_pitch, const void* y, size_t y_pitch, int64_t y_rows,
                                    const int32_t* positions, const float* weights, void* dy, size_t dy_pitch,
                                    float* dweights, void* stream) {
  PLR_TRY(check_combine(dtype, tokens, k, cols, y_rows));
  if (tokens == 0) return PLR_OK;
  if (!dout || !positions || (y_rows > 0 && !dy) || (y_rows > 0 && dweights && !y)) return PLR_EINVAL;
  if (!a16(dout) || !a16(y) || !a16(dy) || !a4(positions) || !a4(weights) || !a4(dweights)) return PLR_EALIGN;
  const uint64_t len = cols * elem(dtype), pairs = (uint64_t)tokens * k * 4;
  PLR_TRY(check_pitch(dout_pitch, len, tokens));
  if (dweights) PLR_TRY(check_pitch(y_pitch, len, y_rows));
  PLR_TRY(check_pitch(dy_pitch, len, y_rows));
  const Rows o = rows_of(dy, len, dy_pitch, y_rows), dw = block_of(dweights, pairs);
  const Rows ins[4] = {rows_of(dout, len, dout_pitch, tokens), block_of(positions, pairs), block_of(weights, pairs),
                       rows_of(dweights ? y : nullptr, len, y_pitch, y_rows)};
  for (int i = 0; i < 4; ++i) {
    // dy may take y's own rows: a thread reads each vector of y before it writes there
    if (meets(o, ins[i]) && !(i == 3 && same(o, ins[i]))) return PLR_EINVAL;
    if (meets(dw, ins[i])) return PLR_EINVAL;
  }
  if (meets(o, dw)) return PLR_EINVAL;
  CombineBackArgs a{};
  a.dout = static_cast<const char*>(dout);
  a.y = static_cast<const char*>(y);
  a.positions = positions;
  a.weights = weights;
  a.dy = static_cast<char*>(dy);
  a.dweights = dweights;
  a.dout_pitch = dout_pitch;
  a.y_pitch = y_pitch;
  a.dy_pitch = dy_pitch;
  a.tokens = tokens;
  a.rows = y_rows;
  a.k = (uint32_t)k;
  a.nvec = (uint32_t)(len / 16);
  return status(launch_combine_back(a, dtype, static_cast<hipStream_t>(stream)));
}
