// C-ABI host layer of the history layer (layer norm, dropout, attention of
// histories): argument validation and workspace sizes. No C++ exception
// crosses the ABI.
#include <hip/hip_runtime.h>

#include <cmath>

#include "emb.h"
#include "seq_internal.h"

using namespace emb;

namespace {

int check_rows_sizes(int64_t rows, int32_t dim, int64_t max_dim) {
  if (rows < 0 || rows >= (1ll << 31)) return fail(EMB_E_INVAL, "rows %lld not in [0, 2^31)", (long long)rows);
  if (dim < 1 || dim > max_dim) return fail(EMB_E_INVAL, "dim %d not in [1, %lld]", dim, (long long)max_dim);
  return EMB_OK;
}

int check_rows(const char* name, const Rows2D& r) {
  if (!r.p) return fail(EMB_E_INVAL, "%s is NULL", name);
  if (!aligned(r.p, (size_t)esize(r.dtype))) return fail(EMB_E_INVAL, "%s is not aligned to its elements", name);
  if (r.stride < 0) return fail(EMB_E_INVAL, "%s has a negative stride", name);
  return EMB_OK;
}

int check_rows_out(const char* name, const Rows2D& r, int64_t rows, int32_t dim) {
  if (int rc = check_rows(name, r)) return rc;
  if (rows > 1 && r.stride < dim) return fail(EMB_E_INVAL, "%s: rows of stride %lld overlap", name, r.stride);
  return EMB_OK;
}

// Overlap of two operands is only allowed as the very same one.
int check_same(const char* in_name, const Rows2D& in, const char* out_name, const Rows2D& out) {
  if (in.p == out.p && (in.stride != out.stride || in.dtype != out.dtype))
    return fail(EMB_E_INVAL, "%s is %s with another stride or type", out_name, in_name);
  return EMB_OK;
}

int check_types(int x_dtype, int y_dtype) {
  if (int rc = check_dtype(x_dtype)) return rc;
  if (int rc = check_dtype(y_dtype)) return rc;
  if (x_dtype != y_dtype && x_dtype != EMB_F32)
    return fail(EMB_E_DTYPE, "y_dtype %d with x_dtype %d: the same, or 16-bit rows of fp32 ones", y_dtype, x_dtype);
  return EMB_OK;
}

}  // namespace

extern "C" {

int emb_layer_norm(int64_t rows, int32_t dim, const void* x, int32_t x_dtype, int64_t x_stride, void* y,
                   int32_t y_dtype, int64_t y_stride, const float* w, const float* b, float eps, void* hip_stream) {
  int rc = check_rows_sizes(rows, dim, EMB_MAX_ROW_DIM);
  if (rc) return rc;
  if ((rc = check_types(x_dtype, y_dtype)) || (rc = check_norm("w", w, eps)) || (rc = check_norm("b", b, eps))) return rc;
  if (rows == 0) return ok();
  const LayerNormArgs a{rows, dim, {x, x_stride, x_dtype}, {y, y_stride, y_dtype}, w, b, eps};
  if ((rc = check_rows("x", a.x)) || (rc = check_rows_out("y", a.y, rows, dim)) || (rc = check_same("x", a.x, "y", a.y)))
    return rc;
  hipError_t e = launch_layer_norm(a, static_cast<hipStream_t>(hip_stream));
  if (e != hipSuccess) return hip_fail(e, "layer norm");
  return ok();
}

size_t emb_layer_norm_workspace_bytes(int64_t rows, int32_t dim) {
  if (check_rows_sizes(rows, dim, EMB_MAX_ROW_DIM)) return 0;
  return (size_t)layer_norm_back_blocks(rows) * 2 * dim * sizeof(float);
}

int emb_layer_norm_backward(int64_t rows, int32_t dim, const void* x, int32_t x_dtype, int64_t x_stride,
                            const void* dy, int32_t y_dtype, int64_t dy_stride, void* dx, int64_t dx_stride,
                            const float* w, float eps, void* ws, size_t ws_bytes, float* dw, float* db,
                            void* hip_stream) {
  int rc = check_rows_sizes(rows, dim, EMB_MAX_ROW_DIM);
  if (rc) return rc;
  if ((rc = check_types(x_dtype, y_dtype)) || (rc = check_norm("w", w, eps))) return rc;
  if (!aligned(dw, 4) || !aligned(db, 4)) return fail(EMB_E_INVAL, "dw/db are misaligned");
  const LayerNormBackArgs a{rows, dim, {x, x_stride, x_dtype}, {dy, dy_stride, y_dtype}, {dx, dx_stride, x_dtype},
                            w, eps, static_cast<float*>(ws), dw, db};
  if (rows > 0) {
    if ((rc = check_rows("x", a.x)) || (rc = check_rows("dy", a.dy)) || (rc = check_rows_out("dx", a.dx, rows, dim)) ||
        (rc = check_same("x", a.x, "dx", a.dx)) || (rc = check_same("dy", a.dy, "dx", a.dx)))
      return rc;
    const size_t need = emb_layer_norm_workspace_bytes(rows, dim);
    if (!ws) return fail(EMB_E_INVAL, "ws is NULL");
    if (!aligned(ws, 16)) return fail(EMB_E_INVAL, "ws is not 16-byte aligned");
    if (ws_bytes < need) return fail(EMB_E_WORKSPACE, "workspace of %zu bytes, need %zu", ws_bytes, need);
  }
  hipError_t e = launch_layer_norm_back(a, static_cast<hipStream_t>(hip_stream));
  if (e != hipSuccess) return hip_fail(e, "gradient of layer norm");
  return ok();
}

int emb_dropout(int64_t rows, int32_t dim, int32_t dtype, const void* x, int64_t x_stride, const void* residual,
                int64_t residual_stride, void* y, int64_t y_stride, double p, uint64_t seed, const int64_t* step,
                void* hip_stream) {
  int rc = check_rows_sizes(rows, dim, (1ll << 31) - 1);
  if (rc) return rc;
  if ((rc = check_dtype(dtype))) return rc;
  if (!(p >= 0.0 && p <= 1.0)) return fail(EMB_E_INVAL, "p is not in [0, 1]");
  if (!aligned(step, 8)) return fail(EMB_E_INVAL, "step is misaligned");
  if (rows == 0) return ok();
  const uint64_t t = (uint64_t)std::floor(p * 0x1p32 + 0.5);
  const float scale = t >> 32 ? 0.f : (float)(1.0 / (1.0 - (double)t * 0x1p-32));
  const DropoutArgs a{rows, dim, {x, x_stride, dtype}, {residual, residual_stride, dtype}, {y, y_stride, dtype},
                      t, scale, seed, reinterpret_cast<const long long*>(step)};
  if ((rc = check_rows("x", a.x)) || (rc = check_rows_out("y", a.y, rows, dim)) || (rc = check_same("x", a.x, "y", a.y)))
    return rc;
  if (residual && ((rc = check_rows("residual", a.res)) || (rc = check_same("residual", a.res, "y", a.y)))) return rc;
  hipError_t e = launch_dropout(a, static_cast<hipStream_t>(hip_stream));
  if (e != hipSuccess) return hip_fail(e, "dropout");
  return ok();
}

}  // extern "C"
