// C ABI of the activation checkpoints and of the operators that read them
// (declared in include/scape.h): argument validation and workspace sizes.
#include "activations.h"

#include <cmath>

using namespace scape;

namespace {

bool rows_ok(int64_t rows) { return rows >= 0 && rows < (int64_t(1) << 31); }
bool cols_ok(int64_t cols) { return cols >= 1 && cols <= kMaxCols; }

scape_status check_size(int64_t rows, int64_t cols) {
  if (!rows_ok(rows) || !cols_ok(cols))
    return fail(SCAPE_ESHAPE, "invalid shape: rows=%lld cols=%lld (need 0<=rows<2^31, 1<=cols<=2^20)",
                (long long)rows, (long long)cols);
  return SCAPE_OK;
}

// `need`: the matrix has to be there (a matrix of no rows need not).
scape_status check_matrix(const char* name, const scape_matrix& m, int64_t rows, int64_t cols, bool need) {
  if (!m.data) return need && rows > 0 ? fail(SCAPE_EINVAL, "%s is null", name) : SCAPE_OK;
  if (m.dtype != SCAPE_F32 && m.dtype != SCAPE_BF16 && m.dtype != SCAPE_F16)
    return fail(SCAPE_EINVAL, "%s: unknown dtype %d", name, m.dtype);
  if ((uintptr_t)m.data % dtype_bytes(m.dtype)) return fail(SCAPE_EINVAL, "%s is not aligned to its type", name);
  if (m.ld < cols || m.ld > (int64_t(1) << 46) / (rows > 0 ? rows : 1))
    return fail(SCAPE_ESHAPE, "%s: ld %lld must be at least cols %lld (and rows * ld at most 2^46)", name,
                (long long)m.ld, (long long)cols);
  return SCAPE_OK;
}

scape_status check_act(const char* name, const scape_act_view& a, int64_t rows, bool need) {
  if (!a.codes && !a.scales && !(need && rows > 0)) return SCAPE_OK;
  if (!a.codes || !a.scales) return fail(SCAPE_EINVAL, "%s is null", name);
  if ((uintptr_t)a.codes & 15u) return fail(SCAPE_EINVAL, "%s: codes must be 16-byte aligned", name);
  return SCAPE_OK;
}

bool misaligned4(const void* p) { return ((uintptr_t)p & 3u) != 0; }

scape_status check_workspace(const void* ws, size_t have, size_t need) {
  if (!ws) return fail(SCAPE_EINVAL, "workspace is null");
  if ((uintptr_t)ws & 255u) return fail(SCAPE_EINVAL, "workspace must be 256-byte aligned");
  if (have < need) return fail(SCAPE_EWORKSPACE, "workspace has %zu bytes, needs %zu", have, need);
  return SCAPE_OK;
}

// An output may be an input's own matrix, element on element, or lie apart.
bool shifted_alias(const scape_matrix& o, const scape_matrix& i, int64_t rows) {
  return o.data && o.data == i.data && rows > 1 && o.ld != i.ld;
}

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

}  // namespace

extern "C" {

int32_t scape_act_block(void) { return kActBlock; }

size_t scape_act_bytes(int64_t rows, int64_t cols) {
  if (!rows_ok(rows) || !cols_ok(cols)) return 0;
  const size_t codes = align256((size_t)rows * (size_t)act_pitch(cols));
  return codes + align256((size_t)rows * (size_t)act_blocks(cols)) + (rows ? 0 : 256);
}

scape_status scape_act_slot(int64_t rows, int64_t cols, void* buffer, scape_act_view* out) {
  scape_status st = check_size(rows, cols);
  if (st) return st;
  if (!buffer || !out) return fail(SCAPE_EINVAL, "buffer or out is null");
  char* base = static_cast<char*>(buffer);
  out->codes = reinterpret_cast<int8_t*>(base);
  out->scales = reinterpret_cast<uint8_t*>(base + align256((size_t)rows * (size_t)act_pitch(cols)));
  return SCAPE_OK;
}

scape_status scape_act_pack(int64_t rows, int64_t cols, scape_matrix x, scape_act_view out, hipStream_t stream) {
  scape_status st = check_size(rows, cols);
  if (st) return st;
  if ((st = check_matrix("x", x, rows, cols, true))) return st;
  if ((st = check_act("out", out, rows, true))) return st;
  return hip_check(launch_act_pack(rows, cols, x, out, stream), "act pack");
}

scape_status scape_act_unpack(int64_t rows, int64_t cols, scape_act_view a, const float* gain, scape_matrix out,
                              hipStream_t stream) {
  scape_status st = check_size(rows, cols);
  if (st) return st;
  if ((st = check_act("a", a, rows, true))) return st;
  if ((st = check_matrix("out", out, rows, cols, true))) return st;
  if (misaligned4(gain)) return fail(SCAPE_EINVAL, "gain must be 4-byte aligned");
  return hip_check(launch_act_unpack(rows, cols, a, gain, out, stream), "act unpack");
}

scape_status scape_rmsnorm_pack(int64_t rows, int64_t cols, scape_matrix x, scape_matrix residual,
                                const float* weight, float eps, scape_matrix h, scape_matrix y, scape_act_view xhat,
                                float* rstd, hipStream_t stream) {
  scape_status st = check_size(rows, cols);
  if (st) return st;
  if ((st = check_matrix("x", x, rows, cols, true))) return st;
  if ((st = check_matrix("residual", residual, rows, cols, false))) return st;
  if ((st = check_matrix("h", h, rows, cols, false))) return st;
  if ((st = check_matrix("y", y, rows, cols, false))) return st;
  if ((st = check_act("xhat", xhat, rows, false))) return st;
  if (rows > 0 && !y.data && !xhat.codes) return fail(SCAPE_EINVAL, "y and xhat are both null");
  if (y.data && !weight) return fail(SCAPE_EINVAL, "weight is null");
  if (misaligned4(weight) || misaligned4(rstd)) return fail(SCAPE_EINVAL, "weight and rstd must be 4-byte aligned");
  if (!(eps > 0.0f) || !std::isfinite(eps)) return fail(SCAPE_EINVAL, "eps must be positive and finite");
  const scape_matrix* same[3] = {&residual, &h, &y};
  for (const scape_matrix* m : same)
    if (m->data && m->dtype != x.dtype) return fail(SCAPE_EINVAL, "residual, h and y must have x's dtype");
  if (h.data && h.data == y.data) return fail(SCAPE_EINVAL, "h and y must be different matrices");
  if (shifted_alias(h, x, rows) || shifted_alias(h, residual, rows) || shifted_alias(y, x, rows) ||
      shifted_alias(y, residual, rows))
    return fail(SCAPE_EINVAL, "an output in an input's place must have its ld");
  return hip_check(launch_rmsnorm_pack(rows, cols, x, residual, weight, eps, h, y, xhat, rstd, stream),
                   "rmsnorm pack");
}

size_t scape_rmsnorm_workspace_bytes(int64_t rows, int64_t cols) {
  if (!rows_ok(rows) || !cols_ok(cols)) return 0;
  return align256((size_t)rmsnorm_parts(rows, cols) * (size_t)cols * 4);
}

scape_status scape_rmsnorm_backward(int64_t rows, int64_t cols, scape_matrix dy, scape_act_view xhat,
                                    const float* rstd, const float* weight, scape_matrix dres, scape_matrix dh,
                                    float* dweight, int32_t accumulate, void* workspace, size_t workspace_bytes,
                                    hipStream_t stream) {
  scape_status st = check_size(rows, cols);
  if (st) return st;
  if ((st = check_matrix("dy", dy, rows, cols, true))) return st;
  if ((st = check_act("xhat", xhat, rows, true))) return st;
  if ((st = check_matrix("dres", dres, rows, cols, false))) return st;
  if ((st = check_matrix("dh", dh, rows, cols, false))) return st;
  if (rows > 0 && !dh.data && !dweight) return fail(SCAPE_EINVAL, "dh and dweight are both null");
  if (rows > 0 && (!rstd || !weight)) return fail(SCAPE_EINVAL, "rstd or weight is null");
  if (misaligned4(weight) || misaligned4(rstd) || misaligned4(dweight))
    return fail(SCAPE_EINVAL, "rstd, weight and dweight must be 4-byte aligned");
  if ((dres.data && dres.dtype != dy.dtype) || (dh.data && dh.dtype != dy.dtype))
    return fail(SCAPE_EINVAL, "dres and dh must have dy's dtype");
  if (shifted_alias(dh, dy, rows) || shifted_alias(dh, dres, rows))
    return fail(SCAPE_EINVAL, "an output in an input's place must have its ld");
  if ((st = check_workspace(workspace, workspace_bytes, scape_rmsnorm_workspace_bytes(rows, cols)))) return st;
  return hip_check(launch_rmsnorm_backward(rows, cols, dy, xhat, rstd, weight, dres, dh, dweight, accumulate != 0,
                                           static_cast<float*>(workspace), stream),
                   "rmsnorm backward");
}

int32_t scape_wgrad_splits(int64_t rows, int64_t in, int64_t out, int32_t dtype, int32_t* tile_out,
                           int32_t* tile_in) {
  if (!rows_ok(rows) || !cols_ok(in) || !cols_ok(out) || in * out > kMaxWeight) return -1;
  if (dtype != SCAPE_F32 && dtype != SCAPE_BF16 && dtype != SCAPE_F16) return -1;
  int m, n;
  const int splits = wgrad_splits(rows, in, out, dtype, &m, &n);
  if (tile_out) *tile_out = m;
  if (tile_in) *tile_in = n;
  return splits;
}

size_t scape_wgrad_workspace_bytes(int64_t rows, int64_t in, int64_t out, scape_matrix dy) {
  if (!rows_ok(rows) || !cols_ok(in) || !cols_ok(out) || in * out > kMaxWeight) return 0;
  return wgrad_workspace(rows, in, out, dy);
}

scape_status scape_wgrad(int64_t rows, int64_t in, int64_t out, scape_matrix dy, scape_act_view x, const float* gain,
                         float* dw, float* dbias, int32_t accumulate, void* workspace, size_t workspace_bytes,
                         hipStream_t stream) {
  scape_status st = check_size(rows, in);
  if (st) return st;
  if ((st = check_size(rows, out))) return st;
  if (in * out > kMaxWeight)
    return fail(SCAPE_ESHAPE, "invalid shape: in=%lld out=%lld (need in*out<=2^37)", (long long)in, (long long)out);
  if ((st = check_matrix("dy", dy, rows, out, true))) return st;
  if ((st = check_act("x", x, rows, true))) return st;
  if (!dw) return fail(SCAPE_EINVAL, "dw is null");
  if (misaligned4(gain) || misaligned4(dw) || misaligned4(dbias))
    return fail(SCAPE_EINVAL, "gain, dw and dbias must be 4-byte aligned");
  if ((st = check_workspace(workspace, workspace_bytes, wgrad_workspace(rows, in, out, dy)))) return st;
  return hip_check(launch_wgrad(rows, in, out, dy, x, gain, dw, dbias, accumulate != 0, workspace, stream),
                   "wgrad");
}

}  // extern "C"
