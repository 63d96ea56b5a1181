// Argument checks shared by the operators' C entry points.
#pragma once

#include "activations.h"

namespace scape {

inline bool rows_ok(int64_t rows) { return rows >= 0 && rows < (int64_t(1) << 31); }
inline bool cols_ok(int64_t cols) { return cols >= 1 && cols <= kMaxCols; }

inline scape_status check_size(int64_t rows, int64_t cols) {
  if (!rows_ok(rows) || !cols_ok(cols))
    return fail(SCAPE_ESHAPE, "invalid shape: rows=%lld cols=%lld (need 0<=rows<2^31, 1<=cols<=2^20)",
                (long long)rows, (long long)cols);
  return SCAPE_OK;
}

// `need`: the matrix has to be there (a matrix of no rows need not).
inline scape_status check_matrix(const char* name, const scape_matrix& m, int64_t rows, int64_t cols, bool need) {
  if (!m.data) return need && rows > 0 ? fail(SCAPE_EINVAL, "%s is null", name) : SCAPE_OK;
  if (m.dtype != SCAPE_F32 && m.dtype != SCAPE_BF16 && m.dtype != SCAPE_F16)
    return fail(SCAPE_EINVAL, "%s: unknown dtype %d", name, m.dtype);
  if ((uintptr_t)m.data % dtype_bytes(m.dtype)) return fail(SCAPE_EINVAL, "%s is not aligned to its type", name);
  if (m.ld < cols || m.ld > (int64_t(1) << 46) / (rows > 0 ? rows : 1))
    return fail(SCAPE_ESHAPE, "%s: ld %lld must be at least cols %lld (and rows * ld at most 2^46)", name,
                (long long)m.ld, (long long)cols);
  return SCAPE_OK;
}

inline scape_status check_act(const char* name, const scape_act_view& a, int64_t rows, bool need) {
  if (!a.codes && !a.scales && !(need && rows > 0)) return SCAPE_OK;
  if (!a.codes || !a.scales) return fail(SCAPE_EINVAL, "%s is null", name);
  if ((uintptr_t)a.codes & 15u) return fail(SCAPE_EINVAL, "%s: codes must be 16-byte aligned", name);
  return SCAPE_OK;
}

inline bool misaligned4(const void* p) { return ((uintptr_t)p & 3u) != 0; }

inline scape_status check_workspace(const void* ws, size_t have, size_t need) {
  if (!ws) return fail(SCAPE_EINVAL, "workspace is null");
  if ((uintptr_t)ws & 255u) return fail(SCAPE_EINVAL, "workspace must be 256-byte aligned");
  if (have < need) return fail(SCAPE_EWORKSPACE, "workspace has %zu bytes, needs %zu", have, need);
  return SCAPE_OK;
}

// An output may be an input's own matrix, element on element, or lie apart.
inline bool shifted_alias(const scape_matrix& o, const scape_matrix& i, int64_t rows) {
  return o.data && o.data == i.data && rows > 1 && o.ld != i.ld;
}

inline size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

}  // namespace scape
