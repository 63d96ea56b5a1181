// C ABI of the embedding, the token log probabilities and the gradient
// clipping (declared in include/scape.h): argument validation.
#include "checks.h"
#include "ends.h"

#include <cmath>

using namespace scape;

namespace {

bool table_ok(int64_t rows) { return rows >= 1 && rows < (int64_t(1) << 31); }

scape_status check_ids(const char* name, const scape_ids& ids, int64_t count, bool need) {
  if (!ids.data) return need && count > 0 ? fail(SCAPE_EINVAL, "%s is null", name) : SCAPE_OK;
  if (ids.bits != 32 && ids.bits != 64) return fail(SCAPE_EINVAL, "%s: %d bits (need 32 or 64)", name, ids.bits);
  if ((uintptr_t)ids.data % (ids.bits / 8)) return fail(SCAPE_EINVAL, "%s is not aligned to its type", name);
  return SCAPE_OK;
}

scape_status check_embed_size(int64_t tokens, int64_t vocab, int64_t cols) {
  if (tokens < 0 || tokens > kMaxTokens || !table_ok(vocab) || !cols_ok(cols))
    return fail(SCAPE_ESHAPE,
                "invalid shape: tokens=%lld vocab=%lld cols=%lld (need 0<=tokens<=2^26, 1<=vocab<2^31, 1<=cols<=2^20)",
                (long long)tokens, (long long)vocab, (long long)cols);
  return SCAPE_OK;
}

scape_status check_logits(int64_t rows, int64_t vocab, int32_t top) {
  scape_status st = check_size(rows, vocab);
  if (st) return st;
  if (top < 0 || top > kMaxTop || top > vocab)
    return fail(SCAPE_ESHAPE, "invalid shape: top=%d (need 0<=top<=min(vocab, %d))", top, kMaxTop);
  return SCAPE_OK;
}

scape_status check_scale(float scale) {
  // within 2^+-100, where its products with 32-bit constants keep their digits
  if (!(scale >= 0x1p-100f) || !(scale <= 0x1p100f))
    return fail(SCAPE_EINVAL, "scale must be positive and within 2^-100 and 2^100");
  return SCAPE_OK;
}

// The gradient's own arguments.
scape_status check_dlogits(const LogprobArgs& a) {
  scape_status st = check_matrix("dlogits", a.dlogits, a.rows, a.vocab, true);
  if (st) return st;
  if (a.rows > 0 && !a.dlogp && !a.dentropy) return fail(SCAPE_EINVAL, "dlogp and dentropy are both null");
  if (a.dlogits.data && a.dlogits.dtype != a.logits.dtype)
    return fail(SCAPE_EINVAL, "dlogits must have logits' dtype");
  if (shifted_alias(a.dlogits, a.logits, a.rows))
    return fail(SCAPE_EINVAL, "an output in an input's place must have its ld");
  if (misaligned4(a.dlogp) || misaligned4(a.dentropy))
    return fail(SCAPE_EINVAL, "dlogp and dentropy must be 4-byte aligned");
  return SCAPE_OK;
}

scape_status check_grads(int32_t count, const scape_grad* grads, int32_t groups, bool clip) {
  if (count < 0 || count > kMaxGrads || groups < 1 || groups > kMaxGrads || count % groups)
    return fail(SCAPE_ESHAPE, "invalid list: count=%d groups=%d (need 0<=count<=2^20, 1<=groups<=2^20, "
                "count%%groups==0)", count, groups);
  if (count > 0 && !grads) return fail(SCAPE_EINVAL, "grads is null");
  int64_t total = 0;
  for (int32_t i = 0; i < count; ++i) {
    const scape_grad& g = grads[i];
    if (g.count < 0 || g.count > (int64_t(1) << 46))
      return fail(SCAPE_ESHAPE, "grads[%d]: count %lld (need 0<=count<=2^46)", i, (long long)g.count);
    total += g.count;
    if (total > (int64_t(1) << 46)) return fail(SCAPE_ESHAPE, "the list holds more than 2^46 elements");
    if (g.count == 0) continue;
    if (!g.data) return fail(SCAPE_EINVAL, "grads[%d] is null", i);
    if (g.dtype != SCAPE_F32 && g.dtype != SCAPE_BF16 && g.dtype != SCAPE_F16)
      return fail(SCAPE_EINVAL, "grads[%d]: unknown dtype %d", i, g.dtype);
    if ((uintptr_t)g.data % dtype_bytes(g.dtype)) return fail(SCAPE_EINVAL, "grads[%d] is not aligned to its type", i);
    if (!clip || !g.out) continue;
    if (g.out_dtype != g.dtype && g.out_dtype != SCAPE_F32)
      return fail(SCAPE_EINVAL, "grads[%d]: out must have its dtype or fp32", i);
    if ((uintptr_t)g.out % dtype_bytes(g.out_dtype))
      return fail(SCAPE_EINVAL, "grads[%d]: out is not aligned to its type", i);
    if (g.out == g.data && g.out_dtype != g.dtype)
      return fail(SCAPE_EINVAL, "grads[%d]: out in data's place must have its dtype", i);
  }
  return SCAPE_OK;
}

scape_status run_grads(int32_t count, const scape_grad* grads, int32_t groups, float scale, bool clip, float max_norm,
                       float* norm, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  scape_status st = check_grads(count, grads, groups, clip);
  if (st) return st;
  if ((st = check_scale(scale))) return st;
  if (!norm) return fail(SCAPE_EINVAL, "norm is null");
  if (misaligned4(norm)) return fail(SCAPE_EINVAL, "norm must be 4-byte aligned");
  if ((st = check_workspace(workspace, workspace_bytes, grad_workspace(count, grads, groups)))) return st;
  return hip_check(launch_grads(count, grads, groups, scale, clip, max_norm, norm, workspace, stream),
                   clip ? "grad clip" : "grad norm");
}

}  // namespace

extern "C" {

scape_status scape_embed(int64_t tokens, int64_t vocab, int64_t positions, int64_t cols, scape_ids ids,
                         scape_matrix table, float scale, scape_ids pos, scape_matrix pos_table, scape_matrix out,
                         hipStream_t stream) {
  scape_status st = check_embed_size(tokens, vocab, cols);
  if (st) return st;
  if ((st = check_ids("ids", ids, tokens, true))) return st;
  if ((st = check_matrix("table", table, vocab, cols, tokens > 0))) return st;
  if ((st = check_matrix("out", out, tokens, cols, true))) return st;
  if (!std::isfinite(scale)) return fail(SCAPE_EINVAL, "scale must be finite");
  if (pos_table.data) {
    if (!table_ok(positions))
      return fail(SCAPE_ESHAPE, "invalid shape: positions=%lld (need 1<=positions<2^31)", (long long)positions);
    if ((st = check_ids("pos", pos, tokens, true))) return st;
    if ((st = check_matrix("pos_table", pos_table, positions, cols, true))) return st;
    if (table.data && pos_table.dtype != table.dtype) return fail(SCAPE_EINVAL, "pos_table must have table's dtype");
  }
  return hip_check(launch_embed(tokens, vocab, positions, cols, ids, table, scale, pos, pos_table, out, stream),
                   "embed");
}

size_t scape_embed_workspace_bytes(int64_t tokens, int64_t cols) {
  if (tokens < 0 || tokens > kMaxTokens || !cols_ok(cols)) return 0;
  return embed_workspace(tokens, cols);
}

scape_status scape_embed_backward(int64_t tokens, int64_t vocab, int64_t cols, scape_ids ids, scape_matrix dy,
                                  float scale, float* dtable, int32_t accumulate, void* workspace,
                                  size_t workspace_bytes, hipStream_t stream) {
  scape_status st = check_embed_size(tokens, vocab, cols);
  if (st) return st;
  if ((st = check_ids("ids", ids, tokens, true))) return st;
  if ((st = check_matrix("dy", dy, tokens, cols, true))) return st;
  if (!std::isfinite(scale)) return fail(SCAPE_EINVAL, "scale must be finite");
  if (!dtable) return fail(SCAPE_EINVAL, "dtable is null");
  if (misaligned4(dtable)) return fail(SCAPE_EINVAL, "dtable must be 4-byte aligned");
  if ((st = check_workspace(workspace, workspace_bytes, embed_workspace(tokens, cols)))) return st;
  return hip_check(launch_embed_backward(tokens, vocab, cols, ids, dy, scale, dtable, accumulate != 0, workspace,
                                         stream),
                   "embed backward");
}

int32_t scape_token_logprobs_max_top(void) { return kMaxTop; }

size_t scape_token_logprobs_workspace_bytes(int64_t rows, int64_t vocab, int32_t top) {
  if (!rows_ok(rows) || !cols_ok(vocab) || top < 0 || top > kMaxTop || top > vocab) return 0;
  return kLogprobsWorkspace;
}

scape_status scape_token_logprobs(int64_t rows, int64_t vocab, scape_matrix logits, float scale, scape_ids targets,
                                  float* logp, float* stats, float* entropy, int32_t top, float* top_logp,
                                  int32_t* top_ids, const float* dlogp, const float* dentropy, scape_matrix dlogits,
                                  void* workspace, size_t workspace_bytes, hipStream_t stream) {
  scape_status st = check_logits(rows, vocab, top);
  if (st) return st;
  if ((st = check_matrix("logits", logits, rows, vocab, true))) return st;
  if ((st = check_scale(scale))) return st;
  if ((st = check_ids("targets", targets, rows, logp || dlogp))) return st;
  if (misaligned4(logp) || misaligned4(stats) || misaligned4(entropy) || misaligned4(top_logp) || misaligned4(top_ids))
    return fail(SCAPE_EINVAL, "logp, stats, entropy, top_logp and top_ids must be 4-byte aligned");
  if (rows > 0 && top > 0 && !top_logp && !top_ids) return fail(SCAPE_EINVAL, "top_logp and top_ids are both null");
  if (top == 0 && (top_logp || top_ids)) return fail(SCAPE_EINVAL, "top_logp and top_ids need top > 0");
  if (rows > 0 && !logp && !stats && !entropy && top == 0 && !dlogits.data)
    return fail(SCAPE_EINVAL, "every output is null");
  const LogprobArgs a{rows, vocab, logits, scale, targets, logp, stats, entropy, top, top_logp, top_ids, dlogp,
                      dentropy, dlogits};
  if (dlogits.data) {
    if ((st = check_dlogits(a))) return st;
  } else if (dlogp || dentropy) {
    return fail(SCAPE_EINVAL, "dlogp and dentropy need dlogits");
  }
  if ((st = check_workspace(workspace, workspace_bytes, kLogprobsWorkspace))) return st;
  return hip_check(launch_logprobs(a, stream), "token logprobs");
}

scape_status scape_token_logprobs_backward(int64_t rows, int64_t vocab, scape_matrix logits, float scale,
                                           scape_ids targets, const float* stats, const float* entropy,
                                           const float* dlogp, const float* dentropy, scape_matrix dlogits,
                                           hipStream_t stream) {
  scape_status st = check_logits(rows, vocab, 0);
  if (st) return st;
  if ((st = check_matrix("logits", logits, rows, vocab, true))) return st;
  if ((st = check_scale(scale))) return st;
  if ((st = check_ids("targets", targets, rows, dlogp != nullptr))) return st;
  if (rows > 0 && !stats) return fail(SCAPE_EINVAL, "stats is null");
  if (rows > 0 && dentropy && !entropy) return fail(SCAPE_EINVAL, "entropy is null");
  if (misaligned4(stats) || misaligned4(entropy))
    return fail(SCAPE_EINVAL, "stats and entropy must be 4-byte aligned");
  const LogprobArgs a{rows,    vocab, logits,  scale,   targets, nullptr, const_cast<float*>(stats),
                      const_cast<float*>(entropy), 0,   nullptr, nullptr, dlogp, dentropy, dlogits};
  if ((st = check_dlogits(a))) return st;
  return hip_check(launch_logprobs_backward(a, stream), "token logprobs backward");
}

size_t scape_grad_workspace_bytes(int32_t count, const scape_grad* grads, int32_t groups) {
  if (check_grads(count, grads, groups, false)) return 0;
  return grad_workspace(count, grads, groups);
}

scape_status scape_grad_norm(int32_t count, const scape_grad* grads, int32_t groups, float scale, float* norm,
                             void* workspace, size_t workspace_bytes, hipStream_t stream) {
  return run_grads(count, grads, groups, scale, false, 0.0f, norm, workspace, workspace_bytes, stream);
}

scape_status scape_grad_clip(int32_t count, const scape_grad* grads, int32_t groups, float scale, float max_norm,
                             float* norm, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (!(max_norm > 0.0f)) return fail(SCAPE_EINVAL, "max_norm must be positive");
  return run_grads(count, grads, groups, scale, true, max_norm, norm, workspace, workspace_bytes, stream);
}

}  // extern "C"
