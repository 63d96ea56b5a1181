// Launch wrappers of the operators at the ends of a training step.
#pragma once

#include "activations.h"

namespace scape {

constexpr int64_t kMaxTokens = int64_t(1) << 26;

hipError_t launch_embed(int64_t tokens, int64_t vocab, int64_t positions, int64_t cols, const scape_ids& ids,
                        const scape_matrix& table, float scale, const scape_ids& pos, const scape_matrix& pos_table,
                        const scape_matrix& out, hipStream_t s);
size_t embed_workspace(int64_t tokens, int64_t cols);
hipError_t launch_embed_backward(int64_t tokens, int64_t vocab, int64_t cols, const scape_ids& ids,
                                 const scape_matrix& dy, float scale, float* dtable, bool accumulate, void* ws,
                                 hipStream_t s);

constexpr int kMaxTop = 64;
constexpr int32_t kMaxGrads = 1 << 20;  // tensors of a list, and groups: a launch has a workgroup for each
struct LogprobArgs {
  int64_t rows, vocab;
  scape_matrix logits;
  float scale;
  scape_ids targets;
  float* logp;
  float* stats;
  float* entropy;
  int top;
  float* top_logp;
  int32_t* top_ids;
  const float* dlogp;
  const float* dentropy;
  scape_matrix dlogits;
};
constexpr size_t kLogprobsWorkspace = 256;  // reserved: no kernel writes there
hipError_t launch_logprobs(const LogprobArgs& a, hipStream_t s);
// The gradient alone, from stats and entropy (inputs here).
hipError_t launch_logprobs_backward(const LogprobArgs& a, hipStream_t s);

size_t grad_workspace(int32_t count, const scape_grad* grads, int32_t groups);
// clip false: the norm alone.
hipError_t launch_grads(int32_t count, const scape_grad* grads, int32_t groups, float scale, bool clip, float max_norm,
                        float* norm, void* ws, hipStream_t s);

#ifdef __HIPCC__

template <typename I>
__device__ __forceinline__ int64_t token_at(const void* ids, int64_t i) {
  return static_cast<const I*>(ids)[i];
}
__device__ __forceinline__ int64_t token_at(const scape_ids& ids, int64_t i) {
  return ids.bits == 64 ? token_at<int64_t>(ids.data, i) : token_at<int32_t>(ids.data, i);
}

#endif

}  // namespace scape
