// Norm of gradients over many tensors, and clipping by it.
//
// The tensors of a list go to the kernels by value, so that a call copies no
// table to the device and can be captured.  Each is cut into pieces of one
// size, a workgroup sums one piece, and the pieces' sums are added in their
// order: no atomics, so results do not depend on the order of the workgroups.
#include "ends.h"

namespace scape {
namespace {

constexpr int kSpans = 64;         // tensors of one launch
constexpr int64_t kPieces = 4096;  // pieces of a long list, about

struct Span {
  const void* data;
  void* out;
  int64_t count;
  int32_t first;  // piece of the whole list at which it begins
  int16_t dtype, out_dtype;
  int32_t group;
};

struct SpanArgs {
  Span span[kSpans];
  int32_t n;
  int32_t end;  // one past the last span's last piece
  int64_t piece;
  double* sums;
  const double* factors;
};

struct GroupArgs {
  int32_t first[kSpans + 1];  // pieces of each group
  int32_t n;
  float scale, max_norm;
  bool clip;
  const double* sums;
  double* factors;
  float* norm;
};

__device__ __forceinline__ double block_sum(double x, double* lds) {
  x = wave_sum(x);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
  __syncthreads();
  x = lds[0];
  for (int w = 1; w < kThreads / 64; ++w) x += lds[w];
  return x;
}

// The span of a piece: the last one that begins at or before it and holds
// anything (an empty tensor begins where the next one does).
__device__ __forceinline__ int span_of(const SpanArgs& a, int32_t piece) {
  int lo = 0, hi = a.n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (a.span[mid].first <= piece) lo = mid;
    else hi = mid;
  }
  return lo;
}

template <int DT>
__device__ __forceinline__ double squares(const Span& s, int64_t lo, int64_t hi) {
  double sum = 0.0;
  for (int64_t i = lo + (int64_t)threadIdx.x * 8; i < hi; i += kThreads * 8) {
    float v[8];
    load8<DT>(s.data, 0, i, hi, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) sum = __builtin_fma((double)v[j], (double)v[j], sum);
  }
  return sum;
}

__global__ void __launch_bounds__(kThreads) grad_sum_kernel(SpanArgs a) {
  __shared__ double lds[kThreads / 64];
  const int32_t piece = a.span[0].first + (int32_t)blockIdx.x;
  const Span s = a.span[span_of(a, piece)];
  const int64_t lo = (piece - s.first) * a.piece;
  const int64_t hi = lo + a.piece < s.count ? lo + a.piece : s.count;
  double sum;
  if (s.dtype == SCAPE_F32) sum = squares<SCAPE_F32>(s, lo, hi);
  else if (s.dtype == SCAPE_BF16) sum = squares<SCAPE_BF16>(s, lo, hi);
  else sum = squares<SCAPE_F16>(s, lo, hi);
  sum = block_sum(sum, lds);
  if (threadIdx.x == 0) a.sums[piece] = sum;
}

// One workgroup a group: its norm and the factor of its gradients.
__global__ void __launch_bounds__(kThreads) grad_norm_kernel(GroupArgs a) {
  __shared__ double lds[kThreads / 64];
  const int g = blockIdx.x;
  double sum = 0.0;
  for (int32_t i = a.first[g] + threadIdx.x; i < a.first[g + 1]; i += kThreads) sum += a.sums[i];
  sum = block_sum(sum, lds);
  if (threadIdx.x != 0) return;
  const double norm = sqrt(sum) * (double)a.scale;
  a.norm[g] = (float)norm;
  if (!a.clip) return;
  const bool over = norm > (double)a.max_norm && norm < (double)__builtin_inff();
  a.factors[g] = over ? (double)a.scale * ((double)a.max_norm / norm) : (double)a.scale;
}

template <int DT, int OT>
__device__ __forceinline__ void scale_span(const Span& s, int64_t lo, int64_t hi, double f) {
  for (int64_t i = lo + (int64_t)threadIdx.x * 8; i < hi; i += kThreads * 8) {
    float v[8];
    load8<DT>(s.data, 0, i, hi, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = (float)((double)v[j] * f);
    store8<OT>(s.out, 0, i, hi, v);
  }
}

__global__ void __launch_bounds__(kThreads) grad_scale_kernel(SpanArgs a) {
  const int32_t piece = a.span[0].first + (int32_t)blockIdx.x;
  const Span s = a.span[span_of(a, piece)];
  const int64_t lo = (piece - s.first) * a.piece;
  const int64_t hi = lo + a.piece < s.count ? lo + a.piece : s.count;
  const double f = a.factors[s.group];
  if (f == 1.0 && s.out == s.data) return;
  if (s.dtype == SCAPE_F32) scale_span<SCAPE_F32, SCAPE_F32>(s, lo, hi, f);
  else if (s.dtype == SCAPE_BF16 && s.out_dtype == SCAPE_BF16) scale_span<SCAPE_BF16, SCAPE_BF16>(s, lo, hi, f);
  else if (s.dtype == SCAPE_BF16) scale_span<SCAPE_BF16, SCAPE_F32>(s, lo, hi, f);
  else if (s.out_dtype == SCAPE_F16) scale_span<SCAPE_F16, SCAPE_F16>(s, lo, hi, f);
  else scale_span<SCAPE_F16, SCAPE_F32>(s, lo, hi, f);
}

// Elements of a piece (a multiple of what a workgroup reads at a time), so
// that a list has about kPieces of them at most, and the pieces of each tensor.
int64_t piece_of(int32_t count, const scape_grad* grads) {
  int64_t total = 0;
  for (int32_t i = 0; i < count; ++i) total += grads[i].count;
  const int64_t unit = kThreads * 8;
  const int64_t want = (total + kPieces - 1) / kPieces;
  return (want / unit + 1) * unit;
}
int64_t pieces(int64_t count, int64_t piece) { return (count + piece - 1) / piece; }

int64_t pieces_of(int32_t count, const scape_grad* grads) {
  const int64_t piece = piece_of(count, grads);
  int64_t n = 0;
  for (int32_t i = 0; i < count; ++i) n += pieces(grads[i].count, piece);
  return n;
}

}  // namespace

size_t grad_workspace(int32_t count, const scape_grad* grads, int32_t groups) {
  const size_t n = (size_t)pieces_of(count, grads) + (size_t)groups;
  return (n * sizeof(double) + 255) & ~(size_t)255;
}

hipError_t launch_grads(int32_t count, const scape_grad* grads, int32_t groups, float scale, bool clip, float max_norm,
                        float* norm, void* ws, hipStream_t s) {
  const int64_t piece = piece_of(count, grads);
  const int32_t per = count / groups;
  double* sums = static_cast<double*>(ws);
  double* factors = sums + pieces_of(count, grads);

  const auto walk = [&](bool scaling) {
    SpanArgs a;
    a.piece = piece;
    a.sums = sums;
    a.factors = factors;
    a.n = 0;
    int32_t at = 0;
    for (int32_t i = 0; i <= count; ++i) {
      if (a.n > 0 && (i == count || a.n == kSpans)) {
        a.end = at;
        const dim3 grid((unsigned)(at - a.span[0].first));
        if (scaling) grad_scale_kernel<<<grid, kThreads, 0, s>>>(a);
        else grad_sum_kernel<<<grid, kThreads, 0, s>>>(a);
        a.n = 0;
      }
      if (i == count || grads[i].count == 0) continue;
      const scape_grad& g = grads[i];
      Span& p = a.span[a.n++];
      p.data = g.data;
      p.out = g.out ? g.out : const_cast<void*>(g.data);
      p.count = g.count;
      p.first = at;
      p.dtype = (int16_t)g.dtype;
      p.out_dtype = (int16_t)(g.out ? g.out_dtype : g.dtype);
      p.group = i / per;
      at += (int32_t)pieces(g.count, piece);
    }
  };

  walk(false);
  GroupArgs b;
  b.scale = scale;
  b.max_norm = max_norm;
  b.clip = clip;
  b.sums = sums;
  int32_t at = 0;
  for (int32_t g0 = 0; g0 < groups; g0 += kSpans) {
    b.n = groups - g0 < kSpans ? groups - g0 : kSpans;
    for (int32_t g = 0; g < b.n; ++g) {
      b.first[g] = at;
      for (int32_t i = (g0 + g) * per; i < (g0 + g + 1) * per; ++i) at += (int32_t)pieces(grads[i].count, piece);
    }
    b.first[b.n] = at;
    b.factors = factors + g0;
    b.norm = norm + g0;
    grad_norm_kernel<<<dim3((unsigned)b.n), kThreads, 0, s>>>(b);
  }
  if (clip) walk(true);
  return hipGetLastError();
}

}  // namespace scape
