// Log probabilities of given tokens, entropy, the likeliest alternatives, and
// the gradient of the logits.
#include "ends.h"

namespace scape {
namespace {


// Orders floats as unsigned numbers: NaN above everything, -0 as 0.
__device__ __forceinline__ uint32_t order_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  if (x != x) return 0xffffffffu;
  return (b >> 31) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float of_order(uint32_t k) {
  return __uint_as_float((k >> 31) ? k & 0x7fffffffu : ~k);
}
// The larger key is the larger logit, or of equal ones the lower index.
__device__ __forceinline__ uint64_t key_of(float x, int64_t i) {
  return (uint64_t)order_of(x) << 32 | (0xffffffffu - (uint32_t)i);
}
__device__ __forceinline__ int key_index(uint64_t k) { return (int)(0xffffffffu - (uint32_t)k); }

__device__ __forceinline__ uint64_t block_max(uint64_t x, uint64_t* lds) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) {
    const uint64_t y = __shfl_xor((unsigned long long)x, d, 64);
    x = x > y ? x : y;
  }
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
  __syncthreads();
  for (int w = 0; w < kThreads / 64; ++w) x = x > lds[w] ? x : lds[w];
  return x;
}
__device__ __forceinline__ float block_sum(float x, float* lds) {
  x = wave_sum(x);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
  __syncthreads();
  x = 0.0f;
  for (int w = 0; w < kThreads / 64; ++w) x += lds[w];
  return x;
}

// The gradient of row r, from its m, log-sum and entropy.
template <int DT>
__device__ void emit_gradient(const LogprobArgs& a, int64_t r, float m, float ls, float h) {
  const int64_t y = a.dlogp ? token_at(a.targets, r) : -1;
  const float w = y >= 0 && y < a.vocab ? a.dlogp[r] : 0.0f;
  const float d = a.dentropy ? a.dentropy[r] : 0.0f;
  const int64_t in = r * a.logits.ld, out = r * a.dlogits.ld;
  const bool none = (w == 0.0f && d == 0.0f) || m == -__builtin_inff();
  for (int64_t j = threadIdx.x; j < a.vocab; j += kThreads) {
    float g = 0.0f;
    if (!none) {
      const float lp = (Elem<DT>::get(a.logits.data, in + j) - m) * a.scale - ls;
      const float p = expf(lp);
      g = j == y ? -w * expm1f(lp) : -w * p;
      if (d != 0.0f && !(p == 0.0f)) g -= d * p * (lp + h);
      g *= a.scale;
    }
    Elem<DT>::put(a.dlogits.data, out + j, g);
  }
}

template <int DT>
__global__ void __launch_bounds__(kThreads) logprobs_kernel(LogprobArgs a) {
  __shared__ uint64_t lds8[kThreads / 64];
  __shared__ float lds4[kThreads / 64];
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const int64_t in = r * a.logits.ld;
    uint64_t best = 0;
    for (int64_t j = threadIdx.x; j < a.vocab; j += kThreads) {
      const uint64_t k = key_of(Elem<DT>::get(a.logits.data, in + j), j);
      best = best > k ? best : k;
    }
    best = block_max(best, lds8);
    const float m = of_order((uint32_t)(best >> 32));
    const bool empty = m == -__builtin_inff();
    float o = 0.0f, u = 0.0f;
    if (!empty) {
      for (int64_t j = threadIdx.x; j < a.vocab; j += kThreads) {
        const float z = (Elem<DT>::get(a.logits.data, in + j) - m) * a.scale;
        const float e = expf(z);
        if (j != key_index(best)) o += e;
        if (!(e == 0.0f)) u += e * z;
      }
    }
    o = block_sum(o, lds4);
    u = block_sum(u, lds4);
    if (!(m < __builtin_inff())) o = __builtin_nanf("");
    const float ls = log1pf(o);
    const float h = ls - u / (1.0f + o);
    const float ninf = -__builtin_inff();
    if (threadIdx.x == 0) {
      if (a.logp) {
        const int64_t y = token_at(a.targets, r);
        float v = 0.0f;
        if (y >= 0 && y < a.vocab)
          v = empty ? ninf : (Elem<DT>::get(a.logits.data, in + y) - m) * a.scale - ls;
        a.logp[r] = v;
      }
      if (a.stats) a.stats[2 * r] = m, a.stats[2 * r + 1] = ls;
      if (a.entropy) a.entropy[r] = h;
    }
    uint64_t last = best;
    for (int i = 0; i < a.top; ++i) {
      if (i > 0) {
        uint64_t next = 0;
        for (int64_t j = threadIdx.x; j < a.vocab; j += kThreads) {
          const uint64_t k = key_of(Elem<DT>::get(a.logits.data, in + j), j);
          if (k < last) next = next > k ? next : k;
        }
        last = block_max(next, lds8);
      }
      if (threadIdx.x == 0) {
        if (a.top_ids) a.top_ids[r * a.top + i] = key_index(last);
        if (a.top_logp)
          a.top_logp[r * a.top + i] = empty ? ninf : (of_order((uint32_t)(last >> 32)) - m) * a.scale - ls;
      }
    }
    if (a.dlogits.data) {
      __syncthreads();  // in logits' place: the target's logit has been read
      emit_gradient<DT>(a, r, m, ls, h);
    }
  }
}

template <int DT>
__global__ void __launch_bounds__(kThreads) logprobs_back_kernel(LogprobArgs a) {
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x)
    emit_gradient<DT>(a, r, a.stats[2 * r], a.stats[2 * r + 1], a.dentropy ? a.entropy[r] : 0.0f);
}

unsigned row_grid(int64_t rows) { return (unsigned)(rows > (1 << 20) ? 1 << 20 : rows); }

}  // namespace

size_t logprobs_workspace(int64_t, int64_t, int) { return 256; }

hipError_t launch_logprobs(const LogprobArgs& a, void*, hipStream_t s) {
  if (a.rows == 0) return hipSuccess;
  const dim3 grid(row_grid(a.rows));
  if (a.logits.dtype == SCAPE_F32) logprobs_kernel<SCAPE_F32><<<grid, kThreads, 0, s>>>(a);
  else if (a.logits.dtype == SCAPE_BF16) logprobs_kernel<SCAPE_BF16><<<grid, kThreads, 0, s>>>(a);
  else logprobs_kernel<SCAPE_F16><<<grid, kThreads, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_logprobs_backward(const LogprobArgs& a, hipStream_t s) {
  if (a.rows == 0) return hipSuccess;
  const dim3 grid(row_grid(a.rows));
  if (a.logits.dtype == SCAPE_F32) logprobs_back_kernel<SCAPE_F32><<<grid, kThreads, 0, s>>>(a);
  else if (a.logits.dtype == SCAPE_BF16) logprobs_back_kernel<SCAPE_BF16><<<grid, kThreads, 0, s>>>(a);
  else logprobs_back_kernel<SCAPE_F16><<<grid, kThreads, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace scape
