// Weight gradient of a linear layer from the 8-bit checkpoint of its input:
// dw[o][i] = gain[i] * sum_t dy[t][o] * x[t][i], on the matrix cores in bf16
// with fp32 sums.  A checkpoint's values have at most 8 significant bits and
// a power of two as their scale, so they are exact in bf16; a bf16 dy is
// taken as it is, and fp16 and fp32 are split into 2 and 3 bf16 terms that
// add up to the value.  So every product is exact and only the sums round.

#include "activations.h"

namespace scape {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kBM = 128;         // out per workgroup
constexpr int kBN = 128;         // in per workgroup
constexpr int kBK = 32;          // rows per stage
constexpr int kLdsK = kBK + 8;   // padded k extent of a staged column
constexpr int kMinSplitRows = 128;
constexpr int kTargetBlocks = 512;

constexpr int terms_of(int dt) { return dt == SCAPE_F32 ? 3 : dt == SCAPE_F16 ? 2 : 1; }

struct WgradArgs {
  int64_t rows, in, out, nblk;
  const void* dy;
  int64_t dy_ld;
  const int8_t* codes;
  const uint8_t* scales;
  const float* gain;   // applied here only when there is one split
  float* dw;           // [splits][out][in], or dw itself (one split)
  float* db;           // [splits][out], or dbias itself; null: none
  bool accumulate;     // one split
  int64_t split_rows;  // rows a split sums (a multiple of kBK)
  int tiles_m, tiles_n;
};

// Splits v into its leading 8 significant bits (the upper half of its
// pattern) and the rest.  An infinity leaves nothing; a NaN stays one in the
// rest if its payload is cut off.
__device__ __forceinline__ uint32_t cut_term(float& v) {
  const uint32_t u = __float_as_uint(v) & 0xffff0000u;
  const float h = __uint_as_float(u);
  v = __builtin_isinf(v) ? 0.0f : v - h;
  return u >> 16;
}

template <int DT>
__global__ void __launch_bounds__(256) wgrad_kernel(WgradArgs a) {
  constexpr int NT = terms_of(DT);
  __shared__ __attribute__((aligned(16))) uint16_t lds_a[NT][kBM][kLdsK];
  __shared__ __attribute__((aligned(16))) uint16_t lds_b[kBN][kLdsK];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int tile = blockIdx.x;
  const int64_t m0 = (int64_t)(tile / a.tiles_n) * kBM, n0 = (int64_t)(tile % a.tiles_n) * kBN;
  const int64_t split = blockIdx.y;
  const int64_t t_begin = split * a.split_rows;
  const int64_t t_end = t_begin + a.split_rows < a.rows ? t_begin + a.split_rows : a.rows;
  const bool bias = a.db && n0 == 0;

  f32x16 acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[i][j] = (f32x16)(0.0f);
  float bsum[2] = {0.0f, 0.0f};

  // staging: wave w takes rows 8w .. 8w + 7 of a stage, a lane two columns
  const int64_t mc = m0 + 2 * lane, nc = n0 + 2 * lane;
  const int wm = (wave >> 1) * 64, wn = (wave & 1) * 64;

  for (int64_t t0 = t_begin; t0 < t_end; t0 += kBK) {
    float y[8][2];
    uint32_t xb[2][8];
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      const int64_t t = t0 + wave * 8 + r;
      const bool in_t = t < t_end;
      y[r][0] = in_t && mc < a.out ? Elem<DT>::get(a.dy, t * a.dy_ld + mc) : 0.0f;
      y[r][1] = in_t && mc + 1 < a.out ? Elem<DT>::get(a.dy, t * a.dy_ld + mc + 1) : 0.0f;
      xb[0][r] = xb[1][r] = 0;
      if (in_t && nc < a.nblk * kActBlock) {
        const int64_t b = t * a.nblk + nc / kActBlock;
        const uint16_t q = *reinterpret_cast<const uint16_t*>(a.codes + b * kActBlock + (nc & 31));
        const float f = __uint_as_float((uint32_t)a.scales[b] << 23);
        xb[0][r] = __float_as_uint((float)(int8_t)(q & 0xff) * f) >> 16;
        xb[1][r] = __float_as_uint((float)(int8_t)(q >> 8) * f) >> 16;
      }
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      u32x4 p;
#pragma unroll
      for (int h = 0; h < 4; ++h) p[h] = xb[c][2 * h] | (xb[c][2 * h + 1] << 16);
      *reinterpret_cast<u32x4*>(&lds_b[2 * lane + c][wave * 8]) = p;
      if (bias)
#pragma unroll
        for (int r = 0; r < 8; ++r) bsum[c] += y[r][c];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          const uint32_t lo = cut_term(y[2 * h][c]), hi = cut_term(y[2 * h + 1][c]);
          p[h] = lo | (hi << 16);
        }
        *reinterpret_cast<u32x4*>(&lds_a[n][2 * lane + c][wave * 8]) = p;
      }
    }
    __syncthreads();
#pragma unroll
    for (int kk = 0; kk < kBK; kk += 16) {
      const int k = kk + 8 * (lane >> 5);
      bf16x8 bv[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) bv[j] = *reinterpret_cast<const bf16x8*>(&lds_b[wn + j * 32 + (lane & 31)][k]);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const bf16x8 av = *reinterpret_cast<const bf16x8*>(&lds_a[n][wm + i * 32 + (lane & 31)][k]);
#pragma unroll
          for (int j = 0; j < 2; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(av, bv[j], acc[i][j], 0, 0, 0);
        }
    }
    __syncthreads();
  }

  // element e of a 32x32 accumulator: row 8*(e/4) + 4*(lane/32) + e%4, column lane%32
  float* dw = a.dw + split * a.out * a.in;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int64_t n = n0 + wn + j * 32 + (lane & 31);
    if (n >= a.in) continue;
    const float g = a.gain ? a.gain[n] : 1.0f;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int64_t m = m0 + wm + i * 32 + 8 * (e >> 2) + 4 * (lane >> 5) + (e & 3);
        if (m >= a.out) continue;
        float* p = dw + m * a.in + n;
        const float v = a.gain ? acc[i][j][e] * g : acc[i][j][e];
        *p = a.accumulate ? *p + v : v;
      }
  }
  if (bias) {  // the four waves' sums, in wave order
    float* red = reinterpret_cast<float*>(&lds_b[0][0]);
    red[wave * 128 + 2 * lane] = bsum[0];
    red[wave * 128 + 2 * lane + 1] = bsum[1];
    __syncthreads();
    const int64_t m = m0 + threadIdx.x;
    if (threadIdx.x < kBM && m < a.out) {
      const float v = ((red[threadIdx.x] + red[128 + threadIdx.x]) + red[256 + threadIdx.x]) + red[384 + threadIdx.x];
      float* p = a.db + split * a.out + m;
      *p = a.accumulate ? *p + v : v;
    }
  }
}

// out[i] (+)= gain[i % in] * (the sum of the splits' partial sums, in order).
__global__ void __launch_bounds__(kThreads)
join_kernel(const float* __restrict__ parts, int splits, int64_t n, int64_t in, const float* __restrict__ gain,
            float* __restrict__ out, bool accumulate) {
  const int64_t step = (int64_t)gridDim.x * kThreads;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n; i += step) {
    float s = parts[i];
    for (int p = 1; p < splits; ++p) s += parts[(int64_t)p * n + i];
    if (gain) s *= gain[i % in];
    out[i] = accumulate ? out[i] + s : s;
  }
}

int64_t tiles(int64_t x, int64_t t) { return (x + t - 1) / t; }

void launch_join(const float* parts, int splits, int64_t n, int64_t in, const float* gain, float* out,
                 bool accumulate, hipStream_t s) {
  int64_t grid = tiles(n, kThreads);
  if (grid > 8192) grid = 8192;
  join_kernel<<<(unsigned)grid, kThreads, 0, s>>>(parts, splits, n, in, gain, out, accumulate);
}

}  // namespace

int wgrad_splits(int64_t rows, int64_t in, int64_t out) {
  const int64_t t = tiles(out, kBM) * tiles(in, kBN);
  int64_t s = (kTargetBlocks + t - 1) / t;
  const int64_t most = rows / kMinSplitRows;
  if (s > most) s = most;
  return s < 1 ? 1 : (int)s;
}

size_t wgrad_workspace(int64_t rows, int64_t in, int64_t out) {
  const int s = wgrad_splits(rows, in, out);
  return s == 1 ? 256 : (size_t)s * (size_t)out * (size_t)(in + 1) * 4;
}

hipError_t launch_wgrad(int64_t rows, int64_t in, int64_t out, const scape_matrix& dy, const scape_act_view& x,
                        const float* gain, float* dw, float* dbias, bool accumulate, float* ws, hipStream_t s) {
  if (rows < 1 && accumulate) return hipSuccess;
  const int splits = wgrad_splits(rows, in, out);
  WgradArgs a{};
  a.rows = rows;
  a.in = in;
  a.out = out;
  a.nblk = act_blocks(in);
  a.dy = dy.data;
  a.dy_ld = dy.ld;
  a.codes = x.codes;
  a.scales = x.scales;
  a.split_rows = tiles(tiles(rows, splits), kBK) * kBK;
  a.tiles_m = (int)tiles(out, kBM);
  a.tiles_n = (int)tiles(in, kBN);
  if (splits == 1) {
    a.gain = gain;
    a.dw = dw;
    a.db = dbias;
    a.accumulate = accumulate;
  } else {
    a.dw = ws;
    a.db = dbias ? ws + (int64_t)splits * out * in : nullptr;
  }
  const dim3 grid((unsigned)(a.tiles_m * (int64_t)a.tiles_n), (unsigned)splits);
  switch (dy.dtype) {
    case SCAPE_F32: wgrad_kernel<SCAPE_F32><<<grid, 256, 0, s>>>(a); break;
    case SCAPE_BF16: wgrad_kernel<SCAPE_BF16><<<grid, 256, 0, s>>>(a); break;
    case SCAPE_F16: wgrad_kernel<SCAPE_F16><<<grid, 256, 0, s>>>(a); break;
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || splits == 1) return e;
  launch_join(ws, splits, out * in, in, gain, dw, accumulate, s);
  if (dbias) launch_join(a.db, splits, out, out, nullptr, dbias, accumulate, s);
  return hipGetLastError();
}

}  // namespace scape
