// 8-bit activation checkpoints (pack, unpack) and the RMS norm with its
// packed output, forward and backward.  All of them stream their matrices
// once and are bound by memory; a lane owns 8 consecutive columns (a quad of
// lanes owns the 32 columns that share a scale, so that the block's maximum
// is two lane exchanges).  A large copy runs at 5.2 TB/s on this card.

#include "activations.h"

#include <type_traits>

namespace scape {
namespace {

// ------------------------------------------------------------ pack, unpack

// [16384][5632] bf16: pack 50 us, unpack 46 us, 280 MB each (5.6-6.1 TB/s).
//
// A quad walks (row, block) pairs in row-major order, nquads at a time;
// drow, dblk: nquads as rows and blocks, so that the walk needs no division.
struct BlockWalk {
  int64_t row;
  int64_t blk;
  __device__ __forceinline__ BlockWalk(int64_t quad, int64_t nblk) : row(quad / nblk), blk(quad - row * nblk) {}
  __device__ __forceinline__ void next(int64_t drow, int64_t dblk, int64_t nblk) {
    row += drow;
    blk += dblk;
    if (blk >= nblk) {
      blk -= nblk;
      ++row;
    }
  }
};

template <int DT, bool STREAM>
__global__ void __launch_bounds__(kThreads)
pack_kernel(const void* __restrict__ x, int64_t ld, int64_t rows, int64_t cols, int64_t nblk, int64_t drow,
            int64_t dblk, int8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  const int64_t tid = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int sub = threadIdx.x & 3;
  for (BlockWalk w(tid >> 2, nblk); w.row < rows; w.next(drow, dblk, nblk)) {
    const int64_t c = w.blk * kActBlock + sub * 8;
    float v[8];
    load8<DT, false, STREAM>(x, w.row * ld, c, cols, v);
    const uint32_t amax = quad_max(act_amax8(v));
    uint32_t s;
    const u32x2 q = act_encode(v, amax, &s);
    const int64_t b = w.row * nblk + w.blk;
    *reinterpret_cast<u32x2*>(codes + b * kActBlock + sub * 8) = q;
    if (sub == 0) scales[b] = (uint8_t)s;
  }
}

template <int DT>
__global__ void __launch_bounds__(kThreads)
unpack_kernel(const int8_t* __restrict__ codes, const uint8_t* __restrict__ scales, const float* __restrict__ gain,
              int64_t rows, int64_t cols, int64_t nblk, int64_t drow, int64_t dblk, void* __restrict__ out,
              int64_t ld) {
  const int64_t tid = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int sub = threadIdx.x & 3;
  for (BlockWalk w(tid >> 2, nblk); w.row < rows; w.next(drow, dblk, nblk)) {
    const int64_t b = w.row * nblk + w.blk;
    const int64_t c = w.blk * kActBlock + sub * 8;
    float v[8];
    act_decode(*reinterpret_cast<const u32x2*>(codes + b * kActBlock + sub * 8), scales[b], v);
    if (gain) {
      float g[8];
      load8<SCAPE_F32>(gain, 0, c, cols, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= g[j];
    } else if (DT == SCAPE_F16) {  // 64 quanta of 2^10 are past the type's range, the packed value was not
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = __builtin_fabsf(v[j]) == 65536.0f ? __builtin_copysignf(65504.0f, v[j]) : v[j];
    }
    store8<DT>(out, w.row * ld, c, cols, v);
  }
}

// Whether a call that touches this many matrices, and codes, streams.
bool streams(int dt, int matrices, const int8_t* codes, int64_t rows, int64_t cols) {
  return dt != SCAPE_F32 && rows * cols > kStreamBytes / (matrices * (int64_t)dtype_bytes(dt) + (codes ? 1 : 0));
}

unsigned walk_grid(int64_t rows, int64_t nblk) {
  const int64_t need = (rows * nblk * 4 + kThreads - 1) / kThreads;
  return (unsigned)(need > 16384 ? 16384 : need);
}

// ---------------------------------------------------------------- RMS norm

// Sum over the T threads (64: a wave; more: the workgroup) that share a row;
// every thread gets it, the same one.
template <int T, typename V>
__device__ __forceinline__ V row_sum(V x, V* lds) {
  x = wave_sum(x);
  if (T == 64) return x;
  __syncthreads();  // the previous row's sum has been read
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
  __syncthreads();
  x = lds[0];
#pragma unroll
  for (int w = 1; w < T / 64; ++w) x += lds[w];
  return x;
}

struct NormArgs {
  int64_t rows, cols, nblk;
  const void* x;
  int64_t x_ld;
  const void* res;
  int64_t res_ld;
  const float* weight;
  float eps;
  void* h;
  int64_t h_ld;
  void* y;
  int64_t y_ld;
  int8_t* codes;
  uint8_t* scales;
  float* rstd;
};

template <int DT, bool WHOLE = false, bool STREAM = false>
__device__ __forceinline__ void load_sum(const NormArgs& a, int64_t row, int64_t c, float (&v)[8]) {
  load8<DT, WHOLE, STREAM>(a.x, row * a.x_ld, c, a.cols, v);
  if (a.res) {
    float r[8];
    load8<DT, WHOLE, STREAM>(a.res, row * a.res_ld, c, a.cols, r);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += r[j];
  }
}

// h, y and the code of one lane's 8 columns (a quad writes one scale).
template <int DT, bool WHOLE = false>
__device__ __forceinline__ void norm_emit(const NormArgs& a, int64_t row, int64_t c, const float (&v)[8], float rs) {
  if (a.h && c < a.cols) store8<DT, WHOLE>(a.h, row * a.h_ld, c, a.cols, v);
  float xh[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) xh[j] = v[j] * rs;
  if (a.y && c < a.cols) {
    float w[8];
    load8<SCAPE_F32, WHOLE>(a.weight, 0, c, a.cols, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = xh[j] * w[j];
    store8<DT, WHOLE>(a.y, row * a.y_ld, c, a.cols, w);
  }
  if (a.codes) {
    const uint32_t amax = quad_max(act_amax8(xh));
    uint32_t s;
    const u32x2 q = act_encode(xh, amax, &s);
    if (c < a.nblk * kActBlock) {
      const int64_t b = row * a.nblk + c / kActBlock;
      *reinterpret_cast<u32x2*>(a.codes + b * kActBlock + (c & 31)) = q;
      if ((threadIdx.x & 3) == 0) a.scales[b] = (uint8_t)s;
    }
  }
}

// The reciprocal RMS.  The sum is binary64: how many threads share a row
// changes its order, and with it the last bits of 53, which reach rstd's 24
// practically never (a change of rstd's last bit could move codes across
// rounding borders).  For one row width the order is fixed.
__device__ __forceinline__ float norm_rstd(double sum, int64_t cols, float eps) {
  return (float)(1.0 / sqrt(sum / (double)cols + (double)eps));
}

// Rows held in registers: T threads a row, C chunks of 8 columns a thread
// (T * C * 8 >= cols).  Bound by memory: [16384][2048] bf16 with residual, h,
// y and codes 57 us, 303 MB (5.3 TB/s); [8192][1280] 24 us (3.9 TB/s).
constexpr int group_of(int T) { return T == 64 ? kThreads : T; }  // threads of a workgroup
template <int DT, int T, int C, bool WHOLE, bool STREAM>
__global__ void __launch_bounds__(group_of(T)) norm_kernel(NormArgs a) {
  __shared__ double lds[group_of(T) / 64];
  constexpr int kRows = group_of(T) / T;
  const int t = threadIdx.x % T;
  for (int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / T; row < a.rows; row += (int64_t)gridDim.x * kRows) {
    float v[C][8];
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < C; ++i) {
      load_sum<DT, WHOLE, STREAM>(a, row, (int64_t)(i * T + t) * 8, v[i]);
    }
#pragma unroll
    for (int i = 0; i < C; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) s = fma((double)v[i][j], (double)v[i][j], s);
    s = row_sum<T>(s, lds);
    const float rs = norm_rstd(s, a.cols, a.eps);
    if (a.rstd && t == 0) a.rstd[row] = rs;
#pragma unroll
    for (int i = 0; i < C; ++i) norm_emit<DT, WHOLE>(a, row, (int64_t)(i * T + t) * 8, v[i], rs);
  }
}

// Rows too long for registers: one workgroup a row, two passes over it.
// h and y may be x's or residual's matrix: nothing is written before every
// thread has summed, and then each thread reads what it overwrites first.
template <int DT>
__global__ void __launch_bounds__(kThreads) norm_long_kernel(NormArgs a) {
  __shared__ double lds[4];
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    double s = 0.0;
    for (int64_t c = (int64_t)threadIdx.x * 8; c < a.cols; c += kThreads * 8) {
      float v[8];
      load_sum<DT>(a, row, c, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) s = fma((double)v[j], (double)v[j], s);
    }
    s = row_sum<kThreads>(s, lds);
    const float rs = norm_rstd(s, a.cols, a.eps);
    if (a.rstd && threadIdx.x == 0) a.rstd[row] = rs;
    // whole quads walk to the end of the last block
    for (int64_t c = (int64_t)threadIdx.x * 8; c < a.nblk * kActBlock; c += kThreads * 8) {
      float v[8];
      load_sum<DT>(a, row, c, v);
      norm_emit<DT>(a, row, c, v, rs);
    }
  }
}

struct NormBackArgs {
  int64_t rows, cols, nblk;
  const void* dy;
  int64_t dy_ld;
  const int8_t* codes;
  const uint8_t* scales;
  const float* rstd;
  const float* weight;
  const void* dres;
  int64_t dres_ld;
  void* dh;
  int64_t dh_ld;
  float* dw;  // [gridDim.x][cols] partial sums, or dweight itself (one block)
  bool accumulate;
};

__device__ __forceinline__ void load_hat(const NormBackArgs& a, int64_t row, int64_t c, float (&v)[8]) {
  if (c < a.nblk * kActBlock) {
    const int64_t b = row * a.nblk + c / kActBlock;
    act_decode(*reinterpret_cast<const u32x2*>(a.codes + b * kActBlock + (c & 31)), a.scales[b], v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 0.0f;
  }
}

// dh of one lane's 8 columns, from g = dy * weight and c = mean(g * xh).
template <int DT>
__device__ __forceinline__ void back_emit(const NormBackArgs& a, int64_t row, int64_t c, const float (&g)[8],
                                          const float (&xh)[8], float mean, float rs) {
  if (c >= a.cols) return;
  float o[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) o[j] = rs * (g[j] - xh[j] * mean);
  if (a.dres) {
    float r[8];
    load8<DT>(a.dres, row * a.dres_ld, c, a.cols, r);
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] += r[j];
  }
  store8<DT>(a.dh, row * a.dh_ld, c, a.cols, o);
}

// One row's inputs of a thread, as they lie in memory.
template <int DT, int C, bool WHOLE, bool STREAM>
struct BackRow {
  Raw8<DT, WHOLE, STREAM> dy[C], dres[C];
  u32x2 codes[C];
  uint32_t scale[C];
  float rstd;
  template <int T>
  __device__ __forceinline__ void load(const NormBackArgs& a, int64_t row, int t) {
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int64_t c = (int64_t)(i * T + t) * 8;
      dy[i].load(a.dy, row * a.dy_ld, c, a.cols);
      // past the row: its last codes, whose products are left out of the sum
      const int64_t at = c < a.nblk * kActBlock ? c : a.nblk * kActBlock - 8;
      codes[i] = *reinterpret_cast<const u32x2*>(a.codes + row * a.nblk * kActBlock + at);
      scale[i] = a.scales[row * a.nblk + at / kActBlock];
      if (a.dres) dres[i].load(a.dres, row * a.dres_ld, c, a.cols);
    }
    rstd = a.rstd[row];
  }
};

// Backward: dh, and the block's part of dweight in registers over its rows
// (no atomics, so the order of the sum is fixed).  Bound by memory:
// [16384][2048] bf16 with dres 44 us, 236 MB (5.4 TB/s); [8192][1280] 18.5 us (4.0
// TB/s).  Two rows at a time took 66 us where one took 47.
//
// T threads a row, C chunks of 8 columns a thread.  With one chunk the next
// row is loaded while this one is computed (more would not fit the
// registers of enough waves).  With dh in dy's or dres's place a row is read
// whole before any of it is written, and no other thread reads it.
template <int DT, int T, int C, bool WHOLE, bool STREAM>
__global__ void __launch_bounds__(group_of(T)) norm_back_kernel(NormBackArgs a) {
  __shared__ float lds[group_of(T) / 64];
  __shared__ float part[T == 64 ? 64 * C * 8 : 1];
  constexpr int kRows = group_of(T) / T;
  constexpr bool kAhead = C == 1;
  const int t = threadIdx.x % T;
  const int64_t step = (int64_t)gridDim.x * kRows;
  float dw[C][8], w[C][8];
#pragma unroll
  for (int i = 0; i < C; ++i) {
    load8<SCAPE_F32, WHOLE>(a.weight, 0, (int64_t)(i * T + t) * 8, a.cols, w[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = 0.0f;
  }
  int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / T;
  BackRow<DT, C, WHOLE, STREAM> next;
  if (kAhead && row < a.rows) next.template load<T>(a, row, t);
  for (; row < a.rows; row += step) {
    if (!kAhead) next.template load<T>(a, row, t);
    const BackRow<DT, C, WHOLE, STREAM> cur = next;
    if (kAhead) next.template load<T>(a, row + step < a.rows ? row + step : row, t);
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < C; ++i) {
      float g[8], xh[8];
      cur.dy[i].unpack(g);
      act_decode(cur.codes[i], cur.scale[i], xh);
      float s = sum;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        dw[i][j] = __builtin_fmaf(g[j], xh[j], dw[i][j]);
        s = __builtin_fmaf(g[j] * w[i][j], xh[j], s);
      }
      sum = (int64_t)(i * T + t) * 8 < a.cols ? s : sum;
    }
    if (a.dh) {
      const float mean = row_sum<T>(sum, lds) / (float)a.cols;
#pragma unroll
      for (int i = 0; i < C; ++i) {
        const int64_t c = (int64_t)(i * T + t) * 8;
        if (c >= a.cols) continue;
        float g[8], xh[8];
        cur.dy[i].unpack(g);
        act_decode(cur.codes[i], cur.scale[i], xh);
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] = cur.rstd * (g[j] * w[i][j] - xh[j] * mean);
        if (a.dres) {
          float r[8];
          cur.dres[i].unpack(r);
#pragma unroll
          for (int j = 0; j < 8; ++j) g[j] += r[j];
        }
        store8<DT, WHOLE>(a.dh, row * a.dh_ld, c, a.cols, g);
      }
    }
  }
  if (!a.dw) return;
  if (T == 64) {  // the four waves' sums, in wave order
    for (int w = 0; w < 4; ++w) {
      if (threadIdx.x / 64 == w) {
#pragma unroll
        for (int i = 0; i < C; ++i)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            float* p = &part[(i * 8 + j) * 64 + t];
            *p = w == 0 ? dw[i][j] : *p + dw[i][j];
            dw[i][j] = *p;
          }
      }
      __syncthreads();
    }
    if (threadIdx.x / 64 != 3) return;
  }
  float* out = a.dw + (int64_t)blockIdx.x * a.cols;
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const int64_t c = (int64_t)(i * T + t) * 8;
    if (c >= a.cols) continue;
    if (a.accumulate) {
      float o[8];
      load8<SCAPE_F32>(out, 0, c, a.cols, o);
#pragma unroll
      for (int j = 0; j < 8; ++j) dw[i][j] += o[j];
    }
    store8<SCAPE_F32>(out, 0, c, a.cols, dw[i]);
  }
}

// Long rows: dweight first (dh may overwrite dy), then dh in two passes a row.
template <int DT>
__global__ void __launch_bounds__(kThreads) norm_back_long_dw_kernel(NormBackArgs a) {
  const int64_t c = ((int64_t)blockIdx.y * kThreads + threadIdx.x) * 8;
  if (c >= a.cols) return;
  float dw[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    float g[8], xh[8];
    load8<DT>(a.dy, row * a.dy_ld, c, a.cols, g);
    load_hat(a, row, c, xh);
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[j] = __builtin_fmaf(g[j], xh[j], dw[j]);
  }
  float* out = a.dw + (int64_t)blockIdx.x * a.cols;
  if (a.accumulate) {
    float o[8];
    load8<SCAPE_F32>(out, 0, c, a.cols, o);
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[j] += o[j];
  }
  store8<SCAPE_F32>(out, 0, c, a.cols, dw);
}

template <int DT>
__global__ void __launch_bounds__(kThreads) norm_back_long_kernel(NormBackArgs a) {
  __shared__ float lds[4];
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    float sum = 0.0f;
    for (int64_t c = (int64_t)threadIdx.x * 8; c < a.cols; c += kThreads * 8) {
      float g[8], xh[8], w[8];
      load8<DT>(a.dy, row * a.dy_ld, c, a.cols, g);
      load_hat(a, row, c, xh);
      load8<SCAPE_F32>(a.weight, 0, c, a.cols, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) sum = __builtin_fmaf(g[j] * w[j], xh[j], sum);
    }
    const float mean = row_sum<kThreads>(sum, lds) / (float)a.cols;
    const float rs = a.rstd[row];
    for (int64_t c = (int64_t)threadIdx.x * 8; c < a.cols; c += kThreads * 8) {
      float g[8], xh[8], w[8];
      load8<DT>(a.dy, row * a.dy_ld, c, a.cols, g);
      load_hat(a, row, c, xh);
      load8<SCAPE_F32>(a.weight, 0, c, a.cols, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) g[j] *= w[j];
      back_emit<DT>(a, row, c, g, xh, mean, rs);
    }
  }
}

// out[c] (+)= the sum of parts[0 .. n)[c]: 64 groups of parts a column, each
// in order, then the groups in order.  1024 parts of 2048 columns: 5 us (4
// groups a column: 38 us).
constexpr int kSumCols = 16, kSumGroups = 64;
__global__ void __launch_bounds__(kSumCols * kSumGroups)
sum_parts_kernel(const float* __restrict__ parts, int64_t n, int64_t cols, float* __restrict__ out, bool accumulate) {
  __shared__ float lds[kSumGroups][kSumCols];
  const int lane = threadIdx.x % kSumCols, grp = threadIdx.x / kSumCols;
  const int64_t c = (int64_t)blockIdx.x * kSumCols + lane;
  float s = 0.0f;
  if (c < cols) {
#pragma unroll 8
    for (int64_t p = grp; p < n; p += kSumGroups) s += parts[p * cols + c];
  }
  lds[grp][lane] = s;
  __syncthreads();
  if (grp == 0 && c < cols) {
    s = lds[0][lane];
#pragma unroll
    for (int g = 1; g < kSumGroups; ++g) s += lds[g][lane];
    out[c] = accumulate ? out[c] + s : s;
  }
}

__global__ void __launch_bounds__(kThreads) zero_f32_kernel(float* p, int64_t n) {
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (i < n) p[i] = 0.0f;
}

// Threads that share a row, and chunks of 8 columns a thread: a wave up to
// 512 columns, workgroups of 128, 192 and 256 threads up to 2048 (one chunk
// each; 256 threads for a row of 1280 columns took a tenth longer than 192),
// then 256 and 1024 threads with one or two; longer rows are read twice.
constexpr int64_t kWaveCols = 64 * 8, kGroupCols = 256 * 8 * 2, kWideCols = 1024 * 8 * 2;
constexpr int64_t kBackBlocks = 1024;

unsigned cap_grid(int64_t need, int64_t most) { return (unsigned)(need < most ? need : most); }

template <typename F>
void for_row_shape(int64_t cols, F&& f) {
  if (cols <= 64 * 8) f(std::integral_constant<int, 64>{}, std::integral_constant<int, 1>{});
  else if (cols <= 128 * 8) f(std::integral_constant<int, 128>{}, std::integral_constant<int, 1>{});
  else if (cols <= 192 * 8) f(std::integral_constant<int, 192>{}, std::integral_constant<int, 1>{});
  else if (cols <= 256 * 8) f(std::integral_constant<int, 256>{}, std::integral_constant<int, 1>{});
  else if (cols <= 256 * 16) f(std::integral_constant<int, 256>{}, std::integral_constant<int, 2>{});
  else if (cols <= 1024 * 8) f(std::integral_constant<int, 1024>{}, std::integral_constant<int, 1>{});
  else f(std::integral_constant<int, 1024>{}, std::integral_constant<int, 2>{});
}

template <int DT>
void norm_launch(const NormArgs& a, hipStream_t s) {
  if (a.cols > kWideCols) {
    norm_long_kernel<DT><<<cap_grid(a.rows, 65536), kThreads, 0, s>>>(a);
    return;
  }
  for_row_shape(a.cols, [&](auto t, auto c) {
    constexpr int T = decltype(t)::value, C = decltype(c)::value, per = group_of(T) / T;
    const unsigned grid = cap_grid((a.rows + per - 1) / per, 65536);
    if (a.cols % 8 != 0)
      norm_kernel<DT, T, C, false, false><<<grid, group_of(T), 0, s>>>(a);
    else if (streams(DT, 1 + (a.res != nullptr) + (a.h != nullptr) + (a.y != nullptr), a.codes, a.rows, a.cols))
      norm_kernel<DT, T, C, true, DT != SCAPE_F32><<<grid, group_of(T), 0, s>>>(a);
    else
      norm_kernel<DT, T, C, true, false><<<grid, group_of(T), 0, s>>>(a);
  });
}

template <int DT>
void back_launch(const NormBackArgs& a, unsigned parts, hipStream_t s) {
  if (a.cols > kWideCols) {
    if (a.dw)
      norm_back_long_dw_kernel<DT><<<dim3(parts, (unsigned)((a.cols + 2047) / 2048)), kThreads, 0, s>>>(a);
    if (a.dh) norm_back_long_kernel<DT><<<cap_grid(a.rows, 65536), kThreads, 0, s>>>(a);
    return;
  }
  for_row_shape(a.cols, [&](auto t, auto c) {
    constexpr int T = decltype(t)::value, C = decltype(c)::value;
    if (a.cols % 8 != 0)
      norm_back_kernel<DT, T, C, false, false><<<parts, group_of(T), 0, s>>>(a);
    else if (streams(DT, 1 + (a.dres != nullptr) + (a.dh != nullptr), a.codes, a.rows, a.cols))
      norm_back_kernel<DT, T, C, true, DT != SCAPE_F32><<<parts, group_of(T), 0, s>>>(a);
    else
      norm_back_kernel<DT, T, C, true, false><<<parts, group_of(T), 0, s>>>(a);
  });
}

}  // namespace

hipError_t launch_act_pack(int64_t rows, int64_t cols, const scape_matrix& x, const scape_act_view& out,
                           hipStream_t s) {
  if (rows < 1) return hipSuccess;
  const int64_t nblk = act_blocks(cols);
  const unsigned grid = walk_grid(rows, nblk);
  const int64_t quads = (int64_t)grid * kThreads / 4;
  const int64_t drow = quads / nblk, dblk = quads % nblk;
  const bool stream = streams(x.dtype, 1, out.codes, rows, cols);
#define PACK(DT) \
  case DT: \
    if (stream) \
      pack_kernel<DT, DT != SCAPE_F32><<<grid, kThreads, 0, s>>>(x.data, x.ld, rows, cols, nblk, drow, dblk, out.codes, out.scales); \
    else \
      pack_kernel<DT, false><<<grid, kThreads, 0, s>>>(x.data, x.ld, rows, cols, nblk, drow, dblk, out.codes, out.scales); \
    break;
  switch (x.dtype) { PACK(SCAPE_F32) PACK(SCAPE_BF16) PACK(SCAPE_F16) }
#undef PACK
  return hipGetLastError();
}

hipError_t launch_act_unpack(int64_t rows, int64_t cols, const scape_act_view& a, const float* gain,
                             const scape_matrix& out, hipStream_t s) {
  if (rows < 1) return hipSuccess;
  const int64_t nblk = act_blocks(cols);
  const unsigned grid = walk_grid(rows, nblk);
  const int64_t quads = (int64_t)grid * kThreads / 4;
  const int64_t drow = quads / nblk, dblk = quads % nblk;
#define UNPACK(DT) \
  case DT: unpack_kernel<DT><<<grid, kThreads, 0, s>>>(a.codes, a.scales, gain, rows, cols, nblk, drow, dblk, out.data, out.ld); break;
  switch (out.dtype) { UNPACK(SCAPE_F32) UNPACK(SCAPE_BF16) UNPACK(SCAPE_F16) }
#undef UNPACK
  return hipGetLastError();
}

hipError_t launch_rmsnorm_pack(int64_t rows, int64_t cols, const scape_matrix& x, const scape_matrix& residual,
                               const float* weight, float eps, const scape_matrix& h, const scape_matrix& y,
                               const scape_act_view& xhat, float* rstd, hipStream_t s) {
  if (rows < 1) return hipSuccess;
  NormArgs a{rows, cols, act_blocks(cols), x.data, x.ld, residual.data, residual.ld, weight, eps,
             h.data, h.ld, y.data, y.ld, xhat.codes, xhat.scales, rstd};
  switch (x.dtype) {
    case SCAPE_F32: norm_launch<SCAPE_F32>(a, s); break;
    case SCAPE_BF16: norm_launch<SCAPE_BF16>(a, s); break;
    case SCAPE_F16: norm_launch<SCAPE_F16>(a, s); break;
  }
  return hipGetLastError();
}

int64_t rmsnorm_parts(int64_t rows, int64_t cols) {
  const int64_t per = cols <= kWaveCols ? 4 : 1;  // rows a workgroup works on at a time
  const int64_t need = (rows + per - 1) / per;
  const int64_t most = cols <= kGroupCols ? kBackBlocks : kBackBlocks / 4;
  return need < 1 ? 1 : (need < most ? need : most);
}

hipError_t launch_rmsnorm_backward(int64_t rows, int64_t cols, const scape_matrix& dy, const scape_act_view& xhat,
                                   const float* rstd, const float* weight, const scape_matrix& dres,
                                   const scape_matrix& dh, float* dweight, bool accumulate, float* parts,
                                   hipStream_t s) {
  if (rows < 1) {
    if (dweight && !accumulate)
      zero_f32_kernel<<<(unsigned)((cols + kThreads - 1) / kThreads), kThreads, 0, s>>>(dweight, cols);
    return hipGetLastError();
  }
  const int64_t n = rmsnorm_parts(rows, cols);
  NormBackArgs a{rows, cols, act_blocks(cols), dy.data, dy.ld, xhat.codes, xhat.scales, rstd, weight,
                 dres.data, dres.ld, dh.data, dh.ld, nullptr, false};
  if (dweight) {
    a.dw = n == 1 ? dweight : parts;
    a.accumulate = n == 1 && accumulate;
  }
  switch (dy.dtype) {
    case SCAPE_F32: back_launch<SCAPE_F32>(a, (unsigned)n, s); break;
    case SCAPE_BF16: back_launch<SCAPE_BF16>(a, (unsigned)n, s); break;
    case SCAPE_F16: back_launch<SCAPE_F16>(a, (unsigned)n, s); break;
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !dweight || n == 1) return e;
  sum_parts_kernel<<<(unsigned)((cols + kSumCols - 1) / kSumCols), kSumCols * kSumGroups, 0, s>>>(parts, n, cols, dweight, accumulate);
  return hipGetLastError();
}

}  // namespace scape
