// Shared by the activation kernels: element types, the code format of the
// 8-bit checkpoints, and the launch wrappers.
#pragma once

#include "scape_internal.h"

namespace scape {

constexpr int kActBlock = 32;  // columns that share a scale
constexpr int64_t kMaxCols = int64_t(1) << 20;
constexpr int64_t kMaxWeight = int64_t(1) << 37;  // elements of one weight gradient

inline int64_t act_blocks(int64_t cols) { return (cols + kActBlock - 1) / kActBlock; }
inline int64_t act_pitch(int64_t cols) { return act_blocks(cols) * kActBlock; }
inline size_t dtype_bytes(int dt) { return dt == SCAPE_F32 ? 4 : 2; }

hipError_t launch_act_pack(int64_t rows, int64_t cols, const scape_matrix& x, const scape_act_view& out,
                           hipStream_t s);
hipError_t launch_act_unpack(int64_t rows, int64_t cols, const scape_act_view& a, const float* gain,
                             const scape_matrix& out, hipStream_t s);
hipError_t launch_rmsnorm_pack(int64_t rows, int64_t cols, const scape_matrix& x, const scape_matrix& residual,
                               const float* weight, float eps, const scape_matrix& h, const scape_matrix& y,
                               const scape_act_view& xhat, float* rstd, hipStream_t s);
// Rows of dweight partial sums ([parts][cols] fp32) that the backward writes.
int64_t rmsnorm_parts(int64_t rows, int64_t cols);
hipError_t launch_rmsnorm_backward(int64_t rows, int64_t cols, const scape_matrix& dy, const scape_act_view& xhat,
                                   const float* rstd, const float* weight, const scape_matrix& dres,
                                   const scape_matrix& dh, float* dweight, bool accumulate, float* parts,
                                   hipStream_t s);
// Bytes of scratch of a weight gradient: the checkpoint as bf16, dy's terms
// (those of every type's dy where dy.data is null), the splits' partial sums.
size_t wgrad_workspace(int64_t rows, int64_t in, int64_t out, const scape_matrix& dy);
// The number of splits of the rows, and the tile of dw.
int wgrad_splits(int64_t rows, int64_t in, int64_t out, int dtype, int* tile_out, int* tile_in);
hipError_t launch_wgrad(int64_t rows, int64_t in, int64_t out, const scape_matrix& dy, const scape_act_view& x,
                        const float* gain, float* dw, float* dbias, bool accumulate, void* ws, hipStream_t s);

#ifdef __HIPCC__

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

// 16 bytes at an element type's own alignment (gfx950 takes unaligned global
// accesses); STREAM: past the caches' retention.
typedef u32x4 u32x4_any __attribute__((aligned(2)));
template <bool STREAM>
__device__ __forceinline__ void load16(void* dst, const void* p) {
  const u32x4_any* q = static_cast<const u32x4_any*>(p);
  const u32x4 v = STREAM ? __builtin_nontemporal_load(q) : *q;
  __builtin_memcpy(dst, &v, 16);
}

// Matrices of 16-bit types are read with STREAM where a call touches more
// bytes than the caches (256 MB) will hold next to what else runs.  Repeated
// calls, ordinary against streaming loads, bf16: the norm of [16384][4096]
// (320 MiB) 69 us against 64, its backward pass 72 against 67, and the backward
// pass with dres of [16384][2048] (224 MiB) after its forward pass 49 against
// 44; but pack of [16384][4096] (198 MiB) 30 against 35.5 and of [4096][2048]
// 6.0 against 6.8, whose matrices the caches still hold.  fp32 gains nothing
// (norm of [8192][4096] 58 us either way) and loses in the backward pass (73
// against 78).
constexpr int64_t kStreamBytes = int64_t(208) << 20;

// 8 consecutive elements of a row as fp32, and back (rounded to nearest
// even), as one or two 16-byte accesses.
template <int DT>
struct Elem;

template <>
struct Elem<SCAPE_F32> {
  typedef float T;
  template <bool STREAM>
  static __device__ __forceinline__ void load(const void* p, int64_t i, float (&v)[8]) {
    const float* q = static_cast<const float*>(p) + i;
    load16<STREAM>(&v[0], q);
    load16<STREAM>(&v[4], q + 4);
  }
  static __device__ __forceinline__ void store(void* p, int64_t i, const float (&v)[8]) {
    float* q = static_cast<float*>(p) + i;
    __builtin_memcpy(q, &v[0], 16);
    __builtin_memcpy(q + 4, &v[4], 16);
  }
  static __device__ __forceinline__ float get(const void* p, int64_t i) { return static_cast<const float*>(p)[i]; }
  static __device__ __forceinline__ void put(void* p, int64_t i, float v) { static_cast<float*>(p)[i] = v; }
};

template <>
struct Elem<SCAPE_BF16> {
  typedef uint16_t T;
  template <bool STREAM>
  static __device__ __forceinline__ void load(const void* p, int64_t i, float (&v)[8]) {
    uint32_t u[4];
    load16<STREAM>(u, static_cast<const uint16_t*>(p) + i);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = __uint_as_float(u[j] << 16);
      v[2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ void store(void* p, int64_t i, const float (&v)[8]) {
    bf16x2 u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) u[j] = __builtin_convertvector(f32x2{v[2 * j], v[2 * j + 1]}, bf16x2);
    __builtin_memcpy(static_cast<uint16_t*>(p) + i, u, 16);
  }
  static __device__ __forceinline__ float get(const void* p, int64_t i) {
    return __uint_as_float((uint32_t) static_cast<const uint16_t*>(p)[i] << 16);
  }
  static __device__ __forceinline__ void put(void* p, int64_t i, float v) { static_cast<__bf16*>(p)[i] = (__bf16)v; }
};

template <>
struct Elem<SCAPE_F16> {
  typedef uint16_t T;
  template <bool STREAM>
  static __device__ __forceinline__ void load(const void* p, int64_t i, float (&v)[8]) {
    _Float16 u[8];
    load16<STREAM>(u, static_cast<const uint16_t*>(p) + i);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = (float)u[j];
  }
  static __device__ __forceinline__ void store(void* p, int64_t i, const float (&v)[8]) {
    _Float16 u[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) u[j] = (_Float16)v[j];
    __builtin_memcpy(static_cast<uint16_t*>(p) + i, u, 16);
  }
  static __device__ __forceinline__ float get(const void* p, int64_t i) {
    return (float)static_cast<const _Float16*>(p)[i];
  }
  static __device__ __forceinline__ void put(void* p, int64_t i, float v) {
    static_cast<_Float16*>(p)[i] = (_Float16)v;
  }
};

// The same 8 elements as they lie in memory, for loads that are kept under
// way while something else is computed.  With WHOLE a chunk past the row is
// the row's last one.
template <int DT, bool WHOLE, bool STREAM>
struct Raw8 {
  static constexpr int kWords = DT == SCAPE_F32 ? 8 : 4;
  uint32_t u[kWords];
  __device__ __forceinline__ void load(const void* p, int64_t row0, int64_t c, int64_t cols) {
    const char* q = static_cast<const char*>(p) + (row0 + (!WHOLE || c < cols ? c : cols - 8)) * (kWords / 2);
    if (WHOLE || c + 8 <= cols) {
      load16<STREAM>(u, q);
      if (kWords == 8) load16<STREAM>(u + kWords / 2, q + 16);
    } else {
#pragma unroll
      for (int j = 0; j < kWords; ++j) u[j] = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (c + j < cols) {
          if (kWords == 8) {
            __builtin_memcpy(&u[j % kWords], q + 4 * j, 4);
          } else {
            uint16_t h;
            __builtin_memcpy(&h, q + 2 * j, 2);
            u[j / 2] |= (uint32_t)h << (16 * (j & 1));
          }
        }
    }
  }
  __device__ __forceinline__ void unpack(float (&v)[8]) const {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (DT == SCAPE_F32) {
        v[j] = __uint_as_float(u[j % kWords]);
      } else if (DT == SCAPE_BF16) {
        v[j] = __uint_as_float((j & 1) ? u[j / 2] & 0xffff0000u : u[j / 2] << 16);
      } else {
        v[j] = (float)__builtin_bit_cast(_Float16, (uint16_t)(u[j / 2] >> (16 * (j & 1))));
      }
    }
  }
};

// Elements [c, c + 8) of a row of cols elements that starts at row0.  WHOLE:
// cols is a multiple of 8, so a chunk is all there or not at all, and one
// past the row is loaded from the row's end and set to zero: no branch, behind
// which the compiler would wait for every load under way.
template <int DT, bool WHOLE = false, bool STREAM = false>
__device__ __forceinline__ void load8(const void* p, int64_t row0, int64_t c, int64_t cols, float (&v)[8]) {
  if (WHOLE) {
    Elem<DT>::template load<STREAM>(p, row0 + (c < cols ? c : cols - 8), v);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = c < cols ? v[j] : 0.0f;
  } else if (c + 8 <= cols) {
    Elem<DT>::template load<STREAM>(p, row0 + c, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = c + j < cols ? Elem<DT>::get(p, row0 + c + j) : 0.0f;
  }
}
template <int DT, bool WHOLE = false>
__device__ __forceinline__ void store8(void* p, int64_t row0, int64_t c, int64_t cols, const float (&v)[8]) {
  if (WHOLE ? c < cols : c + 8 <= cols) {
    Elem<DT>::store(p, row0 + c, v);
  } else if (!WHOLE) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (c + j < cols) Elem<DT>::put(p, row0 + c + j, v[j]);
  }
}

// Sum over a wave; every lane gets it, the same one.
template <typename V>
__device__ __forceinline__ V wave_sum(V x) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) x += __shfl_xor(x, d, 64);
  return x;
}

// Maximum over the 4 lanes of a quad (one block of 32 columns, 8 a lane).
__device__ __forceinline__ uint32_t quad_max(uint32_t x) {
  uint32_t y = (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0xB1, 0xf, 0xf, true);  // lanes 1 0 3 2
  x = x > y ? x : y;
  y = (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x4E, 0xf, 0xf, true);  // lanes 2 3 0 1
  return x > y ? x : y;
}

// The code of 8 values whose block's largest magnitude has the bit pattern
// amax.  With amax = m * 2^E (1 <= m < 2) the quantum is 2^(E - 6), or
// 2^(E - 5) where m > 127/64.  x * 2^-e + 1.5*2^23 in one fused operation
// rounds x * 2^-e to an integer (half to even: the addend is even), which
// the sum's low byte holds in two's complement.
__device__ __forceinline__ u32x2 act_encode(const float (&v)[8], uint32_t amax, uint32_t* scale) {
  const bool bad = amax >= 0x7f800000u;
  int s = (int)(amax >> 23) - 6 + ((amax & 0x7fffffu) > 0x7e0000u ? 1 : 0);
  s = s < 1 ? 1 : s;
  const float inv = __uint_as_float((uint32_t)(254 - s) << 23);
  uint32_t q[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) q[j] = __float_as_uint(__builtin_fmaf(v[j], inv, 12582912.0f));
  if (s == 249) {  // 64 quanta would read back as an infinity
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int k = (int)(q[j] - 0x4b400000u);
      q[j] = (uint32_t)(k > 63 ? 63 : (k < -63 ? -63 : k));
    }
  }
  u32x2 r;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t lo = __builtin_amdgcn_perm(q[4 * h + 1], q[4 * h], 0x0c0c0400u);
    const uint32_t hi = __builtin_amdgcn_perm(q[4 * h + 3], q[4 * h + 2], 0x04000c0cu);
    r[h] = bad ? 0u : (lo | hi);
  }
  *scale = bad ? 255u : (amax == 0 ? 0u : (uint32_t)s);
  return r;
}

__device__ __forceinline__ uint32_t act_amax8(const float (&v)[8]) {
  uint32_t a = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t b = __float_as_uint(v[j]) & 0x7fffffffu;
    a = a > b ? a : b;
  }
  return a;
}

// 8 codes at one scale byte as fp32 (exact).
__device__ __forceinline__ void act_decode(u32x2 q, uint32_t scale, float (&v)[8]) {
  const float f = __uint_as_float(scale << 23);
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = (float)(int8_t)(q[j >> 2] >> (8 * (j & 3))) * f;
}

#endif  // __HIPCC__

}  // namespace scape
