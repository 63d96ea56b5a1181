// Weight gradient of a linear layer from the 8-bit checkpoint of its input:
// dw[o][i] = gain[i] * sum_t dy[t][o] * x[t][i], on the matrix cores in bf16
// with fp32 sums.  A checkpoint's values have at most 8 significant bits and
// a power of two as their scale, so they are exact in bf16; a bf16 dy is
// taken as it is, and an fp32 one is split into 3 bf16 terms that add up to
// the value.  So every product is exact and only the sums round.  The terms are
// summed one after the other over all rows of a split, the smallest first: in
// the other order each of their sums' roundings is one at the size of the whole
// sum, and what lies below its last place is lost (999 rows, 777 -> 1531: off
// by 0.9e-7 of the norm, the bias by 0.6e-7; largest first 2.4e-7 and 2.9e-7).
//
// An fp16 dy is multiplied in fp16 (two bf16 terms took twice the time).  Each
// 32 columns of the checkpoint are then scaled by a power of two that brings
// their largest scale to 2^8 (127 * 2^8 is in range), and their sums are scaled
// back: values are exact in fp16 down to 2^-32 times that scale, and smaller
// ones round to multiples of 2^-24 before scaling back, by at most 2^-38 of the
// largest value of those columns.
//
// Launches: for fp16 the largest scales; prepare (the checkpoint in 16 bits,
// and dy's terms where dy cannot be read as it lies); the product over row
// splits; with more than one split the join of their partial sums.

#include "activations.h"

namespace scape {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) char lds_char;

constexpr int kBK = 32;     // rows a stage
constexpr int kWaves = 4;
constexpr int terms_of(int dt) { return dt == SCAPE_F32 ? 3 : 1; }

int64_t ceil_div(int64_t x, int64_t t) { return (x + t - 1) / t; }

// ------------------------------------------------------------------ prepare

constexpr int kTopExp = 8;  // fp16: the largest scale of 32 columns becomes 2^kTopExp

// The scales [rows][nblk] as a matrix of rows of `flat` columns: rows of fewer
// than 64 scales are joined in whole numbers up to 64, so that narrow matrices
// occupy the threads, too.  pitch: flat up to whole slabs of 64.
struct Flat {
  int64_t nblk, flat, pitch;
  explicit Flat(int64_t n) : nblk(n), flat(n < 64 ? 64 / n * n : n), pitch((flat + 63) / 64 * 64) {}
  int64_t rows(int64_t scales) const { return (scales + flat - 1) / flat; }
};

// parts[blockIdx.y][flat column] = the largest finite scale byte of its block of
// columns over one in gridDim.y of the groups of 64 flat rows.  A thread takes
// 16 columns of a row.  [8192][1024]: 4.6 us, a launch and its latency (0.3 MB).
constexpr int kMaxParts = 64;
__global__ void __launch_bounds__(kThreads)
scale_max_kernel(const uint8_t* __restrict__ scales, int64_t n, int64_t nblk, int64_t flat, int64_t pitch,
                 uint8_t* __restrict__ parts) {
  static_assert(kThreads == 256, "64 rows of 4 threads");
  __shared__ __attribute__((aligned(16))) uint8_t rows[64][64], quarters[4][64];
  const int64_t col = (int64_t)blockIdx.x * 64 + (threadIdx.x & 3) * 16;
  uint8_t m[16] = {};
  for (int64_t r = (int64_t)blockIdx.y * 64 + (threadIdx.x >> 2); r * flat < n; r += (int64_t)gridDim.y * 64) {
    const int64_t i = r * flat + col, left = flat - col < n - i ? flat - col : n - i;
    uint8_t b[16];
    if (left >= 16) {
      __builtin_memcpy(b, scales + i, 16);
    } else {
#pragma unroll
      for (int j = 0; j < 16; ++j) b[j] = j < left ? scales[i + j] : 0;
    }
#pragma unroll
    for (int j = 0; j < 16; ++j) m[j] = b[j] != 255 && b[j] > m[j] ? b[j] : m[j];
  }
  __builtin_memcpy(&rows[threadIdx.x >> 2][(threadIdx.x & 3) * 16], m, 16);
  __syncthreads();
  const int c = threadIdx.x & 63, g = threadIdx.x >> 6;
  uint8_t t = 0;
#pragma unroll
  for (int j = 0; j < 16; ++j) t = rows[g * 16 + j][c] > t ? rows[g * 16 + j][c] : t;
  quarters[g][c] = t;
  __syncthreads();
  if (g == 0) {
    for (int j = 1; j < 4; ++j) t = quarters[j][c] > t ? quarters[j][c] : t;
    // joined rows (flat <= 64): the columns nblk apart, 2, 4, 8 .. of them
    for (int d = (int)nblk; d < (int)flat; d *= 2) {
      const int o = __shfl((int)t, c + d < (int)flat ? c + d : c + d - (int)flat, 64);
      t = o > t ? (uint8_t)o : t;
    }
    parts[blockIdx.y * pitch + (int64_t)blockIdx.x * 64 + c] = t;
  }
}

struct PrepArgs {
  int64_t rows, rows_pad, nblk, out, out_pad;
  const int8_t* codes;
  const uint8_t* scales;
  uint16_t* x;  // [rows_pad][nblk * 32] bf16 (fp16 for an fp16 dy), zero past rows
  const uint8_t* max_parts;  // fp16: partial maxima [n_parts][pitch] of the scales
  int n_parts;
  int64_t flat, pitch;  // fp16: those of Flat
  float* back;          // fp16: [nblk], receives what each block's sums are multiplied by
  const void* dy;
  int64_t dy_ld;
  // dy's terms, smallest first, [terms][t_rows][out_pad] in 16 bits of rows t_first .., zero past
  // dy's rows and columns: all rows, or the last, partial stage of a dy that
  // is read as it lies (none: t_rows = 0)
  uint16_t* terms;
  int64_t t_first, t_rows;
  unsigned x_blocks;
};

// Splits v into its leading 8 significant bits (the upper half of its
// pattern) and the rest.  An infinity leaves nothing; a NaN stays one in the
// rest if its payload is cut off.
__device__ __forceinline__ uint32_t cut_term(float& v) {
  const uint32_t u = __float_as_uint(v) & 0xffff0000u;
  const float h = __uint_as_float(u);
  v = __builtin_isinf(v) ? 0.0f : v - h;
  return u;
}
// The upper halves of two words, a's in the lower half.
__device__ __forceinline__ uint32_t upper_halves(uint32_t a, uint32_t b) {
  return __builtin_amdgcn_perm(b, a, 0x07060302u);
}

// fp16: a workgroup takes one in (x_blocks / slabs) of the flat rows in a slab of
// 64 flat columns, 4 threads a column, so that a thread's shift of the scale
// byte is found once.  [8192][1024]: 9.3 us (26 MB, 2.8 TB/s; 8.1 with one shift
// for the whole checkpoint).
__device__ __forceinline__ void prepare_x_f16(const PrepArgs& a) {
  __shared__ __attribute__((aligned(16))) uint8_t parts[kMaxParts][64], quarters[4][64];
  const int64_t slabs = a.pitch / 64, slab = blockIdx.x % slabs;
  const int64_t first = blockIdx.x / slabs, step = a.x_blocks / slabs;
  u32x4 p = {0, 0, 0, 0};
  if ((int)(threadIdx.x >> 2) < a.n_parts)
    __builtin_memcpy(&p, __builtin_assume_aligned(a.max_parts + (threadIdx.x >> 2) * a.pitch + slab * 64 + (threadIdx.x & 3) * 16, 16), 16);
  __builtin_memcpy(&parts[threadIdx.x >> 2][(threadIdx.x & 3) * 16], &p, 16);
  __syncthreads();
  const int c = threadIdx.x & 63, g = threadIdx.x >> 6;
  uint8_t t = 0;
#pragma unroll
  for (int j = 0; j < 16; ++j) t = parts[g * 16 + j][c] > t ? parts[g * 16 + j][c] : t;
  quarters[g][c] = t;
  __syncthreads();
  const int64_t col = slab * 64 + (threadIdx.x >> 2);
  if (col >= a.flat) return;
  int m = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) m = quarters[j][col & 63] > m ? quarters[j][col & 63] : m;
  const int shift = 127 + kTopExp - m;
  if (first == 0 && col < a.nblk && (threadIdx.x & 3) == 0) a.back[col] = ldexpf(1.0f, -shift);
  const int64_t full = a.rows * a.nblk, n = a.rows_pad * a.nblk;  // blocks
  for (int64_t b = first * a.flat + col; b < n; b += step * a.flat) {
    u32x4 o = {0, 0, 0, 0};
    const int64_t i = b * 4 + (threadIdx.x & 3);
    if (b < full) {
      float v[8];
      const uint32_t s = a.scales[b];
      const int e = (int)s + shift;  // under 1: less than any fp16 number
      act_decode(reinterpret_cast<const u32x2*>(a.codes)[i], s == 0 || s == 255 ? s : (e < 1 ? 0u : (uint32_t)e), v);
#pragma unroll
      for (int h = 0; h < 4; ++h)
        o[h] = __builtin_bit_cast(uint32_t, f16x2{(_Float16)v[2 * h], (_Float16)v[2 * h + 1]});
    }
    reinterpret_cast<u32x4*>(a.x)[i] = o;
  }
}

// Bound by memory: [16384][2048] codes to bf16 18 us (102 MB, 5.6 TB/s).
template <int DT>
__global__ void __launch_bounds__(kThreads) wgrad_prepare_kernel(PrepArgs a) {
  if (blockIdx.x < a.x_blocks) {
    if constexpr (DT == SCAPE_F16) {
      prepare_x_f16(a);
    } else {
      const int64_t n = a.rows_pad * a.nblk * 4, step = (int64_t)a.x_blocks * kThreads;
      const int64_t full = a.rows * a.nblk * 4;
      for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n; i += step) {
        u32x4 p = {0, 0, 0, 0};
        if (i < full) {
          float v[8];
          act_decode(reinterpret_cast<const u32x2*>(a.codes)[i], a.scales[i >> 2], v);
#pragma unroll
          for (int h = 0; h < 4; ++h) p[h] = upper_halves(__float_as_uint(v[2 * h]), __float_as_uint(v[2 * h + 1]));
        }
        reinterpret_cast<u32x4*>(a.x)[i] = p;
      }
    }
    return;
  }
  const int64_t chunks = a.out_pad / 8, n = a.t_rows * chunks;
  const int64_t step = (int64_t)(gridDim.x - a.x_blocks) * kThreads;
  for (int64_t i = (int64_t)(blockIdx.x - a.x_blocks) * kThreads + threadIdx.x; i < n; i += step) {
    const int64_t r = i / chunks, c = (i - r * chunks) * 8, t = a.t_first + r;
    float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (t < a.rows) load8<DT>(a.dy, t * a.dy_ld, c, a.out, v);
#pragma unroll
    for (int k = 0; k < terms_of(DT); ++k) {
      u32x4 p;
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        if (DT == SCAPE_F16) {
          p[h] = __builtin_bit_cast(uint32_t, f16x2{(_Float16)v[2 * h], (_Float16)v[2 * h + 1]});
        } else {
          const uint32_t lo = cut_term(v[2 * h]), hi = cut_term(v[2 * h + 1]);
          p[h] = upper_halves(lo, hi);
        }
      }
      *reinterpret_cast<u32x4*>(a.terms + ((terms_of(DT) - 1 - k) * a.t_rows + r) * a.out_pad + c) = p;
    }
  }
}

// ------------------------------------------------------------------ product

struct WgradArgs {
  int64_t rows, in, out;
  const char* a;         // dy or its terms: 16-bit rows a_step bytes apart
  int64_t a_step;
  int64_t a_plane;       // bytes between terms
  int64_t a_cols;        // columns that may be read (a multiple of 8)
  int terms;
  const char* tail;      // the last, partial stage of a's rows, zero filled; null: none
  int64_t tail_step;
  const char* b;         // the checkpoint in 16 bits, zero past rows to a whole stage
  int64_t b_step, b_cols;
  const float* back;     // fp16: the sums' scale for each 32 columns.  It and gain
  const float* gain;     // are applied here only when there is one split
  float* dw;             // [splits][out][in], or dw itself (one split)
  float* db;             // [splits][out], or dbias itself; null: none
  bool accumulate;       // one split
  int64_t split_rows;    // rows a split sums (a multiple of kBK)
  int tiles_n, tiles;    // tiles along in, and in all
};

// A barrier that orders LDS only: loads from memory stay in flight.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// 16 bytes a lane from memory to LDS without a register: lane l's go to
// lds + 16 * l.  The address is base (the same for the wave) + off bytes.
// The compiler does not count it: wait for it with wait_vm.  m0 is the compiler's
// own and declared as overwritten, so that it keeps no value there across this;
// its warning that m0 is not restored says what is meant.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void load_to_lds(const void* base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
               :
               : "s"(lds), "v"(off), "s"(base)
               : "memory", "m0");
}
#pragma clang diagnostic pop
// Waits until at most N of the wave's loads from memory are under way.
template <int N>
__device__ __forceinline__ void wait_vm() {
  asm volatile("s_waitcnt vmcnt(%0)" : : "n"(N) : "memory");
}

// A stage of an operand lies in LDS as in memory, [row][W columns] of 16 bits.
// The 4 rows that a transposed read takes have to fall on different banks
// (256 bytes hold all 64), so the 64-byte pieces of a row are permuted by
// bits of the row number.
template <int W>
__device__ __forceinline__ int piece_at(int piece, int row) {
  return W == 192 ? piece ^ ((row >> 1) & 1) : piece ^ (row & 3);
}

// 16384 rows, 2048 -> 5632, bf16: 315-400 us for 378 GFLOP (0.95-1.2 PFLOP/s;
// the library's product of the same bf16 operands takes 412 us), 8192 rows,
// 4096 -> 4096: 210-230 us (1.2-1.3).  With the loads left out the first takes
// 295, with everything but the loads left out 260: it is held by the products
// (whose clock falls with the data's power: all-zero inputs take 278) and by
// the latency of loads that miss the XCD's L2.  Two waves a SIMD instead of
// one, blocks of tiles for each XCD, and loads issued earlier or more evenly
// took the same time or more.
//
// One workgroup sums a BM x BN tile of dw over the rows of one split.  Both
// operands have the summed index (the rows) as their slow axis and come to
// LDS as they lie, without a register; the transposed LDS read gives the
// fragments.  A ring of kRing stages keeps kRing - 2 of them under way.
template <bool F16, int BM, int BN, int WM, int WN, int kRing>
__global__ void __launch_bounds__(kWaves * 64) wgrad_kernel(WgradArgs a) {
  constexpr int FM = BM / WM / 32, FN = BN / WN / 32;
  constexpr int kBytesA = BM * kBK * 2, kStage = (BM + BN) * kBK * 2;
  constexpr int LA = kBytesA / 1024 / kWaves, LB = BN * kBK * 2 / 1024 / kWaves;  // 1 KB loads a wave and stage
  constexpr int kLoads = LA + LB;
  static_assert(WM * WN == kWaves && FM * WM * 32 == BM && FN * WN * 32 == BN, "tile shape");
  static_assert(LA * kWaves * 1024 == kBytesA && LB * kWaves * 1024 == BN * kBK * 2, "whole loads");
  static_assert(kRing * kStage <= 160 * 1024 && kRing >= 3, "ring");
  __shared__ __attribute__((aligned(1024))) char lds[kRing * kStage];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // Workgroups are dealt to the 8 XCDs in turn: give each XCD consecutive
  // tiles, which share dy's columns and the checkpoint's in its L2.
  const int total = gridDim.x, q8 = total >> 3, r8 = total & 7;
  const int xcd = blockIdx.x & 7;
  const int id = xcd * q8 + (xcd < r8 ? xcd : r8) + (blockIdx.x >> 3);
  const int split = id / a.tiles, tile = id - split * a.tiles;
  const int64_t m0 = (int64_t)(tile / a.tiles_n) * BM, n0 = (int64_t)(tile % a.tiles_n) * BN;
  const int64_t t_begin = (int64_t)split * a.split_rows;
  const int64_t t_end = t_begin + a.split_rows < a.rows ? t_begin + a.split_rows : a.rows;
  const int stages = t_begin < t_end ? (int)((t_end - t_begin + kBK - 1) / kBK) : 0;  // of one term
  const int all = stages * a.terms;

  // ---- loads: this lane's place in each 1 KB of this wave.  Columns past
  // the edge are read from inside the row, multiplied and never stored.
  uint32_t a_off[LA], t_off[LA], b_off[LB];
#pragma unroll
  for (int i = 0; i < LA; ++i) {
    const int at = (wave * LA + i) * 64 + lane, row = at / (BM / 8), place = at % (BM / 8);
    int64_t c = m0 + (piece_at<BM>(place >> 2, row) * 4 + (place & 3)) * 8;
    if (c > a.a_cols - 8) c = a.a_cols - 8;
    a_off[i] = (uint32_t)(row * a.a_step + c * 2);
    t_off[i] = (uint32_t)(row * a.tail_step + c * 2);
  }
#pragma unroll
  for (int i = 0; i < LB; ++i) {
    const int at = (wave * LB + i) * 64 + lane, row = at / (BN / 8), place = at % (BN / 8);
    int64_t c = n0 + (piece_at<BN>(place >> 2, row) * 4 + (place & 3)) * 8;
    if (c > a.b_cols - 8) c = a.b_cols - 8;
    b_off[i] = (uint32_t)(row * a.b_step + c * 2);
  }
  const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_char*)lds;
  const uint32_t lds_a = __builtin_amdgcn_readfirstlane(lds0 + wave * LA * 1024);
  const uint32_t lds_b = __builtin_amdgcn_readfirstlane(lds0 + kBytesA + wave * LB * 1024);

  // the next stage to load; past the last one it is loaded again, into slots
  // that nobody reads, so that every stage has the same loads under way
  const char* a_next = a.a + t_begin * a.a_step;
  const char* b_next = a.b + t_begin * a.b_step;
  int next = 0;
  uint32_t next_at = 0;  // of its slot
  int left = stages;     // of its term
  const bool has_tail = a.tail && t_end == a.rows;
  auto load_a = [&](int i) {
    const bool t = has_tail && left == 1;
    load_to_lds(t ? a.tail : a_next, t ? t_off[i] : a_off[i], lds_a + next_at + i * 1024);
  };
  auto load_b = [&](int i) { load_to_lds(b_next, b_off[i], lds_b + next_at + i * 1024); };
  auto advance = [&]() {
    if (++next < all) {
      a_next += kBK * a.a_step;
      b_next += kBK * a.b_step;
      if (--left == 0) {  // the next term, from the split's first row
        left = stages;
        a_next += a.a_plane - stages * (kBK * a.a_step);
        b_next -= stages * (kBK * a.b_step);
      }
    }
    next_at = next_at + kStage == kRing * kStage ? 0 : next_at + kStage;
  };

  // ---- fragments.  A transposed read takes, in each 16 lanes, 4 rows of 16
  // columns (lane l: row l/4, columns 4 (l%4) ..) and gives lane l column l.
  const int wm = wave / WN * (FM * 32), wn = wave % WN * (FN * 32);
  const int tr = (lane & 15) >> 2;
  int a_at[FM], b_at[FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
    a_at[i] = ((lane >> 5) * 8 + tr) * (BM * 2) + (piece_at<BM>((wm >> 5) + i, tr) << 6) + ((lane >> 4) & 1) * 32 +
              (lane & 3) * 8;
#pragma unroll
  for (int j = 0; j < FN; ++j)
    b_at[j] = kBytesA + ((lane >> 5) * 8 + tr) * (BN * 2) + (piece_at<BN>((wn >> 5) + j, tr) << 6) +
              ((lane >> 4) & 1) * 32 + (lane & 3) * 8;

  f32x16 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = (f32x16)(0.0f);
  const bool bias = a.db && n0 == 0 && wn == 0;
  float bsum[FM] = {};

  union Frag {
    s16x4 h[2];
    bf16x8 v;
    f16x8 f;
    bf16x2 b2[4];
    f16x2 f2[4];
  };
  Frag av[2][FM], bv[2][FN];
  auto read4 = [&](int at) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(lds + at));
  };
  // The fragments' reads in the order in which the products need them: the
  // first of A, all of B, the others of A; two halves each.
  constexpr int kReads = 2 * (FM + FN), kMul = FM * FN;
  auto read_piece = [&](int kk, int at, int r) {
    const int f = r >> 1, h = r & 1;
    if (f >= 1 && f <= FN) {
      bv[kk][f - 1].h[h] = read4(at + b_at[f - 1] + (kk * 16 + h * 4) * (BN * 2));
    } else {
      const int i = f == 0 ? 0 : f - FN;
      av[kk][i].h[h] = read4(at + a_at[i] + (kk * 16 + h * 4) * (BM * 2));
    }
  };
  // The products of fragments kk, with the reads of the next fragments
  // between the first half of them and the loads between the second: a wave
  // has its SIMD to itself, and whatever it issues in one piece leaves the
  // matrix unit idle.
  auto block = [&](int kk, int read_kk, int read_at, bool loads_a) {
    constexpr int kHalf = kMul / 2;
    constexpr int kPer = (kReads + kHalf - 1) / kHalf;
    const int n_loads = loads_a ? LA : LB;
    const int per_load = (n_loads + kHalf - 1) / kHalf;
#pragma unroll
    for (int q = 0; q < kMul; ++q) {
      const int i = q / FN, j = q % FN;
      if (F16) {
        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(av[kk][i].f, bv[kk][j].f, acc[i][j], 0, 0, 0);
      } else {
        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(av[kk][i].v, bv[kk][j].v, acc[i][j], 0, 0, 0);
      }
#pragma unroll
      for (int r = 0; r < kPer; ++r)
        if (q < kHalf && q * kPer + r < kReads) read_piece(read_kk, read_at, q * kPer + r);
#pragma unroll
      for (int r = 0; r < per_load; ++r)
        if (q >= kHalf && (q - kHalf) * per_load + r < n_loads) {
          if (loads_a) {
            load_a((q - kHalf) * per_load + r);
          } else {
            load_b((q - kHalf) * per_load + r);
          }
        }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  auto add_bias = [&](int kk) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        // one fused sum of two elements times one and the sum so far
        if (F16) {
          bsum[i] = __builtin_amdgcn_fdot2(av[kk][i].f2[h], f16x2{(_Float16)1.0f, (_Float16)1.0f}, bsum[i], false);
        } else {
          bsum[i] = __builtin_amdgcn_fdot2_f32_bf16(av[kk][i].b2[h], bf16x2{(__bf16)1.0f, (__bf16)1.0f}, bsum[i], false);
        }
      }
  };

  // ---- the pipeline.  At the start of stage s stage s + 1 has arrived for
  // every wave, so that its first fragments can be read while s is
  // multiplied; stage s + kRing - 1 is loaded into the slot of s - 1, which
  // every wave has read.
  if (all > 0) {
#pragma unroll
    for (int p = 0; p < kRing - 1; ++p) {
#pragma unroll
      for (int i = 0; i < LA; ++i) load_a(i);
#pragma unroll
      for (int i = 0; i < LB; ++i) load_b(i);
      advance();
    }
    wait_vm<(kRing - 2) * kLoads>();
    lds_barrier();
#pragma unroll
    for (int r = 0; r < kReads; ++r) read_piece(0, 0, r);
    int at = 0;
    for (int s = 0; s < all; ++s) {
      wait_vm<(kRing - 3) * kLoads>();
      lds_barrier();
      const int after = at + kStage == kRing * kStage ? 0 : at + kStage;
      block(0, 1, at, true);
      if (bias) add_bias(0);
      block(1, 0, after, false);
      if (bias) add_bias(1);
      advance();
      at = after;
    }
    wait_vm<0>();  // nothing may land in LDS that is no longer this workgroup's
  }

  // Element e of a 32x32 accumulator: row 8*(e/4) + 4*(lane/32) + e%4, column
  // lane%32.  The address is a uniform row start and the lane's offset.
  const int64_t m_first = m0 + wm, n_first = n0 + wn;
  const uint32_t lane_off = (uint32_t)(4 * (lane >> 5) * a.in + (lane & 31));
  const int64_t rows_left = a.out - m_first - 4 * (lane >> 5), cols_left = a.in - n_first - (lane & 31);
  float* const dw = a.dw + (int64_t)split * a.out * a.in + m_first * a.in + n_first;
  auto store_tile = [&](auto whole, auto adds) {
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      const bool col = whole.value || j * 32 < cols_left;
      const float back = F16 && a.back && n_first + j * 32 < a.in ? a.back[(n_first >> 5) + j] : 1.0f;
      const float g = a.gain && col ? (a.gain + n_first + j * 32)[lane & 31] : 1.0f;
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int m = i * 32 + 8 * (e >> 2) + (e & 3);
          float* const p = dw + m * a.in + j * 32;
          const float v = (F16 ? acc[i][j][e] * back : acc[i][j][e]) * g;
          if (whole.value || (col && m < rows_left)) p[lane_off] = adds.value ? p[lane_off] + v : v;
        }
    }
  };
  const bool whole = m0 + BM <= a.out && n0 + BN <= a.in;
  if (a.accumulate) {
    store_tile(std::false_type{}, std::true_type{});
  } else if (whole) {
    store_tile(std::true_type{}, std::false_type{});
  } else {
    store_tile(std::false_type{}, std::false_type{});
  }
  if (bias) {
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const float v = bsum[i] + __shfl_xor(bsum[i], 32, 64);  // the two halves of the rows
      const int64_t m = m0 + wm + i * 32 + (lane & 31);
      if (lane < 32 && m < a.out) {
        float* p = a.db + (int64_t)split * a.out + m;
        *p = a.accumulate ? *p + v : v;
      }
    }
  }
}

// --------------------------------------------------------------------- join

// out[i] (+)= gain[i % in] * back[i % in / 32] * (the sum of the splits' partial
// sums, in order), and for the bias behind them the plain sum.  VEC: 4 elements a
// thread (in % 4 == 0, out 16-byte aligned).  5 splits of 1280 x 1280: 8.7 us
// (39 MB, 4.5 TB/s).
template <bool VEC>
__global__ void __launch_bounds__(kThreads)
join_kernel(const float* __restrict__ parts, int splits, int64_t n, int64_t in, const float* __restrict__ back,
            const float* __restrict__ gain, float* __restrict__ out, const float* __restrict__ b_parts,
            int64_t n_bias, float* __restrict__ bias, bool accumulate) {
  constexpr int V = VEC ? 4 : 1;
  const int64_t step = (int64_t)gridDim.x * kThreads, tid = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  for (int64_t i = tid * V; i < n; i += step * V) {
    float s[V];
    __builtin_memcpy(s, __builtin_assume_aligned(parts + i, 4 * V), 4 * V);
    for (int p = 1; p < splits; ++p) {
      float q[V];
      __builtin_memcpy(q, __builtin_assume_aligned(parts + p * n + i, 4 * V), 4 * V);
#pragma unroll
      for (int j = 0; j < V; ++j) s[j] += q[j];
    }
    const int64_t c = !gain && !back ? 0 : n < (int64_t(1) << 32) ? (int64_t)((uint32_t)i % (uint32_t)in) : i % in;
    const float k = back ? back[c / kActBlock] : 1.0f;
    float* o = out + i;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      s[j] *= k;
      if (gain) s[j] *= gain[c + j];
      if (accumulate) s[j] = o[j] + s[j];
    }
    __builtin_memcpy(__builtin_assume_aligned(o, 4 * V), s, 4 * V);
  }
  for (int64_t i = tid; i < n_bias; i += step) {
    float s = b_parts[i];
    for (int p = 1; p < splits; ++p) s += b_parts[p * n_bias + i];
    bias[i] = accumulate ? bias[i] + s : s;
  }
}

// --------------------------------------------------------------------- plan

// Tile shapes, and the time in ns that a round of them over the CUs was
// measured to take a row (all CUs at work; two 128x128 tiles share a CU).
struct Shape {
  int bm, bn;
  double row_ns, pair_ns;  // one tile a CU; two (0: they do not fit)
};
constexpr Shape kShapes[] = {{256, 256, 23.3, 0.0}, {256, 192, 19.1, 0.0}, {256, 128, 13.4, 0.0}, {128, 128, 8.6, 14.3}};
constexpr int kNumShapes = 4;
constexpr int kCus = 256;
constexpr int kMaxSplits = 32;
constexpr int kMinSplitRows = 128;
constexpr double kBytesPerNs = 5000.0;  // of partial sums and results
constexpr double kRoundNs = 5000.0, kLaunchNs = 4000.0;

struct Plan {
  int shape, splits;
  int64_t split_rows;
};

// The tile shape and the number of splits with the least estimated time: the
// rounds of workgroups, the tiles written, and for splits the partial sums
// read again and one more launch.
Plan wgrad_plan(int64_t rows, int64_t in, int64_t out, int terms) {
  Plan best{0, 1, kBK};
  double best_ns = 0.0;
  for (int i = 0; i < kNumShapes; ++i) {
    const Shape& sh = kShapes[i];
    const int64_t t = ceil_div(out, sh.bm) * ceil_div(in, sh.bn);
    for (int s = 1; s <= kMaxSplits; ++s) {
      if (s > 1 && (rows < (int64_t)s * kMinSplitRows || t * (s - 1) >= 4 * kCus)) break;
      const int64_t sr = ceil_div(ceil_div(rows, s), kBK) * kBK;
      const double work = (double)(sr * terms), bytes = (double)out * (double)in * 4.0;
      double ns;
      if (sh.pair_ns > 0.0) {
        const int64_t full = t * s / (2 * kCus), rest = t * s - full * 2 * kCus;
        ns = (double)full * (work * sh.pair_ns + kRoundNs);
        if (rest) ns += work * (rest <= kCus ? sh.row_ns : sh.pair_ns) + kRoundNs;
      } else {
        ns = (double)ceil_div(t * s, kCus) * (work * sh.row_ns + kRoundNs);
      }
      ns += (double)s * bytes / kBytesPerNs;
      if (s > 1) ns += kLaunchNs + (double)(s + 1) * bytes / kBytesPerNs;
      if (best_ns == 0.0 || ns < best_ns) {
        best_ns = ns;
        best = Plan{i, s, sr < kBK ? kBK : sr};
      }
    }
  }
  return best;
}

// Whether the product reads this dy as it lies: 16-bit rows of whole, aligned
// 16-byte chunks whose stages span less than 2^32 bytes.
bool direct(const scape_matrix& dy, int64_t out) {
  return dy.dtype != SCAPE_F32 && ((uintptr_t)dy.data & 15u) == 0 && dy.ld % 8 == 0 && out % 8 == 0 &&
         dy.ld < (int64_t(1) << 25);
}

struct Layout {  // of the workspace, in bytes
  bool as_it_lies;
  int terms;
  int64_t rows_pad, out_pad, t_first, t_rows;
  size_t max, back, x, dy, parts, total;
};
size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

Layout layout_of(int64_t rows, int64_t in, int64_t out, const scape_matrix& dy, const Plan& p) {
  Layout l;
  l.as_it_lies = direct(dy, out);
  l.terms = terms_of(dy.dtype);
  l.rows_pad = ceil_div(rows, kBK) * kBK;
  l.out_pad = ceil_div(out, 8) * 8;
  l.t_first = l.as_it_lies ? rows / kBK * kBK : 0;
  l.t_rows = l.rows_pad - l.t_first;
  l.max = 0;
  l.back = l.x = 256;
  if (dy.dtype == SCAPE_F16) {
    const Flat f(act_blocks(in));
    l.back = align256((size_t)(kMaxParts * f.pitch));
    l.x = l.back + align256((size_t)f.nblk * 4);
  }
  l.dy = l.x + align256((size_t)l.rows_pad * (size_t)act_pitch(in) * 2);
  l.parts = l.dy + align256((size_t)l.terms * (size_t)l.t_rows * (size_t)l.out_pad * 2);
  l.total = l.parts + (p.splits == 1 ? 0 : align256((size_t)p.splits * (size_t)out * (size_t)(in + 1) * 4));
  return l;
}

template <bool F16>
void launch_product(const WgradArgs& a, int shape, unsigned grid, hipStream_t s) {
  switch (shape) {
    case 0: wgrad_kernel<F16, 256, 256, 2, 2, 5><<<grid, kWaves * 64, 0, s>>>(a); break;
    case 1: wgrad_kernel<F16, 256, 192, 2, 2, 5><<<grid, kWaves * 64, 0, s>>>(a); break;
    case 2: wgrad_kernel<F16, 256, 128, 2, 2, 6><<<grid, kWaves * 64, 0, s>>>(a); break;
    case 3: wgrad_kernel<F16, 128, 128, 2, 2, 5><<<grid, kWaves * 64, 0, s>>>(a); break;
  }
}

}  // namespace

size_t wgrad_workspace(int64_t rows, int64_t in, int64_t out, const scape_matrix& dy) {
  if (dy.data) return layout_of(rows, in, out, dy, wgrad_plan(rows, in, out, terms_of(dy.dtype))).total;
  size_t most = 0;  // of any type, aligned or not
  for (int dt : {SCAPE_F32, SCAPE_BF16, SCAPE_F16}) {
    const scape_matrix m{reinterpret_cast<void*>(uintptr_t(4)), out, dt};  // not 16-byte aligned
    const size_t t = wgrad_workspace(rows, in, out, m);
    most = t > most ? t : most;
  }
  return most;
}

int wgrad_splits(int64_t rows, int64_t in, int64_t out, int dtype, int* tile_out, int* tile_in) {
  const Plan p = wgrad_plan(rows, in, out, terms_of(dtype));
  *tile_out = kShapes[p.shape].bm;
  *tile_in = kShapes[p.shape].bn;
  return p.splits;
}

hipError_t launch_wgrad(int64_t rows, int64_t in, int64_t out, const scape_matrix& dy, const scape_act_view& x,
                        const float* gain, float* dw, float* dbias, bool accumulate, void* ws, hipStream_t s) {
  if (rows < 1 && accumulate) return hipSuccess;
  const bool f16 = dy.dtype == SCAPE_F16;
  const Plan plan = wgrad_plan(rows, in, out, terms_of(dy.dtype));
  const Layout l = layout_of(rows, in, out, dy, plan);
  char* const base = static_cast<char*>(ws);
  uint8_t* const max_parts = reinterpret_cast<uint8_t*>(base + l.max);
  float* const back = f16 && rows > 0 ? reinterpret_cast<float*>(base + l.back) : nullptr;
  hipError_t e = hipSuccess;
  if (rows > 0) {
    const Flat f(act_blocks(in));
    const int64_t scales = rows * f.nblk, groups = ceil_div(f.rows(scales), 64);
    const unsigned n_parts = (unsigned)(groups < kMaxParts ? groups : kMaxParts);
    if (f16) {
      scale_max_kernel<<<dim3((unsigned)(f.pitch / 64), n_parts), kThreads, 0, s>>>(x.scales, scales, f.nblk, f.flat,
                                                                                   f.pitch, max_parts);
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    PrepArgs p{rows, l.rows_pad, f.nblk, out, l.out_pad, x.codes, x.scales, reinterpret_cast<uint16_t*>(base + l.x),
               max_parts, (int)n_parts, f.flat, f.pitch, back, dy.data, dy.ld,
               reinterpret_cast<uint16_t*>(base + l.dy), l.t_first, l.t_rows, 0};
    int64_t xb = ceil_div(l.rows_pad * p.nblk * 4, kThreads), db = ceil_div(l.t_rows * (l.out_pad / 8), kThreads);
    if (xb > 8192) xb = 8192;
    if (db > 8192) db = 8192;
    if (f16) {  // every slab as many workgroups: at most its rows, and about 4096 in all
      const int64_t slabs = f.pitch / 64, most = slabs < 4096 ? 4096 / slabs : 1, need = f.rows(l.rows_pad * f.nblk);
      xb = slabs * (need < most ? need : most);
    }
    p.x_blocks = (unsigned)xb;
    const unsigned grid = (unsigned)(xb + db);
    switch (dy.dtype) {
      case SCAPE_F32: wgrad_prepare_kernel<SCAPE_F32><<<grid, kThreads, 0, s>>>(p); break;
      case SCAPE_BF16: wgrad_prepare_kernel<SCAPE_BF16><<<grid, kThreads, 0, s>>>(p); break;
      case SCAPE_F16: wgrad_prepare_kernel<SCAPE_F16><<<grid, kThreads, 0, s>>>(p); break;
    }
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  const int splits = plan.splits;
  float* const parts = reinterpret_cast<float*>(base + l.parts);
  WgradArgs a{};
  a.rows = rows;
  a.in = in;
  a.out = out;
  if (l.as_it_lies) {
    a.a = static_cast<const char*>(dy.data);
    a.a_step = dy.ld * 2;
    a.a_cols = out;
    a.terms = 1;
    a.tail = l.t_rows ? base + l.dy : nullptr;
  } else {
    a.a = base + l.dy;
    a.a_step = l.out_pad * 2;
    a.a_plane = l.t_rows * l.out_pad * 2;
    a.a_cols = l.out_pad;
    a.terms = l.terms;
  }
  a.tail_step = l.out_pad * 2;
  a.b = base + l.x;
  a.b_step = act_pitch(in) * 2;
  a.b_cols = act_pitch(in);
  a.split_rows = plan.split_rows;
  a.tiles_n = (int)ceil_div(in, kShapes[plan.shape].bn);
  a.tiles = (int)(ceil_div(out, kShapes[plan.shape].bm) * a.tiles_n);
  if (splits == 1) {
    a.back = back;
    a.gain = gain;
    a.dw = dw;
    a.db = dbias;
    a.accumulate = accumulate;
  } else {
    a.dw = parts;
    a.db = dbias ? parts + (int64_t)splits * out * in : nullptr;
  }
  const unsigned grid = (unsigned)((int64_t)a.tiles * splits);
  if (f16) {
    launch_product<true>(a, plan.shape, grid, s);
  } else {
    launch_product<false>(a, plan.shape, grid, s);
  }
  e = hipGetLastError();
  if (e != hipSuccess || splits == 1) return e;
  const int64_t n = out * in, nb = dbias ? out : 0;
  const bool vec = in % 4 == 0 && ((uintptr_t)dw & 15u) == 0;
  int64_t jb = ceil_div(vec ? n / 4 : n, kThreads);
  if (jb > 8192) jb = 8192;
  if (vec)
    join_kernel<true><<<(unsigned)jb, kThreads, 0, s>>>(parts, splits, n, in, back, gain, dw, a.db, nb, dbias, accumulate);
  else
    join_kernel<false><<<(unsigned)jb, kThreads, 0, s>>>(parts, splits, n, in, back, gain, dw, a.db, nb, dbias, accumulate);
  return hipGetLastError();
}

}  // namespace scape
