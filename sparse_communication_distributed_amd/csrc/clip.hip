// Norm of gradients over many tensors, and clipping by it.
//
// The tensors of a list go to the kernels by value, so that a call copies no
// table to the device and can be captured.  Each is cut into pieces of one
// size, a workgroup takes a piece, and the pieces' sums are added in their
// order: no atomics, so results do not depend on the order of the workgroups.
// Bound by memory: every gradient is read once for the norm (355 million in fp32
// 225 us, 6.3 TB/s) and once for the clipping (515 us, 5.5 TB/s), which begins
// with the pieces that were read last.
#include "ends.h"

namespace scape {
namespace {

constexpr int kSpans = 128;         // tensors of one launch: arguments of less than 4 KB
constexpr int kFewSpans = 8;        // of a short list's: a call for one small tensor 9 us, with 4 KB to pass 13
constexpr int kLaunchGroups = 4096;  // groups of one launch: 12 bits
constexpr int64_t kPieces = 16384;  // pieces of a long list, about
constexpr int kFewPieces = 1024;   // of a group: the clipping adds their sums itself

struct Span {
  const void* data;
  void* out;
  uint64_t what;  // elements; from bit 48 on data's type, out's type, and the group less the launch's first
};

// The same in the workspace, where the sums' launches leave it if there are
// several: the scaling is one launch then.
struct Listed {
  const void* data;
  void* out;
  uint64_t what;  // elements and types
  int32_t first, group;
};

template <int NS>
struct SpanArgs {
  Span span[NS];
  int32_t first[NS];  // piece of the whole list at which each span begins; past the last: none
  int32_t begin;          // the first span's
  int32_t end;            // one past the last span's last piece
  int32_t group;          // of the first span
  int64_t piece;
  double* sums;
  Listed* listed;    // the first span's place in the list; null: not wanted
  int32_t* span_at;  // of each piece, the span's place in the list
  int32_t index;     // the first span's
};

struct ListArgs {
  const Listed* listed;
  const int32_t* span_at;
  const double* sums;
  int32_t pieces;
  int64_t piece;
};

struct Scaling {
  const double* factors;  // of each group; null: found from the sums
  float* norm;            // written where factors is null
  float scale, max_norm;
  int32_t group_pieces;  // where factors is null: of every group
  bool stream;           // past the caches
};

struct GroupArgs {
  int32_t first[kSpans + 1];  // pieces of each group
  Scaling s;
  bool clip;
  const double* sums;
  double* factors;
  float* norm;
};

// Over the T threads of a workgroup; every one gets it, the same one.
template <int T>
__device__ __forceinline__ double block_sum(double x, double* lds) {
  x = wave_sum(x);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
  __syncthreads();
  x = lds[0];
#pragma unroll
  for (int w = 1; w < T / 64; ++w) x += lds[w];
  return x;
}

// Sum of a group's pieces.
template <int T>
__device__ __forceinline__ double group_sum(const double* sums, int32_t n, double* lds) {
  double sum = 0.0;
#pragma unroll 4
  for (int32_t i = threadIdx.x; i < n; i += T) sum += sums[i];
  return block_sum<T>(sum, lds);
}

__device__ __forceinline__ double factor_of(double norm, const Scaling& s) {
  const bool over = norm > (double)s.max_norm && norm < (double)__builtin_inff();
  return over ? (double)s.scale * ((double)s.max_norm / norm) : (double)s.scale;
}

// The span of a piece: the number of those that begin at or before it, less
// one, counted by all lanes at once.
template <int NS>
__device__ __forceinline__ int span_of(const SpanArgs<NS>& a, int32_t piece) {
  const int lane = threadIdx.x & 63;
  int n = 0;
#pragma unroll
  for (int k = 0; k < NS; k += 64) n += __popcll(__ballot(k + lane < NS && a.first[k + lane] <= piece));
  return n - 1;
}

struct Piece {
  const void* data;
  void* out;
  int64_t lo, hi;
  int dtype, out_dtype, group;
  __device__ __forceinline__ Piece(const void* d, void* o, uint64_t what, int group_, int32_t nth, int64_t piece) {
    data = d;
    out = o;
    const int64_t count = (int64_t)(what & ((uint64_t(1) << 48) - 1));
    dtype = (int)(what >> 48) & 3;
    out_dtype = (int)(what >> 50) & 3;
    group = group_;
    lo = nth * piece;
    hi = lo + piece < count ? lo + piece : count;
  }
};
template <int NS>
__device__ __forceinline__ Piece piece_at(const SpanArgs<NS>& a, int32_t piece, int span) {
  const Span& s = a.span[span];
  return Piece(s.data, s.out, s.what, a.group + (int)(s.what >> 52), piece - a.first[span], a.piece);
}

// N elements as they lie in memory: 8 or 16 bytes.
template <int DT, int N>
struct Some {
  static constexpr int kBytes = N * (DT == SCAPE_F32 ? 4 : 2);
  uint32_t u[kBytes / 4];
  __device__ __forceinline__ void load(const char* p) {
    if (kBytes == 16) {
      load16<false>(u, p);
    } else {
      typedef u32x2 u32x2_any __attribute__((aligned(2)));
      const u32x2 v = *reinterpret_cast<const u32x2_any*>(p);
      __builtin_memcpy(u, &v, 8);
    }
  }
  __device__ __forceinline__ void widen(float (&v)[N]) const {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      if (DT == SCAPE_F32) v[j] = __uint_as_float(u[j % (kBytes / 4)]);
      else if (DT == SCAPE_BF16) v[j] = __uint_as_float((j & 1) ? u[j / 2] & 0xffff0000u : u[j / 2] << 16);
      else v[j] = (float)__builtin_bit_cast(_Float16, (uint16_t)(u[j / 2] >> (16 * (j & 1))));
    }
  }
};

// Calls many(i, x) for N elements at a time where they lie wholly in [lo, hi),
// DEEP of a thread's on the way, and one(i) for the elements behind them.
template <int DT, int N, int DEEP, typename F, typename G>
__device__ __forceinline__ void walk(const void* data, int64_t lo, int64_t hi, F many, G one) {
  constexpr int kSize = DT == SCAPE_F32 ? 4 : 2;
  const char* const base = static_cast<const char*>(data);
  constexpr int64_t step = (int64_t)kThreads * N;
  int64_t i = lo + (int64_t)threadIdx.x * N;
  for (; lo + DEEP * step <= hi; lo += DEEP * step, i += DEEP * step) {
    Some<DT, N> x[DEEP];
#pragma unroll
    for (int k = 0; k < DEEP; ++k) x[k].load(base + (i + k * step) * kSize);
#pragma unroll
    for (int k = 0; k < DEEP; ++k) many(i + k * step, x[k]);
  }
  for (; i + N <= hi; i += step) {
    Some<DT, N> x;
    x.load(base + i * kSize);
    many(i, x);
  }
  for (int64_t j = i; j < hi; ++j) one(j);
}

template <int DT>
__device__ __forceinline__ double squares(const Piece& p) {
  double sum[4] = {0.0, 0.0, 0.0, 0.0};
  constexpr int N = DT == SCAPE_F32 ? 4 : 8;
  walk<DT, N, 4>(
      p.data, p.lo, p.hi,
      [&](int64_t, const Some<DT, N>& x) {
        float v[N];
        x.widen(v);
#pragma unroll
        for (int j = 0; j < N; ++j) sum[j & 3] = __builtin_fma((double)v[j], (double)v[j], sum[j & 3]);
      },
      [&](int64_t i) {
        const double x = Elem<DT>::get(p.data, i);
        sum[0] = __builtin_fma(x, x, sum[0]);
      });
  return (sum[0] + sum[1]) + (sum[2] + sum[3]);
}

template <int NS>
__global__ void __launch_bounds__(kThreads) grad_sum_kernel(SpanArgs<NS> a) {
  __shared__ double lds[kThreads / 64];
  const int32_t piece = a.begin + (int32_t)blockIdx.x;
  const int span = span_of(a, piece);
  const Piece p = piece_at(a, piece, span);
  if (a.listed && threadIdx.x == 0) {
    a.span_at[piece] = a.index + span;
    if (piece == a.first[span]) a.listed[span] = Listed{p.data, p.out, a.span[span].what, piece, p.group};
  }
  double sum;
  if (p.dtype == SCAPE_F32) sum = squares<SCAPE_F32>(p);
  else if (p.dtype == SCAPE_BF16) sum = squares<SCAPE_BF16>(p);
  else sum = squares<SCAPE_F16>(p);
  sum = block_sum<kThreads>(sum, lds);
  if (threadIdx.x == 0) a.sums[piece] = sum;
}

// One workgroup a group: its norm and the factor of its gradients.
constexpr int kNormThreads = 1024;
__global__ void __launch_bounds__(kNormThreads) grad_norm_kernel(GroupArgs a) {
  __shared__ double lds[kNormThreads / 64];
  const int g = blockIdx.x;
  const double sum = group_sum<kNormThreads>(a.sums + a.first[g], a.first[g + 1] - a.first[g], lds);
  if (threadIdx.x != 0) return;
  const double norm = sqrt(sum) * (double)a.s.scale;
  a.norm[g] = (float)norm;
  if (a.clip) a.factors[g] = factor_of(norm, a.s);
}

// A binary64 product as fp32 that Elem<OT>::put rounds as it would the product
// itself.  For 16 bits fp32 takes the neighbour towards zero with its last bit
// set wherever digits are lost: that is neither a 16-bit value nor halfway
// between two of them, so what is next to one of these stays on its side.
template <int OT>
__device__ __forceinline__ float narrowed(double x) {
  const float f = (float)x;
  if (OT == SCAPE_F32) return f;
  const double back = f;
  uint32_t u = __float_as_uint(f);
  if (back != x) u = (u - (fabs(back) > fabs(x) ? 1u : 0u)) | 1u;
  return __uint_as_float(u);
}

template <int DT, int OT, bool STREAM>
__device__ __forceinline__ void scale_piece(const Piece& p, double f) {
  // 16 bytes of the wider side a lane, so that neighbouring lanes' accesses
  // join: bf16 to fp32 at 32 bytes a lane took 970 us where this takes 620
  // (557 million elements)
  constexpr int N = OT == SCAPE_F32 ? 4 : 8;
  walk<DT, N, DT == OT ? 4 : 8>(
      p.data, p.lo, p.hi,
      [&](int64_t i, const Some<DT, N>& x) {
        float v[N];
        x.widen(v);
        // one rounding of the binary64 product, which is exact or next to it
        typename Elem<OT>::T o[N];
#pragma unroll
        for (int j = 0; j < N; ++j) Elem<OT>::put(o, j, narrowed<OT>((double)v[j] * f));
        u32x4 w;
        __builtin_memcpy(&w, o, 16);
        u32x4_any* q = reinterpret_cast<u32x4_any*>(static_cast<typename Elem<OT>::T*>(p.out) + i);
        if (STREAM) __builtin_nontemporal_store(w, q);
        else *q = w;
        // one chunk's conversions after another's: interleaved they take 129 registers of every call's threads, three
        // waves a SIMD and not seven, 11.5 us and not 9.9 for two fp32 tensors of 2^20
        if (OT != SCAPE_F32) __builtin_amdgcn_sched_barrier(0);
      },
      [&](int64_t i) { Elem<OT>::put(p.out, i, narrowed<OT>((double)Elem<DT>::get(p.data, i) * f)); });
}

template <int DT, int OT>
__device__ __forceinline__ void scale_some(const Piece& p, double f, bool stream) {
  if (stream) scale_piece<DT, OT, true>(p, f);
  else scale_piece<DT, OT, false>(p, f);
}

__device__ __forceinline__ void scale_group_piece(const Piece& p, int32_t piece, const double* sums, const Scaling& s) {
  __shared__ double lds[kThreads / 64];
  double f;
  if (s.factors) {
    f = s.factors[p.group];
  } else {
    const int32_t first = p.group * s.group_pieces;
    const double norm = sqrt(group_sum<kThreads>(sums + first, s.group_pieces, lds)) * (double)s.scale;
    f = factor_of(norm, s);
    if (piece == first && threadIdx.x == 0) s.norm[p.group] = (float)norm;
  }
  if (f == 1.0 && p.out == p.data) return;
  if (p.dtype == SCAPE_F32) scale_some<SCAPE_F32, SCAPE_F32>(p, f, s.stream);
  else if (p.dtype == SCAPE_BF16 && p.out_dtype == SCAPE_BF16) scale_some<SCAPE_BF16, SCAPE_BF16>(p, f, s.stream);
  else if (p.dtype == SCAPE_BF16) scale_some<SCAPE_BF16, SCAPE_F32>(p, f, s.stream);
  else if (p.out_dtype == SCAPE_F16) scale_some<SCAPE_F16, SCAPE_F16>(p, f, s.stream);
  else scale_some<SCAPE_F16, SCAPE_F32>(p, f, s.stream);
}

template <int NS>
__global__ void __launch_bounds__(kThreads) grad_scale_kernel(SpanArgs<NS> a, Scaling s) {
  const int32_t piece = a.end - 1 - (int32_t)blockIdx.x;
  scale_group_piece(piece_at(a, piece, span_of(a, piece)), piece, a.sums, s);
}

__global__ void __launch_bounds__(kThreads) grad_scale_list_kernel(ListArgs a, Scaling s) {
  const int32_t piece = a.pieces - 1 - (int32_t)blockIdx.x;
  const Listed l = a.listed[a.span_at[piece]];
  scale_group_piece(Piece(l.data, l.out, l.what, l.group, piece - l.first, a.piece), piece, a.sums, s);
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

// The list's tensors in launches of at most NS: the sums of their pieces, or
// (with `how`) their scaling.  per: tensors of a group.
template <int NS>
void launch_spans(int32_t count, const scape_grad* grads, int32_t per, int64_t piece, double* sums, Listed* listed,
                  int32_t* span_at, const Scaling* how, hipStream_t s) {
  SpanArgs<NS> a;
  a.piece = piece;
  a.sums = sums;
  a.listed = listed;
  a.span_at = span_at;
  a.index = 0;
  int32_t at = 0, n = 0;
  for (int32_t i = 0; i <= count; ++i) {
    const bool far = n > 0 && i < count && i / per - a.group >= kLaunchGroups;
    if (n > 0 && (i == count || n == NS || far)) {
      a.begin = a.first[0];
      a.end = at;
      for (int32_t j = n; j < NS; ++j) a.first[j] = INT32_MAX;
      const dim3 grid((unsigned)(a.end - a.begin));
      if (how) grad_scale_kernel<NS><<<grid, kThreads, 0, s>>>(a, *how);
      else grad_sum_kernel<NS><<<grid, kThreads, 0, s>>>(a);
      if (a.listed) a.listed += n;
      a.index += n;
      n = 0;
    }
    if (i == count || grads[i].count == 0) continue;
    const scape_grad& g = grads[i];
    if (n == 0) a.group = i / per;
    a.first[n] = at;
    Span& p = a.span[n++];
    p.data = g.data;
    p.out = g.out ? g.out : const_cast<void*>(g.data);
    p.what = (uint64_t)g.count | (uint64_t)g.dtype << 48 | (uint64_t)(g.out ? g.out_dtype : g.dtype) << 50 |
             (uint64_t)(i / per - a.group) << 52;
    at += (int32_t)pieces(g.count, piece);
  }
}

}  // namespace

size_t grad_workspace(int32_t count, const scape_grad* grads, int32_t groups) {
  const size_t n = (size_t)pieces_of(count, grads);
  // the sums and the factors; the list, and each piece's place in it
  const size_t bytes = (n + (size_t)groups) * sizeof(double) + (size_t)count * sizeof(Listed) + n * sizeof(int32_t);
  return (bytes + 255) & ~(size_t)255;
}

hipError_t launch_grads(int32_t count, const scape_grad* grads, int32_t groups, float scale, bool clip, float max_norm,
                        float* norm, void* ws, hipStream_t s) {
  const int64_t piece = piece_of(count, grads);
  const int32_t per = count / groups;
  double* sums = static_cast<double*>(ws);
  const int64_t all = pieces_of(count, grads);
  double* factors = sums + all;
  Listed* listed = reinterpret_cast<Listed*>(factors + groups);
  int32_t* span_at = reinterpret_cast<int32_t*>(listed + count);
  // 393 small tensors: 21.5 us, with as many launches for the scaling as for the sums 32 or more
  const bool list = clip && count > kSpans;
  int64_t bytes = 0;
  for (int32_t i = 0; i < count; ++i)
    bytes += grads[i].count * (int64_t)(dtype_bytes(grads[i].dtype) +
                                        (grads[i].out ? dtype_bytes(grads[i].out_dtype) : 0));

  // groups of as many pieces each, and few: one launch less
  int64_t each = 0;
  bool alike = clip;
  for (int32_t g = 0; alike && g < groups; ++g) {
    int64_t n = 0;
    for (int32_t i = g * per; i < (g + 1) * per; ++i) n += pieces(grads[i].count, piece);
    if (g == 0) each = n;
    alike = n == each && n > 0 && n <= kFewPieces;
  }
  const Scaling how{alike ? nullptr : factors, norm, scale, max_norm, (int32_t)each, bytes > kStreamBytes};

  const auto walk = [&](const Scaling* scaling) {
    Listed* const to = list ? listed : nullptr;
    if (count <= kFewSpans) launch_spans<kFewSpans>(count, grads, per, piece, sums, to, span_at, scaling, s);
    else launch_spans<kSpans>(count, grads, per, piece, sums, to, span_at, scaling, s);
  };

  walk(nullptr);
  if (!alike) {
    GroupArgs b;
    b.s = how;
    b.clip = clip;
    b.sums = sums;
    int32_t at = 0;
    for (int32_t g0 = 0; g0 < groups; g0 += kSpans) {
      const int32_t n = groups - g0 < kSpans ? groups - g0 : kSpans;
      for (int32_t g = 0; g < n; ++g) {
        b.first[g] = at;
        for (int32_t i = (g0 + g) * per; i < (g0 + g + 1) * per; ++i) at += (int32_t)pieces(grads[i].count, piece);
      }
      b.first[n] = at;
      b.factors = factors + g0;
      b.norm = norm + g0;
      grad_norm_kernel<<<dim3((unsigned)n), kNormThreads, 0, s>>>(b);
    }
  }
  if (list && all > 0) {
    const ListArgs a{listed, span_at, sums, (int32_t)all, piece};
    grad_scale_list_kernel<<<dim3((unsigned)all), kThreads, 0, s>>>(a, how);
  } else if (clip) {
    walk(&how);
  }
  return hipGetLastError();
}

}  // namespace scape
