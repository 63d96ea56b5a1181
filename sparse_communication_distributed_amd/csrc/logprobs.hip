// Log probabilities of given tokens, entropy, the likeliest alternatives, and
// the gradient of the logits.
//
// With m the largest logit, t = scale (x - m) and o the sum of e^t over all
// words but one of the likeliest: logp = t_y - log(1 + o), entropy = log(1 + o)
// - sum(e^t t) / (1 + o), and the gradient is a function of each logit alone.
// A row is read once, into registers, from which the maximum, the sums and the
// gradient are taken.  One too long for that passes by, its sums kept relative
// to the maximum so far, and is read again for its gradient.
#include "ends.h"

#include <type_traits>

namespace scape {
namespace {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.693147180559945309417f;
constexpr int kCandidates = 512;  // logits that compete for a row's alternatives, at most

__device__ __forceinline__ float neg_inf() { return -__builtin_inff(); }
// An exponent of 2 that is not positive, -256 at least: 2^-256 is 0, and 0 times
// it nothing, which 0 times -inf is not.
__device__ __forceinline__ float floored(float x) { return __builtin_amdgcn_fmed3f(x, -256.0f, 0.0f); }

// Orders floats as unsigned numbers: NaN above everything, -0 as 0.
__device__ __forceinline__ uint32_t order_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  if (x != x) return 0xffffffffu;
  return (b >> 31) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float of_order(uint32_t k) {
  return __uint_as_float((k >> 31) ? k & 0x7fffffffu : ~k);
}
constexpr uint32_t kOrderNegInf = 0x007fffffu;
// The larger key is the larger logit, or of equal ones the lower index; no key
// is all ones.
__device__ __forceinline__ uint64_t key_of(float x, uint32_t i) {
  return (uint64_t)order_of(x) << 32 | (0xfffffffeu - i);
}
__device__ __forceinline__ uint32_t key_index(uint64_t k) { return 0xfffffffeu - (uint32_t)k; }

__device__ __forceinline__ uint32_t lanes_below(uint64_t mask) {
  return __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0u));
}

// ------------------------------------------------------- threads of a row

// T threads share a row: a wave of a workgroup of four, or a whole workgroup.
template <int T>
struct Team {
  static constexpr int kRows = T == 64 ? 4 : 1;  // rows of a workgroup
  static constexpr int kWaves = T / 64;
  static __device__ __forceinline__ int thread() { return threadIdx.x % T; }
  static __device__ __forceinline__ void sync() {
    if (T == 64) {
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    } else {
      __syncthreads();
    }
  }
};

template <int T>
struct RowLds {
  float most[Team<T>::kWaves], sum[3][Team<T>::kWaves], again[1][Team<T>::kWaves];
  uint64_t key[Team<T>::kWaves];
  uint32_t order[T];
  uint64_t cand[kCandidates];
  uint32_t n, ties[Team<T>::kWaves];
  float target;
};

// Over a wave, the same for every lane: the 16 lanes of a row by exchanges
// within the registers, then the rows.
template <typename F>
__device__ __forceinline__ float wave_join(float x, F f) {
  const auto other = [&](auto ctrl) {
    return __int_as_float(
        __builtin_amdgcn_update_dpp(0, __float_as_int(x), decltype(ctrl)::value, 0xf, 0xf, true));
  };
  x = f(x, other(std::integral_constant<int, 0xB1>{}));   // lanes 1 0 3 2
  x = f(x, other(std::integral_constant<int, 0x4E>{}));   // lanes 2 3 0 1
  x = f(x, other(std::integral_constant<int, 0x141>{}));  // the 8 lanes mirrored
  x = f(x, other(std::integral_constant<int, 0x140>{}));  // the 16 lanes mirrored
  const auto row = [&](int lane) { return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), lane)); };
  return f(f(row(0), row(16)), f(row(32), row(48)));
}

template <int T>
__device__ __forceinline__ float team_max(float x, RowLds<T>& l) {
  const auto larger = [](float a, float b) { return __builtin_fmaxf(a, b); };
  x = wave_join(x, larger);
  if (T == 64) return x;
  if ((threadIdx.x & 63) == 0) l.most[threadIdx.x >> 6] = x;
  __syncthreads();
  x = l.most[0];
#pragma unroll
  for (int w = 1; w < Team<T>::kWaves; ++w) x = __builtin_fmaxf(x, l.most[w]);
  return x;
}

template <int T, int N, int M>
__device__ __forceinline__ void team_sum(float (&x)[N], float (&lds)[M][Team<T>::kWaves]) {
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = wave_join(x[i], [](float a, float b) { return a + b; });
  if (T == 64) return;
  if ((threadIdx.x & 63) == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) lds[i][threadIdx.x >> 6] = x[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    x[i] = lds[i][0];
#pragma unroll
    for (int w = 1; w < Team<T>::kWaves; ++w) x[i] += lds[i][w];
  }
}

template <int T>
__device__ __forceinline__ uint64_t team_max_key(uint64_t x, RowLds<T>& l) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) {
    const uint64_t y = __shfl_xor((unsigned long long)x, d, 64);
    x = x > y ? x : y;
  }
  if (T == 64) return x;
  __syncthreads();
  if ((threadIdx.x & 63) == 0) l.key[threadIdx.x >> 6] = x;
  __syncthreads();
  for (int w = 0; w < Team<T>::kWaves; ++w) x = x > l.key[w] ? x : l.key[w];
  return x;
}

// ------------------------------------------------------------ a row's logits
//
// A thread's chunks of 16 aligned bytes, and one of the few logits before the
// first and behind the last of them (61 rows of 50257 fp16 took 10.7 us from
// where each row begins, 8.4 if they begin aligned).  each(f) calls f(first, n, v)
// for them with the index of the first and their number as a Number; what a
// thread holds past the row is -inf, with an index that is not below its end.
template <int N>
using Number = std::integral_constant<int, N>;

template <int DT>
struct Chunk {
  static constexpr int kSize = DT == SCAPE_F32 ? 4 : 2;
  static constexpr int N = 16 / kSize;
  u32x4 u;
  // From `first` logits behind p, the same for all threads that share a row.
  __device__ __forceinline__ void load(const char* p, int first) {
    load16<false>(&u, p + (uint32_t)first * (uint32_t)kSize);
  }
  template <bool STREAM>
  __device__ __forceinline__ static void store(char* p, int first, const float* v) {
    typename Elem<DT>::T o[N];
#pragma unroll
    for (int j = 0; j < N; ++j) Elem<DT>::put(o, j, v[j]);
    u32x4 w;
    __builtin_memcpy(&w, o, 16);
    u32x4_any* const q = reinterpret_cast<u32x4_any*>(p + (uint32_t)first * (uint32_t)kSize);
    if (STREAM) __builtin_nontemporal_store(w, q);
    else *q = w;
  }
  __device__ __forceinline__ void unpack(float (&v)[N]) const {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      if (DT == SCAPE_F32) v[j] = __uint_as_float(u[j & 3]);
      else if (DT == SCAPE_BF16) v[j] = __uint_as_float((j & 1) ? u[j / 2] & 0xffff0000u : u[j / 2] << 16);
      else v[j] = (float)__builtin_bit_cast(_Float16, (uint16_t)(u[j / 2] >> (16 * (j & 1))));
    }
  }
  __device__ __forceinline__ void none() {
    const uint32_t inf = DT == SCAPE_F32 ? 0xff800000u : DT == SCAPE_BF16 ? 0xff80ff80u : 0xfc00fc00u;
    u = u32x4{inf, inf, inf, inf};
  }
  // Hides from the compiler that the logits are what they were before.
  __device__ __forceinline__ void keep() { asm volatile("" : "+v"(u)); }
};

// How a row is cut: `head` single logits, `whole` chunks, and the rest single.
template <int DT>
struct Cut {
  static constexpr int N = Chunk<DT>::N;
  const char* p;
  int vocab, head, whole;
  __device__ __forceinline__ Cut(const char* row, int64_t cols) {
    p = row;
    vocab = (int)cols;
    head = (int)((16 - ((uintptr_t)row & 15)) & 15) / Chunk<DT>::kSize;
    head = head < vocab ? head : vocab;
    whole = (vocab - head) / N;
  }
  __device__ __forceinline__ int chunk(int i) const { return head + i * N; }  // its first logit
  __device__ __forceinline__ int chunks_end() const { return chunk(whole); }
  __device__ __forceinline__ int singles() const { return vocab - whole * N; }
  __device__ __forceinline__ int single(int i) const { return i < head ? i : i < singles() ? i + whole * N : vocab; }
  // The chunk that holds logit y; behind the chunks, the singles.
  __device__ __forceinline__ int unit_of(int y) const {
    return y < head ? whole + y : y < chunks_end() ? (y - head) / N : y - whole * N + whole;
  }
  __device__ __forceinline__ float get(int i) const { return i < vocab ? Elem<DT>::get(p, i) : neg_inf(); }
  // The last chunk in the place of one past it: loaded and dropped, without a
  // branch, behind which the loads under way would be waited for.
  __device__ __forceinline__ void load(Chunk<DT>& x, int i) const { x.load(p, chunk(i < whole ? i : whole - 1)); }
};

// C chunks a thread in registers.
template <int DT, int T, int C>
struct Row : Cut<DT> {
  using Cut<DT>::N;
  using Cut<DT>::whole;
  Chunk<DT> r[C];
  float one;
  __device__ __forceinline__ Row(const char* row, int64_t cols) : Cut<DT>(row, cols) {
    if (whole == 0) {
#pragma unroll
      for (int i = 0; i < C; ++i) r[i].none();
    } else {
#pragma unroll
      for (int i = 0; i < C; ++i) Cut<DT>::load(r[i], index(i));
    }
    one = Cut<DT>::get(Cut<DT>::single(Team<T>::thread()));
    if (whole == 0) return;
#pragma unroll
    for (int i = 0; i < C; ++i)
      if ((i + 1) * T > whole && index(i) >= whole) r[i].none();
  }
  __device__ __forceinline__ int index(int i) const { return i * T + Team<T>::thread(); }
  // One chunk after the other, widened again in every pass: kept in 32 bits
  // from one pass to the next they would take the registers of half the waves.
  template <typename F>
  __device__ __forceinline__ void each(F f) {
#pragma unroll
    for (int i = 0; i < C; ++i) {
      float v[N];
      r[i].keep();
      if (i * T < whole) {  // of some thread
        r[i].unpack(v);
        f(Cut<DT>::chunk(index(i)), Number<N>{}, v);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    f(Cut<DT>::single(Team<T>::thread()), Number<1>{}, &one);
  }
  // For an f that the threads of a wave take part in together.
  template <typename F>
  __device__ __forceinline__ void each_in_turn(F f) {
    each(f);
  }
};

// Read from memory each time.
template <int DT, int T>
struct Row<DT, T, 0> : Cut<DT> {
  using Cut<DT>::N;
  using Cut<DT>::whole;
  __device__ __forceinline__ Row(const char* row, int64_t cols) : Cut<DT>(row, cols) {}
  template <int U = 4, typename F>
  __device__ __forceinline__ void each(F f) const {
    const int t = Team<T>::thread();
#pragma unroll U
    for (int i = t; i < whole; i += T) {
      Chunk<DT> x;
      float v[N];
      x.load(Cut<DT>::p, Cut<DT>::chunk(i));
      x.unpack(v);
      f(Cut<DT>::chunk(i), Number<N>{}, v);
    }
    const int i = Cut<DT>::single(t);
    float one = Cut<DT>::get(i);
    f(i, Number<1>{}, &one);
  }
  template <typename F>
  __device__ __forceinline__ void each_in_turn(F f) const {
    each<1>(f);
  }
};

// -------------------------------------------------------------- alternatives

// Calls f(rank, key) for the `top` largest keys of any row, in a pass for each.
template <int T, typename M, typename F>
__device__ __forceinline__ void top_slowly(const M& memory, int top, RowLds<T>& l, F f) {
  uint64_t last = ~0ull;
  for (int i = 0; i < top; ++i) {
    uint64_t best = 0;
    memory.each_in_turn([&](int first, auto n, const float* v) {
#pragma unroll 1
      for (int j = 0; j < n; ++j) {
        const uint64_t k = key_of(v[j], (uint32_t)(first + j));
        best = first + j < memory.vocab && k < last && k > best ? k : best;
      }
    });
    last = team_max_key<T>(best, l);
    if (Team<T>::thread() == 0) f(i, last);
  }
}

// The largest `bits`-bit prefix of an order that at least k of 128 values (two
// a lane) reach.
__device__ __forceinline__ uint32_t kth_prefix(uint32_t a, uint32_t b, int k, int bits) {
  const auto reach = [&](uint32_t q) { return __popcll(__ballot(a >= q)) + __popcll(__ballot(b >= q)) >= k; };
  uint32_t p = 0;
  for (int s = 30; s >= 32 - bits; s -= 2) {  // two bits a step
    const uint32_t q1 = p | 1u << s, q2 = p | 2u << s, q3 = p | 3u << s;
    const bool r1 = reach(q1), r2 = reach(q2), r3 = reach(q3);
    p = r3 ? q3 : r2 ? q2 : r1 ? q1 : p;
  }
  return p;
}

// The same for a row without a NaN.  `most`: this thread's largest logit;
// `memory`: the row, which may be the same.
//
// The k-th largest of 64 or 128 groups' maxima bounds the k-th largest logit
// from below, and few logits beside the k reach it: those are collected, and
// each one's rank is the number of larger ones.  Where too many are equal to
// the bound, those above it are collected, and the equal ones taken by index.
template <int T, typename R, typename M, typename F>
__device__ __forceinline__ void top_of(R& row, const M& memory, int top, float most, RowLds<T>& l, F f) {
  constexpr int W = Team<T>::kWaves;
  const int t = Team<T>::thread(), lane = threadIdx.x & 63;
  const auto collect = [&](auto pass, float bound, auto equal) {
    constexpr bool kEqual = decltype(equal)::value;
    Team<T>::sync();
    if (t == 0) l.n = 0;
    Team<T>::sync();
    pass([&](int first, auto n, const float* v) {
      float most = v[0];  // of a wave's chunks few hold any
#pragma unroll
      for (int j = 1; j < n; ++j) most = __builtin_fmaxf(most, v[j]);
      if (!__any(kEqual ? most >= bound : most > bound)) return;
      uint32_t mask = 0;  // a bit for each logit that reaches the bound
#pragma unroll
      for (int j = 0; j < n; ++j) mask |= (kEqual ? v[j] >= bound : v[j] > bound) ? 1u << j : 0u;
      if (first >= (n > 1 ? memory.chunks_end() : memory.vocab)) mask = 0;  // -inf that stand for none
      for (; mask; mask &= mask - 1) {
        const int j0 = __builtin_ctz(mask);
        float x = v[0];
#pragma unroll
        for (int j = 1; j < n; ++j) x = j == j0 ? v[j] : x;
        const uint32_t at = atomicAdd(&l.n, 1u);  // of LDS; the ranks do not depend on the places
        if (at < kCandidates) l.cand[at] = key_of(x, (uint32_t)(first + j0));
      }
    });
    Team<T>::sync();
    return l.n;
  };
  const auto rank = [&](uint32_t n) {
    for (uint32_t i = t; i < n; i += T) {
      const uint64_t k = l.cand[i];
      int r = 0;
#pragma unroll 8
      for (uint32_t j = 0; j < n; ++j) r += l.cand[j] > k;
      if (r < top) f(r, k);
    }
  };
  uint32_t a = order_of(most), b = 0;
  if (W > 1) {
    Team<T>::sync();
    l.order[t] = a;
    Team<T>::sync();
    a = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const uint32_t o = l.order[w * 64 + lane];
      if (w < W / 2) a = a > o ? a : o;
      else b = b > o ? b : o;
    }
  }
  // with fewer threads than alternatives that hold a logit, all are collected
  const bool enough = memory.whole >= top;
  const auto bound_of = [&](int bits) {
    const uint32_t p = enough ? kth_prefix(a, b, top, bits) : 0;
    return p <= kOrderNegInf ? neg_inf() : of_order(p);
  };
  uint32_t n = collect([&](auto f) { row.each_in_turn(f); }, bound_of(20), std::true_type{});
  if (n <= kCandidates) {
    rank(n);
    return;
  }
  const float bound = bound_of(32);
  n = collect([&](auto f) { memory.each_in_turn(f); }, bound, std::false_type{});
  if (n > kCandidates) {
    top_slowly<T>(memory, top, l, f);
    return;
  }
  rank(n);
  // the equal ones in the row's order, T at a time; the row holds enough of them
  uint32_t found = n;
  for (int c0 = 0; found < (uint32_t)top && c0 < memory.vocab; c0 += T) {
    const int c = c0 + t;
    const bool is = c < memory.vocab && memory.get(c) == bound;
    const uint64_t mask = __ballot(is);
    uint32_t at = found + lanes_below(mask);
    if (W > 1) {
      Team<T>::sync();  // the counts before have been read
      if (lane == 0) l.ties[t >> 6] = (uint32_t)__popcll(mask);
      Team<T>::sync();
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const uint32_t x = l.ties[w];
        at += w < t >> 6 ? x : 0;
        found += x;
      }
    } else {
      found += (uint32_t)__popcll(mask);
    }
    if (is && at < (uint32_t)top) f((int)at, key_of(bound, (uint32_t)c));
  }
}

// ------------------------------------------------------------------ gradient

// What a row's gradient is a function of.
struct RowGradient {
  float m, c, ls2, w, d, h, scale;
  int y;  // negative: none
  bool none;
  __device__ __forceinline__ RowGradient(const LogprobArgs& a, int64_t r, float m_, float ls, float entropy) {
    m = m_;
    c = a.scale * kLog2e;
    ls2 = ls * kLog2e;
    h = entropy;
    scale = a.scale;
    const int64_t id = a.dlogp ? token_at(a.targets, r) : -1;
    y = id >= 0 && id < a.vocab ? (int)id : -1;
    w = y >= 0 ? a.dlogp[r] : 0.0f;
    d = a.dentropy ? a.dentropy[r] : 0.0f;
    none = (w == 0.0f && d == 0.0f) || m == neg_inf();
    w += ls - ls;  // NaN of a row that holds one
  }
  // Replaces a chunk's logits by their gradients; the target's is put by itself.
  template <bool ENT, int M>
  __device__ __forceinline__ void of(float* v, Number<M> n) const {
#pragma unroll
    for (int j = 0; j < n; ++j) {
      float l = __builtin_fmaf(v[j] - m, c, -ls2);  // log2 of the probability
      if (ENT) {
        l = floored(l);
        v[j] = -__builtin_amdgcn_exp2f(l) * __builtin_fmaf(d, __builtin_fmaf(l, kLn2, h), w) * scale;
      } else {
        v[j] = __builtin_amdgcn_exp2f(l) * (-w * scale);
      }
    }
  }
  // The target's, from its logit x: 1 - p keeps its precision next to p = 1.
  __device__ __forceinline__ float at_target(float x) const {
    const float lp = (x - m) * scale - ls2 * kLn2;
    float g = -w * expm1f(lp);
    if (d != 0.0f && lp > neg_inf()) g -= d * expf(lp) * (lp + h);
    return g * scale;
  }
};

// Writes the gradient of n logits from `first` on, those of them that the row has.
template <int DT, bool ENT, bool STREAM, int M>
__device__ __forceinline__ void emit_some(const RowGradient& g, char* out, int first, Number<M> n, int vocab, float* v) {
  if (first >= vocab) return;
  g.of<ENT>(v, n);
  if (n > 1) Chunk<DT>::template store<STREAM>(out, first, v);
  else Elem<DT>::put(out, first, v[0]);
}

// Zeros for the units [from, to) of a row, chunks and behind them single logits,
// every T-th of them: what a row without a gradient gets, which is not read.
template <int DT, int T, bool STREAM>
__device__ __forceinline__ void put_zeros(const Cut<DT>& row, char* out, int from, int to) {
  constexpr int N = Cut<DT>::N;
  float zeros[N];
#pragma unroll
  for (int j = 0; j < N; ++j) zeros[j] = 0.0f;
  const int units = row.whole + row.singles();
  for (int i = from; i < to && i < units; i += T) {
    if (i < row.whole) Chunk<DT>::template store<STREAM>(out, row.chunk(i), zeros);
    else Elem<DT>::put(out, row.single(i - row.whole), 0.0f);
  }
}

// ------------------------------------------------------------------- kernels

// What a row's outputs are a function of.
struct RowResult {
  float m, ls, h;
  bool nan;
  // o: the sum of e^t but for one 1; u: the sum of e^t t in powers of 2.
  __device__ __forceinline__ RowResult(float most, float o, float u, bool holds_nan) {
    m = holds_nan ? __builtin_nanf("") : most;
    nan = holds_nan;
    if (!(m < __builtin_inff())) o = __builtin_nanf("");
    ls = log1pf(o);
    h = ls - u * kLn2 / (1.0f + o);
  }
};

// A row's outputs but for its gradient.  y: its target, negative: none.
template <int DT, int T, bool TOP, typename R>
__device__ __forceinline__ void put_row(const LogprobArgs& a, int64_t r, R& row, const Row<DT, T, 0>& memory,
                                        const RowResult& x, int64_t y, float most, RowLds<T>& l) {
  const float m = x.m;
  if (Team<T>::thread() == 0) {
    if (a.logp) a.logp[r] = y < 0 ? 0.0f : m == neg_inf() ? m : (l.target - m) * a.scale - x.ls;
    if (a.stats) {
      a.stats[2 * r] = m;
      a.stats[2 * r + 1] = x.ls;
    }
    if (a.entropy) a.entropy[r] = x.h;
  }
  if (TOP) {
    const auto put = [&](int i, uint64_t key) {
      if (a.top_ids) a.top_ids[r * a.top + i] = (int32_t)key_index(key);
      if (a.top_logp)
        a.top_logp[r * a.top + i] = m == neg_inf() ? m : (of_order((uint32_t)(key >> 32)) - m) * a.scale - x.ls;
    };
    if (x.nan) top_slowly<T>(memory, a.top, l, put);
    else top_of<T>(row, memory, a.top, most, l, put);
    if (a.dlogits.data) Team<T>::sync();  // in logits' place: they have been read
  }
}

template <int DT, int T, bool ENT, bool STREAM, typename R>
__device__ __forceinline__ void put_gradient(const LogprobArgs& a, int64_t r, R& row, const RowResult& x,
                                             const RowLds<T>& l) {
  const RowGradient g(a, r, x.m, x.ls, x.h);
  char* const out = static_cast<char*>(a.dlogits.data) + r * a.dlogits.ld * Chunk<DT>::kSize;
  if (g.none) {
    put_zeros<DT, T, STREAM>(row, out, Team<T>::thread(), INT32_MAX);
    return;
  }
  row.each([&](int first, auto n, float* v) {
    emit_some<DT, ENT, STREAM>(g, out, first, n, n > 1 ? row.chunks_end() : row.vocab, v);
  });
  // by the thread that wrote its place before
  if (g.y < 0) return;
  const int unit = row.unit_of(g.y);
  if (Team<T>::thread() == (unit < row.whole ? unit % T : unit - row.whole))
    Elem<DT>::put(out, g.y, g.at_target(l.target));
}

// No kernel loops over rows: what does not depend on the row would be kept in
// registers across it, as many as the row's own.
template <int DT, int T>
__device__ __forceinline__ int64_t row_of(int64_t r0) {
  return r0 + (int64_t)blockIdx.x * Team<T>::kRows + __builtin_amdgcn_readfirstlane(threadIdx.x / T);
}

// A row's target (negative: none); its logit goes to l.target.
template <int DT, int T>
__device__ __forceinline__ int64_t load_target(const LogprobArgs& a, int64_t r, const char* in, RowLds<T>& l) {
  int64_t y = a.logp || a.dlogp ? token_at(a.targets, r) : -1;
  if (y >= a.vocab) y = -1;
  if (Team<T>::thread() == 0) l.target = y >= 0 ? Elem<DT>::get(in, y) : 0.0f;
  return y;
}

// With the row in registers.  Bound by memory: 8192 x 32000 bf16 with the
// gradient 191 us (1.05 GB, 5.5 TB/s; a pass takes up to 225 where the card comes
// from idling or waits between launches), 4096 x 32000 bf16 without 60 us.  One
// row of 32000 takes 5 us: half of that is arithmetic on one CU.
// (Alternatives take the registers of a second
// workgroup of a CU: forced into half, 2097 x 32001 bf16 with 20 of them takes 69
// us instead of 83, but one row 11.2 instead of 9.6.)
template <int DT, int T, int C, bool ENT, bool TOP>
__global__ void __launch_bounds__(T == 64 ? 256 : T) logprobs_kernel(LogprobArgs a, int64_t r0) {
  __shared__ RowLds<T> all[Team<T>::kRows];
  RowLds<T>& l = all[T == 64 ? threadIdx.x / 64 : 0];
  const float c = a.scale * kLog2e;
  const int64_t r = row_of<DT, T>(r0);
  if (r >= a.rows) return;  // a team as a whole; a workgroup of one team has a row
  const char* const in = static_cast<const char*>(a.logits.data) + r * a.logits.ld * Chunk<DT>::kSize;
  Row<DT, T, C> row(in, a.vocab);
  const int64_t y = load_target<DT, T>(a, r, in, l);

  float most = neg_inf();
  row.each([&](int, auto n, const float* v) {
#pragma unroll
    for (int j = 0; j < n; ++j) most = __builtin_fmaxf(most, v[j]);
  });
  const float m = team_max<T>(most, l);
  const float base = m == neg_inf() ? 0.0f : m;
  // sums of e^t and e^t t (in powers of 2), and the number of logits that are
  // the largest, which only the waves that hold one look for
  float s[3] = {0.0f, 0.0f, 0.0f};
  const bool largest = __any(most == m);
  row.each([&](int, auto n, const float* v) {
    const auto add = [&](auto look) {
#pragma unroll
      for (int j = 0; j < n; ++j) {
        const float x = (v[j] - base) * c;
        float e = __builtin_amdgcn_exp2f(x);
        if (decltype(look)::value) {
          s[2] += v[j] == m ? 1.0f : 0.0f;
          e = v[j] == m ? 0.0f : e;
        }
        s[0] += e;
        if (ENT) s[1] = __builtin_fmaf(e, floored(x), s[1]);
      }
    };
    if (largest) add(std::true_type{});  // a branch a chunk: one around the pass would keep the row twice
    else add(std::false_type{});
  });
  team_sum<T, 3>(s, l.sum);
  if (T == 64) Team<T>::sync();  // the target's logit
  const RowResult x(m, m == neg_inf() ? s[0] : s[0] + (s[2] - 1.0f), s[1], s[0] != s[0]);
  const Row<DT, T, 0> memory(in, a.vocab);
  put_row<DT, T, TOP>(a, r, row, memory, x, y, most, l);
  if (a.dlogits.data) put_gradient<DT, T, ENT, false>(a, r, row, x, l);
}

// With the row passing by: sums relative to the thread's maximum so far, joined
// at the end.  A row whose likeliest word leaves little to the others has the
// thread that holds it sum its logits again without it, since the sum of the
// others next to a 1 has lost digits.
constexpr int kStep = 4;  // chunks of a thread on the way
constexpr float kLittle = 0.25f;

template <int DT, int T, bool ENT, bool TOP>
__global__ void __launch_bounds__(T) logprobs_online_kernel(LogprobArgs a, int64_t r0) {
  __shared__ RowLds<T> l;
  const float c = a.scale * kLog2e;
  const int64_t r = row_of<DT, T>(r0);
  const char* const in = static_cast<const char*>(a.logits.data) + r * a.logits.ld * Chunk<DT>::kSize;
  Row<DT, T, 0> row(in, a.vocab);
  const int64_t y = load_target<DT, T>(a, r, in, l);

  float most = neg_inf(), s = 0.0f, u = 0.0f;
  const auto rebase = [&](float to) {  // the sums relative to another maximum
    const float d = floored((most - to) * c), f = __builtin_amdgcn_exp2f(d);
    if (ENT) u = __builtin_fmaf(s, d, u) * f;
    s *= f;
  };
  const auto join = [&](const float* v, auto n) {
    float top = most;
#pragma unroll
    for (int j = 0; j < n; ++j) top = __builtin_fmaxf(top, v[j]);
    const float base = top == neg_inf() ? 0.0f : top;
    rebase(base);
#pragma unroll
    for (int j = 0; j < n; ++j) {
      const float x = (v[j] - base) * c;
      const float e = __builtin_amdgcn_exp2f(x);
      s += e;
      if (ENT) u = __builtin_fmaf(e, floored(x), u);
    }
    most = top;
  };
  const int t = threadIdx.x;
  for (int i = t; i < row.whole; i += kStep * T) {
    Chunk<DT> x[kStep];
#pragma unroll
    for (int k = 0; k < kStep; ++k) row.Cut<DT>::load(x[k], i + k * T);
#pragma unroll
    for (int k = 0; k < kStep; ++k) {
      float v[Chunk<DT>::N];
      if (i + k * T >= row.whole) x[k].none();
      x[k].unpack(v);
      join(v, Number<Chunk<DT>::N>{});
    }
  }
  const float one = row.get(row.single(t));
  join(&one, Number<1>{});

  const float m = team_max<T>(most, l);
  const float base = m == neg_inf() ? 0.0f : m;
  const float mine = most;
  rebase(base);
  float sum[2] = {s, u};
  team_sum<T, 2>(sum, l.sum);
  float o = m == neg_inf() ? sum[0] : sum[0] - 1.0f;
  bool nan = false;
  if (sum[0] != sum[0]) {  // a NaN, or +inf less +inf
    bool any = false;
    row.each_in_turn([&](int, auto n, const float* v) {
      for (int j = 0; j < n; ++j) any |= v[j] != v[j];
    });
    nan = __syncthreads_or(any);
  } else if (o < kLittle && m > neg_inf()) {
    const uint64_t holds = __ballot(mine == m);
    if ((t & 63) == 0) l.ties[t >> 6] = holds != 0;
    __syncthreads();
    int first = 0;
    while (!l.ties[first]) ++first;
    if (t >> 6 == first && (t & 63) == __builtin_ctzll(holds)) {
      s = 0.0f;
      bool left_out = false;
      row.each_in_turn([&](int, auto n, const float* v) {
        for (int j = 0; j < n; ++j) {
          const bool out = v[j] == m && !left_out;
          left_out |= out;
          s += out ? 0.0f : __builtin_amdgcn_exp2f((v[j] - m) * c);
        }
      });
    }
    float others[1] = {s};
    team_sum<T, 1>(others, l.again);
    o = others[0];
  }
  const RowResult x(m, o, sum[1], nan);
  put_row<DT, T, TOP>(a, r, row, row, x, y, mine, l);
  if (a.dlogits.data) put_gradient<DT, T, ENT, true>(a, r, row, x, l);
}

// The gradient alone: T threads take kBackChunks chunks each of one row.  Bound by
// memory: 1999 x 32000 fp32 75 us (512 MB, a part of them in the caches).
constexpr int kBackChunks = 4;
template <int DT, int T, bool STREAM>
__global__ void __launch_bounds__(kThreads) logprobs_back_kernel(LogprobArgs a, int64_t pieces) {
  const int64_t count = a.rows * pieces;
  constexpr int kTeams = kThreads / T;
  const int team = __builtin_amdgcn_readfirstlane(threadIdx.x / T);
  for (int64_t k = (int64_t)blockIdx.x * kTeams + team; k < count; k += (int64_t)gridDim.x * kTeams) {
    const int64_t i = count - 1 - k;  // the last rows, which the first call read last, are in the caches
    const int64_t r = i / pieces;
    const int i0 = (int)(i - r * pieces) * (kBackChunks * T) + threadIdx.x % T;
    const RowGradient g(a, r, a.stats[2 * r], a.stats[2 * r + 1], a.dentropy ? a.entropy[r] : 0.0f);
    const char* const in = static_cast<const char*>(a.logits.data) + r * a.logits.ld * Chunk<DT>::kSize;
    char* const out = static_cast<char*>(a.dlogits.data) + r * a.dlogits.ld * Chunk<DT>::kSize;
    constexpr int N = Chunk<DT>::N;
    const Cut<DT> row(in, a.vocab);
    if (g.none) {  // of all threads that share the row
      put_zeros<DT, T, STREAM>(row, out, i0, i0 + kBackChunks * T);
      continue;
    }
    // in logits' place the target's is read before its chunk is written, by the same thread
    const int unit = row.unit_of(g.y);
    const bool mine = g.y >= 0 && unit >= i0 && (unit - i0) % T == 0 && unit - i0 < kBackChunks * T;
    const float target = mine ? Elem<DT>::get(in, g.y) : 0.0f;
    const auto emit = [&](auto with_entropy) {
      constexpr bool ent = decltype(with_entropy)::value;
      Chunk<DT> x[kBackChunks];
#pragma unroll
      for (int k = 0; k < kBackChunks; ++k) {
        const int n = i0 + k * T;
        if (row.whole > 0) row.load(x[k], n);
      }
#pragma unroll
      for (int k = 0; k < kBackChunks; ++k) {
        const int n = i0 + k * T;  // a chunk, or behind them a single logit
        float v[N];
        if (n < row.whole) {
          x[k].unpack(v);
          emit_some<DT, ent, STREAM>(g, out, row.chunk(n), Number<N>{}, row.vocab, v);
        } else if (n - row.whole < row.singles()) {
          const int i = row.single(n - row.whole);
          v[0] = Elem<DT>::get(in, i);
          emit_some<DT, ent, STREAM>(g, out, i, Number<1>{}, row.vocab, v);
        }
      }
    };
    if (a.dentropy) emit(std::true_type{});
    else emit(std::false_type{});
    if (mine) Elem<DT>::put(out, g.y, g.at_target(target));
  }
}

constexpr int64_t kLaunchRows = int64_t(1) << 21;  // a launch has less than 2^32 threads

unsigned capped(int64_t blocks) { return (unsigned)(blocks > (1 << 21) ? 1 << 21 : blocks); }

// C 0: the row passes by.
template <int DT, int T, int C, bool ENT, bool TOP>
void launch(const LogprobArgs& a, dim3 grid, int64_t r0, hipStream_t s) {
  if constexpr (C > 0) logprobs_kernel<DT, T, C, ENT, TOP><<<grid, T == 64 ? 256 : T, 0, s>>>(a, r0);
  else logprobs_online_kernel<DT, T, ENT, TOP><<<grid, T, 0, s>>>(a, r0);
}

template <int DT, int T, int C>
void run(const LogprobArgs& a, hipStream_t s) {
  constexpr int kRows = Team<T>::kRows;
  const bool ent = a.entropy || a.dentropy;
  for (int64_t r0 = 0; r0 < a.rows; r0 += kLaunchRows) {
    const int64_t rows = a.rows - r0 < kLaunchRows ? a.rows - r0 : kLaunchRows;
    const dim3 grid((unsigned)((rows + kRows - 1) / kRows));
    if (a.top && ent) launch<DT, T, C, true, true>(a, grid, r0, s);
    else if (a.top) launch<DT, T, C, false, true>(a, grid, r0, s);
    else if (ent) launch<DT, T, C, true, false>(a, grid, r0, s);
    else launch<DT, T, C, false, false>(a, grid, r0, s);
  }
}

template <int DT>
void run_type(const LogprobArgs& a, hipStream_t s) {
  const int64_t v = a.vocab;
  // As few threads a row as hold it in 16 registers each (32 for fp32, and for
  // 16 bits past 32768 logits), so that a CU has two rows or more.  Longer rows
  // pass by: 1335 x 50257 fp32 49 us, in 64 registers 65; 1023 x 65537 bf16 34
  // against 42; with the gradient 65 against 69, though they are read twice.
  constexpr int W = DT == SCAPE_F32 ? 2 : 1;  // chunks of 8 logits
  if (v <= 64 * 8) run<DT, 64, W>(a, s);
  else if (v <= 64 * 32) run<DT, 64, 4 * W>(a, s);
  else if (v <= 256 * 32) run<DT, 256, 4 * W>(a, s);
  else if (v <= 512 * 32) run<DT, 512, 4 * W>(a, s);
  else if (v <= 1024 * 32) run<DT, 1024, 4 * W>(a, s);
  else if (W == 1 && v <= 1024 * 64) run<DT, 1024, W == 1 ? 8 : 0>(a, s);
  else run<DT, 1024, 0>(a, s);
}

template <int DT, int T>
void run_back(const LogprobArgs& a, bool stream, hipStream_t s) {
  constexpr int N = Chunk<DT>::N;
  const int64_t units = a.vocab / N + 2 * N;  // chunks and single logits, at most
  const int64_t pieces = (units + kBackChunks * T - 1) / (kBackChunks * T);
  const dim3 grid(capped((a.rows * pieces + kThreads / T - 1) / (kThreads / T)));
  if (stream) logprobs_back_kernel<DT, T, true><<<grid, kThreads, 0, s>>>(a, pieces);
  else logprobs_back_kernel<DT, T, false><<<grid, kThreads, 0, s>>>(a, pieces);
}

template <int DT>
void run_back(const LogprobArgs& a, bool stream, hipStream_t s) {
  if (a.vocab <= 64 * 16) run_back<DT, 64>(a, stream, s);  // a wave a row
  else run_back<DT, kThreads>(a, stream, s);
}

}  // namespace

hipError_t launch_logprobs(const LogprobArgs& a, hipStream_t s) {
  if (a.rows == 0) return hipSuccess;
  if (a.logits.dtype == SCAPE_F32) run_type<SCAPE_F32>(a, s);
  else if (a.logits.dtype == SCAPE_BF16) run_type<SCAPE_BF16>(a, s);
  else run_type<SCAPE_F16>(a, s);
  return hipGetLastError();
}

hipError_t launch_logprobs_backward(const LogprobArgs& a, hipStream_t s) {
  if (a.rows == 0) return hipSuccess;
  // What the first call read is still in the caches: past them, dlogits does
  // not drive it out.  1999 x 32000 fp32, both calls: 121 us, without it 152.
  // The call that does both keeps dlogits in the caches, for the products that
  // read it next: 1024 x 32000 bf16 and one product of it 49.7 us, with stores
  // past the caches 55.2.  Where it is more than they hold these would win: 8192
  // x 32000 191 either way alone, with the product 302 and 284; 4096 x 50257 159
  // and 154, 241 and 236.
  const bool stream = 2 * a.rows * a.vocab * (int64_t)dtype_bytes(a.logits.dtype) > kStreamBytes;
  if (a.logits.dtype == SCAPE_F32) run_back<SCAPE_F32>(a, stream, s);
  else if (a.logits.dtype == SCAPE_BF16) run_back<SCAPE_BF16>(a, stream, s);
  else run_back<SCAPE_F16>(a, stream, s);
  return hipGetLastError();
}

}  // namespace scape
