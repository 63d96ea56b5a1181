// Log probabilities of given tokens, entropy, the likeliest alternatives, and
// the gradient of the logits.
//
// With m the largest logit, t = scale (x - m) and o the sum of e^t over all
// words but one of the likeliest: logp = t_y - log(1 + o), entropy = log(1 + o)
// - sum(e^t t) / (1 + o), and the gradient is a function of each logit alone.
// A row is read once, into registers, where the maximum, the sums, the
// alternatives and the gradient take it from; only rows too long for the
// registers of a workgroup are read again, from the caches.
#include "ends.h"

#include <type_traits>

namespace scape {
namespace {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.693147180559945309417f;
constexpr int kCandidates = 512;  // logits that compete for a row's alternatives, at most

__device__ __forceinline__ float neg_inf() { return -__builtin_inff(); }

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
  float value[3][Team<T>::kWaves];
  uint64_t key[Team<T>::kWaves];
  uint32_t order[T];
  uint64_t cand[kCandidates];
  uint32_t n, ties[Team<T>::kWaves];
  float target;
};

__device__ __forceinline__ float wave_max(float x) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) x = __builtin_fmaxf(x, __shfl_xor(x, d, 64));
  return x;
}

template <int T>
__device__ __forceinline__ float team_max(float x, RowLds<T>& l) {
  x = wave_max(x);
  if (T == 64) return x;
  if ((threadIdx.x & 63) == 0) l.value[0][threadIdx.x >> 6] = x;
  __syncthreads();
  x = l.value[0][0];
#pragma unroll
  for (int w = 1; w < Team<T>::kWaves; ++w) x = __builtin_fmaxf(x, l.value[0][w]);
  return x;
}

template <int T, int N>
__device__ __forceinline__ void team_sum(float (&x)[N], RowLds<T>& l) {
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = wave_sum(x[i]);
  if (T == 64) return;
  __syncthreads();  // the maxima have been read
  if ((threadIdx.x & 63) == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) l.value[i][threadIdx.x >> 6] = x[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    x[i] = l.value[i][0];
#pragma unroll
    for (int w = 1; w < Team<T>::kWaves; ++w) x[i] += l.value[i][w];
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
// A thread's chunks of 8 logits, and one of the up to 7 logits behind the last
// whole chunk.  each(f) calls f(first, n, v) for them with the index of the
// first and their number, 8 or 1 (a constant where f is inlined); a chunk past
// the row is -inf.
template <int DT>
struct Chunk {
  static constexpr int kSize = DT == SCAPE_F32 ? 4 : 2;
  static constexpr int kWords = 2 * kSize;
  uint32_t u[kWords];
  // A row begins at `row`, the same for all threads that share it.
  __device__ __forceinline__ void load(const char* row, int first) {
    const char* p = row + (uint32_t)first * (uint32_t)kSize;
    load16<false>(u, p);
    if (kWords == 8) load16<false>(u + kWords / 2, p + 16);
  }
  __device__ __forceinline__ void unpack(float (&v)[8]) const {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (DT == SCAPE_F32) v[j] = __uint_as_float(u[j % kWords]);
      else if (DT == SCAPE_BF16) v[j] = __uint_as_float((j & 1) ? u[j / 2] & 0xffff0000u : u[j / 2] << 16);
      else v[j] = (float)__builtin_bit_cast(_Float16, (uint16_t)(u[j / 2] >> (16 * (j & 1))));
    }
  }
  __device__ __forceinline__ void none() {
#pragma unroll
    for (int k = 0; k < kWords; ++k)
      u[k] = DT == SCAPE_F32 ? 0xff800000u : DT == SCAPE_BF16 ? 0xff80ff80u : 0xfc00fc00u;
  }
  __device__ __forceinline__ void keep() {
#pragma unroll
    for (int k = 0; k < kWords; ++k) asm volatile("" : "+v"(u[k]));
  }
};

// C chunks in registers.
template <int DT, int T, int C>
struct Row {
  Chunk<DT> r[C];
  float tail;
  int whole;  // chunks of the row
  int vocab;
  __device__ __forceinline__ void load(const char* row, int cols) {
    vocab = cols;
    whole = cols / 8;
    const int t = Team<T>::thread();
    tail = whole * 8 + t < cols ? Elem<DT>::get(row, whole * 8 + t) : neg_inf();
    if (whole == 0) {
#pragma unroll
      for (int i = 0; i < C; ++i) r[i].none();
      return;
    }
    // a chunk past the row is the last one, loaded and dropped: no branch,
    // behind which the loads under way would be waited for
#pragma unroll
    for (int i = 0; i < C; ++i) r[i].load(row, (index(i) < whole ? index(i) : whole - 1) * 8);
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
      float v[8];
      r[i].keep();
      r[i].unpack(v);
      f(index(i) * 8, 8, v);
      __builtin_amdgcn_sched_barrier(0);
    }
    f(whole * 8 + Team<T>::thread(), 1, &tail);
  }
};

// Read from memory each time.
template <int DT, int T>
struct Row<DT, T, 0> {
  const char* p;
  int whole, vocab;
  __device__ __forceinline__ void load(const char* row, int cols) {
    p = row;
    vocab = cols;
    whole = cols / 8;
  }
  __device__ __forceinline__ float get(int i) const { return Elem<DT>::get(p, i); }
  template <int U = 4, typename F>
  __device__ __forceinline__ void each(F f) const {
    const int t = Team<T>::thread();
#pragma unroll U
    for (int i = t; i < whole; i += T) {
      Chunk<DT> x;
      float v[8];
      x.load(p, i * 8);
      x.unpack(v);
      f(i * 8, 8, v);
    }
    float last = whole * 8 + t < vocab ? Elem<DT>::get(p, whole * 8 + t) : neg_inf();
    f(whole * 8 + t, 1, &last);
  }
};

// -------------------------------------------------------------- alternatives

// Calls f(rank, key) for the `top` largest keys of any row, in a pass for each.
template <int T, typename M, typename F>
__device__ __forceinline__ void top_slowly(const M& memory, int top, RowLds<T>& l, F f) {
  uint64_t last = ~0ull;
  for (int i = 0; i < top; ++i) {
    uint64_t best = 0;
    memory.template each<1>([&](int first, int n, const float* v) {
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
  uint32_t p = 0;
  for (int s = 31; s >= 32 - bits; --s) {
    const uint32_t q = p | 1u << s;
    if (__popcll(__ballot(a >= q)) + __popcll(__ballot(b >= q)) >= k) p = q;
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
  const auto collect = [&](auto& from, float bound, bool equal) {
    Team<T>::sync();
    if (t == 0) l.n = 0;
    Team<T>::sync();
    const auto some = [&](int first, int n, const float* v) {
      uint32_t mask = 0;  // a bit for each logit that reaches the bound
#pragma unroll
      for (int j = 0; j < n; ++j) mask |= (equal ? v[j] >= bound : v[j] > bound) ? 1u << j : 0u;
      for (; mask; mask &= mask - 1) {
        const int i = first + __builtin_ctz(mask);
        if (i >= (n == 8 ? memory.whole * 8 : memory.vocab)) break;  // a -inf that stands for none
        const uint32_t at = atomicAdd(&l.n, 1u);  // of LDS; the ranks do not depend on the places
        if (at < kCandidates) l.cand[at] = key_of(memory.get(i), (uint32_t)i);
      }
    };
    from.each(some);
    Team<T>::sync();
    return l.n;
  };
  const auto rank = [&](uint32_t n) {
    for (uint32_t i = t; i < n; i += T) {
      const uint64_t k = l.cand[i];
      int r = 0;
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
  const bool enough = (row.vocab + 7) / 8 >= top;
  const auto bound_of = [&](int bits) {
    const uint32_t p = enough ? kth_prefix(a, b, top, bits) : 0;
    return p <= kOrderNegInf ? neg_inf() : of_order(p);
  };
  uint32_t n = collect(row, bound_of(20), true);
  if (n <= kCandidates) {
    rank(n);
    return;
  }
  const float bound = bound_of(32);
  n = collect(memory, bound, false);
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
  template <bool ENT>
  __device__ __forceinline__ void of(float* v, int n) const {
#pragma unroll
    for (int j = 0; j < n; ++j) {
      float l = __builtin_fmaf(v[j] - m, c, -ls2);  // log2 of the probability
      if (ENT) {
        l = __builtin_fmaxf(l, -256.0f);  // of probability 0: nothing, not 0 times -inf
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
template <int DT, bool ENT>
__device__ __forceinline__ void emit_some(const RowGradient& g, char* out, int first, int n, int vocab, float* v) {
  if (first >= vocab) return;
  if (g.none) {
#pragma unroll
    for (int j = 0; j < n; ++j) v[j] = 0.0f;
  } else {
    g.of<ENT>(v, n);
  }
  if (n == 8) Elem<DT>::store(out + (uint32_t)first * (uint32_t)Chunk<DT>::kSize, 0, *reinterpret_cast<float(*)[8]>(v));
  else Elem<DT>::put(out, first, v[0]);
}

// ------------------------------------------------------------------- kernels

template <int DT, int T, int C, bool ENT, bool TOP>
__global__ void __launch_bounds__(T == 64 ? 256 : T) logprobs_kernel(LogprobArgs a, int64_t r0) {
  __shared__ RowLds<T> all[Team<T>::kRows];
  RowLds<T>& l = all[T == 64 ? threadIdx.x / 64 : 0];
  const int t = Team<T>::thread();
  const float c = a.scale * kLog2e;
  // no loop over rows: what does not depend on the row would be kept in
  // registers across it, as many as the row's own
  const int64_t r = r0 + (int64_t)blockIdx.x * Team<T>::kRows + __builtin_amdgcn_readfirstlane(threadIdx.x / T);
  if (r >= a.rows) return;  // a team as a whole; a workgroup of one team has a row
  const char* const in = static_cast<const char*>(a.logits.data) + r * a.logits.ld * Chunk<DT>::kSize;
  Row<DT, T, C> row;
  row.load(in, (int)a.vocab);
  int64_t y = a.logp || a.dlogp ? token_at(a.targets, r) : -1;
  if (y >= a.vocab) y = -1;
  if (t == 0) l.target = y >= 0 ? Elem<DT>::get(in, y) : 0.0f;

  float most = neg_inf();
  row.each([&](int, int n, const float* v) {
#pragma unroll
    for (int j = 0; j < n; ++j) most = __builtin_fmaxf(most, v[j]);
  });
  float m = team_max<T>(most, l);
  const float base = m == neg_inf() ? 0.0f : m;
  // sums of e^t and e^t t (in powers of 2), and the number of logits that are
  // the largest, which only the waves that hold one look for
  float s[3] = {0.0f, 0.0f, 0.0f};
  const bool largest = __any(most == m);
  row.each([&](int, int n, const float* v) {
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
        if (ENT) s[1] = __builtin_fmaf(e, __builtin_fmaxf(x, -256.0f), s[1]);
      }
    };
    if (largest) add(std::true_type{});  // a branch a chunk: one around the pass would keep the row twice
    else add(std::false_type{});
  });
  team_sum<T, 3>(s, l);
  if (T == 64) Team<T>::sync();  // the target's logit
  const bool nan = s[0] != s[0];
  float o = m == neg_inf() ? s[0] : s[0] + (s[2] - 1.0f);
  if (m == __builtin_inff()) o = __builtin_nanf("");
  if (nan) m = __builtin_nanf("");
  const float ls = log1pf(o);
  const float h = ls - s[1] * kLn2 / (1.0f + o);
  if (t == 0) {
    if (a.logp) a.logp[r] = y < 0 ? 0.0f : m == neg_inf() ? m : (l.target - m) * a.scale - ls;
    if (a.stats) {
      a.stats[2 * r] = m;
      a.stats[2 * r + 1] = ls;
    }
    if (a.entropy) a.entropy[r] = h;
  }
  if (TOP) {
    const auto put = [&](int i, uint64_t key) {
      if (a.top_ids) a.top_ids[r * a.top + i] = (int32_t)key_index(key);
      if (a.top_logp)
        a.top_logp[r * a.top + i] = m == neg_inf() ? m : (of_order((uint32_t)(key >> 32)) - m) * a.scale - ls;
    };
    Row<DT, T, 0> memory;
    memory.load(in, (int)a.vocab);
    if (nan) top_slowly<T>(memory, a.top, l, put);
    else top_of<T>(row, memory, a.top, most, l, put);
    if (a.dlogits.data) Team<T>::sync();  // in logits' place: they have been read
  }
  if (a.dlogits.data) {
    const RowGradient g(a, r, m, ls, h);
    char* const out = static_cast<char*>(a.dlogits.data) + r * a.dlogits.ld * Chunk<DT>::kSize;
    row.each([&](int first, int n, float* v) {
      emit_some<DT, ENT>(g, out, first, n, n == 8 ? row.whole * 8 : row.vocab, v);
    });
    // by the thread that wrote its place before
    const int owner = g.y / 8 < row.whole ? g.y / 8 % T : g.y - row.whole * 8;
    if (!g.none && g.y >= 0 && t == owner) Elem<DT>::put(out, g.y, g.at_target(l.target));
  }
}

// The gradient alone: a workgroup takes kBackChunks chunks a thread of one row.
constexpr int kBackChunks = 4;
template <int DT>
__global__ void __launch_bounds__(kThreads) logprobs_back_kernel(LogprobArgs a, int64_t pieces) {
  const int64_t count = a.rows * pieces;
  for (int64_t i = blockIdx.x; i < count; i += gridDim.x) {
    const int64_t r = i / pieces;
    const int i0 = (int)(i - r * pieces) * (kBackChunks * kThreads) + threadIdx.x;
    const RowGradient g(a, r, a.stats[2 * r], a.stats[2 * r + 1], a.dentropy ? a.entropy[r] : 0.0f);
    const char* const in = static_cast<const char*>(a.logits.data) + r * a.logits.ld * Chunk<DT>::kSize;
    char* const out = static_cast<char*>(a.dlogits.data) + r * a.dlogits.ld * Chunk<DT>::kSize;
    const int vocab = (int)a.vocab, whole = vocab / 8;
    // in logits' place the target's is read before its chunk is written, by the same thread
    const int owner = g.y / 8 < whole ? g.y / 8 : whole + (g.y & 7);
    const bool mine = !g.none && g.y >= 0 && owner >= i0 && (owner - i0) % kThreads == 0 &&
                      owner - i0 < kBackChunks * kThreads;
    const float target = mine ? Elem<DT>::get(in, g.y) : 0.0f;
    const auto emit = [&](auto with_entropy) {
      constexpr bool ent = decltype(with_entropy)::value;
      Chunk<DT> x[kBackChunks];
#pragma unroll
      for (int k = 0; k < kBackChunks; ++k) {
        const int n = i0 + k * kThreads;
        if (whole > 0) x[k].load(in, (n < whole ? n : whole - 1) * 8);
      }
#pragma unroll
      for (int k = 0; k < kBackChunks; ++k) {
        const int n = i0 + k * kThreads;  // a chunk, or behind them one of the last logits
        float v[8];
        if (n < whole) {
          x[k].unpack(v);
          emit_some<DT, ent>(g, out, n * 8, 8, vocab, v);
        } else if (whole * 8 + (n - whole) < vocab) {
          v[0] = Elem<DT>::get(in, whole * 8 + (n - whole));
          emit_some<DT, ent>(g, out, whole * 8 + (n - whole), 1, vocab, v);
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

template <int DT, int T, int C>
void run(const LogprobArgs& a, hipStream_t s) {
  constexpr int kRows = Team<T>::kRows;
  const dim3 block(T == 64 ? 256 : T);
  const bool ent = a.entropy || a.dentropy;
  for (int64_t r0 = 0; r0 < a.rows; r0 += kLaunchRows) {
    const int64_t rows = a.rows - r0 < kLaunchRows ? a.rows - r0 : kLaunchRows;
    const dim3 grid((unsigned)((rows + kRows - 1) / kRows));
    if (a.top && ent) logprobs_kernel<DT, T, C, true, true><<<grid, block, 0, s>>>(a, r0);
    else if (a.top) logprobs_kernel<DT, T, C, false, true><<<grid, block, 0, s>>>(a, r0);
    else if (ent) logprobs_kernel<DT, T, C, true, false><<<grid, block, 0, s>>>(a, r0);
    else logprobs_kernel<DT, T, C, false, false><<<grid, block, 0, s>>>(a, r0);
  }
}

// As few threads a row as hold it in registers, 64 logits each at most.
template <int DT>
void run_type(const LogprobArgs& a, hipStream_t s) {
  const int64_t v = a.vocab;
  if (v <= 64 * 8) run<DT, 64, 1>(a, s);
  else if (v <= 64 * 32) run<DT, 64, 4>(a, s);
  else if (v <= 256 * 32) run<DT, 256, 4>(a, s);
  else if (v <= 512 * 64) run<DT, 512, 8>(a, s);
  else if (v <= 1024 * 64) run<DT, 1024, 8>(a, s);
  else if (DT != SCAPE_F32 && v <= 1024 * 128) run<DT, 1024, DT == SCAPE_F32 ? 0 : 16>(a, s);
  else run<DT, 1024, 0>(a, s);
}

}  // namespace

size_t logprobs_workspace(int64_t, int64_t, int) { return 256; }

hipError_t launch_logprobs(const LogprobArgs& a, void*, hipStream_t s) {
  if (a.rows == 0) return hipSuccess;
  if (a.logits.dtype == SCAPE_F32) run_type<SCAPE_F32>(a, s);
  else if (a.logits.dtype == SCAPE_BF16) run_type<SCAPE_BF16>(a, s);
  else run_type<SCAPE_F16>(a, s);
  return hipGetLastError();
}

hipError_t launch_logprobs_backward(const LogprobArgs& a, hipStream_t s) {
  if (a.rows == 0) return hipSuccess;
  const int64_t units = a.vocab / 8 + a.vocab % 8;  // chunks and single logits
  const int64_t pieces = (units + kBackChunks * kThreads - 1) / (kBackChunks * kThreads);
  const dim3 grid(capped(a.rows * pieces));
  if (a.logits.dtype == SCAPE_F32) logprobs_back_kernel<SCAPE_F32><<<grid, kThreads, 0, s>>>(a, pieces);
  else if (a.logits.dtype == SCAPE_BF16) logprobs_back_kernel<SCAPE_BF16><<<grid, kThreads, 0, s>>>(a, pieces);
  else logprobs_back_kernel<SCAPE_F16><<<grid, kThreads, 0, s>>>(a, pieces);
  return hipGetLastError();
}

}  // namespace scape
