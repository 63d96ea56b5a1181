// Rows of an embedding table by token, and the table's gradient.
#include "ends.h"

namespace scape {
namespace {

struct EmbedArgs {
  int64_t tokens, vocab, positions, cols;
  scape_ids ids, pos;
  const void* table;
  int64_t table_ld;
  const void* pos_table;
  int64_t pos_ld;
  float scale;
  void* out;
  int64_t out_ld;
};

// out[t] = scale * table[ids[t]] + pos_table[pos[t]]: one read and one write,
// bound by memory: 16384 tokens of 32000 x 2048, fp32 to bf16, tables that change
// from pass to pass: 28 us, 81 MB of rows read and 67 written (5.3 TB/s).  `lanes`
// (a power of two) threads share a token.
template <int TT, int OT>
__global__ void __launch_bounds__(kThreads) embed_kernel(EmbedArgs a, int lanes) {
  const int per = kThreads / lanes;
  for (int64_t t = (int64_t)blockIdx.x * per + threadIdx.x / lanes; t < a.tokens; t += (int64_t)gridDim.x * per) {
    const int64_t id = token_at(a.ids, t);
    const int64_t at = a.pos_table ? token_at(a.pos, t) : -1;
    for (int64_t c = (threadIdx.x & (lanes - 1)) * 8; c < a.cols; c += lanes * 8) {
      float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
      if (id >= 0 && id < a.vocab) load8<TT>(a.table, id * a.table_ld, c, a.cols, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= a.scale;
      if (at >= 0 && at < a.positions) {
        float p[8];
        load8<TT>(a.pos_table, at * a.pos_ld, c, a.cols, p);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] += p[j];
      }
      store8<OT>(a.out, t * a.out_ld, c, a.cols, v);
    }
  }
}

// ----------------------------------------------------------------- gradient
//
// The tokens are sorted by word, equal words by token, and cut into chunks of
// the sorted order, so that the work of a chunk does not depend on how often a
// word occurs.  A chunk sums the rows of each word in it, in their order: a
// word that begins and ends in the chunk goes to the table, one that crosses
// its border to a partial row, and the partial rows of a word are joined in
// order.  No atomics: the sums are the same every time.

constexpr uint32_t kNoWord = 0xfffffffeu;  // above every word, and 1 more is no overflow
constexpr int kSortTile = 512;             // tokens that are sorted by counting
constexpr int kBatch = 8;                  // rows of dy on the way at a time

struct SortArgs {
  int64_t tokens, vocab;
  const void* ids;
  int tile;       // a power of two, at least 64
  int lanes;      // that count for one token
  uint32_t* word;  // [tiles * tile], each tile sorted
  uint32_t* token;
};

// Sorts tiles by counting: a token's place is the number of tokens of its tile
// that come before it.  The comparisons do not wait for each other and spread
// over the card: 6 us, where exchanges in one workgroup took 20 us for tiles of
// 2048.  (Counting in larger tiles: 10 us at 2048, 22 us at 8192.)
template <typename I>
__global__ void __launch_bounds__(kThreads) embed_sort_kernel(SortArgs a) {
  extern __shared__ uint32_t lds[];
  const int per = kThreads / a.lanes;      // tokens of a workgroup
  const int parts = a.tile / per;          // workgroups of a tile
  const int64_t t0 = (int64_t)(blockIdx.x / parts) * a.tile;
  // eight loads on the way at a time; past the end, the last token's word again
  for (int i0 = threadIdx.x; i0 < a.tile; i0 += 8 * kThreads) {
    int64_t id[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int64_t t = t0 + i0 + j * kThreads;
      id[j] = token_at<I>(a.ids, t < a.tokens ? t : a.tokens - 1);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int i = i0 + j * kThreads;
      if (i < a.tile) lds[i] = t0 + i < a.tokens && id[j] >= 0 && id[j] < a.vocab ? (uint32_t)id[j] : kNoWord;
    }
  }
  __syncthreads();
  const int p = (int)(blockIdx.x % parts) * per + threadIdx.x / a.lanes;
  const uint32_t w = lds[p];
  // tokens in front of p come before it if their word is at most w, those
  // behind it if it is below w; four at a time, p's own four as if behind it
  uint32_t place = 0;
  const int l = threadIdx.x & (a.lanes - 1);
#pragma unroll 4
  for (int q = l; q < a.tile / 4; q += a.lanes) {
    const u32x4 k = *reinterpret_cast<const u32x4*>(lds + 4 * q);
    const uint32_t bound = w + (4 * q + 3 < p ? 1u : 0u);
    place += (k[0] < bound) + (k[1] < bound) + (k[2] < bound) + (k[3] < bound);
  }
  for (int d = a.lanes >> 1; d >= 1; d >>= 1) place += __shfl_xor((int)place, d, 64);
  for (int i = p & ~3; i < p; ++i) place += lds[i] == w;
  if (l == 0) {
    a.word[t0 + place] = w;
    a.token[t0 + place] = (uint32_t)t0 + (uint32_t)p;
  }
}

// Sorts by slabs of the vocabulary, in one launch: a workgroup owns `slab`
// words and goes through all tokens.  Its waves take a stretch of them each,
// list those of the slab in LDS and count them by word; a token's place is the
// number of tokens of lower words, of the same word in the stretches before,
// and of the same word before it in its own.  Where a list has no room for all
// of a stretch, the waves go through it a second time instead.
constexpr int kSlabThreads = 1024;
constexpr int kSlabWaves = kSlabThreads / 64;
constexpr int kSlabMax = 512;
// LDS for counts and lists: a CU's 160 KB, less 8 for what else the kernel holds.
// 32000 words x 64, all of the call, with lists and with a second walk: 20000
// tokens 24.3 and 32.7 us, 36000 tokens 29.4 and 45.1; 131072 words, 30000 tokens
// 29.2 and 41.6.
constexpr int64_t kSlabLds = 152 << 10;
constexpr int64_t kSlabs = 1024;                 // workgroups at most: each goes through all tokens
constexpr int64_t kSlabWork = int64_t(1) << 28;  // tokens that they go through in all, at most
constexpr int kAhead = 8;                        // tokens of a lane on the way at a time

struct SlabArgs {
  int64_t tokens, vocab, padded;
  const void* ids;
  int slab;        // words of a workgroup, at most kSlabMax
  int stretch;     // tokens of a wave, a multiple of 64
  uint32_t* word;  // [padded]
  uint32_t* token;
};

// The word of a token number, or one above every word.
__device__ __forceinline__ uint32_t word_of(int64_t id) { return (uint64_t)id >> 32 ? kNoWord : (uint32_t)id; }
__device__ __forceinline__ uint32_t word_of(int32_t id) { return id < 0 ? kNoWord : (uint32_t)id; }

__device__ __forceinline__ uint32_t lanes_below(uint64_t mask) {
  return __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0u));
}

template <typename I, bool LIST>
__global__ void __launch_bounds__(kSlabThreads) embed_slab_kernel(SlabArgs a) {
  extern __shared__ uint32_t lds[];  // [kSlabWaves][slab] counts, then places; [kSlabWaves][stretch] lists
  __shared__ uint32_t first[kSlabThreads], wave_lower[kSlabWaves], wave_total[kSlabWaves];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const uint32_t lo = blockIdx.x * (uint32_t)a.slab;
  const uint32_t words = (uint32_t)(a.vocab - lo < a.slab ? a.vocab - lo : a.slab);
  uint32_t* const mine = lds + wave * a.slab;
  uint32_t* const list = lds + kSlabWaves * a.slab + wave * a.stretch;
  for (int i = lane; i < a.slab; i += 64) mine[i] = 0;
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");

  const int64_t from = (int64_t)wave * a.stretch;
  const int64_t left = a.tokens - from;
  const int own = (int)(left < a.stretch ? left : a.stretch);  // not positive: none
  const I* const ids = static_cast<const I*>(a.ids) + from;
  // Calls f(word, place in the stretch) for the stretch, 64 tokens at a time.
  const auto walk = [&](auto f) {
    for (int t0 = lane; t0 - lane < own; t0 += 64 * kAhead) {
      I id[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int t = t0 + j * 64;
        id[j] = ids[t < own ? t : own - 1];
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int t = t0 + j * 64;
        f(t < own ? word_of(id[j]) : kNoWord, t);
      }
    }
  };
  uint32_t lower = 0, listed = 0;
  walk([&](uint32_t w, int t) {
    const uint32_t r = w - lo;
    lower += w < lo ? 1 : 0;
    const uint64_t in = __ballot(r < words);
    if (in) {
      if (r < words) {
        if (LIST) list[listed + lanes_below(in)] = r << 16 | (uint32_t)t;
        atomicAdd(&mine[r], 1u);  // of LDS; a sum of ones has no order
      }
      listed += (uint32_t)__popcll(in);
    }
  });
  lower = wave_sum(lower);
  if (lane == 0) wave_lower[wave] = lower;
  __syncthreads();
  // a word's tokens, the waves' shares of them, then the words before it
  uint32_t sum = 0;
  if (threadIdx.x < (unsigned)a.slab) {
    for (int w = 0; w < kSlabWaves; ++w) {
      const uint32_t n = lds[w * a.slab + threadIdx.x];
      lds[w * a.slab + threadIdx.x] = sum;
      sum += n;
    }
  }
  uint32_t scan = sum;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t y = __shfl_up(scan, d, 64);
    if (lane >= d) scan += y;
  }
  if (lane == 63) wave_total[wave] = scan;
  __syncthreads();
  uint32_t base = 0, end = 0;
  for (int w = 0; w < kSlabWaves; ++w) {
    base += wave_lower[w] + (w < wave ? wave_total[w] : 0);
    end += wave_lower[w] + wave_total[w];
  }
  first[threadIdx.x] = base + scan - sum;
  __syncthreads();

  // Places up to 64 tokens of the slab in their order; r: none of its words.
  const auto place = [&](uint32_t r, uint32_t t) {
    for (uint64_t open = __ballot(r < words); open;) {
      const uint32_t x = (uint32_t)__builtin_amdgcn_readlane((int)r, __builtin_ctzll(open));
      const uint64_t same = __ballot(r == x);
      open &= ~same;
      const uint32_t at = first[x] + mine[x] + lanes_below(same);
      if (r == x) {
        a.word[at] = lo + x;
        a.token[at] = t;
      }
      if (lane == 0) mine[x] += (uint32_t)__popcll(same);
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    }
  };
  if (LIST) {
    for (uint32_t i0 = 0; i0 < listed; i0 += 64) {
      const uint32_t e = i0 + lane < listed ? list[i0 + lane] : 0xffffffffu;
      place(e >> 16, (uint32_t)from + (e & 0xffffu));
    }
  } else if (listed) {
    walk([&](uint32_t w, int t) { place(w - lo, (uint32_t)from + (uint32_t)t); });
  }
  if (blockIdx.x == gridDim.x - 1)  // the places behind the last word's
    for (int64_t i = end + threadIdx.x; i < a.padded; i += kSlabThreads) {
      a.word[i] = kNoWord;
      a.token[i] = 0;
    }
}

// Number of elements of a sorted run below w (or not above it).
__device__ __forceinline__ int64_t below(const uint32_t* run, int64_t n, uint32_t w, bool equal) {
  int64_t lo = 0;
  while (n > 0) {
    const int64_t half = n >> 1;
    const uint32_t x = run[lo + half];
    const bool right = x < w || (equal && x == w);
    lo += right ? half + 1 : 0;
    n = right ? n - half - 1 : half;
  }
  return lo;
}

// Joins kFan sorted runs of `run` elements (the last of all may be shorter)
// into one: an element's place is its place in its own run plus the number of
// elements of every other run before it.  `lanes` lanes (a power of two) look
// it up in a run each at a time.
constexpr int kFan = 64;
__global__ void __launch_bounds__(kThreads)
embed_merge_kernel(const uint32_t* word, const uint32_t* token, int64_t n, int64_t run, int lanes, uint32_t* out_word,
                   uint32_t* out_token) {
  const int l = threadIdx.x & (lanes - 1);
  const int64_t step = (int64_t)gridDim.x * (kThreads / lanes);
  for (int64_t i = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / lanes; i < n; i += step) {
    const uint32_t w = word[i];
    const int64_t base = i / (run * kFan) * (run * kFan);
    int64_t place = 0;
    for (int j = l; j < kFan; j += lanes) {
      const int64_t r0 = base + j * run;
      if (r0 >= n) break;
      if (i >= r0 && i < r0 + run) place += i - r0;
      else place += below(word + r0, n - r0 < run ? n - r0 : run, w, r0 < i);
    }
    for (int d = lanes >> 1; d >= 1; d >>= 1) place += __shfl_xor((long long)place, d, 64);
    if (l == 0) {
      out_word[base + place] = w;
      out_token[base + place] = token[i];
    }
  }
}

struct ChunkArgs {
  int64_t cols;
  const uint32_t* word;   // sorted, [chunks * chunk]
  const uint32_t* token;
  int chunk;              // a multiple of kBatch
  int32_t chunks;
  int lanes;              // that share a row of up to 512 columns
  int32_t slabs;          // pieces of a row
  const void* dy;
  int64_t dy_ld;
  float scale;
  float* dtable;
  bool accumulate;
  float* part;            // [chunks][2][pitch]: the first word's and the last word's sums
  int64_t pitch;
  int64_t blocks;         // that sum chunks; the others clear rows of no token
  int64_t vocab;
  int rows;               // that a wave clears, below 64
  bool stream;            // past the caches
};

// Clears those of a wave's rows that no token has: one look-up a lane finds
// where each row's word would stand among the sorted ones, and neighbouring
// rows without one are one range.
__device__ __forceinline__ void clear_rows(const ChunkArgs& a, int64_t wave) {
  const int lane = threadIdx.x & 63;
  const int64_t v0 = wave * a.rows;
  const int64_t rows = a.vocab - v0 < a.rows ? a.vocab - v0 : a.rows;
  if (rows <= 0) return;
  const int64_t n = (int64_t)a.chunks * a.chunk;
  const int64_t at = lane <= rows ? below(a.word, n, (uint32_t)(v0 + lane), false) : 0;
  const int64_t next = __shfl_down((long long)at, 1, 64);
  uint64_t clear = __ballot(lane < rows && at == next);
  while (clear) {
    const int from = __builtin_ctzll(clear);
    const uint64_t rest = ~(clear >> from);
    const int count = rest ? __builtin_ctzll(rest) : 64;
    clear &= count + from >= 64 ? 0 : ~0ull << (from + count);
    float* const p = a.dtable + (v0 + from) * a.cols;
    const int64_t size = count * a.cols;
    // 16-byte stores from the first aligned element on
    const int64_t lead0 = (4 - (int64_t)(((uintptr_t)p >> 2) & 3)) & 3;
    const int64_t lead = lead0 < size ? lead0 : size;
    const int64_t whole = (size - lead) / 4;
    f32x4* body = reinterpret_cast<f32x4*>(p + lead);
    if (a.stream) {
      for (int64_t i = lane; i < whole; i += 64) __builtin_nontemporal_store(f32x4{0, 0, 0, 0}, body + i);
    } else {
      for (int64_t i = lane; i < whole; i += 64) body[i] = f32x4{0, 0, 0, 0};
    }
    if (lane < lead) p[lane] = 0.0f;
    if (lane < 4 && lead + whole * 4 + lane < size) p[lead + whole * 4 + lane] = 0.0f;
  }
}

__device__ __forceinline__ void put_row(const ChunkArgs& a, int64_t w, int64_t c, float (&v)[8]) {
  float* row = a.dtable;
  const int64_t at = w * a.cols;
  if (a.accumulate) {
    float o[8];
    load8<SCAPE_F32>(row, at, c, a.cols, o);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = __builtin_fmaf(a.scale, v[j], o[j]);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] *= a.scale;
  }
  store8<SCAPE_F32>(row, at, c, a.cols, v);
}

// Sums the rows of each word of a chunk, and clears rows beside it.  Bound by
// memory: 16384 tokens of 32000 x 2048 bf16, inputs and tables that change from
// pass to pass: 67 us, 66 MB read and 265 written (4.9 TB/s; 56 us over one table
// that stays in the caches); without rows to clear it is bound by the latency of
// two loads, a token's number and its row.
template <int DT, bool WHOLE>
__global__ void __launch_bounds__(kThreads) embed_chunk_kernel(ChunkArgs a) {
  if ((int64_t)blockIdx.x >= a.blocks) {
    clear_rows(a, ((blockIdx.x - a.blocks) * kThreads + threadIdx.x) >> 6);
    return;
  }
  const int64_t wave = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 6;
  const int lane = threadIdx.x & 63;
  const int64_t group = (wave / a.slabs) * (64 / a.lanes) + lane / a.lanes;
  const int64_t c = ((wave % a.slabs) * a.lanes + (lane & (a.lanes - 1))) * 8;
  if (group >= a.chunks || c >= a.cols) return;
  const int64_t p0 = group * a.chunk;
  const uint32_t before = p0 > 0 ? a.word[p0 - 1] : kNoWord;
  const uint32_t after = group + 1 < a.chunks ? a.word[p0 + a.chunk] : kNoWord;
  uint32_t cur = a.word[p0];
  if (cur == kNoWord) return;
  const uint32_t first = a.token[p0];
  bool open = before == cur;  // cur's sum began in an earlier chunk
  float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  const auto flush = [&](bool last) {
    if (open || (last && after == cur)) {
      float* p = a.part + (group * 2 + (open ? 0 : 1)) * a.pitch + c;
      __builtin_memcpy(p, &acc[0], 16);
      __builtin_memcpy(p + 4, &acc[4], 16);
    } else {
      put_row(a, cur, c, acc);
    }
    open = false;
  };
  // the rows of a batch are on the way while those of the one before are added
  struct Batch {
    uint32_t w[kBatch];
    Raw8<DT, WHOLE, false> r[kBatch];
  } now, next;
  const auto fetch = [&](Batch& x, int b) {
    uint32_t t[kBatch];
    __builtin_memcpy(x.w, a.word + p0 + b, 4 * kBatch);
    __builtin_memcpy(t, a.token + p0 + b, 4 * kBatch);
    // no word: any token's row, which is left out of the sums
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const uint32_t row = x.w[j] == kNoWord ? first : t[j];
      x.r[j].load(a.dy, (int64_t)row * a.dy_ld, c, a.cols);
    }
  };
  fetch(next, 0);
  for (int b = 0; b < a.chunk; b += kBatch) {
    now = next;
    if (b + kBatch < a.chunk) fetch(next, b + kBatch);
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      if (now.w[j] != cur) {
        if (cur != kNoWord) flush(false);
        cur = now.w[j];
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
      }
      float v[8];
      now.r[j].unpack(v);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] += v[i];
    }
  }
  if (cur != kNoWord) flush(true);
}

// Partial rows of the word that crosses from chunk k into the next and begins
// in k: k's last, then the first of each chunk that begins with it.  0: none.
__device__ __forceinline__ int64_t partial_rows(const ChunkArgs& a, int32_t k, uint32_t* word) {
  const int64_t p0 = (int64_t)k * a.chunk, p1 = p0 + a.chunk;
  const uint32_t w = a.word[p1 - 1], after = a.word[p1], first = a.word[p0];
  const uint32_t before = a.word[p0 > 0 ? p0 - 1 : 0];
  const auto begin_of = [&](int64_t chunk) { return chunk < a.chunks ? a.word[chunk * a.chunk] : kNoWord; };
  uint32_t begins = begin_of(k + 1 + (threadIdx.x & 63));
  *word = w;
  if (w == kNoWord || after != w) return 0;
  if (first == w && p0 > 0 && before == w) return 0;  // begins further ahead
  const uint64_t others = __ballot(begins != w);
  if (others) return 1 + __builtin_ctzll(others);
  // the first chunk behind these that begins with another word: 64 of what is
  // left are looked at a time, since the words are sorted
  int64_t lo = k + 65, hi = a.chunks;
  while (lo < hi) {
    const int64_t step = (hi - lo + 63) / 64;
    const int64_t at = lo + (threadIdx.x & 63) * step;
    const uint64_t past = __ballot(at >= hi || begin_of(at) != w);
    const int first_past = past ? __builtin_ctzll(past) : 64;
    if (first_past == 0) break;
    const int64_t end = lo + first_past * step;
    hi = end < hi ? end : hi;
    lo += (first_past - 1) * step + 1;
  }
  return lo - k;
}

// The sum of partial rows [from, to) of chunk k's word at columns [c, c + 4),
// eight at a time in pairs: they are on the way together, and a long sum is an
// eighth as many additions deep.
__device__ __forceinline__ f32x4 part_sum(const ChunkArgs& a, int32_t k, int64_t from, int64_t to, int64_t c) {
  constexpr int kAtOnce = 8;
  const auto row = [&](int64_t i) {
    return *reinterpret_cast<const f32x4*>(a.part + ((k + i) * 2 + (i == 0 ? 1 : 0)) * a.pitch + c);
  };
  f32x4 sum = {0, 0, 0, 0};
  int64_t i = from;
  for (; i + kAtOnce <= to; i += kAtOnce) {
    f32x4 x[kAtOnce];
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) x[j] = row(i + j);
#pragma unroll
    for (int d = 1; d < kAtOnce; d *= 2)
#pragma unroll
      for (int j = 0; j < kAtOnce; j += 2 * d) x[j] += x[j + d];
    sum += x[0];
  }
  for (; i < to; ++i) sum += row(i);
  return sum;
}

__device__ __forceinline__ void put_sum(const ChunkArgs& a, uint32_t w, int64_t c, f32x4 sum) {
  float* row = a.dtable + (int64_t)w * a.cols;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (c + j < a.cols) row[c + j] = a.accumulate ? __builtin_fmaf(a.scale, sum[j], row[c + j]) : a.scale * sum[j];
}

// Joins the sums of words that cross chunks: a wave a chunk, 4 columns a lane.
// A word with many partial rows (only one can begin in the chunks of a
// workgroup) is shared by all waves, and by the groups of lanes of a wave where
// a row has fewer than 256 columns, a consecutive part each, joined in a fixed
// order.  Ordinary words: 6.5 us for 511 borders of 2048 columns, the latency of
// three loads.  65536 tokens of one word, 64 and 1024 columns, all of the call:
// 114 and 172 us; in four parts, read one after the other, 283 and 201.  (16
// waves: 114 and 136, but 0.5 to 1 us more for ordinary words.)
constexpr int kLongJoin = 16;
constexpr int kJoinWaves = 8;
__global__ void __launch_bounds__(kJoinWaves * 64) embed_join_kernel(ChunkArgs a) {
  __shared__ f32x4 lds[kJoinWaves][64];
  __shared__ int64_t rows[kJoinWaves];
  __shared__ uint32_t words[kJoinWaves];
  const int q = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int64_t c0 = (int64_t)blockIdx.y * 256, c = c0 + lane * 4;
  for (int64_t k0 = (int64_t)blockIdx.x * kJoinWaves; k0 + 1 < a.chunks; k0 += (int64_t)gridDim.x * kJoinWaves) {
    const int32_t k = (int32_t)k0 + q;
    uint32_t w = kNoWord;
    const int64_t n = k + 1 < a.chunks ? partial_rows(a, k, &w) : 0;
    if (n > 0 && n <= kLongJoin && c < a.pitch) put_sum(a, w, c, part_sum(a, k, 0, n, c));
    if (lane == 0) {
      rows[q] = n > kLongJoin ? n : 0;
      words[q] = w;
    }
    __syncthreads();
    const uint64_t is_long = __ballot(rows[lane % kJoinWaves] != 0);
    if (is_long) {
      const int b = __builtin_ctzll(is_long);
      const int64_t m = rows[b];
      int across = 64;  // lanes that share a row, a power of two
      while (across > 1 && c0 + across * 2 >= a.pitch) across /= 2;
      const int parts = kJoinWaves * (64 / across), part = q * (64 / across) + lane / across;
      const int64_t mine = c0 + (lane & (across - 1)) * 4;
      f32x4 sum = {0, 0, 0, 0};
      if (mine < a.pitch) sum = part_sum(a, (int32_t)k0 + b, m * part / parts, m * (part + 1) / parts, mine);
      for (int d = across; d < 64; d *= 2)
#pragma unroll
        for (int j = 0; j < 4; ++j) sum[j] += __shfl_xor(sum[j], d, 64);
      lds[q][lane] = sum;
      __syncthreads();
      if (q == 0 && lane < across && mine < a.pitch) {
#pragma unroll
        for (int i = 1; i < kJoinWaves; ++i) sum += lds[i][lane];
        put_sum(a, words[b], mine, sum);
      }
    }
    __syncthreads();  // rows and words have been read
  }
}

// Rows of no token are cleared past the caches where the table and dy together
// are more than a part of them.  Inputs and tables that change from pass to pass,
// with the forward pass, us past the caches and through them: table and dy of 62
// and 8 MiB 31.9 and 31.0, 93 and 0.1 27.9 and 26.8, 93 and 8 37.7 and 39.9, 125
// and 16 49.3 and 52.0, 196 and 16 (50257 x 1024, 8192 tokens) 63.3 and 68.1, 250
// and 64 (32000 x 2048, 16384 tokens) 109 and 114.6.  (One table over and over,
// with nothing beside it, stays in the caches: 250 MiB and 64 tokens 58 and 44.
// A training step moves more than they hold between two of its gradients.)
constexpr int64_t kClearStream = int64_t(96) << 20;

// How a gradient's tokens are cut, and its workspace.
struct BackPlan {
  int tile, count_lanes, chunk, lanes;
  int32_t tiles, chunks, slabs;
  int64_t padded, pitch;
  size_t word[2], token[2], part, bytes;  // offsets; the tiles go to the first pair, merges to and fro
};

BackPlan back_plan(int64_t tokens, int64_t cols) {
  BackPlan p;
  p.tile = 64;
  while (p.tile < tokens && p.tile < kSortTile) p.tile *= 2;
  p.count_lanes = 4;
  p.tiles = (int32_t)((tokens + p.tile - 1) / p.tile);
  p.padded = (int64_t)p.tiles * p.tile;
  const int64_t eights = (cols + 7) / 8;
  p.lanes = 1;
  while (p.lanes < 64 && p.lanes < eights) p.lanes *= 2;
  p.slabs = (int32_t)((eights + p.lanes - 1) / p.lanes);
  p.pitch = eights * 8;
  // long chunks write few partial rows, short ones fill the card
  p.chunk = 32;
  while (p.chunk > 8 && p.padded / p.chunk * p.slabs * p.lanes < 1024 * 64) p.chunk /= 2;
  p.chunks = (int32_t)(p.padded / p.chunk);
  size_t at = 0;
  const auto take = [&](size_t n) {
    const size_t here = at;
    at += (n + 255) & ~(size_t)255;
    return here;
  };
  for (int i = 0; i < (p.tiles > 1 ? 2 : 1); ++i) {
    p.word[i] = take((size_t)p.padded * 4);
    p.token[i] = take((size_t)p.padded * 4);
  }
  p.part = take((size_t)p.chunks * 2 * (size_t)p.pitch * 4);
  p.bytes = at + 256;
  return p;
}

unsigned capped(int64_t blocks, int64_t most) { return (unsigned)(blocks > most ? most : blocks); }

template <int DT>
void launch_chunks(const ChunkArgs& a, dim3 grid, hipStream_t s) {
  if (a.cols % 8 == 0) embed_chunk_kernel<DT, true><<<grid, kThreads, 0, s>>>(a);
  else embed_chunk_kernel<DT, false><<<grid, kThreads, 0, s>>>(a);
}

template <int TT>
void embed_out(const EmbedArgs& a, int out, hipStream_t s) {
  int lanes = 1;
  while (lanes < kThreads && lanes * 8 < a.cols) lanes *= 2;
  const dim3 grid(capped((a.tokens * lanes + kThreads - 1) / kThreads, 1 << 20));
  if (out == SCAPE_F32) embed_kernel<TT, SCAPE_F32><<<grid, kThreads, 0, s>>>(a, lanes);
  else if (out == SCAPE_BF16) embed_kernel<TT, SCAPE_BF16><<<grid, kThreads, 0, s>>>(a, lanes);
  else embed_kernel<TT, SCAPE_F16><<<grid, kThreads, 0, s>>>(a, lanes);
}

// Words that a workgroup of the slab sort owns: about one workgroup a CU.  0:
// sorted by tiles, which can be any number.  16384 tokens of 32000 words: slabs
// 7.5 us, tiles and their merge 16.5; 1531 of 4099: 5.2 against 10.5; 65536 of
// 32000 x 1024, all of the call: 184 against 222.  Few words share few
// workgroups, and still: 8 columns, all of the call, 262144 tokens of 2 words 286
// against 320, of 1024 104 against 307, 1048576 of 2 1150 against 1870.  (Tiles
// win where a word of many has most tokens, which is not known here: 262144 of
// 32000 x 64, half of them one word, 408 against 310.)
int slab_of(int64_t tokens, int64_t vocab) {
  int slab = 4;
  while (slab < kSlabMax && (vocab + slab - 1) / slab > 256) slab *= 2;
  const int64_t slabs = (vocab + slab - 1) / slab;
  return slabs <= kSlabs && tokens * slabs <= kSlabWork ? slab : 0;
}

// Sorts tiles and merges them; which pair of buffers holds the result.
int sort_tiles(const BackPlan& p, int64_t tokens, int64_t vocab, const scape_ids& ids, char* base, hipStream_t s) {
  const auto at = [&](size_t off) { return reinterpret_cast<uint32_t*>(base + off); };
  const SortArgs sa{tokens, vocab, ids.data, p.tile, p.count_lanes, at(p.word[0]), at(p.token[0])};
  const dim3 sorting((unsigned)(p.padded * p.count_lanes / kThreads));
  if (ids.bits == 64) embed_sort_kernel<int64_t><<<sorting, kThreads, p.tile * 4, s>>>(sa);
  else embed_sort_kernel<int32_t><<<sorting, kThreads, p.tile * 4, s>>>(sa);
  int from = 0;
  for (int64_t run = p.tile; run < p.padded; run *= kFan, from ^= 1) {
    const int64_t runs = (p.padded + run - 1) / run;
    int lanes = 1;
    while (lanes < kFan && lanes < runs) lanes *= 2;
    const dim3 grid(capped((p.padded * lanes + kThreads - 1) / kThreads, 1 << 22));
    embed_merge_kernel<<<grid, kThreads, 0, s>>>(at(p.word[from]), at(p.token[from]), p.padded, run, lanes,
                                                 at(p.word[from ^ 1]), at(p.token[from ^ 1]));
  }
  return from;
}

}  // namespace

hipError_t launch_embed(int64_t tokens, int64_t vocab, int64_t positions, int64_t cols, const scape_ids& ids,
                        const scape_matrix& table, float scale, const scape_ids& pos, const scape_matrix& pos_table,
                        const scape_matrix& out, hipStream_t s) {
  if (tokens == 0) return hipSuccess;
  const EmbedArgs a{tokens, vocab, positions, cols, ids, pos, table.data, table.ld, pos_table.data, pos_table.ld,
                    scale, out.data, out.ld};
  if (table.dtype == SCAPE_F32) embed_out<SCAPE_F32>(a, out.dtype, s);
  else if (table.dtype == SCAPE_BF16) embed_out<SCAPE_BF16>(a, out.dtype, s);
  else embed_out<SCAPE_F16>(a, out.dtype, s);
  return hipGetLastError();
}

size_t embed_workspace(int64_t tokens, int64_t cols) { return back_plan(tokens, cols).bytes; }

hipError_t launch_embed_backward(int64_t tokens, int64_t vocab, int64_t cols, const scape_ids& ids,
                                 const scape_matrix& dy, float scale, float* dtable, bool accumulate, void* ws,
                                 hipStream_t s) {
  if (tokens == 0 && accumulate) return hipSuccess;
  const BackPlan p = back_plan(tokens, cols);
  char* base = static_cast<char*>(ws);
  const auto at = [&](size_t off) { return reinterpret_cast<uint32_t*>(base + off); };
  int from = 0;
  const int slab = slab_of(tokens, vocab);
  if (slab && tokens > 0) {
    const int stretch = (int)((tokens + kSlabThreads - 1) / kSlabThreads) * 64;
    const SlabArgs a{tokens, vocab, p.padded, ids.data, slab, stretch, at(p.word[0]), at(p.token[0])};
    const dim3 grid((unsigned)((vocab + slab - 1) / slab));
    // (a stretch that passes is far below the 2^16 places of a list's entry)
    const bool list = (int64_t)(slab + stretch) * kSlabWaves * 4 <= kSlabLds;
    const size_t lds = (size_t)(slab + (list ? stretch : 0)) * kSlabWaves * 4;
    const auto go = [&](auto kernel) { kernel<<<grid, kSlabThreads, lds, s>>>(a); };
    if (ids.bits == 64) go(list ? embed_slab_kernel<int64_t, true> : embed_slab_kernel<int64_t, false>);
    else go(list ? embed_slab_kernel<int32_t, true> : embed_slab_kernel<int32_t, false>);
  } else if (tokens > 0) {
    from = sort_tiles(p, tokens, vocab, ids, base, s);
  }
  const int64_t waves = ((int64_t)p.chunks * p.lanes + 63) / 64 * p.slabs;
  const int64_t blocks = (waves + 3) / 4;
  // rows to clear: about 64 KB a wave
  int64_t rows = (64 << 10) / (cols * 4);
  rows = rows < 1 ? 1 : rows > 63 ? 63 : rows;
  const int64_t clearing = accumulate ? 0 : (vocab + 4 * rows - 1) / (4 * rows);
  const ChunkArgs ca{cols, at(p.word[from]), at(p.token[from]), p.chunk, p.chunks, p.lanes, p.slabs, dy.data, dy.ld,
                     scale, dtable, accumulate, reinterpret_cast<float*>(base + p.part), p.pitch, blocks, vocab,
                     (int)rows, (vocab * 4 + tokens * (int64_t)dtype_bytes(dy.dtype)) * cols > kClearStream};
  const dim3 grid((unsigned)(blocks + clearing));
  if (dy.dtype == SCAPE_F32) launch_chunks<SCAPE_F32>(ca, grid, s);
  else if (dy.dtype == SCAPE_BF16) launch_chunks<SCAPE_BF16>(ca, grid, s);
  else launch_chunks<SCAPE_F16>(ca, grid, s);
  if (p.chunks > 1)
    embed_join_kernel<<<dim3(capped((p.chunks + kJoinWaves - 2) / kJoinWaves, 1 << 20), (unsigned)((p.pitch + 255) / 256)),
                        kJoinWaves * 64, 0, s>>>(ca);
  return hipGetLastError();
}

}  // namespace scape
