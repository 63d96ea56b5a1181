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
// bound by memory.
template <int TT, int OT>
__global__ void __launch_bounds__(kThreads) embed_kernel(EmbedArgs a) {
  const int64_t chunks = (a.cols + 7) / 8;
  for (int64_t t = blockIdx.x; t < a.tokens; t += gridDim.x) {
    const int64_t id = token_at(a.ids, t);
    const int64_t at = a.pos_table ? token_at(a.pos, t) : -1;
    for (int64_t i = threadIdx.x; i < chunks; i += kThreads) {
      float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
      if (id >= 0 && id < a.vocab) load8<TT>(a.table, id * a.table_ld, i * 8, a.cols, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= a.scale;
      if (at >= 0 && at < a.positions) {
        float p[8];
        load8<TT>(a.pos_table, at * a.pos_ld, i * 8, a.cols, p);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] += p[j];
      }
      store8<OT>(a.out, t * a.out_ld, i * 8, a.cols, v);
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

constexpr uint32_t kNoWord = 0xffffffffu;
constexpr int kTileMax = 2048;  // tokens that a workgroup sorts in LDS
constexpr int kSortThreads = 1024;
constexpr unsigned kFillBlocks = 4096;
constexpr int kBatch = 8;  // rows of dy on the way at a time

struct SortArgs {
  int64_t tokens, vocab;
  scape_ids ids;
  int tile;         // a power of two
  int32_t tiles;
  uint32_t* word;   // [tiles * tile], each tile sorted
  uint32_t* token;
  float* fill;      // set to zero by the other workgroups
  int64_t fill_n;
};

// Sorts (word, place) pairs of a tile by bitonic exchanges in LDS.  The pairs
// that a wave exchanges at distances of 64 and less lie in a part of the tile
// of its own, so only the larger distances need the workgroup's barrier.
__device__ __forceinline__ void sort_tile(uint64_t* lds, int n) {
  for (int k = 2; k <= n; k <<= 1) {
    for (int j = k >> 1; j > 0; j >>= 1) {
      for (int i = threadIdx.x; i < n / 2; i += kSortThreads) {
        const int lo = ((i & ~(j - 1)) << 1) | (i & (j - 1));
        const uint64_t x = lds[lo], y = lds[lo + j];
        if ((x > y) == ((lo & k) == 0)) {
          lds[lo] = y;
          lds[lo + j] = x;
        }
      }
      if (j > 64) {
        __syncthreads();
      } else {
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        if (j == 1 && k >= 128) __syncthreads();  // the next k exchanges across waves
      }
    }
  }
  __syncthreads();
}

__global__ void __launch_bounds__(kSortThreads) embed_sort_kernel(SortArgs a) {
  __shared__ uint64_t lds[kTileMax];
  if ((int32_t)blockIdx.x < a.tiles) {
    const int64_t t0 = (int64_t)blockIdx.x * a.tile;
    for (int i = threadIdx.x; i < a.tile; i += kSortThreads) {
      uint32_t w = kNoWord;
      if (t0 + i < a.tokens) {
        const int64_t id = token_at(a.ids, t0 + i);
        if (id >= 0 && id < a.vocab) w = (uint32_t)id;
      }
      lds[i] = (uint64_t)w << 32 | (uint32_t)i;
    }
    __syncthreads();
    sort_tile(lds, a.tile);
    for (int i = threadIdx.x; i < a.tile; i += kSortThreads) {
      a.word[t0 + i] = (uint32_t)(lds[i] >> 32);
      a.token[t0 + i] = (uint32_t)t0 + (uint32_t)lds[i];
    }
    return;
  }
  // 16-byte stores from the first aligned element on
  const int64_t lead0 = (4 - (int64_t)(((uintptr_t)a.fill >> 2) & 3)) & 3;
  const int64_t lead = lead0 < a.fill_n ? lead0 : a.fill_n;
  const int64_t whole = (a.fill_n - lead) / 4;
  const int64_t at = (int64_t)(blockIdx.x - a.tiles) * kSortThreads + threadIdx.x;
  const int64_t step = (int64_t)(gridDim.x - a.tiles) * kSortThreads;
  f32x4* body = reinterpret_cast<f32x4*>(a.fill + lead);
  for (int64_t i = at; i < whole; i += step) body[i] = f32x4{0, 0, 0, 0};
  if (at < lead) a.fill[at] = 0.0f;
  const int64_t tail = lead + whole * 4 + at;
  if (at < 4 && tail < a.fill_n) a.fill[tail] = 0.0f;
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
};

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

template <int DT, bool WHOLE>
__global__ void __launch_bounds__(kThreads) embed_chunk_kernel(ChunkArgs a) {
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
  for (int b = 0; b < a.chunk; b += kBatch) {
    uint32_t w[kBatch], t[kBatch];
    __builtin_memcpy(w, a.word + p0 + b, 4 * kBatch);
    __builtin_memcpy(t, a.token + p0 + b, 4 * kBatch);
    if (w[0] == kNoWord) break;
    Raw8<DT, WHOLE, false> r[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j)
      r[j].load(a.dy, (int64_t)(w[j] == kNoWord ? t[0] : t[j]) * a.dy_ld, c, a.cols);
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      if (w[j] != cur) {
        if (cur != kNoWord) flush(false);
        cur = w[j];
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
      }
      float v[8];
      r[j].unpack(v);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] += v[i];
    }
  }
  if (cur != kNoWord) flush(true);
}

// Joins the sums of a word that crosses chunks, in the chunk k where it begins:
// four waves add a quarter of its partial rows each, in order, then the
// quarters.  A lane owns 4 columns.
__device__ __forceinline__ void join_word(const ChunkArgs& a, int32_t k, f32x4 (*lds)[64]) {
  const int64_t p0 = (int64_t)k * a.chunk, p1 = p0 + a.chunk;
  const uint32_t w = a.word[p1 - 1];
  if (w == kNoWord || a.word[p1] != w) return;
  if (a.word[p0] == w && p0 > 0 && a.word[p0 - 1] == w) return;  // begins further ahead
  int64_t lo = p1, hi = (int64_t)a.chunks * a.chunk;  // the word's end
  while (hi - lo > 1) {
    const int64_t mid = (lo + hi) >> 1;
    if (a.word[mid] == w) lo = mid;
    else hi = mid;
  }
  const int64_t n = lo / a.chunk - k + 1;  // partial rows: k's last, then the first of each chunk up to lo's
  const int q = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t c = ((int64_t)blockIdx.y * 64 + lane) * 4;
  const bool mine = c < a.pitch;
  const int64_t from = n * q / 4, to = n * (q + 1) / 4;
  f32x4 sum = {0, 0, 0, 0};
  if (mine) {
#pragma unroll 8
    for (int64_t i = from; i < to; ++i) {
      const float* p = a.part + ((k + i) * 2 + (i == 0 ? 1 : 0)) * a.pitch + c;
      sum += *reinterpret_cast<const f32x4*>(p);
    }
  }
  __syncthreads();  // the sums of the word before have been read
  if (q > 0) lds[q - 1][lane] = sum;
  __syncthreads();
  if (q > 0 || !mine) return;
  sum = ((sum + lds[0][lane]) + lds[1][lane]) + lds[2][lane];
  float* row = a.dtable + (int64_t)w * a.cols;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (c + j < a.cols) row[c + j] = a.accumulate ? __builtin_fmaf(a.scale, sum[j], row[c + j]) : a.scale * sum[j];
}

__global__ void __launch_bounds__(kThreads) embed_join_kernel(ChunkArgs a) {
  __shared__ f32x4 lds[3][64];
  for (int32_t k = blockIdx.x; k + 1 < a.chunks; k += gridDim.x) join_word(a, k, lds);
}

// How a gradient's tokens are cut, and its workspace.
struct BackPlan {
  int tile, chunk, lanes;
  int32_t tiles, chunks, slabs;
  int64_t padded, pitch;
  size_t word[2], token[2], part, bytes;  // offsets; the tiles go to the first pair, merges to and fro
};

BackPlan back_plan(int64_t tokens, int64_t cols) {
  BackPlan p;
  p.tile = 64;
  while (p.tile < kTileMax && p.tile < tokens) p.tile *= 2;
  p.tiles = (int32_t)((tokens + p.tile - 1) / p.tile);
  p.padded = (int64_t)p.tiles * p.tile;
  const int64_t eights = (cols + 7) / 8;
  p.lanes = 1;
  while (p.lanes < 64 && p.lanes < eights) p.lanes *= 2;
  p.slabs = (int32_t)((eights + p.lanes - 1) / p.lanes);
  p.pitch = eights * 8;
  // long chunks write few partial rows, short ones fill the card
  p.chunk = 32;
  while (p.chunk > 8 && p.padded / p.chunk * p.slabs * p.lanes < 2048 * 64) p.chunk /= 2;
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
  const dim3 grid(capped(a.tokens, 1 << 20));
  if (out == SCAPE_F32) embed_kernel<TT, SCAPE_F32><<<grid, kThreads, 0, s>>>(a);
  else if (out == SCAPE_BF16) embed_kernel<TT, SCAPE_BF16><<<grid, kThreads, 0, s>>>(a);
  else embed_kernel<TT, SCAPE_F16><<<grid, kThreads, 0, s>>>(a);
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
  const SortArgs sa{tokens, vocab, ids, p.tile, p.tiles, at(p.word[0]), at(p.token[0]), dtable,
                    accumulate ? 0 : vocab * cols};
  const unsigned fill = capped((sa.fill_n / 4 + kSortThreads - 1) / kSortThreads + (sa.fill_n > 0), kFillBlocks);
  embed_sort_kernel<<<dim3((unsigned)p.tiles + fill), kSortThreads, 0, s>>>(sa);
  if (tokens == 0) return hipGetLastError();
  int from = 0;
  for (int64_t run = p.tile; run < p.padded; run *= kFan, from ^= 1) {
    const int64_t runs = (p.padded + run - 1) / run;
    int lanes = 1;
    while (lanes < kFan && lanes < runs) lanes *= 2;
    const dim3 grid(capped((p.padded * lanes + kThreads - 1) / kThreads, 1 << 22));
    embed_merge_kernel<<<grid, kThreads, 0, s>>>(at(p.word[from]), at(p.token[from]), p.padded, run, lanes,
                                                 at(p.word[from ^ 1]), at(p.token[from ^ 1]));
  }
  const ChunkArgs ca{cols, at(p.word[from]), at(p.token[from]), p.chunk, p.chunks, p.lanes, p.slabs, dy.data, dy.ld,
                     scale, dtable, accumulate, reinterpret_cast<float*>(base + p.part), p.pitch};
  const int64_t waves = ((int64_t)p.chunks * p.lanes + 63) / 64 * p.slabs;
  const dim3 grid((unsigned)((waves + 3) / 4));
  if (dy.dtype == SCAPE_F32) launch_chunks<SCAPE_F32>(ca, grid, s);
  else if (dy.dtype == SCAPE_BF16) launch_chunks<SCAPE_BF16>(ca, grid, s);
  else launch_chunks<SCAPE_F16>(ca, grid, s);
  if (p.chunks > 1)
    embed_join_kernel<<<dim3(capped(p.chunks - 1, 1 << 20), (unsigned)((p.pitch + 255) / 256)), kThreads, 0, s>>>(ca);
  return hipGetLastError();
}

}  // namespace scape
