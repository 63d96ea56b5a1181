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

struct EmbedBackArgs {
  int64_t tokens, vocab, cols;
  scape_ids ids;
  const void* dy;
  int64_t dy_ld;
  float scale;
  float* dtable;
  bool accumulate;
};

constexpr int kSlab = 64;  // rows of the table that a workgroup owns

// A workgroup owns kSlab rows of the table, goes through all tokens in their
// order, and adds the rows of those that are its own; a thread owns its
// columns, so no two write the same element.
template <int DT>
__global__ void __launch_bounds__(kThreads) embed_back_kernel(EmbedBackArgs a) {
  for (int64_t lo = (int64_t)blockIdx.x * kSlab; lo < a.vocab; lo += (int64_t)gridDim.x * kSlab) {
    const int64_t hi = lo + kSlab < a.vocab ? lo + kSlab : a.vocab;
    if (!a.accumulate)
      for (int64_t v = lo; v < hi; ++v)
        for (int64_t c = threadIdx.x; c < a.cols; c += kThreads) a.dtable[v * a.cols + c] = 0.0f;
    for (int64_t t0 = 0; t0 < a.tokens; t0 += 64) {
      const int64_t t = t0 + (threadIdx.x & 63);
      const int64_t id = t < a.tokens ? token_at(a.ids, t) : -1;
      for (uint64_t mine = __ballot(id >= lo && id < hi); mine; mine &= mine - 1) {
        const int l = __builtin_ctzll(mine);
        const int64_t v = lo + __shfl((int)(id - lo), l);
        for (int64_t c = threadIdx.x; c < a.cols; c += kThreads) {
          float* p = a.dtable + v * a.cols + c;
          *p = __builtin_fmaf(a.scale, Elem<DT>::get(a.dy, (t0 + l) * a.dy_ld + c), *p);
        }
      }
    }
  }
}

unsigned capped(int64_t blocks, int64_t most) { return (unsigned)(blocks > most ? most : blocks); }

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

size_t embed_workspace(int64_t, int64_t) { return 256; }

hipError_t launch_embed_backward(int64_t tokens, int64_t vocab, int64_t cols, const scape_ids& ids,
                                 const scape_matrix& dy, float scale, float* dtable, bool accumulate, void*,
                                 hipStream_t s) {
  const EmbedBackArgs a{tokens, vocab, cols, ids, dy.data, dy.ld, scale, dtable, accumulate};
  const dim3 grid(capped((vocab + kSlab - 1) / kSlab, 1 << 20));
  if (dy.dtype == SCAPE_F32) embed_back_kernel<SCAPE_F32><<<grid, kThreads, 0, s>>>(a);
  else if (dy.dtype == SCAPE_BF16) embed_back_kernel<SCAPE_BF16><<<grid, kThreads, 0, s>>>(a);
  else embed_back_kernel<SCAPE_F16><<<grid, kThreads, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace scape
