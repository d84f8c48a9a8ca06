// Attention over parts of the keys: each part leaves its rows' normalised
// result and log-sum (fp32), and attn_join_kernel weighs them together.
#pragma once

#include "sequence.h"

namespace vswin {

struct Split {
  int n;           // parts of the keys (1: results go out directly)
  long long rows;  // rows that are split
  int first;       // first split tile of 128 rows (rows by tile), or -1: rows are (b, h, i)
  float* o;        // [n][rows][d]
  float* lse;      // [n][rows], log2
};

inline size_t split_bytes(const Split& s, int d) { return s.n > 1 ? (size_t)s.n * s.rows * (d + 1) * 4 : 0; }
inline void split_place(Split* s, int d, void* scratch) {
  s->o = static_cast<float*>(scratch);
  s->lse = s->n > 1 ? s->o + (size_t)s->n * s->rows * d : nullptr;
}

// Query tile `tile` of a launch: head and batch fastest, the last rows first.
struct QueryTile {
  int b, h, qt;
};
__host__ __device__ inline QueryTile query_tile(const BiasAttnArgs& a, unsigned tile) {
  const unsigned heads = (unsigned)a.B * a.hq, tiles = (unsigned)(a.Lq + 127) / 128;
  const unsigned rest = tile % heads;
  return {(int)(rest / a.hq), (int)(rest % a.hq), (int)(tiles - 1 - tile / heads)};
}

template <class T, int D>
cudaError_t launch_attention_join(const BiasAttnArgs& a, const Split& sp, cudaStream_t st);

// The form for few rows (bias_attention_token.cu).
bool token_form(const BiasAttnArgs& a);
Split token_split(const BiasAttnArgs& a);
cudaError_t launch_token_attention(const BiasAttnArgs& a, int dtype, void* scratch, cudaStream_t st);

}  // namespace vswin
