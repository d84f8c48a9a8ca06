// Attention over parts of the keys: each part leaves its rows' normalised
// result and log-sum (fp32), and attn_join_kernel weighs them together.
#pragma once

#include "sequence.h"

namespace vswin {

struct Split {
  int n;       // parts of the keys (1: results go out directly)
  float* o;    // [n][B hq Lq][d]
  float* lse;  // [n][B hq Lq], log2
};

inline size_t split_bytes(const BiasAttnArgs& a, int n) {
  return n > 1 ? (size_t)n * a.B * a.hq * a.Lq * (a.d + 1) * 4 : 0;
}
inline Split split_of(const BiasAttnArgs& a, int n, void* scratch) {
  float* o = static_cast<float*>(scratch);
  return Split{n, o, n > 1 ? o + (size_t)n * a.B * a.hq * a.Lq * a.d : nullptr};
}

template <class T, int D>
cudaError_t launch_attention_join(const BiasAttnArgs& a, const Split& sp, cudaStream_t st);

// The form for few rows (bias_attention_token.cu).
bool token_form(const BiasAttnArgs& a);
int token_splits(const BiasAttnArgs& a);
cudaError_t launch_token_attention(const BiasAttnArgs& a, int dtype, void* scratch, cudaStream_t st);

}  // namespace vswin
