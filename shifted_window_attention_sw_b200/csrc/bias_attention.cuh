// What the kernels of the attention with bucketed bias share: the lengths and
// positions of a sequence and the bias of an offset.
#pragma once

#include "sequence.h"

namespace vswin {

// A bias at or below this takes its key out of the softmax, as -inf does (so
// that the lowest value of a type works as a mask).
constexpr float kExclude = -1e30f;

struct SeqLens {
  int nq, nk;  // query rows and keys that take part
  int start;   // position of query 0
};

// Lengths outside the tensors are recorded in the error word and clamped;
// positions are held within +-2^30, so that differences fit an int.
__device__ __forceinline__ SeqLens seq_lens(const BiasAttnArgs& a, int b) {
  SeqLens s;
  s.nq = a.q_lens ? a.q_lens[b] : a.Lq;
  s.nk = a.kv_lens ? a.kv_lens[b] : a.Lk;
  s.start = a.q_start ? a.q_start[b] : 0;
  constexpr int kMaxPos = 1 << 30;
  if (s.nq < 0 || s.nq > a.Lq || s.nk < 0 || s.nk > a.Lk || s.start < -kMaxPos || s.start > kMaxPos) {
    atomicCAS(a.ctx.err, 0, kErrBounds);
    s.nq = s.nq < 0 ? 0 : (s.nq > a.Lq ? a.Lq : s.nq);
    s.nk = s.nk < 0 ? 0 : (s.nk > a.Lk ? a.Lk : s.nk);
    s.start = s.start < -kMaxPos ? -kMaxPos : (s.start > kMaxPos ? kMaxPos : s.start);
  }
  return s;
}

// Bias of head h at offset `rel` = key - position of the query, -inf for a key
// that it takes out; a bucket outside the table is recorded in the error word
// and its bias is 0 (bucket 0 for the gradient).
template <class T>
__device__ __forceinline__ float bias_of(const BiasAttnArgs& a, int rel, int h, int* bucket = nullptr) {
  const int at = (rel < -a.D ? -a.D : (rel > a.D ? a.D : rel)) + a.D;
  int k = __ldg(a.map + at);
  if (k < 0 || k >= a.buckets) {
    atomicCAS(a.ctx.err, 0, kErrBounds);
    if (bucket) *bucket = 0;
    return 0.f;
  }
  if (bucket) *bucket = k;
  const float v = to_f(static_cast<const T*>(a.table)[(long long)k * a.hq + h]);
  return v <= kExclude ? -INFINITY : v;
}

}  // namespace vswin
