// Gradient of the attention with bucketed bias.
#include "bias_attention.cuh"

namespace vswin {
namespace {

constexpr int kWarps = 4;

// One query row per warp: D = dO . o, dS = P (dP - D), dq = scale dS k.
template <class T>
__global__ void __launch_bounds__(32 * kWarps) attn_dq_kernel(BiasAttnArgs a, float* D, float* dtab) {
  const int lane = threadIdx.x & 31;
  const long long row = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (row >= (long long)a.B * a.hq * a.Lq) return;
  const int i = (int)(row % a.Lq), h = (int)(row / a.Lq % a.hq), b = (int)(row / a.Lq / a.hq);
  const int hk = h / (a.hq / a.hk);
  const SeqLens sl = seq_lens(a, b);
  const int pos = sl.start + i;
  const T* q = static_cast<const T*>(a.q.p) + a.q.at(b, i, h);
  const T* o = static_cast<const T*>(a.o.p) + a.o.at(b, i, h);
  const T* go = static_cast<const T*>(a.dout.p) + a.dout.at(b, i, h);
  const float lse = a.lse[row];
  const int nk = i < sl.nq && lse > -INFINITY ? (a.causal ? min(sl.nk, pos + 1) : sl.nk) : 0;
  float dd = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
  if (nk > 0)
    for (int c = lane; c < a.d; c += 32) dd = fmaf(to_f(o[c]), to_f(go[c]), dd);
  for (int k = 16; k; k >>= 1) dd += __shfl_xor_sync(~0u, dd, k);
  if (lane == 0) D[row] = dd;
  for (int j0 = 0; j0 < nk; j0 += 32) {
    const int j = j0 + lane;
    float ds = 0.f;
    if (j < nk) {
      const T* k = static_cast<const T*>(a.k.p) + a.k.at(b, j, hk);
      const T* v = static_cast<const T*>(a.v.p) + a.v.at(b, j, hk);
      float s = 0.f, dp = 0.f;
      for (int c = 0; c < a.d; ++c) {
        s = fmaf(to_f(q[c]), to_f(k[c]), s);
        dp = fmaf(to_f(go[c]), to_f(v[c]), dp);
      }
      int bucket;
      s = s * a.scale + bias_of<T>(a, j - pos, h, &bucket);
      ds = expf(s - lse) * (dp - dd);
      if (ds != 0.f) atomicAdd(&dtab[(long long)bucket * a.hq + h], ds);
    }
    for (int jj = 0; jj < 32 && j0 + jj < nk; ++jj) {
      const float x = __shfl_sync(~0u, ds, jj);
      const T* k = static_cast<const T*>(a.k.p) + a.k.at(b, j0 + jj, hk);
      for (int c = 0; c < a.d / 32; ++c) acc[c] = fmaf(x, to_f(k[lane + 32 * c]), acc[c]);
    }
  }
  T* dq = static_cast<T*>(a.dq.p) + a.dq.at(b, i, h);
  for (int c = 0; c < a.d / 32; ++c) dq[lane + 32 * c] = from_f<T>(acc[c] * a.scale);
}

// One key row per warp: dv = P^T dO and dk = scale dS^T q over the queries and heads that read it.
template <class T>
__global__ void __launch_bounds__(32 * kWarps) attn_dkv_kernel(BiasAttnArgs a, const float* D) {
  const int lane = threadIdx.x & 31;
  const long long row = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (row >= (long long)a.B * a.hk * a.Lk) return;
  const int j = (int)(row % a.Lk), hk = (int)(row / a.Lk % a.hk), b = (int)(row / a.Lk / a.hk);
  const SeqLens sl = seq_lens(a, b);
  const T* k = static_cast<const T*>(a.k.p) + a.k.at(b, j, hk);
  const T* v = static_cast<const T*>(a.v.p) + a.v.at(b, j, hk);
  float dk[4] = {0.f, 0.f, 0.f, 0.f}, dv[4] = {0.f, 0.f, 0.f, 0.f};
  const int i_lo = a.causal ? max(0, j - sl.start) : 0;
  const int i_hi = j < sl.nk ? sl.nq : 0;
  for (int h = hk * (a.hq / a.hk); h < (hk + 1) * (a.hq / a.hk); ++h)
    for (int i0 = i_lo; i0 < i_hi; i0 += 32) {
      const int i = i0 + lane;
      float p = 0.f, ds = 0.f;
      if (i < i_hi) {
        const long long r = ((long long)b * a.hq + h) * a.Lq + i;
        const float lse = a.lse[r];
        if (lse > -INFINITY) {
          const T* q = static_cast<const T*>(a.q.p) + a.q.at(b, i, h);
          const T* go = static_cast<const T*>(a.dout.p) + a.dout.at(b, i, h);
          float s = 0.f, dp = 0.f;
          for (int c = 0; c < a.d; ++c) {
            s = fmaf(to_f(q[c]), to_f(k[c]), s);
            dp = fmaf(to_f(go[c]), to_f(v[c]), dp);
          }
          p = expf(s * a.scale + bias_of<T>(a, j - sl.start - i, h) - lse);
          ds = p * (dp - D[r]);
        }
      }
      for (int ii = 0; ii < 32 && i0 + ii < i_hi; ++ii) {
        const float x = __shfl_sync(~0u, p, ii), y = __shfl_sync(~0u, ds, ii);
        const T* q = static_cast<const T*>(a.q.p) + a.q.at(b, i0 + ii, h);
        const T* go = static_cast<const T*>(a.dout.p) + a.dout.at(b, i0 + ii, h);
        for (int c = 0; c < a.d / 32; ++c) {
          dv[c] = fmaf(x, to_f(go[lane + 32 * c]), dv[c]);
          dk[c] = fmaf(y, to_f(q[lane + 32 * c]), dk[c]);
        }
      }
    }
  T* ok = static_cast<T*>(a.dk.p) + a.dk.at(b, j, hk);
  T* ov = static_cast<T*>(a.dv.p) + a.dv.at(b, j, hk);
  for (int c = 0; c < a.d / 32; ++c) {
    ok[lane + 32 * c] = from_f<T>(dk[c] * a.scale);
    ov[lane + 32 * c] = from_f<T>(dv[c]);
  }
}

template <class T>
__global__ void dtable_round_kernel(BiasAttnArgs a, const float* dtab) {
  const int n = a.buckets * a.hq;
  for (int k = blockIdx.x * blockDim.x + threadIdx.x; k < n; k += gridDim.x * blockDim.x)
    static_cast<T*>(a.dtable)[k] = from_f<T>(dtab[k]);
}

template <class T>
cudaError_t backward(const BiasAttnArgs& a, void* scratch, cudaStream_t st) {
  const long long rows = (long long)a.B * a.hq * a.Lq, keys = (long long)a.B * a.hk * a.Lk;
  float* D = static_cast<float*>(scratch);
  float* dtab = D + rows;
  cudaError_t e = cudaMemsetAsync(dtab, 0, (size_t)a.buckets * a.hq * 4, st);
  if (e != cudaSuccess) return e;
  attn_dq_kernel<T><<<(unsigned)((rows + kWarps - 1) / kWarps), 32 * kWarps, 0, st>>>(a, D, dtab);
  attn_dkv_kernel<T><<<(unsigned)((keys + kWarps - 1) / kWarps), 32 * kWarps, 0, st>>>(a, D);
  dtable_round_kernel<T><<<(a.buckets * a.hq + 255) / 256, 256, 0, st>>>(a, dtab);
  count_launch(3);
  return cudaGetLastError();
}

}  // namespace

size_t bias_attention_backward_scratch_bytes(const BiasAttnArgs& a) {
  return ((size_t)a.B * a.hq * a.Lq + (size_t)a.buckets * a.hq) * 4;
}
cudaError_t launch_bias_attention_backward(const BiasAttnArgs& a, int dtype, void* scratch, cudaStream_t st) {
  return dtype == kBF16 ? backward<__nv_bfloat16>(a, scratch, st) : backward<__half>(a, scratch, st);
}

}  // namespace vswin
