// Internal declarations of the operators over token sequences (qk_norm.cu,
// bias_attention*.cu) and of the optimizer step (adamw.cu).
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "internal.h"

namespace vswin {

// Element types, numbered as VSWIN_BF16, VSWIN_FP16 and VSWIN_F32.
enum : int { kBF16 = 0, kFP16 = 1, kF32 = 2 };

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
template <class T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ float from_f<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half from_f<__half>(float x) { return __float2half_rn(x); }

// A kernel that may start while the one before it in the stream still runs, and
// waits for its end (after_previous) before it reads what that one wrote: its
// launch and prologue then cost nothing. The one before lets it start as soon as
// all of its own blocks have (let_next_start).
template <class... P, class... A>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, const A&... args) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c{};
  c.gridDim = grid;
  c.blockDim = dim3(threads);
  c.dynamicSmemBytes = smem;
  c.stream = st;
  c.attrs = &attr;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kernel, static_cast<P>(args)...);
}
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;"); }
__device__ __forceinline__ void after_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// A (batch, token, head, channel) tensor whose channels are contiguous;
// strides in elements.
struct Heads {
  void* p;
  long long sb, st, sh;
  __host__ __device__ long long at(long long b, long long t, long long h) const { return b * sb + t * st + h * sh; }
};

struct QkNormArgs {
  int B, L, d, rot, interleaved;
  int heads[2];       // of q, k
  Heads x[2], y[2];   // inputs; outputs (forward) or output gradients (backward)
  Heads dx[2];        // backward: input gradients
  const void* gamma[2];
  const float* cosp;  // [rows][rot / 2]
  const float* sinp;
  const int* positions;  // [B][L] or null (token l uses row l)
  int rows;
  float eps;
  float* dgamma[2];  // backward: [d]
  int* err;
};
cudaError_t launch_qk_norm_forward(const QkNormArgs& a, int dtype, cudaStream_t st);
size_t qk_norm_scratch_bytes(const QkNormArgs& a, int dtype);
cudaError_t launch_qk_norm_backward(const QkNormArgs& a, int dtype, void* scratch, cudaStream_t st);

constexpr int kMaxBuckets = 512;

struct BiasAttnArgs {
  int B, Lq, Lk, hq, hk, d;
  Heads q, k, v, o;
  float* lse;  // [B][hq][Lq], natural logarithm
  float scale;
  const void* table;  // [buckets][hq]
  const int* map;     // [2 D + 1]
  int buckets, D;
  const int* q_lens;   // [B] or null
  const int* kv_lens;  // [B] or null
  const int* q_start;  // [B] or null
  int causal;
  // backward
  Heads dout, dq, dk, dv;
  void* dtable;  // [buckets][hq]
  KernelCtx ctx;
};
size_t bias_attention_scratch_bytes(const BiasAttnArgs& a);
cudaError_t launch_bias_attention(const BiasAttnArgs& a, int dtype, void* scratch, cudaStream_t st);
size_t bias_attention_backward_scratch_bytes(const BiasAttnArgs& a);
cudaError_t launch_bias_attention_backward(const BiasAttnArgs& a, int dtype, void* scratch, cudaStream_t st);

// One tensor of an optimizer step.
struct AdamwTensor {
  void* p;
  float* master;
  const void* g;
  void* m;
  void* v;
  float* ms;
  float* vs;
  long long n;
  float keep;     // 1 - lr * weight decay
  int p_type, g_type;
  int vec;        // every pointer 16-byte aligned
};
struct AdamwHyper {
  float b1, c1, b2, c2;  // betas and 1 - beta
  float eps, step_size, inv_sqrt_bc2;
  double lr, beta1, beta2;
  const int* step_dev;      // device step count (then the bias corrections are computed in the kernel) or null
  const float* grad_scale;  // device scalar or null
};
constexpr int kAdamwBlock = 256;  // elements of one scale (8-bit moments)
cudaError_t launch_adamw(const AdamwTensor* t, int count, int bits, const AdamwHyper& h, cudaStream_t st);
cudaError_t launch_adamw_decode(const int8_t* m, const float* ms, const uint8_t* v, const float* vs, long long n,
                                int dtype, void* m_out, void* v_out, cudaStream_t st);

int sm_count();

}  // namespace vswin
