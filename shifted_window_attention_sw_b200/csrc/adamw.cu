// One AdamW step over many tensors in one launch (per kCap tensors):
//
//   g' = g s,  m = b1 m + (1 - b1) g',  v = b2 v + (1 - b2) g'^2,
//   p = p (1 - lr wd) - (lr / (1 - b1^t)) m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// in fp32; p in bf16, fp16 or fp32, optionally with an fp32 master copy that
// is updated and rounded into p. Moments are fp32, or 8-bit codes with one fp32
// scale s (the block's largest value) per 256 elements of a tensor:
//   m: code c in [-127, 127], value s sgn(c) (c / 127)^2   (square-root spacing)
//   v: code c in [0, 255],    value s (c / 255)^4          (fourth-root spacing)
// rounded to the nearest code in that spacing; a positive v keeps a code of at
// least 1, so that it never reads back as zero under the square root.
//
// Bound by HBM: each state is read and written once. A tensor is cut into
// chunks of kChunk elements; the blocks walk the chunks of all tensors (whose
// records travel as the kernel's parameter, so that nothing is uploaded and the
// step can be captured), eight elements per thread. With 8-bit moments a warp
// holds one block of 256 and finds its scale by shuffles.
#include <cmath>

#include "sequence.h"

namespace vswin {
namespace {

constexpr int kThreads = 256;
constexpr int kChunk = kThreads * 8;

template <int kCap>
struct Table {
  AdamwTensor t[kCap];
  long long first[kCap + 1];  // chunks before tensor i
  int count;
};

// Eight elements from index i of n; elements past n read as zero.
__device__ __forceinline__ void load_elems(const void* p, int type, bool vec, long long i, long long n, float (&f)[8]) {
  if (vec && i + 8 <= n) {
    if (type == kF32) {
      const float4 a = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i)[0];
      const float4 b = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i)[1];
      f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
    } else {
      const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (type == kBF16) {
          f[2 * k] = __uint_as_float(w[k] << 16);
          f[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
        } else {
          const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
          f[2 * k] = h.x;
          f[2 * k + 1] = h.y;
        }
      }
    }
    return;
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    f[k] = 0.f;
    if (i + k < n)
      f[k] = type == kF32    ? static_cast<const float*>(p)[i + k]
             : type == kBF16 ? to_f(static_cast<const __nv_bfloat16*>(p)[i + k])
                             : to_f(static_cast<const __half*>(p)[i + k]);
  }
}

__device__ __forceinline__ void store_elems(void* p, int type, bool vec, long long i, long long n,
                                            const float (&f)[8]) {
  if (vec && i + 8 <= n) {
    if (type == kF32) {
      float4* o = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
      o[0] = make_float4(f[0], f[1], f[2], f[3]);
      o[1] = make_float4(f[4], f[5], f[6], f[7]);
    } else {
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (type == kBF16) {
          const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * k], f[2 * k + 1]);
          w[k] = *reinterpret_cast<const uint32_t*>(&h);
        } else {
          const __half2 h = __floats2half2_rn(f[2 * k], f[2 * k + 1]);
          w[k] = *reinterpret_cast<const uint32_t*>(&h);
        }
      }
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    return;
  }
#pragma unroll
  for (int k = 0; k < 8; ++k)
    if (i + k < n) {
      if (type == kF32)
        static_cast<float*>(p)[i + k] = f[k];
      else if (type == kBF16)
        static_cast<__nv_bfloat16*>(p)[i + k] = from_f<__nv_bfloat16>(f[k]);
      else
        static_cast<__half*>(p)[i + k] = from_f<__half>(f[k]);
    }
}

__device__ __forceinline__ uint2 load_codes(const void* p, bool vec, long long i, long long n) {
  const uint8_t* b = static_cast<const uint8_t*>(p);
  if (vec && i + 8 <= n) return *reinterpret_cast<const uint2*>(b + i);
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int k = 0; k < 8; ++k)
    if (i + k < n) w[k >> 2] |= (uint32_t)b[i + k] << (8 * (k & 3));
  return make_uint2(w[0], w[1]);
}
__device__ __forceinline__ void store_codes(void* p, bool vec, long long i, long long n, uint2 c) {
  uint8_t* b = static_cast<uint8_t*>(p);
  if (vec && i + 8 <= n) {
    *reinterpret_cast<uint2*>(b + i) = c;
    return;
  }
  const uint32_t w[2] = {c.x, c.y};
#pragma unroll
  for (int k = 0; k < 8; ++k)
    if (i + k < n) b[i + k] = (uint8_t)(w[k >> 2] >> (8 * (k & 3)));
}

__device__ __forceinline__ float decode_m(int c, float s) {
  const float x = (float)c * (1.f / 127.f);
  return s * x * fabsf(x);
}
__device__ __forceinline__ float decode_v(int c, float s) {
  const float x = (float)c * (1.f / 255.f);
  const float x2 = x * x;
  return s * (x2 * x2);
}

// The largest value of a warp, a NaN anywhere making it NaN (so that the block
// reads back as NaN and is not silently lost).
__device__ __forceinline__ float warp_max_nan(float x, bool nan) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return __any_sync(0xffffffffu, nan) ? __int_as_float(0x7fffffff) : x;
}

template <int kCap, int kBits>
__global__ void __launch_bounds__(kThreads) adamw_kernel(const __grid_constant__ Table<kCap> tab, AdamwHyper h) {
  float step_size = h.step_size, inv_bc2 = h.inv_sqrt_bc2;
  if (h.step_dev) {  // the bias corrections of a step count that lives on the device
    __shared__ float s[2];
    if (threadIdx.x == 0) {
      const int n = *h.step_dev;
      s[0] = (float)(h.lr / (1.0 - pow(h.beta1, (double)n)));
      s[1] = (float)(1.0 / sqrt(1.0 - pow(h.beta2, (double)n)));
    }
    __syncthreads();
    step_size = s[0];
    inv_bc2 = s[1];
  }
  const float gs = h.grad_scale ? *h.grad_scale : 1.f;
  const int lane = threadIdx.x & 31;
  for (long long chunk = blockIdx.x; chunk < tab.first[tab.count]; chunk += gridDim.x) {
    int lo = 0, hi = tab.count - 1;  // the tensor of this chunk
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (tab.first[mid] <= chunk)
        lo = mid;
      else
        hi = mid - 1;
    }
    const AdamwTensor& t = tab.t[lo];
    const long long n = t.n, i = (chunk - tab.first[lo]) * kChunk + threadIdx.x * 8;
    if (kBits == 32 && i >= n) continue;
    if (kBits == 8 && i - lane * 8 >= n) continue;  // a whole warp's block lies behind the tensor
    const bool vec = t.vec != 0;
    float p[8], g[8], m[8], v[8];
    load_elems(t.master ? (const void*)t.master : t.p, t.master ? kF32 : t.p_type, vec, i, n, p);
    load_elems(t.g, t.g_type, vec, i, n, g);
    if (kBits == 32) {
      load_elems(t.m, kF32, vec, i, n, m);
      load_elems(t.v, kF32, vec, i, n, v);
    } else {
      const uint2 cm = load_codes(t.m, vec, i, n), cv = load_codes(t.v, vec, i, n);
      const float sm = t.ms[i / kAdamwBlock], sv = t.vs[i / kAdamwBlock];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        m[k] = decode_m((int)(int8_t)((k < 4 ? cm.x : cm.y) >> (8 * (k & 3))), sm);
        v[k] = decode_v((int)(((k < 4 ? cv.x : cv.y) >> (8 * (k & 3))) & 255u), sv);
      }
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float gr = g[k] * gs;
      m[k] = h.b1 * m[k] + h.c1 * gr;
      v[k] = h.b2 * v[k] + h.c2 * (gr * gr);
      p[k] = t.keep * p[k] - step_size * (m[k] / (sqrtf(v[k]) * inv_bc2 + h.eps));
    }
    if (t.master) store_elems(t.master, kF32, vec, i, n, p);
    store_elems(t.p, t.p_type, vec, i, n, p);
    if (kBits == 32) {
      store_elems(t.m, kF32, vec, i, n, m);
      store_elems(t.v, kF32, vec, i, n, v);
    } else {
      float am = 0.f, av = 0.f;
      bool nan_m = false, nan_v = false;
#pragma unroll
      for (int k = 0; k < 8; ++k) {  // elements behind the tensor are zero here
        am = fmaxf(am, fabsf(m[k]));
        av = fmaxf(av, v[k]);
        nan_m |= m[k] != m[k];
        nan_v |= v[k] != v[k];
      }
      const float sm = warp_max_nan(am, nan_m), sv = warp_max_nan(av, nan_v);
      const float im = sm > 0.f ? 1.f / sm : 0.f, iv = sv > 0.f ? 1.f / sv : 0.f;
      uint32_t cm[2] = {0, 0}, cv[2] = {0, 0};
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        // the clamps matter where 1 / s overflows (s below 2^-128)
        const int a = (int)fminf(rintf(sqrtf(fabsf(m[k]) * im) * 127.f), 127.f);
        int b = (int)fminf(rintf(sqrtf(sqrtf(v[k] * iv)) * 255.f), 255.f);
        b = v[k] > 0.f && b < 1 ? 1 : b;
        cm[k >> 2] |= (uint32_t)((m[k] < 0.f ? -a : a) & 255) << (8 * (k & 3));
        cv[k >> 2] |= (uint32_t)(b & 255) << (8 * (k & 3));
      }
      store_codes(t.m, vec, i, n, make_uint2(cm[0], cm[1]));
      store_codes(t.v, vec, i, n, make_uint2(cv[0], cv[1]));
      if (lane == 0) {
        t.ms[i / kAdamwBlock] = sm;
        t.vs[i / kAdamwBlock] = sv;
      }
    }
  }
}

__global__ void __launch_bounds__(kThreads) adamw_decode_kernel(const int8_t* m, const float* ms, const uint8_t* v,
                                                               const float* vs, long long n, int dtype, bool vec,
                                                               void* mo, void* vo) {
  for (long long i = ((long long)blockIdx.x * kThreads + threadIdx.x) * 8; i < n;
       i += (long long)gridDim.x * kThreads * 8) {
    const uint2 cm = load_codes(m, vec, i, n), cv = load_codes(v, vec, i, n);
    const float sm = ms[i / kAdamwBlock], sv = vs[i / kAdamwBlock];
    float fm[8], fv[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      fm[k] = decode_m((int)(int8_t)((k < 4 ? cm.x : cm.y) >> (8 * (k & 3))), sm);
      fv[k] = decode_v((int)(((k < 4 ? cv.x : cv.y) >> (8 * (k & 3))) & 255u), sv);
    }
    store_elems(mo, dtype, vec, i, n, fm);
    store_elems(vo, dtype, vec, i, n, fv);
  }
}

template <int kCap>
cudaError_t launch_cap(const AdamwTensor* t, int count, int bits, const AdamwHyper& h, cudaStream_t st) {
  Table<kCap> tab;
  long long chunks = 0;
  for (int i = 0; i < count; ++i) {
    tab.t[i] = t[i];
    tab.first[i] = chunks;
    chunks += (t[i].n + kChunk - 1) / kChunk;
  }
  tab.first[count] = chunks;
  tab.count = count;
  if (chunks == 0) return cudaSuccess;
  const long long cap = (long long)sm_count() * 8;
  const int grid = (int)(chunks < cap ? chunks : cap);
  prof_begin(kKindOther, st);
  if (bits == 32)
    adamw_kernel<kCap, 32><<<grid, kThreads, 0, st>>>(tab, h);
  else
    adamw_kernel<kCap, 8><<<grid, kThreads, 0, st>>>(tab, h);
  prof_end(kKindOther, st);
  count_launch();
  return cudaGetLastError();
}

}  // namespace

// Records travel as the kernel's parameter: 16 of them in a small launch, at
// most 192 (about 17 KB) in a large one.
cudaError_t launch_adamw(const AdamwTensor* t, int count, int bits, const AdamwHyper& h, cudaStream_t st) {
  constexpr int kSmall = 16, kLarge = 192;
  for (int i = 0; i < count; i += kLarge) {
    const int n = count - i < kLarge ? count - i : kLarge;
    const cudaError_t e = n <= kSmall ? launch_cap<kSmall>(t + i, n, bits, h, st) : launch_cap<kLarge>(t + i, n, bits, h, st);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_adamw_decode(const int8_t* m, const float* ms, const uint8_t* v, const float* vs, long long n,
                                int dtype, void* m_out, void* v_out, cudaStream_t st) {
  if (n == 0) return cudaSuccess;
  const uintptr_t all = reinterpret_cast<uintptr_t>(m) | reinterpret_cast<uintptr_t>(v) |
                        reinterpret_cast<uintptr_t>(m_out) | reinterpret_cast<uintptr_t>(v_out);
  const long long need = (n + kChunk - 1) / kChunk, cap = (long long)sm_count() * 8;
  prof_begin(kKindOther, st);
  adamw_decode_kernel<<<(int)(need < cap ? need : cap), kThreads, 0, st>>>(m, ms, v, vs, n, dtype, all % 16 == 0,
                                                                          m_out, v_out);
  prof_end(kKindOther, st);
  count_launch();
  return cudaGetLastError();
}

}  // namespace vswin
