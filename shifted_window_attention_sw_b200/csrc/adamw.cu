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
// Bound by HBM: each state is read and written once. 25 M bf16 weights with fp32
// moments and copies: 117 us for 809 MB (6.9 TB/s; a part stays in L2). With 8-bit
// moments the coding counts (0.64 of the issue slots, 0.37 of the special-function
// units): 63 M bf16 weights, 190 us for 635 MB; the decoding of their moments 76 us
// for 378 MB. A tensor is cut into chunks; the blocks walk the chunks of all tensors (whose
// records travel as the kernel's parameter, so that nothing is uploaded and the
// step can be captured), eight elements per thread. With 8-bit moments a warp
// holds one block of 256 and finds its scale by shuffles.
#include <cmath>

#include "sequence.h"

namespace vswin {
namespace {

constexpr int kThreads = 256;
constexpr int kRun = kThreads * 8;  // elements of a block's run

template <int kCap>
struct Table {
  AdamwTensor t[kCap];
  long long first[kCap + 1];  // chunks before tensor i
  int count;
  int chunk;                  // elements of a chunk: one run, or two when there are chunks for every block
};

// Eight elements from index i of n, as they stand in memory (a 16-bit type fills
// the first half); elements past n read as zero. Fetched first and converted when
// every buffer's loads are under way: a conversion beside its load would wait for
// each in turn (25 M weights with fp32 moments and copies: 134 us instead of 121; 63 M with
// 8-bit moments: 220 instead of 196).
struct Raw {
  uint32_t w[8];
};
__device__ __forceinline__ Raw fetch(const void* p, int type, bool vec, long long i, long long n) {
  Raw r;
  const bool wide = type == kF32;
  if (vec && i + 8 <= n) {
    const uint4* at = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p) + i * (wide ? 4 : 2));
    const uint4 x = at[0];
    uint4 y = make_uint4(0, 0, 0, 0);
    if (wide) y = at[1];
    r = Raw{{x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w}};
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) r.w[k] = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (i + k >= n) continue;
      if (wide)
        r.w[k] = static_cast<const uint32_t*>(p)[i + k];
      else
        r.w[k / 2] |= (uint32_t) static_cast<const uint16_t*>(p)[i + k] << (16 * (k & 1));
    }
  }
  return r;
}
__device__ __forceinline__ void convert(const Raw& r, int type, float (&f)[8]) {
  if (type == kF32) {
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = __uint_as_float(r.w[k]);
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (type == kBF16) {
        f[2 * k] = __uint_as_float(r.w[k] << 16);
        f[2 * k + 1] = __uint_as_float(r.w[k] & 0xffff0000u);
      } else {
        const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&r.w[k]));
        f[2 * k] = h.x;
        f[2 * k + 1] = h.y;
      }
    }
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

// Byte k of w as a float, and back: 2^23 + n has n in its low bits, so a byte
// permutation and one addition convert (the conversion instructions run at a
// quarter of the rate).
__device__ __forceinline__ float byte_bits(uint32_t w, int k) {  // 2^23 + byte
  return __uint_as_float(__byte_perm(w, 0x4b000000u, 0x7540 + k));
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 round_bytes(float2 x) { return __fadd2_rn(x, both(12582912.f)); }  // low byte of each: rint(x)
__device__ __forceinline__ uint32_t pack_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}
// Values of codes, with s / 127^2 and s / 255^4 for s. Signed codes come as bytes
// with the sign bit flipped (code + 128).
constexpr float kUnitM = 1.f / (127.f * 127.f), kUnitV = 1.f / (255.f * 255.f * 255.f * 255.f);
__device__ __forceinline__ float2 decode_m2(uint32_t w, int k, float s) {  // bytes k and k + 1
  const float2 c = __fadd2_rn(make_float2(byte_bits(w, k), byte_bits(w, k + 1)), both(-8388736.f));
  return __fmul2_rn(both(s), make_float2(c.x * fabsf(c.x), c.y * fabsf(c.y)));
}
__device__ __forceinline__ float2 decode_v2(uint32_t w, int k, float s) {
  const float2 c = __fadd2_rn(make_float2(byte_bits(w, k), byte_bits(w, k + 1)), both(-8388608.f));
  const float2 c2 = __fmul2_rn(c, c);
  return __fmul2_rn(both(s), __fmul2_rn(c2, c2));
}
constexpr uint32_t kFlip = 0x80808080u;

// Hardware square roots, within 2 units of the last place.
__device__ __forceinline__ float sqrt_fast(float x) {
  float y;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float sqrt_flush(float x) {
  float y;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Largest magnitudes, a NaN anywhere making them NaN (so that its block reads
// back as NaN and is not silently lost).
__device__ __forceinline__ float max3_nan(float x, float y, float z) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
  return r;
}
__device__ __forceinline__ float warp_max_nan(float x) {
  float r;
  asm volatile("redux.sync.max.abs.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}
// The larger of two, NaN when one of them is.
__device__ __forceinline__ float max_nan(float x, float y) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float rcp_fast(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
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
  int at = 0;  // tensor of the chunk: chunks only go up
  for (long long chunk = blockIdx.x; chunk < tab.first[tab.count]; chunk += gridDim.x) {
    if (chunk >= tab.first[at + 1]) {
      int hi = tab.count - 1;
      while (at < hi) {
        const int mid = (at + hi + 1) / 2;
        if (tab.first[mid] <= chunk)
          at = mid;
        else
          hi = mid - 1;
      }
    }
    const AdamwTensor& t = tab.t[at];
    const long long n = t.n, start = (chunk - tab.first[at]) * tab.chunk + threadIdx.x * 8;
    for (long long i = start; i < start + tab.chunk; i += kRun) {
      if (kBits == 32 && i >= n) break;
      if (kBits == 8 && i - lane * 8 >= n) break;  // a whole warp's block lies behind the tensor
      const bool vec = t.vec != 0;
      float p[8], g[8], m[8], v[8];
      const int from_type = t.master ? kF32 : t.p_type;
      const Raw rp = fetch(t.master ? (const void*)t.master : t.p, from_type, vec, i, n);
      const Raw rg = fetch(t.g, t.g_type, vec, i, n);
      if constexpr (kBits == 32) {
        const Raw rm = fetch(t.m, kF32, vec, i, n), rv = fetch(t.v, kF32, vec, i, n);
        convert(rp, from_type, p);
        convert(rg, t.g_type, g);
        convert(rm, kF32, m);
        convert(rv, kF32, v);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float gr = g[k] * gs;
          m[k] = h.b1 * m[k] + h.c1 * gr;
          v[k] = h.b2 * v[k] + (h.c2 * gr) * gr;
          p[k] = t.keep * p[k] - (step_size * m[k]) * rcp_fast(sqrt_fast(v[k]) * inv_bc2 + h.eps);
        }
      } else {
        const uint2 cm = load_codes(t.m, vec, i, n), cv = load_codes(t.v, vec, i, n);
        const float sm = t.ms[i / kAdamwBlock] * kUnitM, sv = t.vs[i / kAdamwBlock] * kUnitV;
        convert(rp, from_type, p);
        convert(rg, t.g_type, g);
        float root[8];  // sqrt(v)
        // (bound by the instructions issued, hence two elements per instruction)
#pragma unroll
        for (int k = 0; k < 8; k += 2) {
          const float2 old_m = decode_m2((k < 4 ? cm.x : cm.y) ^ kFlip, k & 3, sm);
          const float2 old_v = decode_v2(k < 4 ? cv.x : cv.y, k & 3, sv);
          const float2 gr = __fmul2_rn(make_float2(g[k], g[k + 1]), both(gs));
          const float2 m2 = __ffma2_rn(both(h.b1), old_m, __fmul2_rn(both(h.c1), gr));
          const float2 v2 = __ffma2_rn(both(h.b2), old_v, __fmul2_rn(__fmul2_rn(both(h.c2), gr), gr));
          // (8-bit moments do not resolve v below 2^-126: the root may flush)
          root[k] = sqrt_flush(v2.x);
          root[k + 1] = sqrt_flush(v2.y);
          const float2 d = __ffma2_rn(make_float2(root[k], root[k + 1]), both(inv_bc2), both(h.eps));
          // (a NaN v has to reach the weight)
          const float2 inv = make_float2(rcp_fast(max_nan(d.x, 0x1p-66f)), rcp_fast(max_nan(d.y, 0x1p-66f)));
          const float2 p2 = __ffma2_rn(__fmul2_rn(both(-step_size), m2), inv, __fmul2_rn(both(t.keep), make_float2(p[k], p[k + 1])));
          m[k] = m2.x, m[k + 1] = m2.y, v[k] = v2.x, v[k + 1] = v2.y, p[k] = p2.x, p[k + 1] = p2.y;
        }
        if (i + 8 > n) {  // elements behind the tensor (their code 0 of an infinite or NaN scale is NaN)
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (i + k >= n) m[k] = v[k] = 0.f;
        }
        const float top_m = warp_max_nan(max3_nan(max3_nan(m[0], m[1], m[2]), max3_nan(m[3], m[4], m[5]), max3_nan(m[6], m[7], 0.f)));
        const float top_v = warp_max_nan(max3_nan(max3_nan(v[0], v[1], v[2]), max3_nan(v[3], v[4], v[5]), max3_nan(v[6], v[7], 0.f)));
        // code = 127 sqrt(|m| / s), 255 sqrt(sqrt(v) / sqrt(s)); blocks below 2^-100 have no use for codes, and 1 / s no overflow
        const float im = top_m >= 0x1p-100f ? 127.f * 127.f / top_m : 0.f;
        const float iv = top_v >= 0x1p-100f ? 255.f * 255.f * rsqrtf(top_v) : 0.f;
        uint32_t um[8], uv[8];
#pragma unroll
        for (int k = 0; k < 8; k += 2) {
          const float2 x = __fmul2_rn(make_float2(m[k], m[k + 1]), both(im));
          const float2 y = __fmul2_rn(make_float2(root[k], root[k + 1]), both(iv));
          const float2 a = round_bytes(make_float2(copysignf(sqrt_flush(fabsf(x.x)), x.x), copysignf(sqrt_flush(fabsf(x.y)), x.y)));
          const float2 c = round_bytes(make_float2(fmaxf(sqrt_flush(y.x), v[k] > 0.f ? 1.f : 0.f),
                                                   fmaxf(sqrt_flush(y.y), v[k + 1] > 0.f ? 1.f : 0.f)));
          um[k] = __float_as_uint(a.x), um[k + 1] = __float_as_uint(a.y);
          uv[k] = __float_as_uint(c.x), uv[k + 1] = __float_as_uint(c.y);
        }
        store_codes(t.m, vec, i, n, make_uint2(pack_bytes(um[0], um[1], um[2], um[3]), pack_bytes(um[4], um[5], um[6], um[7])));
        store_codes(t.v, vec, i, n, make_uint2(pack_bytes(uv[0], uv[1], uv[2], uv[3]), pack_bytes(uv[4], uv[5], uv[6], uv[7])));
        if (lane == 0) {
          t.ms[i / kAdamwBlock] = top_m;
          t.vs[i / kAdamwBlock] = top_v;
        }
      }
      if (t.master) store_elems(t.master, kF32, vec, i, n, p);
      store_elems(t.p, t.p_type, vec, i, n, p);
      if constexpr (kBits == 32) {
        store_elems(t.m, kF32, vec, i, n, m);
        store_elems(t.v, kF32, vec, i, n, v);
      }
    }
  }
}

// Sixteen elements a thread, so that 32 bytes of codes are in flight.
template <int kType>
__global__ void __launch_bounds__(kThreads) adamw_decode_kernel(const int8_t* m, const float* ms, const uint8_t* v,
                                                               const float* vs, long long n, bool vec, void* mo, void* vo) {
  const long long i = ((long long)blockIdx.x * kThreads + threadIdx.x) * 16;
  if (i >= n) return;
  const float sm = ms[i / kAdamwBlock] * kUnitM, sv = vs[i / kAdamwBlock] * kUnitV;
  uint4 cm, cv;
  if (vec && i + 16 <= n) {
    cm = *reinterpret_cast<const uint4*>(m + i);
    cv = *reinterpret_cast<const uint4*>(v + i);
  } else {
    const uint2 a = load_codes(m, false, i, n), b = load_codes(m, false, i + 8, n);
    const uint2 c = load_codes(v, false, i, n), d = load_codes(v, false, i + 8, n);
    cm = make_uint4(a.x, a.y, b.x, b.y);
    cv = make_uint4(c.x, c.y, d.x, d.y);
  }
  const uint32_t wm[4] = {cm.x ^ kFlip, cm.y ^ kFlip, cm.z ^ kFlip, cm.w ^ kFlip}, wv[4] = {cv.x, cv.y, cv.z, cv.w};
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    float fm[8], fv[8];
#pragma unroll
    for (int k = 0; k < 8; k += 2) {
      const float2 x = decode_m2(wm[2 * e + k / 4], k & 3, sm), y = decode_v2(wv[2 * e + k / 4], k & 3, sv);
      fm[k] = x.x, fm[k + 1] = x.y, fv[k] = y.x, fv[k + 1] = y.y;
    }
    store_elems(mo, kType, vec, i + 8 * e, n, fm);
    store_elems(vo, kType, vec, i + 8 * e, n, fv);
  }
}

template <int kCap>
cudaError_t launch_cap(const AdamwTensor* t, int count, int bits, const AdamwHyper& h, cudaStream_t st) {
  Table<kCap> tab;
  // 32 bits: short-lived blocks, whose loads overlap others' stores (4, 8, 16 blocks per SM: 129, 121, 117 us for 25 M
  // weights with fp32 copies); 8 bits: the resident ones (4, 8, 16: 189, 197, 202 us for 63 M)
  const long long cap = (long long)sm_count() * (bits == 32 ? 16 : 4);
  long long chunks = 0;
  for (int i = 0; i < count; ++i) chunks += (t[i].n + kRun - 1) / kRun;
  tab.chunk = chunks > 2 * cap ? 2 * kRun : kRun;
  chunks = 0;
  for (int i = 0; i < count; ++i) {
    tab.t[i] = t[i];
    tab.first[i] = chunks;
    chunks += (t[i].n + tab.chunk - 1) / tab.chunk;
  }
  tab.first[count] = chunks;
  tab.count = count;
  if (chunks == 0) return cudaSuccess;
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
  const bool vec = all % 16 == 0;
  const long long blocks = (n + 16 * kThreads - 1) / (16 * kThreads);
  if (blocks > 2147483647LL) return cudaErrorInvalidConfiguration;
  prof_begin(kKindOther, st);
  if (dtype == kBF16)
    adamw_decode_kernel<kBF16><<<(unsigned)blocks, kThreads, 0, st>>>(m, ms, v, vs, n, vec, m_out, v_out);
  else if (dtype == kFP16)
    adamw_decode_kernel<kFP16><<<(unsigned)blocks, kThreads, 0, st>>>(m, ms, v, vs, n, vec, m_out, v_out);
  else
    adamw_decode_kernel<kF32><<<(unsigned)blocks, kThreads, 0, st>>>(m, ms, v, vs, n, vec, m_out, v_out);
  prof_end(kKindOther, st);
  count_launch();
  return cudaGetLastError();
}

}  // namespace vswin
