// Norms of queries and keys for each head with the position rotation in the
// same pass, and its gradient. For a head's channels x[0..d):
//
//   r = 1 / sqrt(mean(x^2) + eps),  n = x r gamma,
//   y_a = n_a cos - n_b sin,  y_b = n_b cos + n_a sin
//
// for the channel pairs (a, b) of the first `rot` channels ((i, i + rot/2), or
// (2i, 2i+1) when interleaved), y = n for the rest; cos and sin come from the
// row of a table that the token's position names. The rotation is orthogonal,
// so with g = R^T dy:
//
//   dgamma = sum over rows of g x r,   h = g gamma,
//   dx = r (h - x r mean(h x r)).
//
// Both directions are bound by HBM: forward reads x and writes y once, backward
// reads x and dy and writes dx. 32 x 3136 tokens, 12 + 12 heads of 32, bf16: 62 us
// for 309 MB (4.9 TB/s, 0.77 of the measured copy); 4 x 4099 tokens, 16 + 4 heads
// of 128, fp16: forward 35 us for 168 MB, backward 52 us for 252 MB. What is left
// is issue (0.5 - 0.6 of the slots) beside the loads' latency. Vector path: a row is held by d/16 lanes, each
// with 16 channels as eight (a, b) pairs in registers, so that the rotation
// needs no exchange between lanes. A block takes a few whole tokens at a time,
// consecutive lanes consecutive heads, and walks the tokens: a lane keeps its
// head and its gamma, and a position advances by additions alone; the next row's
// pieces are fetched before the current one is worked on (73 us without). The
// arithmetic goes two channels per instruction. Rows whose width, alignment or
// rotation does not split into 16-byte pieces (the rule is vec_ok) go one row per
// warp, element by element (the 309 MB above from an odd address: 500 us).
#include "sequence.h"

namespace vswin {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxD = 256;

template <class T>
struct Vec8 {  // 8 elements, 16-byte pieces
  static constexpr int N = sizeof(T) * 8 / 16;
  uint4 u[N];
};
template <class T>
__device__ __forceinline__ void load8(const T* p, Vec8<T>& v) {
#pragma unroll
  for (int k = 0; k < Vec8<T>::N; ++k) v.u[k] = reinterpret_cast<const uint4*>(p)[k];
}
template <class T>
__device__ __forceinline__ void unpack8(const Vec8<T>& v, float (&f)[8]) {
  const T* e = reinterpret_cast<const T*>(v.u);
#pragma unroll
  for (int k = 0; k < 8; ++k) f[k] = to_f(e[k]);
}
template <class T>
__device__ __forceinline__ void store8(T* p, const float (&f)[8]) {
  Vec8<T> v;
  T* e = reinterpret_cast<T*>(v.u);
#pragma unroll
  for (int k = 0; k < 8; ++k) e[k] = from_f<T>(f[k]);
#pragma unroll
  for (int k = 0; k < Vec8<T>::N; ++k) reinterpret_cast<uint4*>(p)[k] = v.u[k];
}

// Row of the angle tables for token (b, l); a position outside the tables is
// recorded in the error word and the nearest row is used.
__device__ __forceinline__ long long angle_row(const QkNormArgs& a, int b, int l) {
  if (!a.positions) return l;
  int pos = a.positions[(long long)b * a.L + l];
  if (pos < 0 || pos >= a.rows) {
    atomicCAS(a.err, 0, kErrBounds);
    pos = pos < 0 ? 0 : a.rows - 1;
  }
  return pos;
}

// Channels of lane t of a row: two runs of 8, and the first of its eight angles (or -1).
struct LaneChannels {
  int c0, c1;
  int angle;
};
template <bool kInter>
__device__ __forceinline__ LaneChannels lane_channels(const QkNormArgs& a, int t) {
  LaneChannels c;
  const int turned = a.rot / 16;
  c.angle = t < turned ? 8 * t : -1;
  if (!kInter && t < turned) {
    c.c0 = 8 * t;
    c.c1 = 8 * t + a.rot / 2;
  } else {
    c.c0 = 16 * t;
    c.c1 = 16 * t + 8;
  }
  return c;
}

// The two runs as pairs: (a, b) = (run 0, run 1), or even and odd channels.
template <bool kInter>
__device__ __forceinline__ void to_pairs(float (&a)[8], float (&b)[8]) {
  if constexpr (kInter) {
    float x[16];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      x[k] = a[k];
      x[8 + k] = b[k];
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      a[k] = x[2 * k];
      b[k] = x[2 * k + 1];
    }
  }
}
template <bool kInter>
__device__ __forceinline__ void from_pairs(float (&a)[8], float (&b)[8]) {
  if constexpr (kInter) {
    float x[16];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      x[2 * k] = a[k];
      x[2 * k + 1] = b[k];
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      a[k] = x[k];
      b[k] = x[8 + k];
    }
  }
}

__device__ __forceinline__ void load_angles(const QkNormArgs& a, const LaneChannels& c, long long row, float (&cs)[8],
                                            float (&sn)[8]) {
  if (c.angle >= 0) {
    const float4* cp = reinterpret_cast<const float4*>(a.cosp + row * (a.rot / 2) + c.angle);
    const float4* sp = reinterpret_cast<const float4*>(a.sinp + row * (a.rot / 2) + c.angle);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float4 u = __ldg(cp + k), w = __ldg(sp + k);
      cs[4 * k] = u.x, cs[4 * k + 1] = u.y, cs[4 * k + 2] = u.z, cs[4 * k + 3] = u.w;
      sn[4 * k] = w.x, sn[4 * k + 1] = w.y, sn[4 * k + 2] = w.z, sn[4 * k + 3] = w.w;
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) cs[k] = 1.f, sn[k] = 0.f;
  }
}

template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o, G);
  return v;
}

// Tokens of a block's step: whole tokens, a group of G lanes per row; all heads
// of one token in turns when they outnumber the groups.
template <int G>
__host__ __device__ __forceinline__ int tokens_per_step(int heads) {
  return kThreads / G / heads > 0 ? kThreads / G / heads : 1;
}

// The first `qblocks` blocks walk q's tokens, the others k's.
template <class T, int G, bool kBackward, bool kInter>
__global__ void __launch_bounds__(kThreads, kBackward ? 2 : 3)
    qk_norm_vec_kernel(const __grid_constant__ QkNormArgs a, int qblocks, float* partial) {
  if (kBackward) let_next_start();
  const int w = blockIdx.x < qblocks ? 0 : 1;
  const int block = w ? blockIdx.x - qblocks : blockIdx.x;
  const int blocks = w ? gridDim.x - qblocks : qblocks;
  const int heads = a.heads[w];
  const int groups = kThreads / G, per = tokens_per_step<G>(heads), hpb = heads < groups ? heads : groups;
  const int t = threadIdx.x % G, g = threadIdx.x / G;
  const bool live = t < a.d / 16 && g / hpb < per;
  const LaneChannels c = lane_channels<kInter>(a, t);
  const float inv_d = 1.f / (float)a.d;
  float ga[8], gb[8], cs[8], sn[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) ga[k] = gb[k] = 0.f, cs[k] = 1.f, sn[k] = 0.f;
  if (live) {
    Vec8<T> g0, g1;
    load8(static_cast<const T*>(a.gamma[w]) + c.c0, g0);
    load8(static_cast<const T*>(a.gamma[w]) + c.c1, g1);
    unpack8(g0, ga);
    unpack8(g1, gb);
    to_pairs<kInter>(ga, gb);
  }
  float sum_a[8], sum_b[8];
  if (kBackward) {
#pragma unroll
    for (int k = 0; k < 8; ++k) sum_a[k] = sum_b[k] = 0.f;
  }
  // token n of the walk is token l of sequence b; of its heads, h0 on are next
  const int tokens = a.B * a.L;  // below 2^31
  const int step = blocks * per, step_b = step / a.L, step_l = step % a.L;
  int n = block * per + g / hpb, b = n / a.L, l = n % a.L, h0 = 0;
  int left = tokens - block * per;  // the block's first token is there while this is positive: same for every lane
  Vec8<T> u0, u1, d0, d1;
  auto fetch = [&]() {  // a row's pieces, one step ahead of their use (row 0 where there is none)
    const int h = h0 + g % hpb;
    const bool on = live && n < tokens && h < heads;
    const T* xp = static_cast<const T*>(a.x[w].p) + (on ? a.x[w].at(b, l, h) : 0);
    load8(xp + (on ? c.c0 : 0), u0);
    load8(xp + (on ? c.c1 : 0), u1);
    if (kBackward) {
      const T* yp = static_cast<const T*>(a.y[w].p) + (on ? a.y[w].at(b, l, h) : 0);
      load8(yp + (on ? c.c0 : 0), d0);
      load8(yp + (on ? c.c1 : 0), d1);
    }
  };
  if (left > 0) fetch();
  // every lane of a warp makes the same number of turns (the sums below are warp-wide)
  while (left > 0) {
    const int bn = b, ln = l, hn = h0 + g % hpb;
    const bool on = live && n < tokens && hn < heads;
    if (h0 == 0 && on && c.angle >= 0) load_angles(a, c, angle_row(a, b, l), cs, sn);
    float xa[8], xb[8], ya[8], yb[8];
    unpack8(u0, xa);
    unpack8(u1, xb);
    to_pairs<kInter>(xa, xb);
    if (kBackward) {
      unpack8(d0, ya);
      unpack8(d1, yb);
      to_pairs<kInter>(ya, yb);
    }
    h0 += hpb;
    if (h0 >= heads) {
      h0 = 0;
      n += step;
      left -= step;
      b += step_b;
      l += step_l;
      if (l >= a.L) l -= a.L, ++b;
    }
    if (left > 0) fetch();
    float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < 8; k += 2) {
      s2 = __ffma2_rn(make_float2(xa[k], xa[k + 1]), make_float2(xa[k], xa[k + 1]), s2);
      s2 = __ffma2_rn(make_float2(xb[k], xb[k + 1]), make_float2(xb[k], xb[k + 1]), s2);
    }
    // lanes behind the row's width hold another row's channels: their share is not taken
    const float r = rsqrtf(group_sum<G>(t < a.d / 16 ? s2.x + s2.y : 0.f) * inv_d + a.eps);
    const float2 r2 = make_float2(r, r);
    if (!kBackward) {
#pragma unroll
      for (int k = 0; k < 8; k += 2) {
        const float2 cc = make_float2(cs[k], cs[k + 1]), ss = make_float2(sn[k], sn[k + 1]);
        const float2 na = __fmul2_rn(__fmul2_rn(make_float2(xa[k], xa[k + 1]), r2), make_float2(ga[k], ga[k + 1]));
        const float2 nb = __fmul2_rn(__fmul2_rn(make_float2(xb[k], xb[k + 1]), r2), make_float2(gb[k], gb[k + 1]));
        const float2 p = __fmul2_rn(nb, ss);
        const float2 u = __ffma2_rn(na, cc, make_float2(-p.x, -p.y));
        const float2 v = __ffma2_rn(nb, cc, __fmul2_rn(na, ss));
        ya[k] = u.x, ya[k + 1] = u.y, yb[k] = v.x, yb[k + 1] = v.y;
      }
      if (on) {
        from_pairs<kInter>(ya, yb);
        T* yp = static_cast<T*>(a.y[w].p) + a.y[w].at(bn, ln, hn);
        store8(yp + c.c0, ya);
        store8(yp + c.c1, yb);
      }
    } else {
      float2 along2 = make_float2(0.f, 0.f);
#pragma unroll
      for (int k = 0; k < 8; k += 2) {
        const float2 cc = make_float2(cs[k], cs[k + 1]), ss = make_float2(sn[k], sn[k + 1]);
        const float2 da = make_float2(ya[k], ya[k + 1]), db = make_float2(yb[k], yb[k + 1]);
        const float2 p = __fmul2_rn(da, ss);
        const float2 gya = __ffma2_rn(da, cc, __fmul2_rn(db, ss));                   // R^T dy
        const float2 gyb = __ffma2_rn(db, cc, make_float2(-p.x, -p.y));
        const float2 ua = __fmul2_rn(make_float2(xa[k], xa[k + 1]), r2), ub = __fmul2_rn(make_float2(xb[k], xb[k + 1]), r2);
        if (on) {
          const float2 sa = __ffma2_rn(gya, ua, make_float2(sum_a[k], sum_a[k + 1]));
          const float2 sb = __ffma2_rn(gyb, ub, make_float2(sum_b[k], sum_b[k + 1]));
          sum_a[k] = sa.x, sum_a[k + 1] = sa.y, sum_b[k] = sb.x, sum_b[k + 1] = sb.y;
        }
        const float2 ha = __fmul2_rn(gya, make_float2(ga[k], ga[k + 1])), hb = __fmul2_rn(gyb, make_float2(gb[k], gb[k + 1]));
        along2 = __ffma2_rn(ha, ua, along2);
        along2 = __ffma2_rn(hb, ub, along2);
        xa[k] = ua.x, xa[k + 1] = ua.y, xb[k] = ub.x, xb[k + 1] = ub.y;
        ya[k] = ha.x, ya[k + 1] = ha.y, yb[k] = hb.x, yb[k + 1] = hb.y;
      }
      const float along = group_sum<G>(t < a.d / 16 ? along2.x + along2.y : 0.f) * inv_d;
      const float2 m2 = make_float2(-along, -along);
#pragma unroll
      for (int k = 0; k < 8; k += 2) {
        const float2 u = __fmul2_rn(r2, __ffma2_rn(make_float2(xa[k], xa[k + 1]), m2, make_float2(ya[k], ya[k + 1])));
        const float2 v = __fmul2_rn(r2, __ffma2_rn(make_float2(xb[k], xb[k + 1]), m2, make_float2(yb[k], yb[k + 1])));
        ya[k] = u.x, ya[k + 1] = u.y, yb[k] = v.x, yb[k + 1] = v.y;
      }
      if (on) {
        from_pairs<kInter>(ya, yb);
        T* dp = static_cast<T*>(a.dx[w].p) + a.dx[w].at(bn, ln, hn);
        store8(dp + c.c0, ya);
        store8(dp + c.c1, yb);
      }
    }
  }
  if (kBackward) {
    // this block's share of dgamma: lanes of the same channels, then warps, in a fixed order
    __shared__ float s[kThreads / 32][kMaxD];
    from_pairs<kInter>(sum_a, sum_b);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
#pragma unroll
      for (int o = 16; o >= G; o >>= 1) {
        sum_a[k] += __shfl_xor_sync(0xffffffffu, sum_a[k], o);
        sum_b[k] += __shfl_xor_sync(0xffffffffu, sum_b[k], o);
      }
      if (t < a.d / 16 && (threadIdx.x & 31) < G) {
        s[threadIdx.x >> 5][c.c0 + k] = sum_a[k];
        s[threadIdx.x >> 5][c.c1 + k] = sum_b[k];
      }
    }
    __syncthreads();
    for (int ch = threadIdx.x; ch < a.d; ch += kThreads) {
      float v = 0.f;
#pragma unroll
      for (int k = 0; k < kThreads / 32; ++k) v += s[k][ch];
      partial[(long long)blockIdx.x * a.d + ch] = v;
    }
  }
}

// One row per warp, element by element: any even rot, width up to kMaxD, any
// alignment and strides.
template <class T, bool kBackward, int kPer>  // kPer: channels per lane
__global__ void __launch_bounds__(kThreads) qk_norm_any_kernel(QkNormArgs a, int qblocks, float* partial) {
  if (kBackward) let_next_start();
  const int w = blockIdx.x < qblocks ? 0 : 1;
  const int block = w ? blockIdx.x - qblocks : blockIdx.x;
  const int blocks = w ? gridDim.x - qblocks : qblocks;
  const int heads = a.heads[w], d = a.d, half = a.rot / 2;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const T* gamma = static_cast<const T*>(a.gamma[w]);
  float sums[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k) sums[k] = 0.f;
  // the partner of channel c, its angle, and the sign of its sine term
  auto pair = [&](int c, int* other, int* angle, float* sign) {
    *angle = a.interleaved ? c >> 1 : (c < half ? c : c - half);
    const bool first = a.interleaved ? (c & 1) == 0 : c < half;
    *other = a.interleaved ? c ^ 1 : (first ? c + half : c - half);
    *sign = first ? -1.f : 1.f;
  };
  // row after row: head, token and sequence advance by additions
  const int first = block * (kThreads / 32) + warp, step = blocks * (kThreads / 32);
  const int step_h = step % heads, step_l = step / heads % a.L, step_b = step / heads / a.L;
  int h = first % heads, l = first / heads % a.L, b = first / heads / a.L;
  auto next = [&]() {
    h += step_h;
    l += step_l;
    b += step_b;
    if (h >= heads) h -= heads, ++l;
    if (l >= a.L) l -= a.L, ++b;
  };
  for (; b < a.B; next()) {
    const long long arow = a.rot > 0 ? angle_row(a, b, l) : 0;
    const T* xp = static_cast<const T*>(a.x[w].p) + a.x[w].at(b, l, h);
    const T* yp = static_cast<const T*>(a.y[w].p) + a.y[w].at(b, l, h);
    float x[kPer], part[kPer], ss = 0.f;  // own channel, and its partner's of the rotation
    float g[kPer], gpart[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int c = lane + 32 * k;
      x[k] = part[k] = g[k] = gpart[k] = 0.f;
      if (c >= d) continue;
      x[k] = to_f(xp[c]);
      ss = fmaf(x[k], x[k], ss);
      int other = c, angle;
      float sign;
      if (c < a.rot) pair(c, &other, &angle, &sign);
      part[k] = to_f(xp[other]);
      if (kBackward) {
        g[k] = to_f(yp[c]);
        gpart[k] = to_f(yp[other]);
      }
    }
    __syncwarp();  // every element is read before the row may be overwritten in place
    const float r = rsqrtf(group_sum<32>(ss) / (float)d + a.eps);
    float along = 0.f;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int c = lane + 32 * k;
      if (c >= d) continue;
      int other = c, angle = 0;
      float sign = 0.f, cs = 1.f, sn = 0.f;
      if (c < a.rot) {
        pair(c, &other, &angle, &sign);
        cs = a.cosp[arow * half + angle];
        sn = a.sinp[arow * half + angle];
      }
      if (!kBackward) {
        const float n = x[k] * r * to_f(gamma[c]), m = part[k] * r * to_f(gamma[other]);
        static_cast<T*>(a.y[w].p)[a.y[w].at(b, l, h) + c] = from_f<T>(n * cs + sign * m * sn);
      } else {
        const float gy = g[k] * cs - sign * gpart[k] * sn;
        x[k] *= r;
        sums[k] = fmaf(gy, x[k], sums[k]);
        g[k] = gy * to_f(gamma[c]);
        along = fmaf(g[k], x[k], along);
      }
    }
    if (kBackward) {
      along = group_sum<32>(along) / (float)d;
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        const int c = lane + 32 * k;
        if (c < d) static_cast<T*>(a.dx[w].p)[a.dx[w].at(b, l, h) + c] = from_f<T>(r * (g[k] - x[k] * along));
      }
    }
  }
  if (kBackward) {
    __shared__ float s[kThreads / 32][kMaxD];
#pragma unroll
    for (int k = 0; k < kPer; ++k) s[warp][lane + 32 * k] = sums[k];
    __syncthreads();
    for (int ch = threadIdx.x; ch < d; ch += kThreads) {
      float v = 0.f;
#pragma unroll
      for (int k = 0; k < kThreads / 32; ++k) v += s[k][ch];
      partial[(long long)blockIdx.x * d + ch] = v;
    }
  }
}

// dgamma = the blocks' shares added in a fixed order: 32 channels per block, 32
// runs of shares side by side.
__global__ void __launch_bounds__(1024) qk_norm_dgamma_kernel(QkNormArgs a, int qblocks, int blocks,
                                                             const float* partial) {
  after_previous();
  __shared__ float s[32][33];
  const int w = blockIdx.y, lane = threadIdx.x & 31, run = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  const int lo = w ? qblocks : 0, hi = w ? blocks : qblocks;
  float v = 0.f;
  if (c < a.d) {
#pragma unroll 4
    for (int b = lo + run; b < hi; b += 32) v += partial[(long long)b * a.d + c];
  }
  s[run][lane] = v;
  __syncthreads();
  if (run == 0 && c < a.d) {
    for (int k = 1; k < 32; ++k) v += s[k][lane];
    a.dgamma[w][c] = v;
  }
}

bool view_ok(const Heads& v, int esize) {
  const long long m = 16 / esize;
  return reinterpret_cast<uintptr_t>(v.p) % 16 == 0 && v.sb % m == 0 && v.st % m == 0 && v.sh % m == 0;
}

// The vector path needs rows and rotated parts of whole 16-channel pieces and
// 16-byte aligned rows.
bool vec_ok(const QkNormArgs& a, int esize, bool backward) {
  if (a.d % 16 || a.rot % 16 || a.d > kMaxD) return false;
  for (int w = 0; w < 2; ++w) {
    if (!view_ok(a.x[w], esize) || !view_ok(a.y[w], esize) || (backward && !view_ok(a.dx[w], esize))) return false;
    if (reinterpret_cast<uintptr_t>(a.gamma[w]) % 16) return false;
  }
  return a.rot == 0 || (reinterpret_cast<uintptr_t>(a.cosp) % 16 == 0 && reinterpret_cast<uintptr_t>(a.sinp) % 16 == 0);
}

int group_of(int d) {
  int g = 1;
  while (g < d / 16) g *= 2;
  return g;
}

// Blocks of q and of k for steps of `need` rows or tokens: as many as are
// resident, at most one step each when there are few.
void grid_of(const QkNormArgs& a, const long long (&need)[2], int per_sm, int* q, int* k) {
  const long long cap = (long long)sm_count() * per_sm;
  if (need[0] + need[1] <= cap) {
    *q = (int)need[0];
    *k = (int)need[1];
    return;
  }
  long long nq = cap * a.heads[0] / (a.heads[0] + a.heads[1]);
  nq = nq < 1 ? 1 : (nq > cap - 1 ? cap - 1 : nq);
  *q = (int)(nq < need[0] ? nq : need[0]);
  *k = (int)(cap - nq < need[1] ? cap - nq : need[1]);
}

template <class T, bool kBackward>
void plan(const QkNormArgs& a, bool* vec, int* G, int* nq, int* nk) {
  *vec = vec_ok(a, (int)sizeof(T), kBackward);
  *G = *vec ? group_of(a.d) : 32;
  long long need[2];
  for (int w = 0; w < 2; ++w) {
    const long long tokens = (long long)a.B * a.L;
    const int groups = kThreads / *G, per = groups / a.heads[w] > 0 ? groups / a.heads[w] : 1;
    need[w] = *vec ? (tokens + per - 1) / per : (tokens * a.heads[w] + groups - 1) / groups;
  }
  grid_of(a, need, !*vec ? 8 : (kBackward ? 2 : 3), nq, nk);
}

template <class T, bool kBackward, bool kInter>
void launch_vec(const QkNormArgs& a, int G, int grid, int nq, float* partial, cudaStream_t st) {
  if (G == 1)
    qk_norm_vec_kernel<T, 1, kBackward, kInter><<<grid, kThreads, 0, st>>>(a, nq, partial);
  else if (G == 2)
    qk_norm_vec_kernel<T, 2, kBackward, kInter><<<grid, kThreads, 0, st>>>(a, nq, partial);
  else if (G == 4)
    qk_norm_vec_kernel<T, 4, kBackward, kInter><<<grid, kThreads, 0, st>>>(a, nq, partial);
  else if (G == 8)
    qk_norm_vec_kernel<T, 8, kBackward, kInter><<<grid, kThreads, 0, st>>>(a, nq, partial);
  else
    qk_norm_vec_kernel<T, 16, kBackward, kInter><<<grid, kThreads, 0, st>>>(a, nq, partial);
}

template <class T, bool kBackward>
cudaError_t launch(const QkNormArgs& a, float* partial, cudaStream_t st) {
  bool vec;
  int G, nq, nk;
  plan<T, kBackward>(a, &vec, &G, &nq, &nk);
  const int grid = nq + nk;
  prof_begin(kKindOther, st);
  if (!vec && a.d <= 32)
    qk_norm_any_kernel<T, kBackward, 1><<<grid, kThreads, 0, st>>>(a, nq, partial);
  else if (!vec && a.d <= 64)
    qk_norm_any_kernel<T, kBackward, 2><<<grid, kThreads, 0, st>>>(a, nq, partial);
  else if (!vec && a.d <= 128)
    qk_norm_any_kernel<T, kBackward, 4><<<grid, kThreads, 0, st>>>(a, nq, partial);
  else if (!vec)
    qk_norm_any_kernel<T, kBackward, 8><<<grid, kThreads, 0, st>>>(a, nq, partial);
  else if (a.interleaved && a.rot)
    launch_vec<T, kBackward, true>(a, G, grid, nq, partial, st);
  else
    launch_vec<T, kBackward, false>(a, G, grid, nq, partial, st);
  prof_end(kKindOther, st);
  count_launch();
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !kBackward) return e;
  prof_begin(kKindOther, st);
  e = launch_after(qk_norm_dgamma_kernel, dim3((a.d + 31) / 32, 2), 1024, 0, st, a, nq, grid, partial);
  prof_end(kKindOther, st);
  count_launch();
  return e;
}

}  // namespace

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
      n < 1)
    return 1;
  return n;
}

cudaError_t launch_qk_norm_forward(const QkNormArgs& a, int dtype, cudaStream_t st) {
  if (dtype == kBF16) return launch<__nv_bfloat16, false>(a, nullptr, st);
  if (dtype == kFP16) return launch<__half, false>(a, nullptr, st);
  return launch<float, false>(a, nullptr, st);
}

size_t qk_norm_scratch_bytes(const QkNormArgs& a, int dtype) {
  bool vec;
  int G, nq, nk;
  if (dtype == kF32)
    plan<float, true>(a, &vec, &G, &nq, &nk);
  else
    plan<__half, true>(a, &vec, &G, &nq, &nk);
  return (size_t)(nq + nk) * a.d * sizeof(float);
}

cudaError_t launch_qk_norm_backward(const QkNormArgs& a, int dtype, void* scratch, cudaStream_t st) {
  float* partial = static_cast<float*>(scratch);
  if (dtype == kBF16) return launch<__nv_bfloat16, true>(a, partial, st);
  if (dtype == kFP16) return launch<__half, true>(a, partial, st);
  return launch<float, true>(a, partial, st);
}

}  // namespace vswin
