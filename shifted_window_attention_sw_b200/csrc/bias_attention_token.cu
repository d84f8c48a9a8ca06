// Attention with bucketed bias for few query rows (new tokens against a cache),
// and the join of partial results.
//
// attn_token_kernel: one CTA per 16 rows (the Lq tokens of the query heads that
// share a key head: row r is token r / G, head r % G of the G), and part of the
// keys. Bound by HBM: K and V are read once per 16 rows. Each of the four warps
// walks its own 16-key pieces, fetched with cp.async into a ring of its own (no
// block-wide barrier in the loop), multiplies them with mma.sync m16n8k16
// (16 rows; at so few rows tcgen05's 128 would be seven eighths empty, and the
// copies are the bound either way) and keeps its own running maximum, sum and
// O; the warps' results join in shared memory, the key parts' in
// attn_join_kernel. One token of 16 sequences, caches of up to 16384 tokens, 16
// heads over 4 of 64: 41 + 6 us for 201 MB (31 us at the measured copy's rate). P
// is rounded to 16 bits as an operand; sums and statistics are fp32. The pieces are
// swizzled tiles, which cp.async writes and ldmatrix reads without bank conflicts.
#include "bias_attention.cuh"
#include "bias_attention_split.h"

namespace vswin {
namespace {

constexpr int kWarps = 4;
constexpr int kPiece = 16;  // keys
constexpr int kRows = 16;

template <int D>
struct TokCfg {
  static constexpr int ST = D == 32 ? 4 : 3;       // pieces of a warp's ring
  static constexpr int CTAS = D == 128 ? 2 : 4;    // per SM: warps hide each other's latencies
  static constexpr int kTile = kPiece * D * 2;
  static constexpr int kWarpBytes = ST * 2 * kTile;
  static constexpr int SMEM = kWarps * kWarpBytes;
  static_assert(SMEM >= kWarps * kRows * (D + 2) * 4, "the warps' results fit in the ring");
};

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
template <class T>
__device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (std::is_same<T, __half>::value)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <class T, int D>
__global__ void __launch_bounds__(32 * kWarps, TokCfg<D>::CTAS)
    attn_token_kernel(const __grid_constant__ BiasAttnArgs a, Split sp, int blocks) {
  using C = TokCfg<D>;
  if (sp.n > 1) let_next_start();
  extern __shared__ __align__(1024) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gr = lane >> 2, qc = lane & 3;
  const int group = a.hq / a.hk, rows = a.Lq * group;
  // consecutive CTAs: the row blocks of one part of the keys (they share it in L2)
  int id = blockIdx.x;
  const int rb = id % blocks;
  id /= blocks;
  const int split = id % sp.n;
  id /= sp.n;
  const int hk = id % a.hk, b = id / a.hk;
  const SeqLens sl = seq_lens(a, b);
  const int r0 = rb * kRows;
  // the two rows of this lane's fragments
  int head[2], tok[2], pos[2];
  bool row_ok[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int r = r0 + gr + 8 * e;
    tok[e] = r / group;
    head[e] = hk * group + r % group;
    row_ok[e] = r < rows && tok[e] < sl.nq;
    if (r >= rows) tok[e] = 0, head[e] = hk * group;
    pos[e] = sl.start + tok[e];
  }
  const int first_tok = r0 / group, last_tok = min((r0 + kRows - 1) / group, a.Lq - 1);
  int nk = first_tok < sl.nq ? sl.nk : 0;
  if (a.causal) nk = min(nk, max(0, sl.start + min(last_tok + 1, sl.nq)));
  // the sequence's keys in sp.n equal parts of whole rounds of the warps
  const int chunk = (sl.nk + sp.n * kPiece * kWarps - 1) / (sp.n * kPiece * kWarps) * (kPiece * kWarps);
  const int j_lo = min(split * chunk, nk), j_hi = min(j_lo + chunk, nk);

  // q fragments: lane (gr, qc) holds channels 16 k + 2 qc, + 1 (and + 8) of rows gr and gr + 8
  uint32_t qf[D / 16][4];
#pragma unroll
  for (int k = 0; k < D / 16; ++k)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const T* q = static_cast<const T*>(a.q.p) + a.q.at(b, tok[e], head[e]) + 16 * k + 2 * qc;
      qf[k][e] = row_ok[e] ? *reinterpret_cast<const uint32_t*>(q) : 0u;
      qf[k][e + 2] = row_ok[e] ? *reinterpret_cast<const uint32_t*>(q + 8) : 0u;
    }
  float far[2];  // bias left of the map
#pragma unroll
  for (int e = 0; e < 2; ++e) far[e] = bias_of<T>(a, -a.D, head[e]) * kLog2E;

  const uint32_t ring = smem_u32(smem + warp * C::kWarpBytes);
  const T* kh = static_cast<const T*>(a.k.p) + a.k.at(b, 0, hk);
  const T* vh = static_cast<const T*>(a.v.p) + a.v.at(b, 0, hk);
  const int pieces = (j_hi - j_lo + kPiece - 1) / kPiece;
  const int mine = pieces > warp ? (pieces - warp + kWarps - 1) / kWarps : 0;
  auto fetch = [&](int n) {  // the warp's n-th piece
    if (n < mine) {
      const int j = j_lo + (warp + n * kWarps) * kPiece;
      const uint32_t to = ring + (n % C::ST) * 2 * C::kTile;
      load_tile<T, D, kPiece, 32>(to, kh, a.k.st, j, j_hi, lane);
      load_tile<T, D, kPiece, 32>(to + C::kTile, vh, a.v.st, j, j_hi, lane);
    }
    cp_async_commit();
  };
#pragma unroll
  for (int n = 0; n < C::ST - 1; ++n) fetch(n);

  float m[2] = {0.f, 0.f}, l[2] = {0.f, 0.f};
  bool any[2] = {false, false};  // some key seen so far (in this lane's quad)
  float o[D / 8][4];
#pragma unroll
  for (int n = 0; n < D / 8; ++n)
#pragma unroll
    for (int k = 0; k < 4; ++k) o[n][k] = 0.f;
  const float c = a.scale * kLog2E;
  for (int n = 0; n < mine; ++n) {
    __syncwarp();  // the slot that is fetched into has been read by every lane
    fetch(n + C::ST - 1);
    cp_async_wait<C::ST - 1>();
    __syncwarp();
    const int j0 = j_lo + (warp + n * kWarps) * kPiece;
    const uint32_t at = ring + (n % C::ST) * 2 * C::kTile;
    float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
    // lanes 8 x .. 8 x + 7 address matrix x: channels 8 (2 k + x % 2).. of keys 8 (x / 2)..
    const int krow = (lane >> 4) * 8 + (lane & 7), kchunk = (lane >> 3) & 1;
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      uint32_t f[4];
      ldmatrix4(f, at + TileOf<D>::offset(kPiece, krow, 2 * k + kchunk));
      mma16<T>(s[0], qf[k], f[0], f[1]);
      mma16<T>(s[1], qf[k], f[2], f[3]);
    }
    // s[t][2 e + u]: row gr + 8 e, key j0 + 8 t + 2 qc + u
    const bool far_piece = j0 + kPiece - 1 - (sl.start + first_tok) <= -a.D;
    const bool whole = j0 + kPiece <= j_hi && (!a.causal || j0 + kPiece - 1 <= sl.start + first_tok);
    float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int e = k >> 1, j = j0 + 8 * t + 2 * qc + (k & 1);
        const float bias = far_piece ? far[e] : bias_of<T>(a, j - pos[e], head[e]) * kLog2E;
        float x = fmaf(s[t][k], c, bias);
        // (a score of NaN or infinity plus a bias of -inf would be NaN)
        if (bias == -INFINITY || (!whole && (j >= j_hi || (a.causal && j > pos[e])))) x = -INFINITY;
        s[t][k] = x;
        top[e] = fmaxf(top[e], x);
      }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 1));
      top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 2));
    }
    const bool move[2] = {any[0] ? top[0] > m[0] : top[0] > -INFINITY, any[1] ? top[1] > m[1] : top[1] > -INFINITY};
    if (__any_sync(0xffffffffu, move[0] || move[1])) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float al = move[e] ? (any[e] ? ex2(m[e] - top[e]) : 0.f) : 1.f;
        if (move[e]) m[e] = top[e], any[e] = true;
        l[e] *= al;
#pragma unroll
        for (int x = 0; x < D / 8; ++x) o[x][2 * e] *= al, o[x][2 * e + 1] *= al;
      }
    }
    uint32_t pf[4];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float p0 = ex2(s[t][2 * e] - m[e]), p1 = ex2(s[t][2 * e + 1] - m[e]);
        l[e] += p0 + p1;
        pf[2 * t + e] = pack2<T>(p0, p1);
      }
    // lanes of matrix x: keys 8 (x % 2).., channels 8 (2 y + x / 2)..
    const int vrow = ((lane >> 3) & 1) * 8 + (lane & 7), vchunk = lane >> 4;
#pragma unroll
    for (int y = 0; y < D / 16; ++y) {
      uint32_t f[4];
      ldmatrix4_t(f, at + C::kTile + TileOf<D>::offset(kPiece, vrow, 2 * y + vchunk));
      mma16<T>(o[2 * y], pf, f[0], f[1]);
      mma16<T>(o[2 * y + 1], pf, f[2], f[3]);
    }
  }
  cp_async_wait<0>();
  // the warps' results meet in shared memory (over the rings, all reads done)
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
    l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
  }
  __syncthreads();
  float* so = reinterpret_cast<float*>(smem);          // [warp][row][D]
  float* sm = so + kWarps * kRows * D;                 // [warp][row] (m, l)
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int r = warp * kRows + gr + 8 * e;
#pragma unroll
    for (int x = 0; x < D / 8; ++x)
      *reinterpret_cast<float2*>(so + r * D + 8 * x + 2 * qc) = make_float2(o[x][2 * e], o[x][2 * e + 1]);
    if (qc == 0) {
      sm[2 * r] = any[e] || l[e] != l[e] ? m[e] : -INFINITY;  // (a row of NaN scores has no maximum)
      sm[2 * r + 1] = l[e];
    }
  }
  __syncthreads();
  constexpr int kPer = 8;  // threads per row
  const int row = threadIdx.x / kPer, part = threadIdx.x % kPer;
  const int r = r0 + row;
  if (r >= rows) return;
  const int i = r / group, h = hk * group + r % group;
  float w[kWarps], top = -INFINITY, total = 0.f;
#pragma unroll
  for (int k = 0; k < kWarps; ++k) top = fmaxf(top, sm[2 * (k * kRows + row)]);
#pragma unroll
  for (int k = 0; k < kWarps; ++k) {
    const float mk = sm[2 * (k * kRows + row)], lk = sm[2 * (k * kRows + row) + 1];
    w[k] = mk == -INFINITY ? 0.f : ex2(mk - top);
    total += mk == -INFINITY ? 0.f : w[k] * lk;
  }
  const bool some = i < sl.nq && top > -INFINITY;
  const float inv = some ? 1.f / total : 0.f;
  const long long at = ((long long)b * a.hq + h) * a.Lq + i;
  const long long out_rows = sp.rows;
  if (part == 0) {
    if (sp.n == 1)
      a.lse[at] = some ? (top + log2f(total)) * kLn2 : -INFINITY;
    else
      sp.lse[split * out_rows + at] = some ? top + log2f(total) : -INFINITY;
  }
#pragma unroll
  for (int ch = part * 4; ch < D; ch += kPer * 4) {
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (some) {
#pragma unroll
      for (int k = 0; k < kWarps; ++k) {
        if (w[k] == 0.f) continue;
        const float4 x = *reinterpret_cast<const float4*>(so + (k * kRows + row) * D + ch);
        v.x = fmaf(w[k], x.x, v.x), v.y = fmaf(w[k], x.y, v.y), v.z = fmaf(w[k], x.z, v.z), v.w = fmaf(w[k], x.w, v.w);
      }
      v.x *= inv, v.y *= inv, v.z *= inv, v.w *= inv;
    }
    if (sp.n == 1)
      *reinterpret_cast<uint2*>(static_cast<T*>(a.o.p) + a.o.at(b, i, h) + ch) =
          make_uint2(pack2<T>(v.x, v.y), pack2<T>(v.z, v.w));
    else
      *reinterpret_cast<float4*>(sp.o + (split * out_rows + at) * D + ch) = v;
  }
}

// The parts of the keys joined: a row per warp.
template <class T, int D>
__global__ void __launch_bounds__(128) attn_join_kernel(const __grid_constant__ BiasAttnArgs a, Split sp) {
  const long long rows = sp.rows;
  const long long r = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (r >= rows) return;
  after_previous();
  int i, h, b;
  if (sp.first < 0) {
    i = (int)(r % a.Lq), h = (int)(r / a.Lq % a.hq), b = (int)(r / a.Lq / a.hq);
  } else {
    const QueryTile q = query_tile(a, (unsigned)(sp.first + r / 128));
    i = q.qt * 128 + (int)(r % 128), h = q.h, b = q.b;
    if (i >= a.Lq) return;
  }
  float top = -INFINITY;
  bool nan = false;
  for (int s = lane; s < sp.n; s += 32) {
    const float lse = sp.lse[s * rows + r];
    top = fmaxf(top, lse);
    nan = nan || lse != lse;
  }
  nan = __any_sync(0xffffffffu, nan);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  float total = 0.f, v[D / 32];
#pragma unroll
  for (int k = 0; k < D / 32; ++k) v[k] = 0.f;
  if (top > -INFINITY && !nan) {
#pragma unroll 4
    for (int s = 0; s < sp.n; ++s) {  // (a part without a visible key is zeros with weight 0)
      const float w = ex2(sp.lse[s * rows + r] - top);
      total += w;
#pragma unroll
      for (int k = 0; k < D / 32; ++k) v[k] = fmaf(w, sp.o[(s * rows + r) * D + lane + 32 * k], v[k]);
    }
  }
  if (nan) total = top = __int_as_float(0x7fffffff);
  const float inv = total > 0.f || nan ? 1.f / total : 0.f;
  T* out = static_cast<T*>(a.o.p) + a.o.at(b, i, h);
#pragma unroll
  for (int k = 0; k < D / 32; ++k) out[lane + 32 * k] = from_f<T>(v[k] * inv);
  if (lane == 0) a.lse[((long long)b * a.hq + h) * a.Lq + i] = top > -INFINITY || nan ? (top + log2f(total)) * kLn2 : -INFINITY;
}

// Parts of the keys: enough CTAs for two waves of what is resident (sequences
// have unequal lengths), at least 256 keys (four pieces of every warp) in each.
void token_plan(const BiasAttnArgs& a, int* blocks, int* n) {
  *blocks = (a.Lq * (a.hq / a.hk) + kRows - 1) / kRows;
  const long long ctas = (long long)a.B * a.hk * *blocks;
  const long long want = 2LL * sm_count() * (a.d == 128 ? TokCfg<128>::CTAS : TokCfg<64>::CTAS);
  const long long parts = want / ctas, most = (a.Lk + 255) / 256;
  *n = (int)(parts < 1 ? 1 : (parts > most ? most : parts));
}

template <class T, int D>
cudaError_t token(const BiasAttnArgs& a, void* scratch, cudaStream_t st) {
  using C = TokCfg<D>;
  int blocks, n;
  token_plan(a, &blocks, &n);
  cudaError_t e = cudaFuncSetAttribute(attn_token_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  Split sp = token_split(a);
  split_place(&sp, D, scratch);
  prof_begin(kKindOther, st);
  attn_token_kernel<T, D><<<(unsigned)((long long)a.B * a.hk * blocks * n), 32 * kWarps, C::SMEM, st>>>(a, sp, blocks);
  prof_end(kKindOther, st);
  count_launch();
  e = cudaGetLastError();
  return e == cudaSuccess && n > 1 ? launch_attention_join<T, D>(a, sp, st) : e;
}

template <class T>
cudaError_t token_d(const BiasAttnArgs& a, void* scratch, cudaStream_t st) {
  if (a.d == 32) return token<T, 32>(a, scratch, st);
  if (a.d == 64) return token<T, 64>(a, scratch, st);
  return token<T, 128>(a, scratch, st);
}

}  // namespace

template <class T, int D>
cudaError_t launch_attention_join(const BiasAttnArgs& a, const Split& sp, cudaStream_t st) {
  prof_begin(kKindOther, st);
  const cudaError_t e = launch_after(attn_join_kernel<T, D>, dim3((unsigned)((sp.rows + 3) / 4)), 128, 0, st, a, sp);
  prof_end(kKindOther, st);
  count_launch();
  return e;
}
template cudaError_t launch_attention_join<__nv_bfloat16, 32>(const BiasAttnArgs&, const Split&, cudaStream_t);
template cudaError_t launch_attention_join<__nv_bfloat16, 64>(const BiasAttnArgs&, const Split&, cudaStream_t);
template cudaError_t launch_attention_join<__nv_bfloat16, 128>(const BiasAttnArgs&, const Split&, cudaStream_t);
template cudaError_t launch_attention_join<__half, 32>(const BiasAttnArgs&, const Split&, cudaStream_t);
template cudaError_t launch_attention_join<__half, 64>(const BiasAttnArgs&, const Split&, cudaStream_t);
template cudaError_t launch_attention_join<__half, 128>(const BiasAttnArgs&, const Split&, cudaStream_t);

// Up to 32 rows per key head (two blocks of 16, which share the keys in L2): beyond
// that the products take longer than the copies. Against the form by tiles, 8
// sequences of 8 key heads of 64 and 1024 keys: 4 rows 13 us (21 there), 32 rows
// 17 (21), 64 rows 26 (21); 4 sequences of 8 heads of 128 and 4096 keys: 27 (46),
// 41 (45), 58 (46).
bool token_form(const BiasAttnArgs& a) { return (long long)a.Lq * (a.hq / a.hk) <= 32; }

Split token_split(const BiasAttnArgs& a) {
  int blocks, n;
  token_plan(a, &blocks, &n);
  return Split{n, (long long)a.B * a.hq * a.Lq, -1, nullptr, nullptr};
}

cudaError_t launch_token_attention(const BiasAttnArgs& a, int dtype, void* scratch, cudaStream_t st) {
  return dtype == kBF16 ? token_d<__nv_bfloat16>(a, scratch, st) : token_d<__half>(a, scratch, st);
}

}  // namespace vswin
