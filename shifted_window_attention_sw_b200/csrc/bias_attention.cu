// Attention over token sequences with a learned relative-position bias by
// buckets: for query i of sequence b at position p = q_start[b] + i and key j,
//
//   s_ij = scale q_i . k_j + table[map[clip(j - p, -D, D) + D]][h],
//   P = softmax of s over the visible keys,  o_i = sum_j P_ij v_j,
//   lse_i = log sum_j exp(s_ij).
//
// A key is visible when j < kv_lens[b], j <= p (causal) and its bias is above
// kExclude. Rows behind q_lens[b] and rows without a visible key give o = 0 and
// lse = -inf. Head h reads key head h * hk / hq.
//
// attn_fwd_kernel: one CTA per 128 query rows of a head, two CTAs per SM. The
// keys go by in tiles of 64: S = Q K^T on tcgen05 into one of two TMEM buffers
// (fp32), four softmax warps (TMEM lane = query row) turn it into P (16 bits,
// written over the scores, the A operand of a TS MMA) and O += P V accumulates
// in TMEM. While the warps work on one tile, P V of the tile before and the
// scores of the next run. Two producer warps bring K and V tiles (two or three
// stages, TMA) and prepare each tile's bias; a tile in which the keys end goes
// by cp.async instead, so that nothing behind the lengths is read.
//
// Bias: it depends on j - i alone, so a tile needs 127 + BN values, one line in
// shared memory that row i reads from entry 127 - i on (consecutive rows,
// consecutive banks); the causal rule is part of the line (-inf). Tiles of one
// bucket (all far ones) skip the line: one value for the whole tile.
//
// Softmax in one pass: a tile's P is formed against the row's reference m, the
// maximum as it was when it last moved, so that its exponentials do not wait
// for its maximum. Only when a score exceeds m by more than kSlack (in log2)
// does the warp raise m, form P again and rescale O; P is at most 2^kSlack, exact in fp32 sums and finite in 16 bits, and o and lse do not
// depend on m. TMEM columns: scores [0, 64) and [64, 128), O behind.
//
// Bound: one exponential per visible pair (16 per clock and SM) for D = 32 and
// 64, the tensor cores for D = 128.
#include "bias_attention.cuh"
#include "bias_attention_split.h"

namespace vswin {
namespace {

constexpr int kSoftmaxWarps = 4, kProducerWarps = 2;
constexpr int kMmaWarp = 4;
constexpr int kFwdThreads = 32 * (kSoftmaxWarps + 1 + kProducerWarps);
constexpr int kProducers = 32 * kProducerWarps;
constexpr float kSlack = 8.f;

constexpr int kBn = 64;           // keys per tile
constexpr int kLineN = 127 + kBn;  // offsets in a tile


template <int D>
struct FwdCfg {
  static constexpr int ST = D == 128 ? 2 : 3;  // stages: two CTAs share 227 KB
  using Line = BiasLine<kLineN, false>;
  static constexpr int kTile = kBn * D * 2;
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = 128 * D * 2;
  static constexpr int OFF_V = OFF_K + ST * kTile;
  static constexpr int OFF_BIAS = OFF_V + ST * kTile;
  static constexpr int OFF_BAR = OFF_BIAS + (ST * (int)sizeof(Line) + 15) / 16 * 16;
  static constexpr int SMEM = OFF_BAR + 256;
  static constexpr int kColO = 2 * kBn;
  static constexpr uint32_t kTmem = 256;
  static_assert(kColO + D <= 256, "TMEM columns of a CTA");
};

struct FwdParams {
  HeadMap q, k, v;
  BiasAttnArgs a;
};

template <class T, int D>
__global__ void __launch_bounds__(kFwdThreads, 2) attn_fwd_kernel(const __grid_constant__ FwdParams params, Split sp) {
  const BiasAttnArgs& a = params.a;
  using C = FwdCfg<D>;
  using Line = typename C::Line;
  constexpr int ST = C::ST;
  extern __shared__ __align__(1024) uint8_t smem[];
  Line* lines = reinterpret_cast<Line*>(smem + C::OFF_BIAS);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* k_full = bars;            // [ST]
  uint64_t* k_free = bars + ST;       // [ST]
  uint64_t* v_full = bars + 2 * ST;   // [ST]
  uint64_t* v_free = bars + 3 * ST;   // [ST]
  uint64_t* s_full = bars + 4 * ST;   // [ST] bias line written and scores in TMEM
  uint64_t* p_full = bars + 5 * ST;   // [2] P written over them
  uint64_t* o_done = p_full + 2;      // P V accumulated
  uint64_t* q_full = p_full + 3;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(p_full + 4);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // heavy query tiles (causal: the last) first
  const unsigned per_tile = (unsigned)a.B * a.hq * sp.n;
  const unsigned id = gridDim.x - 1 - blockIdx.x;
  const int qt = (int)(id / per_tile);
  unsigned rest = id % per_tile;
  const int split = (int)(rest % sp.n);
  rest /= sp.n;
  const int h = (int)(rest % a.hq), b = (int)(rest / a.hq), hk = h / (a.hq / a.hk);
  const SeqLens sl = seq_lens(a, b);
  const int i0 = qt * 128, pos0 = sl.start + i0;
  int nk = i0 < sl.nq ? sl.nk : 0;
  if (a.causal) nk = min(nk, max(0, sl.start + min(i0 + 128, sl.nq)));
  const int tiles = (nk + kBn - 1) / kBn;
  const int per = (tiles + sp.n - 1) / sp.n;
  const int t0 = min(split * per, tiles), nt = min(t0 + per, tiles) - t0;

  if (tid == 0) {
    for (int k = 0; k < ST; ++k) {
      mbar_init(&k_full[k], kProducerWarps);
      mbar_init(&k_free[k], 1);
      mbar_init(&v_full[k], kProducerWarps);
      mbar_init(&v_free[k], 1);
      mbar_init(&s_full[k], kProducerWarps + 1);
    }
    for (int k = 0; k < 2; ++k) mbar_init(&p_full[k], kSoftmaxWarps);
    mbar_init(o_done, 1);
    mbar_init(q_full, kProducerWarps);
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(s_tmem, C::kTmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;

  if (warp > kMmaWarp) {
    // ------------------------------------------------------------ producers
    const int p = tid - 32 * (kMmaWarp + 1);
    const uint32_t sq = smem_u32(smem + C::OFF_Q), sk = smem_u32(smem + C::OFF_K), sv = smem_u32(smem + C::OFF_V);
    if (nt > 0) bring_tile<T, D, 128>(sq, params.q, a.q, b, h, i0, sl.nq, a.Lq, q_full, p);
    int s = 0;
    uint32_t parity = 1;  // of the stage's previous use
    for (int t = 0; t < nt; ++t) {
      const int j0 = (t0 + t) * kBn;
      if (t >= ST && !warp_wait(&k_free[s], parity, a.ctx, kErrAttnLoad)) break;
      bring_tile<T, D, kBn>(sk + s * C::kTile, params.k, a.k, b, hk, j0, sl.nk, a.Lk, &k_full[s], p);
      if (t >= ST && !warp_wait(&v_free[s], parity, a.ctx, kErrAttnLoad)) break;
      bring_tile<T, D, kBn>(sv + s * C::kTile, params.v, a.v, b, hk, j0, sl.nk, a.Lk, &v_full[s], p);
      fill_bias_line<T, kLineN, false, kProducers>(&lines[s], a, h, j0 - pos0 - 127, p);
      if (lane == 0) mbar_arrive(&s_full[s]);  // (the line was free when V was)
      if (++s == ST) s = 0, parity ^= 1;
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ MMA issue
    // (the whole warp waits, one elected lane issues)
    const uint32_t sq = smem_u32(smem + C::OFF_Q), sk = smem_u32(smem + C::OFF_K), sv = smem_u32(smem + C::OFF_V);
    constexpr uint32_t id_s = idesc16<T>(128, kBn, 0, 0), id_o = idesc16<T>(128, D, 0, 1);
    int ks = 0, vs = 0;
    uint32_t kp = 0, vp = 0;
    auto scores = [&](int t) {
      if (!warp_wait(&k_full[ks], kp, a.ctx, kErrAttnMma)) return false;
      tc_fence_after();
      if (elect_one()) {
        mma_rows<D, kBn>(tmem + kBn * (t & 1), sq, sk + ks * C::kTile, id_s);
        umma_commit(&s_full[ks]);
        umma_commit(&k_free[ks]);
      }
      __syncwarp();
      if (++ks == ST) ks = 0, kp ^= 1;
      return true;
    };
    bool ok = nt > 0 && warp_wait(q_full, 0, a.ctx, kErrAttnMma);
    for (int t = 0; t < 2 && t < nt && ok; ++t) ok = scores(t);
    for (int t = 0; t < nt && ok; ++t) {
      ok = warp_wait(&v_full[vs], vp, a.ctx, kErrAttnMma) && warp_wait(&p_full[t & 1], (t >> 1) & 1, a.ctx, kErrAttnMma);
      if (!ok) break;
      tc_fence_after();
      if (elect_one()) {
        mma_acc<D, kBn>(tmem + C::kColO, tmem + kBn * (t & 1), sv + vs * C::kTile, id_o, t == 0);
        umma_commit(o_done);
        umma_commit(&v_free[vs]);
      }
      __syncwarp();
      if (++vs == ST) vs = 0, vp ^= 1;
      if (t + 2 < nt) ok = scores(t + 2);  // runs after P V, which reads these columns
    }
  } else {
    // ------------------------------------------------------------ softmax
    const uint32_t tw = tmem + ((uint32_t)(warp * 32) << 16);
    const int i = i0 + warp * 32 + lane;
    const float c = a.scale * kLog2E;
    const float2 c2 = make_float2(c, c);
    float m = 0.f;  // reference of the row (log2), once l > 0
    float l = 0.f;  // sum of P
    bool ok = true;
    int s = 0;
    uint32_t parity = 0;
    for (int t = 0; t < nt; ++t) {
      ok = warp_wait(&s_full[s], parity, a.ctx, kErrAttnSoftmax);
      if (!ok) break;
      tc_fence_after();
      const uint32_t buf = tw + kBn * (t & 1);
      uint32_t u[kBn];
      tmem_ld32(buf, u);
      tmem_ld32(buf + 32, u + 32);
      const Line& bl = lines[s];
      const bool flat = bl.same[0] && bl.same[1];
      const float value = bl.value;
      const float* line = bl.line + 127 - (warp * 32 + lane);
      const int live = nk - (t0 + t) * kBn;  // columns of the tile that are keys
      tmem_wait_ld_keep(u);
      float x[kBn];  // S c + bias - m
      if (flat) {
        const float2 off = make_float2(value - m, value - m);
#pragma unroll
        for (int k = 0; k < kBn; k += 2) {
          const float2 y = __ffma2_rn(make_float2(__uint_as_float(u[k]), __uint_as_float(u[k + 1])), c2, off);
          x[k] = y.x;
          x[k + 1] = y.y;
        }
      } else {
        const float2 mm = make_float2(-m, -m);
#pragma unroll
        for (int k = 0; k < kBn; k += 2) {
          const float2 off = __fadd2_rn(make_float2(line[k], line[k + 1]), mm);
          const float2 y = __ffma2_rn(make_float2(__uint_as_float(u[k]), __uint_as_float(u[k + 1])), c2, off);
          x[k] = y.x;
          x[k + 1] = y.y;
        }
      }
      if (live < kBn) {
#pragma unroll
        for (int k = 0; k < kBn; ++k) x[k] = k < live ? x[k] : -INFINITY;
      }
      // P against the reference as it stands, while the maximum is found beside it
      uint32_t w[kBn / 2];
      float2 acc;
      auto form = [&]() {
        acc = make_float2(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < kBn; k += 2) {
          const float2 p = make_float2(ex2(x[k]), ex2(x[k + 1]));
          acc = __fadd2_rn(acc, p);
          w[k / 2] = pack2<T>(p.x, p.y);
        }
      };
      form();
      float tops[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
      for (int k = 4; k < kBn; k += 8) {
#pragma unroll
        for (int e = 0; e < 4; ++e) tops[e] = k + 4 + e < kBn ? max3(tops[e], x[k + e], x[k + 4 + e]) : fmaxf(tops[e], x[k + e]);
      }
      const float top = fmaxf(max3(tops[0], tops[1], tops[2]), tops[3]);
      const bool move = l == 0.f ? top > -INFINITY : top > kSlack;
      if (__any_sync(0xffffffffu, move)) {
        const float alpha = move ? (l == 0.f ? 0.f : ex2(-top)) : 1.f;
        const float shift = move ? top : 0.f;
        m += shift;
        l *= alpha;
#pragma unroll
        for (int k = 0; k < kBn; ++k) x[k] -= shift;
        form();
        if (t > 0) {
          ok = warp_wait(o_done, (t - 1) & 1, a.ctx, kErrAttnSoftmax);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int c0 = 0; c0 < D; c0 += 16) {
            uint32_t r[16];
            tmem_ld16(tw + C::kColO + c0, r);
            tmem_wait_ld_keep(r);
#pragma unroll
            for (int k = 0; k < 16; ++k) r[k] = __float_as_uint(__uint_as_float(r[k]) * alpha);
            tmem_st16(tw + C::kColO + c0, r);
          }
        }
      }
      tmem_st16(buf, w);
      tmem_st16(buf + 16, w + 16);
      l += acc.x + acc.y;
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[t & 1]);
      if (++s == ST) s = 0, parity ^= 1;
    }
    if (ok && nt > 0) ok = warp_wait(o_done, (nt - 1) & 1, a.ctx, kErrAttnSoftmax);
    tc_fence_after();
    if (ok) {
      const bool row = i < a.Lq;
      const bool some = i < sl.nq && (l > 0.f || l != l);
      const float inv = some ? 1.f / l : 0.f;
      const long long r = ((long long)b * a.hq + h) * a.Lq + i;
      if (row) {
        if (sp.n == 1)
          a.lse[r] = some ? (m + log2f(l)) * kLn2 : -INFINITY;
        else
          sp.lse[(long long)split * a.B * a.hq * a.Lq + r] = some ? m + log2f(l) : -INFINITY;
      }
      T* out = static_cast<T*>(a.o.p) + (row ? a.o.at(b, i, h) : 0);
      float* part = sp.o + ((long long)split * a.B * a.hq * a.Lq + (row ? r : 0)) * D;
#pragma unroll
      for (int c0 = 0; c0 < D; c0 += 16) {
        uint32_t u[16];
        if (nt > 0) {
          tmem_ld16(tw + C::kColO + c0, u);
          tmem_wait_ld_keep(u);
        }
        float f[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) f[k] = some ? __uint_as_float(u[k]) * inv : 0.f;
        if (row && sp.n == 1) {
#pragma unroll
          for (int k = 0; k < 16; k += 8)
            *reinterpret_cast<uint4*>(out + c0 + k) =
                make_uint4(pack2<T>(f[k], f[k + 1]), pack2<T>(f[k + 2], f[k + 3]), pack2<T>(f[k + 4], f[k + 5]),
                           pack2<T>(f[k + 6], f[k + 7]));
        } else if (row) {
#pragma unroll
          for (int k = 0; k < 16; k += 4)
            *reinterpret_cast<float4*>(part + c0 + k) = make_float4(f[k], f[k + 1], f[k + 2], f[k + 3]);
        }
      }
    }
    tc_fence_before();
  }
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmem);
  }
}

// Parts of the keys when the query tiles alone leave SMs idle: as many as fill
// two CTAs per SM, at least eight key tiles in each.
int forward_splits(const BiasAttnArgs& a) {
  const long long ctas = (long long)a.B * a.hq * ((a.Lq + 127) / 128), slots = 2LL * sm_count();
  const long long tiles = (a.Lk + kBn - 1) / kBn;
  if (2 * ctas > slots) return 1;
  const long long parts = slots / ctas, most = tiles / 8;
  return (int)(parts < most ? parts : (most < 1 ? 1 : most));
}

template <class T, int D>
cudaError_t forward(const BiasAttnArgs& a, void* scratch, cudaStream_t st) {
  using C = FwdCfg<D>;
  static_assert(2 * (C::SMEM + 1024) <= 228 * 1024, "two CTAs per SM");
  cudaError_t e = cudaFuncSetAttribute(attn_fwd_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  const Split sp = split_of(a, forward_splits(a), scratch);
  const int dtype = std::is_same<T, __half>::value ? kFP16 : kBF16;
  FwdParams params;
  params.a = a;
  make_head_map(&params.q, a.q, a.B, a.Lq, a.hq, D, dtype, 128);
  make_head_map(&params.k, a.k, a.B, a.Lk, a.hk, D, dtype, kBn);
  make_head_map(&params.v, a.v, a.B, a.Lk, a.hk, D, dtype, kBn);
  const long long grid = (long long)a.B * a.hq * ((a.Lq + 127) / 128) * sp.n;
  prof_begin(kKindOther, st);
  attn_fwd_kernel<T, D><<<(unsigned)grid, kFwdThreads, C::SMEM, st>>>(params, sp);
  prof_end(kKindOther, st);
  count_launch();
  e = cudaGetLastError();
  return e == cudaSuccess && sp.n > 1 ? launch_attention_join<T, D>(a, sp, st) : e;
}

template <class T>
cudaError_t forward_d(const BiasAttnArgs& a, void* scratch, cudaStream_t st) {
  if (a.d == 32) return forward<T, 32>(a, scratch, st);
  if (a.d == 64) return forward<T, 64>(a, scratch, st);
  return forward<T, 128>(a, scratch, st);
}

}  // namespace

size_t bias_attention_scratch_bytes(const BiasAttnArgs& a) {
  return split_bytes(a, token_form(a) ? token_splits(a) : forward_splits(a));
}
cudaError_t launch_bias_attention(const BiasAttnArgs& a, int dtype, void* scratch, cudaStream_t st) {
  if (token_form(a)) return launch_token_attention(a, dtype, scratch, st);
  return dtype == kBF16 ? forward_d<__nv_bfloat16>(a, scratch, st) : forward_d<__half>(a, scratch, st);
}

}  // namespace vswin
