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
// keys go by in tiles of BN: S = Q K^T on tcgen05 into TMEM (fp32), four
// softmax warps (TMEM lane = query row) turn it into P (16 bits, back to TMEM,
// the A operand of a TS MMA) and O += P V accumulates in TMEM. Two producer
// warps bring K and V tiles (two stages) with cp.async, which zero-fills what
// lies behind the lengths whatever it holds, and prepare each tile's bias.
//
// Bias: it depends on j - i alone, so a tile needs 127 + BN values, one line in
// shared memory that row i reads from entry 127 - i on (consecutive rows,
// consecutive banks); the causal rule is part of the line (-inf). Tiles of one
// bucket (all far ones) skip the line: one value for the whole tile.
//
// Softmax in one pass: a tile's P is formed against the row's reference m, the
// maximum as it was when it last moved. Only when a score exceeds m by more
// than kSlack (in log2) does the warp raise m, rescale O and form the tile
// again; P is at most 2^kSlack, exact in fp32 sums and finite in 16 bits, and o
// and lse do not depend on m. TMEM columns: S [0, BN), P [BN, 3 BN / 2),
// O behind.
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

template <int D>
struct FwdCfg {
  static constexpr int BN = D == 128 ? 64 : 128;
  using Line = BiasLine<127 + BN, false>;
  static constexpr int kTile = BN * D * 2;
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = 128 * D * 2;
  static constexpr int OFF_V = OFF_K + 2 * kTile;
  static constexpr int OFF_BIAS = OFF_V + 2 * kTile;
  static constexpr int OFF_BAR = OFF_BIAS + (2 * (int)sizeof(Line) + 15) / 16 * 16;
  static constexpr int SMEM = OFF_BAR + 256;
  static constexpr int kColP = BN, kColO = BN + BN / 2;
  static constexpr uint32_t kTmem = 256;
  static_assert(kColO + D <= 256, "TMEM columns of a CTA");
};

template <class T, int D>
__global__ void __launch_bounds__(kFwdThreads, 2) attn_fwd_kernel(const __grid_constant__ BiasAttnArgs a, Split sp) {
  using C = FwdCfg<D>;
  constexpr int BN = C::BN;
  using Line = typename C::Line;
  extern __shared__ __align__(1024) uint8_t smem[];
  Line* lines = reinterpret_cast<Line*>(smem + C::OFF_BIAS);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* k_full = bars;         // [2]
  uint64_t* k_free = bars + 2;     // [2]
  uint64_t* v_full = bars + 4;     // [2]
  uint64_t* v_free = bars + 6;     // [2]
  uint64_t* b_full = bars + 8;     // [2] bias line
  uint64_t* b_free = bars + 10;    // [2]
  uint64_t* s_full = bars + 12;    // scores in TMEM
  uint64_t* p_full = bars + 13;    // P written, scores read
  uint64_t* o_done = bars + 14;    // P V accumulated
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(bars + 15);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // heavy query tiles (causal: the last) first
  const long long per_tile = (long long)a.B * a.hq * sp.n;
  const int qt = (int)((gridDim.x - 1 - blockIdx.x) / per_tile);
  int rest = (int)((gridDim.x - 1 - blockIdx.x) % per_tile);
  const int split = rest % sp.n;
  rest /= sp.n;
  const int h = rest % a.hq, b = rest / a.hq, hk = h / (a.hq / a.hk);
  const SeqLens sl = seq_lens(a, b);
  const int i0 = qt * 128, pos0 = sl.start + i0;
  int nk = i0 < sl.nq ? sl.nk : 0;
  if (a.causal) nk = min(nk, max(0, sl.start + min(i0 + 128, sl.nq)));
  const int tiles = (nk + BN - 1) / BN;
  const int per = (tiles + sp.n - 1) / sp.n;
  const int t0 = min(split * per, tiles), nt = min(t0 + per, tiles) - t0;

  if (tid == 0) {
    for (int k = 0; k < 2; ++k) {
      mbar_init(&k_full[k], kProducers);
      mbar_init(&k_free[k], 1);
      mbar_init(&v_full[k], kProducers);
      mbar_init(&v_free[k], 1);
      mbar_init(&b_full[k], kProducers);
      mbar_init(&b_free[k], kSoftmaxWarps);
    }
    mbar_init(s_full, 1);
    mbar_init(p_full, kSoftmaxWarps);
    mbar_init(o_done, 1);
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
    const T* kh = static_cast<const T*>(a.k.p) + a.k.at(b, 0, hk);
    const T* vh = static_cast<const T*>(a.v.p) + a.v.at(b, 0, hk);
    const uint32_t sq = smem_u32(smem + C::OFF_Q), sk = smem_u32(smem + C::OFF_K), sv = smem_u32(smem + C::OFF_V);
    if (nt > 0)
      load_tile<T, D, 128, kProducers>(sq, static_cast<const T*>(a.q.p) + a.q.at(b, 0, h), a.q.st, i0, sl.nq, p);
    for (int t = 0; t < nt; ++t) {
      const int s = t & 1, j0 = (t0 + t) * BN;
      const uint32_t parity = ((t >> 1) & 1) ^ 1;  // the previous use of the stage
      if (t >= 2 && !warp_wait(&k_free[s], parity, a.ctx, kErrAttnLoad)) break;
      load_tile<T, D, BN, kProducers>(sk + s * C::kTile, kh, a.k.st, j0, nk, p);
      cp_async_mbar_arrive_noinc(&k_full[s]);
      if (t >= 2 && !warp_wait(&b_free[s], parity, a.ctx, kErrAttnLoad)) break;
      fill_bias_line<T, 127 + BN, false, kProducers>(&lines[s], a, h, j0 - pos0 - 127, p);
      mbar_arrive(&b_full[s]);
      if (t >= 2 && !warp_wait(&v_free[s], parity, a.ctx, kErrAttnLoad)) break;
      load_tile<T, D, BN, kProducers>(sv + s * C::kTile, vh, a.v.st, j0, nk, p);
      cp_async_mbar_arrive_noinc(&v_full[s]);
    }
    cp_async_wait_all();
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ MMA issue
    if (lane == 0) {
      const uint32_t sq = smem_u32(smem + C::OFF_Q), sk = smem_u32(smem + C::OFF_K), sv = smem_u32(smem + C::OFF_V);
      constexpr uint32_t id_s = idesc16<T>(128, BN, 0, 0), id_o = idesc16<T>(128, D, 0, 1);
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        return mbar_wait(bar, parity, a.ctx.err, kErrAttnMma, a.ctx.wait_limit);
      };
      bool ok = true;
      for (int t = 0; t <= nt && ok; ++t) {
        // scores of tile t once tile t - 1's have been read, then P V of tile t - 1
        if (t > 0) ok = wait(p_full, (t - 1) & 1);
        if (ok && t < nt) {
          ok = wait(&k_full[t & 1], (t >> 1) & 1);
          if (!ok) break;
          fence_proxy_async_smem();  // bytes written by cp.async are read by the tensor core
          tc_fence_after();
          mma_rows<D>(tmem, sq, sk + (t & 1) * C::kTile, id_s);
          umma_commit(s_full);
          umma_commit(&k_free[t & 1]);
        }
        if (ok && t > 0) {
          const int u = t - 1;
          ok = wait(&v_full[u & 1], (u >> 1) & 1);
          if (!ok) break;
          fence_proxy_async_smem();
          tc_fence_after();
          mma_acc<D, BN>(tmem + C::kColO, tmem + C::kColP, sv + (u & 1) * C::kTile, id_o, u == 0);
          umma_commit(o_done);
          umma_commit(&v_free[u & 1]);
        }
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax
    const uint32_t tw = tmem + ((uint32_t)(warp * 32) << 16);
    const int i = i0 + warp * 32 + lane;
    const float c = a.scale * kLog2E;
    float m = 0.f;             // reference of the row (log2), once l > 0
    float l = 0.f;             // sum of P
    bool ok = true;
    for (int t = 0; t < nt; ++t) {
      const int s = t & 1, j0 = (t0 + t) * BN;
      ok = warp_wait(&b_full[s], (t >> 1) & 1, a.ctx, kErrAttnSoftmax) &&
           warp_wait(s_full, t & 1, a.ctx, kErrAttnSoftmax);
      if (!ok) break;
      tc_fence_after();
      const Line& bl = lines[s];
      const bool flat = bl.same[0] && bl.same[1];
      const float value = bl.value;
      const float* line = bl.line + 127 - (warp * 32 + lane);
      const int live = nk - j0;  // columns of the tile that are keys
      // maximum of x - m over the tile, x = S c + bias; with `form`, P = 2^(x - m) into TMEM and its sum too
      float sum = 0.f;
      auto pass = [&](bool form) {
        float top = -INFINITY;
        float2 acc = make_float2(0.f, 0.f);
        for (int c0 = 0; c0 < BN; c0 += 32) {
          uint32_t u[32];
          tmem_ld32(tw + c0, u);
          tmem_wait_ld_keep(u);
          float x[32];
          const float2 c2 = make_float2(c, c);
          if (flat) {
            const float2 off = make_float2(value - m, value - m);
#pragma unroll
            for (int k = 0; k < 32; k += 2) {
              const float2 y =
                  __ffma2_rn(make_float2(__uint_as_float(u[k]), __uint_as_float(u[k + 1])), c2, off);
              x[k] = y.x;
              x[k + 1] = y.y;
            }
          } else {
            const float2 mm = make_float2(-m, -m);
#pragma unroll
            for (int k = 0; k < 32; k += 2) {
              const float2 off = __fadd2_rn(make_float2(line[c0 + k], line[c0 + k + 1]), mm);
              const float2 y =
                  __ffma2_rn(make_float2(__uint_as_float(u[k]), __uint_as_float(u[k + 1])), c2, off);
              x[k] = y.x;
              x[k + 1] = y.y;
            }
          }
          if (live < BN) {
#pragma unroll
            for (int k = 0; k < 32; ++k) x[k] = c0 + k < live ? x[k] : -INFINITY;
          }
#pragma unroll
          for (int k = 0; k < 32; ++k) top = fmaxf(top, x[k]);
          if (form) {
            uint32_t w[16];
#pragma unroll
            for (int k = 0; k < 32; k += 2) {
              const float2 p = make_float2(ex2(x[k]), ex2(x[k + 1]));
              acc = __fadd2_rn(acc, p);
              w[k / 2] = pack2<T>(p.x, p.y);
            }
            tmem_st16(tw + C::kColP + c0 / 2, w);
          }
        }
        sum = acc.x + acc.y;
        return top;
      };
      // P of the tile before has been read, and O may be touched
      float top = t == 0 ? pass(false) : -INFINITY;
      if (t > 0) {
        ok = warp_wait(o_done, (t - 1) & 1, a.ctx, kErrAttnSoftmax);
        if (!ok) break;
        tc_fence_after();
        top = pass(true);
      }
      const bool move = l == 0.f ? top > -INFINITY : top > kSlack;
      if (t == 0 || __any_sync(0xffffffffu, move)) {
        const float alpha = move ? (l == 0.f ? 0.f : ex2(-top)) : 1.f;
        if (move) m += top;
        l *= alpha;
        if (t > 0) {
#pragma unroll
          for (int c0 = 0; c0 < D; c0 += 16) {
            uint32_t u[16];
            tmem_ld16(tw + C::kColO + c0, u);
            tmem_wait_ld_keep(u);
#pragma unroll
            for (int k = 0; k < 16; ++k) u[k] = __float_as_uint(__uint_as_float(u[k]) * alpha);
            tmem_st16(tw + C::kColO + c0, u);
          }
        }
        pass(true);
      }
      l += sum;
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(p_full);
        mbar_arrive(&b_free[s]);
      }
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
// two CTAs per SM, at least four key tiles in each.
int forward_splits(const BiasAttnArgs& a) {
  const int bn = a.d == 128 ? 64 : 128;
  const long long ctas = (long long)a.B * a.hq * ((a.Lq + 127) / 128), slots = 2LL * sm_count();
  const long long tiles = (a.Lk + bn - 1) / bn;
  if (2 * ctas > slots) return 1;
  const long long parts = slots / ctas, most = tiles / 4;
  return (int)(parts < most ? parts : (most < 1 ? 1 : most));
}

template <class T, int D>
cudaError_t forward(const BiasAttnArgs& a, void* scratch, cudaStream_t st) {
  using C = FwdCfg<D>;
  static_assert(2 * (C::SMEM + 1024) <= 228 * 1024, "two CTAs per SM");
  cudaError_t e = cudaFuncSetAttribute(attn_fwd_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  const Split sp = split_of(a, forward_splits(a), scratch);
  const long long grid = (long long)a.B * a.hq * ((a.Lq + 127) / 128) * sp.n;
  prof_begin(kKindOther, st);
  attn_fwd_kernel<T, D><<<(unsigned)grid, kFwdThreads, C::SMEM, st>>>(a, sp);
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
