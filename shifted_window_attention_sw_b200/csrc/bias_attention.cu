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
// keys go by in tiles: S = Q K^T on tcgen05 into TMEM (fp32), four softmax warps
// (TMEM lane = query row) turn it into P (16 bits, written over the scores, the
// A operand of a TS MMA) and O += P V accumulates in TMEM. Tiles have 64 keys and
// two or three score buffers, so that the next scores are there when a tile's P
// is done. D = 32 and 64: two groups of four warps take the tiles in turns, each
// with its own softmax statistics and sums, joined at the end (sixteen softmax
// warps per SM), half a tile in registers at a time. D = 128: TMEM has room for
// one group's sums (two CTAs of 256 columns); it takes a whole tile at a time (8192
// causal tokens, 16 heads over 4, short runs: 263 us; half tiles 300; tiles of 128
// keys with one score buffer 276; eight warps that share a tile's columns 279). One
// warp brings K and V tiles
// (TMA; a tile in which the keys end goes by cp.async instead, so that nothing
// behind the lengths is read), one prepares each tile's bias.
//
// Bias: it depends on j - i alone, so a tile needs 127 + BN values, one line in
// shared memory that row i reads from entry 127 - i on (consecutive rows,
// consecutive banks); the causal rule is part of the line (-inf). Tiles of one
// bucket (all far ones) skip the line: one value for the whole tile.
//
// Softmax in one pass over the keys: P is formed against the row's reference m,
// the maximum as it was when it last moved. Only when a score exceeds m by more
// than kSlack (in log2) does the warp raise m, by a whole number, and rescale what
// it has by that power of two (without rounding); o and lse do not depend on m.
// P is rounded to the tensors' 16 bits once, as the MMA's operand (at most
// 2^kSlack, so finite in either type; half a step per key, or 2^-25 in fp16 where
// that is more), while l sums it unrounded in fp32. TMEM columns: scores first, O behind.
//
// Bound: for D = 32 and 64 one exponential per visible pair (16 per clock and
// SM), for D = 128 the tensor cores; in front of both stands the chain of a
// softmax warp (wait, TMEM load, maximum, exponentials, store, hand-over: ~1.9 K
// cycles per 64 keys at D = 128). Measured: 3136 tokens of 4 clips, 12 heads of
// 32, 171 us of 105 for the exponentials alone; 4096 causal tokens, 24 heads of
// 64, 92 us (560 TFLOP/s); 8192 causal, 16 heads of 128, 263 us in a short run (1.05
// PFLOP/s, 0.62 of the measured burst peak) and 301-312 us a call in a long one, under
// the power cap. Without any exponential they take 0.82-0.87 of that.
#include "bias_attention.cuh"
#include "bias_attention_split.h"

namespace vswin {
namespace {

constexpr int kProducerWarps = 2;
constexpr int kRing = 4;         // bias lines, and the barriers of scores and P
constexpr float kSlack = 8.f;

template <int D>
struct FwdCfg {
  static constexpr int G = D == 128 ? 1 : 2;     // groups of four softmax warps, each with its own sums O
  static constexpr int BN = 64;                   // keys per tile
  static constexpr int NBUF = D == 32 ? 3 : 2;    // score buffers: what TMEM holds
  static constexpr int ST = D == 128 ? 2 : 3;     // stages of K and V: two CTAs share 227 KB
  static constexpr int kMmaWarp = 4 * G;
  static constexpr int THREADS = 32 * (4 * G + 1 + kProducerWarps);
  static constexpr int kLineN = 127 + BN;         // offsets in a tile
  using Line = BiasLine<kLineN, false>;           // kRing stages
  static constexpr int kTile = BN * D * 2;
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = 128 * D * 2;
  static constexpr int OFF_V = OFF_K + ST * kTile;
  static constexpr int OFF_BIAS = OFF_V + ST * kTile;
  static constexpr int OFF_BAR = OFF_BIAS + (kRing * (int)sizeof(Line) + 15) / 16 * 16;
  static constexpr int OFF_ML = OFF_BAR + 256;  // [G][128] (m, l) of the groups' rows
  static constexpr int SMEM = OFF_ML + (G == 2 ? 2 * 128 * 8 : 0);
  static constexpr int kColO = NBUF * BN;
  static constexpr uint32_t kTmem = 256;
  static_assert(kColO + G * D <= 256, "TMEM columns of a CTA");
};

struct FwdParams {
  HeadMap q, k, v;
  BiasAttnArgs a;
};

template <class T, int D>
__global__ void __launch_bounds__(FwdCfg<D>::THREADS, 2) attn_fwd_kernel(const __grid_constant__ FwdParams params, Split sp) {
  const BiasAttnArgs& a = params.a;
  using C = FwdCfg<D>;
  using Line = typename C::Line;
  constexpr int ST = C::ST, G = C::G, NBUF = C::NBUF, kBn = C::BN, kMmaWarp = C::kMmaWarp;
  extern __shared__ __align__(1024) uint8_t smem[];
  Line* lines = reinterpret_cast<Line*>(smem + C::OFF_BIAS);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* k_full = bars;            // [ST] K tile
  uint64_t* s_full = bars + ST;       // [kRing] bias line written and scores in TMEM (K has been read)
  uint64_t* p_full = s_full + kRing;  // [kRing] V tile, and P written over the scores (line and scores have been read)
  uint64_t* o_done = p_full + kRing;  // [kRing] P V accumulated (V has been read)
  uint64_t* q_full = o_done + kRing;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(q_full + 1);
  uint32_t* gave_up = s_tmem + 1;  // a wait ran out
  float2* ml = reinterpret_cast<float2*>(smem + C::OFF_ML);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // the tiles before sp.first whole, then those from there on in sp.n parts of the keys
  const unsigned whole = sp.n > 1 ? (unsigned)sp.first : gridDim.x;
  const unsigned extra = blockIdx.x < whole ? 0 : blockIdx.x - whole;
  const bool is_split = blockIdx.x >= whole;
  const int split = (int)(extra % sp.n), parts = is_split ? sp.n : 1;
  const unsigned id = is_split ? whole + extra / sp.n : blockIdx.x;
  const QueryTile q = query_tile(a, id);
  const int h = q.h, b = q.b, hk = h / (a.hq / a.hk);
  const SeqLens sl = seq_lens(a, b);
  const int i0 = q.qt * 128, pos0 = sl.start + i0;
  int nk = i0 < sl.nq ? sl.nk : 0;
  if (a.causal) nk = min(nk, max(0, sl.start + min(i0 + 128, sl.nq)));
  const int tiles = (nk + kBn - 1) / kBn;
  const int per = (tiles + parts - 1) / parts;
  const int t0 = min(split * per, tiles), nt = min(t0 + per, tiles) - t0;

  if (tid == 0) {
    for (int k = 0; k < ST; ++k) mbar_init(&k_full[k], 1);
    for (int k = 0; k < kRing; ++k) {
      mbar_init(&s_full[k], 2);
      mbar_init(&p_full[k], 5);
      mbar_init(&o_done[k], 1);
    }
    mbar_init(q_full, 1);
    *gave_up = 0;
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
  if (sp.n > 1) let_next_start();

  if (warp > kMmaWarp) {
    // ------------------------------------------------------------ producers: tiles, bias lines
    const uint32_t sq = smem_u32(smem + C::OFF_Q), sk = smem_u32(smem + C::OFF_K), sv = smem_u32(smem + C::OFF_V);
    if (warp == kMmaWarp + 1) {
      if (nt > 0) bring_tile<T, D, 128>(sq, params.q, a.q, b, h, i0, sl.nq, a.Lq, q_full);
      // K runs a tile ahead of V: its stage is free a tile earlier
      auto wait_tile = [&](uint64_t* done, int t) {
        return t < 0 || warp_wait(&done[t % kRing], (t / kRing) & 1, a.ctx, kErrAttnLoad, gave_up);
      };
      for (int t = 0; t <= nt; ++t) {
        if (t < nt) {
          if (!wait_tile(s_full, t - ST)) break;
          bring_tile<T, D, kBn>(sk + t % ST * C::kTile, params.k, a.k, b, hk, (t0 + t) * kBn, sl.nk, a.Lk, &k_full[t % ST]);
        }
        if (t > 0) {
          const int u = t - 1;
          if (!wait_tile(o_done, u - ST)) break;
          bring_tile<T, D, kBn>(sv + u % ST * C::kTile, params.v, a.v, b, hk, (t0 + u) * kBn, sl.nk, a.Lk, &p_full[u % kRing]);
        }
      }
    } else if (nt > 0) {
      const LineWriter<T, C::kLineN, false> writer(a, h);
      for (int t = 0; t < nt; ++t) {
        if (t >= kRing && !warp_wait(&p_full[t % kRing], (t / kRing - 1) & 1, a.ctx, kErrAttnLoad, gave_up)) break;
        writer.write(&lines[t % kRing], (t0 + t) * kBn - pos0 - 127);
        if (lane == 0) mbar_arrive(&s_full[t % kRing]);
      }
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ MMA issue
    // (the whole warp waits, one elected lane issues)
    const uint32_t sq = smem_u32(smem + C::OFF_Q), sk = smem_u32(smem + C::OFF_K), sv = smem_u32(smem + C::OFF_V);
    constexpr uint32_t id_s = idesc16<T>(128, kBn, 0, 0), id_o = idesc16<T>(128, D, 0, 1);
    auto scores = [&](int t) {  // by the elected lane
      mma_rows<D, kBn>(tmem + kBn * (t % NBUF), sq, sk + t % ST * C::kTile, id_s);
      umma_commit(&s_full[t % kRing]);
    };
    auto wait_k = [&](int t) { return warp_wait(&k_full[t % ST], (t / ST) & 1, a.ctx, kErrAttnMma, gave_up); };
    bool ok = nt > 0 && warp_wait(q_full, 0, a.ctx, kErrAttnMma, gave_up);
    for (int t = 0; t < NBUF && t < nt && ok; ++t) {
      ok = wait_k(t);
      if (!ok) break;
      tc_fence_after();
      if (elect_one()) scores(t);
      __syncwarp();
    }
    for (int t = 0; t < nt && ok; ++t) {
      const int u = t + NBUF;  // the tile whose scores take this one's buffer
      ok = warp_wait(&p_full[t % kRing], (t / kRing) & 1, a.ctx, kErrAttnMma, gave_up);
      if (!ok) break;
      // the scores that follow go out at once when their keys are there
      const bool now = u < nt && __all_sync(0xffffffffu, mbar_test(&k_full[u % ST], (u / ST) & 1));
      tc_fence_after();
      if (elect_one()) {
        mma_acc<D, kBn>(tmem + C::kColO + (G == 2 ? (t & 1) * D : 0), tmem + kBn * (t % NBUF), sv + t % ST * C::kTile, id_o,
                        t < G);
        umma_commit(&o_done[t % kRing]);
        if (now) scores(u);  // runs after P V, which reads these columns
      }
      __syncwarp();
      if (u < nt && !now) {
        ok = wait_k(u);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) scores(u);
        __syncwarp();
      }
    }
  } else {
    // ------------------------------------------------------------ softmax
    const int g = warp >> 2, row = (warp & 3) * 32 + lane, i = i0 + row;
    const uint32_t tw = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t to = tw + C::kColO + g * D;
    const float c = a.scale * kLog2E;
    const float2 c2 = make_float2(c, c);
    float m = 0.f;  // reference of the row (log2), once l > 0
    float l = 0.f;  // sum of P
    constexpr int kPart = G == 1 ? kBn : kBn / 2;  // columns in registers at a time (120 or 80 registers)
    bool ok = true;
    for (int t = g; t < nt; t += G) {
      ok = warp_wait(&s_full[t % kRing], (t / kRing) & 1, a.ctx, kErrAttnSoftmax, gave_up);
      if (!ok) break;
      tc_fence_after();
      const uint32_t buf = tw + kBn * (t % NBUF);
      const Line& bl = lines[t % kRing];
      const bool flat = bl.flat != 0;
      const float value = bl.value;
      const float* line = bl.line + 127 - row;
      const int live = nk - (t0 + t) * kBn;  // columns of the tile that are keys
      // one part of the tile: of one bucket or not, with keys missing or not; kRedo when a score is NaN, then again
      // with `careful`, where NaN or infinity in a key that the bias or the causal rule takes out does not count
      enum { kDone, kRedo, kWait };
      // the group's sums so far are complete: these scores came after them if they took the buffer of its last tile;
      // else a part that has to rescale them says kWait and goes again
      bool settled = NBUF == G || t < G;
      auto part = [&](auto second_, auto flat_, auto cut_, auto careful_) -> int {
        constexpr int c0 = decltype(second_)::value ? kPart : 0;
        constexpr bool kFlat = decltype(flat_)::value, kCut = decltype(cut_)::value, kCareful = decltype(careful_)::value;
        uint32_t u[kPart];
#pragma unroll
        for (int e = 0; e < kPart; e += 32) tmem_ld32(buf + c0 + e, u + e);
        tmem_wait_ld_keep(u);
        float x[kPart];  // S c + bias - m
        const float off = kFlat ? value - m : -m;
#pragma unroll
        for (int k = 0; k < kPart; k += 2) {
          float2 y = make_float2(off, off);
          float2 bias;
          if (!kFlat) {
            bias = kCareful && flat ? make_float2(value, value) : make_float2(line[c0 + k], line[c0 + k + 1]);
            y = __fadd2_rn(bias, y);
          }
          y = __ffma2_rn(make_float2(__uint_as_float(u[k]), __uint_as_float(u[k + 1])), c2, y);
          x[k] = !kCut || c0 + k < live ? y.x : -INFINITY;
          x[k + 1] = !kCut || c0 + k + 1 < live ? y.y : -INFINITY;
          if (kCareful && bias.x == -INFINITY) x[k] = -INFINITY;
          if (kCareful && bias.y == -INFINITY) x[k + 1] = -INFINITY;
        }
        auto largest = [&](auto max_of) {
          float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int k = 0; k < kPart; k += 2) tops[k / 2 % 4] = max_of(tops[k / 2 % 4], x[k], x[k + 1]);
          return max_of(max_of(tops[0], tops[1], tops[2]), tops[3], tops[3]);
        };
        const float top = kCareful ? largest(max3) : largest(max3_nan);
        // (unordered comparisons: a NaN enters, too)
        if (__any_sync(0xffffffffu, l == 0.f ? top != -INFINITY : !(top <= kSlack))) {
          if (!kCareful && __any_sync(0xffffffffu, top != top)) return kRedo;
          if (!settled) return kWait;
          const bool move = l == 0.f ? top > -INFINITY : top > kSlack;
          // by whole powers of two, so that what is there already is rescaled without rounding
          const float step = move ? ceilf(top) : 0.f;
          const float alpha = step < 127.f ? __int_as_float((127 - max((int)step, 0)) << 23) : 0.f;
          m += step;
          l *= alpha;
#pragma unroll
          for (int k = 0; k < kPart; ++k) x[k] -= step;
          if (c0) {
            const uint32_t a2 = pack2<T>(alpha, alpha);
            tmem_wait_st();
#pragma unroll
            for (int e = 0; e < c0 / 2; e += 8) {
              uint32_t r[8];
              tmem_ld8(buf + e, r);
              tmem_wait_ld_keep(r);
#pragma unroll
              for (int k = 0; k < 8; ++k) r[k] = mul2<T>(r[k], a2);
              tmem_st8(buf + e, r);
            }
          }
          if (t >= G) {  // the sums so far
            tc_fence_after();
#pragma unroll
            for (int e = 0; e < D; e += 8) {
              uint32_t r[8];
              tmem_ld8(to + e, r);
              tmem_wait_ld_keep(r);
#pragma unroll
              for (int k = 0; k < 8; ++k) r[k] = __float_as_uint(__uint_as_float(r[k]) * alpha);
              tmem_st8(to + e, r);
            }
          }
        }
        float2 acc = make_float2(0.f, 0.f);
#pragma unroll
        for (int e = 0; e < kPart; e += 16) {
          uint32_t v[8];
#pragma unroll
          for (int k = 0; k < 16; k += 2) {
            const float2 p = make_float2(ex2(x[e + k]), ex2(x[e + k + 1]));
            acc = __fadd2_rn(acc, p);
            v[k / 2] = pack2<T>(p.x, p.y);
          }
          tmem_st8(buf + (c0 + e) / 2, v);  // over scores that have been read
        }
        l += acc.x + acc.y;
        return kDone;
      };
      using Yes = std::true_type;
      using No = std::false_type;
      auto whole = [&](auto second_, auto flat_, auto cut_) {
        int r;
        while ((r = part(second_, flat_, cut_, No{})) == kWait) {
          settled = warp_wait(&o_done[(t - G) % kRing], ((t - G) / kRing) & 1, a.ctx, kErrAttnSoftmax, gave_up);
          if (!settled) return false;
        }
        if (r == kRedo) {
          if (!settled && !warp_wait(&o_done[(t - G) % kRing], ((t - G) / kRing) & 1, a.ctx, kErrAttnSoftmax, gave_up))
            return false;
          settled = true;
          part(second_, No{}, Yes{}, Yes{});
        }
        return true;
      };
      auto tile = [&](auto flat_, auto cut_) {
        return whole(No{}, flat_, cut_) && (kPart == kBn || whole(Yes{}, flat_, cut_));
      };
      if (live >= kBn)
        ok = flat ? tile(Yes{}, No{}) : tile(No{}, No{});
      else
        ok = flat ? tile(Yes{}, Yes{}) : tile(No{}, Yes{});
      if (!ok) break;
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[t % kRing]);
    }
    const int last = nt - 1 - (G == 2 ? (nt - 1 - g) & 1 : 0);  // the group's last tile
    if (ok && last >= 0) ok = warp_wait(&o_done[last % kRing], (last / kRing) & 1, a.ctx, kErrAttnSoftmax, gave_up);
    tc_fence_after();
    // the groups' sums over their tiles of the row, weighed against the larger reference; a group without any has weight 0
    float weight[2] = {1.f, 0.f};
    if (G == 2) {
      ml[g * 128 + row] = make_float2(m, l);
      tc_fence_before();
      asm volatile("bar.sync 1, 256;" ::: "memory");
      tc_fence_after();
      const float2 x = ml[row], y = ml[128 + row];
      m = y.y == 0.f ? x.x : (x.y == 0.f ? y.x : fmaxf(x.x, y.x));
      weight[0] = x.y == 0.f ? 0.f : ex2(x.x - m);
      weight[1] = y.y == 0.f ? 0.f : ex2(y.x - m);
      l = (x.y == 0.f ? 0.f : x.y * weight[0]) + (y.y == 0.f ? 0.f : y.y * weight[1]);
    }
    if (ok) {
      const bool in = i < a.Lq;
      const bool some = i < sl.nq && (l > 0.f || l != l);
      const float inv = some ? 1.f / l : 0.f;
      const long long r = ((long long)b * a.hq + h) * a.Lq + i;
      const long long pr = split * sp.rows + (is_split ? (long long)(id - sp.first) * 128 + row : 0);
      if (in && g == 0) {
        if (!is_split)
          a.lse[r] = some ? (m + log2f(l)) * kLn2 : -INFINITY;
        else
          sp.lse[pr] = some ? m + log2f(l) : -INFINITY;
      }
      T* out = static_cast<T*>(a.o.p) + (in ? a.o.at(b, i, h) : 0);
      float* part = sp.o + pr * D;
      // each group writes its part of the channels
#pragma unroll
      for (int c0 = 0; c0 < D / G; c0 += 16) {
        const int ch = g * (D / G) + c0;
        float f[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) f[k] = 0.f;
#pragma unroll
        for (int e = 0; e < G; ++e) {
          uint32_t u[16];
          if (nt > e) {
            tmem_ld16(tw + C::kColO + e * D + ch, u);
            tmem_wait_ld_keep(u);
          }
          // (a sum of weight 0 may be anything, a NaN row has l NaN)
#pragma unroll
          for (int k = 0; k < 16; ++k)
            if (some && weight[e] != 0.f) f[k] = fmaf(__uint_as_float(u[k]), weight[e] * inv, f[k]);
        }
        if (in && !is_split) {
#pragma unroll
          for (int k = 0; k < 16; k += 8)
            *reinterpret_cast<uint4*>(out + ch + k) =
                make_uint4(pack2<T>(f[k], f[k + 1]), pack2<T>(f[k + 2], f[k + 3]), pack2<T>(f[k + 4], f[k + 5]),
                           pack2<T>(f[k + 6], f[k + 7]));
        } else if (in) {
#pragma unroll
          for (int k = 0; k < 16; k += 4)
            *reinterpret_cast<float4*>(part + ch + k) = make_float4(f[k], f[k + 1], f[k + 2], f[k + 3]);
        }
      }
    }
    tc_fence_before();
  }
  join_roles(gave_up);
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmem);
  }
}

// Tiles that are split over the keys: all of them when they fill at most half of
// the resident CTAs (two per SM); else, when all tiles cost the same, those that
// would run as a last wave of at most half of them. As many parts as fill one
// wave, at least 512 keys in each, or 4096 when two fill it (one CTA per SM then
// runs nearly as fast as two). With and without parts: 4096 causal tokens, 2 heads
// of 64: 23 and 42 us; 16384, 1 head: 128 and 154; the last wave of 4 x 3136, 12
// heads of 32: 173 and 184; two parts of 4096, 4 heads: 47 and 44, hence not taken.
Split forward_split(const BiasAttnArgs& a) {
  const long long tiles = (long long)a.B * a.hq * ((a.Lq + 127) / 128), wave = 2LL * sm_count();
  long long last = 2 * tiles <= wave ? tiles : (a.causal ? 0 : tiles % wave);
  if (2 * last > wave) last = 0;
  const long long parts = last ? wave / last : 1, most = a.Lk / (parts > 2 ? 512 : 4096);
  const int n = (int)(parts < most ? parts : (most < 1 ? 1 : most));
  return n > 1 ? Split{n, last * 128, (int)(tiles - last), nullptr, nullptr} : Split{1, 0, 0, nullptr, nullptr};
}

template <class T, int D>
cudaError_t forward(const BiasAttnArgs& a, void* scratch, cudaStream_t st) {
  using C = FwdCfg<D>;
  static_assert(2 * (C::SMEM + 1024) <= 228 * 1024, "two CTAs per SM");
  cudaError_t e = cudaFuncSetAttribute(attn_fwd_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  Split sp = forward_split(a);
  split_place(&sp, D, scratch);
  const int dtype = std::is_same<T, __half>::value ? kFP16 : kBF16;
  FwdParams params;
  params.a = a;
  make_head_map(&params.q, a.q, a.B, a.Lq, a.hq, D, dtype, 128);
  make_head_map(&params.k, a.k, a.B, a.Lk, a.hk, D, dtype, C::BN);
  make_head_map(&params.v, a.v, a.B, a.Lk, a.hk, D, dtype, C::BN);
  const long long tiles = (long long)a.B * a.hq * ((a.Lq + 127) / 128);
  const long long grid = sp.n > 1 ? sp.first + (tiles - sp.first) * sp.n : tiles;
  prof_begin(kKindOther, st);
  attn_fwd_kernel<T, D><<<(unsigned)grid, C::THREADS, C::SMEM, st>>>(params, sp);
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
  return split_bytes(token_form(a) ? token_split(a) : forward_split(a), a.d);
}
cudaError_t launch_bias_attention(const BiasAttnArgs& a, int dtype, void* scratch, cudaStream_t st) {
  if (token_form(a)) return launch_token_attention(a, dtype, scratch, st);
  return dtype == kBF16 ? forward_d<__nv_bfloat16>(a, scratch, st) : forward_d<__half>(a, scratch, st);
}

}  // namespace vswin
