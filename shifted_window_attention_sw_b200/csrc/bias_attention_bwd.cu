// Gradient of the attention with bucketed bias. With the forward's P (rebuilt
// from lse), dP = dO v^T and D_i = dO_i . o_i:
//
//   dS = P (dP - D),  dq = scale dS k,  dk = scale dS^T q,  dv = P^T dO,
//   dtable[bucket][h] = sum of dS over the pairs of that bucket.
//
// Two passes of one kernel, each with 128 fixed rows and moving tiles of 64
// rows: queries fixed (dq and the table's gradient; it also leaves D for the
// other pass), then keys fixed (dk and dv, summed over the heads that share
// them). Each recomputes S and dP on tcgen05 (7 products instead of the 5 of a
// single pass), and in return every sum has one owner and a fixed order: no
// atomics, the same result for the same call.
//
// Measured: 4096 causal tokens, 2 x 12 heads of 64: 145 + 155 us, beside 93 of the
// forward (the seven products that both need take 107 us at the measured peak);
// 8 x 577 tokens, 6 heads: 29 + 25 us. At the first size tensor cores are 0.27 and
// 0.32 busy, special functions 0.36 and 0.32, issue 0.42: bound by the chain scores -
// P and dS - sums of a CTA, which the other CTA of the SM covers in part. The whole
// call, one sequence of 4096 causal tokens: 16 heads of 128 349 us, over 4 key heads
// 457; 32 heads of 64 393 us, over one key head 2487; 4 x 3136 tokens, 12 heads of 32:
// 618. With few key heads the second pass has few CTAs: one per 128 keys and key head,
// which walks all the heads that share it. Tried: one CTA per SM with two
// groups of warps and three score buffers (163 instead of 145 us for the first
// pass) or with three groups (slower, too: one warp issues for all), columns'
// (lse, D) fetched a tile earlier (no change).
//
// P and dS are rounded to the tensors' 16 bits once, as operands of the sums; D
// comes from the 16-bit out. dtable sums the unrounded dS in fp32.
//
// Per tile: X = F1 M1^T and Y = F2 M2^T into TMEM (fp32; queries fixed: F = q,
// dO and M = k, v; keys fixed: F = k, v and M = q, dO), eight warps (TMEM lane =
// fixed row, four warps per half of the columns) form P and dS and write them
// back as 16-bit operands over the scores, then the sums += dS M1 (and P M2) as
// TS MMAs. D = 32 and 64: one such group of warps, two CTAs per SM; D = 128: two
// groups on alternating tiles with a score buffer each, one CTA per SM (the sums
// take 256 TMEM columns).
//
// The table's gradient sums dS along diagonals (the bias is one line per tile,
// see BiasLine). A tile of one bucket adds its rows' sums. In the others a
// warp passes partial sums from lane to lane, in four runs of eight columns: after
// column c of a run, lane 31 holds the run's sum of diagonal c - 31. The 63
// diagonals of the warp's 32 x 32 part, the runs added, then go to its bins, equal
// buckets combined in lane order.
#include "bias_attention.cuh"

namespace vswin {
namespace {

constexpr int kBn = 64;             // moving rows per tile
constexpr int kLineN = 127 + kBn;   // offsets in a tile

template <int D, bool kKeys>
struct BwdCfg {
  static constexpr int G = D == 128 ? 2 : 1;  // groups of eight warps
  static constexpr int CTAS = D == 128 ? 1 : 2;
  static constexpr int ST = 3;  // stages of the moving tiles
  static constexpr int kWarps = 8 * G;
  static constexpr int THREADS = 32 * (kWarps + 3);
  using Line = BiasLine<kLineN, !kKeys>;
  static constexpr int kFixed = 128 * D * 2, kMoving = kBn * D * 2;
  static constexpr int OFF_F = 0;                                   // F1, F2
  static constexpr int OFF_M = 2 * kFixed;                          // per stage M1, M2
  static constexpr int OFF_LINE = OFF_M + ST * 2 * kMoving;
  static constexpr int OFF_COL = OFF_LINE + (ST * (int)sizeof(Line) + 15) / 16 * 16;  // per stage and column (-lse, -D)
  static constexpr int OFF_DIAG = OFF_COL + (kKeys ? ST * kBn * 8 : 0);
  static constexpr int OFF_BAR = OFF_DIAG + (kKeys ? 0 : kWarps * 160 * 4);
  static constexpr int OFF_BINS = OFF_BAR + 192;                    // [kWarps][buckets], queries fixed
  static constexpr uint32_t kTmem = D == 128 ? 512 : 256;
  static constexpr int kColAcc = 128 * G;  // sums behind the score buffers
  static_assert(kColAcc + (kKeys ? 2 : 1) * D <= (int)kTmem, "TMEM columns of a CTA");
};

struct BwdArgs {
  HeadMap f1, f2, m1, m2;  // of the fixed and moving tiles
  BiasAttnArgs a;
  float* delta;    // [B][hq][Lq] D
  float* dtab;     // [hq][B * query tiles][buckets] shares of the table's gradient
};

// D[128 x D] (+)= A[128 x 64] B, A packed in TMEM in two halves of 32 rows of B, 32 columns apart.
template <int D>
__device__ __forceinline__ void mma_halves(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_addr, uint32_t idesc, bool first) {
  mma_acc<D, 32, kBn>(d_tmem, a_tmem, b_addr, idesc, first);
  mma_acc<D, 32, kBn>(d_tmem, a_tmem + 32, b_addr + 32 * TileOf<D>::kRow, idesc, false);
}

template <class T, int D, bool kKeys>
__global__ void __launch_bounds__(BwdCfg<D, kKeys>::THREADS, BwdCfg<D, kKeys>::CTAS)
    attn_bwd_kernel(const __grid_constant__ BwdArgs args) {
  using C = BwdCfg<D, kKeys>;
  using Line = typename C::Line;
  constexpr int G = C::G, ST = C::ST;
  constexpr int kMmaWarp = C::kWarps;
  extern __shared__ __align__(1024) uint8_t smem[];
  const BiasAttnArgs& a = args.a;
  Line* lines = reinterpret_cast<Line*>(smem + C::OFF_LINE);
  float2* cols = reinterpret_cast<float2*>(smem + C::OFF_COL);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* full = bars;            // [ST] moving tiles, line and columns
  uint64_t* free_ = bars + ST;      // [ST] their MMAs and reads are done
  uint64_t* s_full = bars + 2 * ST;       // [G] scores in TMEM
  uint64_t* ds_full = s_full + G;         // [G] operands written back
  uint64_t* f_full = ds_full + G;         // fixed tiles
  uint64_t* done = f_full + 1;            // every sum accumulated
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(done + 1);
  uint32_t* gave_up = s_tmem + 1;         // a wait ran out

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int ft = (int)((gridDim.x - 1 - blockIdx.x) / (a.B * (kKeys ? a.hk : a.hq)));
  const int rest = (int)((gridDim.x - 1 - blockIdx.x) % (a.B * (kKeys ? a.hk : a.hq)));
  const int fixed_tiles = gridDim.x / (a.B * (kKeys ? a.hk : a.hq));
  const int group = a.hq / a.hk;
  const int hf = rest % (kKeys ? a.hk : a.hq), b = rest / (kKeys ? a.hk : a.hq);
  const int hk = kKeys ? hf : hf / group;
  const SeqLens sl = seq_lens(a, b);
  // causal: the heavy fixed tiles are the last queries and the first keys
  const int f0 = (kKeys ? fixed_tiles - 1 - ft : ft) * 128;
  // moving rows [m_lo, m_hi) that some fixed row meets
  int m_lo = 0, m_hi;
  if (kKeys) {
    m_hi = f0 < sl.nk ? sl.nq : 0;
    if (a.causal) m_lo = min(max(0, f0 - sl.start), m_hi) / kBn * kBn;
  } else {
    m_hi = f0 < sl.nq ? sl.nk : 0;
    if (a.causal) m_hi = min(m_hi, max(0, sl.start + min(f0 + 128, sl.nq)));
  }
  const int per_head = (m_hi - m_lo + kBn - 1) / kBn;
  const int nt = per_head * (kKeys ? group : 1);

  if (tid == 0) {
    for (int k = 0; k < ST; ++k) {
      mbar_init(&full[k], 3);
      mbar_init(&free_[k], 1 + 8);
    }
    for (int k = 0; k < G; ++k) {
      mbar_init(&s_full[k], 1);
      mbar_init(&ds_full[k], 8);
    }
    mbar_init(f_full, 2);
    mbar_init(done, 1);
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
  // (not before this block has its columns: blocks of the pass that follows hold theirs while they wait for this one)
  let_next_start();
  const uint32_t sf = smem_u32(smem + C::OFF_F), sm = smem_u32(smem + C::OFF_M);
  // the other pass, whose D this one reads (before any bounded wait; and the table's sums count on both having ended)
  if (kKeys) after_previous();

  if (warp > kMmaWarp) {
    // ------------------------------------------------------------ producers: tiles; bias lines and columns
    int s = 0, u = 0, r0 = m_lo, h = kKeys ? hk * group : hf;
    uint32_t parity = 1;  // of the stage's previous use
    if (warp == kMmaWarp + 1) {
      const Heads &F1 = kKeys ? a.k : a.q, &F2 = kKeys ? a.v : a.dout, &M1 = kKeys ? a.q : a.k, &M2 = kKeys ? a.dout : a.v;
      const int fn = kKeys ? sl.nk : sl.nq, fL = kKeys ? a.Lk : a.Lq;
      const int mn = kKeys ? sl.nq : sl.nk, mL = kKeys ? a.Lq : a.Lk;
      if (nt > 0) {
        bring_tile<T, D, 128>(sf, args.f1, F1, b, hf, f0, fn, fL, f_full);
        bring_tile<T, D, 128>(sf + C::kFixed, args.f2, F2, b, hf, f0, fn, fL, f_full);
      }
      for (int t = 0; t < nt; ++t) {
        if (t >= ST && !warp_wait(&free_[s], parity, a.ctx, kErrAttnLoad, gave_up)) break;
        const int hm = kKeys ? h : hk;
        const uint32_t dst = sm + s * 2 * C::kMoving;
        bring_tile<T, D, kBn>(dst, args.m1, M1, b, hm, r0, mn, mL, &full[s]);
        bring_tile<T, D, kBn>(dst + C::kMoving, args.m2, M2, b, hm, r0, mn, mL, &full[s]);
        if (++s == ST) s = 0, parity ^= 1;
        r0 += kBn;
        if (++u == per_head) u = 0, r0 = m_lo, ++h;
      }
    } else if (nt > 0) {
      LineWriter<T, kLineN, !kKeys> writer(a, h);
      for (int t = 0; t < nt; ++t) {
        if (t >= ST && !warp_wait(&free_[s], parity, a.ctx, kErrAttnLoad, gave_up)) break;
        if constexpr (kKeys) {
#pragma unroll
          for (int e = 0; e < kBn; e += 32) {
            const int i = r0 + e + lane;
            float2 c = make_float2(-INFINITY, 0.f);  // a query that takes no part: P = 0
            if (i < m_hi) {
              const long long r = ((long long)b * a.hq + h) * a.Lq + i;
              const float lse = a.lse[r];
              if (lse != -INFINITY) c = make_float2(-lse * kLog2E, -args.delta[r]);
            }
            cols[s * kBn + e + lane] = c;
          }
          writer.head(h);
          writer.write(&lines[s], f0 - (sl.start + r0) - (kBn - 1));
        } else {
          writer.write(&lines[s], r0 - (sl.start + f0) - 127);
        }
        if (lane == 0) mbar_arrive(&full[s]);
        if (++s == ST) s = 0, parity ^= 1;
        r0 += kBn;
        if (++u == per_head) u = 0, r0 = m_lo, ++h;
      }
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ MMA issue
    // (the whole warp waits, one elected lane issues)
    constexpr uint32_t id_s = idesc16<T>(128, kBn, 0, 0), id_acc = idesc16<T>(128, D, 0, 1);
    auto scores = [&](int t) {  // by the elected lane
      const uint32_t buf = tmem + 128 * (t % G), m1 = sm + t % ST * 2 * C::kMoving;
      mma_rows<D, kBn>(buf, sf, m1, id_s);
      mma_rows<D, kBn>(buf + 64, sf + C::kFixed, m1 + C::kMoving, id_s);
      umma_commit(&s_full[t % G]);
    };
    auto wait_tile = [&](int t) { return warp_wait(&full[t % ST], (t / ST) & 1, a.ctx, kErrAttnMma, gave_up); };
    bool ok = nt > 0 && warp_wait(f_full, 0, a.ctx, kErrAttnMma, gave_up);
    for (int t = 0; t < G && t < nt && ok; ++t) {
      ok = wait_tile(t);
      if (!ok) break;
      tc_fence_after();
      if (elect_one()) scores(t);
      __syncwarp();
    }
    for (int t = 0; t < nt && ok; ++t) {
      const int u = t + G;  // the tile whose scores take this one's buffer
      ok = warp_wait(&ds_full[t % G], (t / G) & 1, a.ctx, kErrAttnMma, gave_up);
      if (!ok) break;
      // the scores that follow go out at once when their tiles are there
      const bool now = u < nt && __all_sync(0xffffffffu, mbar_test(&full[u % ST], (u / ST) & 1));
      tc_fence_after();
      if (elect_one()) {
        const uint32_t buf = tmem + 128 * (t % G), m1 = sm + t % ST * 2 * C::kMoving;
        mma_halves<D>(tmem + C::kColAcc, buf + 64, m1, id_acc, t == 0);  // dq += dS k, or dk += dS^T q
        if (kKeys) mma_halves<D>(tmem + C::kColAcc + D, buf, m1 + C::kMoving, id_acc, t == 0);  // dv += P^T dO
        umma_commit(&free_[t % ST]);
        if (t == nt - 1) umma_commit(done);
        if (now) scores(u);  // runs after the sums, which read these columns
      }
      __syncwarp();
      if (u < nt && !now) {
        ok = wait_tile(u);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) scores(u);
        __syncwarp();
      }
    }
  } else {
    // ------------------------------------------------------------ P and dS
    const int quad = warp >> 2, g = quad >> 1, c_first = 32 * (quad & 1);  // group, first column of its half of a tile
    const int row = (warp & 3) * 32 + lane, i = f0 + row;
    const uint32_t tl = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t buf = tmem + tl + 128 * g;
    const float c = a.scale * kLog2E;
    const float2 c2 = make_float2(c, c);
    float* bins = reinterpret_cast<float*>(smem + C::OFF_BINS) + warp * a.buckets;
    float* diag = reinterpret_cast<float*>(smem + C::OFF_DIAG) + warp * 160;  // [4][40]
    float nl = -INFINITY, nd = 0.f;  // queries fixed: -lse (log2) and -D of the row
    float flat_sum = 0.f;            // dS of tiles of one bucket, until the bucket changes
    int flat_bucket = 0;
    if (!kKeys) {
      for (int k = lane; k < a.buckets; k += 32) bins[k] = 0.f;
      if (i < a.Lq) {
        const long long r = ((long long)b * a.hq + hf) * a.Lq + i;
        float dd = 0.f;
        if (i < sl.nq) {
          const float lse = a.lse[r];
          if (lse != -INFINITY) {
            const T* o = static_cast<const T*>(a.o.p) + a.o.at(b, i, hf);
            const T* go = static_cast<const T*>(a.dout.p) + a.dout.at(b, i, hf);
#pragma unroll
            for (int k = 0; k < D; k += 8) {
              const uint4 ou = *reinterpret_cast<const uint4*>(o + k), gu = *reinterpret_cast<const uint4*>(go + k);
              const T *oe = reinterpret_cast<const T*>(&ou), *ge = reinterpret_cast<const T*>(&gu);
#pragma unroll
              for (int e = 0; e < 8; ++e) dd = fmaf(to_f(oe[e]), to_f(ge[e]), dd);
            }
            nl = -lse * kLog2E;
            nd = -dd;
          }
        }
        if (quad == 0) args.delta[r] = dd;
      }
      __syncwarp();
    }
    // a bucket's sum over the warp goes to its bin
    auto flush_flat = [&]() {
      float v = flat_sum;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      if (lane == 0 && flat_bucket != kNoBucket) bins[flat_bucket] += v;
      __syncwarp();
      flat_sum = 0.f;
    };
    int s = g;
    uint32_t sp = 0;
    bool ok = true;
    for (int t = g; t < nt; t += G) {
      ok = warp_wait(&full[s], sp, a.ctx, kErrAttnSoftmax, gave_up) && warp_wait(&s_full[g], (t / G) & 1, a.ctx, kErrAttnSoftmax, gave_up);
      if (!ok) break;
      tc_fence_after();
      const Line& bl = lines[s];
      const bool flat = bl.flat != 0;
      const float value = bl.value;
      const float* line = bl.line + (kKeys ? kBn - 1 + row : 127 - row);
      const float2* col = cols + s * kBn;
      const int live = kKeys ? kBn : m_hi - t * kBn;  // queries fixed: columns of the tile that are keys
      float2 sum = make_float2(0.f, 0.f);
      if (!kKeys && flat && bl.which != flat_bucket) {
        flush_flat();
        flat_bucket = bl.which;
      }
      // this warp's half of the tile, of one bucket or not, with keys missing or not
      auto form = [&](auto flat_, auto cut_) {
        constexpr bool kFlat = decltype(flat_)::value, kCut = decltype(cut_)::value;
#pragma unroll
        for (int e = 0; e < 32; e += 16) {
          const int c0 = c_first + e;
          uint32_t us[16], ud[16], w[8], wp[8];
          tmem_ld16(buf + c0, us);
          tmem_ld16(buf + 64 + c0, ud);
          tmem_wait_ld_keep(us);
          tmem_wait_ld_keep(ud);
          float ds[16];
#pragma unroll
          for (int k = 0; k < 16; k += 2) {
            float2 off = make_float2(nl, nl), d2 = make_float2(nd, nd);
            if (kKeys) {
              const float4 q = *reinterpret_cast<const float4*>(col + c0 + k);  // two columns' (-lse, -D)
              off = make_float2(q.x, q.z);
              d2 = make_float2(q.y, q.w);
            }
            if (kFlat)
              off = __fadd2_rn(off, make_float2(value, value));
            else if (kKeys)
              off = __fadd2_rn(off, make_float2(line[-(c0 + k)], line[-(c0 + k + 1)]));
            else
              off = __fadd2_rn(off, make_float2(line[c0 + k], line[c0 + k + 1]));
            float2 x = __ffma2_rn(make_float2(__uint_as_float(us[k]), __uint_as_float(us[k + 1])), c2, off);
            if (kCut) {
              x.x = c0 + k < live ? x.x : -INFINITY;
              x.y = c0 + k + 1 < live ? x.y : -INFINITY;
            }
            const float2 pr = make_float2(ex2(x.x), ex2(x.y));
            const float2 d =
                __fmul2_rn(pr, __fadd2_rn(make_float2(__uint_as_float(ud[k]), __uint_as_float(ud[k + 1])), d2));
            if (kKeys) wp[k / 2] = pack2<T>(pr.x, pr.y);
            w[k / 2] = pack2<T>(d.x, d.y);
            ds[k] = d.x;
            ds[k + 1] = d.y;
            if (!kKeys && kFlat) sum = __fadd2_rn(sum, d);
          }
          // over scores of this half that have been read
          if (kKeys) tmem_st8(buf + c_first + e / 2, wp);
          tmem_st8(buf + 64 + c_first + e / 2, w);
          if (!kKeys && !kFlat) {  // two runs of eight columns side by side
            float acc[2] = {0.f, 0.f};
#pragma unroll
            for (int k = 0; k < 8; ++k) {
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                const float up = __shfl_up_sync(0xffffffffu, acc[x], 1);
                acc[x] = (lane == 0 ? 0.f : up) + ds[8 * x + k];
                if (lane == 31) diag[(e / 8 + x) * 40 + k] = acc[x];
              }
            }
            if (lane < 31) {
              diag[e / 8 * 40 + 38 - lane] = acc[0];
              diag[(e / 8 + 1) * 40 + 38 - lane] = acc[1];
            }
          }
        }
      };
      using Yes = std::true_type;
      using No = std::false_type;
      if (live >= kBn) {
        if (flat)
          form(Yes{}, No{});
        else
          form(No{}, No{});
      } else if constexpr (!kKeys) {
        if (flat)
          form(Yes{}, Yes{});
        else
          form(No{}, Yes{});
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ds_full[g]);
      if (!kKeys) {
        if (flat) {
          flat_sum += sum.x + sum.y;
        } else {
          __syncwarp();
          float v[2] = {0.f, 0.f};
          int bucket[2], start[2];
          uint32_t heads[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int at = lane + 32 * k;  // diagonal at - 31 of the warp's 32 x 32
#pragma unroll
            for (int x = 0; x < 4; ++x)
              if (at >= 8 * x && at - 8 * x < 39) v[k] += diag[x * 40 + at - 8 * x];
            bucket[k] = at < 63 ? bl.bucket[at + 96 + c_first - 32 * (warp & 3)] : kNoBucket;
            const int before = __shfl_up_sync(0xffffffffu, bucket[k], 1);
            heads[k] = __ballot_sync(0xffffffffu, lane == 0 || before != bucket[k]);
            start[k] = 31 - __clz(heads[k] & (0xffffffffu >> (31 - lane)));
          }
          // a run of one bucket adds up into its last lane
#pragma unroll
          for (int o = 1; o < 32; o *= 2) {
            const float x[2] = {__shfl_up_sync(0xffffffffu, v[0], o), __shfl_up_sync(0xffffffffu, v[1], o)};
#pragma unroll
            for (int k = 0; k < 2; ++k)
              if (lane - o >= start[k]) v[k] += x[k];
          }
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const bool tail = bucket[k] != kNoBucket && (lane == 31 || ((heads[k] >> (lane + 1)) & 1));
            // runs that share a bucket (no map of vswin_bucket_map has them) add up into the first
            const uint32_t equal = __match_any_sync(0xffffffffu, tail ? bucket[k] : -2 - lane);
            const bool first = (equal & ((1u << lane) - 1)) == 0;
            uint32_t others = first ? equal & ~(1u << lane) : 0;
            while (__any_sync(0xffffffffu, others != 0)) {
              const float x = __shfl_sync(0xffffffffu, v[k], others ? __ffs(others) - 1 : lane);
              if (others) {
                v[k] += x;
                others &= others - 1;
              }
            }
            if (tail && first) bins[bucket[k]] += v[k];
            __syncwarp();
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&free_[s]);
      s += G;
      if (s >= ST) s -= ST, sp ^= 1;
    }
    if (!kKeys) flush_flat();
    if (ok && nt > 0) ok = warp_wait(done, 0, a.ctx, kErrAttnSoftmax, gave_up);
    tc_fence_after();
    if (ok) {
      // every quad writes its part of the sums' columns: dq, or dk and then dv
      const int n_out = kKeys ? a.Lk : a.Lq;
      const bool some = i < (kKeys ? sl.nk : sl.nq) && nt > 0;
      constexpr int kCols = (kKeys ? 2 : 1) * D / (2 * G);
      const int first = quad * kCols;
      const bool is_dv = kKeys && first >= D;
      const Heads& out = !kKeys ? a.dq : (is_dv ? a.dv : a.dk);
      const float scale = is_dv ? 1.f : a.scale;
      T* dst = static_cast<T*>(out.p) + (i < n_out ? out.at(b, i, hf) : 0) + (is_dv ? first - D : first);
#pragma unroll
      for (int c0 = 0; c0 < kCols; c0 += 16) {
        uint32_t u[16];
        if (nt > 0) {
          tmem_ld16(tmem + tl + C::kColAcc + first + c0, u);
          tmem_wait_ld_keep(u);
        }
        float f[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) f[k] = some ? __uint_as_float(u[k]) * scale : 0.f;
        if (i < n_out) {
#pragma unroll
          for (int k = 0; k < 16; k += 8)
            *reinterpret_cast<uint4*>(dst + c0 + k) =
                make_uint4(pack2<T>(f[k], f[k + 1]), pack2<T>(f[k + 2], f[k + 3]), pack2<T>(f[k + 4], f[k + 5]),
                           pack2<T>(f[k + 6], f[k + 7]));
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
  if (!kKeys) {  // this CTA's share of the table's gradient
    const float* bins = reinterpret_cast<const float*>(smem + C::OFF_BINS);
    float* out = args.dtab + (((long long)hf * a.B + b) * fixed_tiles + f0 / 128) * a.buckets;
    for (int k = tid; k < a.buckets; k += C::THREADS) {
      float v = 0.f;
      for (int w = 0; w < C::kWarps; ++w) v += bins[w * a.buckets + k];
      out[k] = v;
    }
  }
}

// dtable = the CTAs' shares of a head added in a fixed order: 32 buckets per
// block, eight runs of shares side by side.
template <class T>
__global__ void __launch_bounds__(256) attn_dtable_kernel(const float* dtab, int shares, int buckets, int hq, T* out) {
  after_previous();
  __shared__ float s[8][33];
  const int h = blockIdx.x, lane = threadIdx.x & 31, run = threadIdx.x >> 5;
  const int k = blockIdx.y * 32 + lane;
  float v = 0.f;
  if (k < buckets)
    for (int c = run; c < shares; c += 8) v += dtab[((long long)h * shares + c) * buckets + k];
  s[run][lane] = v;
  __syncthreads();
  if (run == 0 && k < buckets) {
    for (int r = 1; r < 8; ++r) v += s[r][lane];
    out[(long long)k * hq + h] = from_f<T>(v);
  }
}

template <class T, int D, bool kKeys>
cudaError_t pass(BwdArgs& args, cudaStream_t st) {
  using C = BwdCfg<D, kKeys>;
  const BiasAttnArgs& a = args.a;
  const int smem = C::OFF_BINS + (kKeys ? 0 : C::kWarps * a.buckets * 4);
  constexpr int kMost = C::OFF_BINS + (kKeys ? 0 : C::kWarps * kMaxBuckets * 4);
  static_assert(C::CTAS * (kMost + 1024) <= 228 * 1024, "shared memory of an SM");
  cudaError_t e = cudaFuncSetAttribute(attn_bwd_kernel<T, D, kKeys>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
  if (e != cudaSuccess) return e;
  const int dtype = std::is_same<T, __half>::value ? kFP16 : kBF16;
  auto map = [&](HeadMap* m, const Heads& v, bool keys, int rows) {
    make_head_map(m, v, a.B, keys ? a.Lk : a.Lq, keys ? a.hk : a.hq, D, dtype, rows);
  };
  map(&args.f1, kKeys ? a.k : a.q, kKeys, 128);
  map(&args.f2, kKeys ? a.v : a.dout, kKeys, 128);
  map(&args.m1, kKeys ? a.q : a.k, !kKeys, kBn);
  map(&args.m2, kKeys ? a.dout : a.v, !kKeys, kBn);
  const long long grid = (long long)a.B * (kKeys ? a.hk : a.hq) * (((kKeys ? a.Lk : a.Lq) + 127) / 128);
  prof_begin(kKindAttnBwd, st);
  if (kKeys) {
    e = launch_after(attn_bwd_kernel<T, D, kKeys>, dim3((unsigned)grid), C::THREADS, smem, st, args);
  } else {
    attn_bwd_kernel<T, D, kKeys><<<(unsigned)grid, C::THREADS, smem, st>>>(args);
    e = cudaGetLastError();
  }
  prof_end(kKindAttnBwd, st);
  count_launch();
  return e;
}

size_t delta_bytes(const BiasAttnArgs& a) { return ((size_t)a.B * a.hq * a.Lq * 4 + 255) / 256 * 256; }

template <class T, int D>
cudaError_t backward(const BiasAttnArgs& a, void* scratch, cudaStream_t st) {
  BwdArgs args;
  args.a = a;
  args.delta = static_cast<float*>(scratch);
  args.dtab = reinterpret_cast<float*>(static_cast<char*>(scratch) + delta_bytes(a));
  cudaError_t e = pass<T, D, false>(args, st);
  if (e == cudaSuccess) e = pass<T, D, true>(args, st);
  if (e != cudaSuccess) return e;
  prof_begin(kKindOther, st);
  e = launch_after(attn_dtable_kernel<T>, dim3(a.hq, (a.buckets + 31) / 32), 256, 0, st, args.dtab, a.B * ((a.Lq + 127) / 128),
                   a.buckets, a.hq, static_cast<T*>(a.dtable));
  prof_end(kKindOther, st);
  count_launch();
  return e;
}

template <class T>
cudaError_t backward_d(const BiasAttnArgs& a, void* scratch, cudaStream_t st) {
  if (a.d == 32) return backward<T, 32>(a, scratch, st);
  if (a.d == 64) return backward<T, 64>(a, scratch, st);
  return backward<T, 128>(a, scratch, st);
}

}  // namespace

size_t bias_attention_backward_scratch_bytes(const BiasAttnArgs& a) {
  return delta_bytes(a) + (size_t)a.hq * a.B * ((a.Lq + 127) / 128) * a.buckets * 4;
}
cudaError_t launch_bias_attention_backward(const BiasAttnArgs& a, int dtype, void* scratch, cudaStream_t st) {
  return dtype == kBF16 ? backward_d<__nv_bfloat16>(a, scratch, st) : backward_d<__half>(a, scratch, st);
}

}  // namespace vswin
