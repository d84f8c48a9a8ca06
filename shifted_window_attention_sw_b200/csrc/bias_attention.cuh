// What the kernels of the attention with bucketed bias share: the lengths and
// positions of a sequence, the bias of an offset, and the tensor-core tiles.
//
// Tiles in shared memory: rows in pieces of kPiece channels (64, or 32 for D =
// 32), a piece's rows one after another (128 or 64 bytes each) with the 16-byte
// chunk index XORed with the row (its low three bits, or bits 1-2): what TMA
// writes and the tensor core reads with the 128- or 64-byte swizzle. The same
// tile serves as a K-major operand (rows are M or N, channels are K) and as an
// MN-major one (channels are N, rows are K).
#pragma once

#include <cmath>
#include <cuda.h>

#include "sequence.h"
#include "sm100.cuh"

namespace vswin {

// A bias at or below this takes its key out of the softmax, as -inf does (so
// that the lowest value of a type works as a mask).
constexpr float kExclude = -1e30f;
// What a line's buckets hold for an offset whose map entry lies outside the table: its bias is 0 and it belongs to no
// row of the table's gradient.
constexpr int kNoBucket = 0xffff;
static_assert(kMaxBuckets <= kNoBucket, "no bucket of a table");
constexpr float kLog2E = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

enum : int { kErrAttnLoad = 0x121, kErrAttnMma = 0x122, kErrAttnSoftmax = 0x123 };

struct SeqLens {
  int nq, nk;  // query rows and keys that take part
  int start;   // position of query 0
};

// Lengths outside the tensors are recorded in the error word and clamped;
// positions are held within +-2^30, so that differences fit an int.
__device__ __forceinline__ SeqLens seq_lens(const BiasAttnArgs& a, int b) {
  SeqLens s;
  s.nq = a.q_lens ? a.q_lens[b] : a.Lq;
  s.nk = a.kv_lens ? a.kv_lens[b] : a.Lk;
  s.start = a.q_start ? a.q_start[b] : 0;
  constexpr int kMaxPos = 1 << 30;
  if (s.nq < 0 || s.nq > a.Lq || s.nk < 0 || s.nk > a.Lk || s.start < -kMaxPos || s.start > kMaxPos) {
    atomicCAS(a.ctx.err, 0, kErrBounds);
    s.nq = s.nq < 0 ? 0 : (s.nq > a.Lq ? a.Lq : s.nq);
    s.nk = s.nk < 0 ? 0 : (s.nk > a.Lk ? a.Lk : s.nk);
    s.start = s.start < -kMaxPos ? -kMaxPos : (s.start > kMaxPos ? kMaxPos : s.start);
  }
  return s;
}

// Bias of head h at offset `rel` = key - position of the query, -inf for a key
// that it takes out; a bucket outside the table is recorded in the error word
// and its bias is 0 (kNoBucket for the gradient).
template <class T>
__device__ __forceinline__ float bias_of(const BiasAttnArgs& a, int rel, int h, int* bucket = nullptr) {
  const int at = (rel < -a.D ? -a.D : (rel > a.D ? a.D : rel)) + a.D;
  int k = __ldg(a.map + at);
  if (k < 0 || k >= a.buckets) {
    atomicCAS(a.ctx.err, 0, kErrBounds);
    if (bucket) *bucket = kNoBucket;
    return 0.f;
  }
  if (bucket) *bucket = k;
  const float v = to_f(static_cast<const T*>(a.table)[(long long)k * a.hq + h]);
  return v <= kExclude ? -INFINITY : v;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Largest of three, NaN set aside.
__device__ __forceinline__ float max3(float x, float y, float z) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
  return r;
}

// The same, NaN when one of them is.
__device__ __forceinline__ float max3_nan(float x, float y, float z) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
  return r;
}

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}

template <class T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

template <class T>
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
  if constexpr (std::is_same<T, __half>::value) {
    const __half2 v = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&v);
  } else {
    const __nv_bfloat162 v =
        __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&v);
  }
}

// Instruction descriptor of an MMA on T (both operands) with fp32 accumulation.
template <class T>
__host__ __device__ constexpr uint32_t idesc16(int M, int N, int a_mn, int b_mn) {
  return sizeof(T) == 2 && std::is_same<T, __half>::value
             ? idesc_bf16(M, N, a_mn, b_mn) & ~((7u << 7) | (7u << 10))  // format 0: fp16
             : idesc_bf16(M, N, a_mn, b_mn);
}

template <int D>
struct TileOf {
  static constexpr int kPiece = D == 32 ? 32 : 64;      // channels
  static constexpr int kRow = kPiece * 2;               // bytes of a row of a piece
  static constexpr uint64_t kLayout = D == 32 ? 4 : 2;  // 64- or 128-byte swizzle
  static __device__ __forceinline__ int offset(int rows, int r, int c) {  // of 16-byte chunk c of row r
    const int piece = c / (kPiece / 8), x = c % (kPiece / 8);
    return piece * rows * kRow + r * kRow + ((x ^ (D == 32 ? (r >> 1) & 3 : r & 7)) << 4);
  }
};

// Operand descriptors: 8-row groups 8 kRow bytes apart. K-major: 16 channels of
// a piece are 32 bytes further on. MN-major: pieces `lbo` bytes apart, 16 rows
// are 16 kRow bytes further on.
template <int D>
__device__ __forceinline__ uint64_t tile_desc(uint32_t addr, uint32_t lbo) {
  uint64_t d = 0;
  d |= (uint64_t)((addr >> 4) & 0x3FFFu);
  d |= (uint64_t)((lbo >> 4) & 0x3FFFu) << 16;
  d |= (uint64_t)((8 * TileOf<D>::kRow) >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= TileOf<D>::kLayout << 61;
  return d;
}

// D[128 x ROWS] (+)= A B^T, A a tile of 128 rows, B of ROWS, both K-major.
template <int D, int ROWS>
__device__ __forceinline__ void mma_rows(uint32_t d_tmem, uint32_t a_addr, uint32_t b_addr, uint32_t idesc) {
  using Tl = TileOf<D>;
  const uint64_t da = tile_desc<D>(a_addr, 16), db = tile_desc<D>(b_addr, 16);
#pragma unroll
  for (int k = 0; k < D / 16; ++k) {
    const int piece = 16 * k / Tl::kPiece, in = 16 * k % Tl::kPiece * 2;
    umma_ss(d_tmem, da + ((piece * 128 * Tl::kRow + in) >> 4), db + ((piece * ROWS * Tl::kRow + in) >> 4), idesc, k > 0);
  }
}
// D[128 x D] (+)= A[128 x ROWS] B, A packed in TMEM (8 columns per 16 rows of B), B ROWS rows of a tile of TILE.
template <int D, int ROWS, int TILE = ROWS>
__device__ __forceinline__ void mma_acc(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_addr, uint32_t idesc, bool first) {
  const uint64_t db = tile_desc<D>(b_addr, TILE * TileOf<D>::kRow);
#pragma unroll
  for (int k = 0; k < ROWS / 16; ++k)
    umma_ts(d_tmem, a_tmem + 8 * k, db + (uint64_t)(k * TileOf<D>::kRow), idesc, (first && k == 0) ? 0u : 1u);
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// Rows of one head of a tensor, by TMA where a map could be made.
struct HeadMap {
  CUtensorMap map;    // (channels, tokens, heads, batch)
  int use;
  int hmul, bmul;     // 0 for a dimension of stride 0 (its map has one entry)
};

// cp.async of rows [r0, r0 + ROWS) of a head into a tile; rows outside [0, n)
// become zeros. `p` of `THREADS` threads (whole warps); a warp's copy takes 8
// rows of 4 chunks of 16 bytes.
template <class T, int D, int ROWS, int THREADS>
__device__ __forceinline__ void load_tile(uint32_t dst, const T* head, long long row_stride, int r0, int n, int p) {
  const int r = p & 7, c = (p >> 3) & 3;
  constexpr int kGroups = ROWS / 8 * (D / 32);  // groups of 8 rows x 32 channels
#pragma unroll 4
  for (int g = p >> 5; g < kGroups; g += THREADS / 32) {
    const int at = g / (D / 32) * 8 + r, chunk = g % (D / 32) * 4 + c;
    const int row = r0 + at;
    const bool in = row >= 0 && row < n;
    const T* src = head + (in ? (long long)row * row_stride : 0) + chunk * 8;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + TileOf<D>::offset(ROWS, at, chunk)), "l"(src),
                 "r"(in ? 16u : 0u)
                 : "memory");
  }
}

// Rows [r0, r0 + ROWS) of head h of sequence b into a tile, by one warp, whose
// one arrival completes `bar` with the copies. n of the L rows take part: whole
// tiles go by TMA (which reads zeros behind L); a tile in which the length ends
// goes by cp.async, which reads nothing behind it, whatever it holds.
template <class T, int D, int ROWS>
__device__ __forceinline__ void bring_tile(uint32_t dst, const HeadMap& m, const Heads& v, int b, int h, int r0, int n,
                                           int L, uint64_t* bar) {
  using Tl = TileOf<D>;
  const int lane = threadIdx.x & 31;
  if (m.use && (r0 + ROWS <= n || n == L)) {
    if (lane == 0) {
      mbar_arrive_expect_tx(bar, ROWS * D * 2);
#pragma unroll
      for (int c = 0; c < D; c += Tl::kPiece)
        asm volatile(
            "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, "
            "%5}], [%6];" ::"r"(dst + c / Tl::kPiece * ROWS * Tl::kRow),
            "l"(reinterpret_cast<uint64_t>(&m.map)), "r"(c), "r"(r0), "r"(h * m.hmul), "r"(b * m.bmul), "r"(smem_u32(bar))
            : "memory");
    }
  } else {
    load_tile<T, D, ROWS, 32>(dst, static_cast<const T*>(v.p) + v.at(b, 0, h), v.st, r0, n, lane);
    cp_async_wait_all();
    fence_proxy_async_smem();  // bytes written by cp.async are read by the tensor core
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
  }
}

// A whole warp waits; false in every lane, and *gave_up set, when the wait gave
// up (as mbar_wait does). The hardware suspends the warp for up to the hint (ns) per try: waiting
// warps that poll more often take issue slots from the working ones.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const KernelCtx& ctx, int code,
                                          uint32_t* gave_up) {
  auto once = [&]() {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(20000u)
        : "memory");
    return __all_sync(0xffffffffu, ok != 0);
  };
  if (once()) return true;
  const uint64_t t0 = global_timer_ns();
  while (!once()) {
    if (__any_sync(0xffffffffu, global_timer_ns() - t0 > ctx.wait_limit)) {
      if ((threadIdx.x & 31) == 0) atomicCAS(ctx.err, 0, code);
      *gave_up = 1;
      return false;
    }
  }
  return true;
}

// Where a kernel's roles meet at its end. When a wait gave up (`gave_up`, in
// shared memory), copies and MMAs may still be under way: they get a millisecond
// to land before shared memory and TMEM are given back.
__device__ __forceinline__ void join_roles(const volatile uint32_t* gave_up) {
  __syncthreads();
  if (*gave_up) {
    const uint64_t t0 = global_timer_ns();
    for (int k = 0; k < 100000 && global_timer_ns() - t0 < 1000000; ++k) __nanosleep(1000);
  }
}

// One lane of a converged warp, which the compiler knows to be one: MMAs issued
// under it take ~10-30 cycles each, under `lane == 0` ~50-60 (measured: 16
// MMAs of N = 64 issue in 277 against 726 cycles), since their operands then go
// to uniform registers without a loop over the lanes.
__device__ __forceinline__ bool elect_one() {
  uint32_t pred = 0;
  asm volatile(
      "{\n\t.reg .pred P;\n\telect.sync _|P, 0xffffffff;\n\tselp.u32 %0, 1, 0, P;\n\t}"
      : "=r"(pred));
  return pred != 0;
}

// The bias of a 128 x BN tile depends on the offset of key and query alone, so
// it is one line of N = 127 + BN values, entry t at offset base + t: row i and
// column j read entry j - i + 127 (rows are queries) or i - j + BN - 1 (rows are
// keys). A line whose entries are all the same (`flat`; far tiles have one
// bucket) is only `value` and its bucket `which`. With kBuckets the
// buckets are kept too, and entries are the same only if their buckets are.
template <int N, bool kBuckets>
struct BiasLine {
  float line[N + 1];
  uint16_t bucket[kBuckets ? N + 1 : 2];
  float value;
  int which;
  int flat;
};

// One warp writes lines of a head: the values beyond the map's ends are held, so
// that far tiles read nothing.
template <class T, int N, bool kBuckets>
struct LineWriter {
  const BiasAttnArgs& a;
  int h, low_which, high_which;
  float low, high;

  __device__ __forceinline__ float entry(int rel, int* k) const {
    const float v = bias_of<T>(a, rel, h, k) * kLog2E;
    return a.causal && rel > 0 ? -INFINITY : v;  // the causal rule is part of the line
  }
  __device__ __forceinline__ LineWriter(const BiasAttnArgs& args, int head) : a(args), h(head) {
    low = entry(-a.D, &low_which);
    high = entry(a.D + 1, &high_which);
  }
  __device__ __forceinline__ void head(int head) {
    if (head == h) return;
    h = head;
    low = entry(-a.D, &low_which);
    high = entry(a.D + 1, &high_which);
  }
  __device__ __forceinline__ void write(BiasLine<N, kBuckets>* o, int base) const {
    const int lane = threadIdx.x & 31;
    // a tile beyond one of the map's ends, on one side of the causal border
    bool flat = base > a.D || base + N - 1 <= -a.D;
    float value = base > a.D ? high : low;
    int which = base > a.D ? high_which : low_which;
    if (!flat) {
      constexpr int kPer = (N + 31) / 32;
      float v[kPer];
      int k[kPer];
      // the map's entries, then the table's: two rounds of loads in flight at once
#pragma unroll
      for (int t = 0; t < kPer; ++t) {
        const int rel = base + min(32 * t + lane, N - 1);
        k[t] = __ldg(a.map + min(max(rel, -a.D), a.D) + a.D);
      }
      bool bad = false;
#pragma unroll
      for (int t = 0; t < kPer; ++t) {
        const bool in = (unsigned)k[t] < (unsigned)a.buckets;
        bad = bad || !in;
        k[t] = in ? k[t] : kNoBucket;
        v[t] = in ? to_f(static_cast<const T*>(a.table)[(long long)k[t] * a.hq + h]) : 0.f;
      }
      if (bad) atomicCAS(a.ctx.err, 0, kErrBounds);
#pragma unroll
      for (int t = 0; t < kPer; ++t) {
        const bool gone = v[t] <= kExclude || (a.causal && base + min(32 * t + lane, N - 1) > 0);
        v[t] = gone ? -INFINITY : v[t] * kLog2E;
      }
      value = __shfl_sync(0xffffffffu, v[0], 0);
      which = __shfl_sync(0xffffffffu, k[0], 0);
      flat = true;
#pragma unroll
      for (int t = 0; t < (N + 31) / 32; ++t) {
        if (32 * t + lane < N) {
          o->line[32 * t + lane] = v[t];
          if (kBuckets) o->bucket[32 * t + lane] = (uint16_t)k[t];
        }
        flat = flat && v[t] == value && (!kBuckets || k[t] == which);
      }
      flat = __all_sync(0xffffffffu, flat);
    }
    if (lane == 0) {
      o->value = value;
      o->which = which;
      o->flat = flat;
    }
    __syncwarp();  // the leader's arrival stands for the warp
  }
};

// Map of a tensor of B x L x H rows of d channels in boxes of `rows` rows; false
// (m->use = 0) when its strides have no map.
bool make_head_map(HeadMap* m, const Heads& v, int B, int L, int H, int d, int dtype, int rows);

}  // namespace vswin
