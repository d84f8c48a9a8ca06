// C ABI of the operators over token sequences and of the optimizer step:
// argument validation and dispatch. See include/vswin.h.
#include <cmath>
#include <vector>

#include "api.h"
#include "sequence.h"

namespace vswin {
namespace {

int elem_bytes(int dtype) { return dtype == kF32 ? 4 : 2; }
const char* const kTypes = "VSWIN_BF16, VSWIN_FP16 or VSWIN_F32";

struct Extent {
  long long B, L, H, d;
};

// Bytes from the first to one past the last element of a view.
size_t view_bytes(const Heads& v, const Extent& e, int esize) {
  return (size_t)((e.B - 1) * v.sb + (e.L - 1) * v.st + (e.H - 1) * v.sh + e.d) * esize;
}

bool same_view(const Heads& a, const Heads& b) {
  return a.p == b.p && a.sb == b.sb && a.st == b.st && a.sh == b.sh;
}

// Whether `from`, moved by some steps (step k at most lo..hi times), comes into
// (-below, above): the largest steps first, which leave few counts to try when the
// smaller ones span less than they do (every view that holds no element twice).
struct Steps {
  int n = 0;
  long long step[6], lo[6], hi[6];
  void add(long long s, long long first, long long last) {
    if (s == 0) return;
    int at = 0;
    while (at < n && step[at] > s) ++at;
    if (at < n && step[at] == s) {
      lo[at] += first, hi[at] += last;
      return;
    }
    for (int k = n++; k > at; --k) step[k] = step[k - 1], lo[k] = lo[k - 1], hi[k] = hi[k - 1];
    step[at] = s, lo[at] = first, hi[at] = last;
  }
  // (`tries` bounds the search; where it ends, the answer is yes)
  bool reach(int k, long long from, long long below, long long above, int* tries) const {
    if (k == n) return from > -below && from < above;
    long long least = 0, most = 0;  // what the smaller steps can add
    for (int j = k + 1; j < n; ++j) least += step[j] * lo[j], most += step[j] * hi[j];
    auto floor_div = [](long long x, long long y) { return x / y - (x % y < 0); };
    long long x = floor_div(-below - from - most, step[k]) + 1;
    long long last = -floor_div(from + least - above, step[k]) - 1;
    if (x < lo[k]) x = lo[k];
    if (last > hi[k]) last = hi[k];
    for (; x <= last; ++x)
      if (--*tries < 0 || reach(k + 1, from + x * step[k], below, above, tries)) return true;
    return false;
  }
};

// Whether two views share an element: slices of one buffer may interleave without.
bool views_overlap(const Heads& a, const Extent& ea, const Heads& b, const Extent& eb, int esize) {
  if (!overlap(a.p, view_bytes(a, ea, esize), b.p, view_bytes(b, eb, esize))) return false;
  Steps steps;
  const long long sa[3] = {a.sb, a.st, a.sh}, na[3] = {ea.B, ea.L, ea.H};
  const long long sb[3] = {b.sb, b.st, b.sh}, nb[3] = {eb.B, eb.L, eb.H};
  for (int k = 0; k < 3; ++k) {
    steps.add(sa[k] * esize, 0, na[k] - 1);
    steps.add(sb[k] * esize, 1 - nb[k], 0);
  }
  int tries = 4096;
  return steps.reach(0, static_cast<const char*>(a.p) - static_cast<const char*>(b.p), ea.d * esize, eb.d * esize, &tries);
}

// A view's pointer, alignment and strides; an output may not hold an element twice.
int check_view(const vswin_heads* v, const char* name, const Extent& e, size_t align, int esize, bool output,
               Heads* out) {
  if (!v) return fail(VSWIN_ERR_INVALID_ARG, "%s is NULL", name);
  if (!v->data) return fail(VSWIN_ERR_INVALID_ARG, "%s has a NULL pointer", name);
  if (!aligned(v->data, align)) return fail(VSWIN_ERR_INVALID_ARG, "%s is not %zu-byte aligned", name, align);
  const long long s[3] = {v->batch_stride, v->token_stride, v->head_stride};
  const long long n[3] = {e.B, e.L, e.H};
  for (int k = 0; k < 3; ++k) {
    if (n[k] > 1 && (s[k] < 0 || s[k] > (1LL << 48) / n[k]))
      return fail(VSWIN_ERR_INVALID_ARG, "%s: stride %lld is negative or too large", name, s[k]);
    if (align > (size_t)esize && n[k] > 1 && (s[k] * esize) % (long long)align)
      return fail(VSWIN_ERR_INVALID_ARG, "%s: strides must be multiples of %zu bytes", name, align);
  }
  *out = Heads{v->data, n[0] > 1 ? s[0] : 0, n[1] > 1 ? s[1] : 0, n[2] > 1 ? s[2] : 0};
  if (output) {  // dimensions by stride: each must step over what the smaller ones span
    int order[3] = {0, 1, 2};
    for (int a = 0; a < 2; ++a)
      for (int b = 0; b < 2 - a; ++b)
        if (s[order[b]] > s[order[b + 1]]) std::swap(order[b], order[b + 1]);
    long long span = e.d;
    for (int k = 0; k < 3; ++k) {
      const int dim = order[k];
      if (n[dim] <= 1) continue;
      if (s[dim] < span) return fail(VSWIN_ERR_INVALID_ARG, "%s: strides make elements of the output overlap", name);
      span = (n[dim] - 1) * s[dim] + span;
    }
  }
  return VSWIN_OK;
}

// Contiguous memory that a call reads beside its views (p may be NULL).
struct Flat {
  const void* p;
  size_t bytes;
};

bool overlaps_any(const void* p, size_t bytes, const Flat* f, int n) {
  for (int k = 0; k < n; ++k)
    if (f[k].p && overlap(p, bytes, f[k].p, f[k].bytes)) return true;
  return false;
}

// The weights, angles and positions of the norm, and what of the bias and the
// visibility is on the device.
constexpr int kNormFlats = 5, kAttnFlats = 5;
void norm_flats(const QkNormArgs& a, int esize, Flat (&f)[kNormFlats]) {
  const size_t gamma = (size_t)a.d * esize, angles = (size_t)a.rows * (a.rot / 2) * 4;
  const bool turns = a.rot > 0;
  f[0] = {a.gamma[0], gamma}, f[1] = {a.gamma[1], gamma};
  f[2] = {turns ? a.cosp : nullptr, angles}, f[3] = {turns ? a.sinp : nullptr, angles};
  f[4] = {turns ? a.positions : nullptr, (size_t)a.B * a.L * 4};
}
void attention_flats(const BiasAttnArgs& a, Flat (&f)[kAttnFlats]) {
  const size_t per_sequence = (size_t)a.B * 4;
  f[0] = {a.table, (size_t)a.buckets * a.hq * 2}, f[1] = {a.map, (2 * (size_t)a.D + 1) * 4};
  f[2] = {a.q_lens, per_sequence}, f[3] = {a.kv_lens, per_sequence}, f[4] = {a.q_start, per_sequence};
}

// Sizes, views, weights and rotation of the norm; `backward` has output
// gradients in y and input gradients in dx.
int check_qk_norm(int dtype, int B, int L, int hq, int hk, int d, const vswin_heads* q, const vswin_heads* k,
                  const void* gq, const void* gk, float eps, const vswin_rotation* r, const vswin_heads* yq,
                  const vswin_heads* yk, const vswin_heads* dq, const vswin_heads* dk, QkNormArgs* a) {
  const bool backward = dq != nullptr || dk != nullptr;
  if (dtype < kBF16 || dtype > kF32) return fail(VSWIN_ERR_INVALID_ARG, "dtype %d is none of %s", dtype, kTypes);
  if (B <= 0 || L <= 0 || hq <= 0 || hk <= 0 || d <= 0)
    return fail(VSWIN_ERR_INVALID_ARG, "sizes must be positive (B=%d L=%d heads=%d,%d d=%d)", B, L, hq, hk, d);
  if (d > 256) return fail(VSWIN_ERR_UNSUPPORTED, "head width %d: the norm supports up to 256", d);
  const long long most = (long long)B * L;
  if (most > (1LL << 31) - (1LL << 20) || hq > (1 << 20) || hk > (1 << 20) || most * hq > (1LL << 40) ||
      most * hk > (1LL << 40))
    return fail(VSWIN_ERR_UNSUPPORTED, "B * L exceeds 2^31 - 2^20, heads 2^20 or rows 2^40");
  if (!(eps >= 0.f) || !std::isfinite(eps))
    return fail(VSWIN_ERR_INVALID_ARG, "eps must be finite and >= 0 (got %g)", (double)eps);
  const int es = elem_bytes(dtype);
  *a = QkNormArgs{};
  a->B = B, a->L = L, a->d = d, a->eps = eps;
  a->heads[0] = hq, a->heads[1] = hk;
  const Extent ext[2] = {{B, L, hq, d}, {B, L, hk, d}};
  const vswin_heads *x[2] = {q, k}, *y[2] = {yq, yk}, *g[2] = {dq, dk};
  const void* gamma[2] = {gq, gk};
  const char* xn[2] = {"q", "k"};
  const char* yn[2] = {backward ? "dq_out" : "q_out", backward ? "dk_out" : "k_out"};
  const char* gn[2] = {"dq", "dk"};
  const char* wn[2] = {"gamma_q", "gamma_k"};
  for (int w = 0; w < 2; ++w) {
    int st = check_view(x[w], xn[w], ext[w], es, es, false, &a->x[w]);
    if (st == VSWIN_OK) st = check_view(y[w], yn[w], ext[w], es, es, !backward, &a->y[w]);
    if (st == VSWIN_OK && backward) st = check_view(g[w], gn[w], ext[w], es, es, true, &a->dx[w]);
    if (st != VSWIN_OK) return st;
    if (!gamma[w] || !aligned(gamma[w], es))
      return fail(VSWIN_ERR_INVALID_ARG, "%s is NULL or not %d-byte aligned", wn[w], es);
    a->gamma[w] = gamma[w];
  }
  // results may replace the input they come from (forward: x; backward: x or dy), and nothing else
  for (int w = 0; w < 2; ++w) {
    const Heads& o = backward ? a->dx[w] : a->y[w];
    const char* on = backward ? gn[w] : yn[w];
    for (int u = 0; u < 2; ++u) {
      const Heads* in[2] = {&a->x[u], backward ? &a->y[u] : nullptr};
      for (const Heads* i : in)
        if (i && !(u == w && same_view(o, *i)) && views_overlap(o, ext[w], *i, ext[u], es))
          return fail(VSWIN_ERR_INVALID_ARG, "%s overlaps an input that it does not replace", on);
    }
  }
  const Heads* out = backward ? a->dx : a->y;
  if (views_overlap(out[0], ext[0], out[1], ext[1], es))
    return fail(VSWIN_ERR_INVALID_ARG, "%s and %s overlap", backward ? "dq" : "q_out", backward ? "dk" : "k_out");
  if (r) {
    if (r->dim < 0 || r->dim > d || r->dim % 2)
      return fail(VSWIN_ERR_INVALID_ARG, "rotation dim %d must be even and within [0, %d]", r->dim, d);
    if (r->dim > 0) {
      if (!r->cos || !r->sin || !aligned(r->cos, 4) || !aligned(r->sin, 4))
        return fail(VSWIN_ERR_INVALID_ARG, "rotation tables must be non-NULL and 4-byte aligned");
      if (r->rows <= 0) return fail(VSWIN_ERR_INVALID_ARG, "rotation rows %d must be positive", r->rows);
      if (!r->positions && r->rows < L)
        return fail(VSWIN_ERR_INVALID_ARG, "rotation tables have %d rows for %d tokens", r->rows, L);
      if (!aligned(r->positions, 4)) return fail(VSWIN_ERR_INVALID_ARG, "positions are not 4-byte aligned");
    }
    a->rot = r->dim;
    a->interleaved = r->interleaved != 0;
    a->cosp = r->cos, a->sinp = r->sin;
    a->positions = r->positions;
    a->rows = r->rows;
  }
  Flat flats[kNormFlats];
  norm_flats(*a, es, flats);
  for (int w = 0; w < 2; ++w)
    if (overlaps_any(out[w].p, view_bytes(out[w], ext[w], es), flats, kNormFlats))
      return fail(VSWIN_ERR_INVALID_ARG, "%s overlaps a gamma, a rotation table or the positions", backward ? gn[w] : yn[w]);
  return VSWIN_OK;
}

int check_bias_attention(int dtype, int B, int Lq, int Lk, int hq, int hk, int d, const vswin_heads* q,
                         const vswin_heads* k, const vswin_heads* v, float scale, const vswin_bucket_bias* bias,
                         const vswin_visibility* vis, const vswin_heads* out, const float* lse, bool out_written,
                         BiasAttnArgs* a) {
  if (dtype != kBF16 && dtype != kFP16)
    return fail(dtype == kF32 ? VSWIN_ERR_UNSUPPORTED : VSWIN_ERR_INVALID_ARG,
                "attention takes VSWIN_BF16 or VSWIN_FP16 (got %d)", dtype);
  if (B <= 0 || Lq <= 0 || Lk <= 0 || hq <= 0 || hk <= 0 || d <= 0)
    return fail(VSWIN_ERR_INVALID_ARG, "sizes must be positive (B=%d Lq=%d Lk=%d heads=%d,%d d=%d)", B, Lq, Lk, hq, hk,
                d);
  if (hq % hk) return fail(VSWIN_ERR_INVALID_ARG, "heads %d of q are not a multiple of the %d of k and v", hq, hk);
  if (d != 32 && d != 64 && d != 128)
    return fail(VSWIN_ERR_UNSUPPORTED, "attention needs head width 32, 64 or 128 (got %d)", d);
  if (Lq > (1 << 28) || Lk > (1 << 28)) return fail(VSWIN_ERR_UNSUPPORTED, "sequence longer than 2^28");
  if (hq > 4096 || (long long)B * hq > (1LL << 28) || (long long)B * hq * ((Lq + 127) / 128) > (1LL << 31) - 1 ||
      (long long)B * hk * ((Lk + 127) / 128) > (1LL << 31) - 1)
    return fail(VSWIN_ERR_UNSUPPORTED, "B * heads * length too large");
  if (!(std::fabs(scale) <= 1e30f)) return fail(VSWIN_ERR_INVALID_ARG, "scale must be finite, at most 1e30 (got %g)", (double)scale);
  *a = BiasAttnArgs{};
  a->B = B, a->Lq = Lq, a->Lk = Lk, a->hq = hq, a->hk = hk, a->d = d;
  a->scale = scale;
  const Extent eq{B, Lq, hq, d}, ek{B, Lk, hk, d};
  int st = check_view(q, "q", eq, 16, 2, false, &a->q);
  if (st == VSWIN_OK) st = check_view(k, "k", ek, 16, 2, false, &a->k);
  if (st == VSWIN_OK) st = check_view(v, "v", ek, 16, 2, false, &a->v);
  if (st == VSWIN_OK) st = check_view(out, "out", eq, 16, 2, out_written, &a->o);
  if (st != VSWIN_OK) return st;
  if (out_written && (views_overlap(a->o, eq, a->q, eq, 2) || views_overlap(a->o, eq, a->k, ek, 2) ||
                      views_overlap(a->o, eq, a->v, ek, 2)))
    return fail(VSWIN_ERR_INVALID_ARG, "out overlaps an input");
  if (!lse || !aligned(lse, 4)) return fail(VSWIN_ERR_INVALID_ARG, "lse is NULL or not 4-byte aligned");
  a->lse = const_cast<float*>(lse);
  if (!bias || !bias->table || !bias->map) return fail(VSWIN_ERR_INVALID_ARG, "bias, its table or its map is NULL");
  if (!aligned(bias->table, 2) || !aligned(bias->map, 4))
    return fail(VSWIN_ERR_INVALID_ARG, "bias table or map is misaligned");
  if (bias->buckets <= 0 || bias->buckets > kMaxBuckets || bias->max_distance < 0 || bias->max_distance > (1 << 20))
    return fail(VSWIN_ERR_INVALID_ARG, "buckets %d must lie in [1, %d] and max_distance %d in [0, 2^20]",
                bias->buckets, kMaxBuckets, bias->max_distance);
  a->table = bias->table, a->map = bias->map, a->buckets = bias->buckets, a->D = bias->max_distance;
  if (vis) {
    if (!aligned(vis->q_lens, 4) || !aligned(vis->kv_lens, 4) || !aligned(vis->q_start, 4))
      return fail(VSWIN_ERR_INVALID_ARG, "lengths or starts are not 4-byte aligned");
    a->q_lens = vis->q_lens, a->kv_lens = vis->kv_lens, a->q_start = vis->q_start;
    a->causal = vis->causal != 0;
  }
  return VSWIN_OK;
}

}  // namespace
}  // namespace vswin

using namespace vswin;

extern "C" {

int vswin_qk_norm_forward(int dtype, int B, int L, int hq, int hk, int d, const vswin_heads* q, const vswin_heads* k,
                          const void* gamma_q, const void* gamma_k, float eps, const vswin_rotation* rotation,
                          const vswin_heads* q_out, const vswin_heads* k_out, void* stream) {
  NvtxRange nvtx_range("vswin_qk_norm_forward");
  QkNormArgs a;
  int st = check_qk_norm(dtype, B, L, hq, hk, d, q, k, gamma_q, gamma_k, eps, rotation, q_out, k_out, nullptr, nullptr, &a);
  if (st != VSWIN_OK) return st;
  KernelCtx ctx;
  st = make_ctx(&ctx);
  if (st != VSWIN_OK) return st;
  a.err = ctx.err;
  const cudaError_t e = launch_qk_norm_forward(a, dtype, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? VSWIN_OK : fail_cuda(e, "head norm launch");
}

int vswin_qk_norm_backward(int dtype, int B, int L, int hq, int hk, int d, const vswin_heads* q, const vswin_heads* k,
                           const void* gamma_q, const void* gamma_k, float eps, const vswin_rotation* rotation,
                           const vswin_heads* dq_out, const vswin_heads* dk_out, const vswin_heads* dq,
                           const vswin_heads* dk, float* dgamma_q, float* dgamma_k, void* stream) {
  NvtxRange nvtx_range("vswin_qk_norm_backward");
  if (!dq || !dk) return fail(VSWIN_ERR_INVALID_ARG, "dq or dk is NULL");
  QkNormArgs a;
  int st = check_qk_norm(dtype, B, L, hq, hk, d, q, k, gamma_q, gamma_k, eps, rotation, dq_out, dk_out, dq, dk, &a);
  if (st != VSWIN_OK) return st;
  float* dg[2] = {dgamma_q, dgamma_k};
  Flat flats[kNormFlats];
  norm_flats(a, elem_bytes(dtype), flats);
  for (int w = 0; w < 2; ++w) {
    if (!dg[w] || !aligned(dg[w], 4)) return fail(VSWIN_ERR_INVALID_ARG, "dgamma is NULL or not 4-byte aligned");
    const size_t n = (size_t)d * 4, es = elem_bytes(dtype);
    for (int u = 0; u < 2; ++u) {
      const Extent e{B, L, u ? hk : hq, d};
      if (overlap(dg[w], n, a.x[u].p, view_bytes(a.x[u], e, es)) || overlap(dg[w], n, a.y[u].p, view_bytes(a.y[u], e, es)) ||
          overlap(dg[w], n, a.dx[u].p, view_bytes(a.dx[u], e, es)) || overlaps_any(dg[w], n, flats, kNormFlats))
        return fail(VSWIN_ERR_INVALID_ARG, "dgamma overlaps another tensor");
    }
    a.dgamma[w] = dg[w];
  }
  if (overlap(dg[0], (size_t)d * 4, dg[1], (size_t)d * 4))
    return fail(VSWIN_ERR_INVALID_ARG, "dgamma_q and dgamma_k overlap");
  KernelCtx ctx;
  st = make_ctx(&ctx);
  if (st != VSWIN_OK) return st;
  a.err = ctx.err;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  void* scratch = nullptr;
  st = scratch_alloc(&scratch, qk_norm_scratch_bytes(a, dtype), s);
  if (st != VSWIN_OK) return st;
  const cudaError_t e = launch_qk_norm_backward(a, dtype, scratch, s);
  const cudaError_t e2 = cudaFreeAsync(scratch, s);
  if (e != cudaSuccess) return fail_cuda(e, "head norm backward launch");
  return e2 == cudaSuccess ? VSWIN_OK : fail_cuda(e2, "cudaFreeAsync");
}

int vswin_bucket_map(int buckets, int max_distance, int bidirectional, int* map) {
  if (!map) return fail(VSWIN_ERR_INVALID_ARG, "map is NULL");
  const int side = bidirectional ? buckets / 2 : buckets;
  const int near_n = side / 2;
  if (near_n < 1 || (bidirectional && buckets % 2) || max_distance <= near_n || max_distance > (1 << 20))
    return fail(VSWIN_ERR_INVALID_ARG,
                "buckets %d leave %d single distances of a side: at least 1 is needed, an even count when bidirectional, "
                "and max_distance %d in (%d, 2^20]",
                buckets, near_n, max_distance, near_n);
  for (int rel = -max_distance; rel <= max_distance; ++rel) {
    const int away = bidirectional ? std::abs(rel) : (rel < 0 ? -rel : 0);
    int b = away;
    if (away >= near_n) {
      // 1e-9: distances that lie on a bucket's edge start that bucket whatever the logarithm's last bit
      const double far = std::log((double)away / near_n) / std::log((double)max_distance / near_n) * (side - near_n);
      b = near_n + (int)std::floor(far + 1e-9);
      if (b > side - 1) b = side - 1;
    }
    map[rel + max_distance] = b + (bidirectional && rel > 0 ? side : 0);
  }
  return VSWIN_OK;
}

int vswin_bias_attention_forward(int dtype, int B, int Lq, int Lk, int hq, int hk, int d, const vswin_heads* q,
                                 const vswin_heads* k, const vswin_heads* v, float scale, const vswin_bucket_bias* bias,
                                 const vswin_visibility* vis, const vswin_heads* out, float* lse, void* stream) {
  NvtxRange nvtx_range("vswin_bias_attention_forward");
  BiasAttnArgs a;
  int st = check_bias_attention(dtype, B, Lq, Lk, hq, hk, d, q, k, v, scale, bias, vis, out, lse, true, &a);
  if (st != VSWIN_OK) return st;
  const size_t lse_n = (size_t)B * hq * Lq * 4;
  const Extent eq{B, Lq, hq, d}, ek{B, Lk, hk, d};
  if (overlap(lse, lse_n, a.o.p, view_bytes(a.o, eq, 2)) || overlap(lse, lse_n, a.q.p, view_bytes(a.q, eq, 2)) ||
      overlap(lse, lse_n, a.k.p, view_bytes(a.k, ek, 2)) || overlap(lse, lse_n, a.v.p, view_bytes(a.v, ek, 2)))
    return fail(VSWIN_ERR_INVALID_ARG, "lse overlaps another tensor");
  Flat flats[kAttnFlats];
  attention_flats(a, flats);
  if (overlaps_any(a.o.p, view_bytes(a.o, eq, 2), flats, kAttnFlats) || overlaps_any(lse, lse_n, flats, kAttnFlats))
    return fail(VSWIN_ERR_INVALID_ARG, "out or lse overlaps the bias table, its map, lengths or starts");
  st = make_ctx(&a.ctx);
  if (st != VSWIN_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const size_t bytes = bias_attention_scratch_bytes(a);
  void* scratch = nullptr;
  if (bytes) {
    st = scratch_alloc(&scratch, bytes, s);
    if (st != VSWIN_OK) return st;
  }
  const cudaError_t e = launch_bias_attention(a, dtype, scratch, s);
  const cudaError_t e2 = scratch ? cudaFreeAsync(scratch, s) : cudaSuccess;
  if (e != cudaSuccess) return fail_cuda(e, "attention launch");
  return e2 == cudaSuccess ? VSWIN_OK : fail_cuda(e2, "cudaFreeAsync");
}

int vswin_bias_attention_backward(int dtype, int B, int Lq, int Lk, int hq, int hk, int d, const vswin_heads* q,
                                  const vswin_heads* k, const vswin_heads* v, float scale,
                                  const vswin_bucket_bias* bias, const vswin_visibility* vis, const vswin_heads* out,
                                  const float* lse, const vswin_heads* dout, const vswin_heads* dq,
                                  const vswin_heads* dk, const vswin_heads* dv, void* dtable, void* stream) {
  NvtxRange nvtx_range("vswin_bias_attention_backward");
  BiasAttnArgs a;
  int st = check_bias_attention(dtype, B, Lq, Lk, hq, hk, d, q, k, v, scale, bias, vis, out, lse, false, &a);
  if (st != VSWIN_OK) return st;
  const Extent eq{B, Lq, hq, d}, ek{B, Lk, hk, d};
  st = check_view(dout, "dout", eq, 16, 2, false, &a.dout);
  if (st == VSWIN_OK) st = check_view(dq, "dq", eq, 16, 2, true, &a.dq);
  if (st == VSWIN_OK) st = check_view(dk, "dk", ek, 16, 2, true, &a.dk);
  if (st == VSWIN_OK) st = check_view(dv, "dv", ek, 16, 2, true, &a.dv);
  if (st != VSWIN_OK) return st;
  if (!dtable || !aligned(dtable, 2)) return fail(VSWIN_ERR_INVALID_ARG, "dtable is NULL or not 2-byte aligned");
  a.dtable = dtable;
  const size_t tb = (size_t)a.buckets * hq * 2, lse_n = (size_t)B * hq * Lq * 4;
  const Heads* ins[] = {&a.q, &a.k, &a.v, &a.o, &a.dout};
  const Extent in_e[] = {eq, ek, ek, eq, eq};
  const Heads* outs[] = {&a.dq, &a.dk, &a.dv};
  const Extent out_e[] = {eq, ek, ek};
  const char* names[] = {"dq", "dk", "dv"};
  Flat flats[kAttnFlats];
  attention_flats(a, flats);
  for (int o = 0; o < 3; ++o) {
    const size_t n = view_bytes(*outs[o], out_e[o], 2);
    for (int i = 0; i < 5; ++i)
      if (views_overlap(*outs[o], out_e[o], *ins[i], in_e[i], 2))
        return fail(VSWIN_ERR_INVALID_ARG, "%s overlaps an input", names[o]);
    if (overlap(outs[o]->p, n, lse, lse_n) || overlap(outs[o]->p, n, dtable, tb) || overlaps_any(outs[o]->p, n, flats, kAttnFlats))
      return fail(VSWIN_ERR_INVALID_ARG, "%s overlaps lse, the bias table, its gradient or map, lengths or starts", names[o]);
    if (views_overlap(*outs[o], out_e[o], *outs[(o + 1) % 3], out_e[(o + 1) % 3], 2))
      return fail(VSWIN_ERR_INVALID_ARG, "%s and %s overlap", names[o], names[(o + 1) % 3]);
  }
  for (int i = 0; i < 5; ++i)
    if (overlap(dtable, tb, ins[i]->p, view_bytes(*ins[i], in_e[i], 2)))
      return fail(VSWIN_ERR_INVALID_ARG, "dtable overlaps an input");
  if (overlap(dtable, tb, lse, lse_n) || overlaps_any(dtable, tb, flats, kAttnFlats))
    return fail(VSWIN_ERR_INVALID_ARG, "dtable overlaps lse, the table, its map, lengths or starts");
  st = make_ctx(&a.ctx);
  if (st != VSWIN_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  void* scratch = nullptr;
  st = scratch_alloc(&scratch, bias_attention_backward_scratch_bytes(a), s);
  if (st != VSWIN_OK) return st;
  const cudaError_t e = launch_bias_attention_backward(a, dtype, scratch, s);
  const cudaError_t e2 = cudaFreeAsync(scratch, s);
  if (e != cudaSuccess) return fail_cuda(e, "attention backward launch");
  return e2 == cudaSuccess ? VSWIN_OK : fail_cuda(e2, "cudaFreeAsync");
}

int vswin_adamw_step(const vswin_adamw_tensor* tensors, int count, int bits, double lr, double beta1, double beta2,
                     double eps, long long step, const int* step_device, const float* grad_scale, void* stream) {
  NvtxRange nvtx_range("vswin_adamw_step");
  if (count < 0 || (count > 0 && !tensors)) return fail(VSWIN_ERR_INVALID_ARG, "tensors is NULL or count=%d negative", count);
  if (bits != 32 && bits != 8) return fail(VSWIN_ERR_INVALID_ARG, "bits must be 32 or 8 (got %d)", bits);
  if (!(lr >= 0) || !std::isfinite(lr) || !(beta1 >= 0 && beta1 < 1) || !(beta2 >= 0 && beta2 < 1) || !(eps >= 0) ||
      !std::isfinite(eps))
    return fail(VSWIN_ERR_INVALID_ARG, "lr and eps must be finite and >= 0, betas in [0, 1) (lr=%g betas=%g,%g eps=%g)",
                lr, beta1, beta2, eps);
  if (!step_device && step < 1) return fail(VSWIN_ERR_INVALID_ARG, "step %lld must be at least 1", step);
  if (!aligned(step_device, 4) || !aligned(grad_scale, 4))
    return fail(VSWIN_ERR_INVALID_ARG, "step_device or grad_scale is not 4-byte aligned");
  std::vector<AdamwTensor> list;
  try {
    list.reserve(count);
  } catch (...) {
    return fail(VSWIN_ERR_NO_MEMORY, "no host memory for a list of %d tensors", count);
  }
  for (int i = 0; i < count; ++i) {
    const vswin_adamw_tensor& t = tensors[i];
    if (t.n < 0 || t.n > (1LL << 40)) return fail(VSWIN_ERR_INVALID_ARG, "tensor %d: n=%lld", i, t.n);
    if (t.n == 0) continue;
    if (t.param_dtype < kBF16 || t.param_dtype > kF32 || t.grad_dtype < kBF16 || t.grad_dtype > kF32)
      return fail(VSWIN_ERR_INVALID_ARG, "tensor %d: types must be %s", i, kTypes);
    const size_t pe = elem_bytes(t.param_dtype), ge = elem_bytes(t.grad_dtype), se = bits == 32 ? 4 : 1;
    const void* ptr[] = {t.param, t.grad, t.m, t.v, t.m_scale, t.v_scale, t.master};
    const size_t size[] = {pe, ge, se, se, 4, 4, 4};
    const char* name[] = {"param", "grad", "m", "v", "m_scale", "v_scale", "master"};
    const size_t blocks = (size_t)(t.n + kAdamwBlock - 1) / kAdamwBlock;
    const size_t bytes[] = {t.n * pe, t.n * ge, t.n * se, t.n * se, blocks * 4, blocks * 4, (size_t)t.n * 4};
    bool used[7];
    for (int k = 0; k < 7; ++k) {
      used[k] = k < 4 || (k < 6 ? bits == 8 : t.master != nullptr);
      if (used[k] && (!ptr[k] || !aligned(ptr[k], size[k])))
        return fail(VSWIN_ERR_INVALID_ARG, "tensor %d: %s is NULL or not %zu-byte aligned", i, name[k], size[k]);
    }
    for (int k = 0; k < 7; ++k)
      for (int u = k + 1; u < 7; ++u)
        if (used[k] && used[u] && overlap(ptr[k], bytes[k], ptr[u], bytes[u]))
          return fail(VSWIN_ERR_INVALID_ARG, "tensor %d: %s and %s overlap", i, name[k], name[u]);
    if (!std::isfinite(t.weight_decay) || t.weight_decay < 0)
      return fail(VSWIN_ERR_INVALID_ARG, "tensor %d: weight_decay must be finite and >= 0", i);
    AdamwTensor o{t.param, t.master, t.grad, t.m, t.v, bits == 8 ? t.m_scale : nullptr, bits == 8 ? t.v_scale : nullptr,
                  t.n, (float)(1.0 - lr * t.weight_decay), t.param_dtype, t.grad_dtype, 1};
    for (int k = 0; k < 7; ++k)
      if (k != 4 && k != 5 && used[k] && !aligned(ptr[k], 16)) o.vec = 0;
    list.push_back(o);
  }
  AdamwHyper h{};
  h.b1 = (float)beta1, h.c1 = (float)(1 - beta1), h.b2 = (float)beta2, h.c2 = (float)(1 - beta2), h.eps = (float)eps;
  h.lr = lr, h.beta1 = beta1, h.beta2 = beta2;
  if (!step_device) {
    h.step_size = (float)(lr / (1 - std::pow(beta1, (double)step)));
    h.inv_sqrt_bc2 = (float)(1 / std::sqrt(1 - std::pow(beta2, (double)step)));
  }
  h.step_dev = step_device;
  h.grad_scale = grad_scale;
  KernelCtx ctx;
  const int st = make_ctx(&ctx);
  if (st != VSWIN_OK) return st;
  const cudaError_t e = launch_adamw(list.data(), (int)list.size(), bits, h, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? VSWIN_OK : fail_cuda(e, "optimizer step launch");
}

int vswin_adamw_decode(const void* m, const float* m_scale, const void* v, const float* v_scale, long long n,
                       int out_dtype, void* m_out, void* v_out, void* stream) {
  NvtxRange nvtx_range("vswin_adamw_decode");
  if (n < 0 || n > (1LL << 40)) return fail(VSWIN_ERR_INVALID_ARG, "n=%lld", n);
  if (n == 0) return VSWIN_OK;
  if (out_dtype < kBF16 || out_dtype > kF32) return fail(VSWIN_ERR_INVALID_ARG, "dtype %d is none of %s", out_dtype, kTypes);
  const size_t es = elem_bytes(out_dtype), blocks = (size_t)(n + kAdamwBlock - 1) / kAdamwBlock;
  const void* ptr[] = {m, m_scale, v, v_scale, m_out, v_out};
  const size_t size[] = {1, 4, 1, 4, es, es};
  const size_t bytes[] = {(size_t)n, blocks * 4, (size_t)n, blocks * 4, n * es, n * es};
  const char* name[] = {"m", "m_scale", "v", "v_scale", "m_out", "v_out"};
  for (int k = 0; k < 6; ++k) {
    if (!ptr[k] || !aligned(ptr[k], size[k]))
      return fail(VSWIN_ERR_INVALID_ARG, "%s is NULL or not %zu-byte aligned", name[k], size[k]);
    for (int u = 4; u < 6; ++u)
      if (k < u && overlap(ptr[k], bytes[k], ptr[u], bytes[u]))
        return fail(VSWIN_ERR_INVALID_ARG, "%s and %s overlap", name[k], name[u]);
  }
  KernelCtx ctx;
  const int st = make_ctx(&ctx);
  if (st != VSWIN_OK) return st;
  const cudaError_t e = launch_adamw_decode(static_cast<const int8_t*>(m), m_scale, static_cast<const uint8_t*>(v),
                                            v_scale, n, out_dtype, m_out, v_out, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? VSWIN_OK : fail_cuda(e, "moment decoding launch");
}

}  // extern "C"
