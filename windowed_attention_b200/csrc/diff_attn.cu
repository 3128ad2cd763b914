// Entry points of differential attention: argument checks, the geometry that
// the kernels read, workspace sizes.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstdio>
#include <initializer_list>

#include "diff_attn.cuh"

namespace rib {
namespace {

rib_status bad(const char* who, rib_status st, const char* what) {
  char buf[200];
  std::snprintf(buf, sizeof(buf), "%s: %s", who, what);
  return fail(st, buf);
}

// The strides of a tensor [batch][tokens][heads][e]; all zero means contiguous.
struct Strides { long long b, t, h; };
Strides strides(const long long (&s)[3], long long tokens, int heads, int e) {
  if (!s[0] && !s[1] && !s[2]) return {tokens * heads * e, static_cast<long long>(heads) * e, e};
  return {s[0], s[1], s[2]};
}
// The kernels' form of them; token and head strides are ints there.
rib_status narrow(const char* who, const Strides& s, const long long (&n)[3], int rows, DiffStrides* out) {
  if (s.b < 0 || s.t < 0 || s.h < 0 || s.b % 8 || s.t % 8 || s.h % 8)
    return bad(who, RIB_ERR_ALIGNMENT, "strides must be non-negative multiples of 8 elements");
  // a tensor map holds strides below 2^40 bytes (a map's row: width tokens)
  if (s.t > 0x7FFFFFFF || s.h > 0x7FFFFFFF || s.b >= (1ll << 39) || s.t * rows >= (1ll << 39))
    return bad(who, RIB_ERR_UNSUPPORTED, "token or head stride of 2^31 elements, or batch stride of 2^39, or more");
  // an axis that is stepped along needs a stride of its own
  if (n[0] > 0 && n[1] > 0 && ((n[0] > 1 && s.b == 0) || (n[1] > 1 && s.t == 0) || (n[2] > 1 && s.h == 0)))
    return bad(who, RIB_ERR_UNSUPPORTED, "a stride of 0 (a broadcast tensor): give its one copy as an axis of length 1");
  *out = {s.b, static_cast<int>(s.t), static_cast<int>(s.h)};
  return RIB_OK;
}
// Written tensors may not lay two values on one place: the head stride holds a
// row of e, the token stride a token's heads and the batch stride an item.
bool overlaps(const DiffStrides& s, int batch, long long tokens, int heads, int e) {
  if (batch == 0 || tokens == 0) return false;
  struct Axis { long long n, st; } ax[3] = {{heads, s.h}, {tokens, s.t}, {batch, s.b}};
  for (int i = 0; i < 3; ++i)
    for (int j = i + 1; j < 3; ++j)
      if (ax[j].st < ax[i].st) { const Axis x = ax[i]; ax[i] = ax[j]; ax[j] = x; }
  long long reach = e;   // values from the first to behind the last of the axes so far
  for (const Axis& x : ax) {
    if (x.n <= 1) continue;
    if (x.st < reach) return true;
    reach += (x.n - 1) * x.st;
  }
  return false;
}

// Boxes of 64 rows. In a window: the power of two of columns that takes the
// fewest boxes (the widest of them: longer runs of memory).
void boxes(DiffGeom* g) {
  const int tokens = 64 / g->group;
  if (!g->window) {
    g->tck = 64; g->lk = 6; g->trk = 1;
    g->tcq = tokens; g->lq = 31; g->trq = 1;
    return;
  }
  const int w = diff_span_x(*g, 0), h = diff_span_y(*g);
  auto pick = [&](int n, int* tc, int* l, int* tr) {
    int top = 0;
    while ((2 << top) <= n) ++top;   // the largest power of two within n
    long long best = -1;
    for (int i = 0; i <= top; ++i) {
      const int c = 1 << i, r = 1 << (top - i);
      const long long count = static_cast<long long>(ceil_div(w, c)) * ceil_div(h > 0 ? h : 1, r);
      if (best < 0 || count <= best) {
        best = count;
        *tc = c; *l = i; *tr = r;
      }
    }
  };
  pick(64, &g->tck, &g->lk, &g->trk);
  pick(tokens, &g->tcq, &g->lq, &g->trq);
}

rib_status geometry(const char* who, const rib_diff_attn_desc* d, DiffGeom* g) {
  if (!d) return bad(who, RIB_ERR_INVALID_ARG, "null descriptor");
  if (d->batch < 0 || d->q_len < 0 || d->k_len < 0 || d->q_heads <= 0 || d->kv_heads <= 0 || d->d <= 0 || d->dv <= 0)
    return bad(who, RIB_ERR_INVALID_ARG, "sizes: batch and lengths >= 0, heads and widths positive");
  if (d->q_heads % d->kv_heads) return bad(who, RIB_ERR_INVALID_ARG, "q_heads must be a multiple of kv_heads");
  // the kernels' exponents are powers of two
  if (!(d->scale > 0.f) || !std::isfinite(d->scale * kDiffLog2e)) return bad(who, RIB_ERR_INVALID_ARG, "scale must be positive and below 2.3e38");
  if (d->dtype != RIB_BF16 && d->dtype != RIB_F16) return bad(who, RIB_ERR_INVALID_ARG, "dtype must be RIB_BF16 or RIB_F16");
  if (d->lam_dtype != RIB_F32 && d->lam_dtype != d->dtype)
    return bad(who, RIB_ERR_INVALID_ARG, "lam_dtype must be RIB_F32 or dtype");
  if (d->d % 8 || d->dv % 8 || d->d > 64 || d->dv > 128) return bad(who, RIB_ERR_UNSUPPORTED, "needs d <= 64 and dv <= 128, multiples of 8");
  if (d->window < 0 || d->width < 0 || (d->window > 0) != (d->width > 0))
    return bad(who, RIB_ERR_INVALID_ARG, "window and width go together");
  if (d->window > 0) {
    if (d->q_len != d->k_len || d->q_len % d->width) return bad(who, RIB_ERR_INVALID_ARG, "a map has q_len = k_len = height * width");
    if (d->causal) return bad(who, RIB_ERR_INVALID_ARG, "windows have no causal mask");
    if (d->window > 1024) return bad(who, RIB_ERR_UNSUPPORTED, "window above 1024");
  }
  *g = DiffGeom{};
  g->batch = d->batch; g->q_len = d->q_len; g->k_len = d->k_len; g->q_heads = d->q_heads; g->kv_heads = d->kv_heads;
  g->group = d->q_heads / d->kv_heads;
  g->d = d->d; g->dv = d->dv;
  g->window = d->window; g->width = d->width; g->causal = d->causal != 0; g->lam_f32 = d->lam_dtype == RIB_F32;
  if (d->window > 0) {
    g->height = d->q_len / d->width;
    g->nwx = (d->width - 1) / d->window + 1;
    g->nwy = g->height > 0 ? (g->height - 1) / d->window + 1 : 0;
  }
  g->group_magic = div_magic(static_cast<uint32_t>(g->group));
  g->scale = d->scale;
  g->scale_log2 = d->scale * kDiffLog2e;
  rib_status st = RIB_OK;
  if ((st = narrow(who, strides(d->q_stride, d->q_len, d->q_heads, d->d), {d->batch, d->q_len, d->q_heads}, d->window ? d->width : 1, &g->q)) != RIB_OK ||
      (st = narrow(who, strides(d->k_stride, d->k_len, d->kv_heads, d->d), {d->batch, d->k_len, d->kv_heads}, d->window ? d->width : 1, &g->k)) != RIB_OK ||
      (st = narrow(who, strides(d->v_stride, d->k_len, d->kv_heads, d->dv), {d->batch, d->k_len, d->kv_heads}, d->window ? d->width : 1, &g->v)) != RIB_OK ||
      (st = narrow(who, strides(d->o_stride, d->q_len, d->q_heads, d->dv), {d->batch, d->q_len, d->q_heads}, d->window ? d->width : 1, &g->o)) != RIB_OK)
    return st;
  if (g->group > 64) return bad(who, RIB_ERR_UNSUPPORTED, "more than 64 query heads a key head");
  // coordinates and tokens are ints, with a box behind the last
  if (d->q_len > 0x7FFFFFFF - 256 || d->k_len > 0x7FFFFFFF - 256) return bad(who, RIB_ERR_UNSUPPORTED, "sequences too long");
  boxes(g);
  // units of work are ints: (sequences, key heads, tiles, splits)
  const long long seqs = static_cast<long long>(d->batch) * (d->window ? static_cast<long long>(g->nwx) * g->nwy : 1);
  const long long bq = diff_max_q_boxes(*g), bk = diff_max_k_boxes(*g), tiles = (bq > bk ? bq : bk) + 64;
  if (seqs > 0x7FFFFFFFll / d->kv_heads || seqs * d->kv_heads > 0x3FFFFFFFll / tiles)
    return bad(who, RIB_ERR_UNSUPPORTED, "too many sequences and heads");
  if (overlaps(g->o, d->batch, d->q_len, d->q_heads, d->dv)) return bad(who, RIB_ERR_INVALID_ARG, "o_stride lays values of o on one another");
  return RIB_OK;
}

bool misaligned(std::initializer_list<const void*> ps, uintptr_t to) {
  for (const void* p : ps)
    if (reinterpret_cast<uintptr_t>(p) % to) return true;
  return false;
}

// The backward's row constants hold lse / scale in three 16-bit terms; below
// these scales the log-sum-exp of 2^31 equal keys alone leaves their range.
float least_bwd_scale(const rib_diff_attn_desc* d) { return d->dtype == RIB_F16 ? 0x1p-26f : 0x1p-100f; }

uintptr_t lam_size(const rib_diff_attn_desc* d) { return d->lam_dtype == RIB_F32 ? 4 : 2; }

// Query boxes of one (sequence, key head) in the backward's row constants: whole tiles of two.
int row_boxes(const DiffGeom& g) { return ceil_div(diff_max_q_boxes(g), 2) * 2; }
size_t row_bytes(const DiffGeom& g) {
  return static_cast<size_t>(diff_sequences(g)) * g.kv_heads * row_boxes(g) * DiffRows::kBytes;
}

}  // namespace
}  // namespace rib

using namespace rib;

extern "C" {

size_t rib_diff_attention_workspace_size(const rib_diff_attn_desc* d) {
  DiffGeom g;
  return geometry("rib_diff_attention_workspace_size", d, &g) == RIB_OK ? diff_split_bytes(g) : 0;
}

rib_status rib_diff_attention(const rib_diff_attn_desc* d, const void* q1, const void* q2, const void* k1, const void* k2, const void* v,
                              const void* lam, const int* k_lens, void* o, void* o2, float* lse, void* ws, size_t ws_bytes,
                              cudaStream_t stream) {
  const char* who = "rib_diff_attention";
  DiffFwdArgs a{};
  rib_status st = geometry(who, d, &a.g);
  if (st != RIB_OK) return st;
  if (d->batch == 0 || d->q_len == 0) return RIB_OK;   // no rows: nothing is written
  const bool keys = d->k_len > 0;                      // empty tensors may have null pointers
  if (!q1 || !q2 || !lam || !o || (keys && (!k1 || !k2 || !v))) return bad(who, RIB_ERR_INVALID_ARG, "null pointer");
  if (k_lens && d->window) return bad(who, RIB_ERR_INVALID_ARG, "windows have no key lengths");
  if (misaligned({q1, q2, k1, k2, v, o, o2, ws}, 16) || misaligned({lse, k_lens}, 4) || misaligned({lam}, lam_size(d)))
    return bad(who, RIB_ERR_ALIGNMENT, "tensors and workspace need 16 bytes, lam, lse and k_lens their element's");
  a.splits = diff_splits(a.g);
  if (a.splits > 1) {
    if (!ws || ws_bytes < diff_split_bytes(a.g)) return bad(who, RIB_ERR_INVALID_ARG, "workspace missing or too small");
    a.part = static_cast<float*>(ws);
    if (diff_few_rows(a.g)) {
      a.quad = 1;
      a.g.tcq = 32 / a.g.group;   // the rows of one lane quarter
    }
  }
  a.g.k_lens = k_lens;
  a.q1 = q1; a.q2 = q2; a.k1 = k1; a.k2 = k2; a.v = v; a.lam = lam;
  a.o = o; a.o2 = o2; a.lse = lse;
  if (!(a.err = device_error_word())) return bad(who, RIB_ERR_CUDA, "no device error word");
  const cudaError_t e = launch_diff_attn_fwd(a, d->dtype == RIB_F16, stream);
  if (e != cudaSuccess) return cuda_fail(e, "rib_diff_attention launch");
  return RIB_OK;
}

size_t rib_diff_attention_bwd_workspace_size(const rib_diff_attn_desc* d) {
  DiffGeom g;
  return geometry("rib_diff_attention_bwd_workspace_size", d, &g) == RIB_OK ? row_bytes(g) + diff_bwd_part_bytes(g) : 0;
}

rib_status rib_diff_attention_bwd(const rib_diff_attn_desc* d, const void* q1, const void* q2, const void* k1, const void* k2, const void* v,
                                  const void* lam, const int* k_lens, const void* o, const void* o2, const float* lse, const void* dO,
                                  void* dq1, void* dq2, void* dk1, void* dk2, void* dv, void* dlam, void* ws, size_t ws_bytes,
                                  cudaStream_t stream) {
  const char* who = "rib_diff_attention_bwd";
  DiffBwdArgs a{};
  rib_status st = geometry(who, d, &a.g);
  if (st != RIB_OK) return st;
  const DiffGeom& g = a.g;
  if (d->scale < least_bwd_scale(d)) return bad(who, RIB_ERR_UNSUPPORTED, "scale below 2^-26 (fp16) or 2^-100 (bf16)");
  const bool rows = d->batch > 0 && d->q_len > 0, keys = d->batch > 0 && d->k_len > 0;
  if (!lam || !dlam || (rows && (!q1 || !q2 || !o || !o2 || !lse || !dO || !dq1 || !dq2)) ||
      (keys && (!k1 || !k2 || !v || !dk1 || !dk2 || !dv)))
    return bad(who, RIB_ERR_INVALID_ARG, "null pointer");
  if (k_lens && d->window) return bad(who, RIB_ERR_INVALID_ARG, "windows have no key lengths");
  if (misaligned({q1, q2, k1, k2, v, o, o2, dO, dq1, dq2, dk1, dk2, dv, ws}, 16) || misaligned({lse, k_lens}, 4) ||
      misaligned({lam, dlam}, lam_size(d)))
    return bad(who, RIB_ERR_ALIGNMENT, "tensors and workspace need 16 bytes, lam, dlam, lse and k_lens their element's");
  if (overlaps(g.q, d->batch, d->q_len, d->q_heads, d->d) || overlaps(g.k, d->batch, d->k_len, d->kv_heads, d->d) ||
      overlaps(g.v, d->batch, d->k_len, d->kv_heads, d->dv))
    return bad(who, RIB_ERR_INVALID_ARG, "strides lay gradients on one another");
  a.boxes = row_boxes(g);
  if (rows && (!ws || ws_bytes < row_bytes(g) + diff_bwd_part_bytes(g))) return bad(who, RIB_ERR_INVALID_ARG, "workspace missing or too small");
  a.rows = static_cast<uint8_t*>(ws);
  a.splits = rows ? diff_bwd_splits(g) : 1;
  a.part = a.splits > 1 ? reinterpret_cast<float*>(a.rows + row_bytes(g)) : nullptr;
  a.g.k_lens = k_lens;
  a.q1 = q1; a.q2 = q2; a.k1 = k1; a.k2 = k2; a.v = v; a.lam = lam; a.o = o; a.o2 = o2; a.lse = lse; a.dO = dO;
  a.dq1 = dq1; a.dq2 = dq2; a.dk1 = dk1; a.dk2 = dk2; a.dv = dv; a.dlam = dlam;
  if (!(a.err = device_error_word())) return bad(who, RIB_ERR_CUDA, "no device error word");
  const cudaError_t e = launch_diff_attn_bwd(a, d->dtype == RIB_F16, stream);
  if (e != cudaSuccess) return cuda_fail(e, "rib_diff_attention_bwd launch");
  return RIB_OK;
}

}  // extern "C"
