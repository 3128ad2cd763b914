// The join of a block with its residual stream, forward and backward
// (rib_residual_norm, rib_residual_norm_bwd):
//   u  = N_post(y) post_w + post_b        (y itself without a post norm)
//   x' = x + m * scale[group] * gate * u  (m the dropout factor, 0 or 1/keep)
//   h  = N_pre(x') pre_w + pre_b
// with N(v) = (v - mean) / sqrt(var + eps) (LayerNorm, biased variance) or
// v / sqrt(mean(v^2) + eps) (RMSNorm). With t the gradient at N's output
// times its weight and v^ = N(v), the gradient at v is
//   r (t - [LayerNorm] mean(t) - v^ mean(t v^)),   r = 1 / sqrt(var + eps),
// so with dx' the whole gradient at x' (the stream's plus N_pre's):
//   dx = dx',  f = m * scale,  dgate = dx' f u,  dscale = sum dx' m gate u,
//   du = dx' f gate,  dpost_w = sum du y^,  dpost_b = sum du, dy from du post_w,
//   dpre_w = sum dh x'^,  dpre_b = sum dh.
//
// What bounds both: memory. Each tensor is read or written once: a row lives
// in the registers of a group of `lpr` threads (a power of two from 4 to 512,
// each thread NV vectors of V elements), statistics are two passes over those
// registers (mean, then squared deviations: no cancellation), and the backward
// recomputes them from x' and y rather than reading saved ones.
//
// Column sums (weights, scale) of the backward: every thread keeps its own
// columns' sums in fp32 registers over the rows that its group walks; the
// groups of a CTA are added through shared memory and one partial row per CTA
// goes to the workspace; a second kernel adds the partials in their order. No
// atomics: the same bits on every run.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstdio>
#include <type_traits>

#include "philox.cuh"
#include "rib_internal.h"
#include "sm100.cuh"

namespace rib {

bool make_drop_rng(float p, uint64_t seed, uint64_t offset, const uint64_t* step, DropRng* rng);

namespace {

constexpr int kMaxC = 4096;
constexpr int kMaxGroups = 1024;
constexpr int kSums = 5;   // dscale, dpost_w, dpost_b, dpre_w, dpre_b

struct NormParams {
  long long T, rows_per_group;
  int C, pre, post;         // norm kinds: 0 none, 1 LayerNorm, 2 RMSNorm
  float eps, inv_c;
  const void *x, *y, *gate; // backward: x is x'
  const float *scale, *post_w, *post_b, *pre_w, *pre_b;
  void *x_out, *h;
  DropRng rng;
  // backward
  const void *dx_out, *dh;
  void *dx, *dy, *dgate;
  float* partial;           // [CTAs][kSums][C]
  int chunks;               // CTAs of a group
};

// V consecutive elements as fp32.
template <typename T, int V>
__device__ __forceinline__ void load_v(const void* base, size_t at, float (&f)[V]) {
  const T* p = static_cast<const T*>(base) + at;
  if constexpr (sizeof(T) == 4) {
    if constexpr (V == 4) {
      const float4 v = *reinterpret_cast<const float4*>(p);
      f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
    } else {
      f[0] = *reinterpret_cast<const float*>(p);
    }
  } else {
    constexpr bool kHalf = std::is_same<T, __half>::value;
    if constexpr (V == 4) {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      f[0] = kHalf ? f16_lo(v.x) : bf16_lo(v.x);
      f[1] = kHalf ? f16_hi(v.x) : bf16_hi(v.x);
      f[2] = kHalf ? f16_lo(v.y) : bf16_lo(v.y);
      f[3] = kHalf ? f16_hi(v.y) : bf16_hi(v.y);
    } else {
      const uint32_t v = *reinterpret_cast<const uint16_t*>(p);
      f[0] = kHalf ? f16_lo(v) : bf16_lo(v);
    }
  }
}
// SAT: fp16 results beyond +-65504 saturate, as in every forward store of the
// library. Gradients do not: an overflow has to stay visible to loss scaling.
template <typename T, int V, bool SAT>
__device__ __forceinline__ void store_v(void* base, size_t at, const float (&f)[V]) {
  T* p = static_cast<T*>(base) + at;
  if constexpr (sizeof(T) == 4) {
    if constexpr (V == 4) *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
    else *reinterpret_cast<float*>(p) = f[0];
  } else {
    constexpr bool kHalf = std::is_same<T, __half>::value;
    auto pack = [](float a, float b) {
      if constexpr (!kHalf) {
        return pack_bf16x2(a, b);
      } else if constexpr (SAT) {
        return pack_f16x2_sat(a, b);
      } else {
        const __half2 v = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&v);
      }
    };
    if constexpr (V == 4) *reinterpret_cast<uint2*>(p) = make_uint2(pack(f[0], f[1]), pack(f[2], f[3]));
    else *reinterpret_cast<uint16_t*>(p) = static_cast<uint16_t>(pack(f[0], 0.f));
  }
}

// Sums of N values over the lpr threads of a row. WIDE rows span warps: their
// warp sums meet in shared memory, two buffers in turn, so one barrier a sum
// is enough (a thread past the barrier of sum k + 1 knows that every thread
// has read the buffer of sum k). Every thread of the CTA calls it.
template <int N, bool WIDE>
__device__ __forceinline__ void row_sum(float (&v)[N], int lpr, float (*red)[2][32], int& phase) {
  const int w = WIDE ? 32 : lpr;
  for (int o = w >> 1; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xFFFFFFFFu, v[i], o);
  if constexpr (WIDE) {
    const int warp = threadIdx.x >> 5, per = lpr >> 5, first = warp / per * per;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) red[phase][i][warp] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float s = 0.f;
      for (int k = 0; k < per; ++k) s += red[phase][i][first + k];
      v[i] = s;
    }
    phase ^= 1;
  }
}

// The dropout factor of V elements from flat element `at` (V == 4: at % 4 == 0).
template <int V>
__device__ __forceinline__ void drop_factor(const DropRng& rng, uint64_t stream, uint64_t at, float (&m)[V]) {
  const uint4 w = philox4x32_10(at >> 3, stream, rng.seed);
  if constexpr (V == 4) {
    const bool high = (at & 4) != 0;
    const uint32_t a = high ? w.z : w.x, b = high ? w.w : w.y;
    m[0] = (a & 0xFFFFu) >= rng.threshold ? rng.up : 0.f;
    m[1] = (a >> 16) >= rng.threshold ? rng.up : 0.f;
    m[2] = (b & 0xFFFFu) >= rng.threshold ? rng.up : 0.f;
    m[3] = (b >> 16) >= rng.threshold ? rng.up : 0.f;
  } else {
    const uint32_t s = static_cast<uint32_t>(at & 7);
    const uint32_t v = s < 4 ? (s < 2 ? w.x : w.y) : (s < 6 ? w.z : w.w);
    m[0] = ((s & 1) ? v >> 16 : v & 0xFFFFu) >= rng.threshold ? rng.up : 0.f;
  }
}

// v := (v - mean) * r in place; returns r. Elements behind the row's end stay 0.
template <int V, int NV, bool WIDE>
__device__ __forceinline__ float normalise(float (&v)[NV][V], const bool (&in)[NV], int kind, const NormParams& p, int lpr,
                                           float (*red)[2][32], int& phase) {
  float s[1];
  if (kind == 1) {
    s[0] = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int e = 0; e < V; ++e) s[0] += v[k][e];
    row_sum<1, WIDE>(s, lpr, red, phase);
    const float mean = s[0] * p.inv_c;
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int e = 0; e < V; ++e) v[k][e] = in[k] ? v[k][e] - mean : 0.f;
  }
  s[0] = 0.f;
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int e = 0; e < V; ++e) s[0] = fmaf(v[k][e], v[k][e], s[0]);
  row_sum<1, WIDE>(s, lpr, red, phase);
  const float r = 1.f / sqrtf(fmaf(s[0], p.inv_c, p.eps));
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int e = 0; e < V; ++e) v[k][e] *= r;
  return r;
}

// One row per group of lpr threads, CTAs walking blocks of rows.
template <typename XT, typename YT, int V, int NV, bool WIDE>
__global__ void __launch_bounds__(512) residual_norm_fwd_kernel(const NormParams p, int lpr_log2) {
  __shared__ float red[2][2][32];
  int phase = 0;
  const int lpr = 1 << lpr_log2, lane = threadIdx.x & (lpr - 1), slot = threadIdx.x >> lpr_log2;
  const int rows_per_cta = blockDim.x >> lpr_log2;
  const uint64_t stream = p.rng.offset + (p.rng.threshold && p.rng.step ? *p.rng.step : 0ull);
  const long long blocks = (p.T + rows_per_cta - 1) / rows_per_cta;
  for (long long b = blockIdx.x; b < blocks; b += gridDim.x) {
    const long long row = b * rows_per_cta + slot;
    const bool live = row < p.T;
    const size_t base = live ? static_cast<size_t>(row) * p.C : 0;
    bool in[NV];
    float x[NV][V], u[NV][V], g[NV][V];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = (lane + k * lpr) * V;
      in[k] = live && c < p.C;
#pragma unroll
      for (int e = 0; e < V; ++e) x[k][e] = u[k][e] = 0.f, g[k][e] = 1.f;
      if (in[k]) {
        load_v<XT, V>(p.x, base + c, x[k]);
        if (p.y) load_v<YT, V>(p.y, base + c, u[k]);
        if (p.gate) load_v<YT, V>(p.gate, base + c, g[k]);
      }
    }
    if (p.y) {
      if (p.post) normalise<V, NV, WIDE>(u, in, p.post, p, lpr, red, phase);
      const float* scale = p.scale ? p.scale + (live ? row / p.rows_per_group : 0) * p.C : nullptr;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        if (!in[k]) continue;
        const int c = (lane + k * lpr) * V;
        float a[V];
        if (p.post_w) {
          load_v<float, V>(p.post_w, c, a);
#pragma unroll
          for (int e = 0; e < V; ++e) u[k][e] *= a[e];
        }
        if (p.post_b) {
          load_v<float, V>(p.post_b, c, a);
#pragma unroll
          for (int e = 0; e < V; ++e) u[k][e] += a[e];
        }
        if (scale) {
          load_v<float, V>(scale, c, a);
#pragma unroll
          for (int e = 0; e < V; ++e) g[k][e] *= a[e];
        }
        if (p.rng.threshold) {
          // a dropped element adds 0 whatever the branch holds
          drop_factor<V>(p.rng, stream, base + c, a);
#pragma unroll
          for (int e = 0; e < V; ++e) x[k][e] += a[e] != 0.f ? a[e] * g[k][e] * u[k][e] : 0.f;
        } else {
#pragma unroll
          for (int e = 0; e < V; ++e) x[k][e] = fmaf(g[k][e], u[k][e], x[k][e]);
        }
        if (p.x_out) store_v<XT, V, true>(p.x_out, base + c, x[k]);
      }
    }
    if (p.pre) {
      normalise<V, NV, WIDE>(x, in, p.pre, p, lpr, red, phase);
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        if (!in[k]) continue;
        const int c = (lane + k * lpr) * V;
        float a[V];
        if (p.pre_w) {
          load_v<float, V>(p.pre_w, c, a);
#pragma unroll
          for (int e = 0; e < V; ++e) x[k][e] *= a[e];
        }
        if (p.pre_b) {
          load_v<float, V>(p.pre_b, c, a);
#pragma unroll
          for (int e = 0; e < V; ++e) x[k][e] += a[e];
        }
        store_v<YT, V, true>(p.h, base + c, x[k]);
      }
    }
  }
}

// CTA (group, chunk): rows of one scale group, so dscale's partials never mix groups.
template <typename XT, typename YT, int V, int NV, bool WIDE>
__global__ void __launch_bounds__(512) residual_norm_bwd_kernel(const NormParams p, int lpr_log2) {
  extern __shared__ float acc_smem[];   // [slots][lpr * NV * V], one sum at a time
  __shared__ float red[2][2][32];
  int phase = 0;
  const int lpr = 1 << lpr_log2, lane = threadIdx.x & (lpr - 1), slot = threadIdx.x >> lpr_log2;
  const int rows_per_cta = blockDim.x >> lpr_log2;
  const uint64_t stream = p.rng.offset + (p.rng.threshold && p.rng.step ? *p.rng.step : 0ull);
  const long long group = blockIdx.x / p.chunks, chunk = blockIdx.x % p.chunks;
  const long long g0 = group * p.rows_per_group;
  const long long g1 = g0 + p.rows_per_group < p.T ? g0 + p.rows_per_group : p.T;
  const float* scale = p.scale ? p.scale + group * p.C : nullptr;
  float acc[kSums][NV][V];
#pragma unroll
  for (int s = 0; s < kSums; ++s)
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int e = 0; e < V; ++e) acc[s][k][e] = 0.f;

  // every thread of the CTA takes the same number of steps (the row sums meet at barriers)
  for (long long r0 = g0 + chunk * rows_per_cta; r0 < g1; r0 += static_cast<long long>(p.chunks) * rows_per_cta) {
    const long long row = r0 + slot;
    const bool live = row < g1;
    const size_t base = live ? static_cast<size_t>(row) * p.C : 0;
    bool in[NV];
    float xh[NV][V], u[NV][V], g[NV][V], d[NV][V], dh[NV][V];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = (lane + k * lpr) * V;
      in[k] = live && c < p.C;
#pragma unroll
      for (int e = 0; e < V; ++e) xh[k][e] = u[k][e] = d[k][e] = dh[k][e] = 0.f, g[k][e] = 1.f;
      if (in[k]) {
        if (p.pre) {
          load_v<XT, V>(p.x, base + c, xh[k]);
          load_v<YT, V>(p.dh, base + c, dh[k]);
        }
        if (p.y) load_v<YT, V>(p.y, base + c, u[k]);
        if (p.gate) load_v<YT, V>(p.gate, base + c, g[k]);
        if (p.dx_out) load_v<XT, V>(p.dx_out, base + c, d[k]);
      }
    }
    if (p.pre) {
      const float r = normalise<V, NV, WIDE>(xh, in, p.pre, p, lpr, red, phase);
      float s[2] = {0.f, 0.f};
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int c = (lane + k * lpr) * V;
        float w[V];
#pragma unroll
        for (int e = 0; e < V; ++e) w[e] = 1.f;
        if (in[k] && p.pre_w) load_v<float, V>(p.pre_w, c, w);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          acc[3][k][e] = fmaf(dh[k][e], xh[k][e], acc[3][k][e]);
          acc[4][k][e] += dh[k][e];
          dh[k][e] *= w[e];
          s[0] += dh[k][e];
          s[1] = fmaf(dh[k][e], xh[k][e], s[1]);
        }
      }
      row_sum<2, WIDE>(s, lpr, red, phase);
      const float m0 = p.pre == 1 ? s[0] * p.inv_c : 0.f, m1 = s[1] * p.inv_c;
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int e = 0; e < V; ++e) d[k][e] = in[k] ? fmaf(r, dh[k][e] - m0 - xh[k][e] * m1, d[k][e]) : 0.f;
    }
    if (p.dx)
#pragma unroll
      for (int k = 0; k < NV; ++k)
        if (in[k]) store_v<XT, V, false>(p.dx, base + (lane + k * lpr) * V, d[k]);
    if (!p.y) continue;
    float ry = 1.f;
    if (p.post) ry = normalise<V, NV, WIDE>(u, in, p.post, p, lpr, red, phase);
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = (lane + k * lpr) * V;
      float w[V], b[V], sc[V], m[V];
#pragma unroll
      for (int e = 0; e < V; ++e) w[e] = sc[e] = m[e] = 1.f, b[e] = 0.f;
      if (in[k]) {
        if (p.post_w) load_v<float, V>(p.post_w, c, w);
        if (p.post_b) load_v<float, V>(p.post_b, c, b);
        if (scale) load_v<float, V>(scale, c, sc);
        if (p.rng.threshold) drop_factor<V>(p.rng, stream, base + c, m);
      }
      float dg[V];
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float uu = fmaf(u[k][e], w[e], b[e]);   // N_post(y) post_w + post_b
        const float dm = m[e] != 0.f ? d[k][e] * m[e] : 0.f;
        const float dmu = m[e] != 0.f ? dm * uu : 0.f;
        dg[e] = dmu * sc[e];
        acc[0][k][e] = fmaf(dmu, g[k][e], acc[0][k][e]);
        const float du = dm * sc[e] * g[k][e];
        acc[1][k][e] = fmaf(du, u[k][e], acc[1][k][e]);
        acc[2][k][e] += du;
        d[k][e] = du * w[e];
        s[0] += d[k][e];
        s[1] = fmaf(d[k][e], u[k][e], s[1]);
      }
      if (in[k] && p.dgate) store_v<YT, V, false>(p.dgate, base + c, dg);
    }
    if (p.post) {
      row_sum<2, WIDE>(s, lpr, red, phase);
      const float m0 = p.post == 1 ? s[0] * p.inv_c : 0.f, m1 = s[1] * p.inv_c;
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int e = 0; e < V; ++e) d[k][e] = ry * (d[k][e] - m0 - u[k][e] * m1);
    }
    if (p.dy)
#pragma unroll
      for (int k = 0; k < NV; ++k)
        if (in[k]) store_v<YT, V, false>(p.dy, base + (lane + k * lpr) * V, d[k]);
  }

  // the CTA's groups of threads, one sum at a time, in their order
  if (!p.partial) return;
  const int width = lpr * NV * V;
#pragma unroll
  for (int s = 0; s < kSums; ++s) {
    __syncthreads();
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int e = 0; e < V; ++e) acc_smem[slot * width + (lane + k * lpr) * V + e] = acc[s][k][e];
    __syncthreads();
    for (int c = threadIdx.x; c < p.C; c += blockDim.x) {
      float v = 0.f;
      for (int q = 0; q < rows_per_cta; ++q) v += acc_smem[q * width + c];
      p.partial[(static_cast<size_t>(blockIdx.x) * kSums + s) * p.C + c] = v;
    }
  }
}

struct NormSums {
  float* out[kSums];   // dscale [groups][C], dpost_w, dpost_b, dpre_w, dpre_b [C]; null: not wanted
  const float* partial;
  int C, chunks, groups;
};

// blockIdx.y 0..3: dpost_w .. dpre_b over every CTA's partial; 4 + g: dscale of group g.
__global__ void __launch_bounds__(256) residual_norm_sum_kernel(const NormSums p) {
  __shared__ float part[8][33];
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const bool is_scale = blockIdx.y >= 4;
  const int s = is_scale ? 0 : blockIdx.y + 1;
  float* out = p.out[s];
  if (!out) return;
  const int first = is_scale ? (blockIdx.y - 4) * p.chunks : 0;
  const int rows = is_scale ? p.chunks : p.chunks * p.groups;
  float v = 0.f;
  if (c < p.C)
    for (int r = w; r < rows; r += 8) v += p.partial[(static_cast<size_t>(first + r) * kSums + s) * p.C + c];
  part[w][lane] = v;
  __syncthreads();
  if (w == 0 && c < p.C) {
    float t = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) t += part[k][lane];
    out[(is_scale ? static_cast<size_t>(blockIdx.y - 4) * p.C : 0) + c] = t;
  }
}

// The threads of a row and the vectors of a thread: the fewest slots that hold
// C, and among equals rows inside a warp (no barriers), then more threads.
struct RowShape {
  int v, nv, lpr_log2;
};
RowShape row_shape(int C, bool vec, int max_nv) {
  RowShape best{vec ? 4 : 1, 0, 0};
  long best_slots = 1L << 60;
  const int vecs = vec ? C / 4 : C;
  const int options4[] = {1, 2, 3}, options1[] = {4, 8, 8};
  const int order[] = {5, 4, 3, 2, 6, 7, 8, 9};
  for (int l : order)
    for (int i = 0; i < (vec ? max_nv : 2); ++i) {
      const int nv = vec ? options4[i] : options1[i];
      const long slots = static_cast<long>(nv) << l;
      if (slots >= vecs && slots < best_slots) {
        best_slots = slots;
        best.nv = nv;
        best.lpr_log2 = l;
      }
    }
  return best;
}

int cta_threads(int lpr_log2) { return lpr_log2 > 8 ? 512 : 256; }

long long bwd_chunks(long long T, long long rows_per_group, int groups, int rows_per_cta) {
  // two CTAs an SM over all groups, no more than a group has blocks of rows
  const long long target = 2ll * 148;
  long long chunks = (target + groups - 1) / groups;
  const long long rows = rows_per_group < T ? rows_per_group : T;
  const long long blocks = (rows + rows_per_cta - 1) / rows_per_cta;
  return chunks < blocks ? (chunks > 0 ? chunks : 1) : (blocks > 0 ? blocks : 1);
}

template <typename XT, typename YT>
cudaError_t launch_fwd(const NormParams& p, bool vec, cudaStream_t stream) {
  const RowShape s = row_shape(p.C, vec, 3);
  const int threads = cta_threads(s.lpr_log2), rows_per_cta = threads >> s.lpr_log2;
  const long long blocks = (p.T + rows_per_cta - 1) / rows_per_cta;
  const long long most = static_cast<long long>(sm_count()) * (2048 / threads);
  const unsigned grid = static_cast<unsigned>(blocks < most ? blocks : most);
  const bool wide = s.lpr_log2 > 5;
#define RIB_FWD(V, NV)                                                                                              \
  if (s.v == V && s.nv == NV) {                                                                                     \
    if (wide) residual_norm_fwd_kernel<XT, YT, V, NV, true><<<grid, threads, 0, stream>>>(p, s.lpr_log2);           \
    else residual_norm_fwd_kernel<XT, YT, V, NV, false><<<grid, threads, 0, stream>>>(p, s.lpr_log2);               \
    return cudaGetLastError();                                                                                      \
  }
  RIB_FWD(4, 1) RIB_FWD(4, 2) RIB_FWD(4, 3) RIB_FWD(1, 4) RIB_FWD(1, 8)
#undef RIB_FWD
  return cudaErrorInvalidConfiguration;
}

template <typename XT, typename YT>
cudaError_t launch_bwd(NormParams p, bool vec, int groups, cudaStream_t stream) {
  const RowShape s = row_shape(p.C, vec, 2);
  const int threads = cta_threads(s.lpr_log2), rows_per_cta = threads >> s.lpr_log2;
  p.chunks = static_cast<int>(bwd_chunks(p.T, p.rows_per_group, groups, rows_per_cta));
  const unsigned grid = static_cast<unsigned>(p.chunks) * groups;
  const size_t smem = p.partial ? static_cast<size_t>(rows_per_cta) * (s.v * s.nv << s.lpr_log2) * sizeof(float) : 0;
  const bool wide = s.lpr_log2 > 5;
#define RIB_BWD(V, NV)                                                                                              \
  if (s.v == V && s.nv == NV) {                                                                                     \
    if (wide) residual_norm_bwd_kernel<XT, YT, V, NV, true><<<grid, threads, smem, stream>>>(p, s.lpr_log2);        \
    else residual_norm_bwd_kernel<XT, YT, V, NV, false><<<grid, threads, smem, stream>>>(p, s.lpr_log2);            \
    return cudaGetLastError();                                                                                      \
  }
  RIB_BWD(4, 1) RIB_BWD(4, 2) RIB_BWD(1, 4) RIB_BWD(1, 8)
#undef RIB_BWD
  return cudaErrorInvalidConfiguration;
}

rib_status bad(const char* who, rib_status st, const char* what) {
  char buf[200];
  std::snprintf(buf, sizeof(buf), "%s: %s", who, what);
  return fail(st, buf);
}

rib_status check_desc(const char* who, const rib_residual_norm_desc* d) {
  if (!d) return bad(who, RIB_ERR_INVALID_ARG, "null descriptor");
  if (d->T < 0 || d->C <= 0 || d->rows_per_group <= 0) return bad(who, RIB_ERR_INVALID_ARG, "sizes: T >= 0, C and rows_per_group positive");
  if (d->pre < 0 || d->pre > 2 || d->post < 0 || d->post > 2)
    return bad(who, RIB_ERR_INVALID_ARG, "pre and post must be RIB_NORM_NONE, RIB_NORM_LAYER or RIB_NORM_RMS");
  if (!(d->eps > 0.f) || !std::isfinite(d->eps)) return bad(who, RIB_ERR_INVALID_ARG, "eps must be positive and finite");
  if (!(d->p >= 0.f && d->p <= 1.f)) return bad(who, RIB_ERR_INVALID_ARG, "p must be in [0, 1]");
  const int xs = d->x_dtype, ys = d->dtype;
  if (xs < 0 || xs > 2 || ys < 0 || ys > 2) return bad(who, RIB_ERR_INVALID_ARG, "dtypes must be RIB_BF16, RIB_F32 or RIB_F16");
  if (xs != RIB_F32 && xs != ys) return bad(who, RIB_ERR_UNSUPPORTED, "a 16-bit residual stream needs the branch in the same type");
  if (d->C > kMaxC) return bad(who, RIB_ERR_UNSUPPORTED, "needs C <= 4096");
  if (d->T > (1ll << 40)) return bad(who, RIB_ERR_UNSUPPORTED, "T above 2^40");
  if (d->T > 0 && (d->T - 1) / d->rows_per_group + 1 > kMaxGroups)
    return bad(who, RIB_ERR_UNSUPPORTED, "more than 1024 groups of rows");
  return RIB_OK;
}

int group_count(const rib_residual_norm_desc* d) {
  return d->T > 0 ? static_cast<int>((d->T - 1) / d->rows_per_group + 1) : 1;
}

// Vectors of four need C % 4 == 0 and every tensor on a vector's boundary.
struct Aligner {
  bool vec = true, element = true;
  void add(const void* p, int dtype) {
    const uintptr_t size = dtype == RIB_F32 ? 4 : 2, a = reinterpret_cast<uintptr_t>(p);
    if (a % size) element = false;
    if (a % (4 * size)) vec = false;
  }
};

}  // namespace
}  // namespace rib

using namespace rib;

extern "C" {

rib_status rib_residual_norm(const rib_residual_norm_desc* d, const void* x, const void* y, const void* gate,
                             const float* scale, const float* post_w, const float* post_b, const float* pre_w,
                             const float* pre_b, void* x_out, void* h, const uint64_t* step, cudaStream_t stream) {
  const char* who = "rib_residual_norm";
  rib_status st = check_desc(who, d);
  if (st != RIB_OK) return st;
  if (d->T == 0) return RIB_OK;   // empty tensors may have null pointers
  if (!x) return bad(who, RIB_ERR_INVALID_ARG, "null x");
  if (!h != (d->pre == RIB_NORM_NONE)) return bad(who, RIB_ERR_INVALID_ARG, "h goes with a pre norm: both or neither");
  if (!y && (gate || scale || post_w || post_b || d->post != RIB_NORM_NONE || x_out))
    return bad(who, RIB_ERR_INVALID_ARG, "without y there is no gate, scale, post norm or x_out");
  if (!y && !h) return bad(who, RIB_ERR_INVALID_ARG, "nothing to compute: neither y nor a pre norm");
  if (y && !x_out && !h) return bad(who, RIB_ERR_INVALID_ARG, "nothing to write: neither x_out nor h");
  if ((post_w || post_b) && d->post == RIB_NORM_NONE) return bad(who, RIB_ERR_INVALID_ARG, "post_w and post_b need a post norm");
  if ((pre_w || pre_b) && d->pre == RIB_NORM_NONE) return bad(who, RIB_ERR_INVALID_ARG, "pre_w and pre_b need a pre norm");
  Aligner a;
  a.add(x, d->x_dtype);
  a.add(x_out, d->x_dtype);
  for (const void* q : {y, gate, static_cast<const void*>(h)}) a.add(q, d->dtype);
  for (const float* q : {scale, post_w, post_b, pre_w, pre_b}) a.add(q, RIB_F32);
  if (!a.element || reinterpret_cast<uintptr_t>(step) % 8) return bad(who, RIB_ERR_ALIGNMENT, "tensors need their element's alignment, step 8 bytes");
  NormParams p{};
  p.T = d->T; p.C = d->C; p.rows_per_group = d->rows_per_group; p.pre = d->pre; p.post = d->post;
  p.eps = d->eps; p.inv_c = 1.f / d->C;
  p.x = x; p.y = y; p.gate = gate; p.scale = scale; p.post_w = post_w; p.post_b = post_b; p.pre_w = pre_w; p.pre_b = pre_b;
  p.x_out = x_out; p.h = h;
  make_drop_rng(d->p, d->seed, d->offset, step, &p.rng);
  const bool vec = a.vec && d->C % 4 == 0;
  cudaError_t e;
  if (d->x_dtype == RIB_BF16) e = launch_fwd<__nv_bfloat16, __nv_bfloat16>(p, vec, stream);
  else if (d->x_dtype == RIB_F16) e = launch_fwd<__half, __half>(p, vec, stream);
  else if (d->dtype == RIB_BF16) e = launch_fwd<float, __nv_bfloat16>(p, vec, stream);
  else if (d->dtype == RIB_F16) e = launch_fwd<float, __half>(p, vec, stream);
  else e = launch_fwd<float, float>(p, vec, stream);
  if (e != cudaSuccess) return cuda_fail(e, "rib_residual_norm launch");
  return RIB_OK;
}

size_t rib_residual_norm_bwd_workspace_size(const rib_residual_norm_desc* d) {
  if (!d || d->T <= 0 || d->C <= 0 || d->C > kMaxC || d->rows_per_group <= 0) return 0;
  const int groups = group_count(d);
  // the vector and the scalar form take different rows a CTA: the larger of the two
  size_t most = 0;
  for (int vec = 0; vec < 2; ++vec) {
    if (vec && d->C % 4) continue;
    const RowShape s = row_shape(d->C, vec, 2);
    const int rows_per_cta = cta_threads(s.lpr_log2) >> s.lpr_log2;
    const size_t n = static_cast<size_t>(bwd_chunks(d->T, d->rows_per_group, groups, rows_per_cta)) * groups;
    most = n > most ? n : most;
  }
  return most * kSums * d->C * sizeof(float);
}

rib_status rib_residual_norm_bwd(const rib_residual_norm_desc* d, const void* x_out, const void* y, const void* gate,
                                 const float* scale, const float* post_w, const float* post_b, const float* pre_w,
                                 const void* dx_out, const void* dh, void* dx, void* dy, void* dgate, float* dscale,
                                 float* dpost_w, float* dpost_b, float* dpre_w, float* dpre_b, void* ws, size_t ws_bytes,
                                 const uint64_t* step, cudaStream_t stream) {
  const char* who = "rib_residual_norm_bwd";
  rib_status st = check_desc(who, d);
  if (st != RIB_OK) return st;
  const bool pre = d->pre != RIB_NORM_NONE;
  // empty tensors may have null pointers: without rows only the weight gradients count
  const bool rows = d->T > 0;
  if (rows && pre && (!x_out || !dh)) return bad(who, RIB_ERR_INVALID_ARG, "a pre norm needs x_out and dh");
  if (!pre && (dh || pre_w || dpre_w || dpre_b)) return bad(who, RIB_ERR_INVALID_ARG, "dh, pre_w, dpre_w and dpre_b need a pre norm");
  if (rows && !pre && !dx_out) return bad(who, RIB_ERR_INVALID_ARG, "no gradient to start from: neither dx_out nor dh");
  if (rows && !y && (gate || scale || post_w || post_b || d->post != RIB_NORM_NONE || dy || dgate || dscale || dpost_w || dpost_b))
    return bad(who, RIB_ERR_INVALID_ARG, "without y there is no gate, scale or post norm, nor their gradients");
  if (d->post == RIB_NORM_NONE && (post_w || post_b || dpost_w || dpost_b))
    return bad(who, RIB_ERR_INVALID_ARG, "post_w, post_b and their gradients need a post norm");
  if (rows && dgate && !gate) return bad(who, RIB_ERR_INVALID_ARG, "dgate needs gate");
  if (rows && dscale && !scale) return bad(who, RIB_ERR_INVALID_ARG, "dscale needs scale");
  const bool sums = dscale || dpost_w || dpost_b || dpre_w || dpre_b;
  if (sums && rows && !ws) return bad(who, RIB_ERR_INVALID_ARG, "weight gradients need the workspace");
  if (sums && ws_bytes < rib_residual_norm_bwd_workspace_size(d)) return bad(who, RIB_ERR_INVALID_ARG, "workspace too small");
  Aligner a;
  a.add(x_out, d->x_dtype);
  a.add(dx_out, d->x_dtype);
  a.add(dx, d->x_dtype);
  for (const void* q : {y, gate, dh, static_cast<const void*>(dy), static_cast<const void*>(dgate)}) a.add(q, d->dtype);
  for (const float* q : {scale, post_w, post_b, pre_w}) a.add(q, RIB_F32);
  Aligner b;   // written one element at a time
  for (const float* q : {dscale, dpost_w, dpost_b, dpre_w, dpre_b}) b.add(q, RIB_F32);
  b.add(ws, RIB_F32);
  if (!a.element || !b.element || reinterpret_cast<uintptr_t>(step) % 8)
    return bad(who, RIB_ERR_ALIGNMENT, "tensors need their element's alignment, the workspace 4 bytes, step 8");
  if (rows && !sums && !dx && !dy && !dgate) return bad(who, RIB_ERR_INVALID_ARG, "nothing to write");
  const int groups = group_count(d);
  NormSums sp{};
  cudaError_t e = cudaSuccess;
  if (rows) {
    NormParams p{};
    p.T = d->T; p.C = d->C; p.rows_per_group = d->rows_per_group; p.pre = d->pre; p.post = d->post;
    p.eps = d->eps; p.inv_c = 1.f / d->C;
    p.x = x_out; p.y = y; p.gate = gate; p.scale = scale; p.post_w = post_w; p.post_b = post_b; p.pre_w = pre_w;
    p.dx_out = dx_out; p.dh = dh; p.dx = dx; p.dy = dy; p.dgate = dgate;
    p.partial = sums ? static_cast<float*>(ws) : nullptr;
    make_drop_rng(d->p, d->seed, d->offset, step, &p.rng);
    const bool vec = a.vec && d->C % 4 == 0;
    if (d->x_dtype == RIB_BF16) e = launch_bwd<__nv_bfloat16, __nv_bfloat16>(p, vec, groups, stream);
    else if (d->x_dtype == RIB_F16) e = launch_bwd<__half, __half>(p, vec, groups, stream);
    else if (d->dtype == RIB_BF16) e = launch_bwd<float, __nv_bfloat16>(p, vec, groups, stream);
    else if (d->dtype == RIB_F16) e = launch_bwd<float, __half>(p, vec, groups, stream);
    else e = launch_bwd<float, float>(p, vec, groups, stream);
    if (e != cudaSuccess) return cuda_fail(e, "rib_residual_norm_bwd launch");
    const RowShape s = row_shape(d->C, vec, 2);
    sp.chunks = static_cast<int>(bwd_chunks(d->T, d->rows_per_group, groups, cta_threads(s.lpr_log2) >> s.lpr_log2));
  }
  if (!sums) return RIB_OK;
  // no rows: the sums are empty and the gradients zero
  sp.out[0] = dscale; sp.out[1] = dpost_w; sp.out[2] = dpost_b; sp.out[3] = dpre_w; sp.out[4] = dpre_b;
  sp.partial = static_cast<const float*>(ws);
  sp.C = d->C;
  sp.groups = rows ? groups : 0;
  const dim3 grid((d->C + 31) / 32, 4 + (dscale ? sp.groups : 0));
  residual_norm_sum_kernel<<<grid, 256, 0, stream>>>(sp);
  e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "rib_residual_norm_bwd: sums launch");
  return RIB_OK;
}

}  // extern "C"
