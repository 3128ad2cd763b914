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
// Memory is the floor of both: each tensor is read or written once. A CTA walks
// blocks of whole rows, which are contiguous in every tensor: bulk copies
// bring a block into shared memory while the block before is computed, results
// overwrite their inputs there and leave by bulk copies, so no thread waits for
// memory and odd widths move like even ones (blocks at a tensor's end, or of
// tensors off a 16-byte boundary, are copied element by element). A row lives
// in the registers of a group of `lpr` threads (a power of two from 4 to 512,
// each thread NV vectors of V elements), statistics are two passes over those
// registers (mean, then squared deviations: no cancellation), and the backward
// recomputes them from x' and y rather than reading saved ones.
//
// Measured: 640x360 rows of 180, fp32 stream, bf16 branch and gate, forward
// 112-118 us by box (581 MB, 4.9-5.2 TB/s); 16x96x96 rows of 180 with dropout,
// forward 108 and backward 193 us (floors 57 and 89); 4039 rows of 1021 in fp16,
// forward and backward 131-134 us (floor 23). The forward issues in 68 % of its
// cycles, between the barriers of 16-row blocks. The backward (149 instructions
// a warp-wide element, 110 us of issue) issues in 60 %: 15 warps an SM, at 128
// registers, wait for dependent instructions, shared memory and a block's
// barriers. Rows of 1021 take pairs with 150 bytes of spills and 65 KB blocks,
// too large for a second stage, so that loads and arithmetic take turns.
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

enum NormSite : int { SITE_N_FULL = 701 };

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
  // blocks in shared memory: rows of one, the place of x, dx_out, y, gate and dh in a stage, bytes of a stage, stages
  int block, off[5], stage_bytes, stages, bulk;
  int* err;
};
enum { kX = 0, kD, kY, kG, kH };

// V consecutive elements as fp32.
template <typename T, int V>
__device__ __forceinline__ void load_v(const void* base, uint32_t at, float (&f)[V]) {
  const T* p = static_cast<const T*>(base) + at;
  if constexpr (sizeof(T) == 4) {
    if constexpr (V == 4) {
      const float4 v = *reinterpret_cast<const float4*>(p);
      f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
    } else if constexpr (V == 2) {
      const float2 v = *reinterpret_cast<const float2*>(p);
      f[0] = v.x; f[1] = v.y;
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
    } else if constexpr (V == 2) {
      const uint32_t v = *reinterpret_cast<const uint32_t*>(p);
      f[0] = kHalf ? f16_lo(v) : bf16_lo(v);
      f[1] = kHalf ? f16_hi(v) : bf16_hi(v);
    } else {
      const uint32_t v = *reinterpret_cast<const uint16_t*>(p);
      f[0] = kHalf ? f16_lo(v) : bf16_lo(v);
    }
  }
}
// Which of a thread's V elements lie in the row: all or none, but for pairs (V
// == 2) of odd rows, which start one element early so that they are aligned.
template <int V>
struct Inside {
  bool all;
  float f;   // 1 or 0
  __device__ __forceinline__ float one(int) const { return f; }
  __device__ __forceinline__ bool operator[](int) const { return all; }
  __device__ __forceinline__ bool any() const { return all; }
};
template <>
struct Inside<2> {
  bool lo, hi;
  float f[2];
  __device__ __forceinline__ float one(int e) const { return f[e]; }
  __device__ __forceinline__ bool operator[](int e) const { return e ? hi : lo; }
  __device__ __forceinline__ bool any() const { return lo || hi; }
};
template <int V>
__device__ __forceinline__ Inside<V> inside(bool live, int c, int C) {
  if constexpr (V == 2) {
    const bool lo = live && c >= 0 && c < C, hi = live && c + 1 < C;
    return {lo, hi, {lo ? 1.f : 0.f, hi ? 1.f : 0.f}};
  } else {
    const bool all = live && c < C;
    return {all, all ? 1.f : 0.f};
  }
}
// Elements from a stage or the weights beside it, zeros where they are not in the row.
template <typename T, int V>
__device__ __forceinline__ void load_if(const T* base, uint32_t at, const Inside<V>& in, float (&f)[V]) {
#pragma unroll
  for (int e = 0; e < V; ++e) f[e] = 0.f;
  if (in.any()) load_v<T, V>(base, at, f);
  if constexpr (V == 2) {
    if (!in.lo) f[0] = 0.f;
    if (!in.hi) f[1] = 0.f;
  }
}
// SAT: fp16 results beyond +-65504 saturate, as in every forward store of the
// library. Gradients do not: an overflow has to stay visible to loss scaling.
template <typename T, int V, bool SAT>
__device__ __forceinline__ void store_v(void* base, uint32_t at, const float (&f)[V]) {
  T* p = static_cast<T*>(base) + at;
  if constexpr (sizeof(T) == 4) {
    if constexpr (V == 4) *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
    else if constexpr (V == 2) *reinterpret_cast<float2*>(p) = make_float2(f[0], f[1]);
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
    else if constexpr (V == 2) *reinterpret_cast<uint32_t*>(p) = pack(f[0], f[1]);
    else *reinterpret_cast<uint16_t*>(p) = static_cast<uint16_t>(pack(f[0], 0.f));
  }
}

template <typename T, int V, bool SAT>
__device__ __forceinline__ void store_if(T* base, uint32_t at, const Inside<V>& in, const float (&f)[V]) {
  if constexpr (V == 2) {
    if (in.lo && in.hi) {
      store_v<T, 2, SAT>(base, at, f);
    } else {   // the pair's other element is a neighbouring row's
      const float lo[1] = {f[0]}, hi[1] = {f[1]};
      if (in.lo) store_v<T, 1, SAT>(base, at, lo);
      if (in.hi) store_v<T, 1, SAT>(base, at + 1, hi);
    }
  } else {
    if (in.all) store_v<T, V, SAT>(base, at, f);
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
    // the lanes of each warp read the row's warp sums (2 to 16 of them) and add them by shuffles
    const int warp = threadIdx.x >> 5, per = lpr >> 5, lane = threadIdx.x & 31;
    if (lane == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) red[phase][i][warp] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = red[phase][i][(warp & ~(per - 1)) + (lane & (per - 1))];
    for (int o = per >> 1; o > 0; o >>= 1)
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xFFFFFFFFu, v[i], o);
    phase ^= 1;
  }
}

// Blocks of rows between memory and the stages of a CTA. Tensors that are
// absent have null pointers.
template <typename XT, typename YT>
struct BlockIo {
  const NormParams& p;
  uint8_t* smem;
  uint64_t* full;
  volatile uint32_t* abort_flag;
  uint32_t laps = 0u;   // a parity bit a stage

  __device__ __forceinline__ int place(int t) const { return t == kX ? p.off[kX] : (t == kD ? p.off[kD] : (t == kY ? p.off[kY] : p.off[kG])); }
  __device__ __forceinline__ bool whole(long long r0, long long r1) const { return p.bulk && r1 - r0 == p.block; }
  // Thread 0: the stage's last results have left, then the next block comes in.
  __device__ __forceinline__ void start(int st, long long r0, long long r1, const void* const (&src)[5]) const {
    if (threadIdx.x != 0 || !whole(r0, r1)) return;
    asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    const uint32_t n = static_cast<uint32_t>(p.block) * p.C;
    uint32_t bytes = 0;
#pragma unroll
    for (int i = 0; i < 5; ++i)
      if (src[i]) bytes += n * (i < kY ? sizeof(XT) : sizeof(YT));
    mbar_arrive_expect_tx(&full[st], bytes);
#pragma unroll
    for (int i = 0; i < 5; ++i)
      if (src[i]) {
        const uint32_t size = i < kY ? sizeof(XT) : sizeof(YT);
        bulk_load(smem + st * p.stage_bytes + p.off[i], static_cast<const uint8_t*>(src[i]) + static_cast<size_t>(r0) * p.C * size, n * size,
                  &full[st]);
      }
  }
  // All threads: the block is in its stage. False after a wait that ran out.
  __device__ __forceinline__ bool ready(int st, long long r0, long long r1, const void* const (&src)[5]) {
    bool ok = true;
    if (whole(r0, r1)) {
      ok = mbar_wait(&full[st], (laps >> st) & 1u, WaitCtx{abort_flag, p.err}, SITE_N_FULL);
      laps ^= 1u << st;
    } else {
      if (threadIdx.x == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
      __syncthreads();
      const size_t n = static_cast<size_t>(r1 - r0) * p.C, at = static_cast<size_t>(r0) * p.C;
      uint8_t* to = smem + st * p.stage_bytes;
#pragma unroll
      for (int i = 0; i < 5; ++i) {
        if (!src[i]) continue;
        if (i < kY)
          for (size_t e = threadIdx.x; e < n; e += blockDim.x) reinterpret_cast<XT*>(to + p.off[i])[e] = static_cast<const XT*>(src[i])[at + e];
        else
          for (size_t e = threadIdx.x; e < n; e += blockDim.x) reinterpret_cast<YT*>(to + p.off[i])[e] = static_cast<const YT*>(src[i])[at + e];
      }
    }
    return __syncthreads_and(ok) != 0;
  }
  // All threads: results dst[k], held where tensor at[k] was, leave the stage.
  __device__ __forceinline__ void finish(int st, long long r0, long long r1, void* const (&dst)[3], const int (&at)[3]) const {
    const uint8_t* from = smem + st * p.stage_bytes;
    if (whole(r0, r1)) {
      fence_proxy_async_smem();
      __syncthreads();
      if (threadIdx.x == 0) {
        const uint32_t n = static_cast<uint32_t>(p.block) * p.C;
#pragma unroll
        for (int k = 0; k < 3; ++k)
          if (dst[k]) {
            const uint32_t size = at[k] < kY ? sizeof(XT) : sizeof(YT);
            asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;"
                         ::"l"(static_cast<uint8_t*>(dst[k]) + static_cast<size_t>(r0) * p.C * size), "r"(smem_u32(from + place(at[k]))),
                           "r"(n * size) : "memory");
          }
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
      }
    } else {
      __syncthreads();
      const size_t n = static_cast<size_t>(r1 - r0) * p.C, to = static_cast<size_t>(r0) * p.C;
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        if (!dst[k]) continue;
        if (at[k] < kY)
          for (size_t e = threadIdx.x; e < n; e += blockDim.x) static_cast<XT*>(dst[k])[to + e] = reinterpret_cast<const XT*>(from + place(at[k]))[e];
        else
          for (size_t e = threadIdx.x; e < n; e += blockDim.x) static_cast<YT*>(dst[k])[to + e] = reinterpret_cast<const YT*>(from + place(at[k]))[e];
      }
      fence_proxy_async_smem();   // the stage's next block may come by bulk copies
      __syncthreads();
    }
  }
  __device__ __forceinline__ void drain() const {
    if (threadIdx.x == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }
};

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
    const auto half = [](const uint4& w, uint32_t s) {
      const uint32_t v = s < 4 ? (s < 2 ? w.x : w.y) : (s < 6 ? w.z : w.w);
      return (s & 1) ? v >> 16 : v & 0xFFFFu;
    };
    const uint32_t s = static_cast<uint32_t>(at & 7);
    m[0] = half(w, s) >= rng.threshold ? rng.up : 0.f;
    if constexpr (V == 2) {
      const uint4 next = s == 7 ? philox4x32_10((at >> 3) + 1, stream, rng.seed) : w;
      m[1] = half(next, (s + 1) & 7) >= rng.threshold ? rng.up : 0.f;
    }
  }
}

// v := (v - mean) * r in place; returns r. Elements behind the row's end stay 0.
template <int V, int NV, bool WIDE>
__device__ __forceinline__ float normalise(float (&v)[NV][V], const Inside<V> (&in)[NV], int kind, const NormParams& p, int lpr,
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
      for (int e = 0; e < V; ++e) v[k][e] = fmaf(-mean, in[k].one(e), v[k][e]);   // stays 0 outside the row
  }
  s[0] = 0.f;
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int e = 0; e < V; ++e) s[0] = fmaf(v[k][e], v[k][e], s[0]);
  row_sum<1, WIDE>(s, lpr, red, phase);
  const float r = rsqrtf(fmaf(s[0], p.inv_c, p.eps));   // within 2 units in the last place
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int e = 0; e < V; ++e) v[k][e] *= r;
  return r;
}

__device__ __forceinline__ long long group_of(long long row, long long per) {
  if (((row | per) >> 32) == 0) return static_cast<uint32_t>(row) / static_cast<uint32_t>(per);
  return row / per;
}

// Columns of a CTA's weight arrays in shared memory; pairs keep a second copy of
// them, shifted by one element for the rows that start on an odd one.
__host__ __device__ inline int weight_columns(int C) { return (C + 1 + 3) / 4 * 4; }
template <int V>
__device__ __forceinline__ void put_weight(float* weights, int arrays, int which, int c, int C, float v) {
  const int wide = weight_columns(C);
  weights[which * wide + c] = v;
  if constexpr (V == 2) weights[(arrays + which) * wide + c + 1] = v;
}

// One row per group of lpr threads, CTAs walking blocks of rows.
template <typename XT, typename YT, int V, int NV, bool WIDE>
__global__ void __launch_bounds__(512, 2) residual_norm_fwd_kernel(const __grid_constant__ NormParams p, int lpr_log2) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float red[2][2][32];
  __shared__ uint64_t full[2];
  __shared__ uint32_t abort_word;
  if (threadIdx.x == 0) {
    mbar_init(&full[0], 1);
    mbar_init(&full[1], 1);
    abort_word = 0u;
    fence_barrier_init();
  }
  __syncthreads();
  int phase = 0;
  const int lpr = 1 << lpr_log2, lane = threadIdx.x & (lpr - 1), slot = threadIdx.x >> lpr_log2;
  const int rows_per_cta = blockDim.x >> lpr_log2;
  const uint64_t stream = p.rng.offset + (p.rng.threshold && p.rng.step ? *p.rng.step : 0ull);
  const long long blocks = (p.T + p.block - 1) / p.block;
  BlockIo<XT, YT> io{p, smem, full, &abort_word};
  const void* const src[5] = {p.x, nullptr, p.y, p.gate, nullptr};
  void* const dst[3] = {p.y ? p.x_out : nullptr, p.pre ? p.h : nullptr, nullptr};
  const int held[3] = {kX, kY, kY};
  const auto last = [&](long long b) { return (b + 1) * p.block < p.T ? (b + 1) * p.block : p.T; };
  if (blockIdx.x < blocks) io.start(0, static_cast<long long>(blockIdx.x) * p.block, last(blockIdx.x), src);
  int st = 0;
  // the weights of every column, in shared memory: post_w, post_b, pre_w, pre_b, scale (of the first group)
  float* weights = reinterpret_cast<float*>(smem + p.stages * p.stage_bytes);
  const int wide_c = weight_columns(p.C);
  for (int c = threadIdx.x; c < p.C; c += blockDim.x) {
    put_weight<V>(weights, 5, 0, c, p.C, p.post_w ? p.post_w[c] : 1.f);
    put_weight<V>(weights, 5, 1, c, p.C, p.post_b ? p.post_b[c] : 0.f);
    put_weight<V>(weights, 5, 2, c, p.C, p.pre_w ? p.pre_w[c] : 1.f);
    put_weight<V>(weights, 5, 3, c, p.C, p.pre_b ? p.pre_b[c] : 0.f);
    put_weight<V>(weights, 5, 4, c, p.C, p.scale ? p.scale[c] : 1.f);
  }
  const bool many = p.scale && p.rows_per_group < p.T;   // groups
  // pairs: this thread's rows all start on an even element of their block (par 0) or all on an odd one, since the CTA's
  // rows in step are an even number
  const int par = V == 2 && (p.C & 1) ? slot & 1 : 0;
  const float* w0 = weights + (par ? 5 * wide_c : 0) + lane * V;
  for (long long b = blockIdx.x; b < blocks; b += gridDim.x) {
    const long long r0 = b * p.block, r1 = last(b), next = b + gridDim.x;
    if (p.stages == 2 && next < blocks) io.start(st ^ 1, next * p.block, last(next), src);
    if (!io.ready(st, r0, r1, src)) break;
    uint8_t* stage = smem + st * p.stage_bytes;
    for (int rr = slot; rr - slot < p.block; rr += rows_per_cta) {
      const long long row = r0 + rr;
      const bool live = row < r1;
      const uint32_t at = (live ? rr : par) * p.C + lane * V - par;
      XT* sx = reinterpret_cast<XT*>(stage + p.off[kX]) + at;
      YT* sy = reinterpret_cast<YT*>(stage + p.off[kY]) + at;
      const YT* sg = reinterpret_cast<const YT*>(stage + p.off[kG]) + at;
      Inside<V> in[NV];
      float x[NV][V], u[NV][V];
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        in[k] = inside<V>(live, (lane + k * lpr) * V - par, p.C);
        load_if<XT, V>(sx, k * lpr * V, in[k], x[k]);
      }
      if (p.y) {
#pragma unroll
        for (int k = 0; k < NV; ++k) load_if<YT, V>(sy, k * lpr * V, in[k], u[k]);
        if (p.post) normalise<V, NV, WIDE>(u, in, p.post, p, lpr, red, phase);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
          float w[V], c[V];
          load_if<float, V>(w0, k * lpr * V, in[k], w);
          load_if<float, V>(w0, wide_c + k * lpr * V, in[k], c);
#pragma unroll
          for (int e = 0; e < V; ++e) u[k][e] = fmaf(u[k][e], w[e], c[e]);
        }
        if (many) {
          const float* scale = p.scale + (live ? group_of(row, p.rows_per_group) : 0) * p.C;
#pragma unroll
          for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int e = 0; e < V; ++e)
              if (in[k][e]) u[k][e] *= scale[(lane + k * lpr) * V - par + e];
        } else {
#pragma unroll
          for (int k = 0; k < NV; ++k) {
            float w[V];
            load_if<float, V>(w0, 4 * wide_c + k * lpr * V, in[k], w);
#pragma unroll
            for (int e = 0; e < V; ++e) u[k][e] *= w[e];
          }
        }
        if (p.gate) {
#pragma unroll
          for (int k = 0; k < NV; ++k) {
            float g[V];
            load_if<YT, V>(sg, k * lpr * V, in[k], g);
#pragma unroll
            for (int e = 0; e < V; ++e) u[k][e] *= g[e];
          }
        }
        if (p.rng.threshold) {
#pragma unroll
          for (int k = 0; k < NV; ++k) {
            float m[V];
            drop_factor<V>(p.rng, stream, static_cast<uint64_t>(row) * p.C + (lane + k * lpr) * V - par, m);
            // a dropped element adds 0 whatever the branch holds
#pragma unroll
            for (int e = 0; e < V; ++e) u[k][e] = m[e] != 0.f ? m[e] * u[k][e] : 0.f;
          }
        }
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
          for (int e = 0; e < V; ++e) x[k][e] += u[k][e];
        if (p.x_out)
#pragma unroll
          for (int k = 0; k < NV; ++k)
            store_if<XT, V, true>(sx, k * lpr * V, in[k], x[k]);
      }
      if (p.pre) {
        normalise<V, NV, WIDE>(x, in, p.pre, p, lpr, red, phase);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
          float w[V], c[V];
          load_if<float, V>(w0, 2 * wide_c + k * lpr * V, in[k], w);
          load_if<float, V>(w0, 3 * wide_c + k * lpr * V, in[k], c);
#pragma unroll
          for (int e = 0; e < V; ++e) x[k][e] = fmaf(x[k][e], w[e], c[e]);
          store_if<YT, V, true>(sy, k * lpr * V, in[k], x[k]);
        }
      }
    }
    io.finish(st, r0, r1, dst, held);
    if (p.stages == 2) st ^= 1;
    else if (next < blocks) io.start(0, next * p.block, last(next), src);
  }
  io.drain();
}

// CTA (group, chunk): rows of one scale group, so dscale's partials never mix groups.
template <typename XT, typename YT, int V, int NV, bool WIDE>
__global__ void __launch_bounds__(512) residual_norm_bwd_kernel(const __grid_constant__ NormParams p, int lpr_log2) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float red[2][2][32];
  __shared__ uint64_t full[2];
  __shared__ uint32_t abort_word;
  if (threadIdx.x == 0) {
    mbar_init(&full[0], 1);
    mbar_init(&full[1], 1);
    abort_word = 0u;
    fence_barrier_init();
  }
  __syncthreads();
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

  // this chunk's share of the group's blocks, which lie at multiples of p.block of all rows
  const long long b0 = g0 / p.block, n_blocks = g1 > g0 ? (g1 - 1) / p.block - b0 + 1 : 0;
  const long long first = b0 + n_blocks * chunk / p.chunks, behind = b0 + n_blocks * (chunk + 1) / p.chunks;
  BlockIo<XT, YT> io{p, smem, full, &abort_word};
  const bool pre = p.pre != 0;
  const void* const src[5] = {pre ? p.x : nullptr, p.dx_out, p.y, p.gate, pre ? p.dh : nullptr};
  const int dx_at = pre ? kX : kD;
  void* const dst[3] = {p.dx, p.y ? p.dy : nullptr, p.y ? p.dgate : nullptr};
  const int held[3] = {dx_at, kY, kG};
  const auto lo = [&](long long b) { return b * p.block > g0 ? b * p.block : g0; };
  const auto hi = [&](long long b) { return (b + 1) * p.block < g1 ? (b + 1) * p.block : g1; };
  if (first < behind) io.start(0, lo(first), hi(first), src);
  // the weights of every column, in shared memory: pre_w, post_w, post_b, scale
  float* weights = reinterpret_cast<float*>(smem + p.stages * p.stage_bytes);
  const int wide_c = weight_columns(p.C);
  for (int c = threadIdx.x; c < p.C; c += blockDim.x) {
    put_weight<V>(weights, 4, 0, c, p.C, p.pre_w ? p.pre_w[c] : 1.f);
    put_weight<V>(weights, 4, 1, c, p.C, p.post_w ? p.post_w[c] : 1.f);
    put_weight<V>(weights, 4, 2, c, p.C, p.post_b ? p.post_b[c] : 0.f);
    put_weight<V>(weights, 4, 3, c, p.C, scale ? scale[c] : 1.f);
  }
  const int par = V == 2 && (p.C & 1) ? slot & 1 : 0;   // as in the forward
  const float* w0 = weights + (par ? 4 * wide_c : 0) + lane * V;
  int st = 0;
  for (long long blk = first; blk < behind; ++blk) {
    const long long r0 = lo(blk), r1 = hi(blk);
    if (p.stages == 2 && blk + 1 < behind) io.start(st ^ 1, lo(blk + 1), hi(blk + 1), src);
    if (!io.ready(st, r0, r1, src)) break;
    uint8_t* stage = smem + st * p.stage_bytes;
    // every thread of the CTA takes the same number of steps (the row sums meet at barriers)
    for (int rr = slot; rr - slot < p.block; rr += rows_per_cta) {
      const long long row = r0 + rr;
      const bool live = row < r1;
      const uint32_t at = (live ? rr : par) * p.C + lane * V - par;
      XT* sx = reinterpret_cast<XT*>(stage + p.off[kX]) + at;
      XT* sd = reinterpret_cast<XT*>(stage + p.off[kD]) + at;
      YT* sy = reinterpret_cast<YT*>(stage + p.off[kY]) + at;
      YT* sg = reinterpret_cast<YT*>(stage + p.off[kG]) + at;
      const YT* sh = reinterpret_cast<const YT*>(stage + p.off[kH]) + at;
      Inside<V> in[NV];
      float d[NV][V];
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        in[k] = inside<V>(live, (lane + k * lpr) * V - par, p.C);
        load_if<XT, V>(sd, k * lpr * V, inside<V>(live && p.dx_out, (lane + k * lpr) * V - par, p.C), d[k]);
      }
      if (pre) {
        float xh[NV][V], dh[NV][V];
#pragma unroll
        for (int k = 0; k < NV; ++k) {
          load_if<XT, V>(sx, k * lpr * V, in[k], xh[k]);
          load_if<YT, V>(sh, k * lpr * V, in[k], dh[k]);
        }
        const float r = normalise<V, NV, WIDE>(xh, in, p.pre, p, lpr, red, phase);
        float s[2] = {0.f, 0.f};
#pragma unroll
        for (int k = 0; k < NV; ++k) {
          float w[V];
          load_if<float, V>(w0, k * lpr * V, in[k], w);
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
          for (int e = 0; e < V; ++e) d[k][e] = fmaf(r, fmaf(-m1, xh[k][e], fmaf(-m0, in[k].one(e), dh[k][e])), d[k][e]);
      }
      if (p.dx) {
        XT* out = pre ? sx : sd;
#pragma unroll
        for (int k = 0; k < NV; ++k)
          store_if<XT, V, false>(out, k * lpr * V, in[k], d[k]);
      }
      if (!p.y) continue;
      float u[NV][V];
#pragma unroll
      for (int k = 0; k < NV; ++k) load_if<YT, V>(sy, k * lpr * V, in[k], u[k]);
      float ry = 1.f;
      if (p.post) ry = normalise<V, NV, WIDE>(u, in, p.post, p, lpr, red, phase);
      float s[2] = {0.f, 0.f};
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        float w[V], b[V], sc[V], m[V], g[V], dg[V];
        load_if<float, V>(w0, wide_c + k * lpr * V, in[k], w);
        load_if<float, V>(w0, 2 * wide_c + k * lpr * V, in[k], b);
        load_if<float, V>(w0, 3 * wide_c + k * lpr * V, in[k], sc);
#pragma unroll
        for (int e = 0; e < V; ++e) g[e] = 1.f;
        if (p.gate) load_if<YT, V>(sg, k * lpr * V, in[k], g);
        const auto branch = [&](auto drops) {
#pragma unroll
          for (int e = 0; e < V; ++e) {
            const float uu = fmaf(u[k][e], w[e], b[e]);   // N_post(y) post_w + post_b
            // a dropped element has no part in any gradient, whatever the branch, the gate and the scale hold there
            const bool kept = !decltype(drops)::value || m[e] != 0.f;
            float du = 0.f;
            dg[e] = 0.f;
            if (kept) {
              const float dm = decltype(drops)::value ? d[k][e] * m[e] : d[k][e], dmu = dm * uu;
              dg[e] = dmu * sc[e];
              acc[0][k][e] = fmaf(dmu, g[e], acc[0][k][e]);
              du = dm * (sc[e] * g[e]);
            }
            acc[1][k][e] = fmaf(du, u[k][e], acc[1][k][e]);
            acc[2][k][e] += du;
            d[k][e] = du * w[e];
            s[0] += d[k][e];
            s[1] = fmaf(d[k][e], u[k][e], s[1]);
          }
        };
        if (p.rng.threshold) {
          drop_factor<V>(p.rng, stream, static_cast<uint64_t>(row) * p.C + (lane + k * lpr) * V - par, m);
          branch(std::true_type{});
        } else {
          branch(std::false_type{});
        }
        if (p.dgate) store_if<YT, V, false>(sg, k * lpr * V, in[k], dg);
      }
      if (!p.dy) continue;
      if (p.post) {
        row_sum<2, WIDE>(s, lpr, red, phase);
        const float m0 = p.post == 1 ? s[0] * p.inv_c : 0.f, m1 = s[1] * p.inv_c;
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
          for (int e = 0; e < V; ++e) d[k][e] = ry * (d[k][e] - m0 - u[k][e] * m1);
      }
#pragma unroll
      for (int k = 0; k < NV; ++k)
        store_if<YT, V, false>(sy, k * lpr * V, in[k], d[k]);
    }
    io.finish(st, r0, r1, dst, held);
    if (p.stages == 2) st ^= 1;
    else if (blk + 1 < behind) io.start(0, lo(blk + 1), hi(blk + 1), src);
  }
  io.drain();

  // the CTA's groups of threads, one sum at a time, in their order
  if (!p.partial) return;
  float* acc_smem = reinterpret_cast<float*>(smem);   // [slots][lpr * NV * V + 1], one sum at a time, column c at c + 1
  const int width = lpr * NV * V + 1;
#pragma unroll
  for (int s = 0; s < kSums; ++s) {
    __syncthreads();
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int e = 0; e < V; ++e) acc_smem[slot * width + (lane + k * lpr) * V + e - par + 1] = acc[s][k][e];
    __syncthreads();
    for (int c = threadIdx.x; c < p.C; c += blockDim.x) {
      float v = 0.f;
      for (int q = 0; q < rows_per_cta; ++q) v += acc_smem[q * width + c + 1];
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
// Vectors of four where C % 4 == 0 and the tensors are aligned; pairs else,
// which odd rows start one element early (see Inside); single elements for odd
// rows too wide for two of them in step.
struct RowShape {
  int v, nv, lpr_log2;
};
RowShape row_shape(int C, bool vec) {
  const bool odd_wide = C % 2 && C > 2046;
  RowShape best{vec ? 4 : (odd_wide ? 1 : 2), 0, 0};
  long best_slots = 1L << 60;
  const int vecs = vec ? C / 4 : (odd_wide ? C : (C % 2 ? C / 2 + 1 : C / 2));
  const int options4[] = {1, 2, 3}, options2[] = {1, 2, 4}, options1[] = {8, 8, 8};
  const int* options = vec ? options4 : (odd_wide ? options1 : options2);
  const int order[] = {5, 4, 3, 2, 6, 7, 8, 9};
  for (int l : order) {
    if (best.v == 2 && C % 2 && l > 8) continue;   // two rows of 256 threads in step at least
    for (int i = 0; i < 3; ++i) {
      const long slots = static_cast<long>(options[i]) << l;
      if (slots >= vecs && slots < best_slots) {
        best_slots = slots;
        best.nv = options[i];
        best.lpr_log2 = l;
      }
    }
  }
  return best;
}

// Threads of a CTA: 512 for rows of 256 threads or more, and where a block's shared
// memory leaves room for no more than two CTAs an SM.
int cta_threads(int lpr_log2, long long block_bytes) { return lpr_log2 > 7 || block_bytes > 56 * 1024 ? 512 : 256; }
// Rows that make whole 16-byte pieces of a tensor of that element size.
int row_unit(int C, int size) {
  int unit = 1;
  while (unit < 8 && static_cast<long long>(unit) * C * size % 16) unit *= 2;
  return unit;
}

// CTAs of a group in the backward: two an SM over all groups, no more than the group has rows.
long long bwd_chunks(long long T, long long rows_per_group, int groups) {
  const long long chunks = (2ll * sm_count() + groups - 1) / groups;
  const long long rows = rows_per_group < T ? rows_per_group : T;
  return chunks < rows ? chunks : (rows > 0 ? rows : 1);
}

// Rows of a block and its place in shared memory. Bulk copies need whole
// multiples of 16 bytes, that is 8 / gcd(C, 8) rows of a 16-bit tensor. Blocks
// of about 24 KB in two stages leave room for two to four CTAs an SM; wide
// rows get what fits, in one stage.
constexpr int kSmemMost = 224 * 1024;   // of any plan of C <= kMaxC, weights included
void plan_blocks(NormParams* p, const void* const (&src)[5], const bool (&held)[5], int xs, int ys, int rows_per_cta, bool aligned, int extra) {
  int elem = 0;
  for (int i = 0; i < 5; ++i)
    if (src[i] || held[i]) elem += i < kY ? xs : ys;
  const int unit = row_unit(p->C, ys);
  const auto bytes = [&](int rows) {   // each tensor's part on a 16-byte boundary
    int n = 0;
    for (int i = 0; i < 5; ++i) {
      p->off[i] = n;
      if (src[i] || held[i]) n += (rows * p->C * (i < kY ? xs : ys) + 127) / 128 * 128;
    }
    return n;
  };
  int rows = rows_per_cta > unit ? rows_per_cta : unit;
  p->bulk = aligned && bytes(rows) + extra <= kSmemMost;
  if (!p->bulk) rows = rows_per_cta;
  while (static_cast<long long>(rows) * p->C * elem < 16 * 1024 && rows < 512) rows *= 2;
  p->block = rows;
  p->stage_bytes = bytes(rows);
  p->stages = p->bulk && 2 * p->stage_bytes + extra <= kSmemMost / 2 ? 2 : 1;
}

// Beyond 48 KB, static arrays included, a kernel has to ask. The limit belongs to
// the kernel, not to the call, and one instance serves many sizes: it is always
// raised to the most that any plan takes, so that a call of another host thread
// cannot lower it between this call's request and its launch.
template <typename K>
cudaError_t allow_smem(K kernel, int bytes) {
  return bytes > 46 * 1024 ? cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMost) : cudaSuccess;
}

template <typename XT, typename YT>
cudaError_t launch_fwd(NormParams p, bool vec, bool aligned, cudaStream_t stream) {
  const RowShape s = row_shape(p.C, vec);
  const int threads = cta_threads(s.lpr_log2, static_cast<long long>(row_unit(p.C, sizeof(YT))) * p.C * (sizeof(XT) + 2 * sizeof(YT)));
  const int weights = (s.v == 2 ? 10 : 5) * weight_columns(p.C) * static_cast<int>(sizeof(float));
  const int rows_per_cta = threads >> s.lpr_log2;
  plan_blocks(&p, {p.x, nullptr, p.y, p.gate, nullptr}, {true, false, true, false, false}, sizeof(XT), sizeof(YT), rows_per_cta, aligned, weights);
  const int smem = p.stages * p.stage_bytes + weights;
  const long long blocks = (p.T + p.block - 1) / p.block;
  const int by_smem = 227 * 1024 / (smem + 2048), by_threads = 1024 / threads;
  const long long most = static_cast<long long>(sm_count()) * (by_smem < by_threads ? by_smem : by_threads);
  const unsigned grid = static_cast<unsigned>(blocks < most ? blocks : most);
  const bool wide = s.lpr_log2 > 5;
  const auto run = [&](auto kernel) {
    const cudaError_t e = allow_smem(kernel, smem);
    if (e != cudaSuccess) return e;
    kernel<<<grid, threads, smem, stream>>>(p, s.lpr_log2);
    return cudaGetLastError();
  };
#define RIB_FWD(V, NV)                                                                     \
  if (s.v == V && s.nv == NV) return wide ? run(residual_norm_fwd_kernel<XT, YT, V, NV, true>) \
                                          : run(residual_norm_fwd_kernel<XT, YT, V, NV, false>);
  RIB_FWD(4, 1) RIB_FWD(4, 2) RIB_FWD(4, 3) RIB_FWD(2, 1) RIB_FWD(2, 2) RIB_FWD(2, 4) RIB_FWD(1, 8)
#undef RIB_FWD
  return cudaErrorInvalidConfiguration;
}

template <typename XT, typename YT>
cudaError_t launch_bwd(NormParams p, bool vec, bool aligned, int groups, int* chunks, cudaStream_t stream) {
  const RowShape s = row_shape(p.C, vec);
  const int threads = cta_threads(s.lpr_log2, static_cast<long long>(row_unit(p.C, sizeof(YT))) * p.C * (2 * sizeof(XT) + 3 * sizeof(YT)));
  const int weights = (s.v == 2 ? 8 : 4) * weight_columns(p.C) * static_cast<int>(sizeof(float));
  const int rows_per_cta = threads >> s.lpr_log2;
  const bool pre = p.pre != 0;
  plan_blocks(&p, {pre ? p.x : nullptr, p.dx_out, p.y, p.gate, pre ? p.dh : nullptr}, {false, false, false, false, false}, sizeof(XT),
              sizeof(YT), rows_per_cta, aligned, weights);
  const int sums = p.partial ? rows_per_cta * ((s.v * s.nv << s.lpr_log2) + 1) * static_cast<int>(sizeof(float)) : 0;
  const int stages = p.stages * p.stage_bytes + weights, smem = stages > sums ? stages : sums;
  // the CTAs that run at once, in whole chunks a group, and no more than the workspace's partials
  const int by_smem = 227 * 1024 / (smem + 2048), per_sm = by_smem < 512 / threads ? by_smem : 512 / threads;
  const long long most = bwd_chunks(p.T, p.rows_per_group, groups), fit = static_cast<long long>(sm_count()) * (per_sm > 0 ? per_sm : 1) / groups;
  p.chunks = static_cast<int>(fit < 1 ? 1 : (fit < most ? fit : most));
  *chunks = p.chunks;
  const unsigned grid = static_cast<unsigned>(p.chunks) * groups;
  const bool wide = s.lpr_log2 > 5;
  const auto run = [&](auto kernel) {
    const cudaError_t e = allow_smem(kernel, smem);
    if (e != cudaSuccess) return e;
    kernel<<<grid, threads, smem, stream>>>(p, s.lpr_log2);
    return cudaGetLastError();
  };
#define RIB_BWD(V, NV)                                                                     \
  if (s.v == V && s.nv == NV) return wide ? run(residual_norm_bwd_kernel<XT, YT, V, NV, true>) \
                                          : run(residual_norm_bwd_kernel<XT, YT, V, NV, false>);
  RIB_BWD(4, 1) RIB_BWD(4, 2) RIB_BWD(4, 3) RIB_BWD(2, 1) RIB_BWD(2, 2) RIB_BWD(2, 4) RIB_BWD(1, 8)
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

// Vectors of four need C % 4 == 0 and the tensors that move in blocks on a vector's boundary (weights are read by element).
struct Aligner {
  bool vec = true, element = true, bulk = true;   // bulk: 16 bytes
  void add(const void* p, int dtype) {
    const uintptr_t size = dtype == RIB_F32 ? 4 : 2, a = reinterpret_cast<uintptr_t>(p);
    if (a % size) element = false;
    if (a % (4 * size)) vec = false;
    if (a % 16) bulk = false;
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
  Aligner a;   // the tensors that move in blocks
  a.add(x, d->x_dtype);
  a.add(x_out, d->x_dtype);
  for (const void* q : {y, gate, static_cast<const void*>(h)}) a.add(q, d->dtype);
  Aligner b;   // read one element at a time
  for (const float* q : {scale, post_w, post_b, pre_w, pre_b}) b.add(q, RIB_F32);
  if (!a.element || !b.element || reinterpret_cast<uintptr_t>(step) % 8) return bad(who, RIB_ERR_ALIGNMENT, "tensors need their element's alignment, step 8 bytes");
  NormParams p{};
  p.T = d->T; p.C = d->C; p.rows_per_group = d->rows_per_group; p.pre = d->pre; p.post = d->post;
  p.eps = d->eps; p.inv_c = 1.f / d->C;
  p.x = x; p.y = y; p.gate = gate; p.scale = scale; p.post_w = post_w; p.post_b = post_b; p.pre_w = pre_w; p.pre_b = pre_b;
  p.x_out = x_out; p.h = h;
  if (!(p.err = device_error_word())) return bad(who, RIB_ERR_CUDA, "no device error word");
  make_drop_rng(d->p, d->seed, d->offset, step, &p.rng);
  const bool vec = a.vec && d->C % 4 == 0;
  cudaError_t e;
  if (d->x_dtype == RIB_BF16) e = launch_fwd<__nv_bfloat16, __nv_bfloat16>(p, vec, a.bulk, stream);
  else if (d->x_dtype == RIB_F16) e = launch_fwd<__half, __half>(p, vec, a.bulk, stream);
  else if (d->dtype == RIB_BF16) e = launch_fwd<float, __nv_bfloat16>(p, vec, a.bulk, stream);
  else if (d->dtype == RIB_F16) e = launch_fwd<float, __half>(p, vec, a.bulk, stream);
  else e = launch_fwd<float, float>(p, vec, a.bulk, stream);
  if (e != cudaSuccess) return cuda_fail(e, "rib_residual_norm launch");
  return RIB_OK;
}

size_t rib_residual_norm_bwd_workspace_size(const rib_residual_norm_desc* d) {
  if (!d || d->T <= 0 || d->C <= 0 || d->C > kMaxC || d->rows_per_group <= 0) return 0;
  const int groups = group_count(d);
  return static_cast<size_t>(bwd_chunks(d->T, d->rows_per_group, groups)) * groups * kSums * d->C * sizeof(float);
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
  Aligner a;   // the tensors that move in blocks
  a.add(x_out, d->x_dtype);
  a.add(dx_out, d->x_dtype);
  a.add(dx, d->x_dtype);
  for (const void* q : {y, gate, dh, static_cast<const void*>(dy), static_cast<const void*>(dgate)}) a.add(q, d->dtype);
  Aligner b;   // read or written one element at a time
  for (const float* q : {scale, post_w, post_b, pre_w}) b.add(q, RIB_F32);
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
    if (!(p.err = device_error_word())) return bad(who, RIB_ERR_CUDA, "no device error word");
    make_drop_rng(d->p, d->seed, d->offset, step, &p.rng);
    const bool vec = a.vec && d->C % 4 == 0;
    if (d->x_dtype == RIB_BF16) e = launch_bwd<__nv_bfloat16, __nv_bfloat16>(p, vec, a.bulk, groups, &sp.chunks, stream);
    else if (d->x_dtype == RIB_F16) e = launch_bwd<__half, __half>(p, vec, a.bulk, groups, &sp.chunks, stream);
    else if (d->dtype == RIB_BF16) e = launch_bwd<float, __nv_bfloat16>(p, vec, a.bulk, groups, &sp.chunks, stream);
    else if (d->dtype == RIB_F16) e = launch_bwd<float, __half>(p, vec, a.bulk, groups, &sp.chunks, stream);
    else e = launch_bwd<float, float>(p, vec, a.bulk, groups, &sp.chunks, stream);
    if (e != cudaSuccess) return cuda_fail(e, "rib_residual_norm_bwd launch");
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
