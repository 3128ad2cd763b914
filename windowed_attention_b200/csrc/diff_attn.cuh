// Shared by the differential attention kernels: where a sequence's tokens lie,
// and how their rows reach the swizzled shared-memory tiles that tcgen05.mma
// reads.
//
// A sequence is one batch item (window 0) or one window of a map, cut off at
// the map's edge. Query rows are (token, query head of the group) pairs,
// row = token * G + g: the G query heads that share a key head meet the same
// key tiles, so a tile of 128 rows is full even for a single token with many
// heads, and the gradients of a shared head are sums over rows.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "rib_internal.h"
#include "sm100.cuh"

namespace rib {

constexpr float kDiffLog2e = 1.4426950408889634f;
constexpr float kDiffLn2 = 0.6931471805599453f;

struct DiffStrides {
  long long b, t, h;   // elements between batch items, tokens and heads
};

struct DiffGeom {
  int batch, q_len, k_len, q_heads, kv_heads, group;   // group = q_heads / kv_heads
  int d, dv;
  int window, width, height, nwx, nwy;                 // window 0: sequences
  int causal, lam_f32;
  uint32_t group_magic;                                // see div_by(); 0: group 1
  float scale, scale_log2;
  const int* k_lens;
  DiffStrides q, k, v, o;
};

// t / n for n > 1 with magic = ceil(2^32 / n) (0 for n <= 1): exact while t * n < 2^32.
__host__ __device__ inline uint32_t div_magic(uint32_t n) { return n > 1 ? 0xFFFFFFFFu / n + 1u : 0u; }
__device__ __forceinline__ int div_by(int t, uint32_t magic) {
  return static_cast<int>(__umulhi(static_cast<uint32_t>(t), magic));
}

// Query row r is (token r / G, head r % G of the group).
__device__ __forceinline__ int diff_row_token(const DiffGeom& g, int r) { return g.group_magic ? div_by(r, g.group_magic) : r; }

// One sequence: token t (0 .. nq - 1 of the queries, 0 .. nk - 1 of the keys)
// is batch item b's token t0 + (t / n1) * width + t % n1.
struct DiffSeq {
  int b, t0, nq, nk, n1, width;
  uint32_t magic;   // of n1; 0 with one column (n1 = 1) or a sequence (n1 = 0)

  __device__ __forceinline__ long long token(int t) const {
    const int r = magic ? div_by(t, magic) : (n1 == 1 ? t : 0);
    return static_cast<long long>(t0) + static_cast<long long>(r) * width + (t - r * n1);
  }
};

__device__ __forceinline__ DiffSeq diff_sequence(const DiffGeom& g, int s) {
  DiffSeq q;
  if (g.window) {
    const int wx = s % g.nwx, wy = (s / g.nwx) % g.nwy;
    q.b = s / (g.nwx * g.nwy);
    const int y0 = wy * g.window, x0 = wx * g.window;
    const int hv = min(g.window, g.height - y0), wv = min(g.window, g.width - x0);
    q.t0 = y0 * g.width + x0;
    q.nq = q.nk = hv * wv;
    q.n1 = wv;
    q.width = g.width;
    q.magic = div_magic(static_cast<uint32_t>(wv));
  } else {
    q.b = s;
    q.t0 = 0;
    q.nq = g.q_len;
    q.nk = g.k_lens ? min(max(g.k_lens[s], 0), g.k_len) : g.k_len;
    q.n1 = 0;
    q.width = 0;
    q.magic = 0u;
  }
  return q;
}

// Keys that query token t of a sequence sees (a prefix): all, or with the
// causal mask those up to its own place counted from the end.
__device__ __forceinline__ int diff_visible(const DiffGeom& g, const DiffSeq& s, int t) {
  return g.causal ? min(max(t + 1 + s.nk - s.nq, 0), s.nk) : s.nk;
}

// A tile of ROWS rows of D 16-bit elements as tcgen05.mma operands: atoms of up
// to 64 columns side by side, each [ROWS][RB bytes] with the swizzle of that
// row size. The same bytes serve as a K-major operand (products over D: +32
// bytes a K step, atom to atom every 64) and as an MN-major one (products over
// the rows: +16 rows a K step, atoms along N).
template <int ROWS, int D>
struct DiffTile {
  static constexpr int COLS = D < 64 ? D : 64;
  static constexpr int RB = COLS * 2;
  static constexpr int ATOM = ROWS * RB;
  static constexpr int BYTES = ROWS * D * 2;
  static constexpr uint32_t SW = RB == 128 ? SW_128B : (RB == 64 ? SW_64B : SW_32B);
  static constexpr int CHUNKS = D / 8;   // 16-byte pieces of a row
  static_assert(D == 16 || D == 32 || D == 64 || D == 128, "operand widths");

  __device__ static __forceinline__ uint32_t offset(int row, int chunk) {
    constexpr int per = COLS / 8;
    const int a = chunk / per, c = chunk % per;
    const int x = RB == 128 ? (row & 7) : (RB == 64 ? ((row >> 1) & 3) : ((row >> 2) & 1));
    return static_cast<uint32_t>(a * ATOM + row * RB + ((c ^ x) << 4));
  }
  // K-major descriptor of K step ks (16 columns)
  __device__ static __forceinline__ uint64_t kmajor(uint32_t base, int ks) {
    constexpr int per = COLS / 16;
    return make_sdesc(base + (ks / per) * ATOM + (ks % per) * 32, 16, 8 * RB, SW);
  }
  // MN-major descriptor of K step ks (16 rows)
  __device__ static __forceinline__ uint64_t mnmajor(uint32_t base, int ks) {
    return make_sdesc(base + ks * 16 * RB, ATOM, 8 * RB, SW);
  }
};

// 16 bytes into shared memory, or 16 zero bytes (nothing is read then).
__device__ __forceinline__ void cp_async_16_or_zero(uint32_t dst, const void* src, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
}

// Rows first .. first + ROWS - 1 of a key-side tensor (one row a token) into a
// tile; rows at or behind n and columns at or behind d become zero, so what a
// mask hides never reaches a product.
template <int ROWS, int D, int THREADS>
__device__ __forceinline__ void diff_load_keys(uint32_t tile, const uint16_t* base, long long stride, const DiffSeq& s, int first, int n,
                                               int d, int tid) {
  using T = DiffTile<ROWS, D>;
  static_assert(THREADS % T::CHUNKS == 0, "a thread keeps its column");
  const int ch = tid % T::CHUNKS;
#pragma unroll 4
  for (int row = tid / T::CHUNKS; row < ROWS; row += THREADS / T::CHUNKS) {
    const int t = first + row;
    const bool real = t < n && ch * 8 < d;
    cp_async_16_or_zero(tile + T::offset(row, ch), real ? base + s.token(t) * stride + ch * 8 : base, real);
  }
}

// The same for a query-side tensor.
template <int ROWS, int D, int THREADS>
__device__ __forceinline__ void diff_load_queries(uint32_t tile, const uint16_t* base, const DiffStrides& st, const DiffGeom& g,
                                                  const DiffSeq& s, int first, int n, int d, int tid) {
  using T = DiffTile<ROWS, D>;
  static_assert(THREADS % T::CHUNKS == 0, "a thread keeps its column");
  const int ch = tid % T::CHUNKS;
#pragma unroll 4
  for (int row = tid / T::CHUNKS; row < ROWS; row += THREADS / T::CHUNKS) {
    const int r = first + row;
    const bool real = r < n && ch * 8 < d;
    const int t = diff_row_token(g, r), h = r - t * g.group;
    cp_async_16_or_zero(tile + T::offset(row, ch), real ? base + s.token(t) * st.t + h * st.h + ch * 8 : base, real);
  }
}

__host__ __device__ constexpr uint32_t diff_idesc(bool f16, int N, bool b_mn) {
  return f16 ? idesc_f16(128, N, false, b_mn) : idesc_bf16(128, N, false, b_mn);
}

// Two fp32 as a packed pair of the operand type.
template <bool F16>
__device__ __forceinline__ uint32_t diff_pack(float lo, float hi) {
  if constexpr (F16) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  } else {
    return pack_bf16x2(lo, hi);
  }
}
template <bool F16>
__device__ __forceinline__ float diff_lo(uint32_t v) { return F16 ? f16_lo(v) : bf16_lo(v); }
template <bool F16>
__device__ __forceinline__ float diff_hi(uint32_t v) { return F16 ? f16_hi(v) : bf16_hi(v); }
template <bool F16>
__device__ __forceinline__ float diff_lambda(const void* lam, int lam_f32, int h) {
  return lam_f32 ? static_cast<const float*>(lam)[h] : diff_lo<F16>(static_cast<const uint16_t*>(lam)[h]);
}

// What the launches get.
struct DiffFwdArgs {
  DiffGeom g;
  const void *q1, *q2, *k1, *k2, *v, *lam;
  void *o, *o2;
  float* lse;        // [2][batch][q_heads][q_len] or null
  float* part;       // split keys: [splits][rows][2][dv] then [splits][rows][2] (log2 of the row sums); null without
  int splits;
  int* err;
};
// Row constants of the backward, one array each, for the query rows of every
// (sequence, key head) padded to a multiple of 128: -log2e lse1, -log2e lse2,
// -dO.O1, -dO.O2, -lambda and the keys that the row sees (an int; 0 for the padding).
enum { kRowL1 = 0, kRowL2, kRowD1, kRowD2, kRowLam, kRowSeen, kRowArrays };
struct DiffBwdArgs {
  DiffGeom g;
  const void *q1, *q2, *k1, *k2, *v, *lam, *o, *o2, *dO;
  const float* lse;
  void *dq1, *dq2, *dk1, *dk2, *dv, *dlam;
  float* rows;       // [kRowArrays][row_stride]
  long long row_stride;
  int rows_pad;      // rows of one (sequence, key head)
  int* err;
};
inline int diff_sequences(const DiffGeom& g) { return g.window ? g.batch * g.nwx * g.nwy : g.batch; }
// Query rows of the longest sequence, of one key head.
inline long long diff_max_rows(const DiffGeom& g) {
  const long long nq = g.window ? static_cast<long long>(g.window < g.height ? g.window : g.height) * (g.window < g.width ? g.window : g.width)
                                : g.q_len;
  return nq * g.group;
}
inline int diff_max_keys(const DiffGeom& g) { return g.window ? static_cast<int>(diff_max_rows(g) / g.group) : g.k_len; }
// The operand widths of the kernels: the smallest pair that holds d and dv.
inline int diff_class(int d, int dv) { return d <= 16 && dv <= 32 ? 0 : (d <= 32 && dv <= 64 ? 1 : 2); }
int diff_splits(const DiffGeom& g);
size_t diff_split_bytes(const DiffGeom& g);
long long diff_rows_pad(const DiffGeom& g);
cudaError_t launch_diff_attn_fwd(const DiffFwdArgs& a, bool f16, cudaStream_t stream);
cudaError_t launch_diff_attn_bwd(const DiffBwdArgs& a, bool f16, cudaStream_t stream);

}  // namespace rib
