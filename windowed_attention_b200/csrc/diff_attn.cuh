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

// One row of a tensor into a tile, by a pair of lanes (par = 0, 1: they share
// 32-byte sectors): two instructions a 16-byte piece, since the swizzle is an
// exclusive or of the row's place. `size` is 16, or 0 for a row of zeros (src is
// not read then). Pieces at or behind n (the tensor's width) are left as they are.
template <int ROWS, int D>
__device__ __forceinline__ void diff_load_row(uint32_t tile, int row, int par, const uint16_t* src, int size, int n) {
  using T = DiffTile<ROWS, D>;
  constexpr int per = T::COLS / 8;
  const uint32_t dst = tile + T::offset(row, par);
  const uint16_t* from = src + par * 8;
#pragma unroll
  for (int k = 0; k < T::CHUNKS / 2; ++k)
    if (2 * k + par < n)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                   ::"r"((dst ^ ((2 * k % per) << 4)) + 2 * k / per * T::ATOM), "l"(from + 16 * k), "r"(size) : "memory");
}

// Rows first .. first + ROWS - 1 of the key side (a row a token): k1, k2 and v
// into three tiles one behind the other. Rows at or behind n become zero, so
// what a mask hides never reaches a product. Every row is a pair of lanes.
template <int ROWS, int D, int DV, int THREADS>
__device__ __forceinline__ void diff_load_keys(uint32_t tile, const uint16_t* k1, const uint16_t* k2, const uint16_t* v, const DiffGeom& g,
                                               const DiffSeq& s, int first, int n, int tid) {
  const int par = tid & 1, nd = g.d / 8, nv = g.dv / 8;
#pragma unroll
  for (int row = tid >> 1; row < ROWS; row += THREADS / 2) {
    const int t = first + row, size = t < n ? 16 : 0;
    const long long token = t < n ? s.token(t) : 0;
    diff_load_row<ROWS, D>(tile, row, par, k1 + token * g.k.t, size, nd);
    diff_load_row<ROWS, D>(tile + DiffTile<ROWS, D>::BYTES, row, par, k2 + token * g.k.t, size, nd);
    diff_load_row<ROWS, DV>(tile + 2 * DiffTile<ROWS, D>::BYTES, row, par, v + token * g.v.t, size, nv);
  }
}

// The same for the query side: q1, q2 and (dO not null) dO.
template <int ROWS, int D, int DV, int THREADS>
__device__ __forceinline__ void diff_load_queries(uint32_t tile, const uint16_t* q1, const uint16_t* q2, const uint16_t* dO, const DiffGeom& g,
                                                  const DiffSeq& s, int first, int n, int tid) {
  const int par = tid & 1, nd = g.d / 8, nv = g.dv / 8;
#pragma unroll
  for (int row = tid >> 1; row < ROWS; row += THREADS / 2) {
    const int r = first + row, size = r < n ? 16 : 0;
    const int t = r < n ? diff_row_token(g, r) : 0, h = r < n ? r - t * g.group : 0;
    const long long token = s.token(t), at = token * g.q.t + h * g.q.h;
    diff_load_row<ROWS, D>(tile, row, par, q1 + at, size, nd);
    diff_load_row<ROWS, D>(tile + DiffTile<ROWS, D>::BYTES, row, par, q2 + at, size, nd);
    if (dO) diff_load_row<ROWS, DV>(tile + 2 * DiffTile<ROWS, D>::BYTES, row, par, dO + token * g.o.t + h * g.o.h, size, nv);
  }
}

// Zeros for the columns behind the tensors' widths, which no load writes: the
// loader warps clear their tiles once (barrier 2 is theirs).
template <int D, int DV, int THREADS>
__device__ __forceinline__ void diff_clear(uint8_t* tiles, int bytes, const DiffGeom& g, int tid) {
  if (g.d == D && g.dv == DV) return;
  for (int i = tid * 16; i < bytes; i += THREADS * 16) *reinterpret_cast<uint4*>(tiles + i) = make_uint4(0u, 0u, 0u, 0u);
  asm volatile("bar.sync 2, %0;" ::"n"(THREADS) : "memory");
}

__host__ __device__ constexpr uint32_t diff_idesc(bool f16, int N, bool b_mn) {
  return f16 ? idesc_f16(128, N, false, b_mn) : idesc_bf16(128, N, false, b_mn);
}

// 2^x for a pair of x in [-inf, 127] on the FMA pipe, for the share of the
// exponentials that relieves the MUFU (16 a cycle and SM): exp2_poly_x2 with a
// polynomial of degree 4, fitted for relative error on [-1/2, 1/2] (2.8e-6,
// against 1.0e-4 of the cubic): the log-sum-exp goes out in fp32. A NaN gives
// 0; callers see it in the other elements of its row.
__device__ __forceinline__ void diff_exp2_poly(float x0, float x1, float& y0, float& y1) {
  constexpr float kRound = 12582912.0f;   // 1.5 * 2^23
  const uint64_t x = f2_pack(fmaxf(x0, -127.f), fmaxf(x1, -127.f));
  const uint64_t t = f2_add(x, f2_pack(kRound, kRound));
  const uint64_t j = f2_add(t, f2_pack(-kRound, -kRound));
  const uint64_t f = f2_fma(j, f2_pack(-1.f, -1.f), x);
  uint64_t p = f2_fma(f2_pack(0.00958285201f, 0.00958285201f), f, f2_pack(0.0559064262f, 0.0559064262f));
  p = f2_fma(p, f, f2_pack(0.240240991f, 0.240240991f));
  p = f2_fma(p, f, f2_pack(0.693124175f, 0.693124175f));
  p = f2_fma(p, f, f2_pack(1.f, 1.f));
  float p0, p1, t0, t1;
  f2_unpack(p, p0, p1);
  f2_unpack(t, t0, t1);
  y0 = __uint_as_float(__float_as_uint(p0) + (__float_as_uint(t0) << 23));
  y1 = __uint_as_float(__float_as_uint(p1) + (__float_as_uint(t1) << 23));
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
