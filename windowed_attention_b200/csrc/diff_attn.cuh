// Shared by the differential attention kernels: where a sequence's tokens lie,
// and how their rows reach the swizzled shared-memory tiles that tcgen05.mma
// reads.
//
// A sequence is one batch item, or one window of a map, cut off at the map's
// edge. Both are rectangles of tokens (a sequence is one row of them), and TMA
// loads a rectangle of at most 64 rows, a "box":
//   keys     64 tokens, tck x trk
//   queries  tcq x trq tokens times the G query heads that share a key head,
//            row = token * G + head: boxes are full even for single tokens of
//            many heads, and gradients of a shared head are sums over rows.
// The order of a window's tokens does not matter to attention, so boxes need
// not follow it. Rows of a box outside the sequence are masked; where they
// hold other tokens (a neighbouring window, keys behind a length) the streamed
// side's are also cleared, since 0 * NaN is NaN in a product.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "rib_internal.h"
#include "sm100.cuh"

namespace rib {

constexpr float kDiffLog2e = 1.4426950408889634f;
constexpr float kDiffLn2 = 0.6931471805599453f;

struct DiffStrides {
  long long b;   // elements between batch items,
  int t, h;      // tokens and heads
};

struct DiffGeom {
  int batch, q_len, k_len, q_heads, kv_heads, group;   // group = q_heads / kv_heads
  int d, dv;
  int window, width, height, nwx, nwy;                 // window 0: sequences
  int tck, lk, trk;                                    // key boxes; lk = log2 tck
  int tcq, lq, trq;                                    // query boxes; lq = log2 tcq, 31 for sequences (one row)
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
__host__ __device__ inline int ceil_div(int a, int b) { return (a + b - 1) / b; }
__device__ __forceinline__ long long wide(int a, int b) { return static_cast<long long>(a) * b; }

__device__ __forceinline__ int diff_row_token(const DiffGeom& g, int r) { return g.group_magic ? div_by(r, g.group_magic) : r; }

// One sequence: a rectangle of queries wq x hq and one of keys wk x hk at (x0, y0) of batch item b.
struct DiffSeq {
  int b, x0, y0, wq, hq, wk, hk, width;
  __device__ __forceinline__ int token(int x, int y) const { return (y0 + y) * width + x0 + x; }
};

__device__ __forceinline__ DiffSeq diff_sequence(const DiffGeom& g, int s) {
  DiffSeq q;
  if (g.window) {
    const int wx = s % g.nwx, wy = (s / g.nwx) % g.nwy;
    q.b = s / (g.nwx * g.nwy);
    q.x0 = wx * g.window;
    q.y0 = wy * g.window;
    q.wq = q.wk = min(g.window, g.width - q.x0);
    q.hq = q.hk = min(g.window, g.height - q.y0);
    q.width = g.width;
  } else {
    q.b = s;
    q.x0 = q.y0 = 0;
    q.wq = g.q_len;
    q.wk = g.k_lens ? min(max(g.k_lens[s], 0), g.k_len) : g.k_len;
    q.hq = q.hk = 1;
    q.width = 0;
  }
  return q;
}

// Keys that query x of a sequence sees (a prefix; windows see all, see below):
// with the causal mask those up to its own place counted from the end.
__device__ __forceinline__ int diff_visible(const DiffGeom& g, const DiffSeq& s, int x) {
  return g.causal ? min(max(x + 1 + s.wk - s.wq, 0), s.wk) : s.wk;
}
__device__ __forceinline__ int diff_q_boxes(const DiffGeom& g, const DiffSeq& s) {
  return ceil_div(s.wq, g.tcq) * ceil_div(s.hq, g.trq);
}

// Row r6 of a query box.
struct DiffRow {
  int x, y, head;   // place in the sequence; head in its group
  bool live;
};
__device__ __forceinline__ DiffRow diff_query_row(const DiffGeom& g, const DiffSeq& s, int box, int r6) {
  DiffRow r;
  const int idx = g.group_magic ? div_by(r6, g.group_magic) : r6;
  r.head = r6 - idx * g.group;
  const int nx = ceil_div(s.wq, g.tcq), by = box / nx, bx = box - by * nx;
  const int yy = idx >> g.lq, xx = idx - (yy << g.lq);
  r.x = bx * g.tcq + xx;
  r.y = by * g.trq + yy;
  r.live = idx < g.tcq * g.trq && r.x < s.wq && r.y < s.hq;
  return r;
}

// The keys of box j that exist, a bit each: column c is (c % tck, c / tck) of the box.
struct DiffKeyBox {
  int x, y, vx, vy;   // place in the sequence, existing columns and rows (vx may exceed tck, vy trk)
};
__device__ __forceinline__ DiffKeyBox diff_key_box(const DiffGeom& g, const DiffSeq& s, int nx, int j) {
  DiffKeyBox k;
  const int by = j / nx, bx = j - by * nx;
  k.x = bx * g.tck;
  k.y = by * g.trk;
  k.vx = s.wk - k.x;
  k.vy = s.hk - k.y;
  return k;
}
__device__ __forceinline__ uint64_t diff_key_mask(const DiffGeom& g, int vx, int vy) {
  if (vx <= 0 || vy <= 0) return 0ull;
  const uint64_t row = vx >= g.tck ? (g.tck == 64 ? ~0ull : (1ull << g.tck) - 1ull) : (1ull << vx) - 1ull;
  uint64_t m = 0ull;
  for (int y = 0; y < min(vy, g.trk); ++y) m |= row << (y << g.lk);
  return m;
}

// The keys of box j that a row sees which sees `seen` keys of its sequence.
__device__ __forceinline__ uint64_t diff_seen(const DiffGeom& g, const DiffSeq& s, int nx, int j, int seen) {
  if (g.window) {
    const DiffKeyBox k = diff_key_box(g, s, nx, j);
    return k.vx >= g.tck && k.vy >= g.trk ? ~0ull : diff_key_mask(g, k.vx, k.vy);
  }
  const int left = seen - 64 * j;
  return left >= 64 ? ~0ull : (left > 0 ? (1ull << left) - 1ull : 0ull);
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
  static_assert(D == 16 || D == 32 || D == 64 || D == 128, "operand widths");

  __device__ static __forceinline__ uint32_t offset(int row, int chunk) {
    constexpr int per = COLS / 8;
    const int a = chunk / per, c = chunk % per;
    const int x = RB == 128 ? (row & 7) : (RB == 64 ? ((row >> 1) & 3) : ((row >> 2) & 1));
    return static_cast<uint32_t>(a * ATOM + row * RB + ((c ^ x) << 4));
  }
  // Descriptors of a tile at shared address `base`, and what K step ks adds to
  // them (a descriptor's low bits are the address / 16): one addition a
  // product, since the issuing thread's own instructions bound its rate.
  // K-major: steps of 16 columns; MN-major: steps of 16 rows.
  __device__ static __forceinline__ uint64_t kmajor(uint32_t base) { return make_sdesc(base, 16, 8 * RB, SW); }
  __device__ static constexpr uint32_t kstep(int ks) { return (ks / (COLS / 16) * ATOM + ks % (COLS / 16) * 32) >> 4; }
  __device__ static __forceinline__ uint64_t mnmajor(uint32_t base) { return make_sdesc(base, ATOM, 8 * RB, SW); }
  __device__ static constexpr uint32_t mnstep(int ks) { return (ks * 16 * RB) >> 4; }
  // One box into rows `row` .. of the tile; columns behind the tensor's width
  // arrive as zeros.
  __device__ static __forceinline__ void load(uint8_t* tile, int row, const CUtensorMap* map, uint64_t* bar, int head, int x, int y, int b) {
#pragma unroll
    for (int a = 0; a < D / COLS; ++a) tma_load_5d(tile + a * ATOM + row * RB, map, bar, a * COLS, head, x, y, b);
  }
  __device__ static __forceinline__ uint32_t box_bytes(int rows) { return static_cast<uint32_t>(rows * D * 2); }
  // Zeros into a row, by `lanes` threads.
  __device__ static __forceinline__ void clear_row(uint8_t* tile, int row, int lane, int lanes) {
    for (int c = lane; c < D / 8; c += lanes) *reinterpret_cast<uint4*>(tile + offset(row, c)) = make_uint4(0u, 0u, 0u, 0u);
  }
};

// Zeros into the rows of a box whose bits are set, two tiles of width D and one of DV behind them, by a warp.
template <int ROWS, int D, int DV>
__device__ __forceinline__ void diff_clear_rows(uint8_t* tiles, uint64_t rows, int lane) {
  while (rows) {
    const int row = __ffsll(static_cast<long long>(rows)) - 1;
    rows &= rows - 1;
    DiffTile<ROWS, D>::clear_row(tiles, row, lane, 32);
    DiffTile<ROWS, D>::clear_row(tiles + DiffTile<ROWS, D>::BYTES, row, lane, 32);
    DiffTile<ROWS, DV>::clear_row(tiles + 2 * DiffTile<ROWS, D>::BYTES, row, lane, 32);
  }
}

__host__ __device__ constexpr uint32_t diff_idesc(bool f16, int N, bool b_mn) {
  return f16 ? idesc_f16(128, N, false, b_mn) : idesc_bf16(128, N, false, b_mn);
}

// D = A B^T over every K step of two K-major tiles (columns behind the
// tensors' width are zeros).
template <typename TA, typename TB, int STEPS>
__device__ __forceinline__ void diff_mma_kk(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc) {
#pragma unroll
  for (int ks = 0; ks < STEPS; ++ks) umma_ss(d, a + TA::kstep(ks), b + TB::kstep(ks), idesc, ks > 0 ? 1u : 0u);
}

// A bounded wait of a whole warp.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const WaitCtx& w, int site) {
  return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, w, site));
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
  int splits, quad;  // CTAs of a query tile; the form for few rows
  int* err;
};
// Row constants of the backward for every box of 64 query rows of every
// (sequence, key head). First what the key-side kernel streams:
//  * a [64][16] operand tile (32-byte rows, swizzled) whose columns hold
//    c = -lse / scale of both maps and -D_1, each as three 16-bit terms:
//    2^15 h + 2^4 m + l. One more K step against a constant operand adds them to
//    S_1, S_2 and dP inside the products. The factors are for fp16, whose h ends
//    at 65504: |c| up to 2.1e9 is held, fp32's bits or 2^-25 of it (256 h + m + l
//    ends at 1.7e7, which a row of eight keys passes at scale 1e-7). bf16 holds
//    24 bits by any factors.
//  * D_1 - D_2 and -lambda of each row.
// Then what the query-side kernel reads once: -log2e lse1, -log2e lse2, -D_1,
// -D_2, and where it leaves -sum_k P_2 dP for dlambda. Rows without a query
// hold zeros: their Q and dO are zeros, and so is what they add.
struct DiffRows {
  static constexpr float kHigh = 32768.f, kMiddle = 16.f;   // factors of h and m
  static constexpr int kTile = 64 * 16 * 2;
  static constexpr int kDelta = kTile, kLam = kTile + 256, kStream = kTile + 512;   // bytes streamed
  static constexpr int kL1 = kStream, kL2 = kL1 + 256, kD1 = kL2 + 256, kD2 = kD1 + 256, kSum = kD2 + 256, kBytes = kSum + 256;
};
struct DiffBwdArgs {
  DiffGeom g;
  const void *q1, *q2, *k1, *k2, *v, *lam, *o, *o2, *dO;
  const float* lse;
  void *dq1, *dq2, *dk1, *dk2, *dv, *dlam;
  uint8_t* rows;     // [sequences * key heads][boxes] of DiffRows
  int boxes;         // of one (sequence, key head), an even number
  float* part;       // key-side sums of `splits` shares of the rows, [unit][key tile][split][128][2 d + dv]; null without
  int splits;
  int* err;
};
inline int diff_sequences(const DiffGeom& g) { return g.window ? g.batch * g.nwx * g.nwy : g.batch; }
// The longest sequence's extents and boxes.
inline int diff_span_x(const DiffGeom& g, int len) { return g.window ? (g.window < g.width ? g.window : g.width) : len; }
inline int diff_span_y(const DiffGeom& g) { return g.window ? (g.window < g.height ? g.window : g.height) : 1; }
inline int diff_max_q_boxes(const DiffGeom& g) { return ceil_div(diff_span_x(g, g.q_len), g.tcq) * ceil_div(diff_span_y(g), g.trq); }
inline int diff_max_k_boxes(const DiffGeom& g) { return ceil_div(diff_span_x(g, g.k_len), g.tck) * ceil_div(diff_span_y(g), g.trk); }
// The operand widths of the kernels: the smallest pair that holds d and dv.
inline int diff_class(int d, int dv) { return d <= 16 && dv <= 32 ? 0 : (d <= 32 && dv <= 64 ? 1 : 2); }
// Few query rows over split keys take a form of the kernel that splits them over its warps too.
inline bool diff_few_rows(const DiffGeom& g) { return !g.window && static_cast<long long>(g.q_len) * g.group <= 32; }
int diff_splits(const DiffGeom& g);
size_t diff_split_bytes(const DiffGeom& g);
int diff_bwd_splits(const DiffGeom& g);
size_t diff_bwd_part_bytes(const DiffGeom& g);
// Tensor maps (columns, heads, x, y, batch) of the query and the key side with
// their boxes; `cols` is the width of an operand atom.
bool diff_map(CUtensorMap* map, const DiffGeom& g, bool query, bool f16, const void* p, const DiffStrides& s, int e, int cols);
cudaError_t launch_diff_attn_fwd(const DiffFwdArgs& a, bool f16, cudaStream_t stream);
cudaError_t launch_diff_attn_bwd(const DiffBwdArgs& a, bool f16, cudaStream_t stream);

}  // namespace rib
