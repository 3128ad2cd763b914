// Differential attention, backward (rib_diff_attention_bwd). With
// P_i = softmax(s Q_i K_i^T), O_i = P_i V, O = O_1 - lambda O_2 and
// dP = dO V^T (the same for both maps):
//   D_i = rowsum(dO * O_i),            O_1 = O + lambda O_2
//   dS_1 = P_1 (dP - D_1),             dS_2 = -lambda P_2 (dP - D_2)
//   dQ_i = s dS_i K_i,  dK_i = s dS_i^T Q_i,  dV = (P_1 - lambda P_2)^T dO
//   dlambda = -sum over the head's rows of sum_k P_2 dP
// P_i is formed again from the forward's log-sum-exps. Gradients of a key head
// that several query heads share are sums over its rows, in one accumulator.
//
// Three launches:
//  * rows: D_1, D_2 and the other row constants, box by box of 64 query rows.
//    D comes from the stored O and O_2 in their 16-bit type, half a step of each
//    term, in place of a sum over the keys of P dP (a pass more over the scores).
//  * dq: one CTA owns 128 query rows and streams key boxes of 64. It also sums
//    P_2 dP in fp32, which spares dlambda the rounding of a stored O_2.
//  * dkv: one CTA owns 128 keys of a key head and streams query boxes, keys in
//    the TMEM lanes (S_i^T = K_i Q_i^T); the last CTAs add up dlambda. Per-row
//    constants lie along its columns: reading them for every element took
//    three quarters of the shared-memory pipe, so lse and D_1 enter inside the
//    products, as one more K step. Where the key tiles alone leave SMs idle or
//    a causal mask gives the first ones most of the work, each one's rows are
//    split over CTAs, whose fp32 sums a fourth launch adds. Every sum has one
//    owner and a fixed order: the same bits on every run, no atomics.
// Both recompute S_i and dP: the alternative, one kernel that adds its dQ
// tiles to memory, needs atomics, whose order changes the result.
//
// Roles in both: 16 elementwise warps (thread = TMEM lane; P and dS take the
// 16-bit type for the products, half a step of each), two MMA issuers (scores;
// gradients), a TMA producer, and a warp that clears the rows of a streamed
// box that are not the sequence's.
//
// Bound: the exponentials (2 per pair and kernel, 16 a cycle and SM) at d <= 32;
// with d = 64, dv = 128 the shared-memory bytes of the products' operands (dkv)
// and the chain of products and elementwise work with two tiles in flight (dq).
// Measured: 2x96x96 windows, 6 heads of 16/32: dq 770 us (MUFU 66 %), dkv 861 us
// (60 %), rows 10 us. Causal 2x4001 tokens, 8 query on 2 key heads of 64/128: dq
// 146, dkv 199 (four splits a key tile) and 15 for their join, rows 16 us.
#include <cuda_runtime.h>

#include "diff_attn.cuh"

namespace rib {
namespace {

constexpr int kOwn = 128, kStream = 64;
constexpr int kWarpS = 16, kWarpX = 17, kWarpLoad = 18, kWarpClear = 19;
constexpr int kThreads = 32 * 20;

enum Site : int {
  SITE_RAW = 620, SITE_OWN = 621, SITE_ST_FULL = 622, SITE_ST_EMPTY = 623, SITE_S_FULL = 624, SITE_S_FREE = 625, SITE_X_FULL = 626,
  SITE_X_DONE = 627, SITE_DONE = 628,
};

// fp16 probabilities and their gradients are held times 2^6, which moves
// fp16's smallest normal value to 2^-20 (rows of a million keys) and still
// leaves |P (dP - D)| up to 1023 below its largest; the epilogues divide it
// out. bf16 has fp32's range.
template <bool F16>
constexpr float kShift = F16 ? 6.f : 0.f;
template <bool F16>
constexpr float kUnshift = F16 ? 1.f / 64.f : 1.f;

// All by the MUFU: the polynomial of the forward made both kernels slower (2 of
// 8 pairs: 2.22 -> 2.25 ms for a 2x96x96 training call).
__device__ __forceinline__ uint64_t exp2_pair(uint64_t x) {
  float x0, x1;
  f2_unpack(x, x0, x1);
  return f2_pack(ex2_approx(x0), ex2_approx(x1));
}
template <bool F16>
__device__ __forceinline__ uint32_t pack_pair(uint64_t x) {
  float x0, x1;
  f2_unpack(x, x0, x1);
  return diff_pack<F16>(x0, x1);
}
__device__ __forceinline__ uint64_t raw_pair(const uint32_t* r) { return f2_pack(__uint_as_float(r[0]), __uint_as_float(r[1])); }

// ---------------------------------------------------------------- row constants
// LPR lanes hold a row's eight columns each; a CTA takes rows of one box.
template <int LPR, bool F16>
__global__ void __launch_bounds__(256) diff_attn_rows_kernel(const DiffBwdArgs a) {
  const DiffGeom& g = a.g;
  constexpr int kRows = 256 / LPR;   // 64, 32 or 16
  const long long box_at = static_cast<long long>(blockIdx.x) * kRows / 64;
  const int r6 = static_cast<int>(static_cast<long long>(blockIdx.x) * kRows % 64) + threadIdx.x / LPR, lane = threadIdx.x % LPR;
  const int unit = static_cast<int>(box_at / a.boxes), box = static_cast<int>(box_at - static_cast<long long>(unit) * a.boxes);
  const int hk = unit % g.kv_heads;
  const DiffSeq s = diff_sequence(g, unit / g.kv_heads);
  const DiffRow q = diff_query_row(g, s, box, r6);
  const bool live = q.live;
  const int hq = hk * g.group + (live ? q.head : 0), token = live ? s.token(q.x, q.y) : 0;
  const float lam = diff_lambda<F16>(a.lam, g.lam_f32, hq);
  float d1 = 0.f, d2 = 0.f;
  if (live && lane * 8 < g.dv) {
    const long long at = s.b * g.o.b + wide(token, g.o.t) + wide(hq, g.o.h) + lane * 8;
    const uint4 dw = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.dO) + at);
    const uint4 ow = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.o) + at);
    const uint4 pw = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.o2) + at);
    const uint32_t dd[4] = {dw.x, dw.y, dw.z, dw.w}, oo[4] = {ow.x, ow.y, ow.z, ow.w}, pp[4] = {pw.x, pw.y, pw.z, pw.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float x0 = diff_lo<F16>(dd[e]), x1 = diff_hi<F16>(dd[e]);
      const float q0 = diff_lo<F16>(pp[e]), q1 = diff_hi<F16>(pp[e]);
      d1 = fmaf(x0, fmaf(lam, q0, diff_lo<F16>(oo[e])), d1);
      d1 = fmaf(x1, fmaf(lam, q1, diff_hi<F16>(oo[e])), d1);
      d2 = fmaf(x0, q0, d2);
      d2 = fmaf(x1, q1, d2);
    }
  }
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) {
    d1 += __shfl_xor_sync(0xFFFFFFFFu, d1, o);
    d2 += __shfl_xor_sync(0xFFFFFFFFu, d2, o);
  }
  if (lane != 0) return;
  // a row that saw nothing (lse -inf) is masked wherever it is met: any finite value will do
  float l[2] = {0.f, 0.f};
  if (live)
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const float v = a.lse[((static_cast<long long>(m) * g.batch + s.b) * g.q_heads + hq) * g.q_len + token];
      if (v != -INFINITY) l[m] = fmaf(-kDiffLog2e, v, kShift<F16>);
    }
  uint8_t* w = a.rows + box_at * DiffRows::kBytes;
  const auto put = [&](int at, float v) { *reinterpret_cast<float*>(w + at + 4 * r6) = v; };
  put(DiffRows::kDelta, d1 - d2);
  put(DiffRows::kLam, live ? -lam : 0.f);
  put(DiffRows::kL1, l[0]);
  put(DiffRows::kL2, l[1]);
  put(DiffRows::kD1, -d1);
  put(DiffRows::kD2, -d2);
  put(DiffRows::kSum, 0.f);
  // x = 2^15 h + 2^4 m + r in the operand type, each term the rounding of what is left
  const auto terms = [](float x, float& h, float& m, float& r) {
    h = diff_lo<F16>(diff_pack<F16>(x * (1.f / DiffRows::kHigh), 0.f));
    const float y = fmaf(-DiffRows::kHigh, h, x);
    m = diff_lo<F16>(diff_pack<F16>(y * (1.f / DiffRows::kMiddle), 0.f));
    r = fmaf(-DiffRows::kMiddle, m, y);
  };
  const float inv = 1.f / g.scale_log2;
  float t[9];
  terms(l[0] * inv, t[0], t[1], t[2]);
  terms(l[1] * inv, t[3], t[4], t[5]);
  terms(-d1, t[6], t[7], t[8]);
  using TT = DiffTile<64, 16>;
  *reinterpret_cast<uint4*>(w + TT::offset(r6, 0)) = make_uint4(diff_pack<F16>(t[0], t[1]), diff_pack<F16>(t[2], t[3]), diff_pack<F16>(t[4], t[5]),
                                                              diff_pack<F16>(t[6], t[7]));
  *reinterpret_cast<uint4*>(w + TT::offset(r6, 1)) = make_uint4(diff_pack<F16>(t[8], 0.f), 0u, 0u, 0u);
}

// ------------------------------------------------------------------- dQ kernel
template <int D, int DV>
struct DqLay {
  using TQ = DiffTile<kOwn, D>;
  using TO = DiffTile<kOwn, DV>;
  using TK = DiffTile<kStream, D>;
  using TV = DiffTile<kStream, DV>;
  static constexpr int OWN = 2 * TQ::BYTES + TO::BYTES;
  static constexpr int STAGE = 2 * TK::BYTES + TV::BYTES;
  static constexpr int NS = 4;
  static constexpr int OFF_ST = OWN;
  static constexpr int OFF_SUM = OFF_ST + NS * STAGE;  // [4][128] fp32: sums of P_2 dP
  static constexpr int OFF_BAR = OFF_SUM + 4 * 128 * 4;
  static constexpr int NBAR = 1 + 3 * NS + 6 + 1;      // own, st_full, st_empty, raw, s_full[2], x_full[2], x_done[2], done
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
  static constexpr int ALLOC = OFF_MISC + 16 + 1024;
  // Two buffers of S_1, S_2, dP (64 columns each); dS_i overwrites the first
  // half of each 32 columns of S_i. Columns of its own for dS, with S freed as
  // soon as it was in registers, cost more in barriers than they saved (0.87
  // for 0.77 ms at 2x96x96).
  static constexpr uint32_t BUF = 192, Q1 = 384, Q2 = 448, COLS = 512;
};

template <int D, int DV, bool F16>
__global__ void __launch_bounds__(kThreads, 1)
diff_attn_dq_kernel(const __grid_constant__ CUtensorMap tm_q1, const __grid_constant__ CUtensorMap tm_q2,
                    const __grid_constant__ CUtensorMap tm_do, const __grid_constant__ CUtensorMap tm_k1,
                    const __grid_constant__ CUtensorMap tm_k2, const __grid_constant__ CUtensorMap tm_v, const DiffBwdArgs a, int q_tiles) {
  using Lay = DqLay<D, DV>;
  using TQ = typename Lay::TQ;
  using TO = typename Lay::TO;
  using TK = typename Lay::TK;
  using TV = typename Lay::TV;
  constexpr int NS = Lay::NS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align_smem_1024(smem_raw);
  uint64_t* own = reinterpret_cast<uint64_t*>(smem + Lay::OFF_BAR);
  uint64_t* st_full = own + 1;
  uint64_t* st_empty = st_full + NS;
  uint64_t* raw = st_empty + NS;
  uint64_t* s_full = raw + NS;
  uint64_t* x_full = s_full + 2;
  uint64_t* x_done = s_full + 4;
  uint64_t* done = s_full + 6;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + Lay::OFF_MISC);
  volatile uint32_t* abort_flag = tmem_holder + 1;
  const DiffGeom& g = a.g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  int u = blockIdx.x;
  const int qt = g.causal ? q_tiles - 1 - u % q_tiles : u % q_tiles;   // most keys first
  u /= q_tiles;
  const int unit = u, hk = u % g.kv_heads;
  const DiffSeq s = diff_sequence(g, u / g.kv_heads);
  const int q_boxes = diff_q_boxes(g, s);
  if (2 * qt >= q_boxes) return;
  const int k_nx = g.causal ? ceil_div(diff_visible(g, s, min((2 * qt + 2) * g.tcq, s.wq) - 1), g.tck) : ceil_div(s.wk, g.tck);
  const int n = k_nx * ceil_div(s.hk, g.trk);
  const bool cut = s.wk % g.tck || s.hk % g.trk;
  const bool clear = cut && (g.window || g.k_lens);

  if (threadIdx.x == 0) {
    mbar_init(own, 1);
    for (int i = 0; i < NS; ++i) {
      mbar_init(&st_full[i], 1);
      mbar_init(&raw[i], 1);
      mbar_init(&st_empty[i], 2);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&x_full[i], 8);
      mbar_init(&x_done[i], 1);
    }
    mbar_init(done, 2);
    tmem_holder[1] = 0u;
    tmem_holder[2] = 0u;
    fence_barrier_init();
  }
  // The tensor maps are fetched while TMEM is allocated: training 2x96x96 2167 -> 2158 us.
  if (warp == kWarpLoad && lane == 0) {
    tma_prefetch_desc(&tm_q1);
    tma_prefetch_desc(&tm_q2);
    tma_prefetch_desc(&tm_do);
    tma_prefetch_desc(&tm_k1);
    tma_prefetch_desc(&tm_k2);
    tma_prefetch_desc(&tm_v);
  }
  if (warp == kWarpS) {
    tmem_alloc(tmem_holder, Lay::COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const WaitCtx wc{abort_flag, a.err};
  const WaitCtx drain{tmem_holder + 2, a.err};
  const uint32_t so = smem_u32(smem), sst = so + Lay::OFF_ST;

  if (warp == kWarpLoad) {
    // --------------------------------------------------------- TMA producer
    if (lane == 0 && n > 0) {
      const int nx_q = ceil_div(s.wq, g.tcq), halves = min(2, q_boxes - 2 * qt), q_rows = g.tcq * g.trq * g.group;
      mbar_arrive_expect_tx(own, halves * (2 * TQ::box_bytes(q_rows) + TO::box_bytes(q_rows)));
      for (int h = 0; h < halves; ++h) {
        const int box = 2 * qt + h, by = box / nx_q, x = s.x0 + (box - by * nx_q) * g.tcq, y = s.y0 + by * g.trq;
        TQ::load(smem, 64 * h, &tm_q1, own, hk * g.group, x, y, s.b);
        TQ::load(smem + TQ::BYTES, 64 * h, &tm_q2, own, hk * g.group, x, y, s.b);
        TO::load(smem + 2 * TQ::BYTES, 64 * h, &tm_do, own, hk * g.group, x, y, s.b);
      }
      const uint32_t bytes = 2 * TK::box_bytes(kStream) + TV::box_bytes(kStream);
      int bx = 0, by = 0, issued = 0;
      uint64_t* to_full = clear ? raw : st_full;
      for (int i = 0; i < n; ++i) {
        const int st = i % NS;
        if (i >= NS && !mbar_wait(&st_empty[st], ((i / NS) - 1) & 1, wc, SITE_ST_EMPTY)) break;
        uint8_t* to = smem + Lay::OFF_ST + st * Lay::STAGE;
        const int x = s.x0 + bx * g.tck, y = s.y0 + by * g.trk;
        mbar_arrive_expect_tx(&to_full[st], bytes);
        TK::load(to, 0, &tm_k1, &to_full[st], hk, x, y, s.b);
        TK::load(to + TK::BYTES, 0, &tm_k2, &to_full[st], hk, x, y, s.b);
        TV::load(to + 2 * TK::BYTES, 0, &tm_v, &to_full[st], hk, x, y, s.b);
        issued = i + 1;
        if (++bx == k_nx) {
          bx = 0;
          ++by;
        }
      }
      mbar_wait(own, 0, drain, SITE_DONE);
      for (int i = max(0, issued - NS); i < issued; ++i) mbar_wait(&to_full[i % NS], (i / NS) & 1, drain, SITE_DONE);
    }
  } else if (warp == kWarpClear) {
    if (clear)
      for (int i = 0; i < n; ++i) {
        const int st = i % NS;
        if (!warp_wait(&raw[st], (i / NS) & 1, wc, SITE_RAW)) break;
        const DiffKeyBox k = diff_key_box(g, s, k_nx, i);
        const uint64_t mask = diff_key_mask(g, k.vx, k.vy);
        uint8_t* to = smem + Lay::OFF_ST + st * Lay::STAGE;
        if (mask != ~0ull) {
          diff_clear_rows<kStream, D, DV>(to, ~mask, lane);
          fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&st_full[st]);
      }
  } else if (warp == kWarpS || warp == kWarpX) {
    // two MMA issuers: the scores and dP, and the gradients
    if (n > 0) {
      const uint32_t id_s = diff_idesc(F16, kStream, false);
      const uint32_t id_q = diff_idesc(F16, (g.d + 15) / 16 * 16, true);
      const uint64_t q1 = TQ::kmajor(so), q2 = TQ::kmajor(so + TQ::BYTES), dO = TO::kmajor(so + 2 * TQ::BYTES);
      const uint64_t kk = TK::kmajor(sst), kv = TV::kmajor(sst + 2 * TK::BYTES), km = TK::mnmajor(sst);
      bool ok = warp_wait(own, 0, wc, SITE_OWN);
      int st = 0;
      uint32_t lap = 0;
      for (int j = 0; ok && j < n; ++j) {
        const int bb = j & 1;
        const uint32_t at = static_cast<uint32_t>(st) * (Lay::STAGE >> 4), t = tmem + Lay::BUF * bb;
        if (warp == kWarpS) {
          ok = warp_wait(&st_full[st], lap, wc, SITE_ST_FULL);
          if (ok && j >= 2) ok = warp_wait(&x_done[bb], ((j - 2) >> 1) & 1, wc, SITE_X_DONE);
          if (ok && elect_one()) {
            tc_fence_after();
            diff_mma_kk<TQ, TK, D / 16>(t, q1, kk + at, id_s);
            diff_mma_kk<TQ, TK, D / 16>(t + 64, q2, kk + at + (TK::BYTES >> 4), id_s);
            diff_mma_kk<TO, TV, DV / 16>(t + 128, dO, kv + at, id_s);
            umma_commit(&s_full[bb]);
            umma_commit(&st_empty[st]);
          }
        } else {
          ok = warp_wait(&x_full[bb], (j >> 1) & 1, wc, SITE_X_FULL);
          if (ok && elect_one()) {
            tc_fence_after();
            const uint32_t acc = j > 0 ? 1u : 0u;
#pragma unroll
            for (int ks = 0; ks < kStream / 16; ++ks)
              umma_ts(tmem + Lay::Q1, t + 32u * (ks >> 1) + 8u * (ks & 1), km + at + TK::mnstep(ks), id_q, ks > 0 ? 1u : acc);
#pragma unroll
            for (int ks = 0; ks < kStream / 16; ++ks)
              umma_ts(tmem + Lay::Q2, t + 64 + 32u * (ks >> 1) + 8u * (ks & 1), km + at + (TK::BYTES >> 4) + TK::mnstep(ks), id_q,
                      ks > 0 ? 1u : acc);
            umma_commit(&x_done[bb]);
            umma_commit(&st_empty[st]);
          }
        }
        __syncwarp();
        if (++st == NS) {
          st = 0;
          lap ^= 1u;
        }
      }
      if (elect_one()) umma_commit(done);
      warp_wait(done, 0, drain, SITE_DONE);
    }
  } else {
    // elementwise: warpgroup (p, h) takes columns 32 h .. of the tiles j = p, p + 2, ...; thread = query row
    const int w = warp >> 2, p = w >> 1, h = w & 1, row = (warp & 3) * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t t = tmem + lane_off + Lay::BUF * p + 32 * h;
    const DiffRow q = diff_query_row(g, s, 2 * qt + (row >> 6), row & 63);
    uint8_t* c = a.rows + (static_cast<long long>(unit) * a.boxes + 2 * qt + (row >> 6)) * DiffRows::kBytes + 4 * (row & 63);
    const auto get = [&](int at) { return *reinterpret_cast<const float*>(c + at); };
    const float l1 = get(DiffRows::kL1), l2 = get(DiffRows::kL2), d1 = get(DiffRows::kD1), d2 = get(DiffRows::kD2), nlam = get(DiffRows::kLam);
    const int seen = q.live ? diff_visible(g, s, q.x) : 0x7FFFFFFF;
    const bool warp_live = __any_sync(0xFFFFFFFFu, q.live);
    const uint64_t sl2 = f2_pack(g.scale_log2, g.scale_log2), L1 = f2_pack(l1, l1), L2 = f2_pack(l2, l2), D1 = f2_pack(d1, d1), D2 = f2_pack(d2, d2);
    const uint64_t NL = f2_pack(nlam, nlam);
    uint64_t sum = f2_pack(0.f, 0.f);   // of P_2 dP
    bool ok = true;
    for (int j = p; j < n; j += 2) {
      ok = warp_wait(&s_full[p], (j >> 1) & 1, wc, SITE_S_FULL);
      if (!ok) break;
      tc_fence_after();
      if (warp_live) {
        uint32_t hidden = 0u;   // a bit for every column that the row does not see
        if (cut || g.causal) {
          const uint64_t mask = diff_seen(g, s, k_nx, j, seen);
          hidden = ~static_cast<uint32_t>(mask >> (32 * h));
        }
        const bool edge = __any_sync(0xFFFFFFFFu, hidden != 0u);
#pragma unroll
        for (int cc = 0; cc < 2; ++cc) {
          uint32_t s1[16], s2[16], dp[16], x1[8], x2[8];
          tmem_ld16(t + 16 * cc, s1);
          tmem_ld16(t + 64 + 16 * cc, s2);
          tmem_ld16(t + 128 + 16 * cc, dp);
          tmem_wait_ld();
          if (edge) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (hidden & (1u << (16 * cc + i))) s1[i] = s2[i] = 0xFF800000u;   // -inf: P = 0
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint64_t dd = raw_pair(dp + 2 * i);
            const uint64_t y1 = f2_fma(raw_pair(s1 + 2 * i), sl2, L1), y2 = f2_fma(raw_pair(s2 + 2 * i), sl2, L2);
            const uint64_t p1 = exp2_pair(y1), p2 = exp2_pair(y2);
            sum = f2_fma(p2, dd, sum);
            x1[i] = pack_pair<F16>(f2_mul(p1, f2_add(dd, D1)));
            x2[i] = pack_pair<F16>(f2_mul(f2_mul(p2, NL), f2_add(dd, D2)));
          }
          tmem_st8(t + 8 * cc, x1);
          tmem_st8(t + 64 + 8 * cc, x2);
        }
        tmem_wait_st();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&x_full[p]);
    }
    float* sums = reinterpret_cast<float*>(smem + Lay::OFF_SUM);
    float s0, s1;
    f2_unpack(sum, s0, s1);
    sums[w * 128 + row] = s0 + s1;
    if (ok && n > 0) ok = warp_wait(done, 0, wc, SITE_DONE);
    asm volatile("bar.sync 1, 512;" ::: "memory");
    tc_fence_after();
    if (ok && warp_live && *abort_flag == 0u) {
      if (w == 0 && q.live)
        *reinterpret_cast<float*>(c + DiffRows::kSum) = -kUnshift<F16> * ((sums[row] + sums[128 + row]) + (sums[256 + row] + sums[384 + row]));
      // warpgroup (p, h) stores columns h D / 2 .. of dQ_(p + 1); without a key in sight the gradient is zero
      const float f = g.scale * kUnshift<F16>;
      uint16_t* out = static_cast<uint16_t*>(p ? a.dq2 : a.dq1);
      if (q.live) out += s.b * g.q.b + wide(s.token(q.x, q.y), g.q.t) + wide(hk * g.group + q.head, g.q.h);
#pragma unroll
      for (int cc = 0; cc < D / 16; ++cc) {
        const int col = h * (D / 2) + 8 * cc;
        uint32_t v[8], o[4];
        tmem_ld8(tmem + lane_off + (p ? Lay::Q2 : Lay::Q1) + col, v);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 4; ++e)
          o[e] = n > 0 ? diff_pack<F16>(__uint_as_float(v[2 * e]) * f, __uint_as_float(v[2 * e + 1]) * f) : 0u;
        if (q.live && col < g.d) *reinterpret_cast<uint4*>(out + col) = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kWarpS) {
    tc_fence_after();
    tmem_dealloc(tmem, Lay::COLS);
  }
}

// -------------------------------------------------------------- dK / dV kernel
template <int D, int DV>
struct DkvLay {
  using TK = DiffTile<kOwn, D>;
  using TV = DiffTile<kOwn, DV>;
  using TQ = DiffTile<kStream, D>;
  using TO = DiffTile<kStream, DV>;
  using TP = DiffTile<kOwn, kStream>;      // P^T, dS_1^T, dS_2^T: [128 keys][64 query rows]
  // Buffers of the scores and of P^T, dS^T. Two where TMEM holds them (dv <=
  // 64): tiles alternate between two pairs of warpgroups. One at dv = 128: the
  // four warpgroups share a tile and free S as soon as it is in registers.
  static constexpr int NB = DV <= 64 ? 2 : 1;
  static constexpr int PER = 16 * NB;      // query rows of a warpgroup's share
  static constexpr int OWN = 2 * TK::BYTES + TV::BYTES;
  using TA = DiffTile<kOwn, 16>;           // the constant operands of the row constants' K step
  static constexpr int CONSTS = DiffRows::kStream;
  static constexpr int STAGE = (2 * TQ::BYTES + TO::BYTES + CONSTS + 1023) / 1024 * 1024;
  static constexpr int NS = DV <= 64 ? 4 : 3;
  // the constant operands: shared memory, or (dv = 128) 24 spare columns of TMEM
  static constexpr bool A_TMEM = DV > 64;
  static constexpr int OFF_A = OWN;
  static constexpr int OFF_ST = OFF_A + (A_TMEM ? 0 : 3 * TA::BYTES);
  static constexpr int OFF_X = OFF_ST + NS * STAGE;
  static constexpr int X = 3 * TP::BYTES;
  static constexpr int OFF_BAR = OFF_X + NB * X;
  static constexpr int NBAR = 1 + 3 * NS + 8 + 1;   // own, st_full, st_empty, raw, s_full[2], s_free[2], x_full[2], x_free[2], done
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
  static constexpr int ALLOC = OFF_MISC + 16 + 1024;
  static_assert(ALLOC <= 232448, "shared memory of an SM");
  static constexpr uint32_t BUF = 192, S2 = 64, DP = 128, V = BUF * NB, K1 = V + DV, K2 = K1 + D, A = K2 + D, COLS = 512;
  static_assert(A + (A_TMEM ? 24 : 0) <= 512, "TMEM columns");
};

// ONE: a key head of one query head, whose lambda is a constant.
template <int D, int DV, bool F16, bool ONE>
__global__ void __launch_bounds__(kThreads, 1)
diff_attn_dkv_kernel(const __grid_constant__ CUtensorMap tm_q1, const __grid_constant__ CUtensorMap tm_q2,
                     const __grid_constant__ CUtensorMap tm_do, const __grid_constant__ CUtensorMap tm_k1,
                     const __grid_constant__ CUtensorMap tm_k2, const __grid_constant__ CUtensorMap tm_v, const DiffBwdArgs a, int k_tiles,
                     int units) {
  using Lay = DkvLay<D, DV>;
  using TQ = typename Lay::TQ;
  using TO = typename Lay::TO;
  using TK = typename Lay::TK;
  using TV = typename Lay::TV;
  using TP = typename Lay::TP;
  constexpr int NS = Lay::NS, NB = Lay::NB;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align_smem_1024(smem_raw);
  const DiffGeom& g = a.g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // work unit: (sequence, key head), key tile, split of its rows
  const int item = blockIdx.x / a.splits, sp = blockIdx.x - item * a.splits, u = item / k_tiles;
  if (u >= units) {
    // dlambda of one head: its rows' sums over every sequence, each thread a
    // strided share, then a tree
    const int hq = blockIdx.x - units * k_tiles * a.splits, hk = hq / g.group, gh = hq - hk * g.group;
    const int per = g.tcq * g.trq;
    const long long total = static_cast<long long>(units / g.kv_heads) * a.boxes * per;
    float sum = 0.f;
    for (long long i = threadIdx.x; i < total; i += kThreads) {
      const long long box = i / per;
      const int idx = static_cast<int>(i - box * per);
      const long long seq = box / a.boxes;
      sum += *reinterpret_cast<const float*>(a.rows + ((seq * g.kv_heads + hk) * a.boxes + (box - seq * a.boxes)) * DiffRows::kBytes +
                                             DiffRows::kSum + 4 * (idx * g.group + gh));
    }
    float* red = reinterpret_cast<float*>(smem);
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    if (lane == 0) red[warp] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
      float v = 0.f;
      for (int i = 0; i < kThreads / 32; ++i) v += red[i];
      if (g.lam_f32) static_cast<float*>(a.dlam)[hq] = v;
      else static_cast<uint16_t*>(a.dlam)[hq] = static_cast<uint16_t>(diff_pack<F16>(v, 0.f));
    }
    return;
  }
  uint64_t* own = reinterpret_cast<uint64_t*>(smem + Lay::OFF_BAR);
  uint64_t* st_full = own + 1;
  uint64_t* st_empty = st_full + NS;
  uint64_t* raw = st_empty + NS;
  uint64_t* s_full = raw + NS;
  uint64_t* s_free = s_full + 2;
  uint64_t* x_full = s_full + 4;
  uint64_t* x_free = s_full + 6;
  uint64_t* done = s_full + 8;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + Lay::OFF_MISC);
  volatile uint32_t* abort_flag = tmem_holder + 1;
  const int kt = item - u * k_tiles;                    // with a causal mask the first keys have the most rows
  const int unit = u, hk = u % g.kv_heads;
  const DiffSeq s = diff_sequence(g, u / g.kv_heads);
  const int all = g.window ? s.wk : g.k_len;            // keys whose gradients are written
  const int k_nx = ceil_div(all, g.tck), k_boxes = k_nx * ceil_div(s.hk, g.trk);
  if (2 * kt >= k_boxes) return;
  const int q_nx = ceil_div(s.wq, g.tcq), q_boxes = diff_q_boxes(g, s);
  // sequences: the first row that sees one of the keys, and the first from which every row sees them all
  const int key0 = kt * kOwn;
  int first = 0, full = 0;
  if (g.causal) {
    first = min(max(key0 - s.wk + s.wq, 0), s.wq);
    full = min(max(min(key0 + kOwn, s.wk) - 1 - s.wk + s.wq, 0), s.wq);
  }
  const int j_all = g.causal ? first / g.tcq : 0, n_all = !g.window && (key0 >= s.wk || first >= s.wq) ? 0 : q_boxes - j_all;
  const int from_box = static_cast<int>(wide(n_all, sp) / a.splits);
  const int j0 = j_all + from_box, n = static_cast<int>(wide(n_all, sp + 1) / a.splits) - from_box;
  const int q_rows = g.tcq * g.trq * g.group;
  const bool clear = g.window && (s.wq % g.tcq || s.hq % g.trq);   // boxes with another window's rows

  if (threadIdx.x == 0) {
    mbar_init(own, 1);
    for (int i = 0; i < NS; ++i) {
      mbar_init(&st_full[i], 1);
      mbar_init(&raw[i], 1);
      mbar_init(&st_empty[i], 2);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_free[i], 16 / NB);
      mbar_init(&x_full[i], 16 / NB);
      mbar_init(&x_free[i], 1);
    }
    mbar_init(done, 2);
    tmem_holder[1] = 0u;
    tmem_holder[2] = 0u;
    fence_barrier_init();
  }
  if (warp == kWarpLoad && lane == 0) {
    tma_prefetch_desc(&tm_q1);
    tma_prefetch_desc(&tm_q2);
    tma_prefetch_desc(&tm_do);
    tma_prefetch_desc(&tm_k1);
    tma_prefetch_desc(&tm_k2);
    tma_prefetch_desc(&tm_v);
  }
  if (warp == kWarpS) {
    tmem_alloc(tmem_holder, Lay::COLS);
    tmem_relinquish();
  }
  if (q_rows < 64) {
    // rows of a stage that no load writes are zeros
    for (int i = Lay::OFF_ST + threadIdx.x * 16; i < Lay::OFF_X; i += kThreads * 16)
      *reinterpret_cast<uint4*>(smem + i) = make_uint4(0u, 0u, 0u, 0u);
  }
  // three [128][16] operands, every row alike: the terms' factors in the columns of S_1's, S_2's and dP's
  const auto constant = [](int which, int c) {
    const auto at = [&](int i) {
      return i == 3 * which ? DiffRows::kHigh : (i == 3 * which + 1 ? DiffRows::kMiddle : (i == 3 * which + 2 ? 1.f : 0.f));
    };
    return diff_pack<F16>(at(c), at(c + 1));
  };
  if (!Lay::A_TMEM)
    for (int i = threadIdx.x; i < 3 * kOwn * 2; i += kThreads) {
      const int which = i / (kOwn * 2), r = i / 2 % kOwn, c = 8 * (i & 1);
      *reinterpret_cast<uint4*>(smem + Lay::OFF_A + which * Lay::TA::BYTES + Lay::TA::offset(r, i & 1)) =
          make_uint4(constant(which, c), constant(which, c + 2), constant(which, c + 4), constant(which, c + 6));
    }
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  if (Lay::A_TMEM) {
    if (warp < 4) {
      for (int which = 0; which < 3; ++which) {
        uint32_t w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = constant(which, 2 * e);
        tmem_st8(tmem + (static_cast<uint32_t>(warp * 32) << 16) + Lay::A + 8 * which, w);
      }
      tmem_wait_st();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
  }
  const WaitCtx wc{abort_flag, a.err};
  const WaitCtx drain{tmem_holder + 2, a.err};
  const uint32_t so = smem_u32(smem), sst = so + Lay::OFF_ST, sx = so + Lay::OFF_X;

  if (warp == kWarpLoad) {
    // --------------------------------------------------------- TMA producer
    if (lane == 0 && n > 0) {
      const int halves = min(2, k_boxes - 2 * kt);
      mbar_arrive_expect_tx(own, halves * (2 * TK::box_bytes(64) + TV::box_bytes(64)));
      for (int h = 0; h < halves; ++h) {
        const int box = 2 * kt + h, by = box / k_nx, x = s.x0 + (box - by * k_nx) * g.tck, y = s.y0 + by * g.trk;
        TK::load(smem, 64 * h, &tm_k1, own, hk, x, y, s.b);
        TK::load(smem + TK::BYTES, 64 * h, &tm_k2, own, hk, x, y, s.b);
        TV::load(smem + 2 * TK::BYTES, 64 * h, &tm_v, own, hk, x, y, s.b);
      }
      const uint32_t bytes = 2 * TQ::box_bytes(q_rows) + TO::box_bytes(q_rows) + Lay::CONSTS;
      const uint8_t* consts = a.rows + (static_cast<long long>(unit) * a.boxes + j0) * DiffRows::kBytes;
      int by = j0 / q_nx, bx = j0 - by * q_nx, issued = 0;
      uint64_t* to_full = clear ? raw : st_full;
      for (int i = 0; i < n; ++i) {
        const int st = i % NS;
        if (i >= NS && !mbar_wait(&st_empty[st], ((i / NS) - 1) & 1, wc, SITE_ST_EMPTY)) break;
        uint8_t* to = smem + Lay::OFF_ST + st * Lay::STAGE;
        const int x = s.x0 + bx * g.tcq, y = s.y0 + by * g.trq;
        mbar_arrive_expect_tx(&to_full[st], bytes);
        TQ::load(to, 0, &tm_q1, &to_full[st], hk * g.group, x, y, s.b);
        TQ::load(to + TQ::BYTES, 0, &tm_q2, &to_full[st], hk * g.group, x, y, s.b);
        TO::load(to + 2 * TQ::BYTES, 0, &tm_do, &to_full[st], hk * g.group, x, y, s.b);
        bulk_load(to + 2 * TQ::BYTES + TO::BYTES, consts + static_cast<long long>(i) * DiffRows::kBytes, Lay::CONSTS, &to_full[st]);
        issued = i + 1;
        if (++bx == q_nx) {
          bx = 0;
          ++by;
        }
      }
      mbar_wait(own, 0, drain, SITE_DONE);
      for (int i = max(0, issued - NS); i < issued; ++i) mbar_wait(&to_full[i % NS], (i / NS) & 1, drain, SITE_DONE);
    }
  } else if (warp == kWarpClear) {
    if (clear)
      for (int i = 0; i < n; ++i) {
        const int st = i % NS;
        if (!warp_wait(&raw[st], (i / NS) & 1, wc, SITE_RAW)) break;
        const int by = (j0 + i) / q_nx, vx = s.wq - (j0 + i - by * q_nx) * g.tcq, vy = s.hq - by * g.trq;
        uint8_t* to = smem + Lay::OFF_ST + st * Lay::STAGE;
        if (vx < g.tcq || vy < g.trq) {
          // rows that the load brought and that are not the window's
          uint64_t dead = 0ull;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int row = 32 * h + lane;
            const uint32_t bits = __ballot_sync(0xFFFFFFFFu, row < q_rows && !diff_query_row(g, s, j0 + i, row).live);
            dead |= static_cast<uint64_t>(bits) << (32 * h);
          }
          diff_clear_rows<kStream, D, DV>(to, dead, lane);
          fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&st_full[st]);
      }
  } else if (warp == kWarpS || warp == kWarpX) {
    if (n > 0) {
      const uint32_t id_s = diff_idesc(F16, kStream, false);
      const uint32_t id_k = diff_idesc(F16, (g.d + 15) / 16 * 16, true), id_v = diff_idesc(F16, (g.dv + 15) / 16 * 16, true);
      const uint64_t k1 = TK::kmajor(so), k2 = TK::kmajor(so + TK::BYTES), v = TV::kmajor(so + 2 * TK::BYTES), x = TP::kmajor(sx);
      using TC = DiffTile<kStream, 16>;
      const uint64_t ca = Lay::TA::kmajor(so + Lay::OFF_A), cb = TC::kmajor(sst + 2 * TQ::BYTES + TO::BYTES);
      const auto add_constants = [&](uint32_t d, int which, uint64_t b) {
        if constexpr (Lay::A_TMEM) umma_ts(d, tmem + Lay::A + 8 * which, b, id_s, 1u);
        else umma_ss(d, ca + static_cast<uint32_t>(which) * (Lay::TA::BYTES >> 4), b, id_s, 1u);
      };
      const uint64_t qk = TQ::kmajor(sst), dk = TO::kmajor(sst + 2 * TQ::BYTES), qm = TQ::mnmajor(sst), dm = TO::mnmajor(sst + 2 * TQ::BYTES);
      bool ok = warp_wait(own, 0, wc, SITE_OWN);
      int st = 0;
      uint32_t lap = 0;
      for (int j = 0; ok && j < n; ++j) {
        const int bb = NB == 2 ? j & 1 : 0, round = NB == 2 ? j >> 1 : j;
        const uint32_t at = static_cast<uint32_t>(st) * (Lay::STAGE >> 4);
        if (warp == kWarpS) {
          const uint32_t t = tmem + Lay::BUF * bb;
          ok = warp_wait(&st_full[st], lap, wc, SITE_ST_FULL);
          if (ok && round >= 1) ok = warp_wait(&s_free[bb], (round - 1) & 1, wc, SITE_S_FREE);
          if (ok && elect_one()) {
            tc_fence_after();
            diff_mma_kk<TK, TQ, D / 16>(t, k1, qk + at, id_s);
            add_constants(t, 0, cb + at);
            diff_mma_kk<TK, TQ, D / 16>(t + Lay::S2, k2, qk + at + (TQ::BYTES >> 4), id_s);
            add_constants(t + Lay::S2, 1, cb + at);
            diff_mma_kk<TV, TO, DV / 16>(t + Lay::DP, v, dk + at, id_s);
            add_constants(t + Lay::DP, 2, cb + at);
            umma_commit(&s_full[bb]);
            umma_commit(&st_empty[st]);
          }
        } else {
          ok = warp_wait(&x_full[bb], round & 1, wc, SITE_X_FULL);
          if (ok && elect_one()) {
            tc_fence_after();
            const uint64_t xb = x + static_cast<uint32_t>(bb) * (Lay::X >> 4);
            const uint32_t acc0 = j > 0 ? 1u : 0u;
#pragma unroll
            for (int ks = 0; ks < kStream / 16; ++ks) {
              const uint32_t acc = ks > 0 ? 1u : acc0;
              umma_ss(tmem + Lay::V, xb + TP::kstep(ks), dm + at + TO::mnstep(ks), id_v, acc);
              umma_ss(tmem + Lay::K1, xb + (TP::BYTES >> 4) + TP::kstep(ks), qm + at + TQ::mnstep(ks), id_k, acc);
              umma_ss(tmem + Lay::K2, xb + 2 * (TP::BYTES >> 4) + TP::kstep(ks), qm + at + (TQ::BYTES >> 4) + TQ::mnstep(ks), id_k, acc);
            }
            umma_commit(&x_free[bb]);
            umma_commit(&st_empty[st]);
          }
        }
        __syncwarp();
        if (++st == NS) {
          st = 0;
          lap ^= 1u;
        }
      }
      if (elect_one()) umma_commit(done);
      warp_wait(done, 0, drain, SITE_DONE);
    }
  } else {
    // elementwise: thread = key = TMEM lane; warpgroup w takes PER query rows of its tiles
    const int w = warp >> 2, p = NB == 2 ? w >> 1 : 0, part = NB == 2 ? w & 1 : w;
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t t = tmem + lane_off + Lay::BUF * p + Lay::PER * part;
    const uint64_t sl2 = f2_pack(g.scale_log2, g.scale_log2);
    const int key = key0 + row;   // of a causal sequence
    const float nl = ONE ? -diff_lambda<F16>(a.lam, g.lam_f32, hk) : 0.f;
    const ulonglong2 nlam = {f2_pack(nl, nl), f2_pack(nl, nl)};
    bool ok = true;
    for (int j = p; j < n; j += NB) {
      const int st = j % NS, round = NB == 2 ? j >> 1 : j;
      ok = warp_wait(&st_full[st], (j / NS) & 1, wc, SITE_ST_FULL);   // the row constants
      ok = ok && warp_wait(&s_full[p], round & 1, wc, SITE_S_FULL);
      if (!ok) break;
      tc_fence_after();
      const float* cs = reinterpret_cast<const float*>(smem + Lay::OFF_ST + st * Lay::STAGE + 2 * TQ::BYTES + TO::BYTES + DiffRows::kDelta) +
                        Lay::PER * part;   // D_1 - D_2; -lambda 64 further
      const int x0 = (j0 + j) * g.tcq;                 // first query of the box
      const bool edge = g.causal && x0 < full;
#pragma unroll
      for (int cc = 0; cc < NB; ++cc) {
        uint32_t s1[16], s2[16], dp[16];
        tmem_ld16(t + 16 * cc, s1);
        tmem_ld16(t + Lay::S2 + 16 * cc, s2);
        tmem_ld16(t + Lay::DP + 16 * cc, dp);
        tmem_wait_ld();
        if (cc == NB - 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s_free[p]);   // the next products may overwrite them
        }
        if (edge) {
          // query x sees the keys up to x + wk - wq
          const int from = key - s.wk + s.wq - x0;   // the first query of the box that sees this key
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int r6 = Lay::PER * part + 16 * cc + i, x = g.group_magic ? div_by(r6, g.group_magic) : r6;
            if (x < from) s1[i] = s2[i] = 0xFF800000u;   // -inf: P = 0
          }
        }
        uint8_t* to = smem + Lay::OFF_X + p * Lay::X;
#pragma unroll
        for (int q = 0; q < 2; ++q) {   // eight query rows: 16 bytes of each operand row
          uint32_t pp[4], x1[4], x2[4];
#pragma unroll
          for (int e = 0; e < 2; ++e) {   // four rows' constants a load
            const int i = 8 * q + 4 * e;
            const ulonglong2* quad = reinterpret_cast<const ulonglong2*>(cs + 16 * cc + i);
            const ulonglong2 DD = quad[0];
            const ulonglong2 NL = ONE ? nlam : quad[16];
#pragma unroll
            for (int f = 0; f < 2; ++f) {
              const int at = i + 2 * f;
              const uint64_t t1 = raw_pair(dp + at);
              const uint64_t y1 = f2_mul(raw_pair(s1 + at), sl2), y2 = f2_mul(raw_pair(s2 + at), sl2);
              const uint64_t p1 = exp2_pair(y1), p2 = f2_mul(exp2_pair(y2), f ? NL.y : NL.x);
              pp[2 * e + f] = pack_pair<F16>(f2_add(p1, p2));
              x1[2 * e + f] = pack_pair<F16>(f2_mul(p1, t1));
              x2[2 * e + f] = pack_pair<F16>(f2_mul(p2, f2_add(t1, f ? DD.y : DD.x)));
            }
          }
          if (cc == 0 && q == 0 && round >= 1) {
            // the products of the buffer's tile before have read P^T and dS^T
            ok = warp_wait(&x_free[p], (round - 1) & 1, wc, SITE_X_DONE);
            if (!ok) break;
          }
          uint8_t* at = to + TP::offset(row, (Lay::PER * part + 16 * cc) / 8 + q);
          *reinterpret_cast<uint4*>(at) = make_uint4(pp[0], pp[1], pp[2], pp[3]);
          *reinterpret_cast<uint4*>(at + TP::BYTES) = make_uint4(x1[0], x1[1], x1[2], x1[3]);
          *reinterpret_cast<uint4*>(at + 2 * TP::BYTES) = make_uint4(x2[0], x2[1], x2[2], x2[3]);
        }
        if (!ok) break;
      }
      if (!ok) break;
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&x_full[p]);
    }
    if (ok && n > 0) ok = warp_wait(done, 0, wc, SITE_DONE);
    tc_fence_after();
    if (ok && *abort_flag == 0u) {
      // this lane's key
      const int box = 2 * kt + (row >> 6), c = row & 63, by = box / k_nx;
      const int x = (box - by * k_nx) * g.tck + (c & (g.tck - 1)), y = by * g.trk + (c >> g.lk);
      const bool live = x < all && y < s.hk, real = n > 0 && x < s.wk;   // keys behind the length have gradient zero
      const int token = live ? s.token(x, y) : 0;
      // warpgroup w stores its quarter of the columns of each gradient: results, or this split's sums
      const int width_all = 2 * g.d + g.dv;
      float* part = a.part ? a.part + (static_cast<long long>(blockIdx.x) * kOwn + row) * width_all : nullptr;
      auto store = [&](uint32_t col, int cols, uint16_t* out, int width, float f, int at) {
        const int share = cols >= 32 ? cols / 4 : 8;
        for (int c0 = w * share; c0 < min(cols, (w + 1) * share); c0 += 8) {
          uint32_t v[8], o[4];
          tmem_ld8(tmem + lane_off + col + c0, v);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = real ? __float_as_uint(__uint_as_float(v[e]) * f) : 0u;
          if (c0 >= width) continue;
          if (part) {
            *reinterpret_cast<uint4*>(part + at + c0) = make_uint4(v[0], v[1], v[2], v[3]);
            *reinterpret_cast<uint4*>(part + at + c0 + 4) = make_uint4(v[4], v[5], v[6], v[7]);
            continue;
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) o[e] = diff_pack<F16>(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1]));
          if (live) *reinterpret_cast<uint4*>(out + c0) = make_uint4(o[0], o[1], o[2], o[3]);
        }
      };
      const long long kv = s.b * g.v.b + wide(token, g.v.t) + wide(hk, g.v.h), kk = s.b * g.k.b + wide(token, g.k.t) + wide(hk, g.k.h);
      store(Lay::V, DV, static_cast<uint16_t*>(a.dv) + kv, g.dv, kUnshift<F16>, 2 * g.d);
      store(Lay::K1, D, static_cast<uint16_t*>(a.dk1) + kk, g.d, g.scale * kUnshift<F16>, 0);
      store(Lay::K2, D, static_cast<uint16_t*>(a.dk2) + kk, g.d, g.scale * kUnshift<F16>, g.d);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kWarpS) {
    tc_fence_after();
    tmem_dealloc(tmem, Lay::COLS);
  }
}

// The splits' sums of one key row, in their order; a thread owns eight columns.
template <bool F16>
__global__ void __launch_bounds__(256) diff_attn_dkv_join_kernel(const DiffBwdArgs a, int k_tiles, long long threads) {
  const DiffGeom& g = a.g;
  const long long at = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  if (at >= threads) return;
  const int width = 2 * g.d + g.dv, pieces = width / 8;
  const long long row_at = at / pieces;
  const int c = static_cast<int>(at - row_at * pieces) * 8, row = static_cast<int>(row_at % kOwn);
  const long long tile = row_at / kOwn;
  const int unit = static_cast<int>(tile / k_tiles), kt = static_cast<int>(tile - static_cast<long long>(unit) * k_tiles), hk = unit % g.kv_heads;
  const DiffSeq s = diff_sequence(g, unit / g.kv_heads);
  const int all = g.window ? s.wk : g.k_len, k_nx = ceil_div(all, g.tck);
  const int box = 2 * kt + (row >> 6), cc = row & 63, by = box / k_nx;
  const int x = (box - by * k_nx) * g.tck + (cc & (g.tck - 1)), y = by * g.trk + (cc >> g.lk);
  if (x >= all || y >= s.hk) return;
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  const float* p = a.part + (tile * a.splits * kOwn + row) * width + c;
  for (int i = 0; i < a.splits; ++i, p += static_cast<long long>(kOwn) * width) {
    const float4 lo = reinterpret_cast<const float4*>(p)[0], hi = reinterpret_cast<const float4*>(p)[1];
    v[0] += lo.x; v[1] += lo.y; v[2] += lo.z; v[3] += lo.w;
    v[4] += hi.x; v[5] += hi.y; v[6] += hi.z; v[7] += hi.w;
  }
  const int token = s.token(x, y);
  const long long kk = s.b * g.k.b + wide(token, g.k.t) + wide(hk, g.k.h);
  uint16_t* out = c < g.d       ? static_cast<uint16_t*>(a.dk1) + kk + c
                  : c < 2 * g.d ? static_cast<uint16_t*>(a.dk2) + kk + c - g.d
                                : static_cast<uint16_t*>(a.dv) + s.b * g.v.b + wide(token, g.v.t) + wide(hk, g.v.h) + c - 2 * g.d;
  *reinterpret_cast<uint4*>(out) =
      make_uint4(diff_pack<F16>(v[0], v[1]), diff_pack<F16>(v[2], v[3]), diff_pack<F16>(v[4], v[5]), diff_pack<F16>(v[6], v[7]));
}

template <int D, int DV, bool F16>
cudaError_t launch_class(const DiffBwdArgs& a, cudaStream_t stream) {
  const DiffGeom& g = a.g;
  const long long units = static_cast<long long>(diff_sequences(g)) * g.kv_heads;
  const int q_tiles = a.boxes / 2, k_tiles = ceil_div(diff_max_k_boxes(g), 2);
  constexpr int LPR = DV / 8;
  const long long row_ctas = units * a.boxes * LPR / 4, q_ctas = units * q_tiles, k_ctas = units * k_tiles * a.splits + g.q_heads;
  if (row_ctas > 0x7FFFFFFFll || q_ctas > 0x7FFFFFFFll || k_ctas > 0x7FFFFFFFll) return cudaErrorInvalidConfiguration;
  using TK = DiffTile<kOwn, D>;
  using TV = DiffTile<kOwn, DV>;
  CUtensorMap q1, q2, dO, k1, k2, v;
  if (!diff_map(&q1, g, true, F16, a.q1, g.q, g.d, TK::COLS) || !diff_map(&q2, g, true, F16, a.q2, g.q, g.d, TK::COLS) ||
      !diff_map(&dO, g, true, F16, a.dO, g.o, g.dv, TV::COLS) || !diff_map(&k1, g, false, F16, a.k1, g.k, g.d, TK::COLS) ||
      !diff_map(&k2, g, false, F16, a.k2, g.k, g.d, TK::COLS) || !diff_map(&v, g, false, F16, a.v, g.v, g.dv, TV::COLS))
    return cudaErrorInvalidValue;
  auto dq = diff_attn_dq_kernel<D, DV, F16>;
  auto dkv = g.group == 1 ? diff_attn_dkv_kernel<D, DV, F16, true> : diff_attn_dkv_kernel<D, DV, F16, false>;
  cudaError_t e = cudaFuncSetAttribute(dq, cudaFuncAttributeMaxDynamicSharedMemorySize, DqLay<D, DV>::ALLOC);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(dkv, cudaFuncAttributeMaxDynamicSharedMemorySize, DkvLay<D, DV>::ALLOC);
  if (e != cudaSuccess) return e;
  if (row_ctas > 0) {
    diff_attn_rows_kernel<LPR, F16><<<static_cast<unsigned>(row_ctas), 256, 0, stream>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    dq<<<static_cast<unsigned>(q_ctas), kThreads, DqLay<D, DV>::ALLOC, stream>>>(q1, q2, dO, k1, k2, v, a, q_tiles);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  // k_tiles 0: dlambda alone, with no tiles before it
  dkv<<<static_cast<unsigned>(k_ctas), kThreads, DkvLay<D, DV>::ALLOC, stream>>>(q1, q2, dO, k1, k2, v, a, k_tiles > 0 ? k_tiles : 1,
                                                                               k_tiles > 0 ? static_cast<int>(units) : 0);
  if ((e = cudaGetLastError()) != cudaSuccess || !a.part) return e;
  const long long threads = units * k_tiles * kOwn * ((2 * g.d + g.dv) / 8);
  if (threads <= 0) return cudaSuccess;
  diff_attn_dkv_join_kernel<F16><<<static_cast<unsigned>((threads + 255) / 256), 256, 0, stream>>>(a, k_tiles, threads);
  return cudaGetLastError();
}

}  // namespace

// Shares of a key tile's rows, of eight boxes at least; one where there are
// three key tiles an SM. Measured, in us of a whole backward by the number of shares:
//   2 x 4001 causal, 8 on 2 heads of 64/128    475 (1)  404 (2)  377 (3)  352 (4)  383 (6)  416 (8)
//   8192 causal, 2 heads of 32/64              262 (1)  213 (2)  225 (3)  227 (4)  244 (6)
//   4096 causal, 4 heads of 64/128             170 (1)  172 (2)  168 (3)  176 (4)  207 (6)
//   4096, the same heads                       172 (1)  197 (2)  211 (3)
//   3000 on 200 keys, 2 on 1 heads of 32/64    119 (1)  58 (4)  47 (8)  43 (12)
//   4 x 2048 causal, 8 heads of 32/64          213 (1)  252 (2)
int diff_bwd_splits(const DiffGeom& g) {
  const long long k_tiles = ceil_div(diff_max_k_boxes(g), 2), boxes = diff_max_q_boxes(g);
  const long long tiles = static_cast<long long>(diff_sequences(g)) * g.kv_heads * k_tiles;
  const int sms = sm_count();
  if (tiles == 0 || boxes < 16 || tiles >= 3ll * sms) return 1;
  const long long most = boxes / 8 < 16 ? boxes / 8 : 16;
  if (g.causal) {
    // the first key tiles have the most rows: so many shares that the longest is two thirds of an SM's part of all the work
    const long long total = tiles * boxes / 2;
    const long long want = (3 * boxes * sms + 2 * total - 1) / (2 * total);
    return static_cast<int>(want < most ? want : most);
  }
  // all tiles are alike: the least estimate of time. A box takes a CTA about 1.2 us, its start and end as much as four;
  // the join 6 us and its sums' bytes, written and read, at 5 TB/s
  int best = 1;
  float least = 0.f;
  for (int s = 1; s <= most; ++s) {
    const float us = static_cast<float>((tiles * s + sms - 1) / sms) * ((boxes + s - 1) / s + 4) * 1.2f +
                     (s > 1 ? 6.f + static_cast<float>(tiles * s) * (2 * g.d + g.dv) / 4900.f : 0.f);
    if (s == 1 || us < least) {
      least = us;
      best = s;
    }
  }
  return best;
}

size_t diff_bwd_part_bytes(const DiffGeom& g) {
  const int s = diff_bwd_splits(g);
  return s > 1 ? static_cast<size_t>(diff_sequences(g)) * g.kv_heads * ceil_div(diff_max_k_boxes(g), 2) * s * kOwn * (2 * g.d + g.dv) * sizeof(float) : 0;
}

cudaError_t launch_diff_attn_bwd(const DiffBwdArgs& a, bool f16, cudaStream_t stream) {
  switch (diff_class(a.g.d, a.g.dv)) {
    case 0: return f16 ? launch_class<16, 32, true>(a, stream) : launch_class<16, 32, false>(a, stream);
    case 1: return f16 ? launch_class<32, 64, true>(a, stream) : launch_class<32, 64, false>(a, stream);
    default: return f16 ? launch_class<64, 128, true>(a, stream) : launch_class<64, 128, false>(a, stream);
  }
}

}  // namespace rib
