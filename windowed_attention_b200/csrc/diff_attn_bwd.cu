// Differential attention, backward (rib_diff_attention_bwd). With
// P_i = softmax(s Q_i K_i^T), O_i = P_i V, O = O_1 - lambda O_2 and
// dP = dO V^T (the same for both maps):
//   D_i = rowsum(dO * O_i),            O_1 = O + lambda O_2
//   dS_1 = P_1 (dP - D_1),             dS_2 = -lambda P_2 (dP - D_2)
//   dQ_i = s dS_i K_i,  dK_i = s dS_i^T Q_i,  dV = (P_1 - lambda P_2)^T dO
//   dlambda = -sum over the head's rows of D_2
// P_i is formed again from the forward's log-sum-exps. Gradients of a key head
// that several query heads share are sums over its rows, in one accumulator.
//
// Three launches:
//  * rows: D_1, D_2 and the other row constants, one array each, so that the
//    key-side kernel reads four neighbouring rows' with one load.
//  * dq: one CTA owns 128 query rows and streams key tiles of 64.
//  * dkv: one CTA owns 128 keys of a key head and streams tiles of 64 query
//    rows, keys in the TMEM lanes (S_i^T = K_i Q_i^T); the last CTAs add up
//    dlambda. Every sum has one owner and a fixed order: the same bits on
//    every run, no atomics.
// Both recompute S_i and dP: the alternative, one kernel that adds its dQ
// tiles to memory, needs atomics, whose order changes the result.
//
// Bound: the exponentials (2 per pair and kernel, 16 a cycle and SM) at d <= 32;
// with d = 64, dv = 128 the products, whose cost per 128 x 64 tile in cycles
// is about 48 per K step of N = 64 and 64 at N = 128: dq 1150, dkv 1400.
#include <cuda_runtime.h>

#include "diff_attn.cuh"

namespace rib {
namespace {

constexpr int kOwn = 128, kStream = 64;
constexpr int kLoadWarps = 4;
constexpr int kLoaders = 32 * kLoadWarps;
constexpr int kThreads = 32 * (10 + kLoadWarps);   // 8 elementwise warps, two MMA issuers, the loaders

enum Site : int {
  SITE_OWN = 421, SITE_ST_FULL = 422, SITE_ST_EMPTY = 423, SITE_S_FULL = 424, SITE_S_FREE = 425, SITE_X_FULL = 426, SITE_X_DONE = 427,
  SITE_DONE = 428,
};

// fp16 probabilities and their gradients are held times 2^6, which moves
// fp16's smallest normal value to 2^-20 (rows of a million keys) and still
// leaves |P (dP - D)| up to 1023 below its largest; the epilogues divide it
// out. bf16 has fp32's range.
template <bool F16>
constexpr float kShift = F16 ? 6.f : 0.f;
template <bool F16>
constexpr float kUnshift = F16 ? 1.f / 64.f : 1.f;

// ---------------------------------------------------------------- row constants
// LPR lanes hold a row's eight columns each.
template <int LPR, bool F16>
__global__ void __launch_bounds__(256) diff_attn_rows_kernel(const DiffBwdArgs a) {
  const DiffGeom& g = a.g;
  constexpr int kRows = 256 / LPR;
  const int per = a.rows_pad / kRows, unit = blockIdx.x / per;
  const int r = (blockIdx.x - unit * per) * kRows + threadIdx.x / LPR, lane = threadIdx.x % LPR;
  const int hk = unit % g.kv_heads;
  const DiffSeq s = diff_sequence(g, unit / g.kv_heads);
  const bool live = r < s.nq * g.group;
  const int t = live ? diff_row_token(g, r) : 0, hq = hk * g.group + (live ? r - t * g.group : 0);
  const long long token = live ? s.token(t) : 0;
  const float lam = diff_lambda<F16>(a.lam, g.lam_f32, hq);
  float d1 = 0.f, d2 = 0.f;
  if (live && lane * 8 < g.dv) {
    const long long at = s.b * g.o.b + token * g.o.t + hq * g.o.h + lane * 8;
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
  float l[2] = {-INFINITY, -INFINITY};   // minus the log-sum-exp: a row that saw nothing has P = 2^(S - inf) = 0
  if (live)
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const float v = a.lse[((static_cast<long long>(m) * g.batch + s.b) * g.q_heads + hq) * g.q_len + token];
      l[m] = v == -INFINITY ? -INFINITY : fmaf(-kDiffLog2e, v, kShift<F16>);
    }
  float* w = a.rows + static_cast<long long>(unit) * a.rows_pad + r;
  w[kRowL1 * a.row_stride] = l[0];
  w[kRowL2 * a.row_stride] = l[1];
  w[kRowD1 * a.row_stride] = -d1;
  w[kRowD2 * a.row_stride] = -d2;
  w[kRowLam * a.row_stride] = live ? -lam : 0.f;
  w[kRowSeen * a.row_stride] = __int_as_float(live ? diff_visible(g, s, t) : 0);
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
  static constexpr int OFF_BAR = OFF_ST + NS * STAGE;
  static constexpr int NBAR = 1 + 2 * NS + 6 + 1;   // own, st_full, st_empty, s_full[2], x_full[2], x_done[2], done
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
  static constexpr int ALLOC = OFF_MISC + 16 + 1024;
  // two buffers of S_1, S_2, dP (64 columns each); dS_i overwrites S_i's first 32
  static constexpr uint32_t BUF = 192, Q1 = 384, Q2 = 448, COLS = 512;
};

template <int D, int DV, bool F16>
__global__ void __launch_bounds__(kThreads, 1) diff_attn_dq_kernel(const DiffBwdArgs a, int q_tiles) {
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
  uint64_t* s_full = st_empty + NS;
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
  const int rows = s.nq * g.group, row0 = qt * kOwn;
  if (row0 >= rows) return;
  const int most = diff_visible(g, s, diff_row_token(g, min(row0 + kOwn, rows) - 1));
  const int least = diff_visible(g, s, diff_row_token(g, row0));   // the keys that every row of the tile sees
  const int n = (most + kStream - 1) / kStream;

  if (threadIdx.x == 0) {
    mbar_init(own, kLoadWarps);
    for (int i = 0; i < NS; ++i) {
      mbar_init(&st_full[i], kLoadWarps);
      mbar_init(&st_empty[i], 2);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&x_full[i], 4);
      mbar_init(&x_done[i], 1);
    }
    mbar_init(done, 2);
    tmem_holder[1] = 0u;
    tmem_holder[2] = 0u;
    fence_barrier_init();
  }
  if (warp == 8) {
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

  if (warp >= 10) {
    // ------------------------------------------------------------ loaders
    const int tid = threadIdx.x - 10 * 32;
    const long long qb = s.b * g.q.b + static_cast<long long>(hk) * g.group * g.q.h;
    const long long ob = s.b * g.o.b + static_cast<long long>(hk) * g.group * g.o.h;
    const long long kb = s.b * g.k.b + hk * g.k.h;
    const uint16_t* k1 = static_cast<const uint16_t*>(a.k1) + kb;
    const uint16_t* k2 = static_cast<const uint16_t*>(a.k2) + kb;
    const uint16_t* v = static_cast<const uint16_t*>(a.v) + s.b * g.v.b + hk * g.v.h;
    int told = -1;   // -1: nothing handed over, 0: the own tiles, i + 1: key tile i
    auto tell = [&](int upto) {
      if (upto <= told) return;
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0)
        for (int i = told + 1; i <= upto; ++i) mbar_arrive(i == 0 ? own : &st_full[(i - 1) % NS]);
      told = upto;
    };
    if (n > 0) {
      diff_clear<D, DV, kLoaders>(smem, Lay::OFF_BAR, g, tid);
      diff_load_queries<kOwn, D, DV, kLoaders>(so, static_cast<const uint16_t*>(a.q1) + qb, static_cast<const uint16_t*>(a.q2) + qb,
                                               static_cast<const uint16_t*>(a.dO) + ob, g, s, row0, rows, tid);
      cp_async_commit();
    }
    for (int i = 0; i < n; ++i) {
      const int st = i % NS;
      if (i >= NS) {
        const uint32_t parity = ((i / NS) - 1) & 1;
        if (!__all_sync(0xFFFFFFFFu, mbar_test_wait(&st_empty[st], parity))) {
          cp_async_wait<0>();
          tell(i);
          if (!__all_sync(0xFFFFFFFFu, mbar_wait(&st_empty[st], parity, wc, SITE_ST_EMPTY))) break;
        }
      }
      const uint32_t b = sst + st * Lay::STAGE;
      diff_load_keys<kStream, D, DV, kLoaders>(b, k1, k2, v, g, s, i * kStream, s.nk, tid);
      cp_async_commit();
      cp_async_wait<1>();
      tell(i);
    }
    cp_async_wait<0>();
    if (n > 0 && *abort_flag == 0u) tell(n);
  } else if (warp == 8 || warp == 9) {
    // two MMA issuers: warp 8 the scores and dP, warp 9 the gradients
    if (lane == 0 && n > 0) {
      const uint32_t id_s = diff_idesc(F16, kStream, false);
      const uint32_t id_q = diff_idesc(F16, (g.d + 15) / 16 * 16, true);
      const int ks_d = (g.d + 15) / 16, ks_v = (g.dv + 15) / 16;
      bool ok = mbar_wait(own, 0, wc, SITE_OWN);
      for (int j = 0; ok && j < n; ++j) {
        const int st = j % NS, bb = j & 1;
        const uint32_t b = sst + st * Lay::STAGE, t = tmem + Lay::BUF * bb;
        if (warp == 8) {
          if (!(ok = mbar_wait(&st_full[st], (j / NS) & 1, wc, SITE_ST_FULL))) break;
          if (j >= 2 && !(ok = mbar_wait(&x_done[bb], ((j - 2) >> 1) & 1, wc, SITE_X_DONE))) break;
          tc_fence_after();
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks)
            if (ks < ks_d) umma_ss(t, TQ::kmajor(so, ks), TK::kmajor(b, ks), id_s, ks > 0 ? 1u : 0u);
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks)
            if (ks < ks_d) umma_ss(t + 64, TQ::kmajor(so + TQ::BYTES, ks), TK::kmajor(b + TK::BYTES, ks), id_s, ks > 0 ? 1u : 0u);
#pragma unroll
          for (int ks = 0; ks < DV / 16; ++ks)
            if (ks < ks_v)
              umma_ss(t + 128, TO::kmajor(so + 2 * TQ::BYTES, ks), TV::kmajor(b + 2 * TK::BYTES, ks), id_s, ks > 0 ? 1u : 0u);
          umma_commit(&s_full[bb]);
        } else {
          if (!(ok = mbar_wait(&x_full[bb], (j >> 1) & 1, wc, SITE_X_FULL))) break;
          tc_fence_after();
#pragma unroll
          for (int ks = 0; ks < kStream / 16; ++ks)
            umma_ts(tmem + Lay::Q1, t + 8u * ks, TK::mnmajor(b, ks), id_q, (j > 0 || ks > 0) ? 1u : 0u);
#pragma unroll
          for (int ks = 0; ks < kStream / 16; ++ks)
            umma_ts(tmem + Lay::Q2, t + 64 + 8u * ks, TK::mnmajor(b + TK::BYTES, ks), id_q, (j > 0 || ks > 0) ? 1u : 0u);
          umma_commit(&x_done[bb]);
        }
        umma_commit(&st_empty[st]);
      }
      umma_commit(done);
      mbar_wait(done, 0, drain, SITE_DONE);
    }
  } else {
    // elementwise: warpgroup w takes the tiles j = w, w + 2, ...; thread = query row = TMEM lane
    const int w = warp >> 2, row = (warp & 3) * 32 + lane, r = row0 + row;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t t = tmem + lane_off + Lay::BUF * w;
    const float* c = a.rows + static_cast<long long>(unit) * a.rows_pad + r;
    const float l1 = c[kRowL1 * a.row_stride], l2 = c[kRowL2 * a.row_stride], d1 = c[kRowD1 * a.row_stride], d2 = c[kRowD2 * a.row_stride];
    const float nlam = c[kRowLam * a.row_stride];
    const int seen = __float_as_int(c[kRowSeen * a.row_stride]);
    const bool warp_live = row0 + (warp & 3) * 32 < rows;
    const uint64_t sl2 = f2_pack(g.scale_log2, g.scale_log2), L1 = f2_pack(l1, l1), L2 = f2_pack(l2, l2), D1 = f2_pack(d1, d1), D2 = f2_pack(d2, d2);
    const uint64_t NL = f2_pack(nlam, nlam);
    bool ok = true;
    for (int j = w; j < n; j += 2) {
      ok = __all_sync(0xFFFFFFFFu, mbar_wait(&s_full[w], (j >> 1) & 1, wc, SITE_S_FULL));
      if (!ok) break;
      tc_fence_after();
      if (warp_live) {
        const bool edge = (j + 1) * kStream > least;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t s1[32], s2[32], dp[32], x1[16], x2[16];
          tmem_ld32(t + 32 * h, s1);
          tmem_ld32(t + 64 + 32 * h, s2);
          tmem_ld32(t + 128 + 32 * h, dp);
          tmem_wait_ld();
          if (edge) {
            const int left = seen - j * kStream - 32 * h;
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (i >= left) s1[i] = s2[i] = 0xFF800000u;   // -inf: P = 0
          }
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const uint64_t y1 = f2_fma(f2_pack(__uint_as_float(s1[2 * i]), __uint_as_float(s1[2 * i + 1])), sl2, L1);
            const uint64_t y2 = f2_fma(f2_pack(__uint_as_float(s2[2 * i]), __uint_as_float(s2[2 * i + 1])), sl2, L2);
            const uint64_t dd = f2_pack(__uint_as_float(dp[2 * i]), __uint_as_float(dp[2 * i + 1]));
            float a0, a1, b0, b1;
            f2_unpack(y1, a0, a1);
            f2_unpack(y2, b0, b1);
            const uint64_t e1 = f2_mul(f2_pack(ex2_approx(a0), ex2_approx(a1)), f2_add(dd, D1));
            const uint64_t e2 = f2_mul(f2_mul(f2_pack(ex2_approx(b0), ex2_approx(b1)), NL), f2_add(dd, D2));
            f2_unpack(e1, a0, a1);
            f2_unpack(e2, b0, b1);
            x1[i] = diff_pack<F16>(a0, a1);
            x2[i] = diff_pack<F16>(b0, b1);
          }
          tmem_st16(t + 16 * h, x1);
          tmem_st16(t + 64 + 16 * h, x2);
        }
        tmem_wait_st();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&x_full[w]);
    }
    if (ok && n > 0) ok = __all_sync(0xFFFFFFFFu, mbar_wait(done, 0, wc, SITE_DONE));
    tc_fence_after();
    if (ok && warp_live && *abort_flag == 0u) {
      // warpgroup w stores dQ_(w + 1); without a key in sight the gradient is zero
      const float f = n > 0 ? g.scale * kUnshift<F16> : 0.f;
      const bool live = r < rows;
      const int tk = diff_row_token(g, r);
      uint16_t* out = static_cast<uint16_t*>(w ? a.dq2 : a.dq1);
      if (live) out += s.b * g.q.b + s.token(tk) * g.q.t + (hk * g.group + r - tk * g.group) * g.q.h;
#pragma unroll
      for (int cc = 0; cc < D / 16; ++cc) {
        uint32_t v[16];
        tmem_ld16(tmem + lane_off + (w ? Lay::Q2 : Lay::Q1) + 16 * cc, v);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = n > 0 ? __float_as_uint(__uint_as_float(v[i]) * f) : 0u;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t o[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) o[e] = diff_pack<F16>(__uint_as_float(v[8 * h + 2 * e]), __uint_as_float(v[8 * h + 2 * e + 1]));
          if (live && 16 * cc + 8 * h < g.d) *reinterpret_cast<uint4*>(out + 16 * cc + 8 * h) = make_uint4(o[0], o[1], o[2], o[3]);
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
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
  static constexpr int OWN = 2 * TK::BYTES + TV::BYTES;
  static constexpr int CONSTS = kRowArrays * kStream * 4;
  static constexpr int STAGE = (2 * TQ::BYTES + TO::BYTES + CONSTS + 1023) / 1024 * 1024;
  static constexpr int NS = STAGE <= 16 * 1024 ? 4 : 3;
  static constexpr int OFF_ST = OWN;
  static constexpr int OFF_X = OFF_ST + NS * STAGE;
  static constexpr int OFF_BAR = OFF_X + 3 * TP::BYTES;
  static constexpr int NBAR = 1 + 2 * NS + 4 + 1;   // own, st_full, st_empty, s_full, s_free, x_full, x_free, done
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
  static constexpr int ALLOC = OFF_MISC + 16 + 1024;
  static_assert(ALLOC <= 232448, "shared memory of an SM");
  static constexpr uint32_t S1 = 0, S2 = 64, DP = 128, V = 192, K1 = V + DV, K2 = K1 + D, COLS = K2 + D <= 256 ? 256 : 512;
};

template <int D, int DV, bool F16>
__global__ void __launch_bounds__(kThreads, 1) diff_attn_dkv_kernel(const DiffBwdArgs a, int k_tiles, int units) {
  using Lay = DkvLay<D, DV>;
  using TQ = typename Lay::TQ;
  using TO = typename Lay::TO;
  using TK = typename Lay::TK;
  using TV = typename Lay::TV;
  using TP = typename Lay::TP;
  constexpr int NS = Lay::NS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align_smem_1024(smem_raw);
  const DiffGeom& g = a.g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  int u = blockIdx.x / k_tiles;
  if (u >= units) {
    // dlambda of one head: its rows' -D_2 over every sequence, each thread a
    // strided share, then a tree
    const int h = blockIdx.x - units * k_tiles, hk = h / g.group;
    float sum = 0.f;
    const long long per = a.rows_pad / g.group, total = static_cast<long long>(units / g.kv_heads) * per;
    for (long long i = threadIdx.x; i < total; i += kThreads) {
      const long long q = i / per, t = i - q * per;
      sum += a.rows[kRowD2 * a.row_stride + (q * g.kv_heads + hk) * a.rows_pad + t * g.group + (h - hk * g.group)];
    }
    float* red = reinterpret_cast<float*>(smem);
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    if (lane == 0) red[warp] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
      float v = 0.f;
      for (int i = 0; i < kThreads / 32; ++i) v += red[i];
      if (g.lam_f32) static_cast<float*>(a.dlam)[h] = v;
      else static_cast<uint16_t*>(a.dlam)[h] = static_cast<uint16_t>(diff_pack<F16>(v, 0.f));
    }
    return;
  }
  uint64_t* own = reinterpret_cast<uint64_t*>(smem + Lay::OFF_BAR);
  uint64_t* st_full = own + 1;
  uint64_t* st_empty = st_full + NS;
  uint64_t* s_full = st_empty + NS;
  uint64_t* s_free = s_full + 1;
  uint64_t* x_full = s_full + 2;
  uint64_t* x_free = s_full + 3;
  uint64_t* done = s_full + 4;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + Lay::OFF_MISC);
  volatile uint32_t* abort_flag = tmem_holder + 1;
  const int key0 = (blockIdx.x - u * k_tiles) * kOwn;   // with a causal mask the first keys have the most rows
  const int unit = u, hk = u % g.kv_heads;
  const DiffSeq s = diff_sequence(g, u / g.kv_heads);
  const int all = g.window ? s.nk : g.k_len;            // keys whose gradients are written
  if (key0 >= all) return;
  const int rows = s.nq * g.group;
  // the first row that sees key0, and the first from which every row sees the whole tile
  int first = 0, full = 0;
  if (g.causal) {
    first = min(max(key0 - s.nk + s.nq, 0), s.nq) * g.group;
    full = min(max(min(key0 + kOwn, s.nk) - 1 - s.nk + s.nq, 0), s.nq) * g.group;
  }
  if (key0 >= s.nk) first = rows;
  const int j0 = first / kStream, n = first < rows ? (rows + kStream - 1) / kStream - j0 : 0;

  if (threadIdx.x == 0) {
    mbar_init(own, kLoadWarps);
    for (int i = 0; i < NS; ++i) {
      mbar_init(&st_full[i], kLoadWarps);
      mbar_init(&st_empty[i], 2);
    }
    mbar_init(s_full, 1);
    mbar_init(s_free, 8);
    mbar_init(x_full, 8);
    mbar_init(x_free, 1);
    mbar_init(done, 2);
    tmem_holder[1] = 0u;
    tmem_holder[2] = 0u;
    fence_barrier_init();
  }
  if (warp == 8) {
    tmem_alloc(tmem_holder, Lay::COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const WaitCtx wc{abort_flag, a.err};
  const WaitCtx drain{tmem_holder + 2, a.err};
  const uint32_t so = smem_u32(smem), sst = so + Lay::OFF_ST, sx = so + Lay::OFF_X;

  if (warp >= 10) {
    // ------------------------------------------------------------ loaders
    const int tid = threadIdx.x - 10 * 32;
    const long long qb = s.b * g.q.b + static_cast<long long>(hk) * g.group * g.q.h;
    const long long kb = s.b * g.k.b + hk * g.k.h;
    const uint16_t* q1 = static_cast<const uint16_t*>(a.q1) + qb;
    const uint16_t* q2 = static_cast<const uint16_t*>(a.q2) + qb;
    const uint16_t* dO = static_cast<const uint16_t*>(a.dO) + s.b * g.o.b + static_cast<long long>(hk) * g.group * g.o.h;
    const float* consts = a.rows + static_cast<long long>(unit) * a.rows_pad;
    int told = -1;
    auto tell = [&](int upto) {
      if (upto <= told) return;
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0)
        for (int i = told + 1; i <= upto; ++i) mbar_arrive(i == 0 ? own : &st_full[(i - 1) % NS]);
      told = upto;
    };
    if (n > 0) {
      diff_clear<D, DV, kLoaders>(smem, Lay::OFF_X, g, tid);
      diff_load_keys<kOwn, D, DV, kLoaders>(so, static_cast<const uint16_t*>(a.k1) + kb, static_cast<const uint16_t*>(a.k2) + kb,
                                            static_cast<const uint16_t*>(a.v) + s.b * g.v.b + hk * g.v.h, g, s, key0, s.nk, tid);
      cp_async_commit();
    }
    for (int i = 0; i < n; ++i) {
      const int st = i % NS;
      if (i >= NS) {
        const uint32_t parity = ((i / NS) - 1) & 1;
        if (!__all_sync(0xFFFFFFFFu, mbar_test_wait(&st_empty[st], parity))) {
          cp_async_wait<0>();
          tell(i);
          if (!__all_sync(0xFFFFFFFFu, mbar_wait(&st_empty[st], parity, wc, SITE_ST_EMPTY))) break;
        }
      }
      const uint32_t b = sst + st * Lay::STAGE;
      const int r0 = (j0 + i) * kStream;
      diff_load_queries<kStream, D, DV, kLoaders>(b, q1, q2, dO, g, s, r0, rows, tid);
      for (int c = tid; c < kRowArrays * kStream / 4; c += kLoaders)   // 16 pieces of 4 rows an array; rows_pad covers the last tile
        cp_async_16(smem + (b - so) + 2 * TQ::BYTES + TO::BYTES + c * 16, consts + (c / 16) * a.row_stride + r0 + (c % 16) * 4);
      cp_async_commit();
      cp_async_wait<1>();
      tell(i);
    }
    cp_async_wait<0>();
    if (n > 0 && *abort_flag == 0u) tell(n);
  } else if (warp == 8 || warp == 9) {
    if (lane == 0 && n > 0) {
      const uint32_t id_s = diff_idesc(F16, kStream, false);
      const uint32_t id_k = diff_idesc(F16, (g.d + 15) / 16 * 16, true), id_v = diff_idesc(F16, (g.dv + 15) / 16 * 16, true);
      const int ks_d = (g.d + 15) / 16, ks_v = (g.dv + 15) / 16;
      bool ok = mbar_wait(own, 0, wc, SITE_OWN);
      for (int j = 0; ok && j < n; ++j) {
        const int st = j % NS;
        const uint32_t b = sst + st * Lay::STAGE;
        if (warp == 8) {
          if (!(ok = mbar_wait(&st_full[st], (j / NS) & 1, wc, SITE_ST_FULL))) break;
          if (j >= 1 && !(ok = mbar_wait(s_free, (j - 1) & 1, wc, SITE_S_FREE))) break;
          tc_fence_after();
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks)
            if (ks < ks_d) umma_ss(tmem + Lay::S1, TK::kmajor(so, ks), TQ::kmajor(b, ks), id_s, ks > 0 ? 1u : 0u);
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks)
            if (ks < ks_d)
              umma_ss(tmem + Lay::S2, TK::kmajor(so + TK::BYTES, ks), TQ::kmajor(b + TQ::BYTES, ks), id_s, ks > 0 ? 1u : 0u);
#pragma unroll
          for (int ks = 0; ks < DV / 16; ++ks)
            if (ks < ks_v)
              umma_ss(tmem + Lay::DP, TV::kmajor(so + 2 * TK::BYTES, ks), TO::kmajor(b + 2 * TQ::BYTES, ks), id_s, ks > 0 ? 1u : 0u);
          umma_commit(s_full);
        } else {
          if (!(ok = mbar_wait(x_full, j & 1, wc, SITE_X_FULL))) break;
          tc_fence_after();
#pragma unroll
          for (int ks = 0; ks < kStream / 16; ++ks) {
            const uint32_t acc = (j > 0 || ks > 0) ? 1u : 0u;
            umma_ss(tmem + Lay::V, TP::kmajor(sx, ks), TO::mnmajor(b + 2 * TQ::BYTES, ks), id_v, acc);
            umma_ss(tmem + Lay::K1, TP::kmajor(sx + TP::BYTES, ks), TQ::mnmajor(b, ks), id_k, acc);
            umma_ss(tmem + Lay::K2, TP::kmajor(sx + 2 * TP::BYTES, ks), TQ::mnmajor(b + TQ::BYTES, ks), id_k, acc);
          }
          umma_commit(x_free);
        }
        umma_commit(&st_empty[st]);
      }
      umma_commit(done);
      mbar_wait(done, 0, drain, SITE_DONE);
    }
  } else {
    // elementwise: thread = key = TMEM lane; warpgroup w takes query rows 32 w .. 32 w + 31 of every tile
    const int w = warp >> 2, row = (warp & 3) * 32 + lane, key = key0 + row;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t t = tmem + lane_off + 32 * w;
    const uint64_t sl2 = f2_pack(g.scale_log2, g.scale_log2);
    bool ok = true;
    for (int j = 0; j < n; ++j) {
      const int st = j % NS, r0 = (j0 + j) * kStream;
      ok = __all_sync(0xFFFFFFFFu, mbar_wait(&st_full[st], (j / NS) & 1, wc, SITE_ST_FULL));   // the row constants
      ok = ok && __all_sync(0xFFFFFFFFu, mbar_wait(s_full, j & 1, wc, SITE_S_FULL));
      if (!ok) break;
      tc_fence_after();
      uint32_t s1[32], s2[32], dp[32];
      tmem_ld32(t + Lay::S1, s1);
      tmem_ld32(t + Lay::S2, s2);
      tmem_ld32(t + Lay::DP, dp);
      tmem_wait_ld();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(s_free);   // the next tile's products may overwrite them
      const float* cs = reinterpret_cast<const float*>(smem + Lay::OFF_ST + st * Lay::STAGE + 2 * TQ::BYTES + TO::BYTES) + 32 * w;
      // rows behind the last one, or (causal) before the first that sees the whole tile
      if (r0 < full || r0 + kStream > rows) {
        const int* seen = reinterpret_cast<const int*>(cs + kRowSeen * kStream);
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (key >= seen[i]) s1[i] = s2[i] = 0xFF800000u;   // -inf: P = 0
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {   // eight query rows: 16 bytes of each operand row
        uint32_t pp[4], x1[4], x2[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int i = 8 * q + 2 * e;
          const uint64_t* pair = reinterpret_cast<const uint64_t*>(cs + i);
          const uint64_t L1 = pair[kRowL1 * kStream / 2], L2 = pair[kRowL2 * kStream / 2], D1 = pair[kRowD1 * kStream / 2],
                         D2 = pair[kRowD2 * kStream / 2], NL = pair[kRowLam * kStream / 2];
          const uint64_t y1 = f2_fma(f2_pack(__uint_as_float(s1[i]), __uint_as_float(s1[i + 1])), sl2, L1);
          const uint64_t y2 = f2_fma(f2_pack(__uint_as_float(s2[i]), __uint_as_float(s2[i + 1])), sl2, L2);
          const uint64_t dd = f2_pack(__uint_as_float(dp[i]), __uint_as_float(dp[i + 1]));
          float a0, a1, b0, b1;
          f2_unpack(y1, a0, a1);
          f2_unpack(y2, b0, b1);
          const uint64_t p1 = f2_pack(ex2_approx(a0), ex2_approx(a1));
          const uint64_t p2 = f2_mul(f2_pack(ex2_approx(b0), ex2_approx(b1)), NL);
          f2_unpack(f2_add(p1, p2), a0, a1);
          pp[e] = diff_pack<F16>(a0, a1);
          f2_unpack(f2_mul(p1, f2_add(dd, D1)), a0, a1);
          x1[e] = diff_pack<F16>(a0, a1);
          f2_unpack(f2_mul(p2, f2_add(dd, D2)), b0, b1);
          x2[e] = diff_pack<F16>(b0, b1);
        }
        if (q == 0 && j >= 1) {
          // the products of the tile before have read P^T and dS^T
          ok = __all_sync(0xFFFFFFFFu, mbar_wait(x_free, (j - 1) & 1, wc, SITE_X_DONE));
          if (!ok) break;
        }
        uint8_t* to = smem + Lay::OFF_X + TP::offset(row, 4 * w + q);
        *reinterpret_cast<uint4*>(to) = make_uint4(pp[0], pp[1], pp[2], pp[3]);
        *reinterpret_cast<uint4*>(to + TP::BYTES) = make_uint4(x1[0], x1[1], x1[2], x1[3]);
        *reinterpret_cast<uint4*>(to + 2 * TP::BYTES) = make_uint4(x2[0], x2[1], x2[2], x2[3]);
      }
      if (!ok) break;
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(x_full);
    }
    if (ok && n > 0) ok = __all_sync(0xFFFFFFFFu, mbar_wait(done, 0, wc, SITE_DONE));
    tc_fence_after();
    if (ok && *abort_flag == 0u) {
      const bool live = key < all, real = n > 0 && key < s.nk;   // keys behind the length have gradient zero
      const long long token = live ? s.token(key) : 0;
      auto store = [&](uint32_t col, int c0, int c1, uint16_t* out, int width, float f) {
        for (int c = c0; c < c1; c += 16) {
          uint32_t v[16];
          tmem_ld16(tmem + lane_off + col + c, v);
          tmem_wait_ld();
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t o[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int i = 8 * h + 2 * e;
              o[e] = real ? diff_pack<F16>(__uint_as_float(v[i]) * f, __uint_as_float(v[i + 1]) * f) : 0u;
            }
            if (live && c + 8 * h < width) *reinterpret_cast<uint4*>(out + c + 8 * h) = make_uint4(o[0], o[1], o[2], o[3]);
          }
        }
      };
      store(Lay::V, w * (DV / 2), (w + 1) * (DV / 2), static_cast<uint16_t*>(a.dv) + s.b * g.v.b + token * g.v.t + hk * g.v.h, g.dv,
            kUnshift<F16>);
      store(w ? Lay::K2 : Lay::K1, 0, D, static_cast<uint16_t*>(w ? a.dk2 : a.dk1) + s.b * g.k.b + token * g.k.t + hk * g.k.h, g.d,
            g.scale * kUnshift<F16>);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, Lay::COLS);
  }
}

template <int D, int DV, bool F16>
cudaError_t launch_class(const DiffBwdArgs& a, cudaStream_t stream) {
  const DiffGeom& g = a.g;
  const long long seqs = diff_sequences(g), units = seqs * g.kv_heads;
  const int q_tiles = static_cast<int>((diff_max_rows(g) + kOwn - 1) / kOwn), k_tiles = (diff_max_keys(g) + kOwn - 1) / kOwn;
  constexpr int LPR = DV / 8;
  const long long row_ctas = units * (a.rows_pad / (256 / LPR)), q_ctas = units * q_tiles, k_ctas = units * k_tiles + g.q_heads;
  if (row_ctas > 0x7FFFFFFFll || q_ctas > 0x7FFFFFFFll || k_ctas > 0x7FFFFFFFll) return cudaErrorInvalidConfiguration;
  auto dq = diff_attn_dq_kernel<D, DV, F16>;
  auto dkv = diff_attn_dkv_kernel<D, DV, F16>;
  cudaError_t e = cudaFuncSetAttribute(dq, cudaFuncAttributeMaxDynamicSharedMemorySize, DqLay<D, DV>::ALLOC);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(dkv, cudaFuncAttributeMaxDynamicSharedMemorySize, DkvLay<D, DV>::ALLOC);
  if (e != cudaSuccess) return e;
  if (row_ctas > 0) {
    diff_attn_rows_kernel<LPR, F16><<<static_cast<unsigned>(row_ctas), 256, 0, stream>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    dq<<<static_cast<unsigned>(q_ctas), kThreads, DqLay<D, DV>::ALLOC, stream>>>(a, q_tiles);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  // k_tiles 0: dlambda alone, with no tiles before it
  dkv<<<static_cast<unsigned>(k_ctas), kThreads, DkvLay<D, DV>::ALLOC, stream>>>(a, k_tiles > 0 ? k_tiles : 1, k_tiles > 0 ? static_cast<int>(units) : 0);
  return cudaGetLastError();
}

}  // namespace

long long diff_rows_pad(const DiffGeom& g) { return (diff_max_rows(g) + kOwn - 1) / kOwn * kOwn; }

cudaError_t launch_diff_attn_bwd(const DiffBwdArgs& a, bool f16, cudaStream_t stream) {
  switch (diff_class(a.g.d, a.g.dv)) {
    case 0: return f16 ? launch_class<16, 32, true>(a, stream) : launch_class<16, 32, false>(a, stream);
    case 1: return f16 ? launch_class<32, 64, true>(a, stream) : launch_class<32, 64, false>(a, stream);
    default: return f16 ? launch_class<64, 128, true>(a, stream) : launch_class<64, 128, false>(a, stream);
  }
}

}  // namespace rib
