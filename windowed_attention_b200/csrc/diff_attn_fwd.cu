// Differential attention, forward (rib_diff_attention):
//   O = (softmax(s Q1 K1^T) - lambda softmax(s Q2 K2^T)) V
// per sequence and head, lambda learned per query head.
//
// One pass over the keys: each of the two maps keeps its own running maximum m
// and sum l, O_i accumulates 2^(s' S_i - m_i) V (s' = s log2 e) and the output
// is O_1 / l_1 - lambda O_2 / l_2, formed once at the end. The maximum is
// raised (and O_i scaled) only when a tile exceeds it by 2^8, so P <= 256.
// P takes the 16-bit type for its product with V (half a step of each term, the
// operand type of one product instead of the two that P in two terms would
// take: in bf16 the output is 0.0025 of its norm off, 0.0017 of which rounding
// the result alone takes); scores, sums and both O_i stay fp32.
//
// One CTA owns 128 query rows and streams key tiles of 64; V is loaded once
// for both maps. S of each map has two buffers in TMEM, so the products of the
// next tile run under the exponentials of this one.
//   warps 0 .. 4 NG - 1  softmax: thread = query row = TMEM lane; P overwrites
//                        S in TMEM. NG = 4 warpgroups at dv <= 64: one for each
//                        map and parity of the key tile, with its own m, l and
//                        O, joined at the end. At dv = 128 TMEM holds two O:
//                        NG = 2, one group a map.
//   then one warp        TMEM owner, issues S
//   then one warp        issues P V (its own stream: neither waits for the other)
//   then one warp        TMA producer
//   then one warp        clears the rows of a key box that are not the sequence's
// TMEM: S of map m and parity q at 64 (2 q + m), O from column 256. (P in columns
// of its own, with S freed as soon as it was in registers, cost more in barriers
// than it saved: 0.97 for 0.87 ms.)
//
// Bound: the exponentials, 2 per (query, key) pair: a tile of 128 x 64 x 2
// takes 1024 cycles of the SM's MUFU, of which the FMA pipe takes over POLY of
// every 8 pairs. Its products take 2 (48 D / 16 + 4 max(DV / 2, 32 + DV / 4)) cycles.
// Measured: 320x180 map, window 64, 6 heads of 16/32: 860 us, MUFU 82 % busy
// (floor 596 us); windows of 32, 16 and 8 320, 182 and 261 us (floors 151, 39
// and 14: a CTA takes all of TMEM, so nothing hides its start, and its lanes are
// half empty at 8). Heads of 32/64 913 us, of 48/32, in the tiles of 64/128, 1059.
// Causal 2x4001 tokens, 8 query on 2 key heads of 64/128: 133 us,
// bound by the chain of product, softmax and product with two tiles in flight
// (four softmax groups that share one reference a map: 129 us there, but 2 %
// more for single tokens; not kept).
#include <cuda_runtime.h>

#include "diff_attn.cuh"

namespace rib {
namespace {

constexpr int kBK = 64;

enum Site : int {
  SITE_RAW = 600, SITE_Q = 601, SITE_KV_FULL = 602, SITE_KV_EMPTY = 603, SITE_S = 604, SITE_P = 605, SITE_PV = 606, SITE_DONE = 607,
};

template <int D, int DV>
struct FwdLay {
  using TQ = DiffTile<128, D>;
  using TK = DiffTile<kBK, D>;
  using TV = DiffTile<kBK, DV>;
  static constexpr int NP = DV <= 64 ? 2 : 1;               // O accumulators of a map
  static constexpr int NG = 2 * NP;
  static constexpr int kThreads = 32 * (4 * NG + 4);
  static constexpr int STAGE = 2 * TK::BYTES + TV::BYTES;
  static constexpr int NS = STAGE <= 16 * 1024 ? 6 : 4;
  static constexpr int OFF_ST = 2 * TQ::BYTES;
  static constexpr int OFF_L = OFF_ST + NS * STAGE;         // [4][128] m, then [4][128] l of each group
  static constexpr int OFF_BAR = OFF_L + 2 * 4 * 128 * 4;
  static constexpr int NBAR = 1 + 3 * NS + 12 + 1;          // q, kv_full, kv_empty, raw, s[4], p[4], pv[4], done
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
  static constexpr int ALLOC = OFF_MISC + 16 + 1024;
  static_assert((128 * 2 * DV + 256) * 4 <= OFF_L, "the quarters' outputs over the tiles");
  static constexpr uint32_t O = 256, COLS = 512;
};

__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// QUAD: one tile of at most 32 query rows over split keys (single tokens). The
// rows stand in all four lane quarters; the warps of a quarter take 16 of a
// box's 64 keys and leave zeros in P for the others; the four O of a row are
// joined at the end. A fourth of the exponentials a warp, where they bound.
template <int D, int DV, bool F16, int POLY, bool QUAD>
__global__ void __launch_bounds__(FwdLay<D, DV>::kThreads, 1)
diff_attn_fwd_kernel(const __grid_constant__ CUtensorMap tm_q1, const __grid_constant__ CUtensorMap tm_q2,
                     const __grid_constant__ CUtensorMap tm_k1, const __grid_constant__ CUtensorMap tm_k2,
                     const __grid_constant__ CUtensorMap tm_v, const DiffFwdArgs a, int q_tiles) {
  using Lay = FwdLay<D, DV>;
  using TQ = typename Lay::TQ;
  using TK = typename Lay::TK;
  using TV = typename Lay::TV;
  constexpr int NS = Lay::NS, NP = Lay::NP, NG = Lay::NG;
  constexpr int kWarpS = 4 * NG, kWarpPV = kWarpS + 1, kWarpLoad = kWarpS + 2, kWarpClear = kWarpS + 3;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align_smem_1024(smem_raw);
  uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + Lay::OFF_BAR);
  uint64_t* kv_full = q_full + 1;
  uint64_t* kv_empty = kv_full + NS;
  uint64_t* raw = kv_empty + NS;      // loaded, to be cleared (used instead of kv_full then)
  uint64_t* s_full = raw + NS;        // [2 q + m], as the two below
  uint64_t* p_full = s_full + 4;
  uint64_t* pv = s_full + 8;
  uint64_t* done = s_full + 12;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + Lay::OFF_MISC);
  volatile uint32_t* abort_flag = tmem_holder + 1;
  const DiffGeom& g = a.g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // work unit: (sequence, key head, query tile, split), query tiles with the most keys first
  int u = blockIdx.x;
  const int sp = u % a.splits;
  u /= a.splits;
  const int qt = g.causal ? q_tiles - 1 - u % q_tiles : u % q_tiles;
  u /= q_tiles;
  const int hk = u % g.kv_heads;
  const DiffSeq s = diff_sequence(g, u / g.kv_heads);
  const int q_boxes = diff_q_boxes(g, s);
  if (2 * qt >= q_boxes) return;   // a window at the map's edge has fewer tiles
  // key boxes: all, or (causal) those that the last row sees
  const int k_nx = g.causal ? ceil_div(diff_visible(g, s, min((2 * qt + 2) * g.tcq, s.wq) - 1), g.tck) : ceil_div(s.wk, g.tck);
  const int tiles = k_nx * ceil_div(s.hk, g.trk);
  const bool cut = s.wk % g.tck || s.hk % g.trk;            // some boxes are not the sequence's alone
  const bool clear = cut && (g.window || g.k_lens);         // what lies behind a tensor's end arrives as zeros
  const int per = (tiles + a.splits - 1) / a.splits;
  const int j0 = sp * per, n = max(0, min(tiles, j0 + per) - j0);

  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    for (int i = 0; i < NS; ++i) {
      mbar_init(&kv_full[i], 1);
      mbar_init(&raw[i], 1);
      mbar_init(&kv_empty[i], 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&pv[i], 1);
    }
    mbar_init(done, 2);
    tmem_holder[1] = 0u;
    tmem_holder[2] = 0u;   // abort word of the teardown drain
    fence_barrier_init();
  }
  // The tensor maps are fetched while TMEM is allocated: 866 -> 860 us (window 64, 320x180), no difference on short grids.
  if (warp == kWarpLoad && lane == 0) {
    tma_prefetch_desc(&tm_q1);
    tma_prefetch_desc(&tm_q2);
    tma_prefetch_desc(&tm_k1);
    tma_prefetch_desc(&tm_k2);
    tma_prefetch_desc(&tm_v);
  }
  if (warp == kWarpS) {
    tmem_alloc(tmem_holder, Lay::COLS);
    tmem_relinquish();
  }
  const int q_rows = g.tcq * g.trq * g.group;   // of a box
  if (q_rows < 64) {
    // rows that no load writes: zeros, so that their scores stay finite
    for (int i = threadIdx.x * 16; i < Lay::OFF_ST; i += Lay::kThreads * 16) *reinterpret_cast<uint4*>(smem + i) = make_uint4(0u, 0u, 0u, 0u);
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const WaitCtx wc{abort_flag, a.err};
  const WaitCtx drain{tmem_holder + 2, a.err};

  if (warp == kWarpLoad) {
    // --------------------------------------------------------- TMA producer
    if (lane == 0 && n > 0) {
      const int nx_q = ceil_div(s.wq, g.tcq), copies = QUAD ? 4 : min(2, q_boxes - 2 * qt);
      mbar_arrive_expect_tx(q_full, 2 * copies * TQ::box_bytes(q_rows));
      for (int h = 0; h < copies; ++h) {
        const int box = QUAD ? 0 : 2 * qt + h, by = box / nx_q, x = s.x0 + (box - by * nx_q) * g.tcq, y = s.y0 + by * g.trq;
        TQ::load(smem, (QUAD ? 32 : 64) * h, &tm_q1, q_full, hk * g.group, x, y, s.b);
        TQ::load(smem + TQ::BYTES, (QUAD ? 32 : 64) * h, &tm_q2, q_full, hk * g.group, x, y, s.b);
      }
      const uint32_t bytes = 2 * TK::box_bytes(kBK) + TV::box_bytes(kBK);
      int by = j0 / k_nx, bx = j0 - by * k_nx, issued = 0;
      uint64_t* full = clear ? raw : kv_full;
      for (int i = 0; i < n; ++i) {
        const int st = i % NS;
        if (i >= NS && !mbar_wait(&kv_empty[st], ((i / NS) - 1) & 1, wc, SITE_KV_EMPTY)) break;
        uint8_t* to = smem + Lay::OFF_ST + st * Lay::STAGE;
        const int x = s.x0 + bx * g.tck, y = s.y0 + by * g.trk;
        mbar_arrive_expect_tx(&full[st], bytes);
        TK::load(to, 0, &tm_k1, &full[st], hk, x, y, s.b);
        TK::load(to + TK::BYTES, 0, &tm_k2, &full[st], hk, x, y, s.b);
        TV::load(to + 2 * TK::BYTES, 0, &tm_v, &full[st], hk, x, y, s.b);
        issued = i + 1;
        if (++bx == k_nx) {
          bx = 0;
          ++by;
        }
      }
      // nothing is left in flight when the CTA ends
      mbar_wait(q_full, 0, drain, SITE_DONE);
      for (int i = max(0, issued - NS); i < issued; ++i) mbar_wait(&full[i % NS], (i / NS) & 1, drain, SITE_DONE);
    }
  } else if (warp == kWarpClear) {
    // ------------------------------------------------------------- clearing
    if (clear)
      for (int i = 0; i < n; ++i) {
        const int st = i % NS;
        if (!warp_wait(&raw[st], (i / NS) & 1, wc, SITE_RAW)) break;
        const DiffKeyBox k = diff_key_box(g, s, k_nx, j0 + i);
        const uint64_t mask = diff_key_mask(g, k.vx, k.vy);
        uint8_t* to = smem + Lay::OFF_ST + st * Lay::STAGE;
        if (mask != ~0ull) {
          diff_clear_rows<kBK, D, DV>(to, ~mask, lane);
          fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&kv_full[st]);
      }
  } else if (warp == kWarpS) {
    // --------------------------------------------------------- S issuer
    if (n > 0) {
      const uint32_t sq = smem_u32(smem);
      const uint32_t id_s = diff_idesc(F16, kBK, false);
      const uint64_t dq[2] = {TQ::kmajor(sq), TQ::kmajor(sq + TQ::BYTES)}, dk = TK::kmajor(sq + Lay::OFF_ST);
      bool ok = warp_wait(q_full, 0, wc, SITE_Q);
      int st = 0;
      uint32_t lap = 0;   // parity of the stages' lap
      for (int j = 0; ok && j < n; ++j) {
        ok = warp_wait(&kv_full[st], lap, wc, SITE_KV_FULL);
        const uint64_t k = dk + static_cast<uint32_t>(st) * (Lay::STAGE >> 4);
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const int b = 2 * (j & 1) + m;
          // S overwrites the P of two tiles before: its product has to be done with it
          if (ok && j >= 2) ok = warp_wait(&pv[b], ((j - 2) >> 1) & 1, wc, SITE_PV);
          if (ok && elect_one()) {
            tc_fence_after();
            diff_mma_kk<TQ, TK, D / 16>(tmem + 64u * b, dq[m], k + m * (TK::BYTES >> 4), id_s);
            umma_commit(&s_full[b]);
          }
          __syncwarp();
        }
        if (++st == NS) {
          st = 0;
          lap ^= 1u;
        }
      }
      if (elect_one()) umma_commit(done);
      warp_wait(done, 0, drain, SITE_DONE);
    }
  } else if (warp == kWarpPV) {
    // ------------------------------------------------------- P V issuer
    if (n > 0) {
      const uint32_t id_o = diff_idesc(F16, (g.dv + 15) / 16 * 16, true);
      const uint64_t dv = TV::mnmajor(smem_u32(smem) + Lay::OFF_ST + 2 * TK::BYTES);
      bool ok = true;
      int st = 0;
      for (int j = 0; ok && j < n; ++j) {
        const uint64_t v = dv + static_cast<uint32_t>(st) * (Lay::STAGE >> 4);
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const int b = 2 * (j & 1) + m;
          ok = ok && warp_wait(&p_full[b], (j >> 1) & 1, wc, SITE_P);
          if (ok && elect_one()) {
            tc_fence_after();
            const uint32_t o = tmem + Lay::O + DV * (NP == 2 ? b : m), p = tmem + 64u * b, acc = j >= NP ? 1u : 0u;
#pragma unroll
            for (int ks = 0; ks < kBK / 16; ++ks) umma_ts(o, p + 8u * ks, v + TV::mnstep(ks), id_o, ks > 0 ? 1u : acc);
            umma_commit(&pv[b]);
            if (m == 1) umma_commit(&kv_empty[st]);   // S of the tile was done before its P was written
          }
          __syncwarp();
        }
        if (++st == NS) st = 0;
      }
      if (elect_one()) umma_commit(done);
      warp_wait(done, 0, drain, SITE_DONE);
    }
  } else {
    // ------------------------------------------------------------ softmax
    const int gi = warp >> 2, m = gi & 1, p = gi >> 1;   // map and, with NP = 2, the parity of its tiles
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const DiffRow q = QUAD ? diff_query_row(g, s, 0, lane) : diff_query_row(g, s, 2 * qt + (row >> 6), row & 63);
    const bool live = q.live;
    const int hq = hk * g.group + q.head;
    const int seen = live ? diff_visible(g, s, q.x) : 0x7FFFFFFF;   // of a sequence
    const bool warp_live = __any_sync(0xFFFFFFFFu, live);            // a warp without rows only keeps the barriers going
    const float sl2 = g.scale_log2;
    float mx = -INFINITY, l = 0.f;
    bool ok = true;
    for (int j = p; j < n; j += NP) {
      const int b = 2 * (j & 1) + m;
      const uint32_t tS = tmem + lane_off + 64u * b;
      ok = warp_wait(&s_full[b], (j >> 1) & 1, wc, SITE_S);
      if (!ok) break;
      tc_fence_after();
      if (warp_live) {
        constexpr int kChunk = QUAD ? 16 : 32, kChunks = QUAD ? 1 : 2;
        uint32_t sv[kChunks][kChunk];
#pragma unroll
        for (int c = 0; c < kChunks; ++c) tmem_ld_cols<kChunk>(tS + (QUAD ? 16 * (warp & 3) : 32 * c), sv[c]);
        tmem_wait_ld();
        if (cut || g.causal) {
          const uint64_t mask = diff_seen(g, s, k_nx, j0 + j, seen);
          if (__any_sync(0xFFFFFFFFu, mask != ~0ull)) {
            const uint32_t bits[2] = {static_cast<uint32_t>(QUAD ? mask >> (16 * (warp & 3)) : mask), static_cast<uint32_t>(mask >> 32)};
#pragma unroll
            for (int c = 0; c < kChunks; ++c)
#pragma unroll
              for (int i = 0; i < kChunk; ++i)
                if (!(bits[c] & (1u << i))) sv[c][i] = 0xFF800000u;
          }
        }
        constexpr int kRun = kChunks * kChunk / 4;   // four chains
        float tops[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint32_t* x = &sv[c * kRun / kChunk][c * kRun % kChunk];
          float q = max3_nan(__uint_as_float(x[0]), __uint_as_float(x[1]), __uint_as_float(x[2]));
#pragma unroll
          for (int i = 3; i + 1 < kRun; i += 2) q = max3_nan(q, __uint_as_float(x[i]), __uint_as_float(x[i + 1]));
          tops[c] = max_nan(q, __uint_as_float(x[kRun - 1]));
        }
        const float top = max_nan(max3_nan(tops[0], tops[1], tops[2]), tops[3]) * sl2;
        // keep the reference unless the tile exceeds it by 2^8; a NaN score becomes the reference, and the row NaN
        const float m_new = top <= mx + 8.f ? mx : top;
        const float alpha = m_new == mx ? 1.f : ex2_approx(mx - m_new);
        mx = m_new;
        if (j >= NP && __any_sync(0xFFFFFFFFu, alpha != 1.f)) {
          // O has to be complete up to the tile before: with NP = 2 S(j) was issued after that
          if (NP == 1 && !(ok = __all_sync(0xFFFFFFFFu, mbar_wait(&pv[b ^ 2], ((j - 1) >> 1) & 1, wc, SITE_PV)))) break;
          tc_fence_after();
          const uint32_t tO = tmem + lane_off + Lay::O + DV * (NP == 2 ? b : m);
#pragma unroll
          for (int c = 0; c < DV / 8; ++c) {
            uint32_t ov[8];
            tmem_ld8(tO + 8 * c, ov);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 8; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * alpha);
            tmem_st8(tO + 8 * c, ov);
          }
        }
        // rows that have seen nothing (a score of -inf is a key not seen): reference 0; a score of +inf has no softmax
        const float ref = mx == -INFINITY ? 0.f : mx + (mx - mx);
        const uint64_t scale2 = f2_pack(sl2, sl2), ref2 = f2_pack(-ref, -ref);
        uint64_t sum0 = f2_pack(l * alpha, 0.f), sum1 = f2_pack(0.f, 0.f);
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
          uint32_t pk[kChunk / 2];
#pragma unroll
          for (int i = 0; i < kChunk / 2; ++i) {
            const uint64_t x = f2_fma(f2_pack(__uint_as_float(sv[c][2 * i]), __uint_as_float(sv[c][2 * i + 1])), scale2, ref2);
            float x0, x1, p0, p1;
            f2_unpack(x, x0, x1);
            if ((i & 7) < POLY) {
              diff_exp2_poly(x0, x1, p0, p1);
            } else {
              p0 = ex2_approx(x0);
              p1 = ex2_approx(x1);
            }
            if (i & 1) sum1 = f2_add(sum1, f2_pack(p0, p1));
            else sum0 = f2_add(sum0, f2_pack(p0, p1));
            pk[i] = diff_pack<F16>(p0, p1);
          }
          if constexpr (QUAD) {
            const uint32_t none[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              if (k == (warp & 3)) tmem_st8(tS + 8 * k, pk);
              else tmem_st8(tS + 8 * k, none);
            }
          } else {
            tmem_st16(tS + 16 * c, pk);
          }
        }
        float s0, s1;
        f2_unpack(f2_add(sum0, sum1), s0, s1);
        l = s0 + s1;
        tmem_wait_st();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[b]);
    }
    const int last = n - 1 - (NP == 2 ? (n - 1 - p) & 1 : 0);   // this group's last tile (negative: none)
    if (ok && last >= 0) ok = warp_wait(&pv[2 * (last & 1) + m], (last >> 1) & 1, wc, SITE_PV);
    tc_fence_after();
    float* sm = reinterpret_cast<float*>(smem + Lay::OFF_L);
    sm[gi * 128 + row] = mx;
    sm[512 + gi * 128 + row] = l;
    // every group's sums and products are complete (all softmax warps meet, on a timeout too)
    asm volatile("bar.sync 1, %0;" ::"n"(128 * NG) : "memory");
    tc_fence_after();
    if (ok && *abort_flag == 0u && warp_live) {
      // c[gi]: what the group's O is multiplied with; 0 where it holds nothing
      float cf[NG], lse2[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float top = sm[i * 128 + row], sum = 0.f;
        if (NP == 2) top = max_nan(top, sm[(2 + i) * 128 + row]);
        const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll
        for (int k = 0; k < NP; ++k) {
          cf[2 * k + i] = ex2_approx(sm[(2 * k + i) * 128 + row] - ref);
          sum = fmaf(cf[2 * k + i], sm[512 + (2 * k + i) * 128 + row], sum);
        }
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
        for (int k = 0; k < NP; ++k) cf[2 * k + i] *= inv;
        lse2[i] = sum == 0.f ? -INFINITY : ref + log2f(sum);
      }
      const long long prow = a.part ? ((wide(s.b, g.kv_heads) + hk) * g.q_len + q.x) * g.group + q.head : 0;   // sequences only
      const long long prows = static_cast<long long>(g.batch) * g.q_heads * g.q_len;
      const int token = live ? s.token(q.x, q.y) : 0;
      const long long part = (static_cast<long long>(sp) * prows + prow) * 2;
      if (!QUAD && live && gi < 2 && a.part) a.part[static_cast<long long>(a.splits) * prows * 2 * g.dv + part + gi] = lse2[gi];
      if (live && gi < 2 && a.lse && !a.part)
        a.lse[((static_cast<long long>(gi) * g.batch + s.b) * g.q_heads + hq) * g.q_len + token] = lse2[gi] * kDiffLn2;
      const float lam = live ? diff_lambda<F16>(a.lam, g.lam_f32, hq) : 0.f;
      uint16_t* o = static_cast<uint16_t*>(a.o) + s.b * g.o.b + wide(token, g.o.t) + wide(hq, g.o.h);
      uint16_t* o2 = a.o2 ? static_cast<uint16_t*>(a.o2) + s.b * g.o.b + wide(token, g.o.t) + wide(hq, g.o.h) : nullptr;
      // group gi stores its share of the columns
#pragma unroll
      for (int c = 0; c < DV / NG / 8; ++c) {
        const int col = gi * (DV / NG) + 8 * c;
        float f[2][8];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int k = 0; k < NP; ++k) {
            uint32_t v[8];
            tmem_ld8(tmem + lane_off + Lay::O + DV * (2 * k + i) + col, v);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float x = cf[2 * k + i] == 0.f ? 0.f : __uint_as_float(v[e]) * cf[2 * k + i];
              f[i][e] = k == 0 ? x : f[i][e] + x;
            }
          }
        if (!live || col >= g.dv) continue;
        if constexpr (QUAD) {
          // [quarter][row][2 DV], then log-sum-exps [2][quarter][row]: the tiles are free by now
          float* w = reinterpret_cast<float*>(smem) + row * 2 * DV + col;
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int e = 0; e < 8; e += 4)
              *reinterpret_cast<float4*>(w + i * DV + e) = make_float4(f[i][e], f[i][e + 1], f[i][e + 2], f[i][e + 3]);
          continue;
        }
        if (a.part) {
          float* w = a.part + part * g.dv + col;
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int e = 0; e < 8; e += 4)
              *reinterpret_cast<float4*>(w + i * g.dv + e) = make_float4(f[i][e], f[i][e + 1], f[i][e + 2], f[i][e + 3]);
          continue;
        }
        uint32_t w[4], w2[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float d0 = fmaf(-lam, f[1][2 * e], f[0][2 * e]), d1 = fmaf(-lam, f[1][2 * e + 1], f[0][2 * e + 1]);
          w[e] = F16 ? pack_f16x2_sat(d0, d1) : pack_bf16x2(d0, d1);
          w2[e] = F16 ? pack_f16x2_sat(f[1][2 * e], f[1][2 * e + 1]) : pack_bf16x2(f[1][2 * e], f[1][2 * e + 1]);
        }
        *reinterpret_cast<uint4*>(o + col) = make_uint4(w[0], w[1], w[2], w[3]);
        if (o2) *reinterpret_cast<uint4*>(o2 + col) = make_uint4(w2[0], w2[1], w2[2], w2[3]);
      }
      if (QUAD && gi < 2) reinterpret_cast<float*>(smem)[128 * 2 * DV + gi * 128 + row] = lse2[gi];
    }
    if constexpr (QUAD) {
      // the quarters' parts of a row into this split's
      asm volatile("bar.sync 1, %0;" ::"n"(128 * NG) : "memory");
      const int live_rows = s.wq * g.group, columns = 2 * g.dv;
      const long long prows = static_cast<long long>(g.batch) * g.q_heads * g.q_len;
      if (ok && *abort_flag == 0u)
        for (int i = threadIdx.x; i < live_rows * columns; i += 128 * NG) {
          const int rr = i / columns, c = i - rr * columns, m = c >= g.dv, cc = c - m * g.dv;
          float l[4], top = -INFINITY;
#pragma unroll
          for (int k = 0; k < 4; ++k) top = max_nan(top, l[k] = reinterpret_cast<const float*>(smem)[128 * 2 * DV + m * 128 + 32 * k + rr]);
          const float ref = top == -INFINITY ? 0.f : top;
          float sum = 0.f, v = 0.f;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float w = exp2f(l[k] - ref);
            sum += w;
            v = fmaf(w, reinterpret_cast<const float*>(smem)[(32 * k + rr) * 2 * DV + m * DV + cc], v);
          }
          const int t = diff_row_token(g, rr);
          const long long prow = ((wide(s.b, g.kv_heads) + hk) * g.q_len + t) * g.group + rr - t * g.group;
          const long long part = (static_cast<long long>(sp) * prows + prow) * 2;
          a.part[part * g.dv + m * g.dv + cc] = sum == 0.f ? 0.f : v / sum;
          if (cc == 0) a.part[static_cast<long long>(a.splits) * prows * 2 * g.dv + part + m] = sum == 0.f ? -INFINITY : ref + log2f(sum);
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

// The parts of one (batch item, key head, token, head of the group) row over
// its key splits, weighted by their sums: a CTA a row. Its threads are
// 2 dv / 4 pieces of the two maps' outputs times groups that share the parts.
constexpr int kJoinThreads = 256, kMostParts = 64;
template <bool F16>
__global__ void __launch_bounds__(kJoinThreads) diff_attn_join_kernel(const DiffFwdArgs a) {
  __shared__ float weight[2][kMostParts];
  __shared__ float lse2[2];
  __shared__ float4 sums[kJoinThreads];
  const DiffGeom& g = a.g;
  const long long prows = static_cast<long long>(g.batch) * g.q_heads * g.q_len, prow = blockIdx.x;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (warp < 2) {
    // warp m: weights of map m's parts
    const float* l = a.part + static_cast<long long>(a.splits) * prows * 2 * g.dv + prow * 2 + warp;
    float top = -INFINITY, sum = 0.f;
    for (int s = lane; s < a.splits; s += 32) top = max_nan(top, weight[warp][s] = l[s * prows * 2]);
    for (int o = 16; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    const float ref = top == -INFINITY ? 0.f : top;
    for (int s = lane; s < a.splits; s += 32) sum += weight[warp][s] = exp2f(weight[warp][s] - ref);
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    for (int s = lane; s < a.splits; s += 32) weight[warp][s] *= inv;
    if (lane == 0) lse2[warp] = sum == 0.f ? -INFINITY : ref + log2f(sum);
  }
  __syncthreads();
  const int pieces = g.dv / 2, groups = kJoinThreads / pieces, piece = threadIdx.x % pieces, gr = threadIdx.x / pieces;
  if (gr < groups) {
    const int m = piece >= g.dv / 4;
    const float* p = a.part + prow * 2 * g.dv + piece * 4;
    float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int s = gr; s < a.splits; s += groups) {
      const float4 v = *reinterpret_cast<const float4*>(p + s * prows * 2 * g.dv);
      const float w = weight[m][s];
      f.x = fmaf(w, v.x, f.x); f.y = fmaf(w, v.y, f.y); f.z = fmaf(w, v.z, f.z); f.w = fmaf(w, v.w, f.w);
    }
    sums[gr * pieces + piece] = f;
  }
  __syncthreads();
  const int gh = static_cast<int>(prow % g.group), t = static_cast<int>(prow / g.group % g.q_len);
  const int hk = static_cast<int>(prow / (static_cast<long long>(g.group) * g.q_len) % g.kv_heads);
  const int b = static_cast<int>(prow / (static_cast<long long>(g.group) * g.q_len * g.kv_heads));
  const int hq = hk * g.group + gh;
  if (threadIdx.x < g.dv / 4) {
    float f[2][4];
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int k = 0; k < groups; ++k) {
        const float4 u = sums[k * pieces + m * (g.dv / 4) + threadIdx.x];
        v.x += u.x; v.y += u.y; v.z += u.z; v.w += u.w;
      }
      f[m][0] = v.x; f[m][1] = v.y; f[m][2] = v.z; f[m][3] = v.w;
    }
    const float lam = diff_lambda<F16>(a.lam, g.lam_f32, hq);
    uint32_t w[2], w2[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float d0 = fmaf(-lam, f[1][2 * e], f[0][2 * e]), d1 = fmaf(-lam, f[1][2 * e + 1], f[0][2 * e + 1]);
      w[e] = F16 ? pack_f16x2_sat(d0, d1) : pack_bf16x2(d0, d1);
      w2[e] = F16 ? pack_f16x2_sat(f[1][2 * e], f[1][2 * e + 1]) : pack_bf16x2(f[1][2 * e], f[1][2 * e + 1]);
    }
    const long long to = b * g.o.b + wide(t, g.o.t) + wide(hq, g.o.h) + threadIdx.x * 4;
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.o) + to) = make_uint2(w[0], w[1]);
    if (a.o2) *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.o2) + to) = make_uint2(w2[0], w2[1]);
  }
  if (a.lse && threadIdx.x < 2)
    a.lse[((static_cast<long long>(threadIdx.x) * g.batch + b) * g.q_heads + hq) * g.q_len + t] = lse2[threadIdx.x] * kDiffLn2;
}

template <int D, int DV, bool F16>
cudaError_t launch_class(const DiffFwdArgs& a, cudaStream_t stream) {
  using Lay = FwdLay<D, DV>;
  // Of 8 pairs, those on the FMA pipe: at dv <= 32 the softmax warps' own instructions bound too (window 64 map: 868 us
  // with none, 872 with two); at 64 and 128 two are best (128 -> 124 us, 140 -> 134 us)
  constexpr int POLY = DV <= 32 ? 0 : 2;
  auto kernel = a.quad ? diff_attn_fwd_kernel<D, DV, F16, 0, true> : diff_attn_fwd_kernel<D, DV, F16, POLY, false>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay::ALLOC);
  if (e != cudaSuccess) return e;
  const DiffGeom& g = a.g;
  const int q_tiles = ceil_div(diff_max_q_boxes(g), 2);
  const long long ctas = static_cast<long long>(diff_sequences(g)) * g.kv_heads * q_tiles * a.splits;
  if (ctas > 0x7FFFFFFFll) return cudaErrorInvalidConfiguration;
  CUtensorMap q1, q2, k1, k2, v;
  using TQ = typename Lay::TQ;
  using TV = typename Lay::TV;
  if (!diff_map(&q1, g, true, F16, a.q1, g.q, g.d, TQ::COLS) || !diff_map(&q2, g, true, F16, a.q2, g.q, g.d, TQ::COLS) ||
      !diff_map(&k1, g, false, F16, a.k1, g.k, g.d, TQ::COLS) || !diff_map(&k2, g, false, F16, a.k2, g.k, g.d, TQ::COLS) ||
      !diff_map(&v, g, false, F16, a.v, g.v, g.dv, TV::COLS))
    return cudaErrorInvalidValue;
  kernel<<<static_cast<unsigned>(ctas), Lay::kThreads, Lay::ALLOC, stream>>>(q1, q2, k1, k2, v, a, q_tiles);
  if ((e = cudaGetLastError()) != cudaSuccess || !a.part) return e;
  const long long rows = static_cast<long long>(g.batch) * g.q_heads * g.q_len;   // few: the keys are split because they are
  diff_attn_join_kernel<F16><<<static_cast<unsigned>(rows), kJoinThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

// CTAs that share a query tile's keys: the number with the least estimate of
// time, of four boxes each at least. A key box takes a CTA about 0.75 us, in the
// form for few rows 0.55; its start and end as much as four; the join 6 us and
// 4.2 ns a row (a CTA each). Measured, in us by the number of parts:
//   16 x 1 token, 8192 keys, 16 on 4 heads of 64/128   121 (1)  72 (2)  88 (3)  78 (4)
//   32 x 1 token, 1024 keys, the same heads             27 (1)  40 (2)  53 (4)
//   128 tokens, 8192 keys, 4 heads of 64/128           119 (1)  49 (4)  31 (16)  29 (32)  41 (64)
//   256 tokens, 4096 keys, 8 heads of 64/128            66 (1)  43 (4)  38 (8)  51 (12)
//   1024 tokens, 1024 keys, 6 heads of 16/32            21 (1)  45 (2)  45 (3)
int diff_splits(const DiffGeom& g) {
  if (g.window || g.q_len == 0 || g.batch == 0) return 1;
  const bool few = diff_few_rows(g);
  const long long units = static_cast<long long>(g.batch) * g.kv_heads * ceil_div(diff_max_q_boxes(g), 2);
  const int sms = sm_count(), boxes = ceil_div(g.k_len, kBK);
  if (units >= (few ? 4ll : 1ll) * sms) return 1;
  const auto rounds = [&](int s) { return static_cast<float>((units * s + sms - 1) / sms) * (ceil_div(boxes, s) + 4); };
  const float join = 6.f + 0.0042f * (static_cast<float>(g.batch) * g.q_heads * g.q_len);
  int best = 1;
  float least = rounds(1) * 0.75f;
  for (int s = 2; s <= kMostParts && 4 * s <= boxes; ++s) {
    const float us = rounds(s) * (few ? 0.55f : 0.75f) + join;
    if (us < least) {
      least = us;
      best = s;
    }
  }
  return best;
}

size_t diff_split_bytes(const DiffGeom& g) {
  const int s = diff_splits(g);
  return s > 1 ? static_cast<size_t>(s) * g.batch * g.q_heads * g.q_len * 2 * (g.dv + 1) * sizeof(float) : 0;
}

bool diff_map(CUtensorMap* map, const DiffGeom& g, bool query, bool f16, const void* p, const DiffStrides& s, int e, int cols) {
  const int heads = query ? g.q_heads : g.kv_heads, len = query ? g.q_len : g.k_len;
  const uint64_t x = static_cast<uint64_t>(g.window ? g.width : len), y = static_cast<uint64_t>(g.window ? g.height : 1);
  *map = CUtensorMap{};
  if (len == 0 || g.batch == 0) return true;   // nothing to load
  const uint64_t dims[5] = {static_cast<uint64_t>(e), static_cast<uint64_t>(heads), x, y, static_cast<uint64_t>(g.batch)};
  const uint64_t raw[4] = {static_cast<uint64_t>(s.h) * 2, static_cast<uint64_t>(s.t) * 2, static_cast<uint64_t>(s.t) * 2 * x,
                           static_cast<uint64_t>(s.b) * 2};
  uint64_t strides[4];
  for (int i = 0; i < 4; ++i) strides[i] = dims[i + 1] > 1 ? raw[i] : 16;   // an axis of one place is never stepped along
  const uint32_t box[5] = {static_cast<uint32_t>(cols), static_cast<uint32_t>(query ? g.group : 1), static_cast<uint32_t>(query ? g.tcq : g.tck),
                           static_cast<uint32_t>(query ? g.trq : g.trk), 1};
  const CUtensorMapSwizzle sw = cols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : (cols == 32 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_32B);
  return encode_tiled(map, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(p), dims, strides, box,
                      sw) == CUDA_SUCCESS;
}

cudaError_t launch_diff_attn_fwd(const DiffFwdArgs& a, bool f16, cudaStream_t stream) {
  switch (diff_class(a.g.d, a.g.dv)) {
    case 0: return f16 ? launch_class<16, 32, true>(a, stream) : launch_class<16, 32, false>(a, stream);
    case 1: return f16 ? launch_class<32, 64, true>(a, stream) : launch_class<32, 64, false>(a, stream);
    default: return f16 ? launch_class<64, 128, true>(a, stream) : launch_class<64, 128, false>(a, stream);
  }
}

}  // namespace rib
