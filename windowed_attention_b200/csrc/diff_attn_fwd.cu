// Differential attention, forward (rib_diff_attention):
//   O = (softmax(s Q1 K1^T) - lambda softmax(s Q2 K2^T)) V
// per sequence and head, lambda learned per query head.
//
// One pass over the keys: each of the two maps keeps its own running maximum m
// and sum l, O_i accumulates 2^(s' S_i - m_i) V (s' = s log2 e) and the output
// is O_1 / l_1 - lambda O_2 / l_2, formed once at the end. The maximum is
// raised (and O_i scaled) only when a tile exceeds it by 2^8, so P <= 256.
// P takes the 16-bit type for its product with V (half a step of each term);
// scores, sums and both O_i stay fp32.
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
//   then kLoadWarps      loaders: cp.async rows into swizzled tiles (any strides,
//                        windows cut anywhere; masked keys become zero rows)
// TMEM: S of map m and parity q at 64 (2 q + m), O from column 256.
//
// Bound: the exponentials, 2 per (query, key) pair: a tile of 128 x 64 x 2
// takes 1024 cycles of the SM's MUFU, of which the FMA pipe takes over POLY of
// every 8 pairs. Its products take 2 (48 D / 16 + 4 max(DV / 2, 32 + DV / 4)) cycles.
#include <cuda_runtime.h>

#include "diff_attn.cuh"

namespace rib {
namespace {

#ifndef RIB_DIFF_POLY_F
#define RIB_DIFF_POLY_F 2
#endif
constexpr int kBK = 64;

enum Site : int {
  SITE_Q = 401, SITE_KV_FULL = 402, SITE_KV_EMPTY = 403, SITE_S = 404, SITE_P = 405, SITE_PV = 406, SITE_DONE = 407,
};

template <int D, int DV>
struct FwdLay {
  using TQ = DiffTile<128, D>;
  using TK = DiffTile<kBK, D>;
  using TV = DiffTile<kBK, DV>;
  static constexpr int NP = DV <= 64 ? 2 : 1;               // O accumulators of a map
  static constexpr int NG = 2 * NP;
  static constexpr int kLoadWarps = 2;
  static constexpr int kThreads = 32 * (4 * NG + 2 + kLoadWarps);
  static constexpr int STAGE = 2 * TK::BYTES + TV::BYTES;
  static constexpr int NS = STAGE <= 16 * 1024 ? 6 : 4;
  static constexpr int OFF_ST = 2 * TQ::BYTES;
  static constexpr int OFF_L = OFF_ST + NS * STAGE;         // [4][128] m, then [4][128] l of each group
  static constexpr int OFF_BAR = OFF_L + 2 * 4 * 128 * 4;
  static constexpr int NBAR = 1 + 2 * NS + 12 + 1;          // q, kv_full, kv_empty, s[4], p[4], pv[4], done
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
  static constexpr int ALLOC = OFF_MISC + 16 + 1024;
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

template <int D, int DV, bool F16, int POLY>
__global__ void __launch_bounds__(FwdLay<D, DV>::kThreads, 1) diff_attn_fwd_kernel(const DiffFwdArgs a, int q_tiles) {
  using Lay = FwdLay<D, DV>;
  using TQ = typename Lay::TQ;
  using TK = typename Lay::TK;
  using TV = typename Lay::TV;
  constexpr int NS = Lay::NS, NP = Lay::NP, NG = Lay::NG, kLoadWarps = Lay::kLoadWarps, kLoaders = 32 * kLoadWarps;
  constexpr int kWarpS = 4 * NG, kWarpPV = kWarpS + 1, kWarpLoad = kWarpS + 2;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align_smem_1024(smem_raw);
  uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + Lay::OFF_BAR);
  uint64_t* kv_full = q_full + 1;
  uint64_t* kv_empty = kv_full + NS;
  uint64_t* s_full = kv_empty + NS;   // [2 q + m], as the two below
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
  const int rows = s.nq * g.group, row0 = qt * 128;
  if (row0 >= rows) return;   // a window at the map's edge has fewer tiles
  const int last_t = diff_row_token(g, min(row0 + 128, rows) - 1);
  const int tiles = (diff_visible(g, s, last_t) + kBK - 1) / kBK;
  const int per = (tiles + a.splits - 1) / a.splits;
  const int j0 = sp * per, n = max(0, min(tiles, j0 + per) - j0);

  if (threadIdx.x == 0) {
    mbar_init(q_full, kLoadWarps);
    for (int i = 0; i < NS; ++i) {
      mbar_init(&kv_full[i], kLoadWarps);
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
  if (warp == kWarpS) {
    tmem_alloc(tmem_holder, Lay::COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const WaitCtx wc{abort_flag, a.err};

  if (warp >= kWarpLoad) {
    // ------------------------------------------------------------ loaders
    const int tid = threadIdx.x - kWarpLoad * 32;
    const uint32_t sq = smem_u32(smem), sst = sq + Lay::OFF_ST;
    const uint16_t* q1 = static_cast<const uint16_t*>(a.q1) + s.b * g.q.b + static_cast<long long>(hk) * g.group * g.q.h;
    const uint16_t* q2 = static_cast<const uint16_t*>(a.q2) + s.b * g.q.b + static_cast<long long>(hk) * g.group * g.q.h;
    const uint16_t* k1 = static_cast<const uint16_t*>(a.k1) + s.b * g.k.b + hk * g.k.h;
    const uint16_t* k2 = static_cast<const uint16_t*>(a.k2) + s.b * g.k.b + hk * g.k.h;
    const uint16_t* v = static_cast<const uint16_t*>(a.v) + s.b * g.v.b + hk * g.v.h;
    int told = -1;   // the last load whose barrier this warp has arrived on (-1: none, 0: Q, i + 1: key tile i)
    auto tell = [&](int upto) {
      if (upto <= told) return;
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0)
        for (int i = told + 1; i <= upto; ++i) mbar_arrive(i == 0 ? q_full : &kv_full[(i - 1) % NS]);
      told = upto;
    };
    if (n > 0) {
      diff_clear<D, DV, kLoaders>(smem, Lay::OFF_L, g, tid);
      diff_load_queries<128, D, DV, kLoaders>(sq, q1, q2, nullptr, g, s, row0, rows, tid);
      cp_async_commit();
    }
    for (int i = 0; i < n; ++i) {
      const int st = i % NS;
      if (i >= NS) {
        const uint32_t parity = ((i / NS) - 1) & 1;
        if (!__all_sync(0xFFFFFFFFu, mbar_test_wait(&kv_empty[st], parity))) {
          // about to wait: first hand over everything that is on its way
          cp_async_wait<0>();
          tell(i);
          if (!__all_sync(0xFFFFFFFFu, mbar_wait(&kv_empty[st], parity, wc, SITE_KV_EMPTY))) break;
        }
      }
      const uint32_t b = sst + st * Lay::STAGE;
      const int first = (j0 + i) * kBK;
      diff_load_keys<kBK, D, DV, kLoaders>(b, k1, k2, v, g, s, first, s.nk, tid);
      cp_async_commit();
      cp_async_wait<2>();
      tell(i - 1);   // all but the two newest groups
    }
    cp_async_wait<0>();
    if (n > 0 && *abort_flag == 0u) tell(n);
  } else if (warp == kWarpS) {
    // --------------------------------------------------------- S issuer
    if (lane == 0 && n > 0) {
      const uint32_t sq = smem_u32(smem), sst = sq + Lay::OFF_ST;
      const uint32_t id_s = diff_idesc(F16, kBK, false);
      const int ks_d = (g.d + 15) / 16;
      bool ok = mbar_wait(q_full, 0, wc, SITE_Q);
      for (int j = 0; ok && j < n; ++j) {
        if (!(ok = mbar_wait(&kv_full[j % NS], (j / NS) & 1, wc, SITE_KV_FULL))) break;
        for (int m = 0; m < 2; ++m) {
          const int b = 2 * (j & 1) + m;
          // S overwrites the P of two tiles before: its product has to be done with it
          if (j >= 2 && !(ok = mbar_wait(&pv[b], ((j - 2) >> 1) & 1, wc, SITE_PV))) break;
          tc_fence_after();
          const uint32_t q = sq + m * TQ::BYTES, k = sst + (j % NS) * Lay::STAGE + m * TK::BYTES;
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks)
            if (ks < ks_d) umma_ss(tmem + 64u * b, TQ::kmajor(q, ks), TK::kmajor(k, ks), id_s, ks > 0 ? 1u : 0u);
          umma_commit(&s_full[b]);
        }
      }
      umma_commit(done);
      const WaitCtx drain{tmem_holder + 2, a.err};
      mbar_wait(done, 0, drain, SITE_DONE);
    }
  } else if (warp == kWarpPV) {
    // ------------------------------------------------------- P V issuer
    if (lane == 0 && n > 0) {
      const uint32_t sst = smem_u32(smem) + Lay::OFF_ST;
      const uint32_t id_o = diff_idesc(F16, (g.dv + 15) / 16 * 16, true);
      bool ok = true;
      for (int j = 0; ok && j < n; ++j) {
        const uint32_t vb = sst + (j % NS) * Lay::STAGE + 2 * TK::BYTES;
        for (int m = 0; m < 2; ++m) {
          const int b = 2 * (j & 1) + m;
          if (!(ok = mbar_wait(&p_full[b], (j >> 1) & 1, wc, SITE_P))) break;
          tc_fence_after();
          const uint32_t o = tmem + Lay::O + DV * (NP == 2 ? b : m);
#pragma unroll
          for (int ks = 0; ks < kBK / 16; ++ks)
            umma_ts(o, tmem + 64u * b + 8u * ks, TV::mnmajor(vb, ks), id_o, (j >= NP || ks > 0) ? 1u : 0u);
          umma_commit(&pv[b]);
          if (m == 1) umma_commit(&kv_empty[j % NS]);   // S of the tile was done before its P was written
        }
      }
      umma_commit(done);
      const WaitCtx drain{tmem_holder + 2, a.err};
      mbar_wait(done, 0, drain, SITE_DONE);
    }
  } else {
    // ------------------------------------------------------------ softmax
    const int gi = warp >> 2, m = gi & 1, p = gi >> 1;   // map and, with NP = 2, the parity of its tiles
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const int r = row0 + row;
    const bool live = r < rows;
    const int t = diff_row_token(g, r), hq = hk * g.group + (r - t * g.group);
    const int seen = live ? diff_visible(g, s, t) : 0;
    const bool warp_live = row0 + (warp & 3) * 32 < rows;   // a warp without rows only keeps the barriers going
    const float sl2 = g.scale_log2;
    float mx = -INFINITY, l = 0.f;
    bool ok = true;
    for (int j = p; j < n; j += NP) {
      const int b = 2 * (j & 1) + m;
      const uint32_t tS = tmem + lane_off + 64u * b;
      ok = __all_sync(0xFFFFFFFFu, mbar_wait(&s_full[b], (j >> 1) & 1, wc, SITE_S));
      if (!ok) break;
      tc_fence_after();
      if (warp_live) {
        uint32_t sv[2][32];
        tmem_ld32(tS, sv[0]);
        tmem_ld32(tS + 32, sv[1]);
        tmem_wait_ld();
        const int left = seen - (j0 + j) * kBK;   // keys of this tile that the row sees
        if (__any_sync(0xFFFFFFFFu, left < kBK)) {
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (32 * c + i >= left) sv[c][i] = 0xFF800000u;
        }
        float tops[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {   // four chains of eight
          const uint32_t* x = &sv[c >> 1][16 * (c & 1)];
          float q = max3_nan(__uint_as_float(x[0]), __uint_as_float(x[1]), __uint_as_float(x[2]));
#pragma unroll
          for (int i = 3; i + 1 < 16; i += 2) q = max3_nan(q, __uint_as_float(x[i]), __uint_as_float(x[i + 1]));
          tops[c] = max_nan(q, __uint_as_float(x[15]));
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
        // rows that have seen nothing: reference 0; an infinite score has no softmax
        const float ref = mx == -INFINITY ? 0.f : mx + (mx - mx);
        const uint64_t scale2 = f2_pack(sl2, sl2), ref2 = f2_pack(-ref, -ref);
        uint64_t sum0 = f2_pack(l * alpha, 0.f), sum1 = f2_pack(0.f, 0.f);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t pk[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
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
          tmem_st16(tS + 16 * c, pk);
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
    if (ok && last >= 0) ok = __all_sync(0xFFFFFFFFu, mbar_wait(&pv[2 * (last & 1) + m], (last >> 1) & 1, wc, SITE_PV));
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
      const long long prow = a.part ? ((static_cast<long long>(s.b) * g.kv_heads + hk) * g.q_len * g.group + r) : 0;   // window 0 only
      const long long prows = static_cast<long long>(g.batch) * g.q_heads * g.q_len;
      const long long token = live ? s.token(t) : 0;
      if (live && gi < 2 && a.part)
        a.part[static_cast<long long>(a.splits) * prows * 2 * g.dv + (static_cast<long long>(sp) * prows + prow) * 2 + gi] = lse2[gi];
      if (live && gi < 2 && a.lse && !a.part)
        a.lse[((static_cast<long long>(gi) * g.batch + s.b) * g.q_heads + hq) * g.q_len + token] = lse2[gi] * kDiffLn2;
      const float lam = live ? diff_lambda<F16>(a.lam, g.lam_f32, hq) : 0.f;
      uint16_t* o = static_cast<uint16_t*>(a.o) + s.b * g.o.b + token * g.o.t + hq * g.o.h;
      uint16_t* o2 = a.o2 ? static_cast<uint16_t*>(a.o2) + s.b * g.o.b + token * g.o.t + hq * g.o.h : nullptr;
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
        if (a.part) {
          float* w = a.part + (static_cast<long long>(sp) * prows + prow) * 2 * g.dv + col;
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
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kWarpS) {
    tc_fence_after();
    tmem_dealloc(tmem, Lay::COLS);
  }
}

// The parts of a row over its key splits, weighted by their sums: a thread
// owns eight columns of one (batch item, query head, token) row of both maps.
template <bool F16>
__global__ void __launch_bounds__(256) diff_attn_join_kernel(const DiffFwdArgs a) {
  const DiffGeom& g = a.g;
  const int pieces = g.dv / 8;
  const long long prows = static_cast<long long>(g.batch) * g.q_heads * g.q_len;
  const long long at = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
  const long long prow = at / pieces;
  const int c = static_cast<int>(at - prow * pieces) * 8;
  if (prow >= prows) return;
  // rows are [batch][key head][token][head of the group]
  const int gh = static_cast<int>(prow % g.group), t = static_cast<int>(prow / g.group % g.q_len);
  const int hk = static_cast<int>(prow / (static_cast<long long>(g.group) * g.q_len) % g.kv_heads);
  const int b = static_cast<int>(prow / (static_cast<long long>(g.group) * g.q_len * g.kv_heads));
  const int hq = hk * g.group + gh;
  const float* sums = a.part + static_cast<long long>(a.splits) * prows * 2 * g.dv;
  float f[2][8], lse2[2];
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    float top = -INFINITY;
    for (int s = 0; s < a.splits; ++s) top = max_nan(top, sums[(s * prows + prow) * 2 + m]);
    const float ref = top == -INFINITY ? 0.f : top;
    float l = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) f[m][e] = 0.f;
    for (int s = 0; s < a.splits; ++s) {
      const float w = exp2f(sums[(s * prows + prow) * 2 + m] - ref);
      const float4* p = reinterpret_cast<const float4*>(a.part + ((s * prows + prow) * 2 + m) * g.dv + c);
      const float4 lo = p[0], hi = p[1];
      l += w;
      const float v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
      for (int e = 0; e < 8; ++e) f[m][e] = fmaf(w, v[e], f[m][e]);
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    lse2[m] = l == 0.f ? -INFINITY : ref + log2f(l);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[m][e] *= inv;
  }
  const float lam = diff_lambda<F16>(a.lam, g.lam_f32, hq);
  uint32_t w[4], w2[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float d0 = fmaf(-lam, f[1][2 * e], f[0][2 * e]), d1 = fmaf(-lam, f[1][2 * e + 1], f[0][2 * e + 1]);
    w[e] = F16 ? pack_f16x2_sat(d0, d1) : pack_bf16x2(d0, d1);
    w2[e] = F16 ? pack_f16x2_sat(f[1][2 * e], f[1][2 * e + 1]) : pack_bf16x2(f[1][2 * e], f[1][2 * e + 1]);
  }
  const long long to = b * g.o.b + t * g.o.t + hq * g.o.h + c;
  *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.o) + to) = make_uint4(w[0], w[1], w[2], w[3]);
  if (a.o2) *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.o2) + to) = make_uint4(w2[0], w2[1], w2[2], w2[3]);
  if (a.lse && c == 0)
#pragma unroll
    for (int m = 0; m < 2; ++m)
      a.lse[((static_cast<long long>(m) * g.batch + b) * g.q_heads + hq) * g.q_len + t] = lse2[m] * kDiffLn2;
}

template <int D, int DV, bool F16>
cudaError_t launch_class(const DiffFwdArgs& a, cudaStream_t stream) {
  using Lay = FwdLay<D, DV>;
  constexpr int POLY = RIB_DIFF_POLY_F;
  auto kernel = diff_attn_fwd_kernel<D, DV, F16, POLY>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay::ALLOC);
  if (e != cudaSuccess) return e;
  const int q_tiles = static_cast<int>((diff_max_rows(a.g) + 127) / 128);
  const long long ctas = static_cast<long long>(diff_sequences(a.g)) * a.g.kv_heads * q_tiles * a.splits;
  if (ctas > 0x7FFFFFFFll) return cudaErrorInvalidConfiguration;
  if (ctas == 0) return cudaSuccess;
  kernel<<<static_cast<unsigned>(ctas), Lay::kThreads, Lay::ALLOC, stream>>>(a, q_tiles);
  if ((e = cudaGetLastError()) != cudaSuccess || !a.part) return e;
  const long long threads = static_cast<long long>(a.g.batch) * a.g.q_heads * a.g.q_len * (a.g.dv / 8);
  diff_attn_join_kernel<F16><<<static_cast<unsigned>((threads + 255) / 256), 256, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

// Keys are split over CTAs when the query tiles alone leave most SMs idle: as
// many splits as fill them, each of at least four tiles of keys.
int diff_splits(const DiffGeom& g) {
  if (g.window || g.q_len == 0 || g.batch == 0) return 1;
  const long long units = static_cast<long long>(g.batch) * g.kv_heads * ((diff_max_rows(g) + 127) / 128);
  const long long tiles = (g.k_len + kBK - 1) / kBK;
  const long long want = 2 * sm_count() / units, most = tiles / 4;
  const long long s = want < most ? want : most;
  return s > 1 ? static_cast<int>(s < 64 ? s : 64) : 1;
}

size_t diff_split_bytes(const DiffGeom& g) {
  const int s = diff_splits(g);
  return s > 1 ? static_cast<size_t>(s) * g.batch * g.q_heads * g.q_len * 2 * (g.dv + 1) * sizeof(float) : 0;
}

cudaError_t launch_diff_attn_fwd(const DiffFwdArgs& a, bool f16, cudaStream_t stream) {
  switch (diff_class(a.g.d, a.g.dv)) {
    case 0: return f16 ? launch_class<16, 32, true>(a, stream) : launch_class<16, 32, false>(a, stream);
    case 1: return f16 ? launch_class<32, 64, true>(a, stream) : launch_class<32, 64, false>(a, stream);
    default: return f16 ? launch_class<64, 128, true>(a, stream) : launch_class<64, 128, false>(a, stream);
  }
}

}  // namespace rib
