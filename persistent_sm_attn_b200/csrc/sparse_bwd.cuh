// Block-sparse attention backward for sm_100a.
//
//   P  = 2^(s S - LSE log2 e) on the visible keys of the picked units, 0 elsewhere
//   dP = dO V^T,  delta = rowsum(dO o O),  dS = P o (dP - delta)
//   dQ = scale dS K,   dK = scale dS^T Q,   dV = P^T dO
//
// Two passes recompute S and dP, each with its result resident in TMEM, so that every sum
// has one owner and a fixed order and no partial of dQ goes through memory:
//   dash_sparse_dq_kernel   walks the listed units of a query tile, as the forward does;
//   dash_sparse_dkdv_kernel a persistent CTA per SM takes items: a unit of 64 keys and a
//                           stretch of the tokens that picked it.
// A unit that many tokens picked (the first block of a causal sequence) is cut into stretches;
// their fp32 partials are added in order by dash_sparse_finish_kernel.  Results are bitwise
// reproducible.
#pragma once
#include "ptx.cuh"
#include "sparse_fwd.cuh"
#include "sparse_plan.cuh"

namespace dash {

// ------------------------------------------------------------------ delta
// delta = rowsum(dO o O) of every row, D / 8 lanes a row, four rows in flight a lane.  Bound
// by reading O and dO: 67 MB in 13.6 us.  (Taken by two warps of the dQ kernel a tile ahead it
// kept the softmax waiting, 276 us for 232 + 13.)
struct SparseDeltaParams {
  const __nv_bfloat16 *o, *dout;
  long long ob, oh, os;  // strides of dout in elements
  float* delta;
  int H, Sq;
  long long rows;
};
template <int D>
__global__ void __launch_bounds__(256) dash_sparse_delta_kernel(const SparseDeltaParams p) {
  constexpr int CH = D / 8, RP = 256 / CH;
  const int c = threadIdx.x % CH;
  const long long row0 = (long long)blockIdx.x * (4 * RP) + threadIdx.x / CH;
  uint4 x[4], z[4];
#pragma unroll
  for (int y = 0; y < 4; ++y) {
    const long long row = min(row0 + y * RP, p.rows - 1);
    const int bh = (int)(row / p.Sq), i = (int)(row - (long long)bh * p.Sq);
    const int b = bh / p.H, h = bh - b * p.H;
    x[y] = __ldcs(reinterpret_cast<const uint4*>(p.o + row * D) + c);
    z[y] = *reinterpret_cast<const uint4*>(p.dout + b * p.ob + h * p.oh + i * p.os + c * 8);
  }
#pragma unroll
  for (int y = 0; y < 4; ++y) {
    const uint32_t xs[4] = {x[y].x, x[y].y, x[y].z, x[y].w};
    const uint32_t zs[4] = {z[y].x, z[y].y, z[y].z, z[y].w};
    float sum = 0.f;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      sum = fmaf(__uint_as_float(xs[q] << 16), __uint_as_float(zs[q] << 16), sum);
      sum = fmaf(__uint_as_float(xs[q] & 0xffff0000u), __uint_as_float(zs[q] & 0xffff0000u), sum);
    }
#pragma unroll
    for (int o = CH / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const long long row = row0 + y * RP;
    if (c == 0 && row < p.rows) p.delta[row] = sum;
  }
}

// The k-th of this CTA's items of a list whose longest come first: the CTAs take them in turns
// that go to and fro, so that all get nearly the same sum.  Ascending in k.
__device__ __forceinline__ int snake_item(int k) {
  const int x = (int)blockIdx.x, g = (int)gridDim.x;
  return k * g + ((k & 1) ? g - 1 - x : x);
}

// ------------------------------------------------------------------ dQ
struct SparseDqParams {
  PlanView plan;
  const float* lse;    // [B,H,Sq]
  const float* delta;  // [B,H,Sq]
  __nv_bfloat16* dq;   // [B,H,Sq,D]
  unsigned* err;
  int Hkv, Sq, Sk, G, T, W, NT, U, tiles, causal;
  int loads;  // units that the producer loads (all, but for a planted fault)
  float scale, scale_log2;
  unsigned long long spin_ns;
};

template <int D>
struct SparseDqCfg {
  static constexpr int kThreads = 384;  // TMA, S and dP of either stream, dQ, 8 warps of softmax
  static constexpr int kTile = kTileRows * D * 2;
  static constexpr int kKV = kUnit * D * 2;
  // tiles of Q and dO, units of K and of V (even: a stage belongs to one stream): K is read
  // twice and stays longer than V
  static constexpr int kQ = D == 128 ? 1 : 2, kK = D == 128 ? 6 : 8, kV = D == 128 ? 4 : 8;
  static constexpr int OFF_Q = 0;  // Q, then dO
  static constexpr int OFF_K = kQ * 2 * kTile;
  static constexpr int OFF_V = OFF_K + kK * kKV;
  static constexpr int OFF_BAR = OFF_V + kV * kKV;
  static constexpr int kBars = 2 * kK + 2 * kV + 2 * 4 + 2 * 6 + 3 + 1;
  static constexpr int OFF_SLOT = OFF_BAR + kBars * 8;
  static constexpr int kSmemBytes = OFF_SLOT + 16;
  static_assert(kSmemBytes <= 232448, "shared memory per block exceeded");
  static_assert(kSmemBytes > 116 * 1024, "one CTA per SM: its 512 TMEM columns are free");
  static constexpr int kAcc = D == 128 ? 1 : 2;  // accumulators
  static constexpr uint32_t TM_S = 0, TM_DQ = 384, kTmemCols = 512;
};

// A persistent CTA per SM takes query tiles, those with the longest lists (the last, under a
// causal mask) first, in turns that go to and fro.  Per listed unit j: S = Q K^T, dP = dO V^T
// (128 x 64, TMEM), dS in bf16 over S, dQ += dS K.  Even and odd units have an issuer of S and dP
// and a softmax warpgroup each, so that one unit's exponentials run beside the other's dS; three
// buffers of S and dP turn, and a unit's products wait only for the dQ product three units back.  (Two buffers,
// free again as they were read: 226 us at 16 heads of 8k, D = 128, 16 picks of 64, 351 us at 8
// heads of 16k, D = 64, 8 picks of 128.  One stream of 128-key products, both warpgroups on
// the same pair: 231 and 408, exponentials and the rest took turns.)  Row t G + g of a tile is
// token t, head g, so a warp holds few tokens and skips the exponentials of units that none
// of them picked.
//
// Measured: 182 us and 312 us in these two cases, 1300 and 1000 cycles a unit of the busiest CTA
// where the products alone take 1160 and 730 (a 128 x 64 x 16 product 48, which is what reading
// its operands from shared memory takes, a commit 35).  That CTA has 8 and 10 % more units than
// the mean; with turns that all go one way 17 and 15 %, and both passes took 10 us more.
//
// kLow: dS enters its product as the sum of two bf16 values instead of one, whose rounding of
// up to 2^-8 is otherwise the larger part of the result's error; see sparse_low_part.
template <int D, bool kLow>
__global__ void __launch_bounds__(384, 1)
    dash_sparse_dq_kernel(const __grid_constant__ CUtensorMap tmQ,
                          const __grid_constant__ CUtensorMap tmDO,
                          const __grid_constant__ CUtensorMap tmK,
                          const __grid_constant__ CUtensorMap tmV,
                          const __grid_constant__ SparseDqParams p) {
  using namespace dev;
  using C = SparseDqCfg<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t sb = smem_u32(smem_raw);
  if (sb & 1023u) {
    if (threadIdx.x == 0) atomicOr(p.err, ERR_MISALIGNED);
    return;
  }
  auto sQ = [&](int k) { return sb + C::OFF_Q + (uint32_t)((k % C::kQ) * 2 * C::kTile); };
  auto sDO = [&](int k) { return sQ(k) + C::kTile; };
  auto sK = [&](int j) { return sb + C::OFF_K + (uint32_t)((j % C::kK) * C::kKV); };
  auto sV = [&](int j) { return sb + C::OFF_V + (uint32_t)((j % C::kV) * C::kKV); };
  const uint32_t bar0 = sb + C::OFF_BAR;
  // per stage of K or V (j: number of the unit)
  auto K_FULL = [&](int j) { return bar0 + 8u * (uint32_t)(j % C::kK); };
  auto K_EMPTY = [&](int j) { return bar0 + 8u * (uint32_t)(C::kK + j % C::kK); };
  auto V_FULL = [&](int j) { return bar0 + 8u * (uint32_t)(2 * C::kK + j % C::kV); };
  auto V_EMPTY = [&](int j) { return bar0 + 8u * (uint32_t)(2 * C::kK + C::kV + j % C::kV); };
  const uint32_t bar1 = bar0 + 16u * (C::kK + C::kV);
  // per tile parity (k: number of the tile)
  auto Q_FULL = [&](int k) { return bar1 + 8u * (uint32_t)(k & 1); };
  auto Q_EMPTY = [&](int k) { return bar1 + 16u + 8u * (uint32_t)(k & 1); };
  auto DONE = [&](int k) { return bar1 + 32u + 8u * (uint32_t)(k & 1); };
  auto ACC_FREE = [&](int k) { return bar1 + 48u + 8u * (uint32_t)(k & 1); };
  // S and dP have three buffers and six barriers each, so that a barrier belongs to one
  // softmax warpgroup (units j mod 2), which sees all its phases.  With three, the phase of
  // unit j + 3 is the other warpgroup's, and j + 6, which the first waits for next, has the
  // parity of j: if S of j + 3 came late, the wait would pass on the phase of j
  const uint32_t bar2 = bar1 + 64u;
  auto S_FULL = [&](int j) { return bar2 + 8u * (uint32_t)(j % 6); };
  auto DP_FULL = [&](int j) { return bar2 + 48u + 8u * (uint32_t)(j % 6); };
  auto ph6 = [](int j) { return (uint32_t)((j / 6) & 1); };
  // per buffer: the issuer of dQ, its only reader, sees all phases
  auto DS_READY = [&](int j) { return bar2 + 96u + 8u * (uint32_t)(j % 3); };
  const uint32_t FINAL = bar2 + 120;
  auto ph3 = [](int j) { return (uint32_t)((j / 3) & 1); };
  auto ph2 = [](int k) { return (uint32_t)((k >> 1) & 1); };
  auto phK = [](int j) { return (uint32_t)((j / C::kK) & 1); };
  auto phV = [](int j) { return (uint32_t)((j / C::kV) & 1); };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem_raw + C::OFF_SLOT);
  const int warp = warp_uniform(), lane = threadIdx.x & 31;
  auto wait = [&](uint32_t bar, uint32_t phase) {
    return mbar_wait_lean(bar, phase, p.spin_ns, p.err);
  };
  // the i-th tile in the order they are taken: K/V head bh, first token t0, plan row gt
  struct Tile {
    int bh, b, hk, t0, n;
    long long gt;
  };
  const int BHk = p.tiles / p.NT;
  auto tile_at = [&](int i) {
    Tile w;
    const int y = i / BHk;
    w.bh = i - y * BHk;
    w.b = w.bh / p.Hkv, w.hk = w.bh - w.b * p.Hkv;
    w.t0 = (p.NT - 1 - y) * p.T;
    w.gt = (long long)w.bh * p.NT + (p.NT - 1 - y);
    w.n = p.plan.count[w.gt];
    return w;
  };

  if (threadIdx.x == 0) {
    for (int s = 0; s < 2 * (C::kK + C::kV); ++s) mbar_init(bar0 + 8u * s, 1);
    for (int k = 0; k < 2; ++k) {
      mbar_init(Q_FULL(k), 1);
      mbar_init(Q_EMPTY(k), 2);
      mbar_init(DONE(k), 1);
      mbar_init(ACC_FREE(k), 8);
    }
    for (int j = 0; j < 6; ++j) {
      mbar_init(S_FULL(j), 1);
      mbar_init(DP_FULL(j), 1);
    }
    for (int j = 0; j < 3; ++j) mbar_init(DS_READY(j), 4);
    mbar_init(FINAL, 3);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // Tiles without a unit take no part in the numbering k of tiles and j of units.
  if (warp == 0 && lane == 0) {
    // ---------------------------------------------------------------- TMA producer
    int m = 0;  // tiles looked at
    auto next_tile = [&](Tile& w) {
      while (snake_item(m) < p.tiles) {
        w = tile_at(snake_item(m++));
        if (w.n > 0) return true;
      }
      return false;
    };
    bool ok = true;                 // no wait has run out: else nothing more is loaded
    int nq = 0, nk = 0, nv = 0;     // loads issued
    // G x T rows of 128 bytes per column half; tokens past Sq arrive as zeros.  Rows G*T to
    // 127 are never written: each row's result stays in its own row
    auto load_q = [&](const Tile& w, int k) {
      if (k >= C::kQ) ok = ok && wait(Q_EMPTY(k - C::kQ), ph2(k - C::kQ));
      if (!ok) return;
      mbar_expect_tx(Q_FULL(k), (uint32_t)(2 * p.G * p.T * D * 2));
#pragma unroll
      for (int cb = 0; cb < D / 64; ++cb) {
        tma_load_4d(sQ(k) + cb * 16384, &tmQ, cb * 64, w.hk * p.G, w.t0, w.b, Q_FULL(k));
        tma_load_4d(sDO(k) + cb * 16384, &tmDO, cb * 64, w.hk * p.G, w.t0, w.b, Q_FULL(k));
      }
      nq = k + 1;
    };
    auto load_unit = [&](uint32_t dst, const CUtensorMap* map, int u, const Tile& w, uint32_t bar) {
      mbar_expect_tx(bar, C::kKV);
#pragma unroll
      for (int cb = 0; cb < D / 64; ++cb)
        tma_load_4d(dst + cb * 8192, map, cb * 64, u * kUnit, w.hk, w.b, bar);
    };
    int k = 0, j = 0;
    Tile w, nw;
    bool on = next_tile(w);
    if (on && C::kQ == 2) load_q(w, 0);
    while (on) {
      const int* units = p.plan.unit + w.gt * p.U;
      const bool more = next_tile(nw);
      int u = units[0];
      for (int e = 0; e < w.n; ++e, ++j) {
        const int next = e + 1 < w.n ? units[e + 1] : 0;
        ok = ok && j < p.loads;
        if (j >= C::kK) ok = ok && wait(K_EMPTY(j), phK(j - C::kK));
        if (ok) load_unit(sK(j), &tmK, u, w, K_FULL(j)), nk = j + 1;
        if (j >= C::kV) ok = ok && wait(V_EMPTY(j), phV(j - C::kV));
        if (!ok) break;
        load_unit(sV(j), &tmV, u, w, V_FULL(j));
        nv = j + 1;
        u = next;
        const bool second = e == min(w.n - 1, 1);
        if (C::kQ == 1 && second) load_q(w, k);
        if (C::kQ == 2 && more && second) load_q(nw, k + 1);
      }
      w = nw;
      on = more && ok;
      ++k;
    }
    // no load may land after the CTA has gone, not even when a wait ran out
    for (int x = max(0, nq - C::kQ); x < nq; ++x)
      mbar_wait_drain(Q_FULL(x), ph2(x), drain_ns(p.spin_ns), p.err, p.err + 1);
    for (int x = max(0, nk - C::kK); x < nk; ++x)
      mbar_wait_drain(K_FULL(x), phK(x), drain_ns(p.spin_ns), p.err, p.err + 1);
    for (int x = max(0, nv - C::kV); x < nv; ++x)
      mbar_wait_drain(V_FULL(x), phV(x), drain_ns(p.spin_ns), p.err, p.err + 1);
  } else if (warp >= 1 && warp < 4) {
    // ---------------------------------------------------------------- product issuers
    // Three of them: warps 1 and 2 S and dP of a stream, warp 3 dQ.  One thread's instructions
    // take longer than the products it issues.  The whole warp walks the loop, one lane issues
    const bool leader = elect_one();
    const uint32_t hi = sdesc_hi(1024);
    bool ok = true;  // no wait has run out: else no more products
    int k = 0, j0 = 0;
#pragma unroll 1
    for (int m = 0; snake_item(m) < p.tiles && ok; ++m) {
      const int i = snake_item(m), y = i / BHk;
      const int n = p.plan.count[(long long)(i - y * BHk) * p.NT + (p.NT - 1 - y)];
      if (n == 0) continue;
      if (warp < 3) {
        constexpr uint32_t ID_S = idesc_bf16_f32(128, kUnit, 0, 0);
        const uint32_t kQ = sdesc_lo(sQ(k), 16), kDO = sdesc_lo(sDO(k), 16);
        ok = wait(Q_FULL(k), ph2(k));
#pragma unroll 1
        for (int e = (j0 ^ (warp - 1)) & 1; e < n && ok; e += 2) {
          const int j = j0 + e;
          const uint32_t kK = sdesc_lo(sK(j), 16), kV = sdesc_lo(sV(j), 16);
          const uint32_t tS = tmem + C::TM_S + 128u * (uint32_t)(j % 3);
          // dS of unit j - 3 lay in S's columns
          ok = wait(K_FULL(j), phK(j)) && (j < 3 || wait(K_EMPTY(j - 3), phK(j - 3)));
          if (!ok) break;
          tc_fence_after();
          if (leader) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              tc_mma_ss_w(tS, kQ + (uint32_t)(((kk >> 2) * 16384 + (kk & 3) * 32) >> 4),
                          kK + (uint32_t)(((kk >> 2) * 8192 + (kk & 3) * 32) >> 4), hi, ID_S,
                          kk > 0 ? 1u : 0u);
            tc_commit(S_FULL(j));
          }
          ok = wait(V_FULL(j), phV(j));
          if (!ok) break;
          tc_fence_after();
          if (leader) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              tc_mma_ss_w(tS + 64, kDO + (uint32_t)(((kk >> 2) * 16384 + (kk & 3) * 32) >> 4),
                          kV + (uint32_t)(((kk >> 2) * 8192 + (kk & 3) * 32) >> 4), hi, ID_S,
                          kk > 0 ? 1u : 0u);
            tc_commit(DP_FULL(j));
            tc_commit(V_EMPTY(j));
          }
        }
        if (leader && ok) tc_commit(Q_EMPTY(k));
      } else {
        constexpr uint32_t ID_Q = idesc_bf16_f32(128, D, 0, 1);  // K MN-major
        const uint32_t tDQ = tmem + C::TM_DQ + (uint32_t)(D * (k % C::kAcc));
        // the accumulator's last tile must have been read
        if (k >= C::kAcc) ok = wait(ACC_FREE(k - C::kAcc), ph2(k - C::kAcc));
#pragma unroll 1
        for (int e = 0; e < n && ok; ++e) {
          const int j = j0 + e;
          const uint32_t mK = sdesc_lo(sK(j), 8192);
          const uint32_t tDS = tmem + C::TM_S + 128u * (uint32_t)(j % 3);
          // K is there whenever dS is, but a softmax that gave up a wait reports dS all the same,
          // and a stage freed before its load has landed would have its barrier armed twice
          ok = wait(K_FULL(j), phK(j)) && wait(DS_READY(j), ph3(j));
          if (!ok) break;
          tc_fence_after();
          if (leader) {
#pragma unroll
            for (int kk = 0; kk < (kLow ? 2 : 1) * kUnit / 16; ++kk)  // high, then low parts
              tc_mma_ts_w(tDQ, tDS + 8 * kk, mK + (kk % 4) * 128, hi, ID_Q, (uint32_t)(e + kk));
            tc_commit(K_EMPTY(j));
            if (e + 1 == n) tc_commit(DONE(k));
          }
        }
      }
      j0 += n;
      ++k;
    }
    if (leader) tc_commit(FINAL);  // the CTA does not go before its products
    mbar_wait_drain(FINAL, 0, drain_ns(p.spin_ns), p.err, p.err + 1);
  } else if (warp >= 4) {
    // ---------------------------------------------------------------- softmax gradient
    const int h = (warp - 4) >> 2, quarter = warp & 3;  // warpgroup h takes units j = h mod 2
    const int r = quarter * 32 + lane;
    const int t = r / p.G, g = r - t * p.G;
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const float sl2 = p.scale_log2;
    const int bit = t & 31, wsel = min(t >> 5, p.W - 1);
    int j0 = 0, k = 0;
    for (int m = 0; snake_item(m) < p.tiles; ++m) {
      const Tile w = tile_at(snake_item(m));
      const int token = w.t0 + t;
      const bool valid = t < p.T && token < p.Sq;
      __nv_bfloat16* out =
          p.dq + (((long long)w.bh * p.G + g) * p.Sq + token) * D + h * (D / 2);
      if (w.n == 0) {
        if (valid)
#pragma unroll
          for (int x = 0; x < D / 16; ++x)
            reinterpret_cast<uint4*>(out)[x] = make_uint4(0, 0, 0, 0);
        continue;
      }
      const int kvlen = p.plan.len[w.b];
      const long long pos = (long long)p.plan.start[w.b] + token;
      const int limit = !valid ? 0
                        : p.causal ? (int)min((long long)kvlen, max(pos + 1, 0ll)) : kvlen;
      const int* units = p.plan.unit + w.gt * p.U;
      const uint32_t* masks = p.plan.mask + w.gt * p.U * p.W + wsel;
      int e = (j0 ^ h) & 1;  // this stream's first unit of the tile
      int u = 0;
      uint32_t word = 0u;
      if (e < w.n) u = units[e], word = masks[(long long)e * p.W];
      const long long row = ((long long)w.bh * p.G + g) * p.Sq + token;
      const float lse2 = valid ? p.lse[row] * 1.4426950408889634f : 0.f;
      const float delta = valid ? p.delta[row] : 0.f;
      for (; e < w.n; e += 2) {
        const int j = j0 + e;
        const int base = u * kUnit;
        const int v = ((word >> bit) & 1u) ? limit - base : 0;  // keys below it count
        const bool partial = base + kUnit > kvlen && kvlen < p.Sk;
        if (e + 2 < w.n) {
          u = units[e + 2];
          word = masks[(long long)(e + 2) * p.W];
        }
        const bool any = __any_sync(0xffffffffu, v > 0);
        const bool clean = __all_sync(0xffffffffu, v >= kUnit || v <= 0);
        const uint32_t keep = v > 0 ? 0xffffffffu : 0u;
        const uint32_t tS = tmem + lane_off + C::TM_S + 128u * (uint32_t)(j % 3), tDP = tS + 64;
        float pr[kUnit];
        wait(S_FULL(j), ph6(j));
        tc_fence_after();
        if (any) {
          uint32_t sv[2][32];
          tmem_ld32x2(tS, tS + 32, sv[0], sv[1]);
#pragma unroll
          for (int x = 0; x < kUnit; x += 2) {
            fma_f32x2(pr[x], pr[x + 1], __uint_as_float(sv[x >> 5][x & 31]),
                      __uint_as_float(sv[x >> 5][(x & 31) + 1]), sl2, -lse2);
            pr[x] = ex2_approx(pr[x]);
            pr[x + 1] = ex2_approx(pr[x + 1]);
          }
        }
        if (partial) {
          // K rows past the sequence hold whatever the cache holds: 0 * NaN would reach dQ
          const int first = max(kvlen - base, 0);
          for (int x = r; x < (kUnit - first) * (D / 8); x += 128) {
            const int kr = first + x / (D / 8), c = x % (D / 8);
            st_shared_v4(sK(j) + (c >> 3) * 8192 + kr * 128 + (c & 7) * 16, 0, 0, 0, 0);
          }
          fence_proxy_async_smem();
        }
        wait(DP_FULL(j), ph6(j));
        tc_fence_after();
        if (any) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t dp[32], pk[16], low[16];
            tmem_ld32(tDP + 32 * c, dp);
#pragma unroll
            for (int x = 0; x < 16; ++x) {
              float d0, d1;
              add_f32x2(d0, d1, __uint_as_float(dp[2 * x]), __uint_as_float(dp[2 * x + 1]), -delta);
              mul_f32x2(d0, d1, pr[32 * c + 2 * x], pr[32 * c + 2 * x + 1], d0, d1);
              if (!clean) {  // selected, not multiplied: S and dP of a masked key may be anything
                if (32 * c + 2 * x >= v) d0 = 0.f;
                if (32 * c + 2 * x + 1 >= v) d1 = 0.f;
              }
              const uint32_t high = pack_bf16x2(d0, d1);
              pk[x] = high & keep;
              if (kLow)
                low[x] = pack_bf16x2(d0 - __uint_as_float(high << 16),
                                     d1 - __uint_as_float(high & 0xffff0000u)) & keep;
            }
            tmem_st16(tS + 16 * c, pk);
            if (kLow) tmem_st16(tS + 32 + 16 * c, low);
          }
        } else {
          const uint32_t zero[16] = {};
#pragma unroll
          for (int c = 0; c < (kLow ? 4 : 2); ++c) tmem_st16(tS + 16 * c, zero);
        }
        tmem_wait_st();
        tc_fence_before();
        warp_arrive(DS_READY(j), lane);
      }
      wait(DONE(k), ph2(k));
      tc_fence_after();
      const uint32_t tDQ =
          tmem + lane_off + C::TM_DQ + (uint32_t)(D * (k % C::kAcc) + h * (D / 2));
      uint32_t ov[D / 64][32];
      if constexpr (D == 128) tmem_ld32x2(tDQ, tDQ + 32, ov[0], ov[1]);
      else tmem_ld32(tDQ, ov[0]);
      tc_fence_before();
      warp_arrive(ACC_FREE(k), lane);
      if (valid) {
        auto val = [&](int x) { return __uint_as_float(ov[x >> 5][x & 31]) * p.scale; };
#pragma unroll
        for (int q = 0; q < D / 16; ++q)
          reinterpret_cast<uint4*>(out)[q] =
              make_uint4(pack_bf16x2(val(8 * q), val(8 * q + 1)),
                         pack_bf16x2(val(8 * q + 2), val(8 * q + 3)),
                         pack_bf16x2(val(8 * q + 4), val(8 * q + 5)),
                         pack_bf16x2(val(8 * q + 6), val(8 * q + 7)));
      }
      j0 += w.n;
      ++k;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// ------------------------------------------------------------------ who reads a unit
// For every unit the tokens that picked it and see it, ascending: counted, given a place by
// prefix sums, written.  8 and 9 us for 35 thousand (tile, unit) pairs.
struct InverseParams {
  PlanView plan;
  int* count;  // [units] tokens of the unit
  int* off;    // [units] its first place in `token`
  int* token;
  int nu, NW, NT, T, U, W;
  long long units;  // B*Hkv*nu
};
// The tokens of query tile t that picked unit u, as a mask.
__device__ __forceinline__ void unit_tokens(const InverseParams& p, long long bh, int u, int t,
                                            uint32_t (&m)[4]) {
#pragma unroll
  for (int x = 0; x < 4; ++x) m[x] = 0u;  // T <= 128 tokens
  if (t >= p.NT) return;
  const long long at = (bh * p.NT + t) * p.NW + (u >> 5);
  const uint32_t w = p.plan.pres[at];
  if (!((w >> (u & 31)) & 1u)) return;
  const int place = p.plan.pre[at] + __popc(w & ((1u << (u & 31)) - 1u));
  const uint32_t* mask = p.plan.mask + ((bh * p.NT + t) * p.U + place) * p.W;
#pragma unroll
  for (int x = 0; x < 4; ++x)
    if (x < p.W) m[x] = mask[x];
}
// A warp per unit, a lane per query tile.
__global__ void __launch_bounds__(128)
    dash_sparse_count_kernel(const __grid_constant__ InverseParams p) {
  const long long gu = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (gu >= p.units) return;
  const int lane = threadIdx.x & 31;
  int n = 0;
  for (int t0 = 0; t0 < p.NT; t0 += 32) {
    uint32_t m[4];
    unit_tokens(p, gu / p.nu, (int)(gu % p.nu), t0 + lane, m);
    n += __popc(m[0]) + __popc(m[1]) + __popc(m[2]) + __popc(m[3]);
  }
  n = __reduce_add_sync(0xffffffffu, n);
  if (lane == 0) p.count[gu] = n;
}
// A CTA per unit, 128 tiles at a time: a thread looks its tile up, a warp writes the tokens of
// its 32 tiles one mask word after the other, a lane per token.
__global__ void __launch_bounds__(128)
    dash_sparse_fill_kernel(const __grid_constant__ InverseParams p) {
  __shared__ int warp_n[4];
  const long long gu = blockIdx.x;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int left = p.count[gu];
  int* out = p.token + p.off[gu];
  for (int t0 = 0; left > 0 && t0 < p.NT; t0 += 128) {
    uint32_t m[4];
    unit_tokens(p, gu / p.nu, (int)(gu % p.nu), t0 + tid, m);
    const int mine = __popc(m[0]) + __popc(m[1]) + __popc(m[2]) + __popc(m[3]);
    const int all = __reduce_add_sync(0xffffffffu, mine);
    __syncthreads();
    if (lane == 0) warp_n[warp] = all;
    __syncthreads();
    int at = 0;
    for (int w = 0; w < warp; ++w) at += warp_n[w];
    for (unsigned on = __ballot_sync(0xffffffffu, mine > 0); on; on &= on - 1) {
      const int src = __ffs(on) - 1, token0 = (t0 + warp * 32 + src) * p.T;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        if (x >= p.W) break;
        const uint32_t word = __shfl_sync(0xffffffffu, m[x], src);
        if ((word >> lane) & 1u) out[at + __popc(word & ((1u << lane) - 1u))] = token0 + 32 * x + lane;
        at += __popc(word);
      }
    }
    const int round = warp_n[0] + warp_n[1] + warp_n[2] + warp_n[3];
    out += round;
    left -= round;
  }
}

// Items of the dK/dV pass: every picked unit, its tokens in tiles of T, cut into stretches of
// at most C tiles with C = max(4, total / kStretches), the longest first (see snake_item).
// Fewer and longer stretches would balance less well, more write more partials.
constexpr int kStretches = 148 * 4;
constexpr int kMinStretch = 4;

struct SparseItem {
  int unit, first, end, slot;   // unit, tiles, partial slot or -1
  int off, tokens, bh, b;       // the unit's token list, its K/V head and batch entry
};
struct ItemParams {
  const int* count;  // [units]
  int* off;          // [units]
  SparseItem* item;
  int* slot0;        // [units] first partial slot of a cut unit, -1 uncut, -2 never picked
  int* head;         // [0] items, [1] C
  int T, nu, Hkv;
  long long units;
};
// One CTA: sums, a histogram of the stretches' lengths, then exclusive prefix sums of the
// tokens and partial slots per unit.  8 us for 512 units, 15 for 2048.
__global__ void __launch_bounds__(1024) dash_sparse_items_kernel(const ItemParams p) {
  constexpr int kHeld = 8192, kBuckets = 64;
  __shared__ int held[kHeld];  // the first units' counts
  __shared__ long long sum[32];
  __shared__ int pre[2][32];
  __shared__ int bucket[kBuckets];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  auto count = [&](long long x) { return x < kHeld ? held[x] : p.count[x]; };
  long long s = 0;
  for (long long x = tid; x < p.units; x += 1024) {
    const int n = p.count[x];
    if (x < kHeld) held[x] = n;
    s += (n + p.T - 1) / p.T;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0) sum[warp] = s;
  if (tid < kBuckets) bucket[tid] = 0;
  __syncthreads();
  long long total = sum[lane];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  const int C = (int)max((long long)kMinStretch, (total + kStretches - 1) / kStretches);
  // bucket 0 holds whole stretches, bucket 63 the shortest rests
  auto rest_bucket = [&](int rest) {
    return kBuckets - 1 - (int)((float)rest / (float)C * (kBuckets - 1));
  };
  for (long long x = tid; x < p.units; x += 1024) {
    const int n = (count(x) + p.T - 1) / p.T;
    if (n / C > 0) atomicAdd(&bucket[0], n / C);
    if (n % C > 0) atomicAdd(&bucket[rest_bucket(n % C)], 1);
  }
  __syncthreads();
  if (tid == 0) {
    int at = 0;
    for (int k = 0; k < kBuckets; ++k) {
      const int n = bucket[k];
      bucket[k] = at;
      at += n;
    }
    p.head[0] = at;
    p.head[1] = C;
  }
  __syncthreads();
  int base[2] = {0, 0};  // slots, tokens
  for (long long x0 = 0; x0 < p.units; x0 += 1024) {
    const long long x = x0 + tid;
    const int tokens = x < p.units ? count(x) : 0;
    const int n = (tokens + p.T - 1) / p.T;
    const int full = n / C, rest = n % C > 0, cut = full + rest > 1 ? full + rest : 0;
    const int own[2] = {cut, tokens};
    int inc[2] = {cut, tokens};  // inclusive prefix sums over the warp
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int y = __shfl_up_sync(0xffffffffu, inc[k], o);
        if (lane >= o) inc[k] += y;
      }
    if (lane == 31)
#pragma unroll
      for (int k = 0; k < 2; ++k) pre[k][warp] = inc[k];
    __syncthreads();
    int at[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int y = pre[k][lane];
      at[k] = base[k] + __reduce_add_sync(0xffffffffu, lane < warp ? y : 0) + inc[k] - own[k];
      base[k] += __reduce_add_sync(0xffffffffu, y);
    }
    if (x < p.units) {
      p.off[x] = at[1];
      p.slot0[x] = n == 0 ? -2 : cut ? at[0] : -1;
      SparseItem w;
      w.unit = (int)x;
      w.off = at[1], w.tokens = tokens;
      w.bh = (int)x / p.nu;
      w.b = w.bh / p.Hkv;
      // places within a bucket go by whoever asks first: they decide only who computes an item
      int place = full > 0 ? atomicAdd(&bucket[0], full) : 0;
      for (int k = 0; k < full + rest; ++k) {
        if (k == full) place = atomicAdd(&bucket[rest_bucket(n % C)], 1);
        w.first = k * C, w.end = min(n, (k + 1) * C);
        w.slot = cut ? at[0] + k : -1;
        p.item[place++] = w;
      }
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------------ dK, dV
struct SparseDkvParams {
  PlanView plan;
  const int* token;
  const SparseItem* item;
  const int* head;
  const __nv_bfloat16 *q, *dout;
  long long qb, qh, qs, ob, oh, os;  // strides of q and dout in elements
  const float* lse;
  const float* delta;
  __nv_bfloat16 *dk, *dv;  // [B,Hkv,Sk,D]
  float* part;             // [slots][2][64][D] (dK, dV)
  unsigned* err;
  int Hkv, Sq, Sk, G, T, nu, causal;
  int loads;  // items whose K and V are loaded (all, but for a planted fault)
  float scale, scale_log2;
  unsigned long long spin_ns;
};

template <int D>
struct SparseDkvCfg {
  static constexpr int kThreads = 640;  // Q rows, dO rows (4 warps each), S and dP, K/V, dV and dK, -, 8 softmax
  static constexpr int kTile = kTileRows * D * 2;
  static constexpr int kKV = kUnit * D * 2;
  static constexpr int kP = kTileRows * kUnit * 2;  // [128][64] bf16
  static constexpr int kStages = D == 128 ? 2 : 3;
  // D = 64 has room for P and dS of two tiles: the warpgroups take tiles in turn
  static constexpr bool kTurns = D == 64;
  static constexpr int OFF_QDO = 0;  // per stage dO, then Q: at D = 64 one [dO | Q] operand
  static constexpr int OFF_KV = kStages * 2 * kTile;  // two of K, then V
  static constexpr int OFF_P = OFF_KV + 4 * kKV;      // P, then dS, then (D = 64) its low part
  static constexpr int kPDS = (D == 64 ? 3 : 2) * kP;
  static constexpr int OFF_BAR = OFF_P + (kTurns ? 2 : 1) * kPDS;
  static constexpr int kBars = 4 * kStages + 12 + 9;
  static constexpr int OFF_SLOT = OFF_BAR + kBars * 8;
  static constexpr int kSmemBytes = OFF_SLOT + 16;
  static_assert(kSmemBytes <= 232448, "shared memory per block exceeded");
  static_assert(kSmemBytes > 116 * 1024, "one CTA per SM: its 512 TMEM columns are free");
  static constexpr uint32_t TM_S = 0, TM_ACC = 256, kTmemCols = 512;
};

// The rows that attend to a unit are gathered: a tile is T tokens of the unit's list with all
// G heads, row t G + g, so that no product is spent on tokens that did not pick the unit (a
// tile of neighbouring tokens would be 2 to 5 times too large at 16 picks of 8k keys).  16-byte
// cp.async writes the rows in the swizzled layout the products read.
//
// Per tile: S = Q K^T and dP = dO V^T as 128 x 64, P and dS in bf16 to shared memory, then
// dV^T += dO^T P and dK^T += Q^T dS with the head dimension as the 128 MMA rows (a 64-key M
// would halve the rate).  At D = 64 the stacked operand [dO | Q] serves both: dV^T is the
// upper half of one product, dK^T the lower of the other.  S and dP of the next tile, K and V
// and the accumulators of the next item have buffers of their own, so that the products of
// one tile run under the exponentials of the other, also from item to item.  D = 128: the two
// softmax warpgroups take 32 keys of every row each, and the dV product is issued before dS
// is computed.  D = 64: they take tiles in turn.  kLow (D = 64, where shared memory has room):
// as in the dQ kernel.
//
// Measured: 16 heads of 8k, 4 K/V heads, D = 128, 16 picks of 64: 177 us, 3100 cycles a tile;
// 8 heads of 16k, D = 64, 8 picks of 128: 142 us, 2500.  The products take 2000 and 1280.  At
// D = 128 two stages are all that fits, and a stage's way from load to last product bounds it.
// Tiles of neighbouring tokens: 544 and 1159 us; dV and dK issued together: 201 and 170.
template <int D, bool kLow>
__global__ void __launch_bounds__(640, 1)
    dash_sparse_dkdv_kernel(const __grid_constant__ CUtensorMap tmK,
                            const __grid_constant__ CUtensorMap tmV,
                            const __grid_constant__ SparseDkvParams p) {
  using namespace dev;
  using C = SparseDkvCfg<D>;
  constexpr int ST = C::kStages;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t sb = smem_u32(smem_raw);
  if (sb & 1023u) {
    if (threadIdx.x == 0) atomicOr(p.err, ERR_MISALIGNED);
    return;
  }
  auto sDO = [&](int s) { return sb + C::OFF_QDO + (uint32_t)(s * 2 * C::kTile); };
  auto sQ = [&](int s) { return sDO(s) + C::kTile; };
  auto sK = [&](int k) { return sb + C::OFF_KV + (uint32_t)((k & 1) * 2 * C::kKV); };
  auto sV = [&](int k) { return sK(k) + C::kKV; };
  auto sP = [&](int j) { return sb + C::OFF_P + (C::kTurns ? (uint32_t)((j & 1) * C::kPDS) : 0u); };
  const uint32_t bar0 = sb + C::OFF_BAR;
  // per stage (Q, dO), per item parity, per tile parity
  auto FULL = [&](int x, int s) { return bar0 + 8u * (uint32_t)(x * ST + s); };
  auto EMPTY = [&](int x, int s) { return bar0 + 8u * (uint32_t)((2 + x) * ST + s); };
  const uint32_t bar1 = bar0 + 32u * ST;
  auto KV_FULL = [&](int k) { return bar1 + 8u * (uint32_t)(k & 1); };
  auto ITEM_DONE = [&](int k) { return bar1 + 16u + 8u * (uint32_t)(k & 1); };
  auto ACC_FREE = [&](int k) { return bar1 + 32u + 8u * (uint32_t)(k & 1); };
  // per tile parity
  auto S_FULL = [&](int j) { return bar1 + 48u + 8u * (uint32_t)(j & 1); };
  auto DP_FULL = [&](int j) { return bar1 + 64u + 8u * (uint32_t)(j & 1); };
  auto SDP_READ = [&](int j) { return bar1 + 80u + 8u * (uint32_t)(j & 1); };
  auto P_READY = [&](int j) { return bar1 + 96u + 8u * (uint32_t)(j & 1); };
  auto P_FREE = [&](int j) { return bar1 + 112u + 8u * (uint32_t)(j & 1); };
  auto DS_READY = [&](int j) { return bar1 + 128u + 8u * (uint32_t)(j & 1); };
  auto DS_FREE = [&](int j) { return bar1 + 144u + 8u * (uint32_t)(j & 1); };
  const uint32_t FINAL = bar1 + 160;
  auto ph2 = [](int k) { return (uint32_t)((k >> 1) & 1); };
  auto phS = [](int j) { return (uint32_t)((j / ST) & 1); };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem_raw + C::OFF_SLOT);
  const int warp = warp_uniform(), lane = threadIdx.x & 31;
  auto wait = [&](uint32_t bar, uint32_t phase) {
    return mbar_wait_lean(bar, phase, p.spin_ns, p.err);
  };
  const int items = p.head[0];
  const uint32_t inv_g = (65536u + p.G - 1) / p.G;  // row / G = row * inv_g >> 16 for row < 128
  const int rows = p.G * p.T;

  if (threadIdx.x == 0) {
    for (int s = 0; s < ST; ++s)
      for (int x = 0; x < 2; ++x) {
        mbar_init(FULL(x, s), 4);
        mbar_init(EMPTY(x, s), 1);
      }
    for (int k = 0; k < 2; ++k) {
      mbar_init(KV_FULL(k), 1);
      mbar_init(ITEM_DONE(k), 1);
      mbar_init(ACC_FREE(k), 8);
      mbar_init(S_FULL(k), 1);
      mbar_init(DP_FULL(k), 1);
      mbar_init(SDP_READ(k), C::kTurns ? 4 : 8);
      mbar_init(P_READY(k), 8);  // D = 128 alone: with kTurns P comes and goes with dS
      mbar_init(P_FREE(k), 1);
      mbar_init(DS_READY(k), C::kTurns ? 4 : 8);
      mbar_init(DS_FREE(k), 1);
    }
    mbar_init(FINAL, 2);
    fence_mbar_init();
  }
  // rows G*T to 127 of a stage are never loaded, but the products sum over all 128 rows
  for (int x = threadIdx.x; x < (kTileRows - rows) * 8 * (2 * ST * D / 64); x += C::kThreads) {
    const int c = x & 7, rest = x >> 3, atom = rest % (2 * ST * D / 64);
    const int row = rows + rest / (2 * ST * D / 64);
    st_shared_v4(sb + C::OFF_QDO + atom * 16384 + row * 128 + c * 16, 0, 0, 0, 0);
  }
  fence_proxy_async_smem();
  if (warp == 8) {
    tmem_alloc(smem_u32(tmem_slot), C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp < 8) {
    // ---------------------------------------------------------------- row loads
    // warps 0-3 Q, 4-7 dO; a warp fills 32 rows of each tile, D / 8 lanes a row, and takes
    // the rows' addresses from the lanes that looked them up
    const int x = warp >> 2, row_l = (warp & 3) * 32 + lane;
    constexpr int CH = D / 8, RP = 32 / CH;  // 16-byte pieces of a row, rows at a time
    const int c = lane % CH, sub = lane / CH;
    const int t = (int)((uint32_t)row_l * inv_g >> 16), g = row_l - t * p.G;
    const long long sB = x ? p.ob : p.qb, sH = x ? p.oh : p.qh, sS_ = x ? p.os : p.qs;
    const __nv_bfloat16* src = (x ? p.dout : p.q) + g * sH;
    const uint32_t col = (uint32_t)((c >> 3) * 16384);
    const int rows_w = min(32, rows - (warp & 3) * 32);  // rows of this warp that are loaded
    int it = 0;
    SparseItem w;
    int token = 0;  // of this lane's row in the next tile
    auto look = [&](const SparseItem& w, int e) {
      const int at = e * p.T + t;
      return t < p.T && at < w.tokens ? p.token[w.off + at] : -1;
    };
    if (snake_item(0) < items) {
      w = p.item[snake_item(0)];
      token = look(w, w.first);
    }
    for (int k = 0; snake_item(k) < items; ++k) {
      const bool more = snake_item(k + 1) < items;
      SparseItem nw = w;
      if (more) nw = p.item[snake_item(k + 1)];
      const int b = w.b, hk = w.bh - b * p.Hkv;
      const __nv_bfloat16* head = src + b * sB + (long long)hk * p.G * sH;
      for (int e = w.first; e < w.end; ++e, ++it) {
        const int s = it % ST;
        const unsigned on = __ballot_sync(0xffffffffu, token >= 0);
        const unsigned long long mine =
            reinterpret_cast<unsigned long long>(head + (long long)max(token, 0) * sS_);
        token = e + 1 < w.end ? look(w, e + 1) : more ? look(nw, nw.first) : 0;
        if (it >= ST) wait(EMPTY(x, s), phS(it - ST));
        const uint32_t dst = (x ? sDO(s) : sQ(s)) + col;
#pragma unroll 8
        for (int y = sub; y < 32; y += RP) {
          const unsigned long long row = __shfl_sync(0xffffffffu, mine, y);
          const int r = (warp & 3) * 32 + y;
          if (y < rows_w)  // rows past the list arrive as zeros
            cp_async16(dst + (uint32_t)(r * 128 + ((c ^ r) & 7) * 16),
                       reinterpret_cast<const void*>(row + c * 16), (on >> y) & 1u ? 16u : 0u);
        }
        cp_async_wait_all();
        fence_proxy_async_smem();
        warp_arrive(FULL(x, s), lane);
      }
      w = nw;
    }
  } else if (warp < 12) {
    if (warp == 9 && lane == 0) {
      // ---------------------------------------------------------------- K and V
      int k = 0;
      for (; snake_item(k) < items; ++k) {
        const SparseItem w = p.item[snake_item(k)];
        const int u = w.unit - w.bh * p.nu, hk = w.bh - w.b * p.Hkv;
        // K and V of item k - 2 are read to the end; nothing is loaded once a wait has run out
        if (k >= p.loads || (k >= 2 && !wait(ITEM_DONE(k), ph2(k - 2)))) break;
        mbar_expect_tx(KV_FULL(k), 2 * C::kKV);
#pragma unroll
        for (int cb = 0; cb < D / 64; ++cb) {
          tma_load_4d(sK(k) + cb * 8192, &tmK, cb * 64, u * kUnit, hk, w.b, KV_FULL(k));
          tma_load_4d(sV(k) + cb * 8192, &tmV, cb * 64, u * kUnit, hk, w.b, KV_FULL(k));
        }
      }
      // no load may land after the CTA has gone, not even when a wait ran out
      for (int j = max(0, k - 2); j < k; ++j)
        mbar_wait_drain(KV_FULL(j), ph2(j), drain_ns(p.spin_ns), p.err, p.err + 1);
    } else if (warp == 8 || warp == 10) {
      // ---------------------------------------------------------------- product issuers
      // Two of them, S and dP and beside them dV and dK (see the dQ kernel)
      const bool leader = elect_one();
      const uint32_t hi = sdesc_hi(1024);
      bool ok = true;  // no wait has run out: else no more products
      int j = 0, k = 0, s = 0;
      uint32_t sph = 0;
#pragma unroll 1
      for (; snake_item(k) < items && ok; ++k) {
        const int first = p.item[snake_item(k)].first, end = p.item[snake_item(k)].end;
        if (warp == 8) {
          constexpr uint32_t ID_S = idesc_bf16_f32(128, kUnit, 0, 0);
          const uint32_t kK = sdesc_lo(sK(k), 16), kV = sdesc_lo(sV(k), 16);
          ok = wait(KV_FULL(k), ph2(k));
#pragma unroll 1
          for (int e = first; e < end && ok; ++e, ++j) {
            const uint32_t kQ = sdesc_lo(sQ(s), 16), kDO = sdesc_lo(sDO(s), 16);
            const uint32_t tS = tmem + C::TM_S + 128u * (uint32_t)(j & 1);
            ok = wait(FULL(0, s), sph) && (j < 2 || wait(SDP_READ(j), ph2(j - 2)));
            if (!ok) break;
            tc_fence_after();
            if (leader) {
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk)
                tc_mma_ss_w(tS, kQ + (uint32_t)(((kk >> 2) * 16384 + (kk & 3) * 32) >> 4),
                            kK + (uint32_t)(((kk >> 2) * 8192 + (kk & 3) * 32) >> 4), hi, ID_S,
                            kk > 0 ? 1u : 0u);
              tc_commit(S_FULL(j));
            }
            ok = wait(FULL(1, s), sph);
            if (!ok) break;
            tc_fence_after();
            if (leader) {
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk)
                tc_mma_ss_w(tS + 64, kDO + (uint32_t)(((kk >> 2) * 16384 + (kk & 3) * 32) >> 4),
                            kV + (uint32_t)(((kk >> 2) * 8192 + (kk & 3) * 32) >> 4), hi, ID_S,
                            kk > 0 ? 1u : 0u);
              tc_commit(DP_FULL(j));
            }
            if (++s == ST) s = 0, sph ^= 1u;
          }
        } else {
          constexpr uint32_t ID_T = idesc_bf16_f32(128, kUnit, 1, 1);  // dV^T, dK^T
          const uint32_t tA = tmem + C::TM_ACC + 128u * (uint32_t)(k & 1);
          // the accumulators of item k - 2 must have been read
          if (k >= 2) ok = wait(ACC_FREE(k), ph2(k - 2));
          // it frees K and V: not before they have landed, even where softmax warps that gave up
          // a wait report P and dS
          ok = ok && wait(KV_FULL(k), ph2(k));
#pragma unroll 1
          for (int e = first; e < end && ok; ++e, ++j) {
            const uint32_t aV = sdesc_lo(sDO(s), 16384);
            const uint32_t aK = D == 128 ? sdesc_lo(sQ(s), 16384) : aV;
            const uint32_t bP = sdesc_lo(sP(j), 16384), bS = sdesc_lo(sP(j) + C::kP, 16384);
            const uint32_t bL = sdesc_lo(sP(j) + 2 * C::kP, 16384);
            // D = 128: P is there before dP, and with it before dO need be.  The dP product has
            // waited for dO and, once done, read it: only then may dV read the stage and its
            // commit free it.  (dP of j + 2 needs that commit, so the phase cannot run ahead.)
            static_assert(C::kTurns || ST == 2, "a stage of dO per parity of the tile");
            ok = C::kTurns ? wait(DS_READY(j), ph2(j))
                           : wait(DP_FULL(j), ph2(j)) && wait(P_READY(j), ph2(j));
            if (!ok) break;
            tc_fence_after();
            if (leader) {
#pragma unroll
              for (int kk = 0; kk < 8; ++kk)
                tc_mma_ss_w(tA, aV + kk * 128, bP + kk * 128, hi, ID_T, (uint32_t)(e - first + kk));
              if (!C::kTurns) {
                tc_commit(P_FREE(j));
                tc_commit(EMPTY(1, s));
              }
            }
            ok = C::kTurns || wait(DS_READY(j), ph2(j));
            if (!ok) break;
            tc_fence_after();
            if (leader) {
#pragma unroll
              for (int kk = 0; kk < 8; ++kk)
                tc_mma_ss_w(tA + 64, aK + kk * 128, bS + kk * 128, hi, ID_T,
                            (uint32_t)(e - first + kk));
              if (kLow)
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)
                  tc_mma_ss_w(tA + 64, aK + kk * 128, bL + kk * 128, hi, ID_T, 1u);
              if (C::kTurns) tc_commit(EMPTY(1, s));
              tc_commit(EMPTY(0, s));
              tc_commit(DS_FREE(j));
              if (e + 1 == end) tc_commit(ITEM_DONE(k));
            }
            if (++s == ST) s = 0;
          }
        }
      }
      if (leader) tc_commit(FINAL);  // the CTA does not go before its products
      mbar_wait_drain(FINAL, 0, drain_ns(p.spin_ns), p.err, p.err + 1);
    }
  } else {
    // ---------------------------------------------------------------- softmax gradient
    const int wg = (warp - 12) >> 2, quarter = warp & 3;
    const int r = quarter * 32 + lane;
    const int t = (int)((uint32_t)r * inv_g >> 16), g = r - t * p.G;
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const float sl2 = p.scale_log2;
    // what this thread's row of a tile needs, fetched one tile ahead
    float lse2 = 0.f, delta = 0.f;
    int vis = 0;  // keys below it are attended to
    auto fetch = [&](const SparseItem& w, int e) {
      const int base = (w.unit - w.bh * p.nu) * kUnit;
      const int kvlen = p.plan.len[w.b];
      // a row without a token has Q = dO = 0: P dO and dS Q are 0 whatever P and a finite
      // dS are; keys past the sequence, which may be anything, are left out for it too
      lse2 = delta = 0.f;
      vis = kvlen - base;
      const int at = e * p.T + t;
      if (t >= p.T || at >= w.tokens) return;
      const int token = p.token[w.off + at];
      const long long row = ((long long)w.bh * p.G + g) * p.Sq + token;
      lse2 = p.lse[row] * 1.4426950408889634f;
      delta = p.delta[row];
      if (p.causal) vis = (int)min((long long)kvlen, (long long)p.plan.start[w.b] + token + 1) - base;
    };
    // the tiles e that this warpgroup takes: all, or with kTurns those of its parity
    constexpr int kStep = C::kTurns ? 2 : 1;
    int it0 = 0, k = 0;  // the item's first tile number, the item's number
    SparseItem w;
    if (snake_item(0) < items) w = p.item[snake_item(0)];
    bool have = false;  // lse2, delta and vis are those of the next tile taken
    for (; snake_item(k) < items; ++k) {
      const bool more = snake_item(k + 1) < items;
      SparseItem nw = w;
      if (more) nw = p.item[snake_item(k + 1)];
      auto first_own = [&](const SparseItem& x, int at) {
        return x.first + (C::kTurns ? ((at ^ wg) & 1) : 0);
      };
      const int it1 = it0 + w.end - w.first, own = first_own(w, it0);
      if (!have && own < w.end) fetch(w, own);
      have = false;
      for (int e = own; e < w.end; e += kStep) {
        const int it = it0 + e - w.first;
        const float l2 = lse2, dl = delta;
        const int v = C::kTurns ? vis : vis - 32 * wg;
        if (e + kStep < w.end) {
          fetch(w, e + kStep);
        } else if (more && first_own(nw, it1) < nw.end) {
          fetch(nw, first_own(nw, it1));
          have = true;
        }
        const bool whole = __all_sync(0xffffffffu, v >= (C::kTurns ? kUnit : 32));
        const uint32_t tS = tmem + lane_off + C::TM_S + 128u * (uint32_t)(it & 1) +
                            (C::kTurns ? 0u : 32u * wg);
        const uint32_t rowP = sP(it) + r * 128, rowS = rowP + C::kP, rowL = rowS + C::kP;
        // two keys of a row from S and dP: dS and P as bf16 pairs
        auto to_ds = [&](int key, float p0, float p1, uint32_t dp0, uint32_t dp1, uint32_t& ds,
                         uint32_t& low) {
          float d0, d1;
          add_f32x2(d0, d1, __uint_as_float(dp0), __uint_as_float(dp1), -dl);
          mul_f32x2(d0, d1, p0, p1, d0, d1);
          if (!whole) {  // selected, not multiplied: S and dP of a masked key may be anything
            if (key >= v) d0 = 0.f;
            if (key + 1 >= v) d1 = 0.f;
          }
          ds = pack_bf16x2(d0, d1);
          if (kLow)
            low = pack_bf16x2(d0 - __uint_as_float(ds << 16), d1 - __uint_as_float(ds & 0xffff0000u));
        };
        if constexpr (C::kTurns) {
          wait(S_FULL(it), ph2(it));
          wait(DP_FULL(it), ph2(it));
          tc_fence_after();
          if (it >= 2) wait(DS_FREE(it), ph2(it - 2));
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t sv[16], dp[16];
            tmem_ld16_async(tS + 16 * c, sv);
            tmem_ld16_async(tS + 64 + 16 * c, dp);
            tmem_wait_ld();
            if (c == 3) {
              tc_fence_before();
              warp_arrive(SDP_READ(it), lane);
            }
            uint32_t pp[8], ds[8], low[8];
#pragma unroll
            for (int x = 0; x < 8; ++x) {
              const int key = 16 * c + 2 * x;
              float p0, p1;
              fma_f32x2(p0, p1, __uint_as_float(sv[2 * x]), __uint_as_float(sv[2 * x + 1]), sl2, -l2);
              p0 = ex2_approx(p0);
              p1 = ex2_approx(p1);
              if (!whole) {
                if (key >= v) p0 = 0.f;
                if (key + 1 >= v) p1 = 0.f;
              }
              pp[x] = pack_bf16x2(p0, p1);
              to_ds(key, p0, p1, dp[2 * x], dp[2 * x + 1], ds[x], low[x]);
            }
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const uint32_t off = (uint32_t)(((2 * c + x) ^ (r & 7)) << 4);
              st_shared_v4(rowP + off, pp[4 * x], pp[4 * x + 1], pp[4 * x + 2], pp[4 * x + 3]);
              st_shared_v4(rowS + off, ds[4 * x], ds[4 * x + 1], ds[4 * x + 2], ds[4 * x + 3]);
              if (kLow)
                st_shared_v4(rowL + off, low[4 * x], low[4 * x + 1], low[4 * x + 2], low[4 * x + 3]);
            }
          }
          fence_proxy_async_smem();
          warp_arrive(DS_READY(it), lane);
          continue;
        }
        wait(S_FULL(it), ph2(it));
        tc_fence_after();
        // P, of which the dV product can be issued while dS is computed
        float pr[32];
#pragma unroll
        for (int c = 0; c < 32; c += 16) {
          uint32_t sv[16];
          tmem_ld16(tS + c, sv);
#pragma unroll
          for (int x = 0; x < 16; x += 2) {
            fma_f32x2(pr[c + x], pr[c + x + 1], __uint_as_float(sv[x]), __uint_as_float(sv[x + 1]),
                      sl2, -l2);
            pr[c + x] = ex2_approx(pr[c + x]);
            pr[c + x + 1] = ex2_approx(pr[c + x + 1]);
          }
        }
        if (!whole)  // selected, not multiplied: S and dP of a masked key may be anything
#pragma unroll
          for (int x = 0; x < 32; ++x)
            if (x >= v) pr[x] = 0.f;
        if (it > 0) wait(P_FREE(it - 1), ph2(it - 1));
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const uint32_t off = (uint32_t)(((4 * wg + x) ^ (r & 7)) << 4);
          st_shared_v4(rowP + off, pack_bf16x2(pr[8 * x], pr[8 * x + 1]),
                       pack_bf16x2(pr[8 * x + 2], pr[8 * x + 3]),
                       pack_bf16x2(pr[8 * x + 4], pr[8 * x + 5]),
                       pack_bf16x2(pr[8 * x + 6], pr[8 * x + 7]));
        }
        fence_proxy_async_smem();
        warp_arrive(P_READY(it), lane);
        wait(DP_FULL(it), ph2(it));
        tc_fence_after();
        if (it > 0) wait(DS_FREE(it - 1), ph2(it - 1));
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t dp[16];
          tmem_ld16(tS + 64 + 16 * c, dp);
          if (c == 1) {
            tc_fence_before();
            warp_arrive(SDP_READ(it), lane);
          }
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            uint32_t ds[4], low[4];
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const int z = 8 * x + 2 * y, q = 16 * c + z;
              to_ds(q, pr[q], pr[q + 1], dp[z], dp[z + 1], ds[y], low[y]);
            }
            const uint32_t off = (uint32_t)(((4 * wg + 2 * c + x) ^ (r & 7)) << 4);
            st_shared_v4(rowS + off, ds[0], ds[1], ds[2], ds[3]);
            if (kLow) st_shared_v4(rowL + off, low[0], low[1], low[2], low[3]);
          }
        }
        fence_proxy_async_smem();
        warp_arrive(DS_READY(it), lane);
      }
      // epilogue: warpgroup 0 writes dV, warpgroup 1 dK; lane = head dimension, column = key
      wait(ITEM_DONE(k), ph2(k));
      tc_fence_after();
      const uint32_t ta = tmem + lane_off + C::TM_ACC + 128u * (uint32_t)(k & 1) + 64u * wg;
      const int base = (w.unit - w.bh * p.nu) * kUnit;
      // at D = 64 dV^T is in lanes 0-63 of its product, dK^T in lanes 64-127 of its own
      const int d = D == 128 ? r : r - (wg == 0 ? 0 : 64);
      const float f = wg == 0 ? 1.f : p.scale;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t acc[32];
        tmem_ld32(ta + 32 * c, acc);
        if (c == 1) {
          tc_fence_before();
          warp_arrive(ACC_FREE(k), lane);
        }
        if (d < 0 || d >= D) continue;
        if (w.slot >= 0) {
          float* out =
              p.part + (((long long)w.slot * 2 + (wg == 0 ? 1 : 0)) * kUnit + 32 * c) * D + d;
#pragma unroll
          for (int key = 0; key < 32; ++key) out[key * D] = __uint_as_float(acc[key]) * f;
        } else {
          __nv_bfloat16* out =
              (wg == 0 ? p.dv : p.dk) + ((long long)w.bh * p.Sk + base + 32 * c) * D + d;
          const int keys = p.Sk - base - 32 * c;
#pragma unroll
          for (int key = 0; key < 32; ++key)
            if (key < keys) out[key * D] = __float2bfloat16_rn(__uint_as_float(acc[key]) * f);
        }
      }
      w = nw;
      it0 = it1;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// Units that no token picked get zeros; the partials of cut units are added in ascending
// order.  A CTA takes 1024 elements of a unit's dK and dV (blockIdx.y).
struct FinishParams {
  const int* slot0;
  const int* count;
  const int* head;
  const float* part;
  __nv_bfloat16 *dk, *dv;
  int Sk, D, nu, T;
};
__global__ void __launch_bounds__(256) dash_sparse_finish_kernel(const FinishParams p) {
  const int gu = blockIdx.x;
  const int s0 = p.slot0[gu];
  if (s0 == -1) return;
  const int bh = gu / p.nu, base = (gu - bh * p.nu) * kUnit;
  const int n = min(kUnit, p.Sk - base) * p.D;
  const int tiles = (p.count[gu] + p.T - 1) / p.T, C = p.head[1];
  const int parts = s0 < 0 ? 0 : (tiles + C - 1) / C;
  const int x = ((int)blockIdx.y * 256 + (int)threadIdx.x) * 4;
  if (x >= n) return;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f), c = a;
  const float* src = p.part + (long long)max(s0, 0) * 2 * kUnit * p.D + x;
#pragma unroll 4
  for (int k = 0; k < parts; ++k, src += 2 * kUnit * p.D) {
    const float4 y = *reinterpret_cast<const float4*>(src);
    const float4 z = *reinterpret_cast<const float4*>(src + kUnit * p.D);
    a.x += y.x, a.y += y.y, a.z += y.z, a.w += y.w;
    c.x += z.x, c.y += z.y, c.z += z.z, c.w += z.w;
  }
  const long long at = ((long long)bh * p.Sk + base) * p.D + x;
  *reinterpret_cast<uint2*>(p.dk + at) =
      make_uint2(dev::pack_bf16x2(a.x, a.y), dev::pack_bf16x2(a.z, a.w));
  *reinterpret_cast<uint2*>(p.dv + at) =
      make_uint2(dev::pack_bf16x2(c.x, c.y), dev::pack_bf16x2(c.z, c.w));
}

}  // namespace dash
