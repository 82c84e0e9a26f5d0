// Block-sparse attention forward for sm_100a.
//
// One CTA per query tile (and per part of its list, when the list is split): 128 rows = T
// tokens x G heads against the tile's listed units of 64 keys.  Per unit j:
//
//   S_j  = Q K_j^T        tcgen05.mma (smem x smem), 128 x 64, TMEM, two buffers
//   P_j  = 2^(s S_j - m)  softmax warps, thread = row = TMEM lane; rows whose token did not
//                         pick the unit, and keys at or past the row's limit, get 0
//   O   += P_j V_j        tcgen05.mma with A = P_j in TMEM
//
// with s = scale log2(e) and m the row's running maximum, moved only when it grows by more
// than kRescaleLog2 (P stays below 2^kRescaleLog2; O / l and m + log2 l do not depend on
// when it moved).  P is rounded once to bf16 for the product; l sums the fp32 values.
//
// 256 threads: TMA, issuers of S and of P V (two, so that S of the next unit does not wait for
// this one's P), four softmax warps.  256 TMEM columns and at most 113 KiB of shared memory,
// so that two CTAs share an SM: one's exponentials run under the other's products.  Row t G + g
// of a tile is token t, head g: a warp holds few tokens and skips the exponentials of units
// that none of them picked.
//
// Measured: 16 heads of 8k, 4 K/V heads, D = 128, 16 picks of 64 (a tile lists 34 units where a
// query picks 15): 134 us; 8 heads of 16k, D = 64, 8 picks of 128 (77 and 16): 224 us.  Bound by
// the softmax warps' way from S to P, some 1600 cycles a unit beside another CTA; a unit's
// products take 710 and 450 cycles.  With one issuer, and a comparison for every key: 191 and
// 335 us.  Lists cut over twice the CTAs, for 376 tiles on 296 places, did not pay for the join
// (94 us for 76).
#pragma once
#include "ptx.cuh"
#include "sparse_plan.cuh"

namespace dash {

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int x, int s,
                                            int h, int b, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(s), "r"(h), "r"(b), "r"(bar)
      : "memory");
}

struct SparseFwdParams {
  PlanView plan;
  __nv_bfloat16* o;  // [B,H,Sq,D]
  float* lse;        // [B,H,Sq]
  float* part_o;     // [splits][B*H*Sq][D] when splits > 1: O of the part, normalised
  float* part_l;     // [splits][B*H*Sq] log2-domain log-sum-exp of the part
  unsigned* err;     // [0] error word, [1] abort flag
  int H, Hkv, Sq, Sk, G, T, W, NT, U, causal, splits;
  int loads;  // units that the producer loads (all, but for a planted fault)
  float scale_log2;
  unsigned long long spin_ns;
};

template <int D>
struct SparseFwdCfg {
  static constexpr int kThreads = 256;
  static constexpr int kQ = kTileRows * D * 2;
  static constexpr int kKV = kUnit * D * 2;
  static constexpr int kK = D == 128 ? 3 : 6, kV = D == 128 ? 2 : 5;  // stages of K and of V
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = kQ;
  static constexpr int OFF_V = OFF_K + kK * kKV;
  static constexpr int OFF_BAR = OFF_V + kV * kKV;
  static constexpr int kBars = 3 + 2 * 3 + 2 * kK + 2 * kV;
  static constexpr int OFF_SLOT = OFF_BAR + kBars * 8;
  static constexpr int kSmemBytes = OFF_SLOT + 16;
  static_assert(kSmemBytes <= 115712, "two CTAs per SM");
  static constexpr uint32_t TM_S = 0, TM_O = 128, kTmemCols = 256;
  static constexpr float kRescaleLog2 = 8.0f;
};

template <int D>
__global__ void __launch_bounds__(256, 2)
    dash_sparse_fwd_kernel(const __grid_constant__ CUtensorMap tmQ,
                           const __grid_constant__ CUtensorMap tmK,
                           const __grid_constant__ CUtensorMap tmV,
                           const __grid_constant__ SparseFwdParams p) {
  using namespace dev;
  using C = SparseFwdCfg<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t sb = smem_u32(smem_raw);
  if (sb & 1023u) {
    if (threadIdx.x == 0) atomicOr(p.err, ERR_MISALIGNED);
    return;
  }
  const uint32_t sQ = sb + C::OFF_Q;
  auto sK = [&](int j) { return sb + C::OFF_K + (uint32_t)((j % C::kK) * C::kKV); };
  auto sV = [&](int j) { return sb + C::OFF_V + (uint32_t)((j % C::kV) * C::kKV); };
  const uint32_t bar0 = sb + C::OFF_BAR;
  const uint32_t Q_FULL = bar0, O_FINAL = bar0 + 8, S_FINAL = bar0 + 16;
  auto S_FULL = [&](int j) { return bar0 + 24u + 8u * (uint32_t)(j & 1); };
  auto P_READY = [&](int j) { return bar0 + 40u + 8u * (uint32_t)(j & 1); };
  auto PV_DONE = [&](int j) { return bar0 + 56u + 8u * (uint32_t)(j & 1); };
  const uint32_t bar1 = bar0 + 72u;
  auto K_FULL = [&](int j) { return bar1 + 8u * (uint32_t)(j % C::kK); };
  auto K_EMPTY = [&](int j) { return bar1 + 8u * (uint32_t)(C::kK + j % C::kK); };
  auto V_FULL = [&](int j) { return bar1 + 8u * (uint32_t)(2 * C::kK + j % C::kV); };
  auto V_EMPTY = [&](int j) { return bar1 + 8u * (uint32_t)(2 * C::kK + C::kV + j % C::kV); };
  auto ph2 = [](int j) { return (uint32_t)((j >> 1) & 1); };
  auto phK = [](int j) { return (uint32_t)((j / C::kK) & 1); };
  auto phV = [](int j) { return (uint32_t)((j / C::kV) & 1); };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem_raw + C::OFF_SLOT);
  const int warp = warp_uniform(), lane = threadIdx.x & 31;
  auto wait = [&](uint32_t bar, uint32_t phase) {
    return mbar_wait_lean(bar, phase, p.spin_ns, p.err);
  };

  // the last tiles (longest lists under a causal mask) first
  const int split = (int)(blockIdx.x % (unsigned)p.splits);
  const unsigned rest = blockIdx.x / (unsigned)p.splits;
  const int BHk = (int)(gridDim.x / (unsigned)p.splits / (unsigned)p.NT);
  const int tile = p.NT - 1 - (int)(rest / (unsigned)BHk), bh = (int)(rest % (unsigned)BHk);
  const int b = bh / p.Hkv, hk = bh % p.Hkv, t0 = tile * p.T;
  const long long gt = (long long)bh * p.NT + tile;
  const int total = p.plan.count[gt];
  const int beg = (int)((long long)total * split / p.splits);
  const int n = (int)((long long)total * (split + 1) / p.splits) - beg;
  const int* units = p.plan.unit + gt * p.U + beg;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kBars; ++i) mbar_init(bar0 + 8u * i, 1);
    for (int i = 0; i < 2; ++i) mbar_init(P_READY(i), 4);
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

  if (warp == 0 && lane == 0) {
    // ---------------------------------------------------------------- TMA producer
    int nk = 0, nv = 0;  // loads issued; nothing more once a wait has run out
    if (n > 0) {
      // T x G rows of 128 bytes per column half; tokens past Sq arrive as zeros.  Rows G*T
      // to 127 of the tile are never written: each row's result stays in its own row
      mbar_expect_tx(Q_FULL, (uint32_t)(p.G * p.T * D * 2));
#pragma unroll
      for (int cb = 0; cb < D / 64; ++cb)
        tma_load_4d(sQ + cb * 16384, &tmQ, cb * 64, hk * p.G, t0, b, Q_FULL);
    }
    int u = n > 0 ? units[0] : 0;
    for (int j = 0; j < n; ++j) {
      const int next = j + 1 < n ? units[j + 1] : 0;
      if (j >= p.loads || (j >= C::kK && !wait(K_EMPTY(j), phK(j - C::kK)))) break;
      mbar_expect_tx(K_FULL(j), C::kKV);
#pragma unroll
      for (int cb = 0; cb < D / 64; ++cb)
        tma_load_4d(sK(j) + cb * 8192, &tmK, cb * 64, u * kUnit, hk, b, K_FULL(j));
      nk = j + 1;
      if (j >= C::kV && !wait(V_EMPTY(j), phV(j - C::kV))) break;
      mbar_expect_tx(V_FULL(j), C::kKV);
#pragma unroll
      for (int cb = 0; cb < D / 64; ++cb)
        tma_load_4d(sV(j) + cb * 8192, &tmV, cb * 64, u * kUnit, hk, b, V_FULL(j));
      nv = j + 1;
      u = next;
    }
    // no load may land after the CTA has gone, not even when a wait ran out
    if (n > 0) mbar_wait_drain(Q_FULL, 0, drain_ns(p.spin_ns), p.err, p.err + 1);
    for (int j = max(0, nk - C::kK); j < nk; ++j)
      mbar_wait_drain(K_FULL(j), phK(j), drain_ns(p.spin_ns), p.err, p.err + 1);
    for (int j = max(0, nv - C::kV); j < nv; ++j)
      mbar_wait_drain(V_FULL(j), phV(j), drain_ns(p.spin_ns), p.err, p.err + 1);
  } else if (warp == 1) {
    // ---------------------------------------------------------------- S issuer
    constexpr uint32_t ID_S = idesc_bf16_f32(128, kUnit, 0, 0);
    const bool leader = elect_one();
    const uint32_t hi = sdesc_hi(1024);
    const uint32_t kQ = sdesc_lo(sQ, 16);
    bool ok = n == 0 || wait(Q_FULL, 0);
#pragma unroll 1
    for (int j = 0; j < n && ok; ++j) {
      const uint32_t kK = sdesc_lo(sK(j), 16);
      const uint32_t tS = tmem + C::TM_S + 64u * (uint32_t)(j & 1);
      // P_{j-2} lay in S_j's buffer
      ok = wait(K_FULL(j), phK(j)) && (j < 2 || wait(PV_DONE(j), ph2(j - 2)));
      if (!ok) break;
      tc_fence_after();
      if (leader) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          tc_mma_ss_w(tS, kQ + (uint32_t)(((kk >> 2) * 16384 + (kk & 3) * 32) >> 4),
                      kK + (uint32_t)(((kk >> 2) * 8192 + (kk & 3) * 32) >> 4), hi, ID_S,
                      kk > 0 ? 1u : 0u);
        tc_commit(S_FULL(j));
        tc_commit(K_EMPTY(j));
      }
    }
    if (leader) tc_commit(S_FINAL);  // the CTA does not go before its products
    mbar_wait_drain(S_FINAL, 0, drain_ns(p.spin_ns), p.err, p.err + 1);
  } else if (warp == 2) {
    // ---------------------------------------------------------------- P V issuer
    constexpr uint32_t ID_PV = idesc_bf16_f32(128, D, 0, 1);
    const bool leader = elect_one();
    const uint32_t hi = sdesc_hi(1024);
    const uint32_t tO = tmem + C::TM_O;
    bool ok = true;
#pragma unroll 1
    for (int j = 0; j < n && ok; ++j) {
      const uint32_t mV = sdesc_lo(sV(j), 8192);
      const uint32_t tP = tmem + C::TM_S + 64u * (uint32_t)(j & 1);
      ok = wait(V_FULL(j), phV(j)) && wait(P_READY(j), ph2(j));
      if (!ok) break;
      tc_fence_after();
      if (leader) {
#pragma unroll
        for (int kk = 0; kk < kUnit / 16; ++kk)
          tc_mma_ts_w(tO, tP + 32 * (kk >> 1) + 8 * (kk & 1), mV + kk * 128, hi, ID_PV,
                      (uint32_t)(j + kk));
        tc_commit(PV_DONE(j));
        tc_commit(V_EMPTY(j));
      }
    }
    if (leader) tc_commit(O_FINAL);
    mbar_wait_drain(O_FINAL, 0, drain_ns(p.spin_ns), p.err, p.err + 1);
  } else if (warp >= 4) {
    // ---------------------------------------------------------------- softmax
    const int quarter = warp & 3;
    const int r = quarter * 32 + lane;
    const int t = r / p.G, g = r - t * p.G, token = t0 + t;
    const bool valid = t < p.T && token < p.Sq;
    const int kvlen = p.plan.len[b];
    const long long pos = (long long)p.plan.start[b] + token;
    const int limit = !valid ? 0
                      : p.causal ? (int)min((long long)kvlen, max(pos + 1, 0ll)) : kvlen;
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const uint32_t tO = tmem + lane_off + C::TM_O;
    const float sl2 = p.scale_log2;
    const uint32_t* masks = p.plan.mask + (gt * p.U + beg) * p.W + min(t >> 5, p.W - 1);
    const int bit = t & 31;
    float m = -INFINITY, l = 0.f;
    int u = n > 0 ? units[0] : 0;
    uint32_t word = n > 0 ? masks[0] : 0u;
    for (int j = 0; j < n; ++j) {
      const int base = u * kUnit;
      const int vis = ((word >> bit) & 1u) ? limit - base : 0;  // keys below it are attended to
      if (j + 1 < n) {
        u = units[j + 1];
        word = masks[(long long)(j + 1) * p.W];
      }
      const bool any = __any_sync(0xffffffffu, vis > 0);
      const bool clean = __all_sync(0xffffffffu, vis >= kUnit || vis <= 0);
      const uint32_t tS = tmem + lane_off + C::TM_S + 64u * (uint32_t)(j & 1);
      if (base + kUnit > kvlen && kvlen < p.Sk) {
        // V rows past the sequence hold whatever the cache holds: 0 * NaN would reach O
        wait(V_FULL(j), phV(j));
        const int first = max(kvlen - base, 0);
        for (int x = r; x < (kUnit - first) * (D / 8); x += 128) {
          const int row = first + x / (D / 8), c = x % (D / 8);
          st_shared_v4(sV(j) + (c >> 3) * 8192 + row * 128 + (c & 7) * 16, 0, 0, 0, 0);
        }
        fence_proxy_async_smem();
      }
      wait(S_FULL(j), ph2(j));
      tc_fence_after();
      if (!any) {
        const uint32_t zero[16] = {};
        tmem_st16(tS, zero);
        tmem_st16(tS + 32, zero);
      } else {
        uint32_t sv[2][32];
        tmem_ld32x2(tS, tS + 32, sv[0], sv[1]);
        if (!clean)  // keys past a row's limit
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if (32 * c + k >= vis) sv[c][k] = 0xff800000u;
        float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int k = 0; k < 32; k += 2)
            top[(k >> 1) & 3] = fmaxf(top[(k >> 1) & 3], fmaxf(__uint_as_float(sv[c][k]),
                                                               __uint_as_float(sv[c][k + 1])));
        const float mt =
            vis > 0 ? fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * sl2 : -INFINITY;
        if (__any_sync(0xffffffffu, mt > m + C::kRescaleLog2)) {
          const float mn = fmaxf(m, mt);
          if (j > 0) {
            const float f = mn == -INFINITY ? 1.f : ex2_approx(m - mn);
            l *= f;
            wait(PV_DONE(j - 1), ph2(j - 1));
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t ov[32];
              tmem_ld32(tO + 32 * c, ov);
              uint32_t lo[16], up[16];
#pragma unroll
              for (int k = 0; k < 16; ++k) {
                lo[k] = __float_as_uint(__uint_as_float(ov[k]) * f);
                up[k] = __float_as_uint(__uint_as_float(ov[16 + k]) * f);
              }
              tmem_st16(tO + 32 * c, lo);
              tmem_st16(tO + 32 * c + 16, up);
            }
          }
          m = mn;
        }
        // a row that did not pick the unit gets zeros by `keep`; -inf - 0 where nothing is seen yet
        const uint32_t keep = vis > 0 ? 0xffffffffu : 0u;
        const float mz = m == -INFINITY ? 0.f : m;
        float l0 = 0.f, l1 = 0.f;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t pk[16];
#pragma unroll
          for (int k = 0; k < 32; k += 2) {
            float p0, p1;
            fma_f32x2(p0, p1, __uint_as_float(sv[c][k]), __uint_as_float(sv[c][k + 1]), sl2, -mz);
            p0 = ex2_approx(p0);
            p1 = ex2_approx(p1);
            l0 += p0;
            l1 += p1;
            pk[k >> 1] = pack_bf16x2(p0, p1) & keep;
          }
          tmem_st16(tS + 32 * c, pk);
        }
        if (vis > 0) l += l0 + l1;
      }
      tmem_wait_st();
      tc_fence_before();
      warp_arrive(P_READY(j), lane);
    }
    // epilogue; a row that attended to nothing gets O = 0 and LSE = -inf
    wait(O_FINAL, 0);
    tc_fence_after();
    const bool some = l > 0.f;
    const bool bad = l != l;  // NaN in the row's own operands stays visible
    const float inv = some ? 1.0f / l : (bad ? l : 0.f);
    const float lse2 = some || bad ? m + log2f(l) : -INFINITY;
    const long long row = ((long long)b * p.H + hk * p.G + g) * p.Sq + token;
#pragma unroll 1
    for (int c = 0; c < D / 32; ++c) {
      uint32_t ov[32];
      tmem_ld32(tO + 32 * c, ov);  // every lane takes part in the load
      if (!valid) continue;
      float x[32];
#pragma unroll
      for (int k = 0; k < 32; ++k) x[k] = (some || bad) ? __uint_as_float(ov[k]) * inv : 0.f;
      if (p.splits > 1) {
        float4* out = reinterpret_cast<float4*>(
            p.part_o + ((long long)split * (gridDim.x / p.splits / p.NT) * p.G * p.Sq + row) * D +
            32 * c);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          out[k] = make_float4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]);
      } else {
        uint4* out = reinterpret_cast<uint4*>(p.o + row * D + 32 * c);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          out[k] = make_uint4(pack_bf16x2(x[8 * k], x[8 * k + 1]),
                              pack_bf16x2(x[8 * k + 2], x[8 * k + 3]),
                              pack_bf16x2(x[8 * k + 4], x[8 * k + 5]),
                              pack_bf16x2(x[8 * k + 6], x[8 * k + 7]));
      }
    }
    if (valid) {
      if (p.splits > 1)
        p.part_l[(long long)split * BHk * p.G * p.Sq + row] = lse2;
      else
        p.lse[row] = lse2 * 0.69314718055994531f;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// Joins the parts of a split list: O = sum_s w_s O_s with w_s = 2^(l_s - l), one warp a
// row, the parts in ascending order.  Bound by reading the parts.
template <int D>
__global__ void __launch_bounds__(128)
    dash_sparse_join_kernel(const float* part_o, const float* part_l, __nv_bfloat16* o, float* lse,
                            long long rows, int splits) {
  const long long row = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (row >= rows) return;
  float top = -INFINITY;
  bool bad = false;
  for (int s = 0; s < splits; ++s) {
    const float x = part_l[s * rows + row];
    bad |= x != x;
    top = fmaxf(top, x);
  }
  float acc[D / 32] = {}, total = 0.f;
  if (top != -INFINITY || bad)
    for (int s = 0; s < splits; ++s) {
      const float w = dev::ex2_approx(part_l[s * rows + row] - top);
      total += w;
      const float* src = part_o + (s * rows + row) * D;
#pragma unroll
      for (int k = 0; k < D / 32; ++k) acc[k] += w * src[32 * k + lane];
    }
  const float inv = total != 0.f ? 1.f / total : 0.f;
#pragma unroll
  for (int k = 0; k < D / 32; ++k) o[row * D + 32 * k + lane] = __float2bfloat16_rn(acc[k] * inv);
  if (lane == 0) lse[row] = (top + log2f(total)) * 0.69314718055994531f;
}

}  // namespace dash
