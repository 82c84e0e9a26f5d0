// Block-sparse attention backward for sm_100a.
//
//   P  = 2^(s S - LSE log2 e) on the visible keys of the picked units, 0 elsewhere
//   dP = dO V^T,  delta = rowsum(dO o O),  dS = P o (dP - delta)
//   dQ = scale dS K,   dK = scale dS^T Q,   dV = P^T dO
//
// Two passes recompute S and dP, each with its result resident in TMEM, so that every sum
// has one owner and a fixed order and no partial of dQ goes through memory:
//   dash_sparse_dq_kernel   a CTA per query tile walks the tile's listed units (as the
//                           forward does) and also writes delta;
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

// ------------------------------------------------------------------ dQ
struct SparseDqParams {
  PlanView plan;
  const __nv_bfloat16* o;  // [B,H,Sq,D]
  const float* lse;        // [B,H,Sq]
  __nv_bfloat16* dq;       // [B,H,Sq,D]
  float* delta;            // [B,H,Sq]
  unsigned* err;
  int H, Hkv, Sq, Sk, G, T, W, NT, U, causal;
  float scale, scale_log2;
  unsigned long long spin_ns;
};

template <int D>
struct SparseDqCfg {
  static constexpr int kThreads = 192;
  static constexpr int kQ = kTileRows * D * 2;
  static constexpr int kKV = kUnit * D * 2;
  static constexpr int kKSt = 2;                  // K is read by S and by dQ
  static constexpr int kVSt = D == 128 ? 1 : 2;   // V is free again after dP
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_DO = kQ;
  static constexpr int OFF_K = 2 * kQ;
  static constexpr int OFF_V = OFF_K + kKSt * kKV;
  static constexpr int OFF_BAR = OFF_V + kVSt * kKV;
  static constexpr int kBars = 6 + 2 * kKSt + 2 * kVSt;
  static constexpr int OFF_SLOT = OFF_BAR + kBars * 8;
  static constexpr int kSmemBytes = OFF_SLOT + 16;
  static_assert(kSmemBytes <= 115712, "two CTAs per SM");
  static constexpr uint32_t TM_S = 0, TM_DP = 64, TM_DQ = 128, kTmemCols = 256;
};

template <int D>
__global__ void __launch_bounds__(192, 2)
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
  const uint32_t sQ = sb + C::OFF_Q, sDO = sb + C::OFF_DO, sK = sb + C::OFF_K, sV = sb + C::OFF_V;
  const uint32_t bar0 = sb + C::OFF_BAR;
  const uint32_t Q_FULL = bar0, S_FULL = bar0 + 8, DP_FULL = bar0 + 16, DS_READY = bar0 + 24;
  const uint32_t DQ_DONE = bar0 + 32, FINAL = bar0 + 40;
  auto K_FULL = [&](int j) { return bar0 + 48u + 8u * (uint32_t)(j % C::kKSt); };
  auto K_EMPTY = [&](int j) { return bar0 + 48u + 8u * (uint32_t)(C::kKSt + j % C::kKSt); };
  auto V_FULL = [&](int j) { return bar0 + 48u + 8u * (uint32_t)(2 * C::kKSt + j % C::kVSt); };
  auto V_EMPTY = [&](int j) {
    return bar0 + 48u + 8u * (uint32_t)(2 * C::kKSt + C::kVSt + j % C::kVSt);
  };
  auto phK = [&](int j) { return (uint32_t)((j / C::kKSt) & 1); };
  auto phV = [&](int j) { return (uint32_t)((j / C::kVSt) & 1); };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem_raw + C::OFF_SLOT);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto wait = [&](uint32_t bar, uint32_t phase) {
    mbar_wait(bar, phase, p.spin_ns, p.err, p.err + 1);
  };
  const int BHk = (int)(gridDim.x / (unsigned)p.NT);
  const int tile = p.NT - 1 - (int)(blockIdx.x / (unsigned)BHk);
  const int bh = (int)(blockIdx.x % (unsigned)BHk);
  const int b = bh / p.Hkv, hk = bh % p.Hkv, t0 = tile * p.T;
  const long long gt = (long long)bh * p.NT + tile;
  const int n = p.plan.count[gt];
  const int* units = p.plan.unit + gt * p.U;
  const int kvlen = p.plan.len[b];

  if (threadIdx.x == 0) {
    mbar_init(Q_FULL, 1);
    mbar_init(S_FULL, 1);
    mbar_init(DP_FULL, 1);
    mbar_init(DS_READY, 128);
    mbar_init(DQ_DONE, 1);
    mbar_init(FINAL, 1);
    for (int i = 0; i < 2 * C::kKSt + 2 * C::kVSt; ++i) mbar_init(bar0 + 48u + 8u * i, 1);
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
    mbar_expect_tx(Q_FULL, (uint32_t)(2 * p.G * p.T * D * 2));
#pragma unroll
    for (int cb = 0; cb < D / 64; ++cb) {
      tma_load_4d(sQ + cb * 16384, &tmQ, cb * 64, t0, hk * p.G, b, Q_FULL);
      tma_load_4d(sDO + cb * 16384, &tmDO, cb * 64, t0, hk * p.G, b, Q_FULL);
    }
    int u = n > 0 ? units[0] : 0;
    for (int j = 0; j < n; ++j) {
      const int next = j + 1 < n ? units[j + 1] : 0;
      if (j >= C::kKSt) wait(K_EMPTY(j), phK(j - C::kKSt));
      mbar_expect_tx(K_FULL(j), C::kKV);
#pragma unroll
      for (int cb = 0; cb < D / 64; ++cb)
        tma_load_4d(sK + (j % C::kKSt) * C::kKV + cb * 8192, &tmK, cb * 64, u * kUnit, hk, b,
                    K_FULL(j));
      if (j >= C::kVSt) wait(V_EMPTY(j), phV(j - C::kVSt));
      mbar_expect_tx(V_FULL(j), C::kKV);
#pragma unroll
      for (int cb = 0; cb < D / 64; ++cb)
        tma_load_4d(sV + (j % C::kVSt) * C::kKV + cb * 8192, &tmV, cb * 64, u * kUnit, hk, b,
                    V_FULL(j));
      u = next;
    }
    // no load may land after the CTA has gone, not even when a wait ran out
    mbar_wait_drain(Q_FULL, 0, p.spin_ns, p.err, p.err + 1);
    for (int j = max(0, n - 2); j < n; ++j) {
      mbar_wait_drain(K_FULL(j), phK(j), p.spin_ns, p.err, p.err + 1);
      if (j >= n - C::kVSt) mbar_wait_drain(V_FULL(j), phV(j), p.spin_ns, p.err, p.err + 1);
    }
  } else if (warp == 1 && lane == 0) {
    // ---------------------------------------------------------------- MMA issuer
    constexpr uint32_t ID_S = idesc_bf16_f32(128, kUnit, 0, 0);  // S, dP
    constexpr uint32_t ID_Q = idesc_bf16_f32(128, D, 0, 1);      // dQ, K MN-major
    const uint32_t hi = sdesc_hi(1024);
    const uint32_t kQ = sdesc_lo(sQ, 16), kDO = sdesc_lo(sDO, 16);
    const uint32_t tS = tmem + C::TM_S, tDP = tmem + C::TM_DP, tDQ = tmem + C::TM_DQ;
    // dS_i lies packed in dP's columns
    auto issue_dq = [&](int i) {
      const uint32_t mK = sdesc_lo(sK + (i % C::kKSt) * C::kKV, 8192);
#pragma unroll
      for (int kk = 0; kk < kUnit / 16; ++kk)
        tc_mma_ts_w(tDQ, tDP + 32 * (kk >> 1) + 8 * (kk & 1), mK + kk * 128, hi, ID_Q,
                    (i > 0 || kk > 0) ? 1u : 0u);
      tc_commit(K_EMPTY(i));
      tc_commit(DQ_DONE);
    };
    if (n > 0) wait(Q_FULL, 0);
    for (int j = 0; j < n; ++j) {
      const uint32_t kK = sdesc_lo(sK + (j % C::kKSt) * C::kKV, 16);
      const uint32_t kV = sdesc_lo(sV + (j % C::kVSt) * C::kKV, 16);
      wait(K_FULL(j), phK(j));
      if (j > 0) wait(DS_READY, (uint32_t)((j - 1) & 1));  // S_{j-1} and dP_{j-1} are read
      tc_fence_after();
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
        tc_mma_ss_w(tS, kQ + (uint32_t)(((kk >> 2) * 16384 + (kk & 3) * 32) >> 4),
                    kK + (uint32_t)(((kk >> 2) * 8192 + (kk & 3) * 32) >> 4), hi, ID_S,
                    kk > 0 ? 1u : 0u);
      tc_commit(S_FULL);
      if (j > 0) {
        issue_dq(j - 1);
        wait(DQ_DONE, (uint32_t)((j - 1) & 1));  // dP_j overwrites dS_{j-1}
      }
      wait(V_FULL(j), phV(j));
      tc_fence_after();
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
        tc_mma_ss_w(tDP, kDO + (uint32_t)(((kk >> 2) * 16384 + (kk & 3) * 32) >> 4),
                    kV + (uint32_t)(((kk >> 2) * 8192 + (kk & 3) * 32) >> 4), hi, ID_S,
                    kk > 0 ? 1u : 0u);
      tc_commit(V_EMPTY(j));
      tc_commit(DP_FULL);
    }
    if (n > 0) {
      wait(DS_READY, (uint32_t)((n - 1) & 1));
      tc_fence_after();
      issue_dq(n - 1);
    }
    tc_commit(FINAL);
    mbar_wait_drain(FINAL, 0, p.spin_ns, p.err, p.err + 1);
  } else if (warp >= 2) {
    // ---------------------------------------------------------------- softmax gradient
    const int quarter = warp & 3;
    const int r = quarter * 32 + lane;
    const int g = r / p.T, t = r - g * p.T, token = t0 + t;
    const bool valid = g < p.G && token < p.Sq;
    const long long row = ((long long)b * p.H + hk * p.G + g) * p.Sq + token;
    const long long pos = (long long)p.plan.start[b] + token;
    const int limit = !valid ? 0
                      : p.causal ? (int)min((long long)kvlen, max(pos + 1, 0ll)) : kvlen;
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const uint32_t tS = tmem + lane_off + C::TM_S, tDP = tmem + lane_off + C::TM_DP;
    const float sl2 = p.scale_log2;
    const uint32_t* masks = p.plan.mask + gt * p.U * p.W + min(t >> 5, p.W - 1);
    const int bit = t & 31;
    const float lse2 = valid ? p.lse[row] * 1.4426950408889634f : 0.f;
    // delta: dO from shared memory (16-byte pieces, swizzled by row), O from memory
    float delta = 0.f;
    wait(Q_FULL, 0);
    if (valid) {
      const uint4* orow = reinterpret_cast<const uint4*>(p.o + row * D);
#pragma unroll 4
      for (int c = 0; c < D / 8; ++c) {
        const uint4 x = orow[c];
        const float4 y = ld_shared_f4(sDO + (c >> 3) * 16384 + r * 128 + (((c & 7) ^ (r & 7)) << 4));
        const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
        const uint32_t ys[4] = {__float_as_uint(y.x), __float_as_uint(y.y), __float_as_uint(y.z),
                                __float_as_uint(y.w)};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          delta = fmaf(__uint_as_float(xs[k] << 16), __uint_as_float(ys[k] << 16), delta);
          delta = fmaf(__uint_as_float(xs[k] & 0xffff0000u),
                       __uint_as_float(ys[k] & 0xffff0000u), delta);
        }
      }
      p.delta[row] = delta;
    }
    int u = n > 0 ? units[0] : 0;
    uint32_t word = n > 0 ? masks[0] : 0u;
    for (int j = 0; j < n; ++j) {
      const int base = u * kUnit;
      const int vis = ((word >> bit) & 1u) ? limit - base : 0;
      if (j + 1 < n) {
        u = units[j + 1];
        word = masks[(long long)(j + 1) * p.W];
      }
      wait(S_FULL, (uint32_t)(j & 1));
      tc_fence_after();
      uint32_t sv[2][32];
      tmem_ld32x2(tS, tS + 32, sv[0], sv[1]);
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int k = 0; k < 32; ++k)
          sv[c][k] = __float_as_uint(
              32 * c + k < vis ? ex2_approx(__uint_as_float(sv[c][k]) * sl2 - lse2) : 0.f);
      wait(DP_FULL, (uint32_t)(j & 1));
      tc_fence_after();
      if (base + kUnit > kvlen && kvlen < p.Sk) {
        // K rows past the sequence hold whatever the cache holds: 0 * NaN would reach dQ
        const int first = kvlen - base;
        const uint32_t sKj = sK + (j % C::kKSt) * C::kKV;
        for (int x = r; x < (kUnit - first) * (D / 8); x += 128) {
          const int kr = first + x / (D / 8), c = x % (D / 8);
          st_shared_v4(sKj + (c >> 3) * 8192 + kr * 128 + (c & 7) * 16, 0, 0, 0, 0);
        }
        fence_proxy_async_smem();
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t dp[32], pk[16];
        tmem_ld32(tDP + 32 * c, dp);
#pragma unroll
        for (int k = 0; k < 32; k += 2) {
          // selected, not multiplied: dP of a masked key may be anything
          const float d0 = 32 * c + k < vis
                               ? __uint_as_float(sv[c][k]) * (__uint_as_float(dp[k]) - delta) : 0.f;
          const float d1 = 32 * c + k + 1 < vis
                               ? __uint_as_float(sv[c][k + 1]) * (__uint_as_float(dp[k + 1]) - delta)
                               : 0.f;
          pk[k >> 1] = pack_bf16x2(d0, d1);
        }
        tmem_st16(tDP + 32 * c, pk);
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(DS_READY);
    }
    wait(FINAL, 0);
    tc_fence_after();
    const uint32_t tDQ = tmem + lane_off + C::TM_DQ;
#pragma unroll 1
    for (int c = 0; c < D / 32; ++c) {
      uint32_t ov[32];
      tmem_ld32(tDQ + 32 * c, ov);
      if (!valid) continue;
      const float f = n > 0 ? p.scale : 0.f;
      float x[32];
#pragma unroll
      for (int k = 0; k < 32; ++k) x[k] = n > 0 ? __uint_as_float(ov[k]) * f : 0.f;
      uint4* out = reinterpret_cast<uint4*>(p.dq + row * D + 32 * c);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        out[k] = make_uint4(pack_bf16x2(x[8 * k], x[8 * k + 1]),
                            pack_bf16x2(x[8 * k + 2], x[8 * k + 3]),
                            pack_bf16x2(x[8 * k + 4], x[8 * k + 5]),
                            pack_bf16x2(x[8 * k + 6], x[8 * k + 7]));
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
// prefix sums, written.  A warp per unit, a lane per query tile.
struct InverseParams {
  PlanView plan;
  int* count;  // [units] tokens of the unit
  int* off;    // [units] its first place in `token`
  int* token;
  int nu, NW, NT, T, U, W;
  long long units;  // B*Hkv*nu
};
template <bool kFill>
__global__ void __launch_bounds__(128)
    dash_sparse_inverse_kernel(const __grid_constant__ InverseParams p) {
  const long long gu = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (gu >= p.units) return;
  const int lane = threadIdx.x & 31;
  const long long bh = gu / p.nu;
  const int u = (int)(gu % p.nu);
  const uint32_t* pres = p.plan.pres + bh * p.NT * p.NW + (u >> 5);
  const int* pre = p.plan.pre + bh * p.NT * p.NW + (u >> 5);
  int* out = kFill ? p.token + p.off[gu] : nullptr;
  int n = 0;
  for (int t0 = 0; t0 < p.NT; t0 += 32) {
    const int t = t0 + lane;
    const uint32_t w = t < p.NT ? pres[(long long)t * p.NW] : 0u;
    const bool on = (w >> (u & 31)) & 1u;
    uint32_t m[4] = {0u, 0u, 0u, 0u};  // T <= 128 tokens
    if (on) {
      const int place = pre[(long long)t * p.NW] + __popc(w & ((1u << (u & 31)) - 1u));
      const uint32_t* mask = p.plan.mask + ((bh * p.NT + t) * p.U + place) * p.W;
#pragma unroll
      for (int x = 0; x < 4; ++x)
        if (x < p.W) m[x] = mask[x];
    }
    const int mine = __popc(m[0]) + __popc(m[1]) + __popc(m[2]) + __popc(m[3]);
    if constexpr (kFill) {
      int before = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += y;
      }
      const int all = __shfl_sync(0xffffffffu, before, 31);
      int at = n + before - mine;
#pragma unroll
      for (int x = 0; x < 4; ++x)
        for (uint32_t rest = m[x]; rest; rest &= rest - 1)
          out[at++] = t * p.T + 32 * x + __ffs(rest) - 1;
      n += all;
    } else {
      n += mine;
    }
  }
  if constexpr (!kFill) {
    n = __reduce_add_sync(0xffffffffu, n);
    if (lane == 0) p.count[gu] = n;
  }
}

// Items of the dK/dV pass: every picked unit, its tokens in tiles of T, cut into stretches of
// at most C tiles with C = max(4, total / kStretches).  Whole stretches come first, so that
// the CTAs that take items in turn get equally many of them.
constexpr int kStretches = 148 * 8;
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
// One CTA: sums, then exclusive prefix sums of the tokens, items and partial slots per unit.
__global__ void __launch_bounds__(1024) dash_sparse_items_kernel(const ItemParams p) {
  __shared__ long long sum[32];
  __shared__ int pre[4][32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  auto block_sum = [&](auto&& f) {
    long long s = 0;
    for (long long x = tid; x < p.units; x += 1024) s += f((p.count[x] + p.T - 1) / p.T);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    __syncthreads();
    if (lane == 0) sum[warp] = s;
    __syncthreads();
    long long t = sum[lane];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    return t;
  };
  const long long total = block_sum([](int n) { return n; });
  const int C = (int)max((long long)kMinStretch, (total + kStretches - 1) / kStretches);
  const int whole = (int)block_sum([&](int n) { return n / C; });
  int base[4] = {0, whole, 0, 0};  // whole stretches, rests, slots, tokens
  for (long long x0 = 0; x0 < p.units; x0 += 1024) {
    const long long x = x0 + tid;
    const int tokens = x < p.units ? p.count[x] : 0;
    const int n = (tokens + p.T - 1) / p.T;
    const int full = n / C, rest = n % C > 0, cut = full + rest > 1 ? full + rest : 0;
    const int own[4] = {full, rest, cut, tokens};
    int inc[4] = {full, rest, cut, tokens};  // inclusive prefix sums over the warp
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int y = __shfl_up_sync(0xffffffffu, inc[k], o);
        if (lane >= o) inc[k] += y;
      }
    if (lane == 31)
#pragma unroll
      for (int k = 0; k < 4; ++k) pre[k][warp] = inc[k];
    __syncthreads();
    int at[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int y = pre[k][lane];
      at[k] = base[k] + __reduce_add_sync(0xffffffffu, lane < warp ? y : 0) + inc[k] - own[k];
      base[k] += __reduce_add_sync(0xffffffffu, y);
    }
    if (x < p.units) {
      p.off[x] = at[3];
      p.slot0[x] = n == 0 ? -2 : cut ? at[2] : -1;
      SparseItem w;
      w.unit = (int)x;
      w.off = at[3], w.tokens = tokens;
      w.bh = (int)(x / p.nu);
      w.b = w.bh / p.Hkv;
      for (int k = 0; k < full + rest; ++k) {
        w.first = k * C, w.end = min(n, (k + 1) * C);
        w.slot = cut ? at[2] + k : -1;
        p.item[k < full ? at[0] + k : at[1]] = w;
      }
    }
    __syncthreads();
  }
  if (tid == 0) {
    p.head[0] = base[1];
    p.head[1] = C;
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
  float scale, scale_log2;
  unsigned long long spin_ns;
};

template <int D>
struct SparseDkvCfg {
  static constexpr int kThreads = 640;  // Q rows, dO rows (4 warps each), MMA, K/V, 8 softmax
  static constexpr int kTile = kTileRows * D * 2;
  static constexpr int kKV = kUnit * D * 2;
  static constexpr int kP = kTileRows * kUnit * 2;  // [128][64] bf16
  static constexpr int kStages = D == 128 ? 2 : 4;
  static constexpr int OFF_QDO = 0;  // per stage dO, then Q: at D = 64 one [dO | Q] operand
  static constexpr int OFF_KV = kStages * 2 * kTile;  // two of K, then V
  static constexpr int OFF_P = OFF_KV + 4 * kKV;      // P, then dS
  static constexpr int OFF_BAR = OFF_P + 2 * kP;
  static constexpr int kBars = 4 * kStages + 6 + 4;
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
// one tile run under the exponentials of the other, also from item to item.  The two softmax
// warpgroups take 32 keys of every row each.
template <int D>
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
  const uint32_t sP = sb + C::OFF_P, sS = sP + C::kP;
  const uint32_t bar0 = sb + C::OFF_BAR;
  // per stage (Q, dO), per item parity, per tile parity
  auto FULL = [&](int x, int s) { return bar0 + 8u * (uint32_t)(x * ST + s); };
  auto EMPTY = [&](int x, int s) { return bar0 + 8u * (uint32_t)((2 + x) * ST + s); };
  const uint32_t bar1 = bar0 + 32u * ST;
  auto KV_FULL = [&](int k) { return bar1 + 8u * (uint32_t)(k & 1); };
  auto ITEM_DONE = [&](int k) { return bar1 + 16u + 8u * (uint32_t)(k & 1); };
  auto ACC_FREE = [&](int k) { return bar1 + 32u + 8u * (uint32_t)(k & 1); };
  auto SDP_FULL = [&](int j) { return bar1 + 48u + 8u * (uint32_t)(j & 1); };
  const uint32_t PDS_READY = bar1 + 64, PDS_FREE = bar1 + 72;
  auto ph2 = [](int k) { return (uint32_t)((k >> 1) & 1); };
  auto phS = [](int j) { return (uint32_t)((j / ST) & 1); };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem_raw + C::OFF_SLOT);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto wait = [&](uint32_t bar, uint32_t phase) {
    mbar_wait(bar, phase, p.spin_ns, p.err, p.err + 1);
  };
  const int items = p.head[0];
  const uint32_t inv_g = (65536u + p.G - 1) / p.G;  // row / G = row * inv_g >> 16 for row < 128
  const int rows = p.G * p.T;

  if (threadIdx.x == 0) {
    for (int s = 0; s < ST; ++s)
      for (int x = 0; x < 2; ++x) {
        mbar_init(FULL(x, s), 128);
        mbar_init(EMPTY(x, s), 1);
      }
    for (int k = 0; k < 2; ++k) {
      mbar_init(KV_FULL(k), 1);
      mbar_init(ITEM_DONE(k), 1);
      mbar_init(ACC_FREE(k), 256);
      mbar_init(SDP_FULL(k), 1);
    }
    mbar_init(PDS_READY, 256);
    mbar_init(PDS_FREE, 1);
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
    if ((int)blockIdx.x < items) {
      w = p.item[blockIdx.x];
      token = look(w, w.first);
    }
    for (int i = blockIdx.x; i < items; i += gridDim.x) {
      const bool more = i + (int)gridDim.x < items;
      SparseItem nw = w;
      if (more) nw = p.item[i + gridDim.x];
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
        mbar_arrive(FULL(x, s));
      }
      w = nw;
    }
  } else if (warp == 9 && lane == 0) {
    // ---------------------------------------------------------------- K and V
    int k = 0;
    for (int i = blockIdx.x; i < items; i += gridDim.x, ++k) {
      const SparseItem w = p.item[i];
      const int u = w.unit - w.bh * p.nu, hk = w.bh - w.b * p.Hkv;
      if (k >= 2) wait(ITEM_DONE(k), ph2(k - 2));  // K and V of item k - 2 are read to the end
      mbar_expect_tx(KV_FULL(k), 2 * C::kKV);
#pragma unroll
      for (int cb = 0; cb < D / 64; ++cb) {
        tma_load_4d(sK(k) + cb * 8192, &tmK, cb * 64, u * kUnit, hk, w.b, KV_FULL(k));
        tma_load_4d(sV(k) + cb * 8192, &tmV, cb * 64, u * kUnit, hk, w.b, KV_FULL(k));
      }
    }
    // no load may land after the CTA has gone, not even when a wait ran out
    for (int j = max(0, k - 2); j < k; ++j)
      mbar_wait_drain(KV_FULL(j), ph2(j), p.spin_ns, p.err, p.err + 1);
  } else if (warp == 8 && lane == 0) {
    // ---------------------------------------------------------------- MMA issuer
    constexpr uint32_t ID_S = idesc_bf16_f32(128, kUnit, 0, 0);
    constexpr uint32_t ID_T = idesc_bf16_f32(128, kUnit, 1, 1);  // dV^T, dK^T
    const uint32_t hi = sdesc_hi(1024);
    const uint32_t bP = sdesc_lo(sP, 16384), bS = sdesc_lo(sS, 16384);
    // two cursors over the CTA's tiles: S and dP run up to two tiles ahead of dV and dK
    struct Cursor {
      int i, k, e, first, end, j;  // item, its number, tile, the item's tiles, tile number
      bool on;
    };
    auto open = [&](Cursor& c) {
      c.on = c.i < items;
      if (c.on) c.first = c.e = p.item[c.i].first, c.end = p.item[c.i].end;
    };
    auto step = [&](Cursor& c) {
      ++c.j;
      if (++c.e == c.end) c.i += gridDim.x, ++c.k, open(c);
    };
    Cursor a{(int)blockIdx.x, 0, 0, 0, 0, 0, false};
    open(a);
    Cursor d = a;
    int last = -1;  // the last item's number
    uint64_t since = 0;
    bool given_up = false;
    while (d.on) {
      bool did = false;
      if (a.on && a.j <= d.j + 1 && (given_up || (mbar_test_wait(FULL(0, a.j % ST), phS(a.j)) &&
                                                  mbar_test_wait(FULL(1, a.j % ST), phS(a.j)) &&
                                                  mbar_test_wait(KV_FULL(a.k), ph2(a.k))))) {
        // S and dP of tile j - 2 were read before its P and dS were ready
        const int s = a.j % ST;
        const uint32_t kQ = sdesc_lo(sQ(s), 16), kDO = sdesc_lo(sDO(s), 16);
        const uint32_t kK = sdesc_lo(sK(a.k), 16), kV = sdesc_lo(sV(a.k), 16);
        const uint32_t tS = tmem + C::TM_S + 128u * (uint32_t)(a.j & 1);
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          tc_mma_ss_w(tS, kQ + (uint32_t)(((kk >> 2) * 16384 + (kk & 3) * 32) >> 4),
                      kK + (uint32_t)(((kk >> 2) * 8192 + (kk & 3) * 32) >> 4), hi, ID_S,
                      kk > 0 ? 1u : 0u);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          tc_mma_ss_w(tS + 64, kDO + (uint32_t)(((kk >> 2) * 16384 + (kk & 3) * 32) >> 4),
                      kV + (uint32_t)(((kk >> 2) * 8192 + (kk & 3) * 32) >> 4), hi, ID_S,
                      kk > 0 ? 1u : 0u);
        tc_commit(SDP_FULL(a.j));
        step(a);
        did = true;
      }
      if (d.j < a.j && (given_up || mbar_test_wait(PDS_READY, (uint32_t)(d.j & 1)))) {
        const int s = d.j % ST;
        const bool first = d.e == d.first;
        // the accumulators of item k - 2 must have been read
        if (first && d.k >= 2) wait(ACC_FREE(d.k), ph2(d.k - 2));
        const uint32_t aV = sdesc_lo(sDO(s), 16384);
        const uint32_t aK = D == 128 ? sdesc_lo(sQ(s), 16384) : aV;
        const uint32_t tA = tmem + C::TM_ACC + 128u * (uint32_t)(d.k & 1);
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          tc_mma_ss_w(tA, aV + kk * 128, bP + kk * 128, hi, ID_T, (!first || kk > 0) ? 1u : 0u);
        if (D == 128) tc_commit(EMPTY(1, s));
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          tc_mma_ss_w(tA + 64, aK + kk * 128, bS + kk * 128, hi, ID_T,
                      (!first || kk > 0) ? 1u : 0u);
        if (D == 64) tc_commit(EMPTY(1, s));
        tc_commit(EMPTY(0, s));
        tc_commit(PDS_FREE);
        last = d.k;
        if (d.e + 1 == d.end) tc_commit(ITEM_DONE(d.k));
        step(d);
        did = true;
      }
      if (did) {
        since = 0;
      } else {
        const uint64_t now = globaltimer();
        if (since == 0) {
          since = now;
        } else if (now - since > p.spin_ns || aborted(p.err + 1)) {
          // go on without waiting, so that every other wait of the CTA ends
          if (!given_up) raise_timeout(p.err, p.err + 1, ERR_WHERE_PIPE);
          given_up = true;
        }
      }
    }
    if (last >= 0) mbar_wait_drain(ITEM_DONE(last), ph2(last), p.spin_ns, p.err, p.err + 1);
  } else if (warp >= 12) {
    // ---------------------------------------------------------------- softmax gradient
    const int wg = (warp - 12) >> 2, quarter = warp & 3;
    const int r = quarter * 32 + lane;
    const int t = (int)((uint32_t)r * inv_g >> 16), g = r - t * p.G;
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const uint32_t rowP = sP + r * 128, rowS = sS + r * 128;
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
    int it = 0, k = 0;
    SparseItem w;
    if ((int)blockIdx.x < items) {
      w = p.item[blockIdx.x];
      fetch(w, w.first);
    }
    for (int i = blockIdx.x; i < items; i += gridDim.x, ++k) {
      const bool more = i + (int)gridDim.x < items;
      SparseItem nw = w;
      if (more) nw = p.item[i + gridDim.x];
      for (int e = w.first; e < w.end; ++e, ++it) {
        const float l2 = lse2, dl = delta;
        const int v = vis - 32 * wg;
        if (e + 1 < w.end) fetch(w, e + 1);
        else if (more) fetch(nw, nw.first);
        const bool whole = __all_sync(0xffffffffu, v >= 32);
        const uint32_t tS = tmem + lane_off + C::TM_S + 128u * (uint32_t)(it & 1) + 32u * wg;
        wait(SDP_FULL(it), ph2(it));
        tc_fence_after();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t sv[16], dp[16];
          tmem_ld16_async(tS + 16 * h, sv);
          tmem_ld16_async(tS + 64 + 16 * h, dp);
          tmem_wait_ld();
          uint32_t pp[8], ds[8];
#pragma unroll
          for (int x = 0; x < 8; ++x) {
            float p0, p1, d0, d1;
            fma_f32x2(p0, p1, __uint_as_float(sv[2 * x]), __uint_as_float(sv[2 * x + 1]), sl2, -l2);
            p0 = ex2_approx(p0);
            p1 = ex2_approx(p1);
            add_f32x2(d0, d1, __uint_as_float(dp[2 * x]), __uint_as_float(dp[2 * x + 1]), -dl);
            mul_f32x2(d0, d1, p0, p1, d0, d1);
            if (!whole) {  // selected, not multiplied: S and dP of a masked key may be anything
              if (16 * h + 2 * x >= v) p0 = d0 = 0.f;
              if (16 * h + 2 * x + 1 >= v) p1 = d1 = 0.f;
            }
            pp[x] = pack_bf16x2(p0, p1);
            ds[x] = pack_bf16x2(d0, d1);
          }
          if (h == 0 && it > 0) wait(PDS_FREE, (uint32_t)((it - 1) & 1));
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const uint32_t off = (uint32_t)(((4 * wg + 2 * h + x) ^ (r & 7)) << 4);
            st_shared_v4(rowP + off, pp[4 * x], pp[4 * x + 1], pp[4 * x + 2], pp[4 * x + 3]);
            st_shared_v4(rowS + off, ds[4 * x], ds[4 * x + 1], ds[4 * x + 2], ds[4 * x + 3]);
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        mbar_arrive(PDS_READY);
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
          mbar_arrive(ACC_FREE(k));
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
