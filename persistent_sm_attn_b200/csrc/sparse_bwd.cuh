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
//                           stretch of the tiles that list it.
// A unit that many tiles list (the first block of a causal sequence) is cut into stretches;
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
// For every unit the tiles that list it, ascending, with the place in the tile's list.
struct InverseParams {
  PlanView plan;
  int2* entry;  // [B*Hkv*nu][NT] (tile, place)
  int* count;   // [B*Hkv*nu]
  int nu, NW, NT;
  long long units;  // B*Hkv*nu
};
__global__ void __launch_bounds__(128) dash_sparse_inverse_kernel(const __grid_constant__ InverseParams p) {
  const long long gu = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (gu >= p.units) return;
  const int lane = threadIdx.x & 31;
  const long long bh = gu / p.nu;
  const int u = (int)(gu % p.nu);
  const uint32_t* pres = p.plan.pres + bh * p.NT * p.NW + (u >> 5);
  const int* pre = p.plan.pre + bh * p.NT * p.NW + (u >> 5);
  int n = 0;
  for (int t0 = 0; t0 < p.NT; t0 += 32) {
    const int t = t0 + lane;
    const uint32_t w = t < p.NT ? pres[(long long)t * p.NW] : 0u;
    const bool on = (w >> (u & 31)) & 1u;
    const unsigned m = __ballot_sync(0xffffffffu, on);
    if (on)
      p.entry[gu * p.NT + n + __popc(m & ((1u << lane) - 1u))] =
          make_int2(t, pre[(long long)t * p.NW] + __popc(w & ((1u << (u & 31)) - 1u)));
    n += __popc(m);
  }
  if (lane == 0) p.count[gu] = n;
}

// Items of the dK/dV pass: every listed unit, cut into stretches of at most C entries with
// C = max(8, total / kStretches), so that the longest item is a small part of an SM's share.
constexpr int kStretches = 148 * 8;
constexpr int kMinStretch = 8;

struct ItemParams {
  const int* count;  // [units]
  int4* item;        // (unit, first entry, end entry, partial slot or -1)
  int* slot0;        // [units] first partial slot of a cut unit, -1 uncut, -2 never listed
  int* head;         // [0] items, [1] C
  long long units;
};
// One CTA: sums, then exclusive prefix sums of the items and partial slots per unit.
__global__ void __launch_bounds__(1024) dash_sparse_items_kernel(const ItemParams p) {
  __shared__ long long sum[32];
  __shared__ int2 pre[32];
  __shared__ long long total;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  long long s = 0;
  for (long long x = tid; x < p.units; x += 1024) s += p.count[x];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0) sum[warp] = s;
  __syncthreads();
  if (tid == 0) {
    long long t = 0;
    for (int w = 0; w < 32; ++w) t += sum[w];
    total = t;
  }
  __syncthreads();
  const int C = (int)max((long long)kMinStretch, (total + kStretches - 1) / kStretches);
  int items = 0, slots = 0;
  for (long long x0 = 0; x0 < p.units; x0 += 1024) {
    const long long x = x0 + tid;
    const int n = x < p.units ? p.count[x] : 0;
    const int parts = (n + C - 1) / C, cut = parts > 1 ? parts : 0;
    int a = parts, c = cut;  // inclusive prefix sums over the CTA
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int ya = __shfl_up_sync(0xffffffffu, a, o), yc = __shfl_up_sync(0xffffffffu, c, o);
      if (lane >= o) a += ya, c += yc;
    }
    if (lane == 31) pre[warp] = make_int2(a, c);
    __syncthreads();
    int ba = items, bc = slots, ta = 0, tc = 0;
    for (int w = 0; w < 32; ++w) {
      if (w < warp) ba += pre[w].x, bc += pre[w].y;
      ta += pre[w].x, tc += pre[w].y;
    }
    if (x < p.units) {
      const int i0 = ba + a - parts, s0 = bc + c - cut;
      p.slot0[x] = n == 0 ? -2 : cut ? s0 : -1;
      for (int k = 0; k < parts; ++k)
        p.item[i0 + k] = make_int4((int)x, k * C, min(n, (k + 1) * C), cut ? s0 + k : -1);
    }
    items += ta;
    slots += tc;
    __syncthreads();
  }
  if (tid == 0) {
    p.head[0] = items;
    p.head[1] = C;
  }
}

// ------------------------------------------------------------------ dK, dV
struct SparseDkvParams {
  PlanView plan;
  const int2* entry;
  const int4* item;
  const int* head;
  const float* lse;
  const float* delta;
  __nv_bfloat16 *dk, *dv;  // [B,Hkv,Sk,D]
  float* part;             // [slots][2][64][D] (dK, dV)
  unsigned* err;
  int H, Hkv, Sq, Sk, G, T, W, NT, U, nu, causal;
  float scale, scale_log2;
  unsigned long long spin_ns;
};

template <int D>
struct SparseDkvCfg {
  static constexpr int kThreads = 320;  // TMA, MMA, two softmax warpgroups
  static constexpr int kTile = kTileRows * D * 2;
  static constexpr int kKV = kUnit * D * 2;
  static constexpr int kP = kTileRows * kUnit * 2;  // [128][64] bf16
  static constexpr int kStages = 2;
  static constexpr int OFF_QDO = 0;  // per stage dO, then Q: at D = 64 one [dO | Q] operand
  static constexpr int OFF_K = kStages * 2 * kTile;
  static constexpr int OFF_V = OFF_K + kKV;
  static constexpr int OFF_P = OFF_V + kKV;  // per warpgroup P, then dS
  static constexpr int OFF_BAR = OFF_P + 4 * kP;
  static constexpr int kBars = 2 * kStages + 2 + 2 * 3 + 1;
  static constexpr int OFF_SLOT = OFF_BAR + kBars * 8;
  static constexpr int kNeed = OFF_SLOT + 16;
  // at least 120 KiB, so one CTA runs per SM and its 512 TMEM columns are free
  static constexpr int kSmemBytes = kNeed > 122880 ? kNeed : 122880;
  static_assert(kSmemBytes <= 232448, "shared memory per block exceeded");
  static constexpr uint32_t TM_S = 0, TM_DV = 256, TM_DK = 320, kTmemCols = 512;
};

// Per entry (a query tile that lists the unit): S = Q K^T and dP = dO V^T as 128 x 64, P and
// dS in bf16 to shared memory, then dV^T += dO^T P and dK^T += Q^T dS with the head dimension
// as the 128 MMA rows (a 64-key M would halve the rate).  At D = 64 the stacked operand
// [dO | Q] serves both: dV^T is the upper half of one product, dK^T the lower of the other.
// The warpgroups take entries in turn, so one's exponentials run under the other's products.
template <int D>
__global__ void __launch_bounds__(320, 1)
    dash_sparse_dkdv_kernel(const __grid_constant__ CUtensorMap tmQ,
                            const __grid_constant__ CUtensorMap tmDO,
                            const __grid_constant__ CUtensorMap tmK,
                            const __grid_constant__ CUtensorMap tmV,
                            const __grid_constant__ SparseDkvParams p) {
  using namespace dev;
  using C = SparseDkvCfg<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t sb = smem_u32(smem_raw);
  if (sb & 1023u) {
    if (threadIdx.x == 0) atomicOr(p.err, ERR_MISALIGNED);
    return;
  }
  const uint32_t sK = sb + C::OFF_K, sV = sb + C::OFF_V;
  auto sDO = [&](int s) { return sb + C::OFF_QDO + (uint32_t)(s * 2 * C::kTile); };
  auto sQ = [&](int s) { return sDO(s) + C::kTile; };
  auto sP = [&](int w) { return sb + C::OFF_P + (uint32_t)(w * 2 * C::kP); };
  const uint32_t bar0 = sb + C::OFF_BAR;
  auto Q_FULL = [&](int s) { return bar0 + 8u * (uint32_t)s; };
  auto Q_EMPTY = [&](int s) { return bar0 + 16u + 8u * (uint32_t)s; };
  const uint32_t KV_FULL = bar0 + 32, ITEM_DONE = bar0 + 40, ACC_FREE = bar0 + 48;
  auto SDP_FULL = [&](int w) { return bar0 + 56u + 8u * (uint32_t)w; };
  auto PDS_READY = [&](int w) { return bar0 + 72u + 8u * (uint32_t)w; };
  auto PDS_FREE = [&](int w) { return bar0 + 88u + 8u * (uint32_t)w; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem_raw + C::OFF_SLOT);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto wait = [&](uint32_t bar, uint32_t phase) {
    mbar_wait(bar, phase, p.spin_ns, p.err, p.err + 1);
  };
  const int items = p.head[0];

  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(Q_FULL(s), 1);
      mbar_init(Q_EMPTY(s), 1);
      mbar_init(SDP_FULL(s), 1);
      mbar_init(PDS_READY(s), 128);
      mbar_init(PDS_FREE(s), 1);
    }
    mbar_init(KV_FULL, 1);
    mbar_init(ITEM_DONE, 1);
    mbar_init(ACC_FREE, 256);
    fence_mbar_init();
  }
  // rows G*T to 127 of a stage are never loaded, but the products sum over all 128 rows
  for (int x = threadIdx.x; x < (kTileRows - p.G * p.T) * 8 * (4 * D / 64); x += C::kThreads) {
    const int c = x & 7, rest = x >> 3, atom = rest % (4 * D / 64);
    const int row = p.G * p.T + rest / (4 * D / 64);
    st_shared_v4(sb + C::OFF_QDO + atom * 16384 + row * 128 + c * 16, 0, 0, 0, 0);
  }
  fence_proxy_async_smem();
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
    int it = 0, k = 0;
    for (int i = blockIdx.x; i < items; i += gridDim.x, ++k) {
      const int4 w = p.item[i];
      const int bh = w.x / p.nu, u = w.x - bh * p.nu, b = bh / p.Hkv, hk = bh - b * p.Hkv;
      const int2* entry = p.entry + (long long)w.x * p.NT;
      if (k > 0) wait(ITEM_DONE, (uint32_t)((k - 1) & 1));  // K and V are read to the end
      mbar_expect_tx(KV_FULL, 2 * C::kKV);
#pragma unroll
      for (int cb = 0; cb < D / 64; ++cb) {
        tma_load_4d(sK + cb * 8192, &tmK, cb * 64, u * kUnit, hk, b, KV_FULL);
        tma_load_4d(sV + cb * 8192, &tmV, cb * 64, u * kUnit, hk, b, KV_FULL);
      }
      int tile = entry[w.y].x;
      for (int e = w.y; e < w.z; ++e, ++it) {
        const int s = it & 1;
        const int next = e + 1 < w.z ? entry[e + 1].x : 0;
        if (it >= 2) wait(Q_EMPTY(s), (uint32_t)(((it >> 1) - 1) & 1));
        mbar_expect_tx(Q_FULL(s), (uint32_t)(2 * p.G * p.T * D * 2));
#pragma unroll
        for (int cb = 0; cb < D / 64; ++cb) {
          tma_load_4d(sQ(s) + cb * 16384, &tmQ, cb * 64, tile * p.T, hk * p.G, b, Q_FULL(s));
          tma_load_4d(sDO(s) + cb * 16384, &tmDO, cb * 64, tile * p.T, hk * p.G, b, Q_FULL(s));
        }
        tile = next;
      }
    }
    // no load may land after the CTA has gone, not even when a wait ran out
    if (k > 0) mbar_wait_drain(KV_FULL, (uint32_t)((k - 1) & 1), p.spin_ns, p.err, p.err + 1);
    for (int j = max(0, it - 2); j < it; ++j)
      mbar_wait_drain(Q_FULL(j & 1), (uint32_t)((j >> 1) & 1), p.spin_ns, p.err, p.err + 1);
  } else if (warp == 1 && lane == 0) {
    // ---------------------------------------------------------------- MMA issuer
    constexpr uint32_t ID_S = idesc_bf16_f32(128, kUnit, 0, 0);
    constexpr uint32_t ID_T = idesc_bf16_f32(128, kUnit, 1, 1);  // dV^T, dK^T
    const uint32_t hi = sdesc_hi(1024);
    const uint32_t kK = sdesc_lo(sK, 16), kV = sdesc_lo(sV, 16);
    int it = 0, k = 0;
    auto issue_acc = [&](int j, bool first) {
      const int s = j & 1;
      const uint32_t aV = sdesc_lo(sDO(s), 16384);
      const uint32_t aK = D == 128 ? sdesc_lo(sQ(s), 16384) : aV;
      const uint32_t bP = sdesc_lo(sP(s), 16384), bS = sdesc_lo(sP(s) + C::kP, 16384);
      wait(PDS_READY(s), (uint32_t)((j >> 1) & 1));
      tc_fence_after();
#pragma unroll
      for (int kk = 0; kk < 8; ++kk)
        tc_mma_ss_w(tmem + C::TM_DV, aV + kk * 128, bP + kk * 128, hi, ID_T,
                    (!first || kk > 0) ? 1u : 0u);
#pragma unroll
      for (int kk = 0; kk < 8; ++kk)
        tc_mma_ss_w(tmem + C::TM_DK, aK + kk * 128, bS + kk * 128, hi, ID_T,
                    (!first || kk > 0) ? 1u : 0u);
      tc_commit(PDS_FREE(s));
      tc_commit(Q_EMPTY(s));
    };
    for (int i = blockIdx.x; i < items; i += gridDim.x, ++k) {
      const int4 w = p.item[i];
      wait(KV_FULL, (uint32_t)(k & 1));
      const int it0 = it;
      for (int e = w.y; e < w.z; ++e, ++it) {
        const int s = it & 1;
        const uint32_t kQ = sdesc_lo(sQ(s), 16), kDO = sdesc_lo(sDO(s), 16);
        const uint32_t tS = tmem + C::TM_S + 128u * (uint32_t)s;
        wait(Q_FULL(s), (uint32_t)((it >> 1) & 1));
        tc_fence_after();
        // S and dP of entry it - 2 were read before its P and dS were ready
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
        tc_commit(SDP_FULL(s));
        if (it > it0) {
          // the accumulators are written first here: the last item's must have been read
          if (it == it0 + 1 && k > 0) {
            wait(ACC_FREE, (uint32_t)((k - 1) & 1));
            tc_fence_after();
          }
          issue_acc(it - 1, it - 1 == it0);
        }
      }
      if (it == it0 + 1 && k > 0) {
        wait(ACC_FREE, (uint32_t)((k - 1) & 1));
        tc_fence_after();
      }
      issue_acc(it - 1, it - 1 == it0);
      tc_commit(ITEM_DONE);
    }
    if (k > 0)
      mbar_wait_drain(ITEM_DONE, (uint32_t)((k - 1) & 1), p.spin_ns, p.err, p.err + 1);
  } else if (warp >= 2) {
    // ---------------------------------------------------------------- softmax gradient
    const int wg = (warp - 2) >> 2, quarter = warp & 3;
    const int r = quarter * 32 + lane;
    const int g = r / p.T, t = r - g * p.T;
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const uint32_t tS = tmem + lane_off + C::TM_S + 128u * (uint32_t)wg;
    const uint32_t rowP = sP(wg) + r * 128, rowS = rowP + C::kP;
    const float sl2 = p.scale_log2;
    const int bit = t & 31, wsel = min(t >> 5, p.W - 1);
    int it = 0, k = 0;
    for (int i = blockIdx.x; i < items; i += gridDim.x, ++k) {
      const int4 w = p.item[i];
      const int bh = w.x / p.nu, u = w.x - bh * p.nu, b = bh / p.Hkv, hk = bh - b * p.Hkv;
      const int2* entry = p.entry + (long long)w.x * p.NT;
      const int base = u * kUnit;
      const int kvlen = p.plan.len[b];
      const long long start = p.plan.start[b];
      const long long row0 = ((long long)b * p.H + hk * p.G + g) * p.Sq;
      // what this thread's row of entry e needs, fetched one entry of its own ahead
      float lse2 = 0.f, delta = 0.f;
      int vis = 0;
      auto fetch = [&](int e, float& f_lse, float& f_delta, int& f_vis) {
        f_lse = f_delta = 0.f;
        f_vis = 0;
        if (e >= w.z) return;
        const int2 at = entry[e];
        const int token = at.x * p.T + t;
        if (g >= p.G || token >= p.Sq) return;
        const long long gt = (long long)bh * p.NT + at.x;
        const uint32_t word = p.plan.mask[(gt * p.U + at.y) * p.W + wsel];
        f_lse = p.lse[row0 + token] * 1.4426950408889634f;
        f_delta = p.delta[row0 + token];
        const long long limit = p.causal ? min((long long)kvlen, max(start + token + 1, 0ll))
                                         : (long long)kvlen;
        f_vis = ((word >> bit) & 1u) ? (int)(limit - base) : 0;
      };
      int e = w.y + ((it ^ wg) & 1);  // this warpgroup takes the steps of its own parity
      fetch(e, lse2, delta, vis);
      for (; e < w.z; e += 2) {
        const int step = it + (e - w.y);
        float n_lse, n_delta;
        int n_vis;
        fetch(e + 2, n_lse, n_delta, n_vis);
        wait(SDP_FULL(wg), (uint32_t)((step >> 1) & 1));
        tc_fence_after();
        if (step >= 2) wait(PDS_FREE(wg), (uint32_t)(((step >> 1) - 1) & 1));
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t sv[32], dp[32];
          tmem_ld32x2(tS + 32 * c, tS + 64 + 32 * c, sv, dp);
#pragma unroll
          for (int c4 = 0; c4 < 4; ++c4) {
            uint32_t pp[4], ds[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const int key = 8 * c4 + 2 * x;
              float p0 = 0.f, p1 = 0.f, d0 = 0.f, d1 = 0.f;
              // selected, not multiplied: S and dP of a masked key may be anything
              if (32 * c + key < vis) {
                p0 = ex2_approx(__uint_as_float(sv[key]) * sl2 - lse2);
                d0 = p0 * (__uint_as_float(dp[key]) - delta);
              }
              if (32 * c + key + 1 < vis) {
                p1 = ex2_approx(__uint_as_float(sv[key + 1]) * sl2 - lse2);
                d1 = p1 * (__uint_as_float(dp[key + 1]) - delta);
              }
              pp[x] = pack_bf16x2(p0, p1);
              ds[x] = pack_bf16x2(d0, d1);
            }
            const uint32_t off = (uint32_t)(((4 * c + c4) ^ (r & 7)) << 4);
            st_shared_v4(rowP + off, pp[0], pp[1], pp[2], pp[3]);
            st_shared_v4(rowS + off, ds[0], ds[1], ds[2], ds[3]);
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        mbar_arrive(PDS_READY(wg));
        lse2 = n_lse, delta = n_delta, vis = n_vis;
      }
      it += w.z - w.y;
      // epilogue: warpgroup 0 writes dV, warpgroup 1 dK; lane = head dimension, column = key
      wait(ITEM_DONE, (uint32_t)(k & 1));
      tc_fence_after();
      uint32_t acc[2][32];
      const uint32_t ta = tmem + lane_off + (wg == 0 ? C::TM_DV : C::TM_DK);
      tmem_ld32x2(ta, ta + 32, acc[0], acc[1]);
      tc_fence_before();
      mbar_arrive(ACC_FREE);
      // at D = 64 dV^T is in lanes 0-63 of its product, dK^T in lanes 64-127 of its own
      const int d = D == 128 ? r : r - (wg == 0 ? 0 : 64);
      if (d >= 0 && d < D) {
        const float f = wg == 0 ? 1.f : p.scale;
        if (w.w >= 0) {
          float* out = p.part + ((long long)w.w * 2 + (wg == 0 ? 1 : 0)) * kUnit * D + d;
#pragma unroll
          for (int key = 0; key < kUnit; ++key)
            out[key * D] = __uint_as_float(acc[key >> 5][key & 31]) * f;
        } else {
          __nv_bfloat16* out = (wg == 0 ? p.dv : p.dk) + ((long long)bh * p.Sk + base) * D + d;
          const int keys = min(kUnit, p.Sk - base);
#pragma unroll
          for (int key = 0; key < kUnit; ++key)
            if (key < keys)
              out[key * D] = __float2bfloat16_rn(__uint_as_float(acc[key >> 5][key & 31]) * f);
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// Units that no tile lists get zeros; the partials of cut units are added in ascending order.
struct FinishParams {
  const int* slot0;
  const int* count;
  const int* head;
  const float* part;
  __nv_bfloat16 *dk, *dv;
  int Sk, D, nu;
};
__global__ void __launch_bounds__(256) dash_sparse_finish_kernel(const FinishParams p) {
  const int gu = blockIdx.x;
  const int s0 = p.slot0[gu];
  if (s0 == -1) return;
  const int bh = gu / p.nu, base = (gu - bh * p.nu) * kUnit;
  const int n = min(kUnit, p.Sk - base) * p.D;
  const int parts = s0 < 0 ? 0 : (p.count[gu] + p.head[1] - 1) / p.head[1];
  const long long at = ((long long)bh * p.Sk + base) * p.D;
  for (int x = threadIdx.x * 2; x < n; x += 512) {
    float2 a = make_float2(0.f, 0.f), c = a;
    for (int k = 0; k < parts; ++k) {
      const float* src = p.part + (long long)(s0 + k) * 2 * kUnit * p.D + x;
      const float2 y = *reinterpret_cast<const float2*>(src);
      const float2 z = *reinterpret_cast<const float2*>(src + kUnit * p.D);
      a.x += y.x, a.y += y.y, c.x += z.x, c.y += z.y;
    }
    *reinterpret_cast<uint32_t*>(p.dk + at + x) = dev::pack_bf16x2(a.x, a.y);
    *reinterpret_cast<uint32_t*>(p.dv + at + x) = dev::pack_bf16x2(c.x, c.y);
  }
}

}  // namespace dash
