// Block-sparse attention of single tokens for sm_100a: no plan, one launch.
//
// A cluster of CTAs takes one token of one K/V head with up to 16 of its query heads.  Its
// warps take 16-key chunks of the picked blocks in turn, each with a running maximum m, a row
// sum l and an output of its own:
//
//   S = Q K^T,  P = 2^(s S - m),  O += P V,  l += rowsum P      (s = scale log2 e)
//
// and the parts are joined at the end, those of a CTA through its shared memory, those of
// the cluster through each other's: O = sum_w 2^(m_w - m) O_w / sum_w 2^(m_w - m) l_w, in the
// order of w.  Bound by reading the picked K and V once: the products (mma.sync, 16 rows) run
// under the loads, three chunks of which each warp keeps in flight (16-byte cp.async).
//
// Measured, 16 picks of 64 keys, 32 heads, 8 K/V heads, D = 128: one token 8.7 us (latency: the
// picks, the keys, the joins), 64 tokens 53 us, 268 MB at 5.1 TB/s.  Two stages took 65, four
// (one CTA an SM) 75.
#pragma once
#include "block_select.cuh"

namespace dash {

constexpr int kTokenWarps = 4, kTokenKeys = 16, kTokenStages = 3;
constexpr int kTokenTopk = 1024, kTokenBlocks = 65536;  // what the list and its bitmap hold

struct SparseTokenParams {
  const __nv_bfloat16 *q, *k, *v;
  long long qb, qh, qs, kb, kh, ks, vb, vh, vs;  // strides in elements
  const int* idx;
  const int* kv_len;
  const int* q_start;
  __nv_bfloat16* o;
  float* lse;
  int H, Hkv, G, RG, Sq, Sk, block, nb, topk, causal;  // RG: groups of 16 heads
  float scale_log2;
};

template <int D>
struct SparseTokenCfg {
  static constexpr int kThreads = kTokenWarps * 32;
  static constexpr int kChunk = kTokenKeys * D * 2;           // of K or of V
  static constexpr int kWarp = kTokenStages * 2 * kChunk;     // a warp's stages
  static constexpr int OFF_ML = kTokenWarps * kWarp;          // m and l of 16 rows, per warp and joined
  static constexpr int OFF_LIST = OFF_ML + (kTokenWarps + 1) * 16 * 8;
  static int smem(int topk, int nb) { return OFF_LIST + topk * 4 + (topk > 32 ? (nb + 31) / 32 * 4 : 0); }
  static_assert(16 * D * 4 <= kWarp, "a warp's output lies over its stages");
};

__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ float ld_shared_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

template <int D>
__global__ void __launch_bounds__(128)
    dash_sparse_token_kernel(const __grid_constant__ SparseTokenParams p) {
  using namespace dev;
  using C = SparseTokenCfg<D>;
  constexpr int CH = D / 8;  // 16-byte pieces of a row
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ int list_n;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int CS = (int)cluster_nctarank(), rank = (int)cluster_ctarank();
  const int unit = (int)blockIdx.x / CS;  // ((b Hkv + hk) Sq + i) RG + group of heads
  const int rg = unit % p.RG, tok = unit / p.RG, i = tok % p.Sq, bh = tok / p.Sq;
  const int b = bh / p.Hkv, hk = bh - b * p.Hkv;
  const int heads = min(16, p.G - rg * 16), h0 = hk * p.G + rg * 16;
  int* const list = reinterpret_cast<int*>(smem_raw + C::OFF_LIST);
  const int len = p.kv_len ? min(max(p.kv_len[b], 0), p.Sk) : p.Sk;
  const long long pos = (long long)(p.q_start ? p.q_start[b] : p.Sk - p.Sq) + i;
  const int limit = p.causal ? (int)min((long long)len, max(pos + 1, 0ll)) : len;

  // ---- Q as MMA operand: row lane/4 (+8), columns 2 (lane%4) (+8); rows past the heads are 0
  uint32_t qa[D / 16][4];
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const int row = half * 8 + (lane >> 2);
    const __nv_bfloat16* q = p.q + b * p.qb + (long long)(h0 + min(row, heads - 1)) * p.qh + i * p.qs +
                             (lane & 3) * 2;
#pragma unroll
    for (int c = 0; c < D / 8; ++c) {
      const uint32_t w = *reinterpret_cast<const uint32_t*>(q + c * 8);
      qa[c >> 1][(c & 1) * 2 + half] = row < heads ? w : 0u;
    }
  }

  // ---- the picked blocks that are seen, each once, in the order of their first mention
  if (warp == 0) {
    uint32_t* const seen = reinterpret_cast<uint32_t*>(list + p.topk);
    if (p.topk > 32)
      for (int x = lane; x < (p.nb + 31) / 32; x += 32) seen[x] = 0u;
    __syncwarp();
    const int* idx = p.idx + ((long long)bh * p.Sq + i) * p.topk;
    int n = 0;
    for (int x0 = 0; x0 < p.topk; x0 += 32) {
      const int e = x0 + lane < p.topk ? idx[x0 + lane] : -1;
      bool on = e >= 0 && e < p.nb && (long long)e * p.block < limit;
      const unsigned same = __match_any_sync(0xffffffffu, on ? e : -1 - lane);
      on = on && (same & ((1u << lane) - 1u)) == 0u;
      if (p.topk > 32) {
        if (on) on = ((seen[e >> 5] >> (e & 31)) & 1u) == 0u;
        __syncwarp();
        if (on) atomicOr(&seen[e >> 5], 1u << (e & 31));
        __syncwarp();
      }
      const unsigned m = __ballot_sync(0xffffffffu, on);
      if (on) list[n + __popc(m & ((1u << lane) - 1u))] = e;
      n += __popc(m);
    }
    if (lane == 0) list_n = n;
  }
  __syncthreads();

  // ---- chunks of 16 keys: warp w of the cluster takes every (4 CS)-th
  const int per = p.block / kTokenKeys, chunks = list_n * per, step = CS * kTokenWarps;
  const uint32_t base = smem_u32(smem_raw) + warp * C::kWarp;
  const __nv_bfloat16* const k = p.k + b * p.kb + hk * p.kh;
  const __nv_bfloat16* const v = p.v + b * p.vb + hk * p.vh;
  const int piece = lane % CH, sub = lane / CH;
  auto first_key = [&](int c) { return list[c / per] * p.block + (c % per) * kTokenKeys; };
  auto load = [&](int c, int stage) {
    if (c < chunks) {
      const int key0 = first_key(c);
      const uint32_t dst = base + stage * 2 * C::kChunk;
#pragma unroll
      for (int r0 = 0; r0 < kTokenKeys; r0 += 32 / CH) {
        const int r = r0 + sub;
        // rows past the sequence are zeros: they may hold anything, and 0 * NaN would reach O
        const uint32_t on = key0 + r < len ? 16u : 0u;
        const long long key = min(key0 + r, p.Sk - 1);
        const uint32_t at = dst + r * (D * 2) + ((piece ^ (r & 7)) << 4);
        cp_async16(at, k + key * p.ks + piece * 8, on);
        cp_async16(at + C::kChunk, v + key * p.vs + piece * 8, on);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  float acc[D / 8][4];
#pragma unroll
  for (int x = 0; x < D / 8; ++x)
#pragma unroll
    for (int y = 0; y < 4; ++y) acc[x][y] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};  // rows lane/4 and lane/4 + 8
  int c = rank * kTokenWarps + warp;
#pragma unroll
  for (int s = 0; s < kTokenStages - 1; ++s) load(c + s * step, s);
  int stage = 0, ahead = kTokenStages - 1;
  for (; c < chunks; c += step) {
    load(c + (kTokenStages - 1) * step, ahead);
    ahead = ahead + 1 == kTokenStages ? 0 : ahead + 1;
    asm volatile("cp.async.wait_group %0;" ::"n"(kTokenStages - 1) : "memory");
    __syncwarp();
    const uint32_t sK = base + stage * 2 * C::kChunk, sV = sK + C::kChunk;
    const int vis = limit - first_key(c);  // keys of the chunk below it are attended to
    float sc[2][4] = {};
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      // keys 0-7, columns 0-7; keys 0-7, columns 8-15; keys 8-15 likewise
      const int row = (lane & 7) + ((lane >> 4) << 3), col = kk * 2 + ((lane >> 3) & 1);
      uint32_t w[4];
      ldmatrix_x4(sK + row * (D * 2) + ((col ^ (row & 7)) << 4), w);
      mma_bf16(sc[0], qa[kk], w[0], w[1]);
      mma_bf16(sc[1], qa[kk], w[2], w[3]);
    }
    float f[2];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      float top = -INFINITY;
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float& s = sc[t][half * 2 + e];
          s = t * 8 + (lane & 3) * 2 + e < vis ? s * p.scale_log2 : -INFINITY;
          top = fmaxf(top, s);
        }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const float mn = fmaxf(m[half], top);
      f[half] = mn == -INFINITY ? 1.f : ex2_approx(m[half] - mn);
      m[half] = mn;
      l[half] *= f[half];
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float& s = sc[t][half * 2 + e];
          s = s == -INFINITY ? 0.f : ex2_approx(s - mn);
          l[half] += s;
        }
    }
    // P is rounded once to bf16 for the product; l sums the fp32 values
    const uint32_t pa[4] = {pack_bf16x2(sc[0][0], sc[0][1]), pack_bf16x2(sc[0][2], sc[0][3]),
                            pack_bf16x2(sc[1][0], sc[1][1]), pack_bf16x2(sc[1][2], sc[1][3])};
    if (__any_sync(0xffffffffu, f[0] != 1.f || f[1] != 1.f))
#pragma unroll
      for (int x = 0; x < D / 8; ++x) {
        acc[x][0] *= f[0], acc[x][1] *= f[0];
        acc[x][2] *= f[1], acc[x][3] *= f[1];
      }
#pragma unroll
    for (int x = 0; x < D / 16; ++x) {
      // keys 0-7, columns 0-7; keys 8-15, columns 0-7; columns 8-15 likewise
      const int row = (lane & 7) + (((lane >> 3) & 1) << 3), col = x * 2 + (lane >> 4);
      uint32_t w[4];
      ldmatrix_x4_trans(sV + row * (D * 2) + ((col ^ (row & 7)) << 4), w);
      mma_bf16(acc[2 * x], pa, w[0], w[1]);
      mma_bf16(acc[2 * x + 1], pa, w[2], w[3]);
    }
    __syncwarp();  // the stage is read by all lanes before it is filled again
    stage = stage + 1 == kTokenStages ? 0 : stage + 1;
  }
  cp_async_wait_all();
  __syncwarp();

  // ---- the warp's part to shared memory, over its stages
  float2* const ml = reinterpret_cast<float2*>(smem_raw + C::OFF_ML);  // [warps + joined][16]
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    l[half] += __shfl_xor_sync(0xffffffffu, l[half], 1);
    l[half] += __shfl_xor_sync(0xffffffffu, l[half], 2);
    const int row = half * 8 + (lane >> 2);
    if ((lane & 3) == 0) ml[warp * 16 + row] = make_float2(m[half], l[half]);
    float* out = reinterpret_cast<float*>(smem_raw + warp * C::kWarp) + row * D + (lane & 3) * 2;
#pragma unroll
    for (int x = 0; x < D / 8; ++x)
      *reinterpret_cast<float2*>(out + x * 8) = make_float2(acc[x][2 * half], acc[x][2 * half + 1]);
  }
  __syncthreads();
  // weights 2^(m_w - m); a part without keys (m = -inf) weighs nothing, a NaN stays visible
  auto weight = [](float mw, float top) { return mw == -INFINITY ? 0.f : ex2_approx(mw - top); };
  // ---- join the CTA's warps, into the first warp's place
  for (int x = tid; x < heads * D; x += C::kThreads) {
    const int row = x / D;
    float top = -INFINITY, sum = 0.f, o = 0.f;
    bool bad = false;
#pragma unroll
    for (int w = 0; w < kTokenWarps; ++w) {
      top = fmaxf(top, ml[w * 16 + row].x);
      bad |= ml[w * 16 + row].y != ml[w * 16 + row].y;
    }
    if (top != -INFINITY || bad)
#pragma unroll
      for (int w = 0; w < kTokenWarps; ++w) {
        const float f = bad ? 1.f : weight(ml[w * 16 + row].x, top);
        sum += f * ml[w * 16 + row].y;
        o += f * reinterpret_cast<const float*>(smem_raw + w * C::kWarp)[x];
      }
    reinterpret_cast<float*>(smem_raw)[x] = o;
    if (x % D == 0) ml[kTokenWarps * 16 + row] = make_float2(top, sum);
  }
  // ---- join the cluster's CTAs; each writes a share of the output
  if (CS > 1) cluster_sync_all();
  else __syncthreads();
  const uint32_t s0 = smem_u32(smem_raw), sml = s0 + C::OFF_ML + kTokenWarps * 16 * 8;
  const long long row_o = ((long long)b * p.H + h0) * p.Sq + i;
  for (int x = rank * C::kThreads + tid; x < heads * D; x += CS * C::kThreads) {
    const int row = x / D;
    float top = -INFINITY, sum = 0.f, o = 0.f;
    bool bad = false;
    for (int r = 0; r < CS; ++r) {
      top = fmaxf(top, ld_shared_cluster_f32(mapa_shared(sml + row * 8, r)));
      const float lr = ld_shared_cluster_f32(mapa_shared(sml + row * 8 + 4, r));
      bad |= lr != lr;
    }
    if (top != -INFINITY || bad)
      for (int r = 0; r < CS; ++r) {
        const float f =
            bad ? 1.f : weight(ld_shared_cluster_f32(mapa_shared(sml + row * 8, r)), top);
        sum += f * ld_shared_cluster_f32(mapa_shared(sml + row * 8 + 4, r));
        o += f * ld_shared_cluster_f32(mapa_shared(s0 + x * 4, r));
      }
    // a row that attended to nothing gets O = 0 and LSE = -inf
    p.o[(row_o + (long long)row * p.Sq) * D + x % D] =
        __float2bfloat16_rn(sum == 0.f ? 0.f : o / sum);
    if (x % D == 0)
      p.lse[row_o + (long long)row * p.Sq] =
          sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.69314718055994531f;
  }
  if (CS > 1) cluster_sync_all();  // a CTA's shared memory outlives its readers
}

}  // namespace dash
