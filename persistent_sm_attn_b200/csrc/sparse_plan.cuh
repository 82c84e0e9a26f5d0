// Tile plans of block-sparse attention.
//
// A query tile is T tokens of one K/V head with all G query heads that share it, T =
// floor(128 / G), row r of the tile being head r / T and token r mod T.  Keys are walked in
// units of 64.  The plan holds for each tile the units that any of its tokens selected and
// may see, ascending, each with a mask of the tokens that did: a block picked by several
// tokens, or twice by one, is visited once.
#pragma once
#include <cstdint>

namespace dash {

constexpr int kUnit = 64;      // keys per unit
constexpr int kTileRows = 128;

// Shapes of a plan and where its parts lie (offsets in bytes, multiples of 16).
struct PlanShape {
  int B, H, Hkv, Sq, Sk, block, topk, causal;
  int G, T, W;        // query heads per K/V head, tokens per tile, mask words
  int NT, nu, U, NW;  // tiles per K/V head, units, units a tile can list, presence words
  long long off_len, off_start, off_count, off_unit, off_mask, off_pres, off_pre, bytes;
};

// A device pointer set of a plan in use.
struct PlanView {
  const int* len;       // [B] keys of each batch entry
  const int* start;     // [B] position of query 0
  const int* count;     // [B*Hkv*NT] listed units
  const int* unit;      // [B*Hkv*NT][U]
  const uint32_t* mask; // [B*Hkv*NT][U][W]
  const uint32_t* pres; // [B*Hkv*NT][NW] a bit per unit
  const int* pre;       // [B*Hkv*NT][NW] listed units before the word
};

struct PlanParams {
  PlanShape s;
  const int* idx;
  const int* kv_len;
  const int* q_start;
  int *len, *start, *count, *unit, *pre;
  uint32_t *mask, *pres;
};

// One CTA per tile: the tokens' picks are OR-ed into a [nu][W] mask in shared memory (an
// OR does not depend on its order), then the non-empty units are numbered by ballots.  1024
// tiles of 32 tokens with 16 picks: 6 us, of a launch's 3 or so.
__global__ void __launch_bounds__(128) dash_sparse_plan_kernel(const __grid_constant__ PlanParams p) {
  extern __shared__ uint32_t plan_mask[];  // [nu][W]
  __shared__ int warp_n[4];
  const PlanShape& s = p.s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const long long tile = blockIdx.x;
  const int bh = (int)(tile / s.NT), t0 = (int)(tile % s.NT) * s.T;
  const int b = bh / s.Hkv;
  const int len = p.kv_len ? min(max(p.kv_len[b], 0), s.Sk) : s.Sk;
  const int pos0 = p.q_start ? p.q_start[b] : s.Sk - s.Sq;
  if (tile == (long long)b * s.Hkv * s.NT && tid == 0) {
    p.len[b] = len;
    p.start[b] = pos0;
  }
  for (int x = tid; x < s.nu * s.W; x += 128) plan_mask[x] = 0u;
  __syncthreads();
  const int nt = min(s.T, s.Sq - t0), nb = (s.Sk + s.block - 1) / s.block, per = s.block / kUnit;
  const int* idx = p.idx + ((long long)bh * s.Sq + t0) * s.topk;
  for (int x = tid; x < nt * s.topk; x += 128) {
    const int t = x / s.topk, e = idx[x];
    if (e < 0 || e >= nb) continue;  // unused places
    const long long pos = (long long)pos0 + t0 + t;
    const long long limit = s.causal ? min((long long)len, pos + 1) : (long long)len;
    for (int u = e * per; u < (e + 1) * per && (long long)u * kUnit < limit; ++u)
      atomicOr(&plan_mask[u * s.W + (t >> 5)], 1u << (t & 31));
  }
  __syncthreads();
  int done = 0;
  for (int u0 = 0; u0 < s.nu; u0 += 128) {
    const int u = u0 + tid;
    uint32_t any = 0;
    if (u < s.nu)
      for (int w = 0; w < s.W; ++w) any |= plan_mask[u * s.W + w];
    const unsigned m = __ballot_sync(0xffffffffu, any != 0);
    if (lane == 0) warp_n[warp] = __popc(m);
    __syncthreads();
    int before = done;
    for (int w = 0; w < warp; ++w) before += warp_n[w];
    if (lane == 0 && u < s.NW * 32) {
      p.pres[tile * s.NW + (u >> 5)] = m;
      p.pre[tile * s.NW + (u >> 5)] = before;
    }
    if (any) {
      const long long at = tile * s.U + before + __popc(m & ((1u << lane) - 1u));
      p.unit[at] = u;
      for (int w = 0; w < s.W; ++w) p.mask[at * s.W + w] = plan_mask[u * s.W + w];
    }
    done += warp_n[0] + warp_n[1] + warp_n[2] + warp_n[3];
    __syncthreads();
  }
  if (tid == 0) p.count[tile] = done;
}

}  // namespace dash
