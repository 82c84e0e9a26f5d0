// Block selection: means of key blocks, and for each query the blocks with the best scores.
//
//   mean[b,hk,j]  = (1 / n_j) sum of the n_j keys of block j below kv_len[b]      (fp32)
//   score(i, j)   = (sum of the group's query heads q[b,h,i]) . mean[b,hk,j]
//
// A query sees the blocks whose first key lies below its limit, min(kv_len, position + 1
// if causal).  The first `sink` and the last `local` of them are always picked, the other
// places go to the highest scores, equal scores to the lowest block.  Which blocks are
// picked must not depend on the order of a sum, so sums and scores are held in fp64: a sum
// of bf16 keys is then exact unless their exponents differ by over 40, and two scores
// closer than fp64 can tell apart do not occur but for equal blocks, which tie exactly.
#pragma once
#include <cuda_bf16.h>
#include <cstdint>

namespace dash {

struct MeansParams {
  const __nv_bfloat16* k;
  long long sb, sh, ss;  // strides of k in elements
  float* means;          // [B, Hkv, nb, D]
  const int* kv_len;     // [B] or null
  const int* start;      // [B] or null: only blocks that hold positions >= start[b]
  int Hkv, Sk, D, block, nb;
};

// One CTA per (block, head): D/8 lanes side by side read a key (16 bytes a lane), the
// 128 threads' rows of keys are added in shared memory.  Bound by reading K.
__global__ void __launch_bounds__(128) dash_block_means_kernel(const MeansParams p) {
  __shared__ double sum[128 * 8];
  const int bh = blockIdx.y, b = bh / p.Hkv, h = bh % p.Hkv;
  const int len = p.kv_len ? min(max(p.kv_len[b], 0), p.Sk) : p.Sk;
  // with a start, the blocks from its own to the last that has keys; the others stay as they are
  const int j0 = p.start ? max(p.start[b], 0) / p.block : 0;
  const int j1 = p.start ? (len + p.block - 1) / p.block : p.nb;
  for (int j = j0 + blockIdx.x; j < j1; j += gridDim.x) {
  const int first = j * p.block;
  const int n = min(p.block, len - first);  // keys of the block that exist (may be <= 0)
  const int lanes = p.D / 8, rows = 128 / lanes;
  const int lane = threadIdx.x % lanes, row = threadIdx.x / lanes;
  const __nv_bfloat16* src = p.k + b * p.sb + h * p.sh + (long long)first * p.ss + lane * 8;
  double acc[8] = {};
  if (row < rows)
    for (int t = row; t < n; t += rows) {
      const uint4 w = *reinterpret_cast<const uint4*>(src + t * p.ss);
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int c = 0; c < 8; ++c)
        acc[c] += (double)__uint_as_float((c & 1) ? (u[c >> 1] & 0xffff0000u) : (u[c >> 1] << 16));
    }
#pragma unroll
  for (int c = 0; c < 8; ++c) sum[threadIdx.x * 8 + c] = acc[c];
  __syncthreads();
  float* dst = p.means + ((long long)bh * p.nb + j) * p.D;
  for (int d = threadIdx.x; d < p.D; d += 128) {
    double s = 0.0;
    for (int r = 0; r < rows; ++r) s += sum[(r * lanes + d / 8) * 8 + d % 8];
    dst[d] = n > 0 ? (float)(s / (double)n) : 0.f;
  }
  __syncthreads();
  }
}

struct SelectParams {
  const __nv_bfloat16* q;
  long long sb, sh, ss;
  const float* means;
  int* idx;  // [B, Hkv, Sq, topk]
  const int* kv_len;
  const int* q_start;
  int Hkv, G, Sq, Sk, block, nb, topk, causal, sink, local;
};

// Monotone map of a double to an unsigned integer (NaN ranks below everything).
__device__ __forceinline__ unsigned long long order_key(double x) {
  if (x != x) return 0ull;
  const long long b = __double_as_longlong(x == 0.0 ? 0.0 : x);  // -0 ties with 0
  return b < 0 ? ~(unsigned long long)b : (unsigned long long)b | 0x8000000000000000ull;
}

// One CTA per QT queries of a K/V head; a warp per query at a time.  Scores of the visible
// blocks go to shared memory in fp64; the picks are then made one at a time by a warp-wide
// maximum over (score, -block).
template <int D, int QT>
__global__ void __launch_bounds__(128) dash_block_select_kernel(const SelectParams p) {
  extern __shared__ __align__(16) unsigned char select_smem[];
  double* qs = reinterpret_cast<double*>(select_smem);             // [QT][D]
  unsigned long long* keys = reinterpret_cast<unsigned long long*>(qs + QT * D);  // [QT][nb]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int bh = blockIdx.y, b = bh / p.Hkv, hk = bh % p.Hkv;
  const int i0 = blockIdx.x * QT;
  const int len = p.kv_len ? min(max(p.kv_len[b], 0), p.Sk) : p.Sk;
  const int pos0 = p.q_start ? p.q_start[b] : p.Sk - p.Sq;
  for (int x = threadIdx.x; x < QT * D; x += 128) {
    const int i = i0 + x / D;
    double s = 0.0;
    if (i < p.Sq)
      for (int g = 0; g < p.G; ++g)
        s += (double)__bfloat162float(
            p.q[b * p.sb + (long long)(hk * p.G + g) * p.sh + (long long)i * p.ss + x % D]);
    qs[x] = s;
  }
  __syncthreads();
  for (int r = warp; r < QT; r += 4) {
    const int i = i0 + r;
    if (i >= p.Sq) break;
    const long long pos = (long long)pos0 + i;
    const long long limit = p.causal ? min((long long)len, pos + 1) : (long long)len;
    const int nvis = limit <= 0 ? 0 : (int)((limit + p.block - 1) / p.block);
    unsigned long long* key = keys + (size_t)r * p.nb;
    for (int j = lane; j < nvis; j += 32) {
      const float* m = p.means + ((long long)bh * p.nb + j) * D;
      double s = 0.0;
      for (int d = 0; d < D; ++d) s += qs[r * D + d] * (double)m[d];
      key[j] = (j < p.sink || j >= nvis - p.local) ? ~0ull : order_key(s);
    }
    __syncwarp();
    const int n = min(p.topk, nvis);
    int* out = p.idx + ((long long)bh * p.Sq + i) * p.topk;
    // n picks, marked by key 0 with their bit kept in the low end of the output order below
    for (int pick = 0; pick < n; ++pick) {
      unsigned long long best = 0;
      int at = 0x7fffffff;
      for (int j = lane; j < nvis; j += 32) {
        const unsigned long long v = key[j];
        if (v != 1ull && (v > best || at == 0x7fffffff)) {
          best = v;
          at = j;
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const unsigned long long ob = __shfl_xor_sync(0xffffffffu, best, o);
        const int oa = __shfl_xor_sync(0xffffffffu, at, o);
        if (oa != 0x7fffffff && (at == 0x7fffffff || ob > best || (ob == best && oa < at))) {
          best = ob;
          at = oa;
        }
      }
      if ((at & 31) == lane) key[at] = 1ull;  // taken (no score maps to 1)
      __syncwarp();
    }
    int done = 0;
    for (int j0 = 0; j0 < nvis; j0 += 32) {
      const bool take = j0 + lane < nvis && key[j0 + lane] == 1ull;
      const unsigned m = __ballot_sync(0xffffffffu, take);
      if (take) out[done + __popc(m & ((1u << lane) - 1u))] = j0 + lane;
      done += __popc(m);
    }
    for (int x = done + lane; x < p.topk; x += 32) out[x] = -1;
    __syncwarp();
  }
}

}  // namespace dash
