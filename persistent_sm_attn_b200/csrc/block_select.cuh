// Block selection: means of key blocks, and for each query the blocks with the best scores.
//
//   mean[b,hk,j]  = (1 / n_j) sum of the n_j keys of block j below kv_len[b]      (fp32)
//   score(i, j)   = (sum of the group's query heads q[b,h,i]) . mean[b,hk,j]
//
// A query sees the blocks whose first key lies below its limit, min(kv_len, position + 1
// if causal).  The first `sink` and the last `local` of them are always picked, the other
// places go to the highest scores, equal scores to the lowest block.  Which blocks are
// picked must not depend on the order of a sum, so the picks are those of fp64 scores: a sum
// of bf16 keys is exact in fp64 unless their exponents differ by over 40, and two scores
// closer than fp64 can tell apart do not occur but for equal blocks, which tie exactly.
// Scores are taken in fp32 first, with a bound on their error, and in fp64 where the bound
// leaves a pick open: for few queries by plain sums (dash_block_select_token_kernel), for many
// by tensor-core products (dash_block_select_kernel).
#pragma once
#include "ptx.cuh"

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
// 128 threads' rows of keys are added in shared memory.  Bound by reading K: 34 MB of keys
// (4 heads of 16k, D = 128) in 6.9 us, 4.9 TB/s.
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

// fp32 bits as an integer that orders like the value, and back
__device__ __forceinline__ int ordered_int(float x) {
  const int b = __float_as_int(x);
  return b ^ ((b >> 31) & 0x7fffffff);
}
__device__ __forceinline__ int ordered_int_inverse(int k) { return k ^ ((k >> 31) & 0x7fffffff); }

// Where query i of batch entry b stands: the number of blocks it sees.
__device__ __forceinline__ int visible_blocks(const SelectParams& p, int b, int i) {
  const int len = p.kv_len ? min(max(p.kv_len[b], 0), p.Sk) : p.Sk;
  const long long pos = (long long)(p.q_start ? p.q_start[b] : p.Sk - p.Sq) + i;
  const long long limit = p.causal ? min((long long)len, pos + 1) : (long long)len;
  return limit <= 0 ? 0 : (int)((limit + p.block - 1) / p.block);
}

// The fp64 score of mean row m, the warp together; the same order of sums for every row, so
// equal rows tie.  qd: this lane's D/32 query sums.
template <int D>
__device__ __forceinline__ double exact_score(const double (&qd)[D / 32], const float* m, int lane) {
  double s = 0.0;
#pragma unroll
  for (int x = 0; x < D / 32; ++x) s += qd[x] * (double)m[32 * x + lane];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

// What a warp knows of its query's picks: of the visible blocks j0 <= j < j1 are contested, r
// places of them are to be given.  Bit x of take and open: block 32 x + lane is taken; is to be
// decided in fp64.  NL: 32-block words that a lane's share of a row has room for.
template <int NL>
struct Picks {
  static constexpr int W = (NL + 31) / 32;
  uint32_t take[W], open[W];
  int nvis, j0, j1, nl, r;
  __device__ Picks(const SelectParams& p, int visible)
      : nvis(visible), j0(p.sink), j1(visible - p.local), nl((visible + 31) / 32),
        r(p.topk - p.sink - p.local) {
#pragma unroll
    for (int w = 0; w < W; ++w) take[w] = open[w] = 0u;
  }
  // Every visible block, or the first `sink` and the last `local` of them, is taken.
  __device__ __forceinline__ void take_all(int lane) { take_where(lane, nvis, nvis); }
  __device__ __forceinline__ void take_forced(int lane) { take_where(lane, j0, j1); }
  __device__ __forceinline__ void take_where(int lane, int below, int from) {
#pragma unroll
    for (int w = 0; w < W; ++w) {
      // bits x of word w with 32 (32 w + x) + lane < n
      auto bits = [&](int n) {
        const int k = (n - lane + 31) / 32 - 32 * w;
        return k <= 0 ? 0u : k >= 32 ? 0xffffffffu : (1u << k) - 1u;
      };
      const uint32_t seen = bits(nvis);
      take[w] |= seen & (bits(max(below, 0)) | ~bits(max(from, 0)));
    }
  }
};

// Picks by approximate scores `row` that are off by at most eps2 / 2 and within +-most_score.
// A cut with exactly r scores above it is found by counting; where the lowest score above and
// the highest below are more than eps2 apart, the picks are those of the exact scores.
// Otherwise the scores within eps2 of the cut stay open; returned is how many of them to take.
// guess: in, where the first counts are taken; out, the cut (both of most_score).  Without one
// (0) they are taken where the cut of normally distributed scores of deviation spread most_score
// would be (Abramowitz and Stegun 26.2.22).  Both only decide how many counts it takes.
template <int NL>
__device__ __forceinline__ int pick_approx(Picks<NL>& k, const float* row, float most_score,
                                           float eps2, float& guess, float spread, int lane) {
  constexpr int W = Picks<NL>::W;
  const int j0 = k.j0, j1 = k.j1, nl = k.nl, r = k.r;
  k.take_forced(lane);
  if (!(eps2 < 1e30f)) {  // a partial sum might have overflowed, or an operand is not finite
    for (int x = 0; x < nl; ++x) {
      const int j = 32 * x + lane;
      if (j >= j0 && j < j1) k.open[W == 1 ? 0 : x >> 5] |= 1u << (x & 31);
    }
    return r;
  }
  // this lane's scores, -inf where not contested: in registers for up to 512 blocks
  constexpr bool kHeld = NL <= 16;
  float held[kHeld ? NL : 1] = {};
  if constexpr (kHeld)
#pragma unroll
    for (int x = 0; x < NL; ++x) {
      if (x % 2 == 0 && x >= nl) break;
      const int j = 32 * x + lane;
      held[x] = j >= j0 && j < j1 ? row[j] : -INFINITY;
    }
  auto each = [&](auto&& f) {
    if constexpr (kHeld) {
#pragma unroll
      for (int x = 0; x < NL; ++x) {
        if (x > 0 && x % 2 == 0 && x >= nl) break;
        f(x, held[x]);
      }
    } else {
#pragma unroll 4
      for (int x = 0; x < nl; ++x) {
        const int j = 32 * x + lane;
        f(x, j >= j0 && j < j1 ? row[j] : -INFINITY);
      }
    }
  };
  // the r-th and the next largest lie in (lo, hi]: no score is beyond |q| max|m|
  float lo = -1.01f * most_score - 1e-30f, hi = -lo, cut = 0.f;
  bool found = false;
  // the range falls to a quarter (a third) with each count: up to 512 blocks leave
  // room for three counts in a word
  constexpr int kBits = kHeld ? 10 : 16;
  if (guess == 0.f) {
    const float t = sqrtf(1.3862944f * __log2f((float)(j1 - j0) / (float)r));  // sqrt(-2 ln p)
    guess = spread * (t - (2.30753f + 0.27061f * t) / (1.f + t * (0.99229f + 0.04481f * t)));
  }
  float near = guess * most_score;
  while (!found && hi - lo > eps2) {
    const float d = kHeld ? 0.25f * hi - 0.25f * lo : (hi - lo) * (1.f / 3.f);
    float m1 = lo + d, m2 = kHeld ? 0.5f * lo + 0.5f * hi : hi - d, m3 = hi - d;
    const float off = 0.2f * fabsf(near);
    if (off > 0.f && near - off > lo && near + off < hi)
      m1 = near - off, m2 = kHeld ? near : near + off, m3 = near + off;
    near = 0.f;
    if (!(m1 > lo && m2 > lo && m1 < hi && m2 < hi)) break;
    // a score above m makes m - score negative: its sign bit is added
    unsigned n1 = 0, n2 = 0, n3 = 0;
    each([&](int, float v) {
      n1 += __float_as_uint(m1 - v) >> 31;
      n2 += __float_as_uint(m2 - v) >> 31;
      if constexpr (kHeld) n3 += __float_as_uint(m3 - v) >> 31;
    });
    const unsigned c =
        __reduce_add_sync(0xffffffffu, n1 + (n2 << kBits) + (kHeld ? n3 << (2 * kBits % 32) : 0u));
    const int c1 = (int)(c & ((1u << kBits) - 1)), c2 = (int)((c >> kBits) & ((1u << kBits) - 1));
    int c3 = 0;
    if constexpr (kHeld) c3 = (int)(c >> (2 * kBits));
    if (c1 == r) cut = m1, found = true;
    else if (c2 == r) cut = m2, found = true;
    else if (kHeld && c3 == r) cut = m3, found = true;
    else if (c1 < r) hi = m1;
    else if (c2 < r) lo = m1, hi = m2;
    else if (!kHeld) lo = m2;
    else if (c3 < r) lo = m2, hi = m3;
    else lo = m3;
  }
  if (found && most_score > 1e-20f) guess = cut / most_score;
  float a = lo, z = hi;
  uint32_t above[W];
#pragma unroll
  for (int w = 0; w < W; ++w) above[w] = 0u;
  if (found) {  // lowest above the cut, highest below
    int ka = 0x7f800000, kz = (int)0x807fffff;  // as integers that order like the floats
    each([&](int x, float v) {
      const int o = ordered_int(v);
      if (v > cut) ka = min(ka, o), above[W == 1 ? 0 : x >> 5] |= 1u << (x & 31);
      else kz = max(kz, o);
    });
    a = __int_as_float(ordered_int_inverse(__reduce_min_sync(0xffffffffu, ka)));
    z = __int_as_float(ordered_int_inverse(__reduce_max_sync(0xffffffffu, kz)));
    if (a - z > eps2) {
#pragma unroll
      for (int w = 0; w < W; ++w) k.take[w] |= above[w];
      return 0;
    }
  }
  const float in_at = z + eps2, open_at = a - eps2;
  int in = 0;
  each([&](int x, float v) {
    if (v > in_at) k.take[W == 1 ? 0 : x >> 5] |= 1u << (x & 31), ++in;
    else if (v >= open_at) k.open[W == 1 ? 0 : x >> 5] |= 1u << (x & 31);
  });
  return r - __reduce_add_sync(0xffffffffu, in);
}

// Decides the open blocks, `need` of which are to be taken, by their fp64 scores.  key: a word
// a block of shared memory.
template <int D, int NL>
__device__ __forceinline__ void pick_exact(Picks<NL>& k, int need, const SelectParams& p, int b,
                                           int hk, int i, const float* means, uint32_t* key,
                                           int lane) {
  constexpr int W = Picks<NL>::W;
  const int j0 = k.j0, j1 = k.j1, nl = k.nl;
  uint32_t(&take)[W] = k.take;
  uint32_t(&open)[W] = k.open;
  int undecided = 0;
#pragma unroll
  for (int w = 0; w < W; ++w) undecided += __popc(open[w]);
  undecided = __reduce_add_sync(0xffffffffu, undecided);
  auto each = [&](auto&& f) {
#pragma unroll 1
    for (int x = 0; x < nl; ++x) {
      const int j = 32 * x + lane;
      if (j >= j0 && j < j1) f(x, j);
    }
  };
  double qd[D / 32] = {};
  const __nv_bfloat16* q = p.q + b * p.sb + (long long)hk * p.G * p.sh + (long long)i * p.ss;
#pragma unroll 4
  for (int g = 0; g < p.G; ++g)
#pragma unroll
    for (int x = 0; x < D / 32; ++x)
      qd[x] += (double)__bfloat162float(q[(long long)g * p.sh + 32 * x + lane]);
  if (undecided <= 32) {
    // the usual case: one open block a lane (ascending), its place among them by 64-bit keys
    int mine = -1, n = 0;
#pragma unroll 1
    for (int x = 0; x < nl; ++x) {
      unsigned m = __ballot_sync(0xffffffffu, (open[W == 1 ? 0 : x >> 5] >> (x & 31)) & 1u);
      for (; m; m &= m - 1, ++n)
        if (lane == n) mine = 32 * x + __ffs(m) - 1;
    }
    unsigned long long key64 = 0;
#pragma unroll 2
    for (int t = 0; t < n; ++t) {
      const int j = __shfl_sync(0xffffffffu, mine, t);
      const unsigned long long k = order_key(exact_score<D>(qd, means + (long long)j * D, lane));
      if (lane == t) key64 = k;
    }
    int place = 0;
#pragma unroll 2
    for (int t = 0; t < n; ++t) {
      const unsigned long long k = __shfl_sync(0xffffffffu, key64, t);
      place += k > key64 || (k == key64 && t < lane);
    }
    const bool in = lane < n && place < need;
#pragma unroll 2
    for (int t = 0; t < n; ++t) {
      const int j = __shfl_sync(0xffffffffu, in ? mine : -1, t);
      if (j >= 0 && (j & 31) == lane)
#pragma unroll
        for (int w = 0; w < W; ++w)
          if (w == j >> 10) take[w] |= 1u << ((j >> 5) & 31);
    }
    need = 0;
  }
  if (need > 0) {  // many open blocks (equal ones, operands that are not finite)
    // exact scores of the open blocks, their keys' upper words in place of the scores;
    // then, among those that tie in it, by the lower words; then by number
#pragma unroll 1
    for (int word = 0; word < 2; ++word) {
#pragma unroll 1
      for (int x = 0; x < nl; ++x) {
        unsigned m = __ballot_sync(0xffffffffu, (open[W == 1 ? 0 : x >> 5] >> (x & 31)) & 1u);
        while (m) {
          const int src = __ffs(m) - 1;
          m &= m - 1;
          const int j = 32 * x + src;
          const unsigned long long k =
              order_key(exact_score<D>(qd, means + (long long)j * D, lane));
          if (lane == src) key[j] = word == 0 ? (uint32_t)(k >> 32) : (uint32_t)k;
        }
      }
      uint32_t t = 0;  // the need-th largest word, bit by bit
#pragma unroll 1
      for (uint32_t bitv = 0x80000000u; bitv; bitv >>= 1) {
        int c = 0;
        each([&](int x, int j) {
          if ((open[W == 1 ? 0 : x >> 5] >> (x & 31)) & 1u) c += key[j] >= (t | bitv);
        });
        if ((int)__reduce_add_sync(0xffffffffu, c) >= need) t |= bitv;
      }
      int in = 0, same = 0;
      each([&](int x, int j) {
        const uint32_t bx = 1u << (x & 31);
        if (!(open[W == 1 ? 0 : x >> 5] & bx)) return;
        if (key[j] > t) take[W == 1 ? 0 : x >> 5] |= bx, open[W == 1 ? 0 : x >> 5] &= ~bx, ++in;
        else if (key[j] < t) open[W == 1 ? 0 : x >> 5] &= ~bx;
        else ++same;
      });
      need -= __reduce_add_sync(0xffffffffu, in);
      same = __reduce_add_sync(0xffffffffu, same);
      if (same == need) {
#pragma unroll
        for (int w = 0; w < W; ++w) take[w] |= open[w], open[w] = 0u;
        need = 0;
        break;
      }
    }
    // exact ties: the lowest numbers
#pragma unroll 1
    for (int x = 0; x < nl && need > 0; ++x) {
      const bool tie = (open[W == 1 ? 0 : x >> 5] >> (x & 31)) & 1u;
      const unsigned m = __ballot_sync(0xffffffffu, tie);
      if (tie && __popc(m & ((1u << lane) - 1u)) < need) take[W == 1 ? 0 : x >> 5] |= 1u << (x & 31);
      need -= __popc(m);
    }
  }
}

// Writes the picks ascending, then -1; topk places, however many blocks are marked.
template <int NL>
__device__ __forceinline__ void put_out(const Picks<NL>& k, int topk, int* out, int lane) {
  constexpr int W = Picks<NL>::W;
  const unsigned below = (1u << lane) - 1u;
  int done = 0;
#pragma unroll (NL <= 16 ? NL : 4)
  for (int x = 0; x < NL; ++x) {
    if (x >= k.nl) break;
    const bool on = (k.take[W == 1 ? 0 : x >> 5] >> (x & 31)) & 1u;
    const unsigned m = __ballot_sync(0xffffffffu, on);
    const int at = done + __popc(m & below);
    if (on && at < topk) out[at] = 32 * x + lane;
    done += __popc(m);
  }
  for (int x = done + lane; x < topk; x += 32) out[x] = -1;
}

// A vector's squared norm as the bounds take it: below 2^-100 the squares of its elements may
// have left fp32's range (those under 2^-63 are 0 or inexact), and no bound comes from it.  From
// there on what is lost, at most 128 squares of 2^-126, is 2^-19 of it.
__device__ __forceinline__ float norm_or_inf(float n2) {
  return n2 < 0x1p-100f ? INFINITY : sqrtf(n2);
}

// Few queries (serving): a CTA per query reads the K/V head's means once, a warp per row with
// 16 (D = 64: 8) bytes a lane, eight rows in flight.  A score is a sum of D products in fp32
// with D/32 + 5 roundings on the way of each, so it is off by less than 2^-20 |q||m|, and by
// what the heads' sum was rounded by (see dash_block_select_kernel); |m| is at most sqrt(D)
// times the largest element.  Queries too small for their norm go to fp64 altogether.  Bound by reading the means: 64 tokens of 8 K/V heads, up to 256
// blocks each, in 12.4 us (all scores in fp64: 21).
template <int D, int NL>
__global__ void __launch_bounds__(256) dash_block_select_token_kernel(const SelectParams p) {
  extern __shared__ __align__(16) unsigned char select_smem[];
  float* sc = reinterpret_cast<float*>(select_smem);  // [nb]
  __shared__ int top_bits;
  constexpr int V = D / 32, kRows = 8;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int bh = blockIdx.y, b = bh / p.Hkv, hk = bh % p.Hkv, i = blockIdx.x;
  const int nvis = visible_blocks(p, b, i);
  const float* means = p.means + (long long)bh * p.nb * D;
  Picks<NL> k(p, nvis);
  const bool contest = nvis > p.topk && k.r > 0;
  if (threadIdx.x == 0) top_bits = 0;
  __syncthreads();
  float n2 = 0.f, a2 = 0.f;  // this lane's share of |q|^2 and of |sum of |heads||^2
  if (contest) {
    const __nv_bfloat16* q = p.q + b * p.sb + (long long)hk * p.G * p.sh + (long long)i * p.ss + lane * V;
    float qs[V] = {}, qa[V] = {};
#pragma unroll 4
    for (int g = 0; g < p.G; ++g)
#pragma unroll
      for (int x = 0; x < V; ++x) {
        const float y = __bfloat162float(q[(long long)g * p.sh + x]);
        qs[x] += y, qa[x] += fabsf(y);
      }
#pragma unroll
    for (int x = 0; x < V; ++x) n2 += qs[x] * qs[x], a2 += qa[x] * qa[x];
    int top = 0;  // largest |element| as bits, so that an infinity or NaN stays the largest
    for (int base = k.j0 + warp * kRows; base < k.j1; base += 8 * kRows) {
      float m[kRows][V], s[kRows];
#pragma unroll
      for (int y = 0; y < kRows; ++y) {
        const float* src = means + (long long)min(base + y, k.j1 - 1) * D + lane * V;
        if constexpr (V == 4) {
          const float4 w = *reinterpret_cast<const float4*>(src);
          m[y][0] = w.x, m[y][1] = w.y, m[y][2] = w.z, m[y][3] = w.w;
        } else {
          const float2 w = *reinterpret_cast<const float2*>(src);
          m[y][0] = w.x, m[y][1] = w.y;
        }
      }
#pragma unroll
      for (int y = 0; y < kRows; ++y) {
        s[y] = 0.f;
#pragma unroll
        for (int x = 0; x < V; ++x) {
          s[y] = fmaf(qs[x], m[y][x], s[y]);
          top = max(top, __float_as_int(m[y][x]) & 0x7fffffff);
        }
      }
      // eight sums over the warp: halves swap what the other sums on
#pragma unroll
      for (int h = 4; h > 0; h >>= 1) {
        const bool up = lane & (h * 4);
#pragma unroll
        for (int y = 0; y < h; ++y) {
          const float give = up ? s[y] : s[y + h], keep = up ? s[y + h] : s[y];
          s[y] = keep + __shfl_xor_sync(0xffffffffu, give, h * 4);
        }
      }
      s[0] += __shfl_xor_sync(0xffffffffu, s[0], 2);
      s[0] += __shfl_xor_sync(0xffffffffu, s[0], 1);
      const int row = base + (lane >> 2);  // bits 4, 3, 2 of the lane chose the row's
      if ((lane & 3) == 0 && row < k.j1) sc[row] = s[0];
    }
    top = __reduce_max_sync(0xffffffffu, top);
    if (lane == 0) atomicMax(&top_bits, top);
  }
  __syncthreads();
  if (warp > 0) return;
  if (contest) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      n2 += __shfl_xor_sync(0xffffffffu, n2, o);
      a2 += __shfl_xor_sync(0xffffffffu, a2, o);
    }
    const float mnorm = sqrtf((float)D) * __int_as_float(top_bits);
    const float qn = norm_or_inf(n2), most = (qn + 0x1p-10f * sqrtf(a2)) * mnorm;
    const float eps2 = 2.f * ((0x1p-20f * qn + 0x1p-24f * p.G * sqrtf(a2)) * mnorm + 1e-35f);
    float guess = 0.f;
    const int need = pick_approx<NL>(k, sc, most, eps2, guess, qn / (most + 1e-30f) *
                                     __int_as_float(top_bits) * 0.25f, lane);
    __syncwarp();
    if (need > 0)
      pick_exact<D, NL>(k, need, p, b, hk, i, means, reinterpret_cast<uint32_t*>(sc), lane);
  } else if (nvis > p.topk) {
    k.take_forced(lane);
  } else {
    k.take_all(lane);
  }
  put_out(k, p.topk, p.idx + ((long long)bh * p.Sq + i) * p.topk, lane);
}

__device__ __forceinline__ void ldmatrix_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// x = hi + lo + rest with hi, lo in bf16: |rest| <= 2^-16 |x|
__device__ __forceinline__ void split_bf16(float x, float y, uint32_t& hi, uint32_t& lo) {
  hi = dev::pack_bf16x2(x, y);
  lo = dev::pack_bf16x2(x - __uint_as_float(hi << 16), y - __uint_as_float(hi & 0xffff0000u));
}

template <int D, int QT>
struct SelectCfg {
  static constexpr int kThreads = 512;
  static constexpr int kRows = QT < 16 ? 16 : QT;  // MMA rows
  static constexpr int RG = kRows / 16;            // 16-row groups; 8 warps over the 64 blocks each
  static constexpr int kLd = D * 2 + 16;           // bytes of a staged row: no bank conflicts
  static constexpr int kQ = 2 * kRows * kLd;       // queries, high and low parts
  static constexpr int kStage = kQ + 2 * 64 * kLd; // and 64 means
  static constexpr float kError = 1.001f * (3 * 0x1p-16f + (3 * D + 3) * 0x1p-23f);
  static int smem(int nb) { return kStage + QT * ((nb + 63) / 64 * 64 + 8) * 4; }
};

// Many queries: QT of one K/V head, all visible blocks, 64 at a time.  16k queries of 16 heads on
// 256 blocks in 126 us, half of it scores, half picks; bound by issuing instructions (some
// 1300 a query and warp).  QT = 64 with 1024 threads, which splits each mean half as often,
// took 136 us: with one CTA an SM nothing runs under its barriers.
//
// Scores: q = q_h + q_l, m = m_h + m_l in bf16, score ~ q_h m_h + q_h m_l + q_l m_h, fp32
// accumulators.  What is left out and rounded is at most 3 * 2^-16 sum|q||m|, the sum of 3 D
// products in fp32 at most (3 D + 3) 2^-23 of the same, and that at most |q| max_j |m_j|
// (Euclidean norms).  The heads' sum q itself is rounded, by at most G 2^-24 sum_g |q_g|, which
// their cancelling may make large against q.  Together, with u = 3 * 2^-16 + (3 D + 3) 2^-23
// and a thousandth for the norms' own rounding, the error is below
//     eps = 1.001 u (|q| + G 2^-24 / u |sum_g |q_g||) max_j |m_j|.
// An eps that is not finite (an infinity or NaN among the operands, a norm too small for fp32's
// squares) leaves everything to fp64.
//
// NL: 32-block words that a lane's share of a row has room for.
template <int D, int QT, int NL>
__global__ void __launch_bounds__(512, 2) dash_block_select_kernel(const SelectParams p) {
  using C = SelectCfg<D, QT>;
  extern __shared__ __align__(16) unsigned char select_smem[];
  __shared__ float qnorm[C::kRows];
  __shared__ int mnorm_bits, todo_n;
  __shared__ int2 todo[QT];
  __shared__ int nv[QT];  // blocks that each query sees
  constexpr int W = (NL + 31) / 32;
  const int ld = (p.nb + 63) / 64 * 64 + 8;
  float* sc = reinterpret_cast<float*>(select_smem + C::kStage);  // [QT][ld]
  const uint32_t stage = dev::smem_u32(select_smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int bh = blockIdx.y, b = bh / p.Hkv, hk = bh % p.Hkv;
  const int i0 = (int)(gridDim.x - 1 - blockIdx.x) * QT;  // the longest rows first
  const int rg = warp / 8, cg = warp % 8;  // one 16 x 8 product a warp
  const int last = min(i0 + QT, p.Sq) - 1;
  const int most = visible_blocks(p, b, last);  // of the CTA's queries (they see ever more)
  if (tid == 0) mnorm_bits = todo_n = 0;
  if (tid < QT) nv[tid] = visible_blocks(p, b, i0 + tid);

  // ---- means: 64 are on their way while the last 64 (first, the queries) are worked on
  const float* means = p.means + (long long)bh * p.nb * D;
  unsigned char* const mstage = select_smem + C::kQ;
  float4 next[D / 32];
  const int mrow = tid >> 3, part = tid & 7;
  auto fetch = [&](int j0) {
    const float4* src = reinterpret_cast<const float4*>(means + (long long)(j0 + mrow) * D) + part;
#pragma unroll
    for (int x = 0; x < D / 32; ++x)
      next[x] = j0 + mrow < most ? src[8 * x] : make_float4(0.f, 0.f, 0.f, 0.f);
  };
  fetch(0);

  // ---- the group's queries, summed, split and staged
  constexpr int CH = D / 8;  // 16-byte pieces of a row, in consecutive lanes
  for (int x = tid; x < C::kRows * CH; x += C::kThreads) {
    const int row = x / CH, c = x % CH;
    const bool on = row < QT && i0 + row < p.Sq;
    const __nv_bfloat16* q = p.q + b * p.sb + (long long)hk * p.G * p.sh +
                             (long long)(on ? i0 + row : 0) * p.ss + c * 8;
    float v[8] = {}, va[8] = {};
    if (on) {
#pragma unroll 4
      for (int g = 0; g < p.G; ++g) {
        const uint4 w = *reinterpret_cast<const uint4*>(q + (long long)g * p.sh);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float x0 = __uint_as_float(u[k] << 16), x1 = __uint_as_float(u[k] & 0xffff0000u);
          v[2 * k] += x0, va[2 * k] += fabsf(x0);
          v[2 * k + 1] += x1, va[2 * k + 1] += fabsf(x1);
        }
      }
    }
    float n2 = 0.f, a2 = 0.f;
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      n2 += v[2 * k] * v[2 * k] + v[2 * k + 1] * v[2 * k + 1];
      a2 += va[2 * k] * va[2 * k] + va[2 * k + 1] * va[2 * k + 1];
      split_bf16(v[2 * k], v[2 * k + 1], hi[k], lo[k]);
    }
    unsigned char* at = select_smem + row * C::kLd + c * 16;
    *reinterpret_cast<uint4*>(at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4*>(at + C::kRows * C::kLd) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
#pragma unroll
    for (int o = CH / 2; o > 0; o >>= 1) {
      n2 += __shfl_xor_sync(0xffffffffu, n2, o);
      a2 += __shfl_xor_sync(0xffffffffu, a2, o);
    }
    if (c == 0) qnorm[row] = norm_or_inf(n2) + 0x1p-24f / C::kError * p.G * sqrtf(a2);
  }

  // ---- scores
  for (int j0 = 0; j0 < most; j0 += 64) {
    __syncthreads();
    {
      float n2 = 0.f;
#pragma unroll
      for (int x = 0; x < D / 32; ++x) {
        const float4 w = next[x];
        n2 += w.x * w.x + w.y * w.y + w.z * w.z + w.w * w.w;
        uint2 hi, lo;
        split_bf16(w.x, w.y, hi.x, lo.x);
        split_bf16(w.z, w.w, hi.y, lo.y);
        unsigned char* at = mstage + mrow * C::kLd + (8 * x + part) * 8;
        *reinterpret_cast<uint2*>(at) = hi;
        *reinterpret_cast<uint2*>(at + 64 * C::kLd) = lo;
      }
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) n2 += __shfl_xor_sync(0xffffffffu, n2, o);
      // as bits, so that an infinity or NaN stays the largest
      const int most_n2 = __reduce_max_sync(0xffffffffu, __float_as_int(n2) & 0x7fffffff);
      if (lane == 0) atomicMax(&mnorm_bits, most_n2);
    }
    __syncthreads();
    if (j0 + 64 < most) fetch(j0 + 64);
    if (rg < C::RG) {
      float acc[3][4] = {};  // high x high, high x low, low x high: three chains of products
      // queries: rows 0-7, rows 8-15, rows 0-7 of the next 8 columns, rows 8-15
      const uint32_t qat = stage + (uint32_t)(rg * 16 + (lane & 15)) * C::kLd + (lane >> 4) * 16;
      // means: high k 0-7, high k 8-15, low k 0-7, low k 8-15
      const uint32_t mat = stage + C::kQ + (lane >> 4) * (64 * C::kLd) + ((lane >> 3) & 1) * 16 +
                           (uint32_t)(cg * 8 + (lane & 7)) * C::kLd;
#pragma unroll 4
      for (int kk = 0; kk < D / 16; ++kk) {
        uint32_t qh[4], ql[4], m[4];
        ldmatrix_x4(qat + kk * 32, qh);
        ldmatrix_x4(qat + C::kRows * C::kLd + kk * 32, ql);
        ldmatrix_x4(mat + kk * 32, m);
        mma_bf16(acc[0], qh, m[0], m[1]);
        mma_bf16(acc[1], qh, m[2], m[3]);
        mma_bf16(acc[2], ql, m[0], m[1]);
      }
#pragma unroll
      for (int x = 0; x < 4; ++x) acc[0][x] += acc[1][x] + acc[2][x];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int row = rg * 16 + half * 8 + (lane >> 2);
        if (row < QT)
          *reinterpret_cast<float2*>(sc + row * ld + j0 + cg * 8 + (lane & 3) * 2) =
              make_float2(acc[0][2 * half], acc[0][2 * half + 1]);
      }
    }
  }
  __syncthreads();

  // ---- picks, a warp per query.  Queries whose picks the bound leaves open are put off, so
  // that the warps share them (one in fifteen on normal data, two blocks each)
  const float mnorm = norm_or_inf(__int_as_float(mnorm_bits));
  uint32_t* saved = reinterpret_cast<uint32_t*>(mstage);  // [QT][2 W][32], over the means
  auto out = [&](int rr) { return p.idx + ((long long)bh * p.Sq + i0 + rr) * p.topk; };
  float guess = 0.f;  // the last cut, of the largest score that could be
  for (int rr = warp; rr < QT && i0 + rr < p.Sq; rr += C::kThreads / 32) {
    Picks<NL> k(p, nv[rr]);
    int need = 0;
    if (k.nvis > p.topk && k.r > 0) {
      const float most_score = qnorm[rr] * mnorm;
      need = pick_approx<NL>(k, sc + rr * ld, most_score,
                             2.f * (C::kError * most_score + 1e-35f), guess, rsqrtf((float)D),
                             lane);
    } else if (k.nvis > p.topk) {
      k.take_forced(lane);
    } else {
      k.take_all(lane);
    }
    if (need > 0) {
#pragma unroll
      for (int w = 0; w < W; ++w) {
        saved[(rr * 2 * W + w) * 32 + lane] = k.take[w];
        saved[(rr * 2 * W + W + w) * 32 + lane] = k.open[w];
      }
      if (lane == 0) {
        const int t = atomicAdd(&todo_n, 1);
        todo[t] = make_int2(rr, need);
      }
    } else {
      put_out(k, p.topk, out(rr), lane);
    }
  }
  __syncthreads();
  for (int t = warp; t < todo_n; t += C::kThreads / 32) {
    const int rr = todo[t].x;
    Picks<NL> k(p, nv[rr]);
#pragma unroll
    for (int w = 0; w < W; ++w) {
      k.take[w] = saved[(rr * 2 * W + w) * 32 + lane];
      k.open[w] = saved[(rr * 2 * W + W + w) * 32 + lane];
    }
    pick_exact<D, NL>(k, todo[t].y, p, b, hk, i0 + rr, means,
                      reinterpret_cast<uint32_t*>(sc + rr * ld), lane);
    put_out(k, p.topk, out(rr), lane);
  }
}

}  // namespace dash
