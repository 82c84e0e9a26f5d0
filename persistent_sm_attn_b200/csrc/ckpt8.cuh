// 8-bit checkpoints of bf16 tensors: groups of 32 consecutive elements share a power of
// two, each element keeps a signed 8-bit multiple of it.
//
//   e = max(floor(log2 max|x|) - 6, -126),  m = clamp(round_half_even(x 2^-e), -127, 127)
//
// so the group's largest element lies in [64, 128) steps and a value m 2^e (7 significant
// bits) is exact in bf16: reading back rounds nothing.  The group's error is at most half
// a step, max|x| 2^-7 (one step, where an element above 127 steps is clamped to 127).  A
// group that holds an infinity or a NaN gets e = -128 and reads back as NaN.
#pragma once
#include "ptx.cuh"

namespace dash {

constexpr int kCkptTensors = 4;  // tensors one launch takes (q, k, v, o)
constexpr int kCkptBad = -128;   // exponent of a group that holds a non-finite value

struct CkptParams {
  const void* src[kCkptTensors];  // pack: bf16; unpack: int8 mantissas
  void* dst[kCkptTensors];        // pack: int8 mantissas; unpack: bf16
  int8_t* exps[kCkptTensors];
  long long groups[kCkptTensors + 1];  // first group of each tensor, and the total
  int n;
};

__device__ __forceinline__ int ckpt_tensor(const CkptParams& p, long long g) {
  int t = 0;
  while (t + 1 < p.n && g >= p.groups[t + 1]) ++t;
  return t;
}
// 2^e as a float, -126 <= e <= 127
__device__ __forceinline__ float exp2_int(int e) { return __int_as_float((e + 127) << 23); }

// Pieces of 8 consecutive elements, four to a group; a warp takes 64 at a time, a thread pieces
// `lane` and `32 + lane`, so that neighbouring threads read and write neighbouring pieces.
// Where piece `x` of a round that starts at piece `c` lies: its tensor and first element there.
struct CkptPlace {
  int t;
  long long at;
};
__device__ __forceinline__ CkptPlace ckpt_place(const CkptParams& p, long long c, int x, int lane) {
  int t = ckpt_tensor(p, c >> 2);  // c is the same in the whole warp
  const long long end = p.groups[t + 1] * 4;
  if (c + 64 <= end) return {t, (c - p.groups[t] * 4) * 8 + x * 256 + lane * 8};
  // the round reaches into the next tensor or past the last piece
  const long long i = min(c + 32 * x + lane, p.groups[p.n] * 4 - 4 + (lane & 3));
  t = ckpt_tensor(p, i >> 2);
  return {t, (i - p.groups[t] * 4) * 8};
}
constexpr int kCkptAhead = 2;  // rounds of 64 pieces a warp has in flight

// Lane pairs swap, so that the even lane stores 16 bytes of the round's first half and the odd
// lane of its second.  Bound by HBM: 2 bytes read and 33/32 written an element, 268 million in
// 158 us, 5.1 TB/s; the same loads and stores with next to no arithmetic take 136.  (Products and
// clamps in bf16 pairs: 167 us.  Stores of 8 bytes and fp32 arithmetic: 198.  Twice the loads in
// flight, fewer or more CTAs, no exponents stored: no faster.)
__global__ void __launch_bounds__(256) dash_ckpt8_pack_kernel(const __grid_constant__ CkptParams p) {
  const long long pieces = p.groups[p.n] * 4, stride = (long long)gridDim.x * 8 * 64;
  const int lane = threadIdx.x & 31;
  const bool odd = lane & 1;
  for (long long c0 = ((long long)blockIdx.x * 8 + dev::warp_uniform()) * 64; c0 < pieces;
       c0 += stride * kCkptAhead) {
    uint4 w[kCkptAhead][2];
    CkptPlace at[kCkptAhead][2];
#pragma unroll
    for (int y = 0; y < kCkptAhead; ++y) {
      const long long c = min(c0 + y * stride, pieces - 1);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        at[y][x] = ckpt_place(p, c, x, lane);
        w[y][x] = __ldcs(reinterpret_cast<const uint4*>(
            static_cast<const __nv_bfloat16*>(p.src[at[y][x].t]) + at[y][x].at));
      }
    }
#pragma unroll
    for (int y = 0; y < kCkptAhead; ++y) {
      const long long c = c0 + y * stride;
      if (c >= pieces) break;
      uint2 pk[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const uint32_t u[4] = {w[y][x].x, w[y][x].y, w[y][x].z, w[y][x].w};
        // |x| as bits orders like |x|; infinities and NaN are the largest
        uint32_t top2 = u[0] & 0x7fff7fffu;
#pragma unroll
        for (int k = 1; k < 4; ++k) top2 = __vmaxu2(top2, u[k] & 0x7fff7fffu);
        top2 = __vmaxu2(top2, __shfl_xor_sync(0xffffffffu, top2, 1));
        top2 = __vmaxu2(top2, __shfl_xor_sync(0xffffffffu, top2, 2));
        const uint32_t top = max(top2 & 0xffffu, top2 >> 16);
        const bool bad = top >= 0x7f80u;
        // the biased exponent of a normal maximum is floor(log2) + 127; below that, clamped
        const int e = max((int)(top >> 7) - 127 - 6, -126);
        // x 2^-e + 1.5 2^10, exact in fp32 (below 2^-6 it rounds, but far from a half), as fp16,
        // whose steps are 1 there: the rounding half to even, and the integer in the low byte
        const float inv = exp2_int(-e);  // -122 <= -e <= 126
        uint32_t r[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float lo, hi;
          dev::fma_f32x2(lo, hi, __uint_as_float(u[k] << 16), __uint_as_float(u[k] & 0xffff0000u),
                         inv, 1536.f);
          const __half2 m = __floats2half2_rn(lo, hi);
          r[k] = *reinterpret_cast<const uint32_t*>(&m);
        }
        // +-127.5 steps, the largest there is, rounds to 128: clamped where a group holds it
        if (__any_sync(0xffffffffu, (top & 0x7fu) == 0x7fu)) {
#pragma unroll
          for (int k = 0; k < 4; ++k) r[k] = __vmaxs2(__vmins2(r[k], 0x667f667fu), 0x65816581u);
        }
        uint32_t q[2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
          q[h] = bad ? 0u : __byte_perm(r[2 * h], r[2 * h + 1], 0x6420);
        pk[x] = make_uint2(q[0], q[1]);
        if ((lane & 3) == 0 && c + 32 * x + lane < pieces)
          p.exps[at[y][x].t][at[y][x].at >> 5] = (int8_t)(bad ? kCkptBad : e);
      }
      const uint2 give = odd ? pk[0] : pk[1], keep = odd ? pk[1] : pk[0];
      const uint2 got = make_uint2(__shfl_xor_sync(0xffffffffu, give.x, 1),
                                   __shfl_xor_sync(0xffffffffu, give.y, 1));
      const int t = odd ? at[y][1].t : at[y][0].t;
      int8_t* dst = static_cast<int8_t*>(p.dst[t]) + (odd ? at[y][1].at - 8 : at[y][0].at);
      if (c + (odd ? 31 + lane : lane) < pieces)  // the pair's first piece
        *reinterpret_cast<uint4*>(dst) = odd ? make_uint4(got.x, got.y, keep.x, keep.y)
                                             : make_uint4(keep.x, keep.y, got.x, got.y);
    }
  }
}

// Bound by HBM: 268 million elements in 135 us, 6.0 TB/s.
__global__ void __launch_bounds__(256) dash_ckpt8_unpack_kernel(const __grid_constant__ CkptParams p) {
  const long long pieces = p.groups[p.n] * 4, stride = (long long)gridDim.x * 8 * 64;
  const int lane = threadIdx.x & 31;
  for (long long c0 = ((long long)blockIdx.x * 8 + dev::warp_uniform()) * 64; c0 < pieces;
       c0 += stride * kCkptAhead) {
    uint2 w[kCkptAhead][2];
    int e[kCkptAhead][2];
    CkptPlace at[kCkptAhead][2];
#pragma unroll
    for (int y = 0; y < kCkptAhead; ++y) {
      const long long c = min(c0 + y * stride, pieces - 1);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        at[y][x] = ckpt_place(p, c, x, lane);
        w[y][x] = __ldcs(reinterpret_cast<const uint2*>(
            static_cast<const int8_t*>(p.src[at[y][x].t]) + at[y][x].at));
        e[y][x] = p.exps[at[y][x].t][at[y][x].at >> 5];
      }
    }
#pragma unroll
    for (int y = 0; y < kCkptAhead; ++y) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if (c0 + y * stride + 32 * x + lane >= pieces) continue;
        // a foreign exponent below the stored range reads as the smallest one
        const float f = e[y][x] == kCkptBad ? __int_as_float(0x7fc00000) : exp2_int(max(e[y][x], -126));
        // a byte b + 128 as the low mantissa bits of 2^23: minus 2^23 + 128 it is b exactly
        const uint32_t words[2] = {w[y][x].x ^ 0x80808080u, w[y][x].y ^ 0x80808080u};
        uint32_t out[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t word = words[k >> 1];
          float lo = __uint_as_float(__byte_perm(word, 0x4b000000u, 0x7540 + 2 * (k & 1)));
          float hi = __uint_as_float(__byte_perm(word, 0x4b000000u, 0x7541 + 2 * (k & 1)));
          lo = (lo - 8388736.f) * f;
          hi = (hi - 8388736.f) * f;
          out[k] = dev::pack_bf16x2(lo, hi);  // exact: at most 7 significant bits
        }
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.dst[at[y][x].t]) + at[y][x].at) =
            make_uint4(out[0], out[1], out[2], out[3]);
      }
    }
  }
}

}  // namespace dash
