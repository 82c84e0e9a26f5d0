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
#include <cuda_bf16.h>
#include <cstdint>

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

// clamp(x s, -127, 127) of two bf16 values and two powers of two
__device__ __forceinline__ uint32_t ckpt_scale(uint32_t x, uint32_t s) {
  const __nv_bfloat162 a = *reinterpret_cast<__nv_bfloat162*>(&x);
  const __nv_bfloat162 b = *reinterpret_cast<__nv_bfloat162*>(&s);
  const __nv_bfloat162 top = __float2bfloat162_rn(127.f), low = __float2bfloat162_rn(-127.f);
  const __nv_bfloat162 m = __hmax2(__hmin2(__hmul2(a, b), top), low);
  return *reinterpret_cast<const uint32_t*>(&m);
}

// A thread takes pieces of 8 consecutive elements, four threads a group, several pieces in
// flight: neighbouring threads read neighbouring pieces.  Bound by HBM: 2 bytes read and 33/32
// written an element.
//
// Packing, a warp takes 64 pieces, a thread pieces `lane` and `32 + lane`; lane pairs swap, so
// that the even lane stores 16 bytes of the first half and the odd lane of the second.  (Stores
// of 8 bytes: 4.1 TB/s; 16 elements a thread, its two loads beside each other: 5.1.)
__global__ void __launch_bounds__(256) dash_ckpt8_pack_kernel(const __grid_constant__ CkptParams p) {
  const long long pieces = p.groups[p.n] * 4, stride = (long long)gridDim.x * 8 * 64;
  const int lane = threadIdx.x & 31;
  constexpr int kAhead = 2;  // rounds of 64 pieces in flight
  for (long long c0 = ((long long)blockIdx.x * 8 + (threadIdx.x >> 5)) * 64; c0 < pieces;
       c0 += stride * kAhead) {
    uint4 w[kAhead][2];
    long long at[kAhead][2];
    int tensor[kAhead][2];
#pragma unroll
    for (int y = 0; y < kAhead; ++y)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const long long i = min(c0 + y * stride + 32 * x + lane, pieces - 4 + (lane & 3)), g = i >> 2;
        const int t = ckpt_tensor(p, g);
        tensor[y][x] = t;
        at[y][x] = (g - p.groups[t]) * 32 + (i & 3) * 8;
        w[y][x] = __ldcs(
            reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.src[t]) + at[y][x]));
      }
#pragma unroll
    for (int y = 0; y < kAhead; ++y) {
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
        // 2^-e, -121 <= -e <= 126, in bf16: x 2^-e is exact there (or rounds to 0 below), and
        // clamping before the rounding gives what clamping after it would
        const uint32_t inv = (uint32_t)(127 - e) << 7;
        uint32_t q[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t r[4];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint32_t m = ckpt_scale(u[2 * h + k], inv | inv << 16);
            // the sum with 1.5 2^23 has the integer, rounded half to even, in its low byte
            r[2 * k] = __float_as_uint(__uint_as_float(m << 16) + 12582912.f);
            r[2 * k + 1] = __float_as_uint(__uint_as_float(m & 0xffff0000u) + 12582912.f);
          }
          const uint32_t bytes =
              __byte_perm(__byte_perm(r[0], r[1], 0x0040), __byte_perm(r[2], r[3], 0x0040), 0x5410);
          q[h] = bad ? 0u : bytes;
        }
        pk[x] = make_uint2(q[0], q[1]);
        if ((lane & 3) == 0 && c0 + y * stride + 32 * x + lane < pieces)
          p.exps[tensor[y][x]][at[y][x] >> 5] = (int8_t)(bad ? kCkptBad : e);
      }
      const bool odd = lane & 1;
      const uint2 give = odd ? pk[0] : pk[1], keep = odd ? pk[1] : pk[0];
      const uint2 got = make_uint2(__shfl_xor_sync(0xffffffffu, give.x, 1),
                                   __shfl_xor_sync(0xffffffffu, give.y, 1));
      const long long i = c0 + y * stride + (odd ? 31 + lane : lane);  // the pair's first piece
      const int t = odd ? tensor[y][1] : tensor[y][0];
      int8_t* dst = static_cast<int8_t*>(p.dst[t]) + (odd ? at[y][1] - 8 : at[y][0]);
      if (i < pieces)
        *reinterpret_cast<uint4*>(dst) = odd ? make_uint4(got.x, got.y, keep.x, keep.y)
                                             : make_uint4(keep.x, keep.y, got.x, got.y);
    }
  }
}

// (One piece of a thread in flight: 5.4 TB/s; four: 5.9.)
constexpr int kCkptAhead = 4;
__global__ void __launch_bounds__(256) dash_ckpt8_unpack_kernel(const __grid_constant__ CkptParams p) {
  const long long pieces = p.groups[p.n] * 4;
  const long long stride = (long long)gridDim.x * blockDim.x;
  for (long long i0 = (long long)blockIdx.x * blockDim.x + threadIdx.x; i0 < pieces;
       i0 += stride * kCkptAhead) {
    uint2 w[kCkptAhead];
    int e[kCkptAhead], tensor[kCkptAhead];
    long long at[kCkptAhead];
#pragma unroll
    for (int y = 0; y < kCkptAhead; ++y) {
      const long long i = min(i0 + y * stride, pieces - 1), g = i >> 2;
      const int t = ckpt_tensor(p, g);
      tensor[y] = t;
      at[y] = (g - p.groups[t]) * 32 + (i & 3) * 8;
      w[y] = __ldcs(reinterpret_cast<const uint2*>(static_cast<const int8_t*>(p.src[t]) + at[y]));
      e[y] = p.exps[t][at[y] >> 5];
    }
#pragma unroll
    for (int y = 0; y < kCkptAhead; ++y) {
      if (i0 + y * stride >= pieces) break;
      // a foreign exponent below the stored range reads as the smallest one
      const float f = e[y] == kCkptBad ? __int_as_float(0x7fc00000) : exp2_int(max(e[y], -126));
      uint32_t out[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t word = k < 2 ? w[y].x : w[y].y;
        const float lo = (float)(int8_t)(word >> (16 * (k & 1))) * f;
        const float hi = (float)(int8_t)(word >> (16 * (k & 1) + 8)) * f;
        // exact: at most 7 significant bits
        __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
        out[k] = *reinterpret_cast<uint32_t*>(&b);
      }
      *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.dst[tensor[y]]) + at[y]) =
          make_uint4(out[0], out[1], out[2], out[3]);
    }
  }
}

}  // namespace dash
