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

// A thread takes 8 consecutive elements (one 16-byte load), four threads a group; the
// group's maximum goes round those four lanes.  Bound by HBM: 2 bytes read and 33/32
// written an element.
__global__ void __launch_bounds__(256) dash_ckpt8_pack_kernel(const __grid_constant__ CkptParams p) {
  const long long total = p.groups[p.n];
  const long long stride = (long long)gridDim.x * blockDim.x;
  // whole groups of four lanes stay together: total * 4 is a multiple of 4
  for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < total * 4; i += stride) {
    const long long g = i >> 2;
    const int t = ckpt_tensor(p, g);
    const long long at = (g - p.groups[t]) * 32 + (i & 3) * 8;
    const uint4 w = __ldcs(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.src[t]) + at));
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
    // |x| as bits orders like |x|; infinities and NaN are the largest
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      top = max(top, u[k] & 0x7fffu);
      top = max(top, (u[k] >> 16) & 0x7fffu);
    }
    const unsigned quad = 0xfu << (threadIdx.x & 28);
    top = max(top, __shfl_xor_sync(quad, top, 1));
    top = max(top, __shfl_xor_sync(quad, top, 2));
    const bool bad = top >= 0x7f80u;
    // the biased exponent of a normal maximum is floor(log2) + 127; below that, clamped
    const int e = max((int)(top >> 7) - 127 - 6, -126);
    const float inv = exp2_int(-e);  // e <= 121, so -e stays in the normal range
    uint32_t pk[2] = {0, 0};
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t h = (k & 1) ? (u[k >> 1] & 0xffff0000u) : (u[k >> 1] << 16);
      int m = __float2int_rn(__uint_as_float(h) * inv);  // the product is exact
      m = bad ? 0 : min(max(m, -127), 127);
      pk[k >> 2] |= (uint32_t)(m & 0xff) << (8 * (k & 3));
    }
    *reinterpret_cast<uint2*>(static_cast<int8_t*>(p.dst[t]) + at) = make_uint2(pk[0], pk[1]);
    if ((i & 3) == 0) p.exps[t][g - p.groups[t]] = (int8_t)(bad ? kCkptBad : e);
  }
}

__global__ void __launch_bounds__(256) dash_ckpt8_unpack_kernel(const __grid_constant__ CkptParams p) {
  const long long total = p.groups[p.n];
  const long long stride = (long long)gridDim.x * blockDim.x;
  for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < total * 4; i += stride) {
    const long long g = i >> 2;
    const int t = ckpt_tensor(p, g);
    const long long at = (g - p.groups[t]) * 32 + (i & 3) * 8;
    const uint2 w = __ldcs(reinterpret_cast<const uint2*>(static_cast<const int8_t*>(p.src[t]) + at));
    const int e = p.exps[t][g - p.groups[t]];
    // a foreign exponent below the stored range reads as the smallest one
    const float f = e == kCkptBad ? __int_as_float(0x7fc00000) : exp2_int(max(e, -126));
    uint32_t out[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t word = k < 2 ? w.x : w.y;
      const float lo = (float)(int8_t)(word >> (16 * (k & 1))) * f;
      const float hi = (float)(int8_t)(word >> (16 * (k & 1) + 8)) * f;
      // exact: at most 7 significant bits
      __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
      out[k] = *reinterpret_cast<uint32_t*>(&b);
    }
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.dst[t]) + at) =
        make_uint4(out[0], out[1], out[2], out[3]);
  }
}

}  // namespace dash
