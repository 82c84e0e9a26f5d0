// 8-bit checkpoints of bf16 tensors: groups of 32 consecutive elements share a power of
// two, each element keeps a signed 8-bit multiple of it.
//
//   e = max(floor(log2 max|x|) - 6, -126),  m = clamp(round_half_even(x 2^-e), -127, 127)
//
// so the group's largest element lies in [64, 128) steps and a value m 2^e (7 significant
// bits) is exact in bf16: reading back rounds nothing.  The group's error is at most half
// a step, max|x| 2^-7 where e is not held at -126: also of the element that is clamped, since
// a bf16 in [64, 128) steps is a whole number of halves, 127.5 at most.  A group that holds an
// infinity or a NaN gets e = -128 and reads back as NaN.
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

// Pieces of 8 consecutive elements, four to a group; a warp takes 128 at a time, a thread pieces
// `32 x + lane`, so that neighbouring threads read and write neighbouring pieces.
constexpr int kCkptTake = 4;                   // pieces of a thread
constexpr int kCkptChunk = 32 * kCkptTake;     // and of a warp
// Where a thread's pieces lie.  Nearly every chunk is within one tensor: one base for all.
template <bool kOne>
struct CkptPlaces {
  int t;
  long long at;  // first element of this thread's piece 0 in tensor t
  __device__ __forceinline__ int tensor(int) const { return t; }
  __device__ __forceinline__ long long elem(int x) const { return at + x * 256; }
  __device__ __forceinline__ bool valid(int) const { return true; }
};
template <>
struct CkptPlaces<false> {
  int t[kCkptTake];
  long long at[kCkptTake];
  bool in[kCkptTake];
  __device__ __forceinline__ int tensor(int x) const { return t[x]; }
  __device__ __forceinline__ long long elem(int x) const { return at[x]; }
  __device__ __forceinline__ bool valid(int x) const { return in[x]; }
};
__device__ __forceinline__ CkptPlaces<false> ckpt_places(const CkptParams& p, long long c, int lane) {
  CkptPlaces<false> r;
#pragma unroll
  for (int x = 0; x < kCkptTake; ++x) {
    const long long pieces = p.groups[p.n] * 4, i = c + 32 * x + lane;
    r.in[x] = i < pieces;
    const long long j = r.in[x] ? i : pieces - 4;  // past the end: read, and not written
    r.t[x] = ckpt_tensor(p, j >> 2);
    r.at[x] = (j - p.groups[r.t[x]] * 4) * 8;
  }
  return r;
}

// Lane pairs swap, so that the even lane stores 16 bytes of pieces x and the odd lane of x + 1.
template <bool kOne>
__device__ __forceinline__ void ckpt_pack_chunk(const CkptParams& p, const CkptPlaces<kOne>& at,
                                                int lane) {
  const bool odd = lane & 1;
  uint4 w[kCkptTake];
#pragma unroll
  for (int x = 0; x < kCkptTake; ++x)
    w[x] = __ldcs(reinterpret_cast<const uint4*>(
        static_cast<const __nv_bfloat16*>(p.src[at.tensor(x)]) + at.elem(x)));
  uint2 pk[kCkptTake];
#pragma unroll
  for (int x = 0; x < kCkptTake; ++x) {
    const uint32_t u[4] = {w[x].x, w[x].y, w[x].z, w[x].w};
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
    for (int h = 0; h < 2; ++h) q[h] = bad ? 0u : __byte_perm(r[2 * h], r[2 * h + 1], 0x6420);
    pk[x] = make_uint2(q[0], q[1]);
    if ((lane & 3) == 0 && at.valid(x))
      p.exps[at.tensor(x)][at.elem(x) >> 5] = (int8_t)(bad ? kCkptBad : e);
  }
#pragma unroll
  for (int x = 0; x < kCkptTake; x += 2) {
    const uint2 give = odd ? pk[x] : pk[x + 1], keep = odd ? pk[x + 1] : pk[x];
    const uint2 got = make_uint2(__shfl_xor_sync(0xffffffffu, give.x, 1),
                                 __shfl_xor_sync(0xffffffffu, give.y, 1));
    int8_t* dst = static_cast<int8_t*>(p.dst[odd ? at.tensor(x + 1) : at.tensor(x)]) +
                  (odd ? at.elem(x + 1) - 8 : at.elem(x));  // the pair's first piece
    if (odd ? at.valid(x + 1) : at.valid(x))
      *reinterpret_cast<uint4*>(dst) = odd ? make_uint4(got.x, got.y, keep.x, keep.y)
                                           : make_uint4(keep.x, keep.y, got.x, got.y);
  }
}

template <bool kOne>
__device__ __forceinline__ void ckpt_unpack_chunk(const CkptParams& p, const CkptPlaces<kOne>& at) {
  uint2 w[kCkptTake];
  int e[kCkptTake];
#pragma unroll
  for (int x = 0; x < kCkptTake; ++x) {
    w[x] = __ldcs(reinterpret_cast<const uint2*>(
        static_cast<const int8_t*>(p.src[at.tensor(x)]) + at.elem(x)));
    e[x] = p.exps[at.tensor(x)][at.elem(x) >> 5];
  }
#pragma unroll
  for (int x = 0; x < kCkptTake; ++x) {
    // a foreign exponent below the stored range reads as the smallest one
    const float f = e[x] == kCkptBad ? __int_as_float(0x7fc00000) : exp2_int(max(e[x], -126));
    // a byte b + 128 as the low mantissa bits of 2^23: minus 2^23 + 128 it is b exactly
    const uint32_t words[2] = {w[x].x ^ 0x80808080u, w[x].y ^ 0x80808080u};
    uint32_t out[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t word = words[k >> 1];
      float lo = __uint_as_float(__byte_perm(word, 0x4b000000u, 0x7540 + 2 * (k & 1)));
      float hi = __uint_as_float(__byte_perm(word, 0x4b000000u, 0x7541 + 2 * (k & 1)));
      dev::add_f32x2(lo, hi, lo, hi, -8388736.f);
      dev::mul_f32x2(lo, hi, lo, hi, f, f);
      out[k] = dev::pack_bf16x2(lo, hi);  // exact: at most 7 significant bits
    }
    if (at.valid(x))
      *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.dst[at.tensor(x)]) + at.elem(x)) =
          make_uint4(out[0], out[1], out[2], out[3]);
  }
}

template <typename One, typename Some>
__device__ __forceinline__ void ckpt_chunks(const CkptParams& p, One&& one, Some&& some) {
  const long long pieces = p.groups[p.n] * 4;
  const int lane = threadIdx.x & 31;
  for (long long c = ((long long)blockIdx.x * 8 + dev::warp_uniform()) * kCkptChunk; c < pieces;
       c += (long long)gridDim.x * 8 * kCkptChunk) {
    const int t = ckpt_tensor(p, c >> 2);
    if (c + kCkptChunk <= p.groups[t + 1] * 4)
      one(CkptPlaces<true>{t, (c - p.groups[t] * 4 + lane) * 8});
    else  // the chunk reaches into the next tensor or past the last piece
      some(ckpt_places(p, c, lane));
  }
}

// Bound by HBM: 2 bytes read and 33/32 written an element, 268 million in 125 us, 6.5 TB/s, a
// copy's rate.  (Places worked out for each piece: 158 us, bound by issue.  Products and clamps in
// bf16 pairs as well: 167.)
__global__ void __launch_bounds__(256) dash_ckpt8_pack_kernel(const __grid_constant__ CkptParams p) {
  const int lane = threadIdx.x & 31;
  ckpt_chunks(p, [&](const CkptPlaces<true>& at) { ckpt_pack_chunk(p, at, lane); },
              [&](const CkptPlaces<false>& at) { ckpt_pack_chunk(p, at, lane); });
}

// Bound by HBM: 268 million elements in 119 us, 6.8 TB/s.  (Places worked out for each piece: 135.)
__global__ void __launch_bounds__(256) dash_ckpt8_unpack_kernel(const __grid_constant__ CkptParams p) {
  ckpt_chunks(p, [&](const CkptPlaces<true>& at) { ckpt_unpack_chunk(p, at); },
              [&](const CkptPlaces<false>& at) { ckpt_unpack_chunk(p, at); });
}

}  // namespace dash
