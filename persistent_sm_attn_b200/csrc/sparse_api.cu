// C ABI of block selection, block-sparse attention and 8-bit checkpoints: argument checks,
// workspace layouts, TMA descriptors and launches.  The operations are documented in
// include/dash_attn.h.  Nothing here allocates device memory: plans and workspaces are the
// caller's, so the calls can be captured into graphs from their first use on.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <climits>
#include <cmath>
#include <cstdint>
#include <map>
#include <mutex>
#include <utility>

#include "../../include/dash_attn.h"
#include "block_select.cuh"
#include "ckpt8.cuh"
#include "internal.h"
#include "sparse_bwd.cuh"
#include "sparse_fwd.cuh"
#include "sparse_plan.cuh"
#include "sparse_token.cuh"

namespace {

using dash::PlanShape;
using dash::PlanView;

#define DASH_CUDA(call)                              \
  do {                                               \
    if ((call) != cudaSuccess) return DASH_ERR_CUDA; \
  } while (0)

// ------------------------------------------------------------------ error words
// Two words per stream, [0] error bits and [1] abort flag, in module memory: no allocation.
// The flag goes up with the first wait that runs out and ends the later waits of the
// stream's launches quickly; dash_attn_sync_status reads and clears both.  Past kSlots
// streams of a device, streams share words (a timeout is then reported to either).
constexpr int kSlots = 256;
static __device__ unsigned g_sparse_words[2 * kSlots];
std::mutex g_mu;
std::map<std::pair<int, uintptr_t>, int> g_slots;
std::map<int, std::pair<unsigned*, int>> g_base;  // device: address of the words, slots given

int words_for(int dev, void* stream, bool create, unsigned** out) {
  std::lock_guard<std::mutex> lk(g_mu);
  auto it = g_slots.find({dev, reinterpret_cast<uintptr_t>(stream)});
  auto& base = g_base[dev];
  if (it == g_slots.end()) {
    *out = nullptr;
    if (!create) return DASH_OK;
    if (!base.first) {
      void* ptr = nullptr;
      if (cudaGetSymbolAddress(&ptr, g_sparse_words) != cudaSuccess || !ptr) {
        cudaGetLastError();
        return DASH_ERR_CUDA;
      }
      base.first = static_cast<unsigned*>(ptr);
    }
    it = g_slots.emplace(std::make_pair(dev, reinterpret_cast<uintptr_t>(stream)),
                         base.second++ % kSlots).first;
  }
  *out = base.first + 2 * it->second;
  return DASH_OK;
}

// Shared memory a kernel may use, raised once per kernel and device (the call costs a
// microsecond) to the most that any launch of it takes: launches of two threads cannot lower
// it for each other.  `done` is the kernel's own array.
constexpr int kMaxDevices = 64;
template <class K>
int allow_smem(K* kern, int most, std::atomic<bool> (&done)[kMaxDevices]) {
  int dev = 0;
  DASH_CUDA(cudaGetDevice(&dev));
  if (dev >= kMaxDevices || !done[dev].load(std::memory_order_acquire)) {
    DASH_CUDA(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, most));
    if (dev < kMaxDevices) done[dev].store(true, std::memory_order_release);
  }
  return DASH_OK;
}
#define DASH_ALLOW_SMEM(kern, most)                       \
  do {                                                    \
    static std::atomic<bool> allowed[kMaxDevices];        \
    const int allow_rc = allow_smem(kern, most, allowed); \
    if (allow_rc) return allow_rc;                        \
  } while (0)

// ------------------------------------------------------------------ checks
bool aligned16(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool aligned4_or_null(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Strides (batch, head, row) of a [B,H,S,D] operand in elements; null means contiguous.
// A dimension of extent 1 has no stride of its own.
struct Strides {
  long long b, h, s;
};
int take_strides(const long long* in, int B, int H, int S, int D, Strides* out) {
  const Strides dense{(long long)H * S * D, (long long)S * D, D};
  *out = dense;
  if (!in) return DASH_OK;
  // (a dense stride may be 0, of an operand without elements)
  auto take = [&](int extent, long long x, long long* to) {
    if (extent <= 1) return true;
    *to = x;
    return x >= 8 && x % 8 == 0 && x < (1LL << 38);
  };
  return take(B, in[0], &out->b) && take(H, in[1], &out->h) && take(S, in[2], &out->s)
             ? DASH_OK : DASH_ERR_INVALID_ARG;
}

// What keeps ceil(Sk / block), the places of a tile's picks and the like within 32 bits
constexpr int kMostKeys = 1 << 30, kMostPicks = 1 << 20;
int check_block(int block, int topk) {
  if (block < dash::kUnit || block % dash::kUnit != 0 || topk < 1) return DASH_ERR_INVALID_ARG;
  return block > kMostKeys || topk > kMostPicks ? DASH_ERR_UNSUPPORTED : DASH_OK;
}

// A block longer than the sequence is one of its whole units: what a kernel walks by blocks
// then ends with the keys
int trim_block(int block, int Sk) {
  return (int)std::min((long long)block, ((long long)Sk + dash::kUnit - 1) / dash::kUnit * dash::kUnit);
}

int check_heads(int B, int H, int Hkv, int Sq, int Sk) {
  if (B < 0 || H < 0 || Sq < 0 || Sk < 1) return DASH_ERR_INVALID_ARG;
  if (Sk > kMostKeys) return DASH_ERR_UNSUPPORTED;
  if (B == 0 || H == 0) return DASH_OK;
  if (Hkv < 1 || H % Hkv != 0) return DASH_ERR_INVALID_ARG;
  if (H / Hkv > dash::kTileRows) return DASH_ERR_UNSUPPORTED;
  if ((long long)B * H * Sq >= (1LL << 31) || (long long)B * Hkv > 65535)
    return DASH_ERR_UNSUPPORTED;
  return DASH_OK;
}

long long align256(long long x) { return (x + 255) & ~255LL; }

int plan_shape(int B, int H, int Hkv, int Sq, int Sk, int block, int topk, int causal,
               PlanShape* s) {
  int rc = check_heads(B, H, Hkv, Sq, Sk);
  if (rc) return rc;
  if ((rc = check_block(block, topk))) return rc;
  if (causal != 0 && causal != 1) return DASH_ERR_INVALID_ARG;
  *s = PlanShape{};
  s->B = B, s->H = H, s->Hkv = Hkv, s->Sq = Sq, s->Sk = Sk;
  s->block = trim_block(block, Sk), s->topk = topk, s->causal = causal;
  if (B == 0 || H == 0 || Sq == 0) return DASH_OK;
  s->G = H / Hkv;
  s->T = dash::kTileRows / s->G;
  s->W = (s->T + 31) / 32;
  s->NT = (Sq + s->T - 1) / s->T;
  s->nu = (int)(((long long)Sk + dash::kUnit - 1) / dash::kUnit);
  const long long picks = (long long)std::min(s->T, Sq) * topk * (s->block / dash::kUnit);
  s->U = (int)std::min((long long)s->nu, picks);
  s->NW = (s->nu + 31) / 32;
  // the plan kernel holds one tile's masks in shared memory
  if ((long long)s->nu * s->W * 4 > 200 * 1024) return DASH_ERR_UNSUPPORTED;
  const long long tiles = (long long)B * Hkv * s->NT;
  if (tiles > 0x7fffffffLL) return DASH_ERR_UNSUPPORTED;
  long long at = 0;
  auto put = [&](long long* off, long long words) {
    *off = at;
    at = align256(at + 4 * words);
  };
  put(&s->off_len, B);
  put(&s->off_start, B);
  put(&s->off_count, tiles);
  put(&s->off_unit, tiles * s->U);
  put(&s->off_mask, tiles * s->U * s->W);
  put(&s->off_pres, tiles * s->NW);
  put(&s->off_pre, tiles * s->NW);
  s->bytes = at;
  return DASH_OK;
}

PlanView plan_view(const PlanShape& s, const void* plan) {
  const char* p = static_cast<const char*>(plan);
  auto i = [&](long long off) { return reinterpret_cast<const int*>(p + off); };
  auto u = [&](long long off) { return reinterpret_cast<const uint32_t*>(p + off); };
  return PlanView{i(s.off_len), i(s.off_start), i(s.off_count), i(s.off_unit),
                  u(s.off_mask), u(s.off_pres), i(s.off_pre)};
}

// ------------------------------------------------------------------ TMA descriptors
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) !=
            cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeTiledFn>(p);
  }();
  return fn;
}

// [B][H][S][D] bf16 with any strides, viewed in boxes of 64 columns x rows x heads with the
// 128-byte swizzle; rows past S read as zero.
int make_tmap4(CUtensorMap* m, const void* base, int B, int H, int S, int D, const Strides& st,
               int rows, int heads) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return DASH_ERR_CUDA;
  cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)S, (cuuint64_t)H, (cuuint64_t)B};
  cuuint64_t strides[3] = {(cuuint64_t)st.s * 2, (cuuint64_t)st.h * 2, (cuuint64_t)st.b * 2};
  cuuint32_t box[4] = {64, (cuuint32_t)rows, (cuuint32_t)heads, 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides,
                  box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? DASH_OK : DASH_ERR_CUDA;
}

// The same with boxes of 64 columns x heads x rows: row t G + g of a tile is row t, head g.
int make_tmap4_rows(CUtensorMap* m, const void* base, int B, int H, int S, int D, const Strides& st,
                    int rows, int heads) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return DASH_ERR_CUDA;
  cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)H, (cuuint64_t)S, (cuuint64_t)B};
  cuuint64_t strides[3] = {(cuuint64_t)st.h * 2, (cuuint64_t)st.s * 2, (cuuint64_t)st.b * 2};
  cuuint32_t box[4] = {64, (cuuint32_t)heads, (cuuint32_t)rows, 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides,
                  box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? DASH_OK : DASH_ERR_CUDA;
}

// Parts that a tile's list is split into: enough CTAs for two on each of 148 SMs, and at
// least two units a part.
int fwd_splits(const PlanShape& s) {
  const long long ctas = (long long)s.B * s.Hkv * s.NT;
  const long long want = (2 * 148 + ctas - 1) / ctas;
  return (int)std::max(1LL, std::min({want, (long long)(s.U + 1) / 2, 64LL}));
}

// Loads of a CTA: all, or with a fault that dash_inject_fault(2) has armed the first few, so that
// waits run out with work in flight.
int take_loads() { return dash::take_sparse_fault() ? 3 : INT_MAX; }

float scale_or_default(float scale, int D) { return scale > 0.f ? scale : 1.0f / sqrtf((float)D); }

template <int D>
int launch_sparse_fwd(const void* q, const void* k, const void* v, const Strides* st,
                      const PlanShape& s, const void* plan, void* o, float* lse, void* work,
                      float scale, cudaStream_t stream) {
  using C = dash::SparseFwdCfg<D>;
  int dev = 0;
  DASH_CUDA(cudaGetDevice(&dev));
  unsigned* words = nullptr;
  int rc = words_for(dev, stream, true, &words);
  if (rc) return rc;
  CUtensorMap tq, tk, tv;
  if ((rc = make_tmap4_rows(&tq, q, s.B, s.H, s.Sq, D, st[0], s.T, s.G)) ||
      (rc = make_tmap4(&tk, k, s.B, s.Hkv, s.Sk, D, st[1], dash::kUnit, 1)) ||
      (rc = make_tmap4(&tv, v, s.B, s.Hkv, s.Sk, D, st[2], dash::kUnit, 1)))
    return rc;
  const long long rows = (long long)s.B * s.H * s.Sq;
  dash::SparseFwdParams p{};
  p.plan = plan_view(s, plan);
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.splits = fwd_splits(s);
  if (p.splits > 1) {
    if (!aligned16(work)) return DASH_ERR_INVALID_ARG;
    p.part_o = static_cast<float*>(work);
    p.part_l = p.part_o + rows * D * p.splits;
  }
  p.err = words;
  p.H = s.H, p.Hkv = s.Hkv, p.Sq = s.Sq, p.Sk = s.Sk, p.G = s.G, p.T = s.T, p.W = s.W;
  p.NT = s.NT, p.U = s.U, p.causal = s.causal;
  p.loads = take_loads();
  p.scale_log2 = scale_or_default(scale, D) * 1.4426950408889634f;
  p.spin_ns = (unsigned long long)dash::spin_limit_us() * 1000ull;
  const long long grid = (long long)s.B * s.Hkv * s.NT * p.splits;
  if (grid > 0x7fffffffLL) return DASH_ERR_UNSUPPORTED;
  auto kern = dash::dash_sparse_fwd_kernel<D>;
  DASH_ALLOW_SMEM(kern, C::kSmemBytes);
  kern<<<(unsigned)grid, C::kThreads, C::kSmemBytes, stream>>>(tq, tk, tv, p);
  DASH_CUDA(cudaGetLastError());
  if (p.splits > 1) {
    dash::dash_sparse_join_kernel<D><<<(unsigned)((rows + 3) / 4), 128, 0, stream>>>(
        p.part_o, p.part_l, p.o, p.lse, rows, p.splits);
    DASH_CUDA(cudaGetLastError());
  }
  return DASH_OK;
}

// CTAs of a cluster that share a token's picks: more than one while there are fewer clusters
// than SMs, with a chunk at least for each warp.  (64 tokens of 8 K/V heads, 16 picks of 64:
// 53 us with one CTA, 68 with two, 89 with four; one token: 8.7 us with eight.)
int token_cluster(long long units, int topk, int block) {
  const long long most = (long long)topk * (block / dash::kTokenKeys) / dash::kTokenWarps;
  int cs = 1;
  while (cs < 8 && units * cs < 148 && 2 * cs <= most) cs *= 2;
  return cs;
}

template <int D>
int launch_sparse_token(dash::SparseTokenParams& p, long long units, cudaStream_t stream) {
  using C = dash::SparseTokenCfg<D>;
  const int cs = token_cluster(units, p.topk, p.block);
  if (units * cs > 0x7fffffffLL) return DASH_ERR_UNSUPPORTED;
  auto kern = dash::dash_sparse_token_kernel<D>;
  const int smem = C::smem(p.topk, p.nb);
  DASH_ALLOW_SMEM(kern, C::smem(dash::kTokenTopk, dash::kTokenBlocks));
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(units * cs));
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = stream;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = (unsigned)cs;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  DASH_CUDA(cudaLaunchKernelEx(&cfg, kern, p));
  return DASH_OK;
}

// Workspace of the backward (offsets in bytes).
struct BwdWork {
  long long units, tokens, slots, off_delta, off_count, off_off, off_token, off_item, off_slot0,
      off_head, off_part, bytes;
};
BwdWork bwd_work(const PlanShape& s, int D) {
  BwdWork w{};
  w.units = (long long)s.B * s.Hkv * s.nu;
  // a token lists a unit at most once, and a unit of a block per pick
  w.tokens = (long long)s.B * s.Hkv * s.Sq *
             std::min((long long)s.nu, (long long)s.topk * (s.block / dash::kUnit));
  // a cut unit of n > C tiles has ceil(n / C) <= 2 n / C parts, and C >= tiles / kStretches
  const long long most = w.units + w.tokens / s.T;
  w.slots = std::min(2LL * dash::kStretches, 2 * most / dash::kMinStretch + 1);
  long long at = 0;
  auto put = [&](long long* off, long long bytes) {
    *off = at;
    at = align256(at + bytes);
  };
  put(&w.off_delta, (long long)s.B * s.H * s.Sq * 4);
  put(&w.off_count, w.units * 4);
  put(&w.off_off, w.units * 4);
  put(&w.off_token, w.tokens * 4);
  put(&w.off_item, (w.units + dash::kStretches) * (long long)sizeof(dash::SparseItem));  // sum of ceil(n / C)
  put(&w.off_slot0, w.units * 4);
  put(&w.off_head, 8);
  put(&w.off_part, w.slots * 2 * dash::kUnit * D * 4);
  w.bytes = at;
  return w;
}

template <int D>
constexpr int kUnitElems = dash::kUnit * D;

// Whether dS keeps a second bf16 part.  It takes much the same off at any length: unit normals,
// causal sequences of 64, 768 and 2048 keys, dQ off by 0.0020, 0.0018 and 0.0018 of its norm in
// place of 0.0026, 0.0025 and 0.0025 (the rounding of the result itself is 0.0017); dK alike at
// D = 64, while at D = 128 shared memory has no room for its part and dK stays at 0.0025.  And it
// costs much the same: a backward of 8 heads of 8k takes 172 us for 156 at 256 picked keys and
// 264 for 237 at 1024 (D = 64), 208 for 191 and 319 for 293 (D = 128).  So the limit is no
// turning point but a choice: few keys, where Delta of the rounded O is the coarsest and the error
// the largest, get it, and the others stay at what dV has from one bf16 part of P.
bool sparse_low_part(const PlanShape& s) {
  return std::min((long long)s.Sk, (long long)s.topk * s.block) <= 768;
}

template <int D>
int launch_sparse_bwd(const void* q, const void* k, const void* v, const void* dout,
                      const Strides* st, const PlanShape& s, const void* plan, const void* o,
                      const float* lse, void* dq, void* dk, void* dv, void* work, float scale,
                      cudaStream_t stream) {
  using Cq = dash::SparseDqCfg<D>;
  using Ck = dash::SparseDkvCfg<D>;
  int dev = 0, sms = 0;
  DASH_CUDA(cudaGetDevice(&dev));
  DASH_CUDA(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
  unsigned* words = nullptr;
  int rc = words_for(dev, stream, true, &words);
  if (rc) return rc;
  const BwdWork w = bwd_work(s, D);
  if (w.units > 0x7fffffffLL || w.tokens > 0x7fffffffLL) return DASH_ERR_UNSUPPORTED;
  CUtensorMap tq, tk, tv, tdo;
  if ((rc = make_tmap4_rows(&tq, q, s.B, s.H, s.Sq, D, st[0], s.T, s.G)) ||
      (rc = make_tmap4(&tk, k, s.B, s.Hkv, s.Sk, D, st[1], dash::kUnit, 1)) ||
      (rc = make_tmap4(&tv, v, s.B, s.Hkv, s.Sk, D, st[2], dash::kUnit, 1)) ||
      (rc = make_tmap4_rows(&tdo, dout, s.B, s.H, s.Sq, D, st[3], s.T, s.G)))
    return rc;
  char* base = static_cast<char*>(work);
  const PlanView view = plan_view(s, plan);
  const float sc = scale_or_default(scale, D);
  const unsigned long long spin = (unsigned long long)dash::spin_limit_us() * 1000ull;

  dash::SparseDeltaParams dl{};
  dl.o = static_cast<const __nv_bfloat16*>(o);
  dl.dout = static_cast<const __nv_bfloat16*>(dout);
  dl.ob = st[3].b, dl.oh = st[3].h, dl.os = st[3].s;
  dl.delta = reinterpret_cast<float*>(base + w.off_delta);
  dl.H = s.H, dl.Sq = s.Sq, dl.rows = (long long)s.B * s.H * s.Sq;
  constexpr int kDeltaRows = 4 * 256 / (D / 8);
  dash::dash_sparse_delta_kernel<D>
      <<<(unsigned)((dl.rows + kDeltaRows - 1) / kDeltaRows), 256, 0, stream>>>(dl);
  DASH_CUDA(cudaGetLastError());

  dash::SparseDqParams a{};
  a.plan = view;
  a.lse = lse;
  a.dq = static_cast<__nv_bfloat16*>(dq);
  a.delta = dl.delta;
  a.err = words;
  a.Hkv = s.Hkv, a.Sq = s.Sq, a.Sk = s.Sk, a.G = s.G, a.T = s.T, a.W = s.W;
  a.NT = s.NT, a.U = s.U, a.causal = s.causal;
  a.tiles = s.B * s.Hkv * s.NT;
  a.loads = take_loads();
  a.scale = sc;
  a.scale_log2 = sc * 1.4426950408889634f;
  a.spin_ns = spin;
  const bool low = sparse_low_part(s);
  auto kq = low ? dash::dash_sparse_dq_kernel<D, true> : dash::dash_sparse_dq_kernel<D, false>;
  if (low) DASH_ALLOW_SMEM(kq, Cq::kSmemBytes);
  else DASH_ALLOW_SMEM(kq, Cq::kSmemBytes);
  kq<<<std::min(sms, a.tiles), Cq::kThreads, Cq::kSmemBytes, stream>>>(tq, tdo, tk, tv, a);
  DASH_CUDA(cudaGetLastError());

  dash::InverseParams iv{};
  iv.plan = view;
  iv.count = reinterpret_cast<int*>(base + w.off_count);
  iv.off = reinterpret_cast<int*>(base + w.off_off);
  iv.token = reinterpret_cast<int*>(base + w.off_token);
  iv.nu = s.nu, iv.NW = s.NW, iv.NT = s.NT, iv.T = s.T, iv.U = s.U, iv.W = s.W;
  iv.units = w.units;
  dash::dash_sparse_count_kernel<<<(unsigned)((w.units + 3) / 4), 128, 0, stream>>>(iv);
  DASH_CUDA(cudaGetLastError());

  dash::ItemParams im{};
  im.count = iv.count;
  im.off = iv.off;
  im.item = reinterpret_cast<dash::SparseItem*>(base + w.off_item);
  im.slot0 = reinterpret_cast<int*>(base + w.off_slot0);
  im.head = reinterpret_cast<int*>(base + w.off_head);
  im.T = s.T, im.nu = s.nu, im.Hkv = s.Hkv;
  im.units = w.units;
  dash::dash_sparse_items_kernel<<<1, 1024, 0, stream>>>(im);
  DASH_CUDA(cudaGetLastError());
  dash::dash_sparse_fill_kernel<<<(unsigned)w.units, 128, 0, stream>>>(iv);
  DASH_CUDA(cudaGetLastError());

  dash::SparseDkvParams c{};
  c.plan = view;
  c.token = iv.token;
  c.q = static_cast<const __nv_bfloat16*>(q);
  c.dout = static_cast<const __nv_bfloat16*>(dout);
  c.qb = st[0].b, c.qh = st[0].h, c.qs = st[0].s;
  c.ob = st[3].b, c.oh = st[3].h, c.os = st[3].s;
  c.item = im.item;
  c.head = im.head;
  c.lse = lse;
  c.delta = a.delta;
  c.dk = static_cast<__nv_bfloat16*>(dk);
  c.dv = static_cast<__nv_bfloat16*>(dv);
  c.part = reinterpret_cast<float*>(base + w.off_part);
  c.err = words;
  c.Hkv = s.Hkv, c.Sq = s.Sq, c.Sk = s.Sk, c.G = s.G, c.T = s.T;
  c.nu = s.nu, c.causal = s.causal;
  c.loads = a.loads;
  c.scale = sc;
  c.scale_log2 = a.scale_log2;
  c.spin_ns = spin;
  auto kk = D == 64 && low ? dash::dash_sparse_dkdv_kernel<D, D == 64>
                           : dash::dash_sparse_dkdv_kernel<D, false>;
  if (low) DASH_ALLOW_SMEM(kk, Ck::kSmemBytes);
  else DASH_ALLOW_SMEM(kk, Ck::kSmemBytes);
  kk<<<sms, Ck::kThreads, Ck::kSmemBytes, stream>>>(tk, tv, c);
  DASH_CUDA(cudaGetLastError());

  dash::FinishParams f{};
  f.slot0 = im.slot0;
  f.count = iv.count;
  f.head = im.head;
  f.part = c.part;
  f.dk = c.dk, f.dv = c.dv;
  f.Sk = s.Sk, f.D = D, f.nu = s.nu, f.T = s.T;
  dash::dash_sparse_finish_kernel<<<dim3((unsigned)w.units, kUnitElems<D> / 1024), 256, 0, stream>>>(f);
  DASH_CUDA(cudaGetLastError());
  return DASH_OK;
}

int ckpt_params(const void* const* src, void* const* dst, signed char* const* exps,
                const long long* elems, int n, dash::CkptParams* p) {
  if (!src || !dst || !exps || !elems || n < 1 || n > dash::kCkptTensors)
    return DASH_ERR_INVALID_ARG;
  p->n = n;
  p->groups[0] = 0;
  for (int t = 0; t < n; ++t) {
    if (elems[t] < 0 || elems[t] % 32 != 0 || elems[t] > (1LL << 40)) return DASH_ERR_INVALID_ARG;
    if (elems[t] > 0 && (!aligned16(src[t]) || !aligned16(dst[t]) || !exps[t]))
      return DASH_ERR_INVALID_ARG;
    p->src[t] = src[t];
    p->dst[t] = dst[t];
    p->exps[t] = reinterpret_cast<int8_t*>(exps[t]);
    p->groups[t + 1] = p->groups[t] + elems[t] / 32;
  }
  return DASH_OK;
}
// A CTA takes 1024 pieces of 8 elements at a time: packing with at most 32 CTAs for each of 148
// SMs and then a stride (268 million elements: 125 us, 130 with a CTA for every 1024 pieces),
// reading back, which keeps less for each piece, with a CTA for all (119 us, 125 with a stride).
unsigned ckpt_grid(const dash::CkptParams& p, long long most) {
  return (unsigned)std::min((p.groups[p.n] * 4 + 1023) / 1024, most);
}

template <int D, int QT, int NL>
int launch_select_tile(const dash::SelectParams& p, int B, cudaStream_t stream) {
  using C = dash::SelectCfg<D, QT>;
  auto kern = dash::dash_block_select_kernel<D, QT, NL>;
  const int smem = C::smem(p.nb);
  DASH_ALLOW_SMEM(kern, C::smem(NL * 32));  // NL blocks a lane
  kern<<<dim3((p.Sq + QT - 1) / QT, B * p.Hkv), C::kThreads, smem, stream>>>(p);
  DASH_CUDA(cudaGetLastError());
  return DASH_OK;
}

// A CTA per query below 16 queries a head: an MMA tile would be mostly empty.  Otherwise as
// many queries a CTA as their scores leave room for in shared memory (two CTAs an SM up to
// 448 blocks at D = 128 and 640 at D = 64, one beyond).
template <int D>
int launch_select(const dash::SelectParams& p, int B, cudaStream_t stream) {
  if (p.Sq < 16) {
    auto kern = p.nb <= 256 ? dash::dash_block_select_token_kernel<D, 8>
                            : dash::dash_block_select_token_kernel<D, 128>;
    kern<<<dim3(p.Sq, B * p.Hkv), 256, (size_t)p.nb * 4, stream>>>(p);
    DASH_CUDA(cudaGetLastError());
    return DASH_OK;
  }
  if (p.nb <= 64) return launch_select_tile<D, 32, 2>(p, B, stream);
  if (p.nb <= 256) return launch_select_tile<D, 32, 8>(p, B, stream);
  if (p.nb <= 512) return launch_select_tile<D, 32, 16>(p, B, stream);
  if (p.nb <= 1024) return launch_select_tile<D, 32, 32>(p, B, stream);
  if (p.nb <= 2048) return launch_select_tile<D, 16, 64>(p, B, stream);
  return launch_select_tile<D, 8, 128>(p, B, stream);
}

}  // namespace

namespace dash {
int sparse_take_status(int dev, void* stream) {
  unsigned* words = nullptr;
  int rc = words_for(dev, stream, false, &words);
  if (rc || !words) return rc;
  unsigned h = 0;
  DASH_CUDA(cudaMemcpy(&h, words, sizeof(unsigned), cudaMemcpyDeviceToHost));
  if (!h) return DASH_OK;
  DASH_CUDA(cudaMemset(words, 0, 2 * sizeof(unsigned)));
  return (h & dev::ERR_TIMEOUT) ? DASH_ERR_TIMEOUT : DASH_ERR_UNSUPPORTED;
}
}  // namespace dash

using dash::no_throw;

extern "C" {

int dash_block_means(const void* k, const long long* k_strides, float* means, const int* kv_len,
                     const int* start, int B, int Hkv, int Sk, int D, int block, void* stream) {
  return no_throw([&]() -> int {
    if (B < 0 || Hkv < 0 || Sk < 1) return DASH_ERR_INVALID_ARG;
    int rc = check_block(block, 1);
    if (rc) return rc;
    if (D != 64 && D != 128) return DASH_ERR_UNSUPPORTED;
    if (Sk > kMostKeys || (long long)B * Hkv > 65535) return DASH_ERR_UNSUPPORTED;
    Strides st;
    rc = take_strides(k_strides, B, Hkv, Sk, D, &st);
    if (rc) return rc;
    if (B == 0 || Hkv == 0) return DASH_OK;
    if (!aligned16(k) || !aligned4(means) || !aligned4_or_null(kv_len) || !aligned4_or_null(start))
      return DASH_ERR_INVALID_ARG;
    dash::MeansParams p;
    p.k = static_cast<const __nv_bfloat16*>(k);
    p.sb = st.b, p.sh = st.h, p.ss = st.s;
    p.means = means;
    p.kv_len = kv_len;
    p.start = start;
    p.Hkv = Hkv, p.Sk = Sk, p.D = D, p.block = trim_block(block, Sk);
    p.nb = (Sk + p.block - 1) / p.block;
    dash::dash_block_means_kernel<<<dim3(start ? std::min(p.nb, 2) : p.nb, B * Hkv), 128, 0,
                                    static_cast<cudaStream_t>(stream)>>>(p);
    DASH_CUDA(cudaGetLastError());
    return DASH_OK;
  }, DASH_ERR_OOM, DASH_ERR_INVALID_ARG);
}

int dash_block_select(const void* q, const long long* q_strides, const float* means, int* idx,
                      const int* kv_len, const int* q_start, int B, int H, int Hkv, int Sq, int Sk,
                      int D, int block, int topk, int causal, int sink, int local, void* stream) {
  return no_throw([&]() -> int {
    int rc = check_heads(B, H, Hkv, Sq, Sk);
    if (rc) return rc;
    if ((rc = check_block(block, topk))) return rc;
    if (sink < 0 || local < 0 || (long long)sink + local > topk || (causal != 0 && causal != 1))
      return DASH_ERR_INVALID_ARG;
    if (D != 64 && D != 128) return DASH_ERR_UNSUPPORTED;
    Strides st;
    if ((rc = take_strides(q_strides, B, H, Sq, D, &st))) return rc;
    if (B == 0 || Sq == 0 || (H == 0 && Hkv == 0)) return DASH_OK;
    if (H == 0) return DASH_ERR_INVALID_ARG;  // places to fill and nothing to score by
    if (!aligned16(q) || !aligned16(means) || !aligned4(idx) || !aligned4_or_null(kv_len) ||
        !aligned4_or_null(q_start))
      return DASH_ERR_INVALID_ARG;
    dash::SelectParams p;
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.sb = st.b, p.sh = st.h, p.ss = st.s;
    p.means = means;
    p.idx = idx;
    p.kv_len = kv_len;
    p.q_start = q_start;
    p.Hkv = Hkv, p.G = H / Hkv, p.Sq = Sq, p.Sk = Sk, p.topk = topk;
    p.block = trim_block(block, Sk);
    p.nb = (Sk + p.block - 1) / p.block;
    p.causal = causal, p.sink = sink, p.local = local;
    if (p.nb > 4096) return DASH_ERR_UNSUPPORTED;  // the queries' scores lie in shared memory
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    return D == 64 ? launch_select<64>(p, B, cs) : launch_select<128>(p, B, cs);
  }, DASH_ERR_OOM, DASH_ERR_INVALID_ARG);
}

long long dash_sparse_plan_bytes(int B, int H, int Hkv, int Sq, int Sk, int block, int topk) {
  PlanShape s;
  const int rc = plan_shape(B, H, Hkv, Sq, Sk, block, topk, 0, &s);
  return rc ? -(long long)rc : s.bytes;
}

int dash_sparse_plan(const int* idx, const int* kv_len, const int* q_start, void* plan, int B,
                     int H, int Hkv, int Sq, int Sk, int block, int topk, int causal,
                     void* stream) {
  return no_throw([&]() -> int {
    dash::PlanParams p{};
    int rc = plan_shape(B, H, Hkv, Sq, Sk, block, topk, causal, &p.s);
    if (rc) return rc;
    if (B == 0 || H == 0 || Sq == 0) return DASH_OK;
    if (!aligned4(idx) || !aligned4_or_null(kv_len) || !aligned4_or_null(q_start) ||
        !aligned16(plan))
      return DASH_ERR_INVALID_ARG;
    p.idx = idx;
    p.kv_len = kv_len;
    p.q_start = q_start;
    char* at = static_cast<char*>(plan);
    auto i = [&](long long off) { return reinterpret_cast<int*>(at + off); };
    p.len = i(p.s.off_len), p.start = i(p.s.off_start), p.count = i(p.s.off_count);
    p.unit = i(p.s.off_unit), p.pre = i(p.s.off_pre);
    p.mask = reinterpret_cast<uint32_t*>(at + p.s.off_mask);
    p.pres = reinterpret_cast<uint32_t*>(at + p.s.off_pres);
    const int smem = p.s.nu * p.s.W * 4;
    auto kern = dash::dash_sparse_plan_kernel;
    DASH_ALLOW_SMEM(kern, 200 * 1024);
    kern<<<(unsigned)((long long)B * Hkv * p.s.NT), 128, smem, static_cast<cudaStream_t>(stream)>>>(p);
    DASH_CUDA(cudaGetLastError());
    return DASH_OK;
  }, DASH_ERR_OOM, DASH_ERR_INVALID_ARG);
}

long long dash_attn_sparse_work_bytes(int B, int H, int Hkv, int Sq, int Sk, int D, int block,
                                      int topk, int backward) {
  PlanShape s;
  const int rc = plan_shape(B, H, Hkv, Sq, Sk, block, topk, 0, &s);
  if (rc) return -(long long)rc;
  if (D != 64 && D != 128) return -(long long)DASH_ERR_UNSUPPORTED;
  if (B == 0 || H == 0 || Sq == 0) return 0;
  if (backward) return bwd_work(s, D).bytes;
  const long long rows = (long long)B * H * Sq;
  const int n = fwd_splits(s);
  return n > 1 ? rows * n * (D + 1) * 4 : 0;
}

int dash_attn_sparse_fwd(const void* q, const void* k, const void* v, const long long* strides,
                         const void* plan, void* o, float* lse, void* work, int B, int H, int Hkv,
                         int Sq, int Sk, int D, int block, int topk, int causal, float scale,
                         void* stream) {
  return no_throw([&]() -> int {
    PlanShape s;
    int rc = plan_shape(B, H, Hkv, Sq, Sk, block, topk, causal, &s);
    if (rc) return rc;
    if (D != 64 && D != 128) return DASH_ERR_UNSUPPORTED;
    if (!(scale >= 0.f) || std::isinf(scale)) return DASH_ERR_INVALID_ARG;
    Strides st[3];
    if ((rc = take_strides(strides, B, H, Sq, D, &st[0])) ||
        (rc = take_strides(strides ? strides + 3 : nullptr, B, Hkv, Sk, D, &st[1])) ||
        (rc = take_strides(strides ? strides + 6 : nullptr, B, Hkv, Sk, D, &st[2])))
      return rc;
    if (B == 0 || H == 0 || Sq == 0) return DASH_OK;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned4(lse) ||
        !aligned16(plan))
      return DASH_ERR_INVALID_ARG;
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    return D == 64 ? launch_sparse_fwd<64>(q, k, v, st, s, plan, o, lse, work, scale, cs)
                   : launch_sparse_fwd<128>(q, k, v, st, s, plan, o, lse, work, scale, cs);
  }, DASH_ERR_OOM, DASH_ERR_INVALID_ARG);
}

int dash_attn_sparse_tokens(const void* q, const void* k, const void* v, const long long* strides,
                            const int* idx, const int* kv_len, const int* q_start, void* o,
                            float* lse, int B, int H, int Hkv, int Sq, int Sk, int D, int block,
                            int topk, int causal, float scale, void* stream) {
  return no_throw([&]() -> int {
    int rc = check_heads(B, H, Hkv, Sq, Sk);
    if (rc) return rc;
    if ((rc = check_block(block, topk))) return rc;
    if ((causal != 0 && causal != 1) || !(scale >= 0.f) || std::isinf(scale))
      return DASH_ERR_INVALID_ARG;
    if (D != 64 && D != 128) return DASH_ERR_UNSUPPORTED;
    Strides st[3];
    if ((rc = take_strides(strides, B, H, Sq, D, &st[0])) ||
        (rc = take_strides(strides ? strides + 3 : nullptr, B, Hkv, Sk, D, &st[1])) ||
        (rc = take_strides(strides ? strides + 6 : nullptr, B, Hkv, Sk, D, &st[2])))
      return rc;
    if (B == 0 || H == 0 || Sq == 0) return DASH_OK;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned4(lse) ||
        !aligned4(idx) || !aligned4_or_null(kv_len) || !aligned4_or_null(q_start))
      return DASH_ERR_INVALID_ARG;
    dash::SparseTokenParams p{};
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.k = static_cast<const __nv_bfloat16*>(k);
    p.v = static_cast<const __nv_bfloat16*>(v);
    p.qb = st[0].b, p.qh = st[0].h, p.qs = st[0].s;
    p.kb = st[1].b, p.kh = st[1].h, p.ks = st[1].s;
    p.vb = st[2].b, p.vh = st[2].h, p.vs = st[2].s;
    p.idx = idx;
    p.kv_len = kv_len;
    p.q_start = q_start;
    p.o = static_cast<__nv_bfloat16*>(o);
    p.lse = lse;
    p.H = H, p.Hkv = Hkv, p.G = H / Hkv, p.RG = (p.G + 15) / 16;
    p.Sq = Sq, p.Sk = Sk, p.topk = topk, p.causal = causal;
    p.block = trim_block(block, Sk);
    p.nb = (Sk + p.block - 1) / p.block;
    if (topk > dash::kTokenTopk || p.nb > dash::kTokenBlocks) return DASH_ERR_UNSUPPORTED;
    p.scale_log2 = scale_or_default(scale, D) * 1.4426950408889634f;
    const long long units = (long long)B * Hkv * Sq * p.RG;
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    return D == 64 ? launch_sparse_token<64>(p, units, cs) : launch_sparse_token<128>(p, units, cs);
  }, DASH_ERR_OOM, DASH_ERR_INVALID_ARG);
}

int dash_attn_sparse_bwd(const void* q, const void* k, const void* v, const void* dout,
                         const long long* strides, const void* plan, const void* o,
                         const float* lse, void* dq, void* dk, void* dv, void* work, int B, int H,
                         int Hkv, int Sq, int Sk, int D, int block, int topk, int causal,
                         float scale, void* stream) {
  return no_throw([&]() -> int {
    PlanShape s;
    int rc = plan_shape(B, H, Hkv, Sq, Sk, block, topk, causal, &s);
    if (rc) return rc;
    if (D != 64 && D != 128) return DASH_ERR_UNSUPPORTED;
    if (!(scale >= 0.f) || std::isinf(scale)) return DASH_ERR_INVALID_ARG;
    Strides st[4];
    if ((rc = take_strides(strides, B, H, Sq, D, &st[0])) ||
        (rc = take_strides(strides ? strides + 3 : nullptr, B, Hkv, Sk, D, &st[1])) ||
        (rc = take_strides(strides ? strides + 6 : nullptr, B, Hkv, Sk, D, &st[2])) ||
        (rc = take_strides(strides ? strides + 9 : nullptr, B, H, Sq, D, &st[3])))
      return rc;
    if (B == 0 || H == 0) return DASH_OK;
    if (!aligned16(dk) || !aligned16(dv)) return DASH_ERR_INVALID_ARG;
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    if (Sq == 0) {  // no query reads a key
      const size_t bytes = (size_t)B * Hkv * Sk * D * 2;
      DASH_CUDA(cudaMemsetAsync(dk, 0, bytes, cs));
      DASH_CUDA(cudaMemsetAsync(dv, 0, bytes, cs));
      return DASH_OK;
    }
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(dout) ||
        !aligned4(lse) || !aligned16(dq) || !aligned16(plan) || !aligned16(work))
      return DASH_ERR_INVALID_ARG;
    return D == 64 ? launch_sparse_bwd<64>(q, k, v, dout, st, s, plan, o, lse, dq, dk, dv, work,
                                           scale, cs)
                   : launch_sparse_bwd<128>(q, k, v, dout, st, s, plan, o, lse, dq, dk, dv, work,
                                            scale, cs);
  }, DASH_ERR_OOM, DASH_ERR_INVALID_ARG);
}

int dash_ckpt8_pack(const void* const* x, void* const* m, signed char* const* e,
                    const long long* elems, int n, void* stream) {
  return no_throw([&]() -> int {
    dash::CkptParams p{};
    int rc = ckpt_params(x, m, e, elems, n, &p);
    if (rc || p.groups[n] == 0) return rc;
    dash::dash_ckpt8_pack_kernel<<<ckpt_grid(p, 148 * 32), 256, 0, static_cast<cudaStream_t>(stream)>>>(p);
    DASH_CUDA(cudaGetLastError());
    return DASH_OK;
  }, DASH_ERR_OOM, DASH_ERR_INVALID_ARG);
}

int dash_ckpt8_unpack(const void* const* m, signed char* const* e, void* const* x,
                      const long long* elems, int n, void* stream) {
  return no_throw([&]() -> int {
    dash::CkptParams p{};
    int rc = ckpt_params(m, x, e, elems, n, &p);
    if (rc || p.groups[n] == 0) return rc;
    dash::dash_ckpt8_unpack_kernel<<<ckpt_grid(p, 0x7fffffff), 256, 0, static_cast<cudaStream_t>(stream)>>>(p);
    DASH_CUDA(cudaGetLastError());
    return DASH_OK;
  }, DASH_ERR_OOM, DASH_ERR_INVALID_ARG);
}

}  // extern "C"
