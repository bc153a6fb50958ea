// Attention of one new token per request over the paged cache.
//
// Output row (b, h) is softmax(s) V over the visible keys of request b, KV head
// h / G, with s_t = cap(scale q.k_t) + slope_h (t - (L - 1)) and visible t:
// t >= L - window or t < n_sink.  "Tree Verification", "Tree Attention": the
// N = 1 case, the token's own K/V already in the cache.
//
// One CTA per row, a warp per key in turn, online softmax per warp in the log2
// domain, the warps' partial sums merged at the end.
#include <algorithm>
#include <cfloat>
#include <cmath>

#include <cuda_bf16.h>

#include "common.h"

namespace {

struct DecodeParams {
  const void* q;
  int64_t q_stride;
  const void* k_cache;
  const void* v_cache;
  int64_t num_blocks;
  int block_size;
  const int32_t* table;
  int max_blocks;
  const int32_t* seq_lens;
  int B, Hq, Hkv, G;
  float scale, softcap;
  int window, n_sink;
  const float* slopes;
  void* out;
  float* lse;
  int32_t* status;
};

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int64_t kCounterBytes = 16384;  // arrival counters, 4096 at most
constexpr int kMaxCtas = 4096;

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void store(float* p, float x) { *p = x; }
__device__ __forceinline__ void store(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

template <typename T, int D>
__global__ void __launch_bounds__(256) decode_kernel(DecodeParams p) {
  constexpr int kE = D / 32;
  const int b = blockIdx.x / p.Hq, h = blockIdx.x % p.Hq, kvh = h / p.G;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  int64_t cap = (int64_t)p.max_blocks * p.block_size;
  const int L = (int)max((int64_t)0, min((int64_t)p.seq_lens[b], cap));
  const int first = p.window > 0 ? max(0, L - p.window) : 0;
  const int sink = min(p.n_sink, first);
  const int n = sink + L - first;
  const T* q = static_cast<const T*>(p.q) + b * p.q_stride + (int64_t)h * D;
  float qv[kE], o[kE];
  for (int e = 0; e < kE; ++e) {
    qv[e] = to_f32(q[lane + 32 * e]);
    o[e] = 0.f;
  }
  const float slope = p.slopes ? p.slopes[h] : 0.f;
  float m = -INFINITY, l = 0.f;
  for (int i = warp; i < n; i += 8) {
    const int t = i < sink ? i : first + i - sink;
    const int64_t blk = p.table[(int64_t)b * p.max_blocks + t / p.block_size];
    const bool ok = blk >= 0 && blk < p.num_blocks;
    if (!ok && p.status && lane == 0) atomicOr(p.status, TV_DEV_BAD_BLOCK);
    const int64_t at = ((blk * p.Hkv + kvh) * p.block_size + t % p.block_size) * D;
    float x = 0.f;
    for (int e = 0; e < kE; ++e) x += ok ? qv[e] * to_f32(static_cast<const T*>(p.k_cache)[at + lane + 32 * e]) : 0.f;
    for (int w = 16; w; w >>= 1) x += __shfl_xor_sync(0xffffffffu, x, w);
    x *= p.scale;
    if (p.softcap > 0.f) x = p.softcap * tanhf(x / p.softcap);
    x = (x + slope * (float)(t - (L - 1))) * kLog2e;
    const float m2 = fmaxf(m, x), c = exp2f(m - m2), w = exp2f(x - m2);
    l = l * c + w;
    for (int e = 0; e < kE; ++e)
      o[e] = o[e] * c + (ok ? w * to_f32(static_cast<const T*>(p.v_cache)[at + lane + 32 * e]) : 0.f);
    m = m2;
  }
  __shared__ float sm[8], sl[8], so[8][D];
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
  for (int e = 0; e < kE; ++e) so[warp][lane + 32 * e] = o[e];
  __syncthreads();
  float mm = -INFINITY, ll = 0.f;
  for (int w = 0; w < 8; ++w) mm = fmaxf(mm, sm[w]);
  if (mm != -INFINITY)
    for (int w = 0; w < 8; ++w) ll += sl[w] * exp2f(sm[w] - mm);
  T* out = static_cast<T*>(p.out) + ((int64_t)b * p.Hq + h) * D;
  for (int d = threadIdx.x; d < D; d += blockDim.x) {
    float v = 0.f;
    if (n > 0)
      for (int w = 0; w < 8; ++w) v += sm[w] == -INFINITY ? 0.f : so[w][d] * exp2f(sm[w] - mm);
    store(out + d, n > 0 ? v / ll : 0.f);
  }
  if (p.lse && threadIdx.x == 0) p.lse[(int64_t)b * p.Hq + h] = n > 0 ? (mm + log2f(ll)) * kLn2 : -INFINITY;
}

template <typename T>
int launch_decode(const DecodeParams& p, int D, cudaStream_t s) {
  const unsigned grid = (unsigned)(p.B * p.Hq);
  switch (D) {
    case 64: decode_kernel<T, 64><<<grid, 256, 0, s>>>(p); break;
    case 128: decode_kernel<T, 128><<<grid, 256, 0, s>>>(p); break;
    default: decode_kernel<T, 256><<<grid, 256, 0, s>>>(p); break;
  }
  TV_LAUNCH_CHECK("decode_kernel");
  return TV_OK;
}

int check_shape(const char* fn, int32_t Hq, int32_t Hkv, int32_t D, int32_t dtype, int32_t num_ctas) {
  if (Hq < 1 || Hkv < 1 || Hq % Hkv || D < 1 || num_ctas < 0 || num_ctas > kMaxCtas)
    return tv::fail(TV_ERR_INVALID_ARG, "%s: bad sizes", fn);
  if (dtype != TV_F32 && dtype != TV_BF16) return tv::fail(TV_ERR_UNSUPPORTED, "%s: dtype %d", fn, dtype);
  if (D != 64 && D != 128 && D != 256)
    return tv::fail(TV_ERR_UNSUPPORTED, "%s: head_dim %d not in {64, 128, 256}", fn, D);
  return TV_OK;
}

}  // namespace

extern "C" int tv_decode_attn_workspace_size(int32_t Hq, int32_t Hkv, int32_t head_dim, int32_t dtype,
                                             int32_t num_ctas, size_t* bytes) {
  tv::clear_error();
  if (int rc = check_shape("tv_decode_attn_workspace_size", Hq, Hkv, head_dim, dtype, num_ctas)) return rc;
  if (!bytes) return tv::fail(TV_ERR_INVALID_ARG, "tv_decode_attn_workspace_size: null pointer");
  *bytes = (size_t)kCounterBytes;
  return TV_OK;
}

extern "C" int tv_decode_attn(const void* q, int64_t q_stride, const void* k_cache, const void* v_cache,
                              int64_t num_blocks, int32_t block_size, const int32_t* block_table, int32_t max_blocks,
                              const int32_t* seq_lens, int32_t B, int32_t Hq, int32_t Hkv, int32_t head_dim,
                              int32_t dtype, float scale, float softcap, int32_t window, int32_t n_sink,
                              const float* slopes, void* out, float* lse, void* workspace, size_t workspace_bytes,
                              int32_t num_ctas, int32_t flags, int32_t* status, void* stream) {
  tv::clear_error();
  if (int rc = check_shape("tv_decode_attn", Hq, Hkv, head_dim, dtype, num_ctas)) return rc;
  if (B < 0 || num_blocks < 1 || block_size < 1 || max_blocks < 1 || window < 0 || n_sink < 0)
    return tv::fail(TV_ERR_INVALID_ARG, "tv_decode_attn: bad sizes");
  if (!std::isfinite(scale) || !(softcap >= 0.f) || !std::isfinite(softcap))
    return tv::fail(TV_ERR_INVALID_ARG, "tv_decode_attn: scale must be finite, softcap finite and not negative");
  if (flags & ~TV_ATTN_WORKSPACE_ZEROED) return tv::fail(TV_ERR_INVALID_ARG, "tv_decode_attn: unknown flags %d", flags);
  if (B == 0) return TV_OK;
  if (!q || !k_cache || !v_cache || !block_table || !seq_lens || !out)
    return tv::fail(TV_ERR_INVALID_ARG, "tv_decode_attn: null pointer");
  const int64_t e = dtype == TV_F32 ? 4 : 2;
  if (q_stride < 0 || (q_stride * e) % 16 ||
      ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k_cache) | reinterpret_cast<uintptr_t>(v_cache) |
        reinterpret_cast<uintptr_t>(out)) & 15))
    return tv::fail(TV_ERR_INVALID_ARG, "tv_decode_attn: buffers and the q stride must be multiples of 16 bytes");
  size_t need = 0;
  if (int rc = tv_decode_attn_workspace_size(Hq, Hkv, head_dim, dtype, num_ctas, &need)) return rc;
  if (!workspace || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255))
    return tv::fail(TV_ERR_WORKSPACE, "tv_decode_attn: needs %zu workspace bytes, 256-byte aligned", need);
  if ((int64_t)B * Hq >= INT32_MAX) return tv::fail(TV_ERR_UNSUPPORTED, "tv_decode_attn: B * Hq exceeds 2^31");
  DecodeParams p{q, q_stride, k_cache, v_cache, num_blocks, block_size, block_table, max_blocks, seq_lens, B, Hq, Hkv,
                 Hq / Hkv, scale, softcap, window, n_sink, slopes, out, lse, status};
  return dtype == TV_BF16 ? launch_decode<__nv_bfloat16>(p, head_dim, (cudaStream_t)stream)
                          : launch_decode<float>(p, head_dim, (cudaStream_t)stream);
}
