// Attention of a chunk of new tokens per request over the paged cache, their
// own keys and values already in it: entry points, and the kernel on CUDA
// cores for float32 and for the shapes that the tcgen05 kernel does not take.
//
// Token j of a chunk of n sits at p = L - n + j; its output row of head h is
// softmax(s) V over the keys t <= p (with a window only t > p - window or
// t < n_sink), s_t = cap(scale q.k_t) + slope_h (t - p).  "Tree Verification",
// "Tree Attention": the chain as a tree, with its K/V in the cache.
//
// CUDA-core kernel: a CTA takes 64 rows (tokens x heads of one KV head) and
// walks their keys in tiles of 32 with the running maximum and sum of a
// softmax; a thread holds 8 rows x 2 scores and 8 rows x D / 16 outputs in
// registers, so 10 16-byte reads of shared memory feed 64 products (heads of 256:
// 32 rows, 4 a thread, 6 reads for 32).  Everything is float32.  Keys that no row of the tile sees are not read.  Few tiles of rows
// share their keys among CTAs, whose parts the last to arrive joins in order.  Bound by the
// latency of its own steps (load, scores, weights, outputs) at 8-16 warps an SM:
// 20-28 TFLOP/s of the FP32 pipe's 80.
#include <algorithm>
#include <climits>
#include <type_traits>

#include <cuda_bf16.h>

#include "attn_score.cuh"
#include "chunk.h"

namespace {

using tv::ChunkOf;
using tv::ChunkParams;

constexpr int kThreads = 128;
constexpr int kKeys = 32;      // of a tile
constexpr int kMaxCtas = 4096;
constexpr size_t kCounterBytes = 4 * kMaxCtas;  // first in the workspace
constexpr int kPieces = 64;       // of a CUDA-core tile's keys at most
constexpr int kSlots = 1216;      // pieces of all tiles at most: about eight CTAs an SM
constexpr size_t kSlotFloats = 64 * (128 + 2);  // a piece's rows with their maxima and sums, enough for 32 rows of 256 too

template <int D>
struct Simt {
  static constexpr int kRows = D == 256 ? 32 : 64;
  static constexpr int kMine = kRows / 8;   // rows of a thread
  static constexpr int kCols = D / 64;      // runs of 4 outputs of a thread
  // few registers for more CTAs an SM (6 x 33-500 tokens, 16 heads of 64, float32: 345 -> 280 us; 8 x 500, 32/8 heads of 128:
  // 725 -> 635 us), but for the longest rows, which gain nothing
  static constexpr int kUnroll = D == 256 ? 2 : 1;
  static constexpr int kPitch = D + 4;      // of a row of Q and K: keys in turn lie in neighbouring banks
  static constexpr int kPitchP = kKeys + 4;
  static constexpr int kBytes = 4 * (kRows * kPitch + kKeys * kPitch + kKeys * D + kRows * kPitchP);
};

__device__ __forceinline__ void cp_async16(float* dst, const void* src, bool read) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src),
               "r"(read ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ float4 as_floats(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 as_floats(const __nv_bfloat16* p) {
  const uint2 r = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xffff0000u), __uint_as_float(r.y << 16),
                     __uint_as_float(r.y & 0xffff0000u));
}
__device__ __forceinline__ void store4(float* p, float a, float b, float c, float d) {
  *reinterpret_cast<float4*>(p) = make_float4(a, b, c, d);
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, float a, float b, float c, float d) {
  uint2 r;
  reinterpret_cast<__nv_bfloat162*>(&r)[0] = __floats2bfloat162_rn(a, b);
  reinterpret_cast<__nv_bfloat162*>(&r)[1] = __floats2bfloat162_rn(c, d);
  *reinterpret_cast<uint2*>(p) = r;
}

// Tile i of request b, found without a scan: request b's tiles start at s0 / tokens + b, and one request's never reach
// the next one's, as ceil(n / tokens) <= (s0 + n) / tokens - s0 / tokens + 1.
__device__ __forceinline__ bool find_tile(const ChunkParams& p, int unit, int tokens, int& b, int& i, ChunkOf& c) {
  if (!p.cu) {
    const int per = (p.T / p.B + tokens - 1) / tokens;
    b = per ? unit / per : p.B;
    i = per ? unit - b * per : 0;
    return b < p.B && tv::chunk_of(p, b, c);
  }
  int lo = 0;
  for (int hi = p.B; hi - lo > 1;) {
    const int mid = lo + (hi - lo) / 2;
    if ((int64_t)__ldg(p.cu + mid) / tokens + mid <= unit) lo = mid; else hi = mid;
  }
  b = lo;
  if (!tv::chunk_of(p, b, c)) return false;
  const int64_t at = (int64_t)unit - (c.s0 / tokens + b);
  i = (int)at;
  return at >= 0 && at * tokens < c.n;
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) chunk_simt_kernel(const __grid_constant__ ChunkParams p, int split) {
  using S = Simt<D>;
  extern __shared__ __align__(16) float sm[];
  float* sq = sm;
  float* sk = sq + S::kRows * S::kPitch;
  float* sv = sk + kKeys * S::kPitch;
  float* sp = sv + kKeys * D;
  __shared__ int64_t row_at[kKeys];  // cache row (of KV head 0) of a key, -1: zeros

  const int kvh = blockIdx.y;
  const int h0 = blockIdx.z / split * S::kRows, heads = min(p.G - h0, S::kRows);  // query heads of the KV head
  const int tokens = S::kRows / min(p.G, S::kRows);
  int b, i;
  ChunkOf c;
  if (p.cu && p.status && blockIdx.x + blockIdx.y + blockIdx.z == 0)
    for (b = threadIdx.x; b < p.B; b += kThreads)
      if (!tv::chunk_of(p, b, c)) atomicOr(p.status, TV_DEV_BAD_OFFSETS);
  if (!find_tile(p, blockIdx.x, tokens, b, i, c)) return;
  const int j0 = i * tokens, nt = min(tokens, c.n - j0);
  const int rows = nt * heads;
  const int tid = threadIdx.x, tx = tid % 16, ty = tid / 16;

  // queries, rows behind the last as zeros
  for (int x = tid; x < S::kRows * (D / 4); x += kThreads) {
    const int r = x / (D / 4), d = x % (D / 4) * 4;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < rows) {
      const int64_t t = c.s0 + j0 + r / heads;
      v = as_floats(reinterpret_cast<const T*>(p.q + t * p.q_stride) + (kvh * p.G + h0 + r % heads) * D + d);
    }
    *reinterpret_cast<float4*>(sq + r * S::kPitch + d) = v;
  }
  const Scorer score(p);
  const int pos0 = c.first + j0, last = pos0 + nt - 1;  // of the tile's first and last token
  const int lo = p.window > 0 ? max(0, max(0, pos0 + 1) - p.window) : 0;
  const int sink = min(p.n_sink, lo);
  int pos[S::kMine];
  float slope[S::kMine], m[S::kMine], l[S::kMine];
#pragma unroll
  for (int r = 0; r < S::kMine; ++r) {
    const int row = ty + 8 * r;
    pos[r] = row < rows ? pos0 + row / heads : -1;
    slope[r] = p.slopes && row < rows ? slope_of(p.slopes, kvh * p.G + h0 + row % heads) : 0.f;
    m[r] = kNoScore;
    l[r] = 0.f;
  }
  float o[S::kMine][S::kCols * 4] = {};

  const int lead = min((sink + kKeys - 1) / kKeys, lo / kKeys);  // tiles of kept first keys before the window's
  const int tiles = last >= 0 ? lead + last / kKeys + 1 - lo / kKeys : 0;
  // few tiles of rows over many keys: several CTAs share one's keys, 128 each at least, and the last to arrive joins
  const int pieces = min(split, max(1, tiles / 4)), piece = blockIdx.z % split;
  if (piece >= pieces) return;
  const int tile1 = (int)((int64_t)tiles * (piece + 1) / pieces);
  for (int tile = (int)((int64_t)tiles * piece / pieces); tile < tile1; ++tile) {
    const int t0 = (tile < lead ? tile : lo / kKeys + tile - lead) * kKeys;
    __syncthreads();
    if (tid < kKeys) {
      const int t = t0 + tid;
      int64_t at = -1;
      if (t <= last && (t >= lo || t < sink)) {
        const int64_t blk = __ldg(p.table + (int64_t)b * p.max_blocks + t / p.block_size);
        if (blk >= 0 && blk < p.num_blocks) at = blk * p.Hkv * p.block_size + t % p.block_size;
        else if (p.status) atomicOr(p.status, TV_DEV_BAD_BLOCK);
      }
      row_at[tid] = at;
    }
    __syncthreads();
    // float32 straight into shared memory, all of K on its way and V behind it while the scores are computed (load by load
    // through registers 1305 against 974 us: 175 tokens over 4648, 32/4 heads of 256)
    if constexpr (std::is_same<T, float>::value) {
      auto load = [&](const char* cache, float* dst, int pitch) {
        for (int x = tid; x < kKeys * (D / 4); x += kThreads) {
          const int key = x / (D / 4), d = x % (D / 4) * 4;
          const int64_t at = row_at[key], from = at < 0 ? 0 : (at + (int64_t)kvh * p.block_size) * D + d;
          cp_async16(dst + key * pitch + d, reinterpret_cast<const float*>(cache) + from, at >= 0);
        }
        cp_async_commit();
      };
      load(p.k_cache, sk, S::kPitch);
      load(p.v_cache, sv, D);
    } else {
      for (int x = tid; x < kKeys * (D / 4); x += kThreads) {
        const int key = x / (D / 4), d = x % (D / 4) * 4;
        const int64_t at = row_at[key];
        float4 k = make_float4(0.f, 0.f, 0.f, 0.f), v = k;
        if (at >= 0) {
          const int64_t off = (at + (int64_t)kvh * p.block_size) * D + d;
          k = as_floats(reinterpret_cast<const T*>(p.k_cache) + off);
          v = as_floats(reinterpret_cast<const T*>(p.v_cache) + off);
        }
        *reinterpret_cast<float4*>(sk + key * S::kPitch + d) = k;
        *reinterpret_cast<float4*>(sv + key * D + d) = v;
      }
    }
    cp_async_wait<1>();
    __syncthreads();
    float s[S::kMine * 2] = {};
#pragma unroll S::kUnroll
    for (int d = 0; d < D; d += 4) {
      const float4 k0 = *reinterpret_cast<const float4*>(sk + tx * S::kPitch + d);
      const float4 k1 = *reinterpret_cast<const float4*>(sk + (tx + 16) * S::kPitch + d);
#pragma unroll
      for (int r = 0; r < S::kMine; ++r) {
        const float4 a = *reinterpret_cast<const float4*>(sq + (ty + 8 * r) * S::kPitch + d);
        s[2 * r] = fmaf(a.w, k0.w, fmaf(a.z, k0.z, fmaf(a.y, k0.y, fmaf(a.x, k0.x, s[2 * r]))));
        s[2 * r + 1] = fmaf(a.w, k1.w, fmaf(a.z, k1.z, fmaf(a.y, k1.y, fmaf(a.x, k1.x, s[2 * r + 1]))));
      }
    }
    score(s);
#pragma unroll
    for (int r = 0; r < S::kMine; ++r) {
      float top = m[r];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int t = t0 + tx + 16 * e;
        float& x = s[2 * r + e];
        if (p.slopes) x = fmaf(slope[r], (float)(t - pos[r]), x);
        const bool seen = t <= pos[r] && (p.window == 0 || pos[r] - t < p.window || t < p.n_sink);
        if (!seen) x = -INFINITY;
        top = fmaxf(top, x);
      }
#pragma unroll
      for (int w = 1; w < 16; w *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
      const float alpha = exp2_approx(m[r] - top);
      const float e0 = exp2_approx(s[2 * r] - top), e1 = exp2_approx(s[2 * r + 1] - top);
      m[r] = top;
      l[r] = l[r] * alpha + (e0 + e1);
#pragma unroll
      for (int k = 0; k < S::kCols * 4; ++k) o[r][k] *= alpha;
      sp[(ty + 8 * r) * S::kPitchP + tx] = e0;
      sp[(ty + 8 * r) * S::kPitchP + tx + 16] = e1;
    }
    cp_async_wait<0>();
    __syncthreads();  // V; a row's weights are its own half warp's
#pragma unroll S::kUnroll
    for (int key = 0; key < kKeys; key += 4) {
      float4 w[S::kMine];
#pragma unroll
      for (int r = 0; r < S::kMine; ++r) w[r] = *reinterpret_cast<const float4*>(sp + (ty + 8 * r) * S::kPitchP + key);
#pragma unroll
      for (int k = 0; k < S::kCols; ++k) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float4 v = *reinterpret_cast<const float4*>(sv + (key + e) * D + k * 64 + tx * 4);
#pragma unroll
          for (int r = 0; r < S::kMine; ++r) {
            const float x = e == 0 ? w[r].x : e == 1 ? w[r].y : e == 2 ? w[r].z : w[r].w;
            o[r][4 * k] = fmaf(x, v.x, o[r][4 * k]);
            o[r][4 * k + 1] = fmaf(x, v.y, o[r][4 * k + 1]);
            o[r][4 * k + 2] = fmaf(x, v.z, o[r][4 * k + 2]);
            o[r][4 * k + 3] = fmaf(x, v.w, o[r][4 * k + 3]);
          }
        }
      }
    }
  }
#pragma unroll
  for (int r = 0; r < S::kMine; ++r)
#pragma unroll
    for (int w = 1; w < 16; w *= 2) l[r] += __shfl_xor_sync(0xffffffffu, l[r], w);
  if (pieces > 1) {
    const int unit = (blockIdx.z / split * gridDim.y + blockIdx.y) * gridDim.x + blockIdx.x;
    float* slot = p.part_o + (int64_t)unit * split * kSlotFloats;  // [piece][rows][D + 2]: outputs, maximum, sum
    float* here = slot + piece * kSlotFloats;
#pragma unroll
    for (int r = 0; r < S::kMine; ++r) {
      float* dst = here + (ty + 8 * r) * (D + 2);
#pragma unroll
      for (int k = 0; k < S::kCols * 4; k += 2)
        *reinterpret_cast<float2*>(dst + k / 4 * 64 + tx * 4 + k % 4) = make_float2(o[r][k], o[r][k + 1]);
      if (tx == 0) *reinterpret_cast<float2*>(dst + D) = make_float2(m[r], l[r]);
    }
    __shared__ bool joins;
    __threadfence();
    __syncthreads();
    if (tid == 0) {
      uint32_t before;
      asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], %2;" : "=r"(before) : "l"(p.arrive + unit), "r"(1u) : "memory");
      joins = before == (uint32_t)pieces - 1;
      if (joins) p.arrive[unit] = 0;
    }
    __syncthreads();
    if (!joins) return;
    __threadfence();
#pragma unroll
    for (int r = 0; r < S::kMine; ++r) {
      m[r] = kNoScore;
      l[r] = 0.f;
#pragma unroll
      for (int k = 0; k < S::kCols * 4; ++k) o[r][k] = 0.f;
    }
#pragma unroll 1
    for (int i = 0; i < pieces; ++i) {
#pragma unroll
      for (int r = 0; r < S::kMine; ++r) {
        const float* src = slot + i * kSlotFloats + (ty + 8 * r) * (D + 2);
        const float2 ml = __ldcg(reinterpret_cast<const float2*>(src + D));
        const float top = fmaxf(m[r], ml.x), keep = exp2_approx(m[r] - top);
        const float w = ml.y == 0.f ? 0.f : exp2_approx(ml.x - top);
        l[r] = fmaf(l[r], keep, w * ml.y);
        m[r] = top;
#pragma unroll
        for (int k = 0; k < S::kCols * 4; k += 2) {
          const float2 x = __ldcg(reinterpret_cast<const float2*>(src + k / 4 * 64 + tx * 4 + k % 4));
          o[r][k] = fmaf(o[r][k], keep, w * x.x);
          o[r][k + 1] = fmaf(o[r][k + 1], keep, w * x.y);
        }
      }
    }
  }
#pragma unroll
  for (int r = 0; r < S::kMine; ++r) {
    const int row = ty + 8 * r;
    if (row >= rows) continue;
    const int64_t at = (int64_t)(c.s0 + j0 + row / heads) * p.Hq + kvh * p.G + h0 + row % heads;
    const float f = inverse(l[r]);
    T* dst = reinterpret_cast<T*>(p.out) + at * D + tx * 4;
#pragma unroll
    for (int k = 0; k < S::kCols; ++k)
      store4(dst + k * 64, o[r][4 * k] * f, o[r][4 * k + 1] * f, o[r][4 * k + 2] * f, o[r][4 * k + 3] * f);
    if (p.lse && tx == 0) p.lse[at] = (m[r] + log2f(l[r])) * kLn2;
  }
}

template <typename T, int D>
int launch_simt(const ChunkParams& p, cudaStream_t stream) {
  using S = Simt<D>;
  const int64_t tokens = S::kRows / std::min(p.G, S::kRows);
  const int64_t units = p.cu ? p.T / tokens + p.B : tv::ceil_div(p.T / p.B, tokens) * p.B;
  const cudaError_t e =
      cudaFuncSetAttribute(chunk_simt_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kBytes);
  if (e != cudaSuccess) return tv::cuda_fail(e, "cudaFuncSetAttribute(chunk_simt_kernel)");
  const int64_t groups = tv::ceil_div(p.G, S::kRows), ctas = units * p.Hkv * groups;
  const int split = (int)std::max<int64_t>(1, std::min<int64_t>(kPieces, kSlots / ctas));
  static_assert((size_t)S::kRows * (D + 2) <= kSlotFloats, "a piece fits its slot");
  const dim3 grid((unsigned)units, (unsigned)p.Hkv, (unsigned)(groups * split));
  chunk_simt_kernel<T, D><<<grid, kThreads, S::kBytes, stream>>>(p, split);
  TV_LAUNCH_CHECK("chunk_simt_kernel");
  return TV_OK;
}

template <typename T>
int dispatch_simt(const ChunkParams& p, int D, cudaStream_t stream) {
  return D == 64    ? launch_simt<T, 64>(p, stream)
         : D == 128 ? launch_simt<T, 128>(p, stream)
                    : launch_simt<T, 256>(p, stream);
}

int check_shape(const char* fn, int32_t Hq, int32_t Hkv, int32_t head_dim, int32_t dtype, int32_t num_ctas) {
  if (Hq < 1 || Hkv < 1 || Hq % Hkv || num_ctas < 0 || num_ctas > kMaxCtas)
    return tv::fail(TV_ERR_INVALID_ARG, "%s: bad sizes", fn);
  if (dtype != TV_F32 && dtype != TV_BF16) return tv::fail(TV_ERR_UNSUPPORTED, "%s: dtype %d", fn, dtype);
  if (head_dim != 64 && head_dim != 128 && head_dim != 256)
    return tv::fail(TV_ERR_UNSUPPORTED, "%s: head_dim %d not in {64, 128, 256}", fn, head_dim);
  if (Hkv > 65535 || (int64_t)Hq * head_dim >= INT32_MAX / 4)
    return tv::fail(TV_ERR_UNSUPPORTED, "%s: more than 65535 KV heads, or a token's heads exceed 2^29 elements", fn);
  if (Hq / Hkv > 65535 * 32)  // the CUDA-core kernel's grid: a CTA has 32 or 64 rows
    return tv::fail(TV_ERR_UNSUPPORTED, "%s: more than %d query heads per KV head", fn, 65535 * 32);
  return TV_OK;
}

// CTAs of the tensor-core kernel's grid
int grid_of(int32_t num_ctas, int* ctas) {
  *ctas = num_ctas;
  if (num_ctas > 0) return TV_OK;
  tv::DeviceInfo dev;
  if (int rc = tv::current_device_info(&dev)) return rc;
  *ctas = dev.sm_count;
  return TV_OK;
}

}  // namespace

extern "C" int tv_chunk_attn_workspace_size(int32_t Hq, int32_t Hkv, int32_t head_dim, int32_t dtype, int32_t num_ctas,
                                            size_t* bytes) {
  tv::clear_error();
  if (!bytes) return tv::fail(TV_ERR_INVALID_ARG, "tv_chunk_attn_workspace_size: null pointer");
  if (int rc = check_shape("tv_chunk_attn_workspace_size", Hq, Hkv, head_dim, dtype, num_ctas)) return rc;
  *bytes = kCounterBytes + kSlots * kSlotFloats * sizeof(float);
  if (dtype != TV_BF16) return TV_OK;  // never the tensor-core kernel
  int ctas = 0;
  if (int rc = grid_of(num_ctas, &ctas)) return rc;
  *bytes = std::max(*bytes, kCounterBytes + tv::chunk_tc_workspace(head_dim, ctas));
  return TV_OK;
}

extern "C" int tv_chunk_attn(const void* q, int64_t q_stride, const void* k_cache, const void* v_cache,
                             int64_t num_blocks, int32_t block_size, const int32_t* block_table, int32_t max_blocks,
                             const int32_t* seq_lens, const int32_t* cu_new, int32_t T, int32_t B, int32_t Hq,
                             int32_t Hkv, int32_t head_dim, int32_t dtype, float scale, float softcap, int32_t window,
                             int32_t n_sink, const float* slopes, void* out, float* lse, void* workspace,
                             size_t workspace_bytes, int32_t num_ctas, int32_t flags, int32_t* status, void* stream) {
  tv::clear_error();
  if (int rc = check_shape("tv_chunk_attn", Hq, Hkv, head_dim, dtype, num_ctas)) return rc;
  if (B < 0 || T < 0 || num_blocks < 1 || block_size < 1 || max_blocks < 1 || window < 0 || n_sink < 0)
    return tv::fail(TV_ERR_INVALID_ARG, "tv_chunk_attn: bad sizes");
  if (!factors_fit(scale, softcap))
    return tv::fail(TV_ERR_INVALID_ARG,
                    "tv_chunk_attn: scale must be finite, softcap finite and not negative, both within 2.3e38");
  if ((flags & ~(3 | TV_ATTN_WORKSPACE_ZEROED)) || (flags & 3) == 3)
    return tv::fail(TV_ERR_INVALID_ARG, "tv_chunk_attn: unknown flags %d", flags);
  if (B == 0) return TV_OK;
  if (!cu_new && T % B)
    return tv::fail(TV_ERR_INVALID_ARG, "tv_chunk_attn: without offsets T (%d) must be a multiple of B (%d)", T, B);
  if (T == 0) return TV_OK;
  if (!q || !k_cache || !v_cache || !block_table || !seq_lens || !out)
    return tv::fail(TV_ERR_INVALID_ARG, "tv_chunk_attn: null pointer");
  const int64_t e = dtype == TV_F32 ? 4 : 2;
  if ((T > 1 && (q_stride < 0 || (q_stride * e) % 16)) ||
      ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k_cache) | reinterpret_cast<uintptr_t>(v_cache) |
        reinterpret_cast<uintptr_t>(out)) & 15))
    return tv::fail(TV_ERR_INVALID_ARG, "tv_chunk_attn: buffers and the q stride must be multiples of 16 bytes");
  size_t need = 0;
  if (int rc = tv_chunk_attn_workspace_size(Hq, Hkv, head_dim, dtype, num_ctas, &need)) return rc;
  if (!workspace || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255))
    return tv::fail(TV_ERR_WORKSPACE, "tv_chunk_attn: needs %zu workspace bytes, 256-byte aligned", need);
  if ((int64_t)T + B >= INT32_MAX)
    return tv::fail(TV_ERR_UNSUPPORTED, "tv_chunk_attn: tokens and requests exceed 2^31");
  cudaStream_t st = (cudaStream_t)stream;
  ChunkParams p{};
  p.q = static_cast<const char*>(q);
  p.q_stride = T > 1 ? q_stride * e : 0;
  p.k_cache = static_cast<const char*>(k_cache);
  p.v_cache = static_cast<const char*>(v_cache);
  p.num_blocks = num_blocks;
  p.block_size = block_size;
  p.table = block_table;
  p.max_blocks = max_blocks;
  p.seq_lens = seq_lens;
  p.cu = cu_new;
  p.T = T;
  p.B = B;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.G = Hq / Hkv;
  p.scale = scale;
  p.softcap = cap_that_matters(scale, softcap);
  p.window = window;
  p.n_sink = n_sink;
  p.slopes = slopes;
  p.out = static_cast<char*>(out);
  p.lse = lse;
  p.status = status;
  p.arrive = static_cast<uint32_t*>(workspace);
  p.part_o = reinterpret_cast<float*>(static_cast<char*>(workspace) + kCounterBytes);
  const char* why = "TV_ATTN_SIMT";
  if ((flags & 3) != TV_ATTN_SIMT) {
    tv::DeviceInfo dev;
    if (int rc = tv::current_device_info(&dev)) return rc;
    why = tv::chunk_tc_unsupported(dev, p, dtype, head_dim);
    if (why && (flags & 3) == TV_ATTN_TCGEN05)
      return tv::fail(TV_ERR_UNSUPPORTED, "tv_chunk_attn: no tcgen05 kernel: %s", why);
  }
  // also where this call cuts no unit and counts nothing: the next one may take the counters as zero
  if (!(flags & TV_ATTN_WORKSPACE_ZEROED)) TV_CUDA_TRY(cudaMemsetAsync(workspace, 0, kCounterBytes, st));
  if (!why) {
    if (int rc = grid_of(num_ctas, &p.ctas)) return rc;
    p.m_tiles = tv::chunk_tc_m_tiles(head_dim);
    p.part_ml = p.part_o + (int64_t)p.ctas * 2 * 128 * p.m_tiles * head_dim;
    return tv::launch_chunk_tc(p, head_dim, st);
  }
  return dtype == TV_BF16 ? dispatch_simt<__nv_bfloat16>(p, head_dim, st) : dispatch_simt<float>(p, head_dim, st);
}
