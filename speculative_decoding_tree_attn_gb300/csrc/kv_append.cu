// Appending new tokens' keys and values to the paged cache, keys (and
// queries) rotated at their positions on the way.
//
// Token j of request b (packed row t = cu_new[b] + j) sits at position
// p = L_b + j: its keys R(p) k and values v go to block
// block_table[b, p / block_size], slot p % block_size, its queries R(p) q to
// q_out, with the rotation of rope_math.cuh (the bits of tv_rope_apply).
// "Tree Verification", "The Cost Side": the cached prefix keys are stored
// rotated, so the tree and one-token attention read them as they are.
//
// Pure movement: (Hq + 2 Hkv) D elements a token read once and written once;
// the rotation is 3 flops an element.  Bound by HBM for a prompt (32 prompts of
// 1-1023 tokens, 32/8 heads of 128, bf16: 65 us, 0.96 of the measured copy rate;
// CTAs of 256 threads 68 us, twice the loads in flight a lane 81 us), by latency
// for a step's tokens (256 requests: 3.3 us).
#include <algorithm>
#include <climits>

#include <cuda_bf16.h>

#include "common.h"
#include "kv_place.cuh"
#include "rope_math.cuh"

namespace {

constexpr int kThreads = 128;

// One warp per (token, slice of its heads): a lane keeps one chunk of 8
// frequency pairs (elements 8c.. and 8c + D/2..), so its cos/sin entries are
// read once for all heads.  The warps behind the tokens' take a request each
// and count its new length.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(AppendParams p) {
  constexpr int kChunks = D / 16;
  constexpr int kHeads = 32 / kChunks;             // heads a warp covers at once
  constexpr int kVec = 8 * (int)sizeof(T) / 16;    // 16-byte vectors per 8 elements
  constexpr int kRow = D * (int)sizeof(T);         // bytes of a head's row
  constexpr int kUnroll = 8 / (int)sizeof(T);      // 128 bytes of a lane on their way at once
  const int lane = threadIdx.x % 32;
  const int64_t w = (int64_t)blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32;
  const int64_t token_warps = (int64_t)p.T * p.slices;
  if (w >= token_warps) {
    if (w - token_warps < p.B) count_request<WarpSearch>(p, (int)(w - token_warps), lane);
    return;
  }
  const int t = (int)(w / p.slices);
  const int s = (int)(w - (int64_t)t * p.slices);
  int b, j;
  if (!find_request<WarpSearch>(p, t, lane, b, j)) return;
  const int L = __ldg(p.seq_lens + b);
  const int64_t pos = (int64_t)L + j;
  if (L < 0 || pos >= p.max_pos) return;
  const int64_t col = pos / p.block_size;
  const int64_t slot = pos - col * p.block_size;
  const int64_t blk = col < p.max_blocks ? __ldg(p.table + (int64_t)b * p.max_blocks + col) : -1;
  const bool placed = blk >= 0 && blk < p.num_blocks;

  const int c = lane % kChunks;
  float co[8], si[8];
  if (p.cs) {
    const float* row = p.cs + pos * D + c * 8;
    Vec8<float>::load(row, co);
    Vec8<float>::load(row + D / 2, si);
  }
  const int Hq = p.q ? p.Hq : 0;
  const int H = Hq + 2 * p.Hkv;
  const int rounds = (H + kHeads - 1) / kHeads;
  const int per = (rounds + p.slices - 1) / p.slices * kHeads;
  const int h_end = min(H, (s + 1) * per);
  const int64_t lo = c * 8 * sizeof(T), hi = lo + kRow / 2;
  for (int h0 = s * per + lane / kChunks; h0 < h_end; h0 += kHeads * kUnroll) {
    Raw<kVec> x1[kUnroll], x2[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int h = h0 + u * kHeads;
      if (h >= h_end) break;
      const char* src = h < Hq ? p.q + t * p.q_stride + (int64_t)h * kRow
                      : h < Hq + p.Hkv ? p.k + t * p.k_stride + (int64_t)(h - Hq) * kRow
                                       : p.v + t * p.v_stride + (int64_t)(h - Hq - p.Hkv) * kRow;
      x1[u] = *reinterpret_cast<const Raw<kVec>*>(src + lo);
      x2[u] = *reinterpret_cast<const Raw<kVec>*>(src + hi);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int h = h0 + u * kHeads;
      if (h >= h_end) break;
      char* dst;
      if (h < Hq) {
        dst = p.q_out + t * p.q_out_stride + (int64_t)h * kRow;
      } else {
        if (!placed) continue;
        const bool is_k = h < Hq + p.Hkv;
        const int kh = h - Hq - (is_k ? 0 : p.Hkv);
        dst = (is_k ? p.k_cache : p.v_cache) + ((blk * p.Hkv + kh) * p.block_size + slot) * kRow;
      }
      if (p.cs && h < Hq + p.Hkv) {
        float a[8], d[8], y1[8], y2[8];
        Vec8<T>::load(reinterpret_cast<const T*>(&x1[u]), a);
        Vec8<T>::load(reinterpret_cast<const T*>(&x2[u]), d);
#pragma unroll
        for (int e = 0; e < 8; ++e) rope_pair(a[e], d[e], co[e], si[e], y1[e], y2[e]);
        Vec8<T>::store(reinterpret_cast<T*>(dst + lo), y1);
        Vec8<T>::store(reinterpret_cast<T*>(dst + hi), y2);
      } else {
        *reinterpret_cast<Raw<kVec>*>(dst + lo) = x1[u];
        *reinterpret_cast<Raw<kVec>*>(dst + hi) = x2[u];
      }
    }
  }
}

// Many tokens of few heads (all of them in one or two rounds of a warp): a token's chain of lookups is longer than its
// copies, so a warp takes 8 tokens, finds their places with a lane each and copies two rounds at a time.  64 prompts of
// up to 2000 tokens, 4/1 heads of 64, bf16: 30 us, a warp per token 58; one round at a time 28 there, but 46 against
// 43 of 2/1 heads of 256; four rounds 36.
constexpr int kTokens = 8;
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) kv_append_narrow_kernel(AppendParams p) {
  constexpr int kChunks = D / 16, kHeads = 32 / kChunks;
  constexpr int kVec = 8 * (int)sizeof(T) / 16;
  constexpr int kRow = D * (int)sizeof(T);
  constexpr int kUnroll = 2;
  const int lane = threadIdx.x % 32;
  const int64_t w = (int64_t)blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32;
  const int64_t token_warps = ((int64_t)p.T + kTokens - 1) / kTokens;
  if (w >= token_warps) {
    if (w - token_warps < p.B) count_request<LaneSearch>(p, (int)(w - token_warps), lane);
    return;
  }
  const int t0 = (int)(w * kTokens);
  int my_pos = -1;       // of token t0 + lane; -1: none
  int64_t my_row = -1;   // its row in the cache for KV head 0; -1: not stored
  if (lane < kTokens && (int64_t)t0 + lane < p.T) {
    const int t = t0 + lane;
    int b, j;
    const bool here = find_request<LaneSearch>(p, t, lane, b, j);
    const int L = __ldg(p.seq_lens + b);
    const int64_t pos = (int64_t)L + j;
    if (here && L >= 0 && pos < p.max_pos) {
      my_pos = (int)pos;
      const int64_t col = pos / p.block_size;
      const int64_t blk = col < p.max_blocks ? __ldg(p.table + (int64_t)b * p.max_blocks + col) : -1;
      if (blk >= 0 && blk < p.num_blocks) my_row = blk * p.Hkv * p.block_size + (pos - col * p.block_size);
    }
  }
  const int c = lane % kChunks;
  const int64_t lo = c * 8 * sizeof(T), hi = lo + kRow / 2;
  const int Hq = p.q ? p.Hq : 0;
  const int H = Hq + 2 * p.Hkv;
  const int two = H > kHeads;  // rounds - 1
#pragma unroll 1
  for (int x0 = 0; x0 < kTokens << two; x0 += kUnroll) {
    Raw<kVec> x1[kUnroll], x2[kUnroll];
    float co[kUnroll][8], si[kUnroll][8];
    char* dst[kUnroll];  // null: nothing to store
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int i = (x0 + u) >> two;
      const int h = lane / kChunks + ((x0 + u) & two) * kHeads;
      const int pos = __shfl_sync(0xffffffffu, my_pos, i);
      const int64_t row = __shfl_sync(0xffffffffu, my_row, i);
      const int64_t t = (int64_t)t0 + i;
      dst[u] = nullptr;
      if (pos < 0 || h >= H) continue;
      const char* src;
      if (h < Hq) {
        src = p.q + t * p.q_stride + (int64_t)h * kRow;
        dst[u] = p.q_out + t * p.q_out_stride + (int64_t)h * kRow;
      } else {
        if (row < 0) continue;
        const bool is_k = h < Hq + p.Hkv;
        const int kh = h - Hq - (is_k ? 0 : p.Hkv);
        src = (is_k ? p.k + t * p.k_stride : p.v + t * p.v_stride) + (int64_t)kh * kRow;
        dst[u] = (is_k ? p.k_cache : p.v_cache) + (row + (int64_t)kh * p.block_size) * kRow;
      }
      x1[u] = *reinterpret_cast<const Raw<kVec>*>(src + lo);
      x2[u] = *reinterpret_cast<const Raw<kVec>*>(src + hi);
      if (p.cs && h < Hq + p.Hkv) {
        const float* cs = p.cs + (int64_t)pos * D + c * 8;
        Vec8<float>::load(cs, co[u]);
        Vec8<float>::load(cs + D / 2, si[u]);
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (!dst[u]) continue;
      if (p.cs && lane / kChunks + ((x0 + u) & two) * kHeads < Hq + p.Hkv) {
        float a[8], d[8], y1[8], y2[8];
        Vec8<T>::load(reinterpret_cast<const T*>(&x1[u]), a);
        Vec8<T>::load(reinterpret_cast<const T*>(&x2[u]), d);
#pragma unroll
        for (int e = 0; e < 8; ++e) rope_pair(a[e], d[e], co[u][e], si[u][e], y1[e], y2[e]);
        Vec8<T>::store(reinterpret_cast<T*>(dst[u] + lo), y1);
        Vec8<T>::store(reinterpret_cast<T*>(dst[u] + hi), y2);
      } else {
        *reinterpret_cast<Raw<kVec>*>(dst[u] + lo) = x1[u];
        *reinterpret_cast<Raw<kVec>*>(dst[u] + hi) = x2[u];
      }
    }
  }
}

template <typename T, int D>
void launch_append(AppendParams p, int sm_count, cudaStream_t stream) {
  constexpr int kHeads = 32 / (D / 16);
  const int H = (p.q ? p.Hq : 0) + 2 * p.Hkv;
  const int rounds = (H + kHeads - 1) / kHeads;
  // 10,000 tokens of one round 6.5 us, 8.1 a warp each, 5000 6.0 and 4.8; of two rounds 10,000 12.4 and 11.1, 19,000 16
  // and 21.  A token of 4 KB fills its warp's copies: 85 us, 82 a warp each.
  if (rounds <= 2 && H * D * (int)sizeof(T) < 4096 && p.T >= 48 * rounds * sm_count) {
    const int64_t warps = ((int64_t)p.T + kTokens - 1) / kTokens + p.B;
    kv_append_narrow_kernel<T, D><<<(unsigned)tv::ceil_div(warps, kThreads / 32), kThreads, 0, stream>>>(p);
    return;
  }
  // few tokens: several warps share one, so that a step's tokens reach every SM
  const int64_t want = (int64_t)sm_count * 8;
  p.slices = (int)std::max<int64_t>(1, std::min<int64_t>(rounds, want / std::max(1, p.T)));
  const int64_t warps = (int64_t)p.T * p.slices + p.B;
  kv_append_kernel<T, D><<<(unsigned)tv::ceil_div(warps, kThreads / 32), kThreads, 0, stream>>>(p);
}

template <typename T>
int dispatch_append(const AppendParams& p, int D, int sm_count, cudaStream_t stream) {
  switch (D) {
    case 16: launch_append<T, 16>(p, sm_count, stream); break;
    case 32: launch_append<T, 32>(p, sm_count, stream); break;
    case 64: launch_append<T, 64>(p, sm_count, stream); break;
    case 128: launch_append<T, 128>(p, sm_count, stream); break;
    case 256: launch_append<T, 256>(p, sm_count, stream); break;
    default: return tv::fail(TV_ERR_UNSUPPORTED, "tv_kv_append: head_dim %d not in {16, 32, 64, 128, 256}", D);
  }
  TV_LAUNCH_CHECK("kv_append_kernel");
  return TV_OK;
}

}  // namespace

extern "C" int tv_kv_append(const void* q, int64_t q_stride, void* q_out, int64_t q_out_stride, int32_t Hq,
                            const void* k_new, int64_t k_stride, const void* v_new, int64_t v_stride,
                            const int32_t* cu_new, int32_t T, void* k_cache, void* v_cache, int64_t num_blocks,
                            int32_t block_size, const int32_t* block_table, int32_t max_blocks,
                            const int32_t* seq_lens, int32_t* new_seq_lens, const float* cos_sin, int32_t max_pos,
                            int32_t B, int32_t Hkv, int32_t head_dim, int32_t dtype, int32_t* status, void* stream) {
  tv::clear_error();
  AppendParams p{};
  bool empty;
  if (int rc = append_params("tv_kv_append", q, q_stride, q_out, q_out_stride, Hq, k_new, k_stride, v_new, v_stride, cu_new,
                             T, k_cache, v_cache, num_blocks, block_size, block_table, max_blocks, seq_lens, new_seq_lens,
                             cos_sin, max_pos, true, B, Hkv, head_dim, dtype, status, &p, &empty))
    return rc;
  if (empty) return TV_OK;
  tv::DeviceInfo dev;
  if (int rc = tv::current_device_info(&dev)) return rc;
  cudaStream_t s = (cudaStream_t)stream;
  return dtype == TV_BF16 ? dispatch_append<__nv_bfloat16>(p, head_dim, dev.sm_count, s)
                          : dispatch_append<float>(p, head_dim, dev.sm_count, s);
}
