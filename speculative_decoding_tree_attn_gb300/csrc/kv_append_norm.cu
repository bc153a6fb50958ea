// Appending new tokens' keys and values to the paged cache, keys and queries
// normalised per head and rotated on the way.
//
// A head's row x of D elements becomes
//   y = x * w / sqrt(sum x^2 / D + eps),   then its leading R elements turned
// by the position's angles, element i with i + R/2 (halves) or 2i with 2i + 1
// (pairs).  Sum, factor and rotation are float32, the row is rounded once.
// Where a token goes is tv_kv_append's (kv_place.cuh); "Tree Verification",
// "The Cost Side": the cached prefix keys are stored as attention reads them.
//
// Bound by HBM: a row is read once and written once.  A head's row lies in the
// registers of D / 16 neighbouring lanes as two runs of 8 elements each, so
// its sum of squares is a sum over 16 registers and log2(D / 16) exchanges,
// and the runs are picked so that a rotation's partners meet in one lane.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include <cuda_bf16.h>

#include "common.h"
#include "kv_place.cuh"
#include "rope_math.cuh"

namespace {

constexpr int kThreads = 128;

struct NormParams {
  AppendParams a;
  const char* q_weight;  // nullable: queries are not normalised
  const char* k_weight;
  float eps;
  int rot;  // elements that are rotated, a multiple of 16
  int pairs;
};

template <typename T>
constexpr int kVec = 8 * (int)sizeof(T) / 16;  // 16-byte vectors per 8 elements

template <typename T>
__device__ __forceinline__ void unpack(const Raw<kVec<T>>& r, float (&v)[8]) {
  Vec8<T>::load(reinterpret_cast<const T*>(&r), v);
}

// One head's row: a lane's two runs of 8, normalised with the weights at w (null: not), runs lo and hi of them, and rotated.
template <typename T, int D>
__device__ __forceinline__ void finish_row(const NormParams& p, const char* w_at, int64_t lo, int64_t hi, bool turn,
                                           const Raw<kVec<T>>& x1, const Raw<kVec<T>>& x2, const float (&co)[8],
                                           const float (&si)[8], float (&a)[8], float (&d)[8]) {
  unpack<T>(x1, a);
  unpack<T>(x2, d);
  float sum = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) sum += a[e] * a[e] + d[e] * d[e];
#pragma unroll
  for (int o = 1; o < D / 16; o *= 2) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (w_at) {  // read for each head (they stay in L1): kept in registers they left a third less room for the rows
    const float f = 1.f / sqrtf(sum * (1.f / D) + p.eps);
    float w[8];
    unpack<T>(*reinterpret_cast<const Raw<kVec<T>>*>(w_at + lo), w);
#pragma unroll
    for (int e = 0; e < 8; ++e) a[e] = a[e] * f * w[e];
    unpack<T>(*reinterpret_cast<const Raw<kVec<T>>*>(w_at + hi), w);
#pragma unroll
    for (int e = 0; e < 8; ++e) d[e] = d[e] * f * w[e];
  }
  if (!turn) return;
  if (p.pairs) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      rope_pair(a[2 * e], a[2 * e + 1], co[e], si[e], a[2 * e], a[2 * e + 1]);
      rope_pair(d[2 * e], d[2 * e + 1], co[4 + e], si[4 + e], d[2 * e], d[2 * e + 1]);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) rope_pair(a[e], d[e], co[e], si[e], a[e], d[e]);
  }
}

// One warp per (token, slice of its heads), as in kv_append.cu; the warps behind the tokens' count the new lengths.  5 CTAs
// an SM leave 96 registers, of which bf16 spills 24 bytes.  With 4 | 5 | 6: 17k tokens of 32/8 heads of 128 in bf16 109 | 72 |
// 73 us, 256 such tokens 5.6 | 5.0 | 5.7, 32 float32 prompts of up to 600 88 | 85 | 81.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 5) kv_append_norm_kernel(const __grid_constant__ NormParams np) {
  const AppendParams& p = np.a;
  constexpr int kChunks = D / 16;
  constexpr int kHeads = 32 / kChunks;          // heads a warp covers at once
  constexpr int kRow = D * (int)sizeof(T);      // bytes of a head's row
  constexpr int kUnroll = 8 / (int)sizeof(T);   // 128 bytes of a lane on their way at once
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

  // the lane's runs: a rotation's partners where the chunk is rotated, the next 16 elements where it is not
  const int c = lane % kChunks;
  const bool turn = c < np.rot / 16;
  const int e1 = turn && !np.pairs ? 8 * c : 16 * c;
  const int e2 = turn && !np.pairs ? np.rot / 2 + 8 * c : 16 * c + 8;
  float co[8], si[8];
  if (turn) {
    const float* row = p.cs + pos * np.rot + c * 8;
    Vec8<float>::load(row, co);
    Vec8<float>::load(row + np.rot / 2, si);
  }
  const int64_t lo = e1 * sizeof(T), hi = e2 * sizeof(T);
  using Run = Raw<kVec<T>>;
  const int Hq = p.q ? p.Hq : 0;
  const int H = Hq + 2 * p.Hkv;
  const int rounds = (H + kHeads - 1) / kHeads;
  const int per = (rounds + p.slices - 1) / p.slices * kHeads;
  const int h_end = min(H, (s + 1) * per);
  // every lane takes the same turns: a row's sum is exchanged within the warp
  for (int g0 = s * per; g0 < h_end; g0 += kHeads * kUnroll) {
    const int h0 = g0 + lane / kChunks;
    Run x1[kUnroll], x2[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int h = h0 + u * kHeads;
      if (h >= h_end) {
        x1[u] = x2[u] = Run{};
        continue;
      }
      const char* src = h < Hq ? p.q + t * p.q_stride + (int64_t)h * kRow
                      : h < Hq + p.Hkv ? p.k + t * p.k_stride + (int64_t)(h - Hq) * kRow
                                       : p.v + t * p.v_stride + (int64_t)(h - Hq - p.Hkv) * kRow;
      x1[u] = *reinterpret_cast<const Run*>(src + lo);
      x2[u] = *reinterpret_cast<const Run*>(src + hi);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (g0 + u * kHeads >= h_end) break;
      const int h = h0 + u * kHeads;
      const bool is_q = h < Hq, is_v = h >= Hq + p.Hkv;
      float y1[8], y2[8];
      finish_row<T, D>(np, is_q ? np.q_weight : is_v ? nullptr : np.k_weight, lo, hi, turn, x1[u], x2[u], co, si, y1, y2);
      if (h >= h_end || (!is_q && !placed)) continue;
      char* dst;
      if (is_q) {
        dst = p.q_out + t * p.q_out_stride + (int64_t)h * kRow;
      } else {
        const int kh = h - Hq - (is_v ? p.Hkv : 0);
        dst = (is_v ? p.v_cache : p.k_cache) + ((blk * p.Hkv + kh) * p.block_size + slot) * kRow;
      }
      if (is_v) {
        *reinterpret_cast<Run*>(dst + lo) = x1[u];
        *reinterpret_cast<Run*>(dst + hi) = x2[u];
      } else {
        Vec8<T>::store(reinterpret_cast<T*>(dst + lo), y1);
        Vec8<T>::store(reinterpret_cast<T*>(dst + hi), y2);
      }
    }
  }
}

template <typename T, int D>
void launch_norm(NormParams p, int sm_count, cudaStream_t stream) {
  constexpr int kHeads = 32 / (D / 16);
  const int H = (p.a.q ? p.a.Hq : 0) + 2 * p.a.Hkv;
  const int rounds = (H + kHeads - 1) / kHeads;
  // few tokens: several warps share one, so that a step's tokens reach every SM
  const int64_t want = (int64_t)sm_count * 8;
  p.a.slices = (int)std::max<int64_t>(1, std::min<int64_t>(rounds, want / std::max(1, p.a.T)));
  const int64_t warps = (int64_t)p.a.T * p.a.slices + p.a.B;
  kv_append_norm_kernel<T, D><<<(unsigned)tv::ceil_div(warps, kThreads / 32), kThreads, 0, stream>>>(p);
}

template <typename T>
int dispatch_norm(const NormParams& p, int D, int sm_count, cudaStream_t stream) {
  switch (D) {
    case 16: launch_norm<T, 16>(p, sm_count, stream); break;
    case 32: launch_norm<T, 32>(p, sm_count, stream); break;
    case 64: launch_norm<T, 64>(p, sm_count, stream); break;
    case 128: launch_norm<T, 128>(p, sm_count, stream); break;
    default: launch_norm<T, 256>(p, sm_count, stream); break;
  }
  TV_LAUNCH_CHECK("kv_append_norm_kernel");
  return TV_OK;
}

}  // namespace

extern "C" int tv_kv_append_norm(const void* q, int64_t q_stride, const void* q_weight, void* q_out,
                                 int64_t q_out_stride, int32_t Hq, const void* k_new, int64_t k_stride,
                                 const void* k_weight, const void* v_new, int64_t v_stride, float eps,
                                 const int32_t* cu_new, int32_t T, void* k_cache, void* v_cache, int64_t num_blocks,
                                 int32_t block_size, const int32_t* block_table, int32_t max_blocks,
                                 const int32_t* seq_lens, int32_t* new_seq_lens, const float* cos_sin, int32_t max_pos,
                                 int32_t rot_dim, int32_t interleaved, int32_t B, int32_t Hkv, int32_t head_dim,
                                 int32_t dtype, int32_t* status, void* stream) {
  tv::clear_error();
  NormParams p{};
  bool empty;
  if (int rc = append_params("tv_kv_append_norm", q, q_stride, q_out, q_out_stride, Hq, k_new, k_stride, v_new, v_stride,
                             cu_new, T, k_cache, v_cache, num_blocks, block_size, block_table, max_blocks, seq_lens,
                             new_seq_lens, cos_sin, max_pos, false, B, Hkv, head_dim, dtype, status, &p.a, &empty))
    return rc;
  if (!(eps >= 0.f) || !std::isfinite(eps))
    return tv::fail(TV_ERR_INVALID_ARG, "tv_kv_append_norm: eps must be finite and not negative");
  if (cos_sin && (rot_dim < 16 || rot_dim % 16 || rot_dim > head_dim))
    return tv::fail(TV_ERR_INVALID_ARG, "tv_kv_append_norm: rot_dim %d not a multiple of 16 in [16, head_dim]", rot_dim);
  if (interleaved != 0 && interleaved != 1)
    return tv::fail(TV_ERR_INVALID_ARG, "tv_kv_append_norm: interleaved must be 0 or 1");
  if (empty) return TV_OK;
  if (q_weight && !q) return tv::fail(TV_ERR_INVALID_ARG, "tv_kv_append_norm: q_weight without q");
  if ((reinterpret_cast<uintptr_t>(q_weight) | reinterpret_cast<uintptr_t>(k_weight)) & 15)
    return tv::fail(TV_ERR_INVALID_ARG, "tv_kv_append_norm: weights must be 16-byte aligned");
  p.q_weight = static_cast<const char*>(q_weight);
  p.k_weight = static_cast<const char*>(k_weight);
  p.eps = eps;
  p.rot = cos_sin ? rot_dim : 0;
  p.pairs = interleaved;
  tv::DeviceInfo dev;
  if (int rc = tv::current_device_info(&dev)) return rc;
  cudaStream_t s = (cudaStream_t)stream;
  return dtype == TV_BF16 ? dispatch_norm<__nv_bfloat16>(p, head_dim, dev.sm_count, s)
                          : dispatch_norm<float>(p, head_dim, dev.sm_count, s);
}
