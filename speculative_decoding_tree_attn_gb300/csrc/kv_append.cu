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
#include "rope_math.cuh"

namespace {

struct AppendParams {
  const char* q;  // nullable
  char* q_out;
  const char* k;
  const char* v;
  int64_t q_stride, q_out_stride, k_stride, v_stride;  // bytes between tokens
  char* k_cache;
  char* v_cache;
  int64_t num_blocks;
  int block_size;
  const int32_t* table;
  int max_blocks;
  const int32_t* cu;  // nullable: T / B tokens each
  const int32_t* seq_lens;
  int32_t* new_lens;  // nullable
  const float* cs;    // nullable: nothing is rotated
  int max_pos;        // rows of cs; without it the largest length an int32 holds
  int B, T, Hq, Hkv;
  int slices;  // warps per token
  int32_t* status;
};

// Largest b with cu[b] <= t.  A search takes the same turns for all rows between two that it leads to b (a turn asks
// whether cu[i] <= t), so a request's first and last row tell whether it finds all of them, in order or not.
// Every lane the same row, 32 probes a round:
struct WarpSearch {
  static __device__ __forceinline__ int request(const AppendParams& p, int t, int lane) {
    int lo = 0, hi = p.B;  // the answer is in [lo, hi)
    while (hi - lo > 1) {
      const int step = (hi - lo + 31) / 32;
      const int64_t i = (int64_t)lo + (int64_t)step * lane;
      const unsigned le = __ballot_sync(0xffffffffu, i < hi && __ldg(p.cu + i) <= t);
      lo += step * (le ? 31 - __clz(le) : 0);
      hi = min(hi, lo + step);
    }
    return lo;
  }
};
// a row a lane:
struct LaneSearch {
  static __device__ __forceinline__ int request(const AppendParams& p, int t, int) {
    int lo = 0;
    for (int hi = p.B; hi - lo > 1;) {
      const int mid = lo + (hi - lo) / 2;
      if (__ldg(p.cu + mid) <= t) lo = mid; else hi = mid;
    }
    return lo;
  }
};

// Request and index within it of packed row t; false for a row of no request.
template <class Search>
__device__ __forceinline__ bool find_request(const AppendParams& p, int t, int lane, int& b, int& j) {
  if (!p.cu) {
    const int per = p.T / p.B;
    b = t / per;
    j = t - b * per;
    return true;
  }
  b = Search::request(p, t, lane);
  const int s0 = __ldg(p.cu + b), s1 = __ldg(p.cu + b + 1);
  j = t - s0;
  return s0 >= 0 && s0 <= t && t < s1 && s1 <= p.T;
}

// New length of request b: the tokens before the first that cannot be placed.  Search is the one that the tokens' warps
// use.  Blocks are looked at 32 a trip to L2, behind the copies: one prompt of 32k tokens, 32/8 heads of 128, takes
// 149 us in blocks of 16 and 638 in blocks of 1, of a floor of 121.
template <class Search>
__device__ void count_request(const AppendParams& p, int b, int lane) {
  const int L = p.seq_lens[b];
  int n, bad = 0;
  if (p.cu) {
    const int s0 = p.cu[b], s1 = p.cu[b + 1];
    n = s1 - s0;
    if (s0 < 0 || s1 < s0 || s1 > p.T) {
      n = 0;
      bad = TV_DEV_BAD_OFFSETS;
    }
    // offsets of others, out of order, may lead some of its rows elsewhere or nowhere
    if (n > 0) {
      const int first = Search::request(p, s0, lane), last = Search::request(p, s1 - 1, lane);
      if (first != b || last != b) {
        n = 0;
        bad = TV_DEV_BAD_OFFSETS;
      }
    }
  } else {
    n = p.T / p.B;
  }
  if (L < 0) {
    n = 0;
    bad |= TV_DEV_BAD_POSITION;
  }
  if ((int64_t)L + n > p.max_pos) {
    n = max(0, p.max_pos - L);
    bad |= TV_DEV_BAD_POSITION;
  }
  if (n > 0) {
    const int64_t c1 = ((int64_t)L + n - 1) / p.block_size;
    for (int64_t c0 = L / p.block_size; c0 <= c1; c0 += 32) {
      const int64_t c = c0 + lane;
      bool miss = false;
      if (c <= c1) {
        const int64_t blk = c < p.max_blocks ? p.table[(int64_t)b * p.max_blocks + c] : -1;
        miss = blk < 0 || blk >= p.num_blocks;
      }
      const unsigned m = __ballot_sync(0xffffffffu, miss);
      if (m) {
        n = (int)max((int64_t)0, (c0 + __ffs(m) - 1) * p.block_size - L);
        bad |= TV_DEV_OUT_OVERFLOW;  // beside positions past the table: their queries are not written
        break;
      }
    }
  }
  if (lane == 0) {
    if (p.new_lens) p.new_lens[b] = L + n;
    if (bad && p.status) atomicOr(p.status, bad);
  }
}

constexpr int kThreads = 128;

template <int N>
struct Raw {
  uint4 v[N];
};

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
  if (B < 0 || T < 0 || Hkv < 1 || head_dim < 1 || block_size < 1 || max_blocks < 1 || num_blocks < 1 ||
      (q && Hq < 1) || (cos_sin && max_pos < 1))
    return tv::fail(TV_ERR_INVALID_ARG, "tv_kv_append: bad sizes");
  if (dtype != TV_F32 && dtype != TV_BF16) return tv::fail(TV_ERR_UNSUPPORTED, "tv_kv_append: dtype %d", dtype);
  if (head_dim != 16 && head_dim != 32 && head_dim != 64 && head_dim != 128 && head_dim != 256)
    return tv::fail(TV_ERR_UNSUPPORTED, "tv_kv_append: head_dim %d not in {16, 32, 64, 128, 256}", head_dim);
  if (B == 0) return TV_OK;
  if (!cu_new && T % B)
    return tv::fail(TV_ERR_INVALID_ARG, "tv_kv_append: without offsets T (%d) must be a multiple of B (%d)", T, B);
  if (!k_cache || !v_cache || !block_table || !seq_lens || (T > 0 && (!k_new || !v_new)))
    return tv::fail(TV_ERR_INVALID_ARG, "tv_kv_append: null pointer");
  if (q && (!cos_sin || !q_out))
    return tv::fail(TV_ERR_INVALID_ARG, "tv_kv_append: q needs cos_sin and q_out");
  // shifted views of one buffer too: lengths are written while other requests' warps read theirs
  const uintptr_t len0 = reinterpret_cast<uintptr_t>(seq_lens), len1 = reinterpret_cast<uintptr_t>(new_seq_lens);
  if (new_seq_lens && (len0 > len1 ? len0 - len1 : len1 - len0) < sizeof(int32_t) * (size_t)B)
    return tv::fail(TV_ERR_INVALID_ARG, "tv_kv_append: new_seq_lens must not alias seq_lens or overlap it");
  const int64_t e = dtype == TV_F32 ? 4 : 2;
  const int64_t kv_row = (int64_t)Hkv * head_dim, q_row = (int64_t)Hq * head_dim;
  const bool many = T > 1;  // one token's strides do not matter
  if (many && (k_stride < 0 || v_stride < 0 || (q && (q_stride < 0 || q_out_stride < q_row))))
    return tv::fail(TV_ERR_INVALID_ARG, "tv_kv_append: bad token stride");
  if ((many && ((k_stride * e) % 16 || (v_stride * e) % 16 || (q && ((q_stride * e) % 16 || (q_out_stride * e) % 16)))) ||
      ((reinterpret_cast<uintptr_t>(k_cache) | reinterpret_cast<uintptr_t>(v_cache) |
        reinterpret_cast<uintptr_t>(k_new) | reinterpret_cast<uintptr_t>(v_new) | reinterpret_cast<uintptr_t>(q) |
        reinterpret_cast<uintptr_t>(q ? q_out : nullptr) | reinterpret_cast<uintptr_t>(cos_sin)) & 15))
    return tv::fail(TV_ERR_INVALID_ARG, "tv_kv_append: buffers and token strides must be multiples of 16 bytes");
  if (kv_row >= INT32_MAX / 4 || (q && q_row >= INT32_MAX / 4))
    return tv::fail(TV_ERR_UNSUPPORTED, "tv_kv_append: a token's heads exceed 2^29 elements");
  tv::DeviceInfo dev;
  if (int rc = tv::current_device_info(&dev)) return rc;
  AppendParams p{};
  p.q = static_cast<const char*>(q);
  p.q_out = static_cast<char*>(q_out);
  p.k = static_cast<const char*>(k_new);
  p.v = static_cast<const char*>(v_new);
  p.q_stride = q_stride * e;
  p.q_out_stride = q_out_stride * e;
  p.k_stride = k_stride * e;
  p.v_stride = v_stride * e;
  p.k_cache = static_cast<char*>(k_cache);
  p.v_cache = static_cast<char*>(v_cache);
  p.num_blocks = num_blocks;
  p.block_size = block_size;
  p.table = block_table;
  p.max_blocks = max_blocks;
  p.cu = cu_new;
  p.seq_lens = seq_lens;
  p.new_lens = new_seq_lens;
  p.cs = cos_sin;
  p.max_pos = cos_sin ? max_pos : INT32_MAX;
  p.B = B;
  p.T = T;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.status = status;
  cudaStream_t s = (cudaStream_t)stream;
  return dtype == TV_BF16 ? dispatch_append<__nv_bfloat16>(p, head_dim, dev.sm_count, s)
                          : dispatch_append<float>(p, head_dim, dev.sm_count, s);
}
