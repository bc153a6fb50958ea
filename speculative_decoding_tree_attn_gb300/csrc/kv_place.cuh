// Where new tokens go in the paged cache, shared by the kernels that append
// them: request and position of a packed row, and a request's new length.
#pragma once

#include <climits>
#include <cstdint>

#include "common.h"

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

template <int N>
struct Raw {
  uint4 v[N];
};

// Checks the arguments of an append call and fills its parameters (all but the split over warps); *empty: no requests.
// q_turned: queries are there to be rotated, so they need the table.
inline int append_params(const char* fn, const void* q, int64_t q_stride, void* q_out, int64_t q_out_stride, int32_t Hq,
                         const void* k_new, int64_t k_stride, const void* v_new, int64_t v_stride,
                         const int32_t* cu_new, int32_t T, void* k_cache, void* v_cache, int64_t num_blocks,
                         int32_t block_size, const int32_t* block_table, int32_t max_blocks, const int32_t* seq_lens,
                         int32_t* new_seq_lens, const float* cos_sin, int32_t max_pos, bool q_turned, int32_t B,
                         int32_t Hkv, int32_t head_dim, int32_t dtype, int32_t* status, AppendParams* out, bool* empty) {
  *empty = B == 0;
  if (B < 0 || T < 0 || Hkv < 1 || head_dim < 1 || block_size < 1 || max_blocks < 1 || num_blocks < 1 ||
      (q && Hq < 1) || (cos_sin && max_pos < 1))
    return tv::fail(TV_ERR_INVALID_ARG, "%s: bad sizes", fn);
  if (dtype != TV_F32 && dtype != TV_BF16) return tv::fail(TV_ERR_UNSUPPORTED, "%s: dtype %d", fn, dtype);
  if (head_dim != 16 && head_dim != 32 && head_dim != 64 && head_dim != 128 && head_dim != 256)
    return tv::fail(TV_ERR_UNSUPPORTED, "%s: head_dim %d not in {16, 32, 64, 128, 256}", fn, head_dim);
  if (B == 0) return TV_OK;
  if (!cu_new && T % B)
    return tv::fail(TV_ERR_INVALID_ARG, "%s: without offsets T (%d) must be a multiple of B (%d)", fn, T, B);
  if (!k_cache || !v_cache || !block_table || !seq_lens || (T > 0 && (!k_new || !v_new)))
    return tv::fail(TV_ERR_INVALID_ARG, "%s: null pointer", fn);
  if (q && q_turned && (!cos_sin || !q_out))
    return tv::fail(TV_ERR_INVALID_ARG, "%s: q needs cos_sin and q_out", fn);
  if (q && !q_out) return tv::fail(TV_ERR_INVALID_ARG, "%s: q needs q_out", fn);
  // shifted views of one buffer too: lengths are written while other requests' warps read theirs
  const uintptr_t len0 = reinterpret_cast<uintptr_t>(seq_lens), len1 = reinterpret_cast<uintptr_t>(new_seq_lens);
  if (new_seq_lens && (len0 > len1 ? len0 - len1 : len1 - len0) < sizeof(int32_t) * (size_t)B)
    return tv::fail(TV_ERR_INVALID_ARG, "%s: new_seq_lens must not alias seq_lens or overlap it", fn);
  const int64_t e = dtype == TV_F32 ? 4 : 2;
  const int64_t kv_row = (int64_t)Hkv * head_dim, q_row = (int64_t)Hq * head_dim;
  const bool many = T > 1;  // one token's strides do not matter
  if (many && (k_stride < 0 || v_stride < 0 || (q && (q_stride < 0 || q_out_stride < q_row))))
    return tv::fail(TV_ERR_INVALID_ARG, "%s: bad token stride", fn);
  if ((many && ((k_stride * e) % 16 || (v_stride * e) % 16 || (q && ((q_stride * e) % 16 || (q_out_stride * e) % 16)))) ||
      ((reinterpret_cast<uintptr_t>(k_cache) | reinterpret_cast<uintptr_t>(v_cache) |
        reinterpret_cast<uintptr_t>(k_new) | reinterpret_cast<uintptr_t>(v_new) | reinterpret_cast<uintptr_t>(q) |
        reinterpret_cast<uintptr_t>(q ? q_out : nullptr) | reinterpret_cast<uintptr_t>(cos_sin)) & 15))
    return tv::fail(TV_ERR_INVALID_ARG, "%s: buffers and token strides must be multiples of 16 bytes", fn);
  if (kv_row >= INT32_MAX / 4 || (q && q_row >= INT32_MAX / 4))
    return tv::fail(TV_ERR_UNSUPPORTED, "%s: a token's heads exceed 2^29 elements", fn);
  AppendParams& p = *out;
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
  return TV_OK;
}

}  // namespace
