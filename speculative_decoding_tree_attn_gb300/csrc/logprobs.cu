// Log probabilities of given tokens under rows of logits, with entropy and
// top alternatives.
//
// With m = max x, S = sum e^(x - m):  ln p_i = x_i - m - ln S,
// H = ln S - (1/S) sum e^(x - m) (x - m).  Alternatives are ordered by one
// whole number per logit: its value's bits in ascending order above its
// index's complement, so equal values go to the lower index.  "Encode branch
// histories in masks and positions": node i's logits predict the token emitted
// at it.
//
// One CTA per entry: a pass for (m, S, sum), then one pass per alternative for
// the largest key below the last one.
#include <cmath>

#include <cuda_bf16.h>

#include "common.h"

namespace {

struct LogprobParams {
  const void* logits;
  const int32_t* tokens;
  const int32_t* node;
  int B, N, C, V;
  float* logprob;
  float* entropy;
  int top_k;
  int32_t* top_ids;
  float* top_logprobs;
  int32_t* status;
};

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }

// Larger key: larger value, then lower index; NaN as -inf, -0 as +0.
__device__ __forceinline__ uint64_t order_key(float x, int i) {
  x = x == x ? x + 0.f : -INFINITY;
  const uint32_t u = __float_as_uint(x);
  const uint32_t o = u & 0x80000000u ? ~u : u | 0x80000000u;
  return (uint64_t)o << 32 | (uint32_t)~i;
}

template <typename T>
__global__ void __launch_bounds__(256) logprob_kernel(LogprobParams p) {
  const int64_t e = blockIdx.x;
  const int b = (int)(e / p.C), c = (int)(e % p.C);
  const int tok = p.tokens[e];
  const int node = p.node ? p.node[e] : c;
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  __shared__ float sm[8], ss[8], sx[8];
  __shared__ uint64_t sk[8];
  if (tok < 0 || tok >= p.V || node < 0 || node >= p.N) {
    if (tid == 0) {
      int bad = 0;
      if (tok != -1 && (tok < 0 || tok >= p.V)) bad |= TV_DEV_BAD_TOKEN;
      if (node != -1 && (node < 0 || node >= p.N)) bad |= TV_DEV_BAD_TOPOLOGY;
      if (bad && p.status) atomicOr(p.status, bad);
      p.logprob[e] = 0.f;
      if (p.entropy) p.entropy[e] = 0.f;
    }
    for (int k = tid; k < p.top_k; k += blockDim.x) {
      p.top_ids[e * p.top_k + k] = -1;
      p.top_logprobs[e * p.top_k + k] = -INFINITY;
    }
    return;
  }
  const T* row = static_cast<const T*>(p.logits) + ((int64_t)b * p.N + node) * p.V;
  float m = -INFINITY;
  for (int i = tid; i < p.V; i += 256) m = fmaxf(m, to_f32(row[i]));
  for (int w = 16; w; w >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, w));
  if (lane == 0) sm[warp] = m;
  __syncthreads();
  for (int w = 0; w < 8; ++w) m = fmaxf(m, sm[w]);
  float s = 0.f, x1 = 0.f;
  for (int i = tid; i < p.V; i += 256) {
    const float d = to_f32(row[i]) - m, ex = expf(d);
    s += ex;
    x1 += d == -INFINITY ? 0.f : ex * d;
  }
  for (int w = 16; w; w >>= 1) {
    s += __shfl_xor_sync(0xffffffffu, s, w);
    x1 += __shfl_xor_sync(0xffffffffu, x1, w);
  }
  if (lane == 0) {
    ss[warp] = s;
    sx[warp] = x1;
  }
  __syncthreads();
  s = x1 = 0.f;
  for (int w = 0; w < 8; ++w) {
    s += ss[w];
    x1 += sx[w];
  }
  const float ln_s = logf(s);
  if (tid == 0) {
    p.logprob[e] = to_f32(row[tok]) - m - ln_s;
    if (p.entropy) p.entropy[e] = ln_s - x1 / s;
  }
  uint64_t last = ~0ull;
  for (int k = 0; k < p.top_k; ++k) {
    uint64_t best = 0;
    for (int i = tid; i < p.V; i += 256) {
      const uint64_t key = order_key(to_f32(row[i]), i);
      if (key < last && key > best) best = key;
    }
    for (int w = 16; w; w >>= 1) {
      const uint64_t o = __shfl_xor_sync(0xffffffffu, best, w);
      best = o > best ? o : best;
    }
    if (lane == 0) sk[warp] = best;
    __syncthreads();
    for (int w = 0; w < 8; ++w) best = sk[w] > best ? sk[w] : best;
    __syncthreads();
    if (tid == 0) {
      const int id = (int)~(uint32_t)best;
      p.top_ids[e * p.top_k + k] = id;
      p.top_logprobs[e * p.top_k + k] = to_f32(row[id]) - m - ln_s;
    }
    last = best;
  }
}

}  // namespace

extern "C" int tv_token_logprobs(const void* logits, const int32_t* tokens, const int32_t* node, int32_t B, int32_t N,
                                 int32_t C, int32_t V, int32_t dtype, float* logprob, float* entropy, int32_t top_k,
                                 int32_t* top_ids, float* top_logprobs, int32_t* status, void* stream) {
  tv::clear_error();
  if (B < 0 || N < 1 || C < 0 || V < 1 || (!node && C > N))
    return tv::fail(TV_ERR_INVALID_ARG, "tv_token_logprobs: bad sizes");
  if (dtype != TV_F32 && dtype != TV_BF16) return tv::fail(TV_ERR_UNSUPPORTED, "tv_token_logprobs: dtype %d", dtype);
  if (top_k < 0 || top_k > TV_MAX_TOP_K || top_k > V)
    return tv::fail(TV_ERR_INVALID_ARG, "tv_token_logprobs: top_k %d not in [0, min(%d, V)]", top_k, TV_MAX_TOP_K);
  if (B == 0 || C == 0) return TV_OK;
  if (!logits || !tokens || !logprob || (top_k && (!top_ids || !top_logprobs)))
    return tv::fail(TV_ERR_INVALID_ARG, "tv_token_logprobs: null pointer");
  if (reinterpret_cast<uintptr_t>(logits) & 15)
    return tv::fail(TV_ERR_INVALID_ARG, "tv_token_logprobs: logits must be 16-byte aligned");
  if ((int64_t)B * C >= INT32_MAX)
    return tv::fail(TV_ERR_UNSUPPORTED, "tv_token_logprobs: B * C exceeds 2^31");
  LogprobParams p{logits, tokens, node, B, N, C, V, logprob, entropy, top_k, top_ids, top_logprobs, status};
  const unsigned grid = (unsigned)(B * C);
  if (dtype == TV_BF16)
    logprob_kernel<__nv_bfloat16><<<grid, 256, 0, (cudaStream_t)stream>>>(p);
  else
    logprob_kernel<float><<<grid, 256, 0, (cudaStream_t)stream>>>(p);
  TV_LAUNCH_CHECK("logprob_kernel");
  return TV_OK;
}
