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
// One pass: a row is read once, by a cluster of 1-8 CTAs (the fewer rows, the
// more), in 16-byte vectors that each thread copies to its own places in shared
// memory two batches ahead (no barrier; 32 KB in flight a CTA, 4 CTAs an SM).
// Bound by HBM for float32 (1000 rows of 128,000: 82 us, 0.92 of the measured copy
// rate), by the issue slots for bf16: an element costs eight instructions
// (unpacking, its place in the maximum, one exponential, three for the sums), ten
// with alternatives; 1999 rows of 128,000 bf16 logits take 94 us with 5
// alternatives (0.80 of the copy rate, 78 % of the slots issued), 82 us without.
// Everything is summed in the log2 domain against r = fl(m log2 e): with S = sum
// 2^(x log2 e - r) the rounding of r cancels in x log2 e - r - log2 S, and a
// distance is one FMA.
//
// The alternatives cost little beside that.  A thread's maximum is kept anyway, and
// the top_k-th of the warps' 4 largest each is a bar that at least top_k elements
// reach, and few more.  Only keys above the bar are written down, in the warp's
// buffer; where one fills up (equal logits, an order of its own), the warp sorts it
// into a list whose top_k-th key is its own bar from then on.  At the end the CTA's
// keys above the last bar are ranked by counting.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include <algorithm>
#include <cfloat>

#include "common.h"

namespace cg = cooperative_groups;

namespace {

struct LogprobParams {
  const char* logits;
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

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kVectors = 4;  // of a thread at a time
constexpr int kStages = 3;
constexpr int kRing = kStages * kVectors * kThreads * 16;
constexpr int kTold = 32 / kWarps;  // thread maxima that a warp tells the others
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLeast = -0x1p100f;

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if either is
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

// Larger key: larger value, then lower index; NaN as -inf, -0 as +0.  0 is below every key.
__device__ __forceinline__ uint64_t order_key(float x, int i) {
  x = x == x ? x + 0.f : -INFINITY;
  const uint32_t u = __float_as_uint(x);
  const uint32_t o = u & 0x80000000u ? ~u : u | 0x80000000u;
  return (uint64_t)o << 32 | (uint32_t)~i;
}
__device__ __forceinline__ float key_value(uint64_t key) {
  const uint32_t o = (uint32_t)(key >> 32);
  return o == 0 ? -INFINITY : __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
}

__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int kN = 4;
  static constexpr uint32_t kMinusInf = 0xff800000u;
  static __device__ __forceinline__ float largest(uint4 v) {  // NaN if one is
    return max_nan(max_nan(__uint_as_float(v.x), __uint_as_float(v.y)),
                   max_nan(__uint_as_float(v.z), __uint_as_float(v.w)));
  }
  static __device__ __forceinline__ uint4 held(uint4 v) {  // at least kLeast
    return make_uint4(__float_as_uint(fmaxf(__uint_as_float(v.x), kLeast)), __float_as_uint(fmaxf(__uint_as_float(v.y), kLeast)),
                      __float_as_uint(fmaxf(__uint_as_float(v.z), kLeast)), __float_as_uint(fmaxf(__uint_as_float(v.w), kLeast)));
  }
  static __device__ __forceinline__ void unpack(uint4 v, float (&x)[kN]) {
    x[0] = __uint_as_float(v.x), x[1] = __uint_as_float(v.y), x[2] = __uint_as_float(v.z), x[3] = __uint_as_float(v.w);
  }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int kN = 8;
  static constexpr uint32_t kMinusInf = 0xff80ff80u;
  static __device__ __forceinline__ float largest(uint4 v) {
    uint32_t m;
    asm("{\n\t.reg .b32 a, b;\n\tmax.NaN.bf16x2 a, %1, %2;\n\tmax.NaN.bf16x2 b, %3, %4;\n\tmax.NaN.bf16x2 %0, a, b;\n\t}"
        : "=r"(m)
        : "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w));
    return max_nan(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
  }
  static __device__ __forceinline__ uint4 held(uint4 v) {
    auto two = [](uint32_t x) {
      uint32_t y;
      asm("max.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(x), "r"(0xf180f180u));  // -2^100
      return y;
    };
    return make_uint4(two(v.x), two(v.y), two(v.z), two(v.w));
  }
  static __device__ __forceinline__ void unpack(uint4 v, float (&x)[kN]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};
__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }

// m: the largest x, or up to 8 less; against r = fl(m log2 e), d = x log2 e - r: s = sum 2^d, t = sum 2^d d.
// Logits are held at -2^100, whose power is 0 (an excluded one's infinite distance
// would make its product NaN).  The maximum's own distance is r's rounding, which
// has to stay small: for |m| > 2^20 (no logits of a model), d = (x - m) log2 e, held
// at -300.
constexpr float kFar = -300.f;
__device__ __forceinline__ float reference(float m) { return m == -INFINITY ? 0.f : __fmul_rn(m, kLog2e); }
__device__ __forceinline__ bool huge(float m) { return fabsf(m) > 1048576.f && m != -INFINITY; }
__device__ __forceinline__ float distance(float x, float m) {
  return huge(m) ? (x - m) * kLog2e : __fmaf_rn(x, kLog2e, -reference(m));
}
// From m's reference to m2's: both rounded, one exact, or both exact.
__device__ __forceinline__ float step(float m, float m2) {
  if (!huge(m)) return huge(m2) ? __fmaf_rn(-m2, kLog2e, reference(m)) : reference(m) - reference(m2);
  return distance(m, m2);
}
struct Sums {
  float m, s, t;
  __device__ __forceinline__ void raise(float m2) {  // to a larger maximum
    const float d = m == -INFINITY ? kFar : fmaxf(step(m, m2), kFar);
    const float c = exp2_approx(d);
    t = c * fmaf(d, s, t);
    s *= c;
    m = m2;
  }
  __device__ __forceinline__ void add(float d) {
    const float e = exp2_approx(d);
    s += e;
    t = fmaf(e, d, t);
  }
};
__device__ __forceinline__ Sums warp_join(Sums a) {  // every lane the same result
  float m = a.m;
#pragma unroll
  for (int w = 16; w; w >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, w));
  if (a.m < m) a.raise(m);
#pragma unroll
  for (int w = 16; w; w >>= 1) {
    a.s += __shfl_xor_sync(0xffffffffu, a.s, w);
    a.t += __shfl_xor_sync(0xffffffffu, a.t, w);
  }
  return a;
}

// n + (a >= b), b > 0, from b's negative: a - b carries out of 32 bits.
__device__ __forceinline__ uint32_t count_ge(uint32_t n, uint32_t a, uint32_t minus_b) {
  asm("{\n\t.reg .u32 t;\n\tadd.cc.u32 t, %1, %2;\n\taddc.u32 %0, %0, 0;\n\t}" : "+r"(n) : "r"(a), "r"(minus_b));
  return n;
}

// The candidates of a warp: keys above the bar wait in its buffer in shared memory;
// when there are 32 they are sorted into a list, one key per lane, descending.
struct Best {
  uint64_t mine = 0, bar = 0;  // top_k keys of the row are at least the bar
  float bar_value = -INFINITY;
  int waiting = 0;

  __device__ __forceinline__ void raise(uint64_t key) {
    if (key > bar) {
      bar = key;
      bar_value = key_value(key);
    }
  }
  __device__ __forceinline__ void offer(uint64_t key, uint64_t* buffer, int k, int lane) {  // every lane its key
    const unsigned hit = __ballot_sync(0xffffffffu, key > bar);
    if (key > bar) buffer[waiting + __popc(hit & ((1u << lane) - 1))] = key;
    waiting += __popc(hit);
    if (waiting >= 32) take(buffer, k, lane);
  }
  __device__ void take(uint64_t* buffer, int k, int lane) {  // the first 32 waiting
    __syncwarp();
    uint64_t x = buffer[lane];
    const uint64_t rest = 32 + lane < waiting ? buffer[32 + lane] : 0;
    __syncwarp();
    if (32 + lane < waiting) buffer[lane] = rest;
    waiting -= 32;
#pragma unroll 1
    for (int size = 2; size <= 32; size <<= 1)
#pragma unroll 1
      for (int w = size >> 1; w; w >>= 1) {
        const uint64_t o = __shfl_xor_sync(0xffffffffu, x, w);
        x = (!(lane & size) == !(lane & w)) == (x > o) ? x : o;  // blocks descend where the size's bit is clear
      }
    join(x, lane);
    raise(__shfl_sync(0xffffffffu, mine, k - 1));
  }
  // The 32 largest of two descending lists.
  __device__ __forceinline__ void join(uint64_t other, int lane) {
    const uint64_t o = __shfl_sync(0xffffffffu, other, 31 - lane);
    mine = o > mine ? o : mine;
#pragma unroll 1
    for (int w = 16; w; w >>= 1) {
      const uint64_t x = __shfl_xor_sync(0xffffffffu, mine, w);
      mine = !(lane & w) == (mine > x) ? mine : x;
    }
  }
  // This warp's 4 largest thread maxima, for the bar.
  __device__ __forceinline__ void tell(uint32_t* shared, float m, int lane) const {
    uint32_t o = (uint32_t)(order_key(m, 0) >> 32), mine4 = 0;
#pragma unroll
    for (int j = 0; j < kTold; ++j) {
      const uint32_t v = __reduce_max_sync(0xffffffffu, o);
      if (lane == j) mine4 = v;
      if (lane == __ffs(__ballot_sync(0xffffffffu, o == v)) - 1) o = 0;
    }
    if (lane < kTold) *(volatile uint32_t*)(shared + lane) = mine4;
  }
  // The k-th of all warps'.  Others may write theirs meanwhile (volatile on both sides: every number is one that its
  // warp told, though four need not be of one time).  A warp's j-th number only grows, as its lanes' maxima do, so a mix
  // of times is nowhere above the latest numbers: no fewer than k elements reach the bar.  (A lane that meets a NaN tells
  // less from then on; the element behind what it told before is still there.)
  __device__ __forceinline__ void heed(const uint32_t* shared, int k, int lane) {
    const uint32_t at = (uint32_t)__cvta_generic_to_shared(shared);
    uint32_t v;
    asm volatile("ld.volatile.shared.u32 %0, [%1];" : "=r"(v) : "r"(at + 4 * lane) : "memory");
    uint32_t reach = 0;
#pragma unroll
    for (int j = 0; j < 32; j += 4) {
      uint4 o;
      asm volatile("ld.volatile.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(o.x), "=r"(o.y), "=r"(o.z), "=r"(o.w)
                   : "r"(at + 4 * j)
                   : "memory");
      reach = count_ge(count_ge(count_ge(count_ge(reach, o.x, -v), o.y, -v), o.z, -v), o.w, -v);
    }
    // under every index of that value
    raise((uint64_t)__reduce_max_sync(0xffffffffu, reach >= (uint32_t)k ? v : 0u) << 32);
  }
};

template <typename T, bool kTop>
__global__ void __launch_bounds__(kThreads, 4) logprob_kernel(const LogprobParams p) {
  using V_ = Vec<T>;
  constexpr int kN = V_::kN;
  cg::cluster_group cluster = cg::this_cluster();
  const int ctas = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int64_t e = blockIdx.x / ctas;
  const int b = (int)(e / p.C), c = (int)(e - (int64_t)b * p.C);
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int tok = __ldg(p.tokens + e);
  const int node = p.node ? __ldg(p.node + e) : c;
  __shared__ Sums s_sums[kWarps + 1];
  __shared__ int s_bad;
  __shared__ uint64_t s_wait[kWarps][64], s_best[32];
  extern __shared__ __align__(16) char s_ring[];
  uint64_t* s_pool = reinterpret_cast<uint64_t*>(s_ring);  // [kWarps * 64], once the stream is over
  __shared__ __align__(16) uint32_t s_bar[32];
  __shared__ int s_pool_size;
  if (tok < 0 || tok >= p.V || node < 0 || node >= p.N) {  // no entry: the same for the whole cluster
    if (rank == 0) {
      if (tid == 0) {
        int bad = 0;
        if (tok != -1 && (tok < 0 || tok >= p.V)) bad |= TV_DEV_BAD_TOKEN;
        if (node != -1 && (node < 0 || node >= p.N)) bad |= TV_DEV_BAD_TOPOLOGY;
        if (bad && p.status) atomicOr(p.status, bad);
        p.logprob[e] = 0.f;
        if (p.entropy) p.entropy[e] = 0.f;
      }
      if (kTop && tid < p.top_k) {
        p.top_ids[e * p.top_k + tid] = -1;
        p.top_logprobs[e * p.top_k + tid] = -INFINITY;
      }
    }
    return;
  }
  const T* row = reinterpret_cast<const T*>(p.logits) + ((int64_t)b * p.N + node) * p.V;
  // elements before the first 16-byte boundary, vectors, elements behind the last
  const int lead = min(p.V, (int)((16 - (reinterpret_cast<uintptr_t>(row) & 15)) % 16 / sizeof(T)));
  const int vectors = (p.V - lead) / kN;
  const int loose = p.V - vectors * kN;
  const uint4* vec = reinterpret_cast<const uint4*>(row + lead);
  const int v0 = (int)((int64_t)vectors * rank / ctas), v1 = (int)((int64_t)vectors * (rank + 1) / ctas);
  const float x_tok = tid == 0 && rank == 0 ? to_f32(row[tok]) : 0.f;

  Sums sums = {-INFINITY, 0.f, 0.f};
  Best best;
  float peak = -INFINITY;  // the largest logit, or a NaN
  // this thread's places in the ring: [stage][vector]; a vector past the end is all -inf there
  constexpr int kBatch = kThreads * kVectors, kStageBytes = kBatch * 16;
  const uint32_t ring = (uint32_t)__cvta_generic_to_shared(s_ring) + tid * 16;
  const uint4* from = vec + v0 + tid;
  int left = v1 - v0 - tid;  // vectors that this thread has yet to fetch, in steps of kThreads
  auto fetch = [&](uint32_t to) {
#pragma unroll
    for (int u = 0; u < kVectors; ++u) {
      if (left > u * kThreads)
        cp_async16(to + u * kThreads * 16, from + u * kThreads);
      else
        asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(to + u * kThreads * 16), "r"(V_::kMinusInf) : "memory");
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    from += kBatch;
    left -= kBatch;
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) fetch(ring + i * kStageBytes);
  if (kTop) {
    if (tid < 32) s_bar[tid] = 0;
    if (tid == 0) s_pool_size = 0;
    __syncthreads();
  }
  uint32_t at = ring, to = ring + (kStages - 1) * kStageBytes;
  float limit = -INFINITY;  // sums are raised to a maximum 8 above their own: powers of up to 2^12 until then
  bool far = false;         // huge(sums.m)
  int refresh = v0;         // the batch after which the bar is raised: the 1st, 2nd, 6th, 22nd, ..
#pragma unroll 1
  for (int base = v0; base < v1; base += kBatch) {  // the same for every warp of the CTA
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
    fetch(to);
    uint4 now[kVectors];
    float top[kVectors];
#pragma unroll
    for (int u = 0; u < kVectors; ++u) {
      now[u] = lds128(at + u * kThreads * 16);
      top[u] = V_::largest(now[u]);
    }
    float m = top[0];
#pragma unroll
    for (int u = 1; u < kVectors; ++u) m = max_nan(m, top[u]);
    peak = max_nan(peak, m);
    if (m > limit) {
      sums.raise(m);
      limit = m + 8.f;
      far = huge(m);
    }
    if (far) {
#pragma unroll 1
      for (int u = 0; u < kVectors; ++u) {
        float x[kN];
        V_::unpack(lds128(at + u * kThreads * 16), x);
#pragma unroll
        for (int i = 0; i < kN; ++i) sums.add(fmaxf((x[i] - sums.m) * kLog2e, kFar));
      }
    } else {
      // two at a time in a register pair: three instructions for both besides their exponentials
      const float r = reference(sums.m);
      const uint64_t scale = pack2(kLog2e, kLog2e), shift = pack2(-r, -r);
      uint64_t s2 = 0, t2 = 0;
#pragma unroll
      for (int u = 0; u < kVectors; ++u) {
        float x[kN];
        V_::unpack(V_::held(now[u]), x);
#pragma unroll
        for (int i = 0; i < kN; i += 2) {
          const uint64_t d = fma2(pack2(x[i], x[i + 1]), scale, shift);
          const float2 y = unpack2(d);
          const uint64_t e = pack2(exp2_approx(y.x), exp2_approx(y.y));
          s2 = add2(s2, e);
          t2 = fma2(e, d, t2);
        }
      }
      const float2 a = unpack2(s2), b = unpack2(t2);
      sums.s += a.x + a.y;
      sums.t += b.x + b.y;
    }
    if (kTop) {
      if (base == refresh) {
        best.tell(s_bar + warp * kTold, peak, lane);
        if (base == v0) __syncthreads();
        best.heed(s_bar, p.top_k, lane);
        refresh = v0 + 4 * (base - v0) + kBatch;
      }
      if (__any_sync(0xffffffffu, !(m < best.bar_value))) {
        unsigned vectors_hit = 0;
#pragma unroll
        for (int u = 0; u < kVectors; ++u)
          if (__any_sync(0xffffffffu, !(top[u] < best.bar_value))) vectors_hit |= 1u << u;
#pragma unroll 1
        while (vectors_hit) {  // few: read again, which leaves the registers to the stream
          const int u = __ffs(vectors_hit) - 1;
          vectors_hit &= vectors_hit - 1;
          const int v = base + tid + u * kThreads;
          float x[kN];
          V_::unpack(lds128(at + u * kThreads * 16), x);
#pragma unroll
          for (int i = 0; i < kN; ++i)
            if (__any_sync(0xffffffffu, !(x[i] < best.bar_value)))
              best.offer(v < v1 ? order_key(x[i], lead + v * kN + i) : 0, s_wait[warp], p.top_k, lane);
        }
      }
    }
    at = at == ring + (kStages - 1) * kStageBytes ? ring : at + kStageBytes;
    to = to == ring + (kStages - 1) * kStageBytes ? ring : to + kStageBytes;
  }
  if (rank == 0 && warp == 0) {  // fewer than 16 elements besides the vectors
    const int i = lane < lead ? lane : lead + vectors * kN + lane - lead;
    const bool here = lane < loose;
    const float x = here ? to_f32(row[i]) : -INFINITY;
    if (x > sums.m) sums.raise(x);
    peak = max_nan(peak, x);
    sums.add(fmaxf(distance(x, sums.m), kFar));
    if (kTop) best.offer(here ? order_key(x, i) : 0, s_wait[warp], p.top_k, lane);
  }

  // ---- the CTA's warps, then the cluster's CTAs ----
  if (kTop) best.tell(s_bar + warp * kTold, peak, lane);
  sums = warp_join(sums);
  if (lane == 0) s_sums[warp] = sums;
  asm volatile("cp.async.wait_group 0;" ::: "memory");  // nothing is left on its way into the ring
  const int any_bad = __syncthreads_or(!(peak <= FLT_MAX));  // a NaN or +inf
  if (kTop) {
    best.heed(s_bar, p.top_k, lane);
    auto keep = [&](uint64_t key) {
      const unsigned hit = __ballot_sync(0xffffffffu, key > best.bar);
      int at = 0;
      if (lane == 0 && hit) at = atomicAdd(&s_pool_size, __popc(hit));
      at = __shfl_sync(0xffffffffu, at, 0) + __popc(hit & ((1u << lane) - 1));
      if (key > best.bar) s_pool[at] = key;
    };
    // the list's own keys reach the bar that came from it
    best.bar = best.bar ? best.bar - 1 : 0;
    keep(best.mine);
    keep(lane < best.waiting ? s_wait[warp][lane] : 0);
    if (tid < 32) s_best[tid] = 0;
    __syncthreads();
    const int n = s_pool_size;
    for (int i = tid; i < n; i += kThreads) {
      const uint64_t key = s_pool[i];
      int above = 0;
      for (int k = 0; k < n; ++k) above += s_pool[k] > key;
      if (above < 32) s_best[above] = key;
    }
  }
  const Sums nothing = {-INFINITY, 0.f, 0.f};
  if (warp == 0) {
    sums = warp_join(lane < kWarps ? s_sums[lane] : nothing);
    if (lane == 0) {
      s_sums[kWarps] = sums;
      s_bad = any_bad;
    }
  }
  if (ctas > 1) {
    cluster.sync();
  } else {
    __syncthreads();
  }
  if (rank == 0 && (warp == 0 || (kTop && ctas > 1))) {
    Sums all = sums;
    int wrong = any_bad, place = lane;
    uint64_t key = kTop ? s_best[lane] : 0;
    if (ctas > 1) {
      // a warp per CTA's list: a key's place is its own in its list and the number of larger ones in each of the others
      if (kTop) key = warp < ctas ? *cluster.map_shared_rank(&s_best[lane], warp) : 0;
      all = warp_join(lane < ctas ? *cluster.map_shared_rank(&s_sums[kWarps], lane) : nothing);
      wrong = __any_sync(0xffffffffu, lane < ctas && *cluster.map_shared_rank(&s_bad, lane));
      if (kTop) {
        s_pool[tid] = key;
        __syncthreads();
        for (int i = 0; i < ctas; ++i) {
          const uint64_t* list = s_pool + 32 * i;
          int above = 0;
#pragma unroll
          for (int w = 16; w; w >>= 1) above += list[above + w - 1] > key ? w : 0;
          above += list[above] > key;
          place += i == warp ? 0 : above;
        }
      }
    }
    // a row without a distribution: a NaN or +inf in it, or nothing above -inf
    const float log2_s = wrong || all.m == -INFINITY ? NAN : log2f(all.s);
    const float log2_sum = log2_s - distance(all.m, all.m);  // log2 sum e^(x - m)
    // A row that one token has to itself: the reference's rounding is in S and taken away again, which leaves a few
    // 2^-24 of either sign.  ln p <= 0 <= H; a NaN stays one.
    auto ln_p = [&](float x) {
      const float y = __fmaf_rn(log2_sum, -kLn2, x - all.m);
      return y > 0.f ? 0.f : y;
    };
    if (tid == 0) {
      p.logprob[e] = ln_p(x_tok);
      const float h = (log2_s - all.t / all.s) * kLn2;
      if (p.entropy) p.entropy[e] = h < 0.f ? 0.f : h;
    }
    if (kTop && key && place < p.top_k) {
      p.top_ids[e * p.top_k + place] = (int)~(uint32_t)key;
      p.top_logprobs[e * p.top_k + place] = ln_p(key_value(key));
    }
  }
  if (ctas > 1) cluster.sync();  // its shared memory is read until here
}

template <typename T>
int launch_logprobs(const LogprobParams& p, int sm_count, cudaStream_t stream) {
  // A row's CTAs; an entry that turns out to be none counts too, as tokens are known on the device only.
  // A cluster costs most of a microsecond, so it has to save more: 4 or 8 CTAs while no SM gets two, of
  // 6144 logits at least (5 rows of 32,000 bf16 and 5 alternatives: 6.8 us by four, 7.4 in one; of 16,000 both 6.7 and
  // 6.2), 2 with 48 KB each (76 rows of 100 KB: 9.1 against 10.1, of 64 KB 8.1 and 8.0), and on SMs with a CTA already
  // 128 KB each (120 rows of 300 KB: 17.0 against 18.0, of 200 KB 11.7 and 10.7; 152 of 100 KB by four 17 and 10).
  const int64_t rows = (int64_t)p.B * p.C, bytes = (int64_t)p.V * sizeof(T);
  int ctas = 1;
  for (int c = 2; c <= 8 && rows * c <= 2 * sm_count; c *= 2) {
    const int64_t least = rows * c > sm_count ? 131072 : c == 2 ? 49152 : 6144 * (int)sizeof(T);
    if (bytes / c >= least) ctas = c;
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(rows * ctas));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kRing;
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = ctas;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  auto kernel = p.top_k ? logprob_kernel<T, true> : logprob_kernel<T, false>;
  TV_CUDA_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRing));
  TV_CUDA_TRY(cudaLaunchKernelEx(&cfg, kernel, p));
  return TV_OK;
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
  if ((int64_t)B * C >= INT32_MAX / 8)
    return tv::fail(TV_ERR_UNSUPPORTED, "tv_token_logprobs: B * C exceeds 2^31 / 8");
  tv::DeviceInfo dev;
  if (int rc = tv::current_device_info(&dev)) return rc;
  LogprobParams p{static_cast<const char*>(logits), tokens, node, B, N, C, V, logprob, entropy, top_k, top_ids,
                  top_logprobs, status};
  return dtype == TV_BF16 ? launch_logprobs<__nv_bfloat16>(p, dev.sm_count, (cudaStream_t)stream)
                          : launch_logprobs<float>(p, dev.sm_count, (cudaStream_t)stream);
}
