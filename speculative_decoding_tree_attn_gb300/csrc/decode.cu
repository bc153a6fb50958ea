// Attention of one new token per request over the paged cache, split over the
// cache's length and joined.
//
// Output row (b, h) is softmax(s) V over the visible keys of request b, KV head
// h / G, with s_t = cap(scale q.k_t) + slope_h (t - (L - 1)) and visible t:
// t >= L - window or t < n_sink.  "Tree Verification", "Tree Attention": the
// N = 1 case, the token's own K/V already in the cache.
//
// Bound by HBM: a key costs 4 D bytes of bf16 K+V and 4 G D flops, G flop a byte
// (4-16), far below the tensor pipes, so every byte is read once for all G heads
// of its KV head and everything else stays off that path:
// - Work is cut as in the tree kernels: a unit is (request, KV head, up to
//   8 or 16 query heads); the units' tiles lie end to end and each CTA of a
//   persistent grid takes an equal run of them.  A tile is one 16-key group per
//   warp.  Each warp copies its own groups through its own ring in shared memory
//   (cp.async, rows looked up in the block table one step ahead), so nothing in
//   the stream waits for another warp.
// - Groups start at multiples of 16 keys.  Rows that are not visible are not read:
//   the copy fills them with zeros, so a window also skips its work.
// - Online softmax per warp in the log2 domain, sums in float32; the warps' sums
//   meet in shared memory at the end of a unit.  A unit cut by a slice boundary
//   leaves (max, sum, output) of each piece in the workspace; the piece that
//   arrives last joins them in order, so results do not depend on timing.
#include <algorithm>
#include <cmath>

#include <cuda_bf16.h>

#include "common.h"

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kMaxCtas = 4096;
constexpr int64_t kCounterBytes = 4 * kMaxCtas;  // first in the workspace whatever the sizes
constexpr int kKeys = 16;                        // keys of a group
constexpr int kZeros = -1;    // cache row of a key that is not read
constexpr int kNoGroup = -2;  // of a warp without a group in the tile

struct DecodeParams {
  const char* q;
  int64_t q_stride;  // bytes
  const char* k_cache;
  const char* v_cache;
  int64_t num_blocks;
  int block_size;
  const int32_t* table;
  int max_blocks;
  const int32_t* seq_lens;
  int B, Hq, Hkv, G;
  int head_groups;  // units per (request, KV head)
  float scale, softcap;
  int window, n_sink;
  const float* slopes;
  char* out;
  float* lse;
  int32_t* status;
  uint32_t* arrive;  // [kMaxCtas], by a split unit's first CTA
  float* part_o;     // [P][2][heads][D]
  float* part_ml;    // [P][2][heads][2]
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool read) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(read ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Counts an arrival; releases what the CTA wrote before its last barrier and
// acquires what the earlier arrivals released.
__device__ __forceinline__ uint32_t arrive(uint32_t* counter) {
  uint32_t before;
  asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(before) : "l"(counter) : "memory");
  return before;
}

// D[16 x 8] += A[16 x 16] B[16 x 8], bf16 operands, float32 sums.
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// The visible keys of one request, in groups of 16 (absolute multiples).
struct Span {
  int L, first, sink;  // t < sink or first <= t < L
  int lead;            // groups [0, lead) before the group of `first`
  int groups;
};

__device__ __forceinline__ Span span_of(const DecodeParams& p, int b) {
  Span s;
  const int64_t cap = (int64_t)p.max_blocks * p.block_size;
  const int64_t L = __ldg(p.seq_lens + b);
  s.L = (int)max((int64_t)0, min(L, cap));
  s.first = p.window > 0 ? max(0, s.L - p.window) : 0;
  s.sink = min(p.n_sink, s.first);
  s.lead = min((s.sink + kKeys - 1) / kKeys, s.first / kKeys);
  s.groups = s.L > 0 ? s.lead + (s.L - 1) / kKeys + 1 - s.first / kKeys : 0;
  return s;
}
__device__ __forceinline__ int group_key(const Span& s, int i) {
  return (i < s.lead ? i : s.first / kKeys + i - s.lead) * kKeys;
}
__device__ __forceinline__ bool visible(const Span& s, int t) { return t < s.L && (t >= s.first || t < s.sink); }

__device__ __forceinline__ int64_t cta_start(int64_t c, int64_t T, int64_t P) { return c * T / P; }
__device__ __forceinline__ int64_t cta_of(int64_t t, int64_t T, int64_t P) { return ((t + 1) * P - 1) / T; }

// Score of one (head, key) in the log2 domain from its raw product.
struct Scorer {
  float mul, cap2, cap_mul;  // mul: scale log2 e;  cap2: softcap log2 e, 0 without
  __device__ __forceinline__ explicit Scorer(const DecodeParams& p)
      : mul(p.scale * kLog2e), cap2(p.softcap * kLog2e), cap_mul(p.softcap > 0.f ? 2.f * kLog2e * p.scale / p.softcap : 0.f) {}
  __device__ __forceinline__ float operator()(float x) const {
    // tanh y = 1 - 2 / (1 + e^2y): absolute error of a few 2^-24, saturating at both ends
    if (cap2 > 0.f) return cap2 - 2.f * cap2 * __frcp_rn(1.f + exp2_approx(x * cap_mul));
    return x * mul;
  }
};

// Position of 16-byte unit u of a head's row in the merge buffer: spreads the
// heads that a warp writes at once over the banks.
__device__ __forceinline__ int merge_unit(int head, int u) {
  const int t = head >> 1;
  return u ^ ((t & 1) | (t & 2) << 1);
}

// ---------------------------------------------------------------------------
// bf16: both products on the warp-level tensor instructions, keys (S) and output
// dimensions (O) as the 16 rows, heads as the 8 columns, so that 8 heads waste
// nothing.  (tcgen05 tiles have 128 rows: 4 or 8 heads would fill a sixteenth of
// one, and its issue and TMEM traffic buys nothing where HBM is the limit.)
//   S^T[key, head] = K Q^T: a thread's A registers are 16-byte pieces of rows g and
//   g + 8; the order of d within the product is free, so Q's pieces are taken alike.
//   O^T[d, head] += V^T P^T: pieces of rows 2t, 2t+1, 2t+8, 2t+9, paired by byte
//   permutes; P^T is S^T's registers with their 8x8 blocks transposed.
// P is held as two bf16 parts (value and remainder, 16 bits together): the
// products are far from the limit, and one part alone would add 2^-9 a weight.
// ---------------------------------------------------------------------------
template <int D, int NB>
struct Bf16Math {
  using Out = __nv_bfloat16;
  static constexpr int kHeads = 8 * NB;
  static constexpr int kRowBytes = 2 * D;
  static constexpr int kWarpScratch = 0;
  uint4 q[NB][D / 32];
  float o[NB][D / 16][4];
  float m[NB][2], l[NB][2], slope[NB][2];

  // 16-byte piece c of row r within a group's K or V tile.
  static __device__ __forceinline__ int piece(int r, int c) { return r * kRowBytes + ((c ^ (r & 7)) << 4); }

  __device__ __forceinline__ void begin(const DecodeParams& p, const char* qrow, int h0, int nh, int lane) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      const int h = 8 * n + g;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const int c = 2 * t + (i & 1) + 8 * (i >> 1);
        q[n][i] = h < nh ? __ldg(reinterpret_cast<const uint4*>(qrow + h * kRowBytes + 16 * c)) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int j = 0; j < D / 16; ++j) o[n][j][0] = o[n][j][1] = o[n][j][2] = o[n][j][3] = 0.f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int hc = 8 * n + 2 * t + e;
        m[n][e] = -INFINITY;
        l[n][e] = 0.f;
        slope[n][e] = p.slopes && hc < nh ? __ldg(p.slopes + h0 + hc) * kLog2e : 0.f;
      }
    }
  }

  __device__ __forceinline__ void group(const DecodeParams& p, const Scorer& score, const Span& sp, int key, uint32_t kt,
                                        uint32_t vt, int lane, float*) {
    const int g = lane >> 2, t = lane & 3;
    float s[NB][4];
#pragma unroll
    for (int n = 0; n < NB; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const int c = 2 * t + (i & 1) + 8 * (i >> 1);
      const uint4 a = lds128(kt + piece(g, c)), b = lds128(kt + piece(g + 8, c));
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        mma(s[n], a.x, b.x, a.y, b.y, q[n][i].x, q[n][i].y);
        mma(s[n], a.z, b.z, a.w, b.w, q[n][i].z, q[n][i].w);
      }
    }
    const bool edge = key + kKeys > sp.L || key < sp.first;
    const bool see0 = visible(sp, key + g), see1 = visible(sp, key + g + 8);
    bool grow = false;
    float mx[NB][2];
#pragma unroll
    for (int n = 0; n < NB; ++n) {
#pragma unroll
      for (int e = 0; e < 4; ++e) s[n][e] = score(s[n][e]);
      if (p.slopes) {
        const float d0 = (float)(key + g - (sp.L - 1)), d1 = (float)(key + g + 8 - (sp.L - 1));
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          s[n][e] = fmaf(slope[n][e], d0, s[n][e]);
          s[n][2 + e] = fmaf(slope[n][e], d1, s[n][2 + e]);
        }
      }
      if (edge) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          if (!see0) s[n][e] = -INFINITY;
          if (!see1) s[n][2 + e] = -INFINITY;
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float v = fmaxf(s[n][e], s[n][2 + e]);
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
        mx[n][e] = v;
        // sums are taken against a maximum up to 2^8 too small before they are scaled again
        grow |= v > m[n][e] + 8.f;
      }
    }
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        float c[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float m2 = fmaxf(m[n][e], mx[n][e]);
          c[e] = m[n][e] == -INFINITY ? 0.f : exp2_approx(m[n][e] - m2);
          m[n][e] = m2;
          l[n][e] *= c[e];
        }
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
          o[n][j][0] *= c[0];
          o[n][j][1] *= c[1];
          o[n][j][2] *= c[0];
          o[n][j][3] *= c[1];
        }
      }
    }
    uint32_t hi[NB][2], lo[NB][2];
#pragma unroll
    for (int n = 0; n < NB; ++n) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float w0 = exp2_approx(s[n][2 * r] - m[n][0]), w1 = exp2_approx(s[n][2 * r + 1] - m[n][1]);
        l[n][0] += w0;
        l[n][1] += w1;
        const __nv_bfloat162 h = __floats2bfloat162_rn(w0, w1);
        const float2 f = __bfloat1622float2(h);
        const __nv_bfloat162 k = __floats2bfloat162_rn(w0 - f.x, w1 - f.y);
        hi[n][r] = transpose8x8(*reinterpret_cast<const uint32_t*>(&h));
        lo[n][r] = transpose8x8(*reinterpret_cast<const uint32_t*>(&k));
      }
    }
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
      const uint4 x0 = lds128(vt + piece(2 * t, g + 8 * i)), x1 = lds128(vt + piece(2 * t + 1, g + 8 * i));
      const uint4 y0 = lds128(vt + piece(2 * t + 8, g + 8 * i)), y1 = lds128(vt + piece(2 * t + 9, g + 8 * i));
      const uint32_t xa[4] = {x0.x, x0.y, x0.z, x0.w}, xb[4] = {x1.x, x1.y, x1.z, x1.w};
      const uint32_t ya[4] = {y0.x, y0.y, y0.z, y0.w}, yb[4] = {y1.x, y1.y, y1.z, y1.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t a0 = __byte_perm(xa[j], xb[j], 0x5410), a1 = __byte_perm(xa[j], xb[j], 0x7632);
        const uint32_t a2 = __byte_perm(ya[j], yb[j], 0x5410), a3 = __byte_perm(ya[j], yb[j], 0x7632);
#pragma unroll
        for (int n = 0; n < NB; ++n) {
          mma(o[n][4 * i + j], a0, a1, a2, a3, hi[n][0], hi[n][1]);
          mma(o[n][4 * i + j], a0, a1, a2, a3, lo[n][0], lo[n][1]);
        }
      }
    }
  }

  // This warp's maxima, sums and outputs of heads 8n .. 8n + 7.
  __device__ __forceinline__ void flush(int n, float* o_out, float* ml, int lane) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int k = 0; k < NB; ++k) {
      if (k != n) continue;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float v = l[k][e];
        v += __shfl_xor_sync(0xffffffffu, v, 4);
        v += __shfl_xor_sync(0xffffffffu, v, 8);
        v += __shfl_xor_sync(0xffffffffu, v, 16);
        const int h = 2 * t + e;
        if (g == 0) {
          ml[2 * h] = m[k][e];
          ml[2 * h + 1] = v;
        }
#pragma unroll
        for (int i = 0; i < D / 64; ++i)
#pragma unroll
          for (int u = 0; u < 2; ++u)
            *reinterpret_cast<float4*>(o_out + h * D + 4 * merge_unit(h, 2 * (g + 8 * i) + u)) =
                make_float4(o[k][4 * i + 2 * u][e], o[k][4 * i + 2 * u][2 + e], o[k][4 * i + 2 * u + 1][e],
                            o[k][4 * i + 2 * u + 1][2 + e]);
      }
    }
  }
};

// ---------------------------------------------------------------------------
// float32: FMAs.  A lane keeps D / 32 dimensions of Q and O for NH heads (the
// least power of two that holds the KV head's, 8 at most).  The partial products
// of 32 (key, head) pairs are summed over the lanes by 31 exchanges that leave
// each lane one pair, and the weights come back through shared memory as
// broadcasts.
// ---------------------------------------------------------------------------
template <int D, int NH>
struct F32Math {
  using Out = float;
  static constexpr int kHeads = NH;
  static constexpr int kRowBytes = 4 * D;
  static constexpr int kWarpScratch = kKeys * NH * 4;  // the group's weights [key][head]
  static constexpr int kE = D / 32;
  static constexpr int kVec = kE < 4 ? kE : 4;                      // consecutive dimensions of a lane
  static constexpr int kPairs = kKeys * NH < 32 ? kKeys * NH : 32;  // (key, head) pairs summed at once
  static constexpr int kAtOnce = kPairs / NH;                       // keys
  static constexpr int kSets = kKeys / kAtOnce;
  float q[NH][kE], o[NH][kE];
  float m, l, slope;  // of head lane % NH

  static __device__ __forceinline__ int piece(int r, int c) { return r * kRowBytes + (c << 4); }
  static __device__ __forceinline__ int dim(int lane, int e) { return lane * kVec + (e / kVec) * 32 * kVec + e % kVec; }
  static __device__ __forceinline__ void lane_row(float (&x)[kE], uint32_t row, int lane) {
#pragma unroll
    for (int e = 0; e < kE; e += kVec) {
      if constexpr (kVec == 4)
        asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(x[e]), "=f"(x[e + 1]), "=f"(x[e + 2]), "=f"(x[e + 3])
                     : "r"(row + 4 * dim(lane, e)));
      else
        asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(x[e]), "=f"(x[e + 1]) : "r"(row + 4 * dim(lane, e)));
    }
  }

  __device__ __forceinline__ void begin(const DecodeParams& p, const char* qrow, int h0, int nh, int lane) {
#pragma unroll
    for (int h = 0; h < NH; ++h)
#pragma unroll
      for (int e = 0; e < kE; ++e) {
        q[h][e] = h < nh ? __ldg(reinterpret_cast<const float*>(qrow + h * kRowBytes) + dim(lane, e)) : 0.f;
        o[h][e] = 0.f;
      }
    m = -INFINITY;
    l = 0.f;
    slope = p.slopes && lane % NH < nh ? __ldg(p.slopes + h0 + lane % NH) * kLog2e : 0.f;
  }

  __device__ __forceinline__ void group(const DecodeParams& p, const Scorer& score, const Span& sp, int key, uint32_t kt,
                                        uint32_t vt, int lane, float* weights) {
    float s[kSets];
    float mx = -INFINITY;
#pragma unroll
    for (int i = 0; i < kSets; ++i) {
      float v[kPairs];
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        float x[kE];
        lane_row(x, kt + (kAtOnce * i + k) * kRowBytes, lane);
#pragma unroll
        for (int h = 0; h < NH; ++h) {
          float a = q[h][0] * x[0];
#pragma unroll
          for (int e = 1; e < kE; ++e) a = fmaf(q[h][e], x[e], a);
          v[NH * k + h] = a;
        }
      }
#pragma unroll
      for (int w = kPairs / 2; w; w >>= 1) {
        const bool up = lane & w;
#pragma unroll
        for (int j = 0; j < w; ++j) {
          const float keep = up ? v[j + w] : v[j], give = up ? v[j] : v[j + w];
          v[j] = keep + __shfl_xor_sync(0xffffffffu, give, w);
        }
      }
      if constexpr (kPairs == 16) v[0] += __shfl_xor_sync(0xffffffffu, v[0], 16);
      const int t = key + kAtOnce * i + lane % kPairs / NH;
      s[i] = fmaf(slope, (float)(t - (sp.L - 1)), score(v[0]));
      if (!visible(sp, t)) s[i] = -INFINITY;
      mx = fmaxf(mx, s[i]);
    }
#pragma unroll
    for (int w = NH; w < kPairs; w <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
    if (__any_sync(0xffffffffu, mx > m + 8.f)) {
      const float m2 = fmaxf(m, mx);
      const float c = m == -INFINITY ? 0.f : exp2_approx(m - m2);
      m = m2;
      l *= c;
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        const float ch = __shfl_sync(0xffffffffu, c, h);
#pragma unroll
        for (int e = 0; e < kE; ++e) o[h][e] *= ch;
      }
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kSets; ++i) {
      const float w = exp2_approx(s[i] - m);
      l += w;
      if (kPairs == 32 || lane < kPairs) weights[kPairs * i + lane] = w;
    }
    __syncwarp();
#pragma unroll 4
    for (int k = 0; k < kKeys; ++k) {
      float x[kE], w[NH];
      lane_row(x, vt + k * kRowBytes, lane);
#pragma unroll
      for (int h = 0; h < NH; ++h) w[h] = weights[NH * k + h];
#pragma unroll
      for (int h = 0; h < NH; ++h)
#pragma unroll
        for (int e = 0; e < kE; ++e) o[h][e] = fmaf(w[h], x[e], o[h][e]);
    }
  }

  __device__ __forceinline__ void flush(int, float* o_out, float* ml, int lane) {
    float v = l;
#pragma unroll
    for (int w = NH; w < kPairs; w <<= 1) v += __shfl_xor_sync(0xffffffffu, v, w);
    if (lane < NH) {
      ml[2 * lane] = m;
      ml[2 * lane + 1] = v;
    }
#pragma unroll
    for (int h = 0; h < NH; ++h)
#pragma unroll
      for (int e = 0; e < kE; ++e) {
        const int d = dim(lane, e);
        o_out[h * D + 4 * merge_unit(h, d >> 2) + (d & 3)] = o[h][e];
      }
  }
};

__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v) {
  __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<uint32_t*>(&a), *reinterpret_cast<uint32_t*>(&b));
}

// Shared memory of a CTA: the rings (192 KB: three groups a warp at 8 KB each, so
// that two are in flight while one is computed), the merge buffer, its weights.
template <class Math, int D>
struct Shape {
  static constexpr int kTile = kKeys * Math::kRowBytes;  // K or V of a group
  static constexpr int kStage = 2 * kTile;
  static constexpr int kWarps = kStage <= 8192 ? 8 : 65536 / kStage;
  static constexpr int kStages = 196608 / (kWarps * kStage);
  static constexpr int kRing = kWarps * kStages * kStage;
  static constexpr int kMerge = kWarps * 8 * D * 4;
  static constexpr int kSmem = kRing + kMerge + kWarps * (8 * 2 * 4 + Math::kWarpScratch);
  static_assert(kSmem <= 227 * 1024 - 256, "shared memory of a CTA");
};

template <class Math, int D>
__global__ void __launch_bounds__(Shape<Math, D>::kWarps * 32, 1) decode_kernel(const DecodeParams p) {
  using S = Shape<Math, D>;
  constexpr int kWarps = S::kWarps, kStages = S::kStages, kThreads = kWarps * 32, kHeads = Math::kHeads;
  constexpr int kPieces = Math::kRowBytes / 16;            // 16-byte pieces of a row
  constexpr int kCopies = kKeys * kPieces / 32;            // copies of a lane for a K or V tile
  extern __shared__ __align__(128) char smem[];
  __shared__ int64_t s_scan[kWarps];
  __shared__ int64_t s_total, s_base;
  __shared__ int s_b;
  __shared__ bool s_last;
  struct Piece {  // this CTA's piece of a cut unit
    int64_t c0;   // the unit's first CTA
    int others;   // its other pieces; -1: no such unit
    int heads;
    int64_t out_row;
  };
  __shared__ Piece s_piece[2];  // of the unit that the slice's start cuts, of the one that its end cuts
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem) + warp * kStages * S::kStage;
  float* merge = reinterpret_cast<float*>(smem + S::kRing);
  float* merge_ml = reinterpret_cast<float*>(smem + S::kRing + S::kMerge);  // [warp][8][2]
  float* scratch = merge_ml + kWarps * 16 + warp * (Math::kWarpScratch / 4);
  const int per_request = p.Hkv * p.head_groups;

  // ---- this CTA's slice of the tiles ----
  auto tiles_of = [&](int b) { return max(1, (span_of(p, b).groups + kWarps - 1) / kWarps); };
  int64_t sum = 0;
  for (int b = tid; b < p.B; b += kThreads) sum += tiles_of(b);
  for (int w = 16; w; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
  if (lane == 0) s_scan[warp] = sum;
  __syncthreads();
  if (tid == 0) {
    int64_t all = 0;
    for (int w = 0; w < kWarps; ++w) all += s_scan[w];
    s_total = all * per_request;
    s_base = 0;
    s_b = -1;
    s_piece[0].others = s_piece[1].others = -1;
  }
  __syncthreads();
  const int64_t T = s_total;
  const int64_t P = min((int64_t)gridDim.x, T);
  if (blockIdx.x >= P) return;
  const int64_t t0 = cta_start(blockIdx.x, T, P), t1 = cta_start(blockIdx.x + 1, T, P);
  for (int base = 0; base < p.B; base += kThreads) {  // request of tile t0
    const int b = base + tid;
    const int64_t n = b < p.B ? (int64_t)tiles_of(b) * per_request : 0;
    int64_t incl = n;
    for (int w = 1; w < 32; w <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, incl, w);
      if (lane >= w) incl += v;
    }
    if (lane == 31) s_scan[warp] = incl;
    __syncthreads();
    int64_t start = s_base + incl - n;
    int64_t all = s_base;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) start += s_scan[w];
      all += s_scan[w];
    }
    __syncthreads();
    if (start <= t0 && t0 < start + n) {
      s_b = b;
      s_base = start;
    } else if (tid == 0 && all <= t0) {
      s_base = all;
    }
    __syncthreads();
    if (s_b >= 0) break;
  }

  struct Place {  // a tile: request, unit in it, tile in the unit
    int b, unit, tile, tiles;
    Span span;
  };
  Place at;
  at.b = s_b;
  at.span = span_of(p, at.b);
  at.tiles = max(1, (at.span.groups + kWarps - 1) / kWarps);
  at.unit = (int)((t0 - s_base) / at.tiles);
  at.tile = (int)((t0 - s_base) % at.tiles);
  auto next_unit = [&](Place& x) {
    x.tile = 0;
    if (++x.unit == per_request) {
      x.unit = 0;
      if (++x.b < p.B) {
        x.span = span_of(p, x.b);
        x.tiles = max(1, (x.span.groups + kWarps - 1) / kWarps);
      }
    }
  };

  // ---- copies, kStages - 1 groups ahead, block table entries one more ----
  Place ahead = at;
  int64_t ahead_left = t1 - t0;
  // cache row of key lane % 16 of the next group
  auto look_up = [&]() -> int64_t {
    int64_t row = kNoGroup;
    if (ahead_left > 0) {
      const int i = ahead.tile * kWarps + warp;
      if (i < ahead.span.groups) {
        const int t = group_key(ahead.span, i) + lane % kKeys;
        row = kZeros;
        if (visible(ahead.span, t)) {
          const int c = t / p.block_size;
          const int64_t blk = __ldg(p.table + (int64_t)ahead.b * p.max_blocks + c);
          if (blk >= 0 && blk < p.num_blocks)
            row = (blk * p.Hkv + ahead.unit / p.head_groups) * p.block_size + (t - c * p.block_size);
          else if (p.status)
            atomicOr(p.status, TV_DEV_BAD_BLOCK);
        }
      }
      --ahead_left;
      if (++ahead.tile == ahead.tiles) next_unit(ahead);
    }
    return row;
  };
  auto copy = [&](int64_t row, int stage) {
    const uint32_t dst = ring + stage * S::kStage;
    if (row != kNoGroup) {  // the same for the whole warp
#pragma unroll
      for (int i = 0; i < kCopies; ++i) {
        const int x = i * 32 + lane;
        const int r = x / kPieces, c = x % kPieces;
        const int64_t from = __shfl_sync(0xffffffffu, row, r);
        const int64_t off = (from < 0 ? 0 : from) * Math::kRowBytes + 16 * c;
        cp_async16(dst + Math::piece(r, c), p.k_cache + off, from >= 0);
        cp_async16(dst + S::kTile + Math::piece(r, c), p.v_cache + off, from >= 0);
      }
    }
    cp_async_commit();
  };
  int64_t row = look_up();
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) {
    const int64_t now = row;
    row = look_up();
    copy(now, s);
  }

  // ---- units ----
  const Scorer score(p);
  int stage = 0;
  Math math;
  uint32_t before_lead = 0, before_tail = 0;  // pieces that arrived before this CTA's (thread 0; not waited for until the end)
  for (int64_t t = t0; t < t1;) {
    const int kvh = at.unit / p.head_groups, hg = at.unit % p.head_groups;
    const int h0 = kvh * p.G + hg * kHeads;                    // first query head
    const int nh = min(kHeads, p.G - hg * kHeads);
    const int tile1 = (int)min((int64_t)at.tiles, at.tile + (t1 - t));
    math.begin(p, p.q + at.b * p.q_stride + (int64_t)h0 * Math::kRowBytes, h0, nh, lane);
    if (t + tile1 - at.tile < t1) {  // the next unit's queries, into this SM's cache
      const bool same = at.unit + 1 < per_request;
      const int unit = same ? at.unit + 1 : 0;
      const int hq = unit / p.head_groups * p.G + unit % p.head_groups * kHeads;
      const int n = min(kHeads, p.G - unit % p.head_groups * kHeads) * (Math::kRowBytes / 128);
      if (tid < n)
        asm volatile("{.reg .b32 x; ld.global.ca.b32 x, [%0];}" ::"l"(
            p.q + (same ? at.b : at.b + 1) * p.q_stride + (int64_t)hq * Math::kRowBytes + tid * 128));
    }
    for (int tile = at.tile; tile < tile1; ++tile) {
      cp_async_wait<kStages - 2>();
      __syncwarp();
      const int64_t now = row;
      row = look_up();
      copy(now, stage == 0 ? kStages - 1 : stage - 1);
      const int i = tile * kWarps + warp;
      if (i < at.span.groups)
        math.group(p, score, at.span, group_key(at.span, i), ring + stage * S::kStage,
                   ring + stage * S::kStage + S::kTile, lane, scratch);
      stage = stage == kStages - 1 ? 0 : stage + 1;
    }

    const int64_t u0 = t - at.tile;  // the unit's first tile
    const bool whole = at.tile == 0 && tile1 == at.tiles;
    const int64_t slot = 2 * (int64_t)blockIdx.x + (at.tile == 0 ? 1 : 0);
    const int64_t out_row = (int64_t)at.b * p.Hq + h0;
    typename Math::Out* out = reinterpret_cast<typename Math::Out*>(p.out) + out_row * D;
#pragma unroll
    for (int n = 0; n < (kHeads + 7) / 8; ++n) {
      const int heads = min(8, nh - 8 * n);
      if (heads <= 0) break;
      __syncthreads();  // the buffer's last readers
      math.flush(n, merge + warp * 8 * D, merge_ml + warp * 16, lane);
      __syncthreads();
      for (int x = tid; x < heads * (D / 4); x += kThreads) {
        const int h = x / (D / 4), u = x % (D / 4);
        float mm = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, merge_ml[w * 16 + 2 * h]);
        float ll = 0.f;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float mw = merge_ml[w * 16 + 2 * h];
          const float c = mw == -INFINITY ? 0.f : exp2_approx(mw - mm);
          const float4 o = *reinterpret_cast<const float4*>(merge + (w * 8 + h) * D + 4 * merge_unit(h, u));
          ll = fmaf(merge_ml[w * 16 + 2 * h + 1], c, ll);
          v.x = fmaf(o.x, c, v.x);
          v.y = fmaf(o.y, c, v.y);
          v.z = fmaf(o.z, c, v.z);
          v.w = fmaf(o.w, c, v.w);
        }
        const int hh = 8 * n + h;
        if (whole) {
          const float r = at.span.groups ? 1.f / ll : 0.f;
          store4(out + hh * D + 4 * u, make_float4(v.x * r, v.y * r, v.z * r, v.w * r));
          if (p.lse && u == 0) p.lse[out_row + hh] = at.span.groups ? (mm + log2f(ll)) * kLn2 : -INFINITY;
        } else {
          __stcg(reinterpret_cast<float4*>(p.part_o + (slot * kHeads + hh) * D + 4 * u), v);
          if (u == 0) __stcg(reinterpret_cast<float2*>(p.part_ml + (slot * kHeads + hh) * 2), make_float2(mm, ll));
        }
      }
    }
    if (!whole) {
      const int64_t c0 = cta_of(u0, T, P), c1 = cta_of(u0 + at.tiles - 1, T, P);
      __syncthreads();  // the piece is written; thread 0's release covers it
      if (tid == 0) {
        const int k = at.tile == 0 ? 1 : 0;
        s_piece[k] = {c0, (int)(c1 - c0), nh, out_row};
        const uint32_t n = arrive(p.arrive + c0);
        if (k) before_tail = n; else before_lead = n;
      }
    }
    t += tile1 - at.tile;
    at.tile = tile1;
    if (at.tile == at.tiles) next_unit(at);
  }
  cp_async_wait<0>();

  // ---- joins ----
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const Piece mine = s_piece[k];
    if (mine.others < 0) continue;
    if (tid == 0) {
      s_last = (k ? before_tail : before_lead) == (uint32_t)mine.others;
      if (s_last) p.arrive[mine.c0] = 0;  // every piece is here
    }
    __syncthreads();
    if (s_last) {
      __threadfence();
      typename Math::Out* out = reinterpret_cast<typename Math::Out*>(p.out) + mine.out_row * D;
      for (int x = tid; x < mine.heads * (D / 4); x += kThreads) {
        const int h = x / (D / 4), u = x % (D / 4);
        // slot 1 of the unit's first CTA, slot 0 of the others
        auto slot = [&](int i) { return ((2 * (mine.c0 + i) + (i == 0)) * kHeads + h); };
        float mm = -INFINITY;
#pragma unroll 8
        for (int i = 0; i <= mine.others; ++i) mm = fmaxf(mm, __ldcg(p.part_ml + slot(i) * 2));
        float ll = 0.f;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
        for (int i = 0; i <= mine.others; ++i) {
          const float2 a = __ldcg(reinterpret_cast<const float2*>(p.part_ml + slot(i) * 2));
          const float4 o = __ldcg(reinterpret_cast<const float4*>(p.part_o + slot(i) * D + 4 * u));
          const float w = a.x == -INFINITY ? 0.f : exp2_approx(a.x - mm);
          ll = fmaf(a.y, w, ll);
          v.x = fmaf(o.x, w, v.x);
          v.y = fmaf(o.y, w, v.y);
          v.z = fmaf(o.z, w, v.z);
          v.w = fmaf(o.w, w, v.w);
        }
        const float r = 1.f / ll;
        store4(out + h * D + 4 * u, make_float4(v.x * r, v.y * r, v.z * r, v.w * r));
        if (p.lse && u == 0) p.lse[mine.out_row + h] = (mm + log2f(ll)) * kLn2;
      }
    }
    __syncthreads();
  }
}

template <class Math, int D>
int launch_decode(DecodeParams p, int ctas, cudaStream_t s) {
  constexpr int smem = Shape<Math, D>::kSmem;
  p.head_groups = (p.G + Math::kHeads - 1) / Math::kHeads;
  TV_CUDA_TRY(cudaFuncSetAttribute(decode_kernel<Math, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
  decode_kernel<Math, D><<<ctas, Shape<Math, D>::kWarps * 32, smem, s>>>(p);
  TV_LAUNCH_CHECK("decode_kernel");
  return TV_OK;
}

// Query heads of a unit.  bf16: 8, or 16 where a KV head serves more than 8 (two
// 8-column products share a key's loads), except where their sums would not fit in
// registers.  float32: as many as the KV head serves, 8 at most.
int unit_heads(int G, int D, int dtype) {
  if (dtype == TV_BF16) return G > 8 && D <= 128 ? 16 : 8;
  return G == 1 ? 1 : G == 2 ? 2 : G <= 4 ? 4 : 8;
}

template <int D>
int dispatch_heads(const DecodeParams& p, int dtype, int ctas, cudaStream_t s) {
  const int heads = unit_heads(p.G, D, dtype);
  if (dtype == TV_BF16) {
    if constexpr (D <= 128)
      if (heads == 16) return launch_decode<Bf16Math<D, 2>, D>(p, ctas, s);
    return launch_decode<Bf16Math<D, 1>, D>(p, ctas, s);
  }
  switch (heads) {
    case 1: return launch_decode<F32Math<D, 1>, D>(p, ctas, s);
    case 2: return launch_decode<F32Math<D, 2>, D>(p, ctas, s);
    case 4: return launch_decode<F32Math<D, 4>, D>(p, ctas, s);
    default: return launch_decode<F32Math<D, 8>, D>(p, ctas, s);
  }
}

int dispatch_decode(const DecodeParams& p, int D, int dtype, int ctas, cudaStream_t s) {
  if (D == 64) return dispatch_heads<64>(p, dtype, ctas, s);
  if (D == 128) return dispatch_heads<128>(p, dtype, ctas, s);
  return dispatch_heads<256>(p, dtype, ctas, s);
}

// One CTA per SM unless the caller asks for another grid.
int grid_of(int num_ctas, int* ctas) {
  if (num_ctas > 0) {
    *ctas = num_ctas;
    return TV_OK;
  }
  tv::DeviceInfo dev;
  if (int rc = tv::current_device_info(&dev)) return rc;
  *ctas = std::min(dev.sm_count, kMaxCtas);
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
  int ctas = 0;
  if (int rc = grid_of(num_ctas, &ctas)) return rc;
  const int heads = unit_heads(Hq / Hkv, head_dim, dtype);
  *bytes = (size_t)kCounterBytes + (size_t)ctas * 2 * heads * (head_dim + 2) * 4;
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
  int ctas = 0;
  if (int rc = grid_of(num_ctas, &ctas)) return rc;
  cudaStream_t st = (cudaStream_t)stream;
  if (!(flags & TV_ATTN_WORKSPACE_ZEROED)) TV_CUDA_TRY(cudaMemsetAsync(workspace, 0, kCounterBytes, st));
  DecodeParams p{};
  p.q = static_cast<const char*>(q);
  p.q_stride = q_stride * e;
  p.k_cache = static_cast<const char*>(k_cache);
  p.v_cache = static_cast<const char*>(v_cache);
  p.num_blocks = num_blocks;
  p.block_size = block_size;
  p.table = block_table;
  p.max_blocks = max_blocks;
  p.seq_lens = seq_lens;
  p.B = B;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.G = Hq / Hkv;
  p.scale = scale;
  p.softcap = softcap;
  p.window = window;
  p.n_sink = n_sink;
  p.slopes = slopes;
  p.out = static_cast<char*>(out);
  p.lse = lse;
  p.status = status;
  p.arrive = static_cast<uint32_t*>(workspace);
  p.part_o = reinterpret_cast<float*>(static_cast<char*>(workspace) + kCounterBytes);
  p.part_ml = p.part_o + (size_t)ctas * 2 * unit_heads(p.G, head_dim, dtype) * head_dim;
  return dispatch_decode(p, head_dim, dtype, ctas, st);
}
