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
// - A unit is (request, KV head, up to 8 or 16 query heads).  A CTA's warps take a
//   team of units at a time, all KV heads of a request where there are 8: they
//   then read whole cache blocks together (one KV head's part of a 16-token block
//   is 4 KB) and meet only at a cut.  64 requests of 1k-8k tokens, 32/8 heads of 128:
//   189 us (0.95 of the measured copy rate), with the warps on one unit's keys 203.
//   Where the lengths leave too few tiles, or too many pieces, several warps share a
//   unit's keys (16 x 32k, 64/8 heads: 320 us, 0.99; as whole teams 334).
// - Teams' tiles (a group of keys per warp) lie end to end and each CTA of a
//   persistent grid takes an equal run of them.  SMs do not get equal shares of the
//   memory: the first CTA is done at 0.87 of the last one's time.  Small runs at the
//   end, taken by whichever CTA is done, gained 4 % in the stream alone and lost it
//   to the pieces that they cut the last requests into.
// - Each warp copies its own groups through its own ring in shared memory
//   (cp.async, rows looked up in the block table one step ahead), so nothing in
//   the stream waits for another warp.
// - Groups start at multiples of their size.  Rows that are not visible are not
//   read: the copy fills them with zeros, so a window also skips its work.
// - Online softmax per warp in the log2 domain, sums in float32; warps that share
//   a unit meet in shared memory at its end.  A team cut by a CTA's boundary
//   leaves (max, sum, output) of each piece in the workspace; the CTA whose piece
//   arrives last joins them in order, so results do not depend on timing (many
//   pieces in two steps).
#include <algorithm>
#include <cfloat>
#include <cmath>
#include <type_traits>

#include <cuda_bf16.h>

#include "attn_score.cuh"
#include "common.h"

namespace {

constexpr int kMaxCtas = 4096;
constexpr int64_t kCounterBytes = 4 * kMaxCtas;  // arrival counters by a cut team's first CTA: first in the workspace
constexpr int kOneStep = 24;  // pieces that are joined at once
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
  int team_log;     // largest team, log2: a power of two that divides a request's units and the warps
  int rows;         // query heads that a unit holds at most
  uint32_t div_mul, div_shift;  // t / block_size = t * div_mul >> div_shift
  float scale, softcap;
  int window, n_sink;
  const float* slopes;
  char* out;
  float* lse;
  int32_t* status;
  uint32_t* arrive;  // [kMaxCtas]
  float* part_o;     // [CTAs][2][team][rows][D]
  float* part_ml;    // [CTAs][2][team][rows][2]
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
// A sum against m as one against top.
__device__ __forceinline__ float scaled(float x, float m, float top) { return x * exp2_approx(m - top); }

// Counts an arrival; releases what the CTA wrote before its last barrier and
// acquires what the earlier arrivals released.
__device__ __forceinline__ uint32_t arrive(uint32_t* counter, uint32_t one) {
  uint32_t before;
  asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], %2;" : "=r"(before) : "l"(counter), "r"(one) : "memory");
  return before;
}

// Joins of n pieces: more than 24 in runs, each joined into its first piece by its last arrival, and then the runs, as
// one CTA reads all of them slowly (one request of 16,000 tokens, 16/1 heads of 128, 152 pieces: 19 us, 37 in one
// step; 8/1 heads of 256: 27 and 83).  A run counts in the lower half of the counter of its first CTA, which no other
// team starts in; the runs of a team in the upper half of the team's.
struct Runs {
  int size, count;
  __device__ __forceinline__ explicit Runs(int n) : size(n), count(1) {
    if (n > kOneStep) {
      size = 5 << (n > 64) + (n > 512);  // about the root of n
      count = n / size;
    }
  }
  __device__ __forceinline__ int of(int i) const { return count == 1 ? 0 : min(i / size, count - 1); }
  __device__ __forceinline__ int pieces(int run, int n) const { return run == count - 1 ? n - run * size : size; }
};

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

// The visible keys of one request, in groups of kKeys (absolute multiples).
struct Span {
  int L, first, sink;  // t < sink or first <= t < L
  int lead;            // groups [0, lead) before the group of `first`
  int groups;
};

template <int kKeys>
__device__ __forceinline__ Span span_of(const DecodeParams& p, int b) {
  Span s;
  const int64_t cap = min((int64_t)p.max_blocks * p.block_size, (int64_t)INT32_MAX - 63);  // a group's end is an int
  const int64_t L = __ldg(p.seq_lens + b);
  s.L = (int)max((int64_t)0, min(L, cap));
  s.first = p.window > 0 ? max(0, s.L - p.window) : 0;
  s.sink = min(p.n_sink, s.first);
  s.lead = min((int)(((uint32_t)s.sink + kKeys - 1) / kKeys), s.first / kKeys);
  s.groups = s.L > 0 ? s.lead + (s.L - 1) / kKeys + 1 - s.first / kKeys : 0;
  return s;
}
template <int kKeys>
__device__ __forceinline__ int group_key(const Span& s, int i) {
  return (i < s.lead ? i : s.first / kKeys + i - s.lead) * kKeys;
}
__device__ __forceinline__ bool visible(const Span& s, int t) { return t < s.L && (t >= s.first || t < s.sink); }

// CTA c of P takes tiles [cta_start(c), cta_start(c + 1)) of T.
__device__ __forceinline__ int cta_start(int c, int T, int P) {  // c T / P in 32 bits, P <= 4096
  return c * (T / P) + (int)((uint32_t)(c * (T % P)) / (uint32_t)P);
}
__device__ __forceinline__ int cta_of(int t, int T, int P) { return (int)((((int64_t)t + 1) * P - 1) / T); }

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
// The sum takes the weight as it was, 2^-17 of it away at most, which is lost in
// the outputs' own rounding (2^-9).
// ---------------------------------------------------------------------------
template <int D, int NB>
struct Bf16Math {
  using Out = __nv_bfloat16;
  static constexpr int kHeads = 8 * NB;
  static constexpr int kFlush = 8;  // heads merged at once
  static constexpr int kKeys = 16;
  static constexpr int kRowBytes = 2 * D;
  static constexpr int kWarpScratch = 0;
  // Q of 16 heads of 256 does not fit beside their sums in registers: each lane's part is in its warp's place of the
  // merge buffer, which holds no sums while keys are read.
  static constexpr bool kQShared = D == 256 && NB == 2;
  static constexpr int kQ = D / 32;
  uint4 q[kQShared ? 1 : NB][kQShared ? 1 : kQ];
  uint32_t q_at;
  float o[NB][D / 16][4];
  float m[NB][2], l[NB][2], slope[NB][2];

  // 16-byte piece c of row r within a group's K or V tile.
  static __device__ __forceinline__ int piece(int r, int c) { return r * kRowBytes + ((c ^ (r & 7)) << 4); }

  __device__ __forceinline__ uint4 query(int n, int i) const {
    if constexpr (kQShared) return lds128(q_at + 512 * (n * kQ + i));
    else return q[n][i];
  }
  __device__ __forceinline__ void begin(const DecodeParams& p, const char* qrow, int h0, int nh, int lane, uint32_t room) {
    const int g = lane >> 2, t = lane & 3;
    q_at = room + 16 * lane;
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      const int h = 8 * n + g;
#pragma unroll
      for (int i = 0; i < kQ; ++i) {
        const int c = 2 * t + (i & 1) + 8 * (i >> 1);
        const uint4 x = h < nh ? __ldg(reinterpret_cast<const uint4*>(qrow + h * kRowBytes + 16 * c)) : make_uint4(0, 0, 0, 0);
        if constexpr (kQShared)
          asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(q_at + 512 * (n * kQ + i)), "r"(x.x), "r"(x.y),
                       "r"(x.z), "r"(x.w)
                       : "memory");
        else
          q[n][i] = x;
      }
#pragma unroll
      for (int j = 0; j < D / 16; ++j) o[n][j][0] = o[n][j][1] = o[n][j][2] = o[n][j][3] = 0.f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int hc = 8 * n + 2 * t + e;
        m[n][e] = kNoScore;
        l[n][e] = 0.f;
        slope[n][e] = p.slopes && hc < nh ? slope_of(p.slopes, h0 + hc) : 0.f;
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
        const uint4 x = query(n, i);
        mma(s[n], a.x, b.x, a.y, b.y, x.x, x.y);
        mma(s[n], a.z, b.z, a.w, b.w, x.z, x.w);
      }
    }
    const bool edge = key + kKeys > sp.L || key < sp.first;
    const bool see0 = visible(sp, key + g), see1 = visible(sp, key + g + 8);
    bool grow = false;
    float mx[NB][2];
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      score(s[n]);
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
          c[e] = exp2_approx(m[n][e] - m2);
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

  __device__ __forceinline__ float4 four(int n, int e, int i, int u) const {
    const float(&a)[4] = o[n][4 * i + 2 * u], (&b)[4] = o[n][4 * i + 2 * u + 1];
    return make_float4(a[e], a[2 + e], b[e], b[2 + e]);
  }
  __device__ __forceinline__ void sum_up() {
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int w = 4; w < 32; w <<= 1) l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], w);
  }
  // The finished rows of a unit that this warp had alone.
  __device__ __forceinline__ void write_out(Out* out, float* lse, int nh, int lane) {
    const int g = lane >> 2, t = lane & 3;
    sum_up();
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int h = 8 * n + 2 * t + e;
        if (h >= nh) continue;
        const float r = inverse(l[n][e]);
        if (lse && g == 0) lse[h] = (m[n][e] + log2f(l[n][e])) * kLn2;
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
          const float4 a = four(n, e, i, 0), b = four(n, e, i, 1);
          const __nv_bfloat162 v[4] = {__floats2bfloat162_rn(a.x * r, a.y * r), __floats2bfloat162_rn(a.z * r, a.w * r),
                                       __floats2bfloat162_rn(b.x * r, b.y * r), __floats2bfloat162_rn(b.z * r, b.w * r)};
          *reinterpret_cast<uint4*>(out + h * D + 8 * (g + 8 * i)) = *reinterpret_cast<const uint4*>(v);
        }
      }
  }
  // Its piece of one: outputs [head][D], (max, sum) [head][2].
  __device__ __forceinline__ void write_piece(float* o_out, float* ml, int nh, int lane) {
    const int g = lane >> 2, t = lane & 3;
    sum_up();
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int h = 8 * n + 2 * t + e;
        if (h >= nh) continue;
        if (g == 0) __stcg(reinterpret_cast<float2*>(ml + 2 * h), make_float2(m[n][e], l[n][e]));
#pragma unroll
        for (int i = 0; i < D / 64; ++i)
#pragma unroll
          for (int u = 0; u < 2; ++u)
            __stcg(reinterpret_cast<float4*>(o_out + h * D + 8 * (g + 8 * i) + 4 * u), four(n, e, i, u));
      }
  }

  // This warp's maxima, sums and outputs of heads 8n .. 8n + 7 into the merge buffer.
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
            *reinterpret_cast<float4*>(o_out + h * D + 4 * merge_unit(h, 2 * (g + 8 * i) + u)) = four(k, e, i, u);
      }
    }
  }
};

// ---------------------------------------------------------------------------
// float32: FMAs.  Groups of 1024 / D keys.  A lane keeps D / 32 dimensions of Q and O for NH heads (the
// least power of two that holds the KV head's, 8 at most).  The partial products
// of 32 (key, head) pairs are summed over the lanes by 31 exchanges that leave
// each lane one pair, and the weights come back through shared memory as
// broadcasts.
// ---------------------------------------------------------------------------
template <int D, int NH>
struct F32Math {
  using Out = float;
  static constexpr int kHeads = NH;
  static constexpr int kFlush = D == 256 && NH == 8 ? 4 : NH;
  static constexpr int kKeys = 1024 / D;  // 8 KB of K and V
  static constexpr int kRowBytes = 4 * D;
  static constexpr int kWarpScratch = kKeys * NH * 4;  // the group's weights [key][head]
  static constexpr bool kQShared = false;
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

  __device__ __forceinline__ void begin(const DecodeParams& p, const char* qrow, int h0, int nh, int lane, uint32_t) {
#pragma unroll
    for (int h = 0; h < NH; ++h)
#pragma unroll
      for (int e = 0; e < kE; ++e) {
        q[h][e] = h < nh ? __ldg(reinterpret_cast<const float*>(qrow + h * kRowBytes) + dim(lane, e)) : 0.f;
        o[h][e] = 0.f;
      }
    m = kNoScore;
    l = 0.f;
    slope = p.slopes && lane % NH < nh ? slope_of(p.slopes, h0 + lane % NH) : 0.f;
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
#pragma unroll
      for (int w = kPairs; w < 32; w <<= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], w);
      s[i] = v[0];
    }
    score(s);
#pragma unroll
    for (int i = 0; i < kSets; ++i) {
      const int t = key + kAtOnce * i + lane % kPairs / NH;
      s[i] = fmaf(slope, (float)(t - (sp.L - 1)), s[i]);
      if (!visible(sp, t)) s[i] = -INFINITY;
      mx = fmaxf(mx, s[i]);
    }
#pragma unroll
    for (int w = NH; w < kPairs; w <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
    if (__any_sync(0xffffffffu, mx > m + 8.f)) {
      const float m2 = fmaxf(m, mx);
      const float c = exp2_approx(m - m2);
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

  __device__ __forceinline__ float sum_up() const {
    float v = l;
#pragma unroll
    for (int w = NH; w < kPairs; w <<= 1) v += __shfl_xor_sync(0xffffffffu, v, w);
    return v;
  }
  static __device__ __forceinline__ void put(float* to, const float (&x)[kE], float r, int lane) {
#pragma unroll
    for (int e = 0; e < kE; e += kVec)
      if constexpr (kVec == 4)
        __stcg(reinterpret_cast<float4*>(to + dim(lane, e)),
               make_float4(x[e] * r, x[e + 1] * r, x[e + 2] * r, x[e + 3] * r));
      else
        __stcg(reinterpret_cast<float2*>(to + dim(lane, e)), make_float2(x[e] * r, x[e + 1] * r));
  }
  __device__ __forceinline__ void write_out(Out* out, float* lse, int nh, int lane) {
    const float v = sum_up();
    if (lse && lane < nh) lse[lane] = (m + log2f(v)) * kLn2;
    const float r = inverse(v);
#pragma unroll
    for (int h = 0; h < NH; ++h) {
      const float rh = __shfl_sync(0xffffffffu, r, h);
      if (h < nh) put(out + h * D, o[h], rh, lane);
    }
  }
  __device__ __forceinline__ void write_piece(float* o_out, float* ml, int nh, int lane) {
    const float v = sum_up();
    if (lane < nh) __stcg(reinterpret_cast<float2*>(ml + 2 * lane), make_float2(m, v));
#pragma unroll
    for (int h = 0; h < NH; ++h)
      if (h < nh) put(o_out + h * D, o[h], 1.f, lane);
  }

  __device__ __forceinline__ void flush(int n, float* o_out, float* ml, int lane) {
    const float v = sum_up();
    if (lane < NH && lane / kFlush == n) {
      ml[2 * (lane % kFlush)] = m;
      ml[2 * (lane % kFlush) + 1] = v;
    }
#pragma unroll
    for (int k = 0; k < NH; ++k) {
      if (k / kFlush != n) continue;
      const int h = k % kFlush;
#pragma unroll
      for (int e = 0; e < kE; ++e) {
        const int d = dim(lane, e);
        o_out[h * D + 4 * merge_unit(h, d >> 2) + (d & 3)] = o[k][e];
      }
    }
  }
};

__device__ __forceinline__ void add(float4& v, float4 o, float w) {
  v.x = fmaf(o.x, w, v.x);
  v.y = fmaf(o.y, w, v.y);
  v.z = fmaf(o.z, w, v.z);
  v.w = fmaf(o.w, w, v.w);
}
__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v) {
  __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<uint32_t*>(&a), *reinterpret_cast<uint32_t*>(&b));
}

// A CTA: 8 warps whose rings take 192 KB, so that 128 KB are in flight while a
// third is computed; 4 warps where a group is 16 KB; 16 where it is 4 KB (twice
// the instructions a byte), which leaves 128 registers a thread: bf16 units of 8
// and 16 heads spill 20 and 38 bytes there (64 requests of 1k-8k, 32/8 heads: 105
// us, 0.84 of the copy rate).
template <class Math, int D>
struct Shape {
  static constexpr int kTile = Math::kKeys * Math::kRowBytes;  // K or V of a group
  static constexpr int kStage = 2 * kTile;
  static constexpr int kWarps = 65536 / kStage;
  static constexpr int kStages = 3;
  static constexpr int kRing = kWarps * kStages * kStage;
  static constexpr int kMerge = kWarps * Math::kFlush * D * 4;
  static constexpr int kSmem = kRing + kMerge + kWarps * (8 * 2 * 4 + Math::kWarpScratch);
  static_assert(kSmem <= 227 * 1024 - 512, "shared memory of a CTA");
};

template <class Math, int D>
__global__ void __launch_bounds__(Shape<Math, D>::kWarps * 32, 1) decode_kernel(const DecodeParams p) {
  using S = Shape<Math, D>;
  constexpr int kWarps = S::kWarps, kStages = S::kStages, kThreads = kWarps * 32, kHeads = Math::kHeads;
  constexpr int kKeys = Math::kKeys, kRowBytes = Math::kRowBytes;
  constexpr int kPieces = kRowBytes / 16;        // 16-byte pieces of a row
  constexpr int kCopies = kKeys * kPieces / 32;  // copies of a lane for a K or V tile
  constexpr int kLogWarps = kWarps == 16 ? 4 : kWarps == 8 ? 3 : 2;
  extern __shared__ __align__(128) char smem[];
  struct Piece {  // this CTA's piece of a cut team
    int c0;       // the team's first CTA
    int others;   // its other pieces
    int b, block;
  };
  __shared__ Piece s_piece[2];  // of the team that the slice's start cuts, of the one that its end cuts
  __shared__ int s_sum[kWarps][kLogWarps + 2];
  __shared__ bool s_last[2], s_top;
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem) + warp * kStages * S::kStage;
  const uint32_t ring_end = (uint32_t)__cvta_generic_to_shared(smem) + S::kRing;
  float* merge = reinterpret_cast<float*>(smem + S::kRing);
  float* merge_ml = reinterpret_cast<float*>(smem + S::kRing + S::kMerge);  // [warp][8][2]
  float* scratch = merge_ml + kWarps * 16 + warp * (Math::kWarpScratch / 4);

  // ---- teams and the cut ----
  // tiles of all requests when 2^k warps share a unit's keys, and the longest request's groups
  int sums[kLogWarps + 1], longest = 0;
#pragma unroll
  for (int k = 0; k <= kLogWarps; ++k) sums[k] = 0;
  const bool few = p.B <= 32;  // every warp sums for itself
  for (int b = few ? lane : tid; b < p.B; b += kThreads) {
    const int n = span_of<kKeys>(p, b).groups;
    longest = max(longest, n);
#pragma unroll
    for (int k = 0; k <= kLogWarps; ++k) sums[k] += max(1, (n + (1 << k) - 1) >> k);
  }
  longest = __reduce_max_sync(0xffffffffu, longest);
#pragma unroll
  for (int k = 0; k <= kLogWarps; ++k) sums[k] = __reduce_add_sync(0xffffffffu, sums[k]);
  if (!few) {
    if (lane == 0) {
#pragma unroll
      for (int k = 0; k <= kLogWarps; ++k) s_sum[warp][k] = sums[k];
      s_sum[warp][kLogWarps + 1] = longest;
    }
    __syncthreads();
    longest = s_sum[0][kLogWarps + 1];
#pragma unroll
    for (int k = 0; k <= kLogWarps; ++k) sums[k] = s_sum[0][k];
    for (int w = 1; w < kWarps; ++w) {
      longest = max(longest, s_sum[w][kLogWarps + 1]);
#pragma unroll
      for (int k = 0; k <= kLogWarps; ++k) sums[k] += s_sum[w][k];
    }
  }
  // The largest team that leaves every CTA 8 tiles and a team about 3 pieces; else a unit at a time.
  const int units = p.Hkv * p.head_groups;  // per request
  int team_log = -1, T = 0;
#pragma unroll
  for (int k = 0; k <= kLogWarps; ++k) {
    const int log = kLogWarps - k;  // of the team
    if (team_log >= 0 || log > p.team_log) continue;
    T = sums[k] * (units >> log);
    const int per = T / (int)gridDim.x;
    if (log == 0 || (per >= 8 && (longest >> k) <= 2 * per)) team_log = log;
  }
  const int share_log = kLogWarps - team_log;        // warps on a unit's keys
  const int member = warp & ((1 << team_log) - 1);   // this warp's unit in the team
  const int share = warp >> team_log;                // and its place among those that share it
  const int blocks = units >> team_log;              // teams per request
  const int P = min((int)gridDim.x, T);
  if (blockIdx.x >= P) return;
  int t = cta_start(blockIdx.x, T, P);
  const int t1 = cta_start(blockIdx.x + 1, T, P);
  auto tiles_of = [&](const Span& s) { return max(1, (s.groups + (1 << share_log) - 1) >> share_log); };

  struct Place {  // a tile: request, team in it, tile in the team
    int b, block, tile, tiles;
    Span span;
  };
  Place at;
  at.b = 0;
  for (int base = 0;; at.b += 32) {  // of tile t, 32 requests at a time
    const int b = at.b + lane;
    const int n = b < p.B ? tiles_of(span_of<kKeys>(p, b)) * blocks : 0;
    int incl = n;
#pragma unroll
    for (int w = 1; w < 32; w <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, w);
      if (lane >= w) incl += v;
    }
    const unsigned behind = __ballot_sync(0xffffffffu, base + incl > t);
    if (behind || at.b + 32 >= p.B) {
      const int x = behind ? __ffs(behind) - 1 : 0;
      base += __shfl_sync(0xffffffffu, incl - n, x);
      at.b += x;
      at.span = span_of<kKeys>(p, at.b);
      at.tiles = tiles_of(at.span);
      at.block = (t - base) / at.tiles;
      at.tile = (t - base) % at.tiles;
      break;
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
  }
  auto next_team = [&](Place& x) {
    x.tile = 0;
    if (++x.block == blocks) {
      x.block = 0;
      if (++x.b < p.B) {
        x.span = span_of<kKeys>(p, x.b);
        x.tiles = tiles_of(x.span);
      }
    }
  };
  struct Unit {
    int kvh, h0, nh;  // KV head, first query head, query heads
  };
  auto unit_of = [&](int block, int who) {
    const int u = (block << team_log) + who;
    Unit x;
    x.kvh = p.head_groups == 1 ? u : u / p.head_groups;
    const int hg = u - x.kvh * p.head_groups;
    x.h0 = x.kvh * p.G + hg * kHeads;
    x.nh = min(kHeads, p.G - hg * kHeads);
    return x;
  };
  auto query = [&](int b, const Unit& u) { return p.q + b * p.q_stride + (int64_t)u.h0 * kRowBytes; };
  auto touch_queries = [&](int b, int block) {  // into this SM's cache
    const Unit u = unit_of(block, member);
    const char* q = query(b, u);
    for (int i = lane; i < u.nh * (kRowBytes / 128); i += 32)
      asm volatile("{.reg .b32 x; ld.global.ca.b32 x, [%0];}" ::"l"(q + i * 128));
  };

  // ---- copies, kStages - 1 groups ahead, block table entries one more ----
  Place ahead = at;
  int ahead_left = t1 - t;
  // cache row of key lane % kKeys of the next group
  auto look_up = [&]() -> int64_t {
    int64_t row = kNoGroup;
    if (ahead_left > 0) {
      const int i = (ahead.tile << share_log) + share;
      if (i < ahead.span.groups) {
        const int t = group_key<kKeys>(ahead.span, i) + lane % kKeys;
        row = kZeros;
        if (visible(ahead.span, t)) {
          const int c = (int)((uint64_t)(uint32_t)t * p.div_mul >> p.div_shift);
          const int64_t blk = __ldg(p.table + (int64_t)ahead.b * p.max_blocks + c);
          if (blk >= 0 && blk < p.num_blocks)
            row = (blk * p.Hkv + unit_of(ahead.block, member).kvh) * p.block_size + (t - c * p.block_size);
          else if (p.status)
            atomicOr(p.status, TV_DEV_BAD_BLOCK);
        }
      }
      --ahead_left;
      if (++ahead.tile == ahead.tiles) next_team(ahead);
    }
    return row;
  };
  auto copy = [&](int64_t row, int stage) {
    const uint32_t dst = ring + stage * S::kStage;
    const int64_t row0 = __shfl_sync(0xffffffffu, row, 0);
    if (__all_sync(0xffffffffu, row == row0 + lane % kKeys && row >= 0)) {  // consecutive rows: one block
      const char* k = p.k_cache + row0 * kRowBytes + 16 * lane;
      const char* v = p.v_cache + row0 * kRowBytes + 16 * lane;
#pragma unroll
      for (int i = 0; i < kCopies; ++i) {
        const int x = i * 32 + lane;
        const uint32_t to = dst + Math::piece(x / kPieces, x % kPieces);
        cp_async16(to, k + 512 * i, true);
        cp_async16(to + S::kTile, v + 512 * i, true);
      }
    } else if (row != kNoGroup) {  // the same for the whole warp
#pragma unroll
      for (int i = 0; i < kCopies; ++i) {
        const int x = i * 32 + lane;
        const int r = x / kPieces, c = x % kPieces;
        const int64_t from = __shfl_sync(0xffffffffu, row, r);
        const int64_t off = (from < 0 ? 0 : from) * kRowBytes + 16 * c;
        cp_async16(dst + Math::piece(r, c), p.k_cache + off, from >= 0);
        cp_async16(dst + S::kTile + Math::piece(r, c), p.v_cache + off, from >= 0);
      }
    }
    cp_async_commit();
  };

  // Row of the workspace's pieces: slot 1 of the CTA that a team starts in, slot 0 of the others.
  auto part_row = [&](int c, bool starts, int who) {
    return ((2 * (int64_t)c + starts) * (1 << p.team_log) + who) * p.rows;
  };

  touch_queries(at.b, at.block);
  int64_t row = look_up();
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) {
    const int64_t now = row;
    row = look_up();
    copy(now, s);
  }

  // ---- the slice's teams ----
  const Scorer score(p);
  int stage = 0;
  bool last[2] = {false, false};  // this CTA's piece was its run's last (thread 0)
  bool cut = false;
  Math math;
  while (t < t1) {
    const Unit unit = unit_of(at.block, member);
    const int tile1 = min(at.tiles, at.tile + (t1 - t));
    math.begin(p, query(at.b, unit), unit.h0, unit.nh, lane, ring_end + warp * Math::kFlush * D * 4);
    if (t + tile1 - at.tile < t1) {
      const bool same = at.block + 1 < blocks;
      touch_queries(same ? at.b : at.b + 1, same ? at.block + 1 : 0);
    }
    for (int tile = at.tile; tile < tile1; ++tile) {
      cp_async_wait<kStages - 2>();
      __syncwarp();
      const int64_t now = row;
      row = look_up();
      copy(now, stage == 0 ? kStages - 1 : stage - 1);
      const int i = (tile << share_log) + share;
      if (i < at.span.groups)
        math.group(p, score, at.span, group_key<kKeys>(at.span, i), ring + stage * S::kStage,
                   ring + stage * S::kStage + S::kTile, lane, scratch);
      stage = stage == kStages - 1 ? 0 : stage + 1;
    }

    const bool whole = at.tile == 0 && tile1 == at.tiles;
    if (share_log == 0) {
      if (whole) {
        const int64_t out_row = (int64_t)at.b * p.Hq + unit.h0;
        math.write_out(reinterpret_cast<typename Math::Out*>(p.out) + out_row * D, p.lse ? p.lse + out_row : nullptr,
                       unit.nh, lane);
      } else {
        const int64_t to = part_row(blockIdx.x, at.tile == 0, member);
        math.write_piece(p.part_o + to * D, p.part_ml + to * 2, unit.nh, lane);
      }
    } else {
#pragma unroll
      for (int n = 0; n < kHeads / Math::kFlush; ++n) {
        if (n * Math::kFlush >= p.rows) break;
        __syncthreads();  // the buffer's last readers
        math.flush(n, merge + warp * Math::kFlush * D, merge_ml + warp * 16, lane);
        __syncthreads();
        for (int x = tid; x < (Math::kFlush * (D / 4)) << team_log; x += kThreads) {
          const int u = x % (D / 4), h = x / (D / 4) % Math::kFlush, who = x / (D / 4) / Math::kFlush;
          const Unit of = unit_of(at.block, who);
          const int hh = Math::kFlush * n + h;
          if (hh >= of.nh) continue;
          float mm = kNoScore;
          for (int w = who; w < kWarps; w += 1 << team_log) mm = fmaxf(mm, merge_ml[w * 16 + 2 * h]);
          float ll = 0.f;
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
          for (int w = who; w < kWarps; w += 1 << team_log) {
            const float c = exp2_approx(merge_ml[w * 16 + 2 * h] - mm);
            const float4 o = *reinterpret_cast<const float4*>(merge + (w * Math::kFlush + h) * D + 4 * merge_unit(h, u));
            ll = fmaf(merge_ml[w * 16 + 2 * h + 1], c, ll);
            add(v, o, c);
          }
          if (whole) {
            const float r = inverse(ll);
            const int64_t out_row = (int64_t)at.b * p.Hq + of.h0 + hh;
            store4(reinterpret_cast<typename Math::Out*>(p.out) + out_row * D + 4 * u,
                   make_float4(v.x * r, v.y * r, v.z * r, v.w * r));
            if (p.lse && u == 0) p.lse[out_row] = (mm + log2f(ll)) * kLn2;
          } else {
            const int64_t to = part_row(blockIdx.x, at.tile == 0, who) + hh;
            __stcg(reinterpret_cast<float4*>(p.part_o + to * D + 4 * u), v);
            if (u == 0) __stcg(reinterpret_cast<float2*>(p.part_ml + to * 2), make_float2(mm, ll));
          }
        }
      }
    }
    if (Math::kQShared && share_log > 0) __syncthreads();  // the buffer is read: the next queries may be written
    if (!whole) {
      cut = true;
      __syncthreads();  // the piece is written; thread 0's release covers it
      if (tid == 0) {
        const int c0 = cta_of(t - at.tile, T, P), c1 = cta_of(t - at.tile + at.tiles - 1, T, P);
        s_piece[at.tile == 0 ? 1 : 0] = {c0, c1 - c0, at.b, at.block};
        const int n = c1 - c0 + 1;
        const Runs runs(n);
        const int run = runs.of(blockIdx.x - c0);
        const bool end = (int)(arrive(p.arrive + c0 + run * runs.size, 1) & 0xffff) == runs.pieces(run, n) - 1;
        if (at.tile == 0) last[1] = end; else last[0] = end;
      }
    }
    t += tile1 - at.tile;
    at.tile = tile1;
    if (at.tile == at.tiles) next_team(at);
  }
  cp_async_wait<0>();
  if (!cut) return;

  // ---- joins of the teams that the slice's ends cut, where this CTA's piece came last ----
  if (tid == 0) {
#pragma unroll
    for (int k = 0; k < 2; ++k) s_last[k] = last[k];
  }
  __syncthreads();
#pragma unroll 1
  for (int k = 0; k < 2; ++k) {
    if (!s_last[k]) continue;
    const Piece mine = s_piece[k];  // read behind the barrier: what thread 0's arrival acquired is there for all
    // row of piece i in the workspace (at most 4096 CTAs, 2 pieces, 64 KB of outputs: under 2^31 floats)
    const int step = (int)part_row(1, false, 0);
    const int first = (int)part_row(mine.c0, true, 0), other = (int)part_row(mine.c0, false, 0);
    auto to_row = [&](int r, bool& here) {  // output row of the pieces' row r
      const Unit unit = unit_of(mine.block, r / p.rows);
      here = r % p.rows < unit.nh;
      return (int64_t)mine.b * p.Hq + unit.h0 + r % p.rows;
    };
    auto put = [&](int64_t row, int u, float4 v, float x) {
      store4(reinterpret_cast<typename Math::Out*>(p.out) + row * D + 4 * u, make_float4(v.x * x, v.y * x, v.z * x, v.w * x));
    };
    const int rows = p.rows << team_log;
    const int items = rows * (D / 4);
    constexpr int kBatch = kThreads > 256 ? 4 : 8;  // pieces that a thread has on their way at once (registers)
    if (mine.others < kBatch) {  // all of them: one trip to L2
      if (tid == 0) p.arrive[mine.c0] = 0;
      for (int x = tid; x < items; x += kThreads) {
        const int r = x / (D / 4), u = x % (D / 4);
        float4 o[kBatch];
        float2 a[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          if (i > mine.others) continue;
          const uint32_t from = (uint32_t)(i ? other + i * step : first) + r;
          a[i] = __ldcg(reinterpret_cast<const float2*>(p.part_ml) + from);
          o[i] = __ldcg(reinterpret_cast<const float4*>(p.part_o) + (from * (D / 4) + u));
        }
        float mm = kNoScore, ll = 0.f;
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
          if (i <= mine.others) mm = fmaxf(mm, a[i].x);
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          if (i > mine.others) continue;
          const float w = scaled(1.f, a[i].x, mm);
          ll = fmaf(a[i].y, w, ll);
          add(v, o[i], w);
        }
        bool here;
        const int64_t row = to_row(r, here);
        if (!here) continue;
        put(row, u, v, inverse(ll));
        if (p.lse && u == 0) p.lse[row] = (mm + log2f(ll)) * kLn2;
      }
      continue;
    }
    const int n = mine.others + 1;
    const Runs runs(n);
    const int run = runs.of(blockIdx.x - mine.c0);
    if (tid == 0) {  // every piece of the run is here; the others' may be counted in the same word
      if (run == 0 && runs.count > 1)
        arrive(p.arrive + mine.c0, -(uint32_t)runs.pieces(0, n));
      else
        p.arrive[mine.c0 + run * runs.size] = 0;
    }
    int base = run * runs.size, count = runs.pieces(run, n), stride = 1;  // pieces base, base + stride, ..
    bool final = runs.count == 1;
    auto part = [&](int i, int row) {
      const int x = base + i * stride;
      return (x ? other + x * step : first) + row;
    };
    for (;;) {
      // every row's maximum and sum: 8 or 32 lanes a row, a piece each in turn
      float* row_max = merge;
      float* row_inv = merge + rows;
      const int wide = rows * 32 <= kThreads ? 32 : 8;
      for (int r0 = 0; r0 < rows; r0 += kThreads / wide) {
        const int r = min(r0 + tid / wide, rows - 1);
        float mm = kNoScore, ll = 0.f;
#pragma unroll 4
        for (int i = tid % wide; i < count; i += wide) {
          const float2 a = __ldcg(reinterpret_cast<const float2*>(p.part_ml) + part(i, r));
          const float m2 = fmaxf(mm, a.x);
          ll = scaled(ll, mm, m2) + scaled(a.y, a.x, m2);
          mm = m2;
        }
        for (int w = 1; w < wide; w <<= 1) {
          const float m1 = __shfl_xor_sync(0xffffffffu, mm, w), l1 = __shfl_xor_sync(0xffffffffu, ll, w);
          const float m2 = fmaxf(mm, m1);
          ll = scaled(ll, mm, m2) + scaled(l1, m1, m2);
          mm = m2;
        }
        if (tid % wide == 0) {
          row_max[r] = mm;
          row_inv[r] = final ? inverse(ll) : ll;
          bool here;
          const int64_t row = to_row(r, here);
          if (p.lse && here && final) p.lse[row] = (mm + log2f(ll)) * kLn2;
        }
      }
      __syncthreads();
      // the outputs: some of a thread's and some pieces at a time, as each step is a trip to L2
      auto sum_up = [&](auto results, auto pieces) {
        constexpr int kAtOnce = decltype(results)::value, kPieces = decltype(pieces)::value;
        for (int x0 = tid; x0 < items; x0 += kThreads * kAtOnce) {
          float4 v[kAtOnce];
#pragma unroll
          for (int j = 0; j < kAtOnce; ++j) v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
          for (int i0 = 0; i0 < count; i0 += kPieces)
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) {
              const int x = x0 + j * kThreads;
              if (x >= items) continue;
              const int r = x / (D / 4);
              const float top = row_max[r];
              float4 o[kPieces];
              float w[kPieces];
#pragma unroll
              for (int k = 0; k < kPieces; ++k) {
                if (i0 + k >= count) continue;
                const uint32_t at_row = (uint32_t)part(i0 + k, r);
                w[k] = __ldcg(p.part_ml + at_row * 2);
                o[k] = __ldcg(reinterpret_cast<const float4*>(p.part_o) + (at_row * (D / 4) + x % (D / 4)));
              }
#pragma unroll
              for (int k = 0; k < kPieces; ++k)
                if (i0 + k < count) add(v[j], o[k], scaled(1.f, w[k], top));
            }
#pragma unroll
          for (int j = 0; j < kAtOnce; ++j) {
            const int x = x0 + j * kThreads, r = x / (D / 4);
            if (x >= items) continue;
            if (!final) {
              __stcg(reinterpret_cast<float4*>(p.part_o) + ((uint32_t)part(0, r) * (D / 4) + x % (D / 4)), v[j]);
              continue;
            }
            bool here;
            const int64_t row = to_row(r, here);
            if (here) put(row, x % (D / 4), v[j], row_inv[r]);
          }
        }
      };
      if (items <= kThreads)
        sum_up(std::integral_constant<int, 1>{}, std::integral_constant<int, 2 * kBatch>{});
      else
        sum_up(std::integral_constant<int, 4>{}, std::integral_constant<int, kBatch>{});
      __syncthreads();  // row_max is read; the next join writes it
      if (final) break;
      for (int r = tid; r < rows; r += kThreads)
        __stcg(reinterpret_cast<float2*>(p.part_ml) + part(0, r), make_float2(row_max[r], row_inv[r]));
      __syncthreads();  // the run's piece is written; thread 0's release covers it
      if (tid == 0) {
        s_top = arrive(p.arrive + mine.c0, 0x10000) >> 16 == (uint32_t)runs.count - 1;
        if (s_top) p.arrive[mine.c0] = 0;  // every run is here
      }
      __syncthreads();
      if (!s_top) break;
      base = 0;
      count = runs.count;
      stride = runs.size;
      final = true;
    }
  }
}

// Largest team of a shape, log2: a power of two that divides a request's units and the warps, with a piece of at
// most 8192 outputs.
int team_log_of(int units, int warps, int heads, int D) {
  int k = 0;
  while ((2 << k) <= warps && units % (2 << k) == 0 && (2 << k) * heads * D <= 8192) ++k;
  return k;
}

// What the workspace holds for a shape and grid, besides the counters.
struct Room {
  int rows, head_groups, team_log;
  size_t floats;  // outputs of all pieces
  size_t bytes;
};

template <class Math, int D>
Room room_of(int Hkv, int G, int ctas) {
  Room r;
  r.rows = std::min(G, Math::kHeads);
  r.head_groups = (G + Math::kHeads - 1) / Math::kHeads;
  // units modulo 16 are all that the team goes by
  r.team_log = team_log_of((int)((int64_t)Hkv * r.head_groups % 16) + 16, Shape<Math, D>::kWarps, r.rows, D);
  const size_t rows = ((size_t)ctas * 2 * r.rows) << r.team_log;
  r.floats = rows * D;
  r.bytes = rows * (D + 2) * 4;
  return r;
}

// What a call asks of the instantiation that fits its shape: its room, or its launch.
struct Call {
  int ctas;
  Room* room;       // non-null: only this
  DecodeParams* p;
  cudaStream_t stream;
};

template <class Math, int D>
int call_decode(const Call& c, int Hkv, int G) {
  const Room r = room_of<Math, D>(Hkv, G, c.ctas);
  if (c.room) {
    *c.room = r;
    return TV_OK;
  }
  constexpr int smem = Shape<Math, D>::kSmem;
  DecodeParams& p = *c.p;
  p.head_groups = r.head_groups;
  p.team_log = r.team_log;
  p.rows = r.rows;
  p.part_ml = p.part_o + r.floats;
  const double tiles = (double)p.max_blocks * p.block_size / Math::kKeys + 2;
  if (tiles * p.B * p.Hkv * p.head_groups >= (double)INT32_MAX)
    return tv::fail(TV_ERR_UNSUPPORTED, "tv_decode_attn: the work could reach 2^31 groups of %d keys", Math::kKeys);
  TV_CUDA_TRY(cudaFuncSetAttribute(decode_kernel<Math, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
  decode_kernel<Math, D><<<c.ctas, Shape<Math, D>::kWarps * 32, smem, c.stream>>>(p);
  TV_LAUNCH_CHECK("decode_kernel");
  return TV_OK;
}

// Query heads of a unit.  bf16: 8, or 16 where a KV head serves more than 8 (two
// 8-column products share a key's loads), rows of 256 only where the units are a
// quarter of the CTAs, as their pieces are twice as large (60 requests of 2k-8.7k,
// 32/2 heads: 138-147 us, 8 heads a unit 203; 8 of 500-2000: 35 and 21).  Units of
// unused slots and short requests count alike: lengths are known on the device
// only.  float32: as many as the KV head serves, 8 at most.
template <int D>
int dispatch_heads(const Call& c, int dtype, int Hkv, int G) {
  if (dtype == TV_BF16) {
    if (G > 8 && (D < 256 || c.room || 4 * (int64_t)c.p->B * Hkv >= c.ctas)) {
      if (D == 256 && c.room) {  // the room that either needs
        if (int rc = call_decode<Bf16Math<D, 1>, D>(c, Hkv, G)) return rc;
        const Room one = *c.room;
        if (int rc = call_decode<Bf16Math<D, 2>, D>(c, Hkv, G)) return rc;
        c.room->bytes = std::max(c.room->bytes, one.bytes);
        return TV_OK;
      }
      return call_decode<Bf16Math<D, 2>, D>(c, Hkv, G);
    }
    return call_decode<Bf16Math<D, 1>, D>(c, Hkv, G);
  }
  if (G == 1) return call_decode<F32Math<D, 1>, D>(c, Hkv, G);
  if (G == 2) return call_decode<F32Math<D, 2>, D>(c, Hkv, G);
  if (G <= 4) return call_decode<F32Math<D, 4>, D>(c, Hkv, G);
  return call_decode<F32Math<D, 8>, D>(c, Hkv, G);
}

int dispatch_decode(const Call& c, int D, int dtype, int Hkv, int G) {
  if (D == 64) return dispatch_heads<64>(c, dtype, Hkv, G);
  if (D == 128) return dispatch_heads<128>(c, dtype, Hkv, G);
  return dispatch_heads<256>(c, dtype, Hkv, G);
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
  Room room;
  if (int rc = dispatch_decode({ctas, &room, nullptr, nullptr}, head_dim, dtype, Hkv, Hq / Hkv)) return rc;
  *bytes = (size_t)kCounterBytes + room.bytes;
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
  if (!factors_fit(scale, softcap))
    return tv::fail(TV_ERR_INVALID_ARG,
                    "tv_decode_attn: scale must be finite, softcap finite and not negative, both within 2.3e38");
  if (flags & ~TV_ATTN_WORKSPACE_ZEROED) return tv::fail(TV_ERR_INVALID_ARG, "tv_decode_attn: unknown flags %d", flags);
  if (B == 0) return TV_OK;
  if (!q || !k_cache || !v_cache || !block_table || !seq_lens || !out)
    return tv::fail(TV_ERR_INVALID_ARG, "tv_decode_attn: null pointer");
  const int64_t e = dtype == TV_F32 ? 4 : 2;
  if ((B > 1 && (q_stride < 0 || (q_stride * e) % 16)) ||
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
  p.softcap = cap_that_matters(scale, softcap);
  p.window = window;
  p.n_sink = n_sink;
  p.slopes = slopes;
  p.out = static_cast<char*>(out);
  p.lse = lse;
  p.status = status;
  p.arrive = static_cast<uint32_t*>(workspace);
  p.part_o = reinterpret_cast<float*>(static_cast<char*>(workspace) + kCounterBytes);
  // t < 2^31, 2^(s-1) < d <= 2^s, m = ceil(2^(31+s) / d) < 2^32: t m / 2^(31+s) has the whole part of t / d, being
  // larger by t (m d - 2^(31+s)) / (d 2^(31+s)) < 1 / d
  uint32_t sh = 0;
  while ((1ll << sh) < block_size) ++sh;
  p.div_shift = 31 + sh;
  p.div_mul = (uint32_t)(((1ull << p.div_shift) + block_size - 1) / block_size);
  return dispatch_decode({ctas, nullptr, &p, st}, head_dim, dtype, Hkv, p.G);
}
