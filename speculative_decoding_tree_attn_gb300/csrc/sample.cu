// Sampling a token from a row of logits with temperature, top-k, min-p and
// top-p, from a given uniform number.
//
// With m = max x and w_i = e^((x_i - m) / T): of the top_k largest logits (equal
// ones by index), those with w_i >= min_p, and of these in descending order the
// shortest run that holds top_p of their sum, are kept; the token is the first
// index whose running sum over the kept ones exceeds u times their total W, and
// w_i / W are the probabilities.  "Implement the lossless speculative sampling
// verifier ...", "Details that matter in review": acceptance has to be given the
// distributions that tokens are drawn from, so both come out of one call.
//
// A draw among V tokens goes wrong wherever a running sum is off by as much as u
// W is away from it, so sums in float32 would give another token in one of a
// hundred draws over 128,000.  Weights are therefore whole numbers, w 2^43 to
// 2^-36 of itself, and their sums exact and independent of order:
//   w = 2^(n / 64) e^t,  (x - m) log2 e / T = n / 64 + r in two floats, t = r ln 2,
// with the 64 powers from a table and e^t by its series (Tang's table-driven
// exponential, ACM TOMS 15, 1989); |t| < 0.0055, so that only its first term needs
// two floats.
//
// A top_k limit: the threads' own largest logits give a bar that top_k elements reach
// and few more; those are sorted in one CTA.  Else a limit is found by a
// histogram of the weights' logarithms (128 bins to a factor of 2), whose
// approximate masses tell the bin that it is in; one pass of exact sums confirms
// it and collects that bin's elements, which are sorted.
//
// A row is read again for each pass, from L2: bound by the instructions of the
// exact pass (45 an element of float32, 15 of bf16) where there is no top_k, by
// the passes' exchanges where there are few rows.  64 registers (two CTAs an SM)
// spill 12 to 32 bytes.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstring>

#include "common.h"

namespace cg = cooperative_groups;

namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kBins = 4096, kPerOctave = 128;
constexpr int kList = 1024;      // elements that are sorted
constexpr int kChunk = 256;      // elements whose kept mass is one number
constexpr int kMaxV = 1 << 20;   // sums stay below 2^64
constexpr int kMaxCluster = 8;
constexpr uint32_t kTableFrom = 0x3c00, kTableSize = 0x600;  // bf16 magnitudes from 2^-7 to 32
constexpr float kLn2Hi = 0.693147182464599609375f, kLn2Lo = -1.904654323148236e-09f;  // ln 2 in two floats
constexpr float kCold = 0x1p-60f;  // a temperature below counts as 0, one above the inverse as that

// 2^(j / 64 + 43), rounded
__constant__ unsigned long long kPowers[64] = {
    8796093022208ull, 8891876195264ull, 8988702378691ull, 9086582930126ull,
    9185529330885ull, 9285553187305ull, 9386666232110ull, 9488880325783ull,
    9592207457961ull, 9696659748838ull, 9802249450589ull, 9908988948806ull,
    10016890763953ull, 10125967552830ull, 10236232110063ull, 10347697369602ull,
    10460376406236ull, 10574282437131ull, 10689428823381ull, 10805829071568ull,
    10923496835354ull, 11042445917079ull, 11162690269381ull, 11284243996830ull,
    11407121357589ull, 11531336765078ull, 11656904789672ull, 11783840160404ull,
    11912157766698ull, 12041872660113ull, 12173000056107ull, 12305555335825ull,
    12439554047902ull, 12575011910285ull, 12711944812080ull, 12850368815412ull,
    12990300157313ull, 13131755251623ull, 13274750690919ull, 13419303248457ull,
    13565429880144ull, 13713147726524ull, 13862474114787ull, 14013426560807ull,
    14166022771192ull, 14320280645363ull, 14476218277651ull, 14633853959423ull,
    14793206181226ull, 14954293634955ull, 15117135216047ull, 15281750025697ull,
    15448157373097ull, 15616376777705ull, 15786427971528ull, 15958330901445ull,
    16132105731538ull, 16307772845465ull, 16485352848846ull, 16664866571680ull,
    16846335070792ull, 17029779632301ull, 17215221774115ull, 17402683248456ull};

struct SampleParams {
  const char* logits;
  int64_t R;
  int V;
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  const float* u;
  int32_t* tokens;
  float* probs;
  int32_t* status;
  int slice;  // elements of a CTA, a multiple of kChunk
};

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Order of elements as one whole number: the value's place, then the lower index first.
__device__ __forceinline__ uint64_t place(float x, int i) {
  const uint32_t bits = __float_as_uint(x + 0.f);  // -0 is 0
  const uint32_t key = bits & 0x80000000u ? ~bits : bits | 0x80000000u;
  return (uint64_t)key << 32 | (uint32_t)~i;
}

struct Scale {
  float m, c1, c2;  // log2 e / T in two floats
  float floor_y;    // a weight whose log2w() lies below is less than min_p, one 2^-8 above is not

  // (x - m) log2 e / T; the first float alone falls with x
  __device__ __forceinline__ float log2w(float x) const { return (x - m) * c1; }

  // w = mantissa 2^(-43 - s) up to 2^-36 of it, the mantissa within [2^42.99, 2^43.993); y > -126.  In units of 2^-39: q's
  // float32 roundings 2.7, the two of e 2, what p >> 12 cuts 1.4, tl's 0.9, the rest 0.1 (3.8 is the most of 40 million).
  __device__ __forceinline__ uint64_t mantissa(float x, const unsigned long long* powers, int& s) const {
    const float dh = x - m, back = dh - x;
    const float dl = (x - (dh - back)) - (m + back);
    const float yh = dh * c1;
    const float yl = fmaf(dh, c1, -yh) + fmaf(dh, c2, dl * c1);
    const float n = rintf(yh * 64.f);
    const float rh = fmaf(n, -0x1p-6f, yh);  // exact
    const float th = rh * kLn2Hi;
    const float tl = fmaf(rh, kLn2Hi, -th) + fmaf(rh, kLn2Lo, yl * kLn2Hi);
    const float t = th + tl;
    const float q = t * t * fmaf(t, fmaf(t, fmaf(t, 1.f / 120.f, 1.f / 24.f), 1.f / 6.f), 0.5f);
    const int e = __float2int_rn(th * 0x1p38f) + __float2int_rn((tl + q) * 0x1p38f);  // (e^t - 1) 2^38
    const int ni = (int)n;
    const unsigned long long p = powers[ni & 63];
    s = -(ni >> 6);
    return p + (uint64_t)(((int64_t)(p >> 12) * e) >> 26);
  }
  // rint(w 2^43)
  __device__ __forceinline__ uint64_t weight(float x, const unsigned long long* powers) const {
    if (!(log2w(x) > -45.f)) return 0;
    int s;
    const uint64_t w = mantissa(x, powers, s);
    return s == 0 ? w : ((w >> (s - 1)) + 1) >> 1;
  }
  // w, to float32
  __device__ __forceinline__ float probability(float x, const unsigned long long* powers) const {
    if (!(log2w(x) > -126.f)) return 0.f;
    int s;
    const uint64_t w = mantissa(x, powers, s);
    return (float)w * 0x1p-43f * __uint_as_float((uint32_t)(127 - s) << 23);
  }
};

__device__ __forceinline__ int bin_of(float y) { return min(kBins - 1, (int)(y * -(float)kPerOctave)); }

struct Shared {
  unsigned long long powers[64];
  unsigned long long warp_sums[kWarps][2];
  unsigned long long totals[2][2];  // exchanged with the cluster's CTAs, in turns
  uint32_t count[kBins], mass[kBins];
  unsigned long long chunk[kMaxV / kMaxCluster / kChunk + 1];  // kept mass
  unsigned long long list_place[kList], list_weight[kList];  // of this CTA
  unsigned long long all_place[kList], all_weight[kList];    // of the cluster
  uint32_t listed, gathered;
  unsigned long long limit, total;
  unsigned long long table[2][kTableSize];  // weights of bf16 logits, by sign and magnitude
  int bin;
  int least_s;
  unsigned long long least;
};

// min_p as least 2^(-43 - least_s), least within [2^43, 2^44).  Below 2^-126 there is no limit: the weights that it would
// take away have a probability of 0 anyway.  By one thread, before the CTA's next barrier.
__device__ __forceinline__ void set_least(Shared& sh, float min_p) {
  int e;
  sh.least = (unsigned long long)(frexpf(fmaxf(fminf(min_p, 1.f), 0.f), &e) * 0x1p24f) << 20;
  sh.least_s = 1 - e;
}
// log2w() is off by 3 2^-24 of itself, 2^-15 at most here, log2f by less.
__device__ __forceinline__ float floor_of(float min_p) { return min_p >= FLT_MIN ? log2f(fminf(min_p, 1.f)) - 0x1p-9f : -FLT_MAX; }
// Whether a weight near the border reaches min_p.  A call of its own: inlined into every pass it took 3-10 % of short rows.
__device__ __noinline__ bool reaches(float m, float c1, float c2, const Shared& sh, float x) {
  const Scale sc{m, c1, c2, 0.f};
  int s;
  const unsigned long long w = sc.mantissa(x, sh.powers, s);  // within [2^42.99, 2^43.993)
  const int d = sh.least_s - s;
  return d >= 0 && (d > 1 || w << d >= sh.least);
}
// Whether min_p leaves x, whose log2w() is y.  All passes ask here: what one counts the others find.
__device__ __forceinline__ bool min_p_leaves(const Scale& sc, const Shared& sh, float x, float y) {
  return y >= sc.floor_y && (y >= sc.floor_y + 0x1p-8f || reaches(sc.m, sc.c1, sc.c2, sh, x));
}

__device__ __forceinline__ unsigned long long warp_sum(unsigned long long x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
__device__ __forceinline__ unsigned long long warp_max(unsigned long long x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x = max(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}

// floor(x u), x < 2^64, u in [0, 1)
__device__ __forceinline__ unsigned long long times(unsigned long long x, float u) {
  if (!(u > 0.f)) return 0;
  int e;
  const unsigned long long f = (unsigned long long)(frexpf(u, &e) * 0x1p24f);  // u = f 2^(e - 24)
  const unsigned long long lo = x * f, hi = __umul64hi(x, f);
  const int s = 24 - e;  // 24 ..
  if (s >= 64) return s >= 128 ? 0 : hi >> (s - 64);
  return hi << (64 - s) | lo >> s;
}
// ceil(x u)
__device__ __forceinline__ unsigned long long times_up(unsigned long long x, float u) {
  const unsigned long long y = times(x, u);
  // x u is whole only if nothing was cut off: u = f 2^(e - 24) cuts the low bits of x f
  int e;
  const unsigned long long f = (unsigned long long)(frexpf(u, &e) * 0x1p24f);
  const int s = 24 - e;
  if (s >= 64) return y + 1;
  return y + ((x * f & ((1ull << s) - 1)) != 0);
}

template <typename T>
struct Row {
  const SampleParams& p;
  Shared& sh;
  cg::cluster_group cluster;
  int rank, turn;
  const T* row;   // of the logits
  int v0, v1;     // this CTA's elements
  bool wide;      // rows of whole vectors

  // Sums (or maxima) of two numbers over the cluster; before0/1: those of the CTAs before this one.
  template <bool kMax>
  __device__ void reduce(unsigned long long& a, unsigned long long& b, unsigned long long* before = nullptr) {
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    a = kMax ? warp_max(a) : warp_sum(a);
    b = kMax ? warp_max(b) : warp_sum(b);
    __syncthreads();
    if (lane == 0) sh.warp_sums[warp][0] = a, sh.warp_sums[warp][1] = b;
    __syncthreads();
    if (warp == 0) {
      a = lane < kWarps ? sh.warp_sums[lane][0] : 0;
      b = lane < kWarps ? sh.warp_sums[lane][1] : 0;
      a = kMax ? warp_max(a) : warp_sum(a);
      b = kMax ? warp_max(b) : warp_sum(b);
      if (lane == 0) sh.totals[turn][0] = a, sh.totals[turn][1] = b;
    }
    cluster.sync();
    a = b = 0;
    const int n = (int)cluster.num_blocks();
    for (int r = 0; r < n; ++r) {
      const unsigned long long* t = cluster.map_shared_rank(&sh.totals[turn][0], r);
      if (before && r == rank) *before = a;
      a = kMax ? max(a, t[0]) : a + t[0];
      b = kMax ? max(b, t[1]) : b + t[1];
    }
    turn ^= 1;
  }

  // bf16 has few values: the weights of nearly all that logits take fit a table, and a weight costs a lookup instead of
  // some 45 instructions.  Filled for every row, as it costs little: 64 rows of 128,000 without limits 42 -> 32 us, with
  // top-p 64 of some 50,000 57.5 -> 54.5, 200 of 32,000 98 -> 95, 200 of 8000 66 -> 67.5, 200 of 500 27 -> 27.5.
  __device__ void fill_table(const Scale& sc) {
    if constexpr (sizeof(T) == 2) {
      for (uint32_t i = threadIdx.x; i < 2 * kTableSize; i += kThreads) {
        const uint32_t sign = i >= kTableSize, mag = kTableFrom + i - sign * kTableSize;
        sh.table[sign][mag - kTableFrom] = sc.weight(fminf(__uint_as_float((sign << 15 | mag) << 16), sc.m), sh.powers);
      }
      __syncthreads();
    }
  }
  __device__ __forceinline__ unsigned long long weight(const Scale& sc, float x) const {
    if constexpr (sizeof(T) == 2) {
      const uint32_t bits = __float_as_uint(x) >> 16, at = (bits & 0x7fff) - kTableFrom;
      if (at < kTableSize) return sh.table[bits >> 15][at];
    }
    return sc.weight(x, sh.powers);
  }

  // Eight elements from i on as they lie in memory; -inf behind the slice's end.
  struct Raw {
    uint4 v[sizeof(T) / 2];
  };
  __device__ __forceinline__ Raw load(int i) const {
    Raw r;
    if (wide && i + 8 <= v1) {
#pragma unroll
      for (int k = 0; k < (int)sizeof(T) / 2; ++k) r.v[k] = __ldg(reinterpret_cast<const uint4*>(row + i) + k);
      return r;
    }
    T x[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = i + k < v1 ? row[i + k] : (T)-INFINITY;
    memcpy(&r, x, sizeof(r));
    return r;
  }
  static __device__ __forceinline__ void unpack(const Raw& r, float (&x)[8]) {
    if constexpr (sizeof(T) == 4) {
      memcpy(x, &r, sizeof(r));
    } else {
      const uint32_t v[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) x[2 * k] = __uint_as_float(v[k] << 16), x[2 * k + 1] = __uint_as_float(v[k] & 0xffff0000u);
    }
  }
  // Calls g(x[8], index of x[0], turn) for this CTA's elements, each thread's in ascending order and every lane of a warp
  // in every turn.  A warp's 256 elements of one turn lie together, the next turns' are on their way.
  template <class G>
  __device__ __forceinline__ void turns(G g) const {
    const int lane = threadIdx.x % 32;
    constexpr int kStep = kThreads * 8;
    int i0 = v0 + (threadIdx.x - lane) * 8;
    if (i0 >= v1) return;
    constexpr bool kTwo = sizeof(T) == 2;  // 64 bytes of a thread on their way
    Raw now = load(i0 + lane * 8), next;
    if constexpr (kTwo) next = load(i0 + kStep + lane * 8);
#pragma unroll 1
    for (; i0 < v1; i0 += kStep) {
      const Raw after = load(i0 + (kTwo ? 2 : 1) * kStep + lane * 8);
      float x[8];
      unpack(now, x);
      g(x, i0 + lane * 8, (i0 - v0) / kChunk);
      now = kTwo ? next : after;
      next = after;
    }
  }
  // Calls f(x, index) for them one by one (and for some -inf behind the slice's end).
  template <class F>
  __device__ __forceinline__ void each(F f) const {
    turns([&](const float (&x)[8], int i, int) {
#pragma unroll
      for (int k = 0; k < 8; ++k) f(x[k], i + k);
    });
  }

  // Bins of the whole row from those of the cluster's CTAs: each adds up its share of them and hands it to the others.
  template <bool kMass>
  __device__ void share_bins() {
    cluster.sync();
    const int n = (int)cluster.num_blocks();
    if (n == 1) return;
    const int each = kBins / n, b0 = rank * each;
    uint32_t c[kBins / kThreads / 2] = {}, w[kBins / kThreads / 2] = {};  // n >= 2
#pragma unroll
    for (int k = 0; k < kBins / kThreads / 2; ++k) {
      const int b = threadIdx.x + k * kThreads;
      if (b >= each) break;
      for (int r = 0; r < n; ++r) {
        c[k] += cluster.map_shared_rank(sh.count, r)[b0 + b];
        if (kMass) w[k] += cluster.map_shared_rank(sh.mass, r)[b0 + b] >> 3;
      }
    }
    cluster.sync();
#pragma unroll
    for (int k = 0; k < kBins / kThreads / 2; ++k) {
      const int b = threadIdx.x + k * kThreads;
      if (b >= each) break;
      for (int r = 0; r < n; ++r) {
        cluster.map_shared_rank(sh.count, r)[b0 + b] = c[k];
        if (kMass) cluster.map_shared_rank(sh.mass, r)[b0 + b] = w[k];
      }
    }
    cluster.sync();
  }

  // First bin at which the running count (or mass, in the weights' unit) reaches target; -1 without one.
  template <bool kMass>
  __device__ int find_bin(unsigned long long target, int last_bin, int unit_bits) {
    constexpr int kPer = kBins / kThreads;
    auto of = [&](int b) -> unsigned long long {
      if (b > last_bin) return 0;
      if (!kMass) return sh.count[b];
      return (unsigned long long)sh.mass[b] << unit_bits >> (b / kPerOctave);
    };
    unsigned long long mine = 0;
    for (int k = 0; k < kPer; ++k) mine += of(threadIdx.x * kPer + k);
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    unsigned long long run = mine;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const unsigned long long y = __shfl_up_sync(0xffffffffu, run, o);
      if (lane >= o) run += y;
    }
    __syncthreads();
    if (lane == 31) sh.warp_sums[warp][0] = run;
    if (threadIdx.x == 0) sh.bin = -1;
    __syncthreads();
    run -= mine;
    for (int k = 0; k < warp; ++k) run += sh.warp_sums[k][0];
    if (run < target && run + mine >= target) {
      for (int k = 0; k < kPer; ++k) {
        const unsigned long long y = of(threadIdx.x * kPer + k);
        if (run < target && run + y >= target) sh.bin = threadIdx.x * kPer + k;
        run += y;
      }
    }
    __syncthreads();
    return sh.bin;
  }
  // Mass of the bins above one, by their approximate masses; the same in every CTA.
  __device__ unsigned long long mass_above(int bin, int unit_bits) {
    unsigned long long a = 0;
    for (int b = threadIdx.x; b < bin; b += kThreads) a += (unsigned long long)sh.mass[b] << unit_bits >> (b / kPerOctave);
    a = warp_sum(a);
    __syncthreads();
    if (threadIdx.x % 32 == 0) sh.warp_sums[threadIdx.x / 32][0] = a;
    __syncthreads();
    a = 0;
    for (int k = 0; k < kWarps; ++k) a += sh.warp_sums[k][0];
    __syncthreads();
    return a;
  }
  // Next bin in a direction with anything in it
  __device__ int next_bin(int b, int step, int last_bin) const {
    for (b += step; b >= 0 && b <= last_bin; b += step)
      if (sh.count[b]) return b;
    return -1;
  }

  // Least and largest place of a bin's kept elements from `from` on.
  template <class Kept>
  __device__ void range_of(const Scale& sc, int bin, unsigned long long from, unsigned long long& lo, unsigned long long& hi,
                           Kept kept) {
    unsigned long long least = 0, most = 0;  // least: inverted
    each([&](float x, int i) {
      const float y = sc.log2w(x);
      if (bin_of(y) != bin || !kept(x, y)) return;
      const unsigned long long at = place(x, i);
      if (at < from) return;
      least = max(least, ~at);
      most = max(most, at);
    });
    reduce<true>(least, most);
    lo = ~least;
    hi = most;
  }

  // Kept elements of bin `bin` with lo <= place <= hi, which are kList at most, in every CTA's list; their number.
  template <class Kept>
  __device__ int gather(const Scale& sc, int bin, unsigned long long lo, unsigned long long hi, Kept kept) {
    __syncthreads();
    if (threadIdx.x == 0) sh.listed = 0;
    __syncthreads();
    each([&](float x, int i) {
      const float y = sc.log2w(x);
      if (bin_of(y) != bin || !kept(x, y)) return;
      const unsigned long long at = place(x, i);
      if (at < lo || at > hi) return;
      const uint32_t k = atomicAdd(&sh.listed, 1u);
      if (k < kList) sh.list_place[k] = at, sh.list_weight[k] = sc.weight(x, sh.powers);
    });
    return merge_lists();
  }
  // The CTAs' lists in every one of them; their number.
  __device__ int merge_lists() {
    cluster.sync();
    const int n = (int)cluster.num_blocks();
    int total = 0;
    for (int r = 0; r < n; ++r) {
      const int c = min((int)*cluster.map_shared_rank(&sh.listed, r), kList);
      for (int k = threadIdx.x; k < c && total + k < kList; k += kThreads) {
        sh.all_place[total + k] = cluster.map_shared_rank(sh.list_place, r)[k];
        sh.all_weight[total + k] = cluster.map_shared_rank(sh.list_weight, r)[k];
      }
      total += c;
    }
    cluster.sync();
    return min(total, kList);
  }
};

// Sorts n places in descending order, their weights along; n2 >= n is a power of two.
__device__ void sort_places(Shared& sh, int n, int n2) {
  for (int i = n + threadIdx.x; i < n2; i += kThreads) sh.all_place[i] = 0, sh.all_weight[i] = 0;
  for (int k = 2; k <= n2; k *= 2)
    for (int j = k / 2; j > 0; j /= 2) {
      __syncthreads();
      for (int x = threadIdx.x; x < n2 / 2; x += kThreads) {
        const int lo = 2 * x - (x & (j - 1)), hi = lo + j;
        const unsigned long long a = sh.all_place[lo], b = sh.all_place[hi];
        if ((a < b) == ((lo & k) == 0)) {
          sh.all_place[lo] = b, sh.all_place[hi] = a;
          const unsigned long long w = sh.all_weight[lo];
          sh.all_weight[lo] = sh.all_weight[hi], sh.all_weight[hi] = w;
        }
      }
    }
  __syncthreads();
}

__device__ void sort_list(Shared& sh, int n) {
  int n2 = 2;
  while (n2 < n) n2 *= 2;
  sort_places(sh, n, n2);
}

// First i < n at which the running sum of the sorted weights exceeds goal, in sh.bin (n - 1 without one), and the running
// sum there in sh.total; returns the sum of all n.
__device__ unsigned long long scan_weights(Shared& sh, int n, unsigned long long goal, bool find) {
  const int per = (n + kThreads - 1) / kThreads, i0 = min(n, (int)threadIdx.x * per), i1 = min(n, i0 + per);
  unsigned long long mine = 0;
  for (int i = i0; i < i1; ++i) mine += sh.all_weight[i];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  unsigned long long run = mine;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const unsigned long long y = __shfl_up_sync(0xffffffffu, run, o);
    if (lane >= o) run += y;
  }
  __syncthreads();
  if (lane == 31) sh.warp_sums[warp][0] = run;
  if (threadIdx.x == 0 && find) sh.bin = n - 1;
  __syncthreads();
  unsigned long long total = 0;
  run -= mine;
  for (int k = 0; k < kWarps; ++k) {
    if (k < warp) run += sh.warp_sums[k][0];
    total += sh.warp_sums[k][0];
  }
  if (find) {
    if (run <= goal && run + mine > goal) {
      for (int i = i0; i < i1; ++i) {
        run += sh.all_weight[i];
        if (run > goal) {
          sh.bin = i;
          sh.total = run;
          break;
        }
      }
    } else if (threadIdx.x == 0 && goal >= total) {
      sh.total = total;
    }
  }
  __syncthreads();
  return total;
}

// A row whose limits leave at most kList candidates: those with a bin up to `bar` and of at least min_p.  They are sorted
// in the cluster's first CTA, which cuts and draws.  False where there are more.
template <typename T>
__device__ bool sample_sorted(Row<T>& r, const Scale& sc, int bar, int top_k, float top_p, float u, int32_t* token) {
  Shared& sh = r.sh;
  __syncthreads();
  if (threadIdx.x == 0) sh.gathered = 0;
  r.cluster.sync();
  uint32_t* count = r.cluster.map_shared_rank(&sh.gathered, 0);
  unsigned long long* places = r.cluster.map_shared_rank(sh.all_place, 0);
  unsigned long long* weights = r.cluster.map_shared_rank(sh.all_weight, 0);
  r.each([&](float x, int i) {
    const float y = sc.log2w(x);
    if (!(y >= sc.floor_y) || bin_of(y) > bar || !min_p_leaves(sc, sh, x, y)) return;
    const uint32_t k = atomicAdd(count, 1u);
    if (k < kList) places[k] = place(x, i), weights[k] = sc.weight(x, sh.powers);
  });
  r.cluster.sync();
  const uint32_t n_all = *count;
  r.cluster.sync();
  if (n_all > kList) return false;
  if (r.rank == 0) {
    int n = (int)n_all;
    sort_list(sh, n);
    if (top_k > 0) n = min(n, top_k);
    unsigned long long total = scan_weights(sh, n, 0, false);
    if (top_p < 1.f) {
      const unsigned long long target = top_p > 0.f ? max(times_up(total, top_p), 1ull) : 1ull;
      scan_weights(sh, n, target - 1, true);
      n = sh.bin + 1;
      total = sh.total;
      __syncthreads();
    }
    if (threadIdx.x == 0) sh.limit = sh.all_place[n - 1];
    const unsigned long long goal = u >= 1.f ? total - 1 : times(total, u);
    __syncthreads();
    // in the order of their index: the place's lower half, inverted, falls with it
    for (int i = threadIdx.x; i < n; i += kThreads) sh.all_place[i] &= 0xffffffffu;
    __syncthreads();
    sort_list(sh, n);
    scan_weights(sh, n, goal, true);
    if (threadIdx.x == 0) {
      *token = (int32_t) ~(uint32_t)sh.all_place[sh.bin];
      sh.total = total;
    }
  }
  return true;
}

// Where the kept elements end: the place of the last of them.  True where the chunks' kept masses, and this thread's in
// kept_here, are known with it.
template <typename T>
__device__ bool find_limits(Row<T>& r, const Scale& sc, int top_k, float top_p, unsigned long long& limit,
                            unsigned long long& kept_here) {
  Shared& sh = r.sh;
  for (int b = threadIdx.x; b < kBins; b += kThreads) sh.count[b] = 0, sh.mass[b] = 0;
  __syncthreads();
  auto kept = [&](float x, float y) { return min_p_leaves(sc, sh, x, y); };
  r.each([&](float x, int) {
    const float y = sc.log2w(x);
    if (!kept(x, y)) return;
    const int b = bin_of(y);
    atomicAdd(&sh.count[b], 1u);
    atomicAdd(&sh.mass[b], (uint32_t)__float2int_rn(exp2_approx(y + (float)(b / kPerOctave)) * 16384.f));
  });
  r.template share_bins<true>();
  const int unit_bits = r.cluster.num_blocks() > 1 ? 29 + 3 : 29;  // 2^-14 in the weights' unit

  int last_bin = kBins - 1;
  if (top_k > 0) {
    const int bin = r.template find_bin<false>(top_k, last_bin, 0);
    if (bin >= 0) {  // else there are no more than top_k
      unsigned long long above = 0, lo = 0, hi = ~0ull, in_range = sh.count[bin];
      {
        unsigned long long a = 0, zero = 0;
        for (int b = threadIdx.x; b < bin; b += kThreads) a += sh.count[b];
        // the same in every CTA: no need to ask the others
        a = warp_sum(a);
        __syncthreads();
        if (threadIdx.x % 32 == 0) sh.warp_sums[threadIdx.x / 32][0] = a;
        __syncthreads();
        for (int k = 0; k < kWarps; ++k) zero += sh.warp_sums[k][0];
        above = zero;
        __syncthreads();
      }
      if (in_range > kList) r.range_of(sc, bin, 0, lo, hi, kept);
      while (in_range > kList) {  // many equal or nearly equal logits: halve the range of places
        const unsigned long long mid = lo + (hi - lo) / 2 + 1;
        unsigned long long n = 0, none = 0;
        r.each([&](float x, int i) {
          const float y = sc.log2w(x);
          if (bin_of(y) != bin || !kept(x, y)) return;
          const unsigned long long at = place(x, i);
          n += at >= mid && at <= hi;
        });
        r.template reduce<false>(n, none);
        if (above + n >= (unsigned)top_k) lo = mid, in_range = n;
        else hi = mid - 1, above += n, in_range -= n;
      }
      const int n = r.gather(sc, bin, lo, hi, kept);
      sort_list(sh, n);
      limit = sh.all_place[top_k - 1 - above];
      last_bin = bin;
      __syncthreads();
    }
  }
  if (!(top_p < 1.f)) return false;

  // the bin by its mass, confirmed by exact sums
  const unsigned long long about = r.mass_above(last_bin + 1, unit_bits);
  int bin = r.template find_bin<true>(max(times_up(about, top_p), 1ull), last_bin, unit_bits);
  if (bin < 0) bin = r.next_bin(last_bin + 1, -1, last_bin);
  unsigned long long target = 0, above = 0, inside = 0, in_bin = 0;
  const int lane = threadIdx.x % 32;
  for (bool first = true;; first = false) {
    // mass above the bin (of every 256 elements, too), in it, and (the first time) behind it; the bin's elements
    __syncthreads();
    if (threadIdx.x == 0) sh.listed = 0;
    __syncthreads();
    unsigned long long a = 0, in = 0, behind = 0, n = 0;
    r.turns([&](const float (&x)[8], int i, int chunk) {
      unsigned long long mass = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float y = sc.log2w(x[k]);
        const int b = bin_of(y);
        if ((b > bin && !first) || !kept(x[k], y)) continue;
        if (limit && place(x[k], i + k) < limit) continue;
        const unsigned long long w = r.weight(sc, x[k]);
        if (b < bin) {
          mass += w;
        } else if (b > bin) {
          behind += w;
        } else {
          in += w;
          ++n;
          const uint32_t j = atomicAdd(&sh.listed, 1u);
          if (j < kList) sh.list_place[j] = place(x[k], i + k), sh.list_weight[j] = w;
        }
      }
      a += mass;
      mass = warp_sum(mass);
      if (lane == 0) sh.chunk[chunk] = mass;
    });
    kept_here = a;
    r.template reduce<false>(a, in);
    r.template reduce<false>(behind, n);
    above = a, inside = in, in_bin = n;
    if (first) target = top_p > 0.f ? max(times_up(above + inside + behind, top_p), 1ull) : 1ull;
    const bool low = above + inside < target;
    if (above < target && !low) break;
    // the first time, by how far the bins' masses were off here; then from bin to bin
    int b = -1;
    if (first) {
      const unsigned long long off = r.mass_above(bin, unit_bits) - above;  // of either sign
      b = r.template find_bin<true>(max(target + off, 1ull), last_bin, unit_bits);
    }
    if (b < 0 || (low ? b <= bin : b >= bin)) b = r.next_bin(bin, low ? 1 : -1, last_bin);
    if (b < 0) return false;  // all of them
    bin = b;
  }
  if (in_bin <= kList) {
    const int n = r.merge_lists();
    sort_list(sh, n);
    scan_weights(sh, n, target - above - 1, true);
    limit = sh.all_place[sh.bin];
    for (int k = threadIdx.x; k < min((int)sh.listed, kList); k += kThreads)
      if (sh.list_place[k] >= limit) {
        kept_here += sh.list_weight[k];
        atomicAdd(&sh.chunk[((int)~(uint32_t)sh.list_place[k] - r.v0) / kChunk], sh.list_weight[k]);
      }
    __syncthreads();
    return true;
  }
  // many equal or nearly equal logits: halve the range of places
  unsigned long long lo = limit, hi = ~0ull, in_range = in_bin;
  r.range_of(sc, bin, limit, lo, hi, kept);
  while (in_range > kList) {
    const unsigned long long mid = lo + (hi - lo) / 2 + 1;
    unsigned long long n = 0, w = 0;
    r.each([&](float x, int i) {
      const float y = sc.log2w(x);
      if (bin_of(y) != bin || !kept(x, y)) return;
      const unsigned long long at = place(x, i);
      if (at >= mid && at <= hi) n += 1, w += sc.weight(x, sh.powers);
    });
    r.template reduce<false>(n, w);
    if (above + w >= target) lo = mid, in_range = n;
    else hi = mid - 1, above += w, in_range -= n;
  }
  const int n = r.gather(sc, bin, lo, hi, kept);
  sort_list(sh, n);
  scan_weights(sh, n, target - above - 1, true);
  limit = sh.all_place[sh.bin];
  __syncthreads();
  return false;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) token_sample_kernel(const __grid_constant__ SampleParams p) {
  extern __shared__ __align__(16) unsigned char raw[];
  Shared& sh = *reinterpret_cast<Shared*>(raw);
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int64_t at = blockIdx.x / C;
  Row<T> r{p, sh, cluster, rank, 0};
  r.row = reinterpret_cast<const T*>(p.logits) + at * p.V;
  r.v0 = min(p.V, rank * p.slice);
  r.v1 = min(p.V, (rank + 1) * p.slice);
  r.wide = (uint64_t)p.V * sizeof(T) % 16 == 0;
  if (threadIdx.x < 64) sh.powers[threadIdx.x] = kPowers[threadIdx.x];
  if (threadIdx.x == 64) set_least(sh, p.min_p ? p.min_p[at] : 0.f);

  float temp = p.temperature ? p.temperature[at] : 1.f;
  int top_k = p.top_k ? p.top_k[at] : 0;
  float top_p = p.top_p ? p.top_p[at] : 1.f;
  const float min_p = p.min_p ? p.min_p[at] : 0.f;
  float u = p.u[at];
  const bool bad_temp = !(temp >= 0.f && temp < INFINITY);
  if (!(top_p > 0.f)) top_p = top_p <= 0.f ? 0.f : 1.f;  // NaN: no limit

  // the largest logit, and whether the row has a distribution
  float mine = -INFINITY;  // this thread's largest
  unsigned long long best, odd;
  {
    bool bad = false;
    r.each([&](float x, int) {
      bad |= !(x < INFINITY);
      mine = fmaxf(mine, x);
    });
    best = place(mine, 0) >> 32, odd = bad;
  }
  r.template reduce<true>(best, odd);
  const uint32_t key = (uint32_t)best;
  const float m = __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
  float* probs = p.probs ? p.probs + at * p.V : nullptr;
  if (odd || bad_temp || !(m > -INFINITY)) {
    if (rank == 0 && threadIdx.x == 0) {
      p.tokens[at] = -1;
      if (bad_temp && p.status) atomicOr(p.status, TV_DEV_BAD_PARAM);
    }
    if (probs)
      for (int i = r.v0 + threadIdx.x; i < r.v1; i += kThreads) probs[i] = NAN;
  } else if (temp < kCold || top_k == 1) {  // the likeliest alone
    unsigned long long first = 0, none = 0;
    r.each([&](float x, int i) {
      if (x == m) first = max(first, (unsigned long long)(uint32_t)~i);
    });
    r.template reduce<true>(first, none);
    const int best_i = (int)~(uint32_t)first;
    if (rank == 0 && threadIdx.x == 0) p.tokens[at] = best_i;
    if (probs)
      for (int i = r.v0 + threadIdx.x; i < r.v1; i += kThreads) probs[i] = i == best_i ? 1.f : 0.f;
  } else {
    Scale sc;
    const double c = 1.4426950408889634074 / (double)fminf(temp, 1.f / kCold);
    sc.m = m;
    sc.c1 = (float)c;
    sc.c2 = (float)(c - (double)sc.c1);
    sc.floor_y = floor_of(min_p);
    if (top_k < 0 || top_k >= p.V) top_k = 0;
    unsigned long long limit = 0;
    // Few candidates: those above a bar that top_k of the threads' largest elements reach.
    int bar = kBins - 1;
    if (top_k > 0 && top_k <= 128 * C) {
      for (int b = threadIdx.x; b < kBins; b += kThreads) sh.count[b] = 0;
      __syncthreads();
      if (mine > -INFINITY) atomicAdd(&sh.count[bin_of(sc.log2w(mine))], 1u);
      r.template share_bins<false>();
      const int b = r.template find_bin<false>(top_k, kBins - 1, 0);
      if (b >= 0) bar = b;
    }
    if (bar < kBins - 1 && sample_sorted(r, sc, bar, top_k, top_p, u, p.tokens + at)) {
      cluster.sync();
      if (probs) {
        limit = *cluster.map_shared_rank(&sh.limit, 0);
        const float inv = (float)(0x1p43 / (double)*cluster.map_shared_rank(&sh.total, 0));
        r.each([&](float x, int i) {
          const float y = sc.log2w(x);
          const bool in = y >= sc.floor_y && place(x, i) >= limit && min_p_leaves(sc, sh, x, y);
          if (i < r.v1) probs[i] = in ? sc.probability(x, sh.powers) * inv : 0.f;
        });
      }
      cluster.sync();
      return;
    }
    r.fill_table(sc);
    bool known = false;
    unsigned long long total = 0, none = 0, before = 0;
    if (top_k > 0 || top_p < 1.f) known = find_limits(r, sc, top_k, top_p, limit, total);

    // kept mass of every 256 elements
    auto kept_weight = [&](float x, int i) -> unsigned long long {
      const float y = sc.log2w(x);
      return y >= sc.floor_y && place(x, i) >= limit && min_p_leaves(sc, sh, x, y) ? r.weight(sc, x) : 0;
    };
    const int lane = threadIdx.x % 32;
    if (!known) total = 0;
    if (!known)
      r.turns([&](const float (&x)[8], int i, int chunk) {
        unsigned long long w = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) w += kept_weight(x[k], i + k);
        total += w;
        w = warp_sum(w);
        if (lane == 0) sh.chunk[chunk] = w;
      });
    r.template reduce<false>(total, none, &before);
    // the draw: in the CTA that u W falls into, by one warp
    const unsigned long long goal = u >= 1.f ? total - 1 : times(total, u);
    if (threadIdx.x < 32 && goal >= before) {
      const int chunks = (r.v1 - r.v0 + kChunk - 1) / kChunk;
      unsigned long long run = before;
      int hit = -1;
      for (int c0 = 0; c0 < chunks && hit < 0; c0 += 32) {
        const unsigned long long w = c0 + lane < chunks ? sh.chunk[c0 + lane] : 0;
        unsigned long long s = w;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
          const unsigned long long y = __shfl_up_sync(0xffffffffu, s, o);
          if (lane >= o) s += y;
        }
        const unsigned over = __ballot_sync(0xffffffffu, run + s > goal);
        if (over) {
          const int k = __ffs(over) - 1;
          hit = c0 + k;
          run += __shfl_sync(0xffffffffu, s - w, k);
        } else {
          run += __shfl_sync(0xffffffffu, s, 31);
        }
      }
      if (hit >= 0) {
        const int i = r.v0 + hit * kChunk + lane * 8;
        float x[8];
        unsigned long long w[8], mine = 0;
        r.unpack(r.load(i), x);
#pragma unroll
        for (int k = 0; k < 8; ++k) w[k] = kept_weight(x[k], i + k), mine += w[k];
        unsigned long long s = mine;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
          const unsigned long long y = __shfl_up_sync(0xffffffffu, s, o);
          if (lane >= o) s += y;
        }
        const unsigned over = __ballot_sync(0xffffffffu, run + s > goal);
        if (over && lane == __ffs(over) - 1) {
          run += s - mine;
          int tok = -1;
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            run += w[k];
            if (tok < 0 && run > goal) tok = i + k;
          }
          p.tokens[at] = tok;
        }
      }
    }
    if (probs) {
      const float inv = (float)(0x1p43 / (double)total);
      r.each([&](float x, int i) {
        const float y = sc.log2w(x);
        const bool in = y >= sc.floor_y && place(x, i) >= limit && min_p_leaves(sc, sh, x, y);
        if (i < r.v1) probs[i] = in ? sc.probability(x, sh.powers) * inv : 0.f;
      });
    }
  }
  cluster.sync();  // the others may still read this CTA's numbers
}

template <typename T>
int launch_sample(SampleParams p, int sm_count, cudaStream_t stream) {
  // CTAs of a row: up to 4 where two waves hold all rows (two CTAs an SM), of 4096 elements at least; more only for what
  // 4 cannot hold.  64 rows of 32,000 float32 with top-p: 44 us by 4, 73 by 8, 54 by 2 (an exchange between CTAs takes
  // longer the more they are); 256 rows of 128,000 bf16: 154 us by 2, 204 by one.
  int C = 1;
  while (C < kMaxCluster && ((int64_t)p.V > (int64_t)C * (kMaxV / kMaxCluster) ||
                             (C < 4 && p.R * C <= 2ll * sm_count && p.V > C * 4096)))
    C *= 2;
  p.slice = (int)(tv::ceil_div(p.V, (int64_t)C * kChunk) * kChunk);
  const int smem = (int)sizeof(Shared);
  cudaError_t e = cudaFuncSetAttribute(token_sample_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return tv::cuda_fail(e, "cudaFuncSetAttribute(token_sample_kernel)");
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.R * C), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = C;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, token_sample_kernel<T>, p);
  if (e != cudaSuccess) return tv::cuda_fail(e, "token_sample_kernel");
  return TV_OK;
}

}  // namespace

extern "C" int tv_token_sample(const void* logits, int64_t R, int32_t V, int32_t dtype, const float* temperature,
                               const int32_t* top_k, const float* top_p, const float* min_p, const float* u,
                               int32_t* tokens, float* probs, int32_t* status, void* stream) {
  tv::clear_error();
  if (R < 0 || V < 1) return tv::fail(TV_ERR_INVALID_ARG, "tv_token_sample: bad sizes");
  if (dtype != TV_F32 && dtype != TV_BF16) return tv::fail(TV_ERR_UNSUPPORTED, "tv_token_sample: dtype %d", dtype);
  if (V > kMaxV) return tv::fail(TV_ERR_UNSUPPORTED, "tv_token_sample: V %d exceeds %d", V, kMaxV);
  if (R > INT32_MAX / kMaxCluster) return tv::fail(TV_ERR_UNSUPPORTED, "tv_token_sample: more than 2^28 rows");
  if (R == 0) return TV_OK;
  if (!logits || !u || !tokens) return tv::fail(TV_ERR_INVALID_ARG, "tv_token_sample: null pointer");
  if ((reinterpret_cast<uintptr_t>(logits) | reinterpret_cast<uintptr_t>(probs)) & 15)
    return tv::fail(TV_ERR_INVALID_ARG, "tv_token_sample: logits and probs must be 16-byte aligned");
  tv::DeviceInfo dev;
  if (int rc = tv::current_device_info(&dev)) return rc;
  SampleParams p{};
  p.logits = static_cast<const char*>(logits);
  p.R = R;
  p.V = V;
  p.temperature = temperature;
  p.top_k = top_k;
  p.top_p = top_p;
  p.min_p = min_p;
  p.u = u;
  p.tokens = tokens;
  p.probs = probs;
  p.status = status;
  cudaStream_t s = (cudaStream_t)stream;
  return dtype == TV_BF16 ? launch_sample<__nv_bfloat16>(p, dev.sm_count, s) : launch_sample<float>(p, dev.sm_count, s);
}
