// Attention of a chunk of new tokens over the paged cache on the
// 5th-generation tensor cores (tcgen05 + TMEM + TMA); chunk.cu has the
// definition.
//
// * Rows: the G query heads of one KV head and floor(128 / G) tokens fill a
//   128-row M tile (row = token * G + head, so rows of one token are
//   neighbours); a unit is two M tiles of one (request, KV head), so a K/V byte
//   that reaches the SM feeds 256 rows.  Q comes by one TMA box per 64 columns.
// * Keys: tiles of 64, K and V in rings of their own, by TMA boxes of (a power
//   of two of) rows within a cache block.  Boxes without a
//   key that the unit sees, and bad blocks, are sent out of bounds: zeros.
// * S_m = Q_m K^T (128 x 64, both operands from shared memory) and O_m += P_m V
//   (P_m from TMEM, bf16, over S_m's columns), issued by a thread each.  Each M
//   tile has two S buffers, so the products of the next tile and of the other M
//   tile run while a tile's softmax does.  (One S buffer, freed once it is in
//   registers, and two for P: 6.0 against 5.7 ms.)
//   S_0 2 x 64 | S_1 2 x 64 | O_0 128 | O_1 128 columns fill the TMEM; with heads
//   of 256 a unit is one M tile, S 2 x 64 | O 256 (4 x 512 tokens, 16/4 heads: 58
//   us, 516 on CUDA cores; the softmax warps spill 44-66 bytes there).
// * Softmax: a thread per row, against a reference that is the first tile's
//   maximum and moves, with O rescaled in TMEM, only when weights pass 2^20; so
//   later tiles need no maximum at all (it took a third of a tile's time).  Weights are rounded to bf16 for
//   P V (an operand of kind::f16 holds no more; half a step, 2^-8 of a weight at
//   most, as much as rounding the output takes), their sum is not.  A second bf16
//   part, as tv_decode_attn has it, would double P V and its reads of V.
// * Work: the units' tiles (with a few virtual ones for a unit's fixed cost) lie
//   end to end and each CTA of a persistent grid takes an equal run.  The sums
//   over a request's units have a closed form (tiles_below), so a CTA finds its
//   run from lengths and offsets alone.  A unit cut by a run's end leaves
//   (max, sum, output) of each piece in the workspace and the CTA whose piece
//   arrives last joins them in order, so results do not depend on timing.
//
// Bound by shared memory and the chain of a tile (scores, softmax, outputs, next
// scores: 1630 cycles, of which the operands' 160 KB take 1250): 8192 tokens
// behind 24576, 64/8 heads of 128, 5.5-5.6 ms, 0.73-0.75 of the measured bf16
// rate; by what a unit costs beside its tiles (about four of them) for prompts of
// a few hundred tokens (32 of 1-1023 tokens: 179 us, 0.29).
//
// Every mbarrier wait is bounded (2 s); past it the CTA sets TV_DEV_TIMEOUT, lets
// its products and loads finish, frees its TMEM and returns.
#include <cuda_bf16.h>

#include <algorithm>
#include <mutex>
#include <type_traits>

#include "attn_score.cuh"
#include "chunk.h"
#include "tc_ptx.cuh"

namespace tv {

namespace {

constexpr int kBlk = 64;           // keys of a tile
constexpr int kQHalf = 128 * 128;  // bytes of 64 columns of a Q tile
constexpr int kHalf = kBlk * 128;  // ... of a K or V tile
constexpr int kThreads = 512;
constexpr unsigned long long kLimitNs = 2000000000ull;
constexpr float kMost = 0x1p20f;   // sum of a row's weights in a tile before its reference moves

template <int D>
struct Cfg {
  static constexpr int kM = D == 256 ? 1 : 2;      // M tiles of a unit: two of 256 columns do not fit the TMEM
  static constexpr int kQTile = D / 64 * kQHalf;
  static constexpr int kTile = D / 64 * kHalf;     // bytes of a K or V tile
  static constexpr int kSlots = D == 64 ? 8 : D == 128 ? 4 : 2;  // of K, and of V
  static constexpr int kOffK = kM * kQTile;        // behind Q_0, Q_1
  static constexpr int kOffV = kOffK + kSlots * kTile;
  static constexpr int kOffOut = kOffV + kSlots * kTile;  // 4 KB a softmax warp: 32 rows of 64 output columns
  static constexpr int kSmem = kOffOut + 8 * 4096 + 1024;
};
static_assert(Cfg<64>::kSmem <= 227 * 1024 - 1024 && Cfg<128>::kSmem <= 227 * 1024 - 1024 &&
                  Cfg<256>::kSmem <= 227 * 1024 - 1024,
              "fits beside the barriers");

__host__ __device__ constexpr uint32_t kColS(int m, uint32_t tile) { return m * 128 + (tile & 1) * 64; }
constexpr uint32_t kColO(int m) { return 256 + m * 128; }

struct Bars {
  uint64_t full[2][8], empty[2][8];  // of K, of V
  uint64_t q_full[2], q_free[2], s_full[2][2], p_full[2][2], pv_done[2][2], v_seen[2], drain[4];
  uint64_t posted, decided;
  uint32_t tmem;
  int abort;
  int last;
};

struct Maps {
  CUtensorMap k, v, q;
  CUtensorMap out;  // boxes of a warp's 32 rows x 64 columns
  int out_tokens;   // of such a box, 0: the group does not fit one and rows are stored directly
};

#ifdef TV_TEST_HOOKS
// Development builds only: a shorter wait limit, and a ring entry of CTA 0 that is left without its loads.
__device__ unsigned long long g_chunk_limit_ns = kLimitNs;
__device__ int g_chunk_withhold = -1;
__device__ __forceinline__ unsigned long long limit_ns() { return *(volatile unsigned long long*)&g_chunk_limit_ns; }
__device__ __forceinline__ bool withhold(uint32_t n) { return blockIdx.x == 0 && (int)n == *(volatile int*)&g_chunk_withhold; }
#else
__device__ __forceinline__ unsigned long long limit_ns() { return kLimitNs; }
__device__ __forceinline__ bool withhold(uint32_t) { return false; }
#endif

// ---------------------------------------------------------------- the plan

// The residues of a step's multiples: a k mod 64 repeats after 64 / gcd(a, 64) turns, a power of two.
struct Residues {
  uint16_t sum[kBlk + 1];  // of the first i of them, up to a period
  uint8_t log_gcd, log_period;
  uint8_t inverse;         // of a / gcd(a, 64) modulo the period
};

Residues residues_of(int a) {
  Residues r{};
  while (r.log_gcd < 6 && a % (2 << r.log_gcd) == 0) ++r.log_gcd;
  r.log_period = 6 - r.log_gcd;
  const int period = 1 << r.log_period;
  for (int k = 0; k < period; ++k) {
    r.sum[k + 1] = r.sum[k] + a * k % kBlk;
    if ((a >> r.log_gcd) * k % period == 1 % period) r.inverse = k;
  }
  return r;
}

// sum over j < n of max(0, floor((b + a j) / 64)), a >= 1: the terms' own sum without their residues'.  With b = 64 .. + g i
// + rest, g = gcd(a, 64), the residues are rest + (a (k + j) mod 64), k = i times the inverse: a run of the table.
__device__ int64_t tiles_below(int64_t n, int a, int64_t b, const Residues& r) {
  if (n <= 0) return 0;
  if (b < 0) {
    const int64_t skip = (-b + a - 1) / a;
    if (skip >= n) return 0;
    n -= skip;
    b += skip * a;
  }
  const int period = 1 << r.log_period, first = (int)(b % kBlk);
  const int k = (first >> r.log_gcd) * r.inverse & (period - 1), end = k + (int)(n & (period - 1));
  const int run = r.sum[min(end, period)] + r.sum[max(0, end - period)] - r.sum[k];
  const int64_t residues = n * (first & ((1 << r.log_gcd) - 1)) + (n >> r.log_period) * r.sum[period] + run;
  return (n * b + n * (n - 1) / 2 * a - residues) / kBlk;
}

// One request's units.
struct Request {
  ChunkOf c;
  int units;   // per KV head
  int step;    // tokens of a unit
  int window, sinks;  // sinks: tiles of kept first keys

  __device__ __forceinline__ void set(const ChunkParams& p, int b) {
    step = p.m_tiles * (128 / p.G);
    chunk_of(p, b, c);
    units = (c.n + step - 1) / step;
    window = p.window;
    sinks = window > 0 ? (int)(((int64_t)p.n_sink + kBlk - 1) / kBlk) : 0;
  }
  // Tiles of unit i (one at least): up to its last position, without those between the kept first keys and the window.
  __device__ __forceinline__ int tiles(int i) const {
    const int first = c.first + i * step, last = c.first + min((i + 1) * step, c.n) - 1;
    const int skipped = window > 0 ? max(0, max(0, max(0, first + 1) - window) / kBlk - sinks) : 0;
    return 1 + max(0, last) / kBlk - skipped;
  }
  // Tiles (and virtual ones) of the units before i, i < units
  __device__ __forceinline__ int64_t before(int i, int cost, const Residues& r) const {
    int64_t n = (int64_t)i * (1 + cost) + tiles_below(i, step, (int64_t)c.first + step - 1, r);
    if (window > 0) n -= tiles_below(i, step, (int64_t)c.first + 1 - window - (int64_t)sinks * kBlk, r);
    return n;
  }
  __device__ __forceinline__ int64_t all(int cost, const Residues& r) const {
    return units ? before(units - 1, cost, r) + tiles(units - 1) + cost : 0;
  }
};

struct Plan {
  int64_t x0, x1, total;  // this CTA's run of [0, total)
  int ctas;               // that take part
  int whole;              // a unit of this length or less is not cut: it goes to the CTA whose run it starts in
  int b, i, kvh;          // the unit that x0 is in
  int64_t at;             // where it starts
};

// a / b, a >= 0, b > 0, without a division of 64 bits where 32 do
__device__ __forceinline__ int64_t divide(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}
__device__ __forceinline__ int64_t run_start(int64_t c, int64_t total, int64_t ctas) { return divide(c * total, ctas); }
__device__ __forceinline__ int64_t run_of(int64_t x, int64_t total, int64_t ctas) { return divide((x + 1) * ctas - 1, total); }

// All threads of the CTA.
__device__ void make_plan(const ChunkParams& p, const Residues& res, int cost, int least, float join_cost, Plan& plan) {
  __shared__ int64_t sums[kThreads / 32 + 1];
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int per = (p.B + kThreads - 1) / kThreads;
  const int b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
  int64_t mine = 0;
  for (int b = b0; b < b1; ++b) {
    Request r;
    r.set(p, b);
    mine += r.all(cost, res);
  }
  mine *= p.Hkv;
  int64_t run = mine;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const int64_t y = __shfl_up_sync(0xffffffffu, run, o);
    if (lane >= o) run += y;
  }
  if (lane == 31) sums[warp] = run;
  if (tid == 0) plan.b = -1;
  __syncthreads();
  int64_t total = 0, start = run - mine;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) start += sums[w];
    total += sums[w];
  }
  // n pieces of a unit of U tiles take U / n tiles, and n pieces' join in one CTA: least for runs of sqrt(U join_cost)
  // (64 tokens over 8000: 74 us over all CTAs, 61 this way)
  least = max(least, (int)sqrtf((float)total * join_cost));
  const int ctas = (int)min((int64_t)p.ctas, max((int64_t)1, divide(total, least)));
  const int c = blockIdx.x;
  const int64_t x0 = c < ctas ? run_start(c, total, ctas) : total;
  const int64_t x1 = c < ctas ? run_start(c + 1, total, ctas) : total;
  if (x0 < x1 && x0 >= start && x0 < start + mine) {  // one thread: its requests hold the run's start
    int b = b0;
    Request r;
    int64_t at = start;
    for (;; ++b) {
      r.set(p, b);
      const int64_t n = r.all(cost, res) * p.Hkv;
      if (x0 < at + n) break;
      at += n;
    }
    int lo = 0;  // the last unit that starts at or before x0
    for (int hi = r.units; hi - lo > 1;) {
      const int mid = lo + (hi - lo) / 2;
      if (at + r.before(mid, cost, res) * p.Hkv <= x0) lo = mid; else hi = mid;
    }
    at += r.before(lo, cost, res) * p.Hkv;
    const int one = r.tiles(lo) + cost;
    plan.kvh = (int)divide(x0 - at, one);
    plan.at = at + (int64_t)plan.kvh * one;
    plan.b = b;
    plan.i = lo;
  }
  if (tid == 0) {
    plan.x0 = x0;
    plan.x1 = x1;
    plan.total = total;
    plan.ctas = ctas;
    // A cut costs about 15 tiles (the pieces written and read back, the wait for the last), an uneven run up to one unit, a
    // quarter of a run at most.  With units up to 0 | 12 | 24 | 48 tiles whole: 32 prompts of 1-1023 tokens 207 | 192 | 180 |
    // 180 us, 64 x 256 tokens with heads of 64 104 | 85 | 85 | 85, 8 x 1000 tokens 116 | 116 | 95 | 95.
    plan.whole = (int)min((int64_t)24, divide(total, ctas) / 4);
  }
  __syncthreads();
}

// A CTA's part of one unit: tiles [a, e) of it.
struct Piece {
  int b, kvh, s0;      // packed row of the unit's first token
  int tokens[2];       // of the M tiles
  int pos0, last;      // positions of the unit's first and last token
  int lo;              // first key of the window of the first token
  int sink;            // keys below it stay visible
  int lead;            // tiles before the window's
  int count[2];        // tiles that an M tile's rows see
  int a, e, tiles;
  int64_t real;        // where its tiles start in [0, total)

  __device__ __forceinline__ int key(int t) const { return (t < lead ? t : lo / kBlk + t - lead) * kBlk; }
  // tiles of this part that M tile m computes
  __device__ __forceinline__ int computed(int m) const { return max(0, min(e, count[m]) - a); }
  // V of a tile at t0 holds keys that no row of the unit sees
  __device__ __forceinline__ bool ragged(int t0) const { return t0 + kBlk - 1 > last || t0 < lo; }
  __device__ __forceinline__ bool split() const { return a > 0 || e < tiles; }
};

struct Walk {
  const ChunkParams& p;
  const Plan& plan;
  int cost, b, i, kvh;
  int64_t at;
  Request r;
  bool fresh = true;  // a new unit's tokens

  __device__ __forceinline__ Walk(const ChunkParams& p_, const Plan& plan_, int cost_)
      : p(p_), plan(plan_), cost(cost_), b(plan_.b), i(plan_.i), kvh(plan_.kvh), at(plan_.at) {
    r.set(p, b);
  }
  // The next part with tiles in this CTA's run; false at its end.  s is the last one, from which the next KV head's differs
  // little (code that runs once a unit is fetched anew each time: the whole of this took 2000 cycles a unit).
  __device__ __forceinline__ bool next(Piece& s) {
    while (at < plan.x1) {
      if (fresh) {
        const int j0 = i * r.step, n = min(r.step, r.c.n - j0), half = 128 / p.G;
        s.b = b;
        s.s0 = r.c.s0 + j0;
        s.tokens[0] = min(n, half);
        s.tokens[1] = max(0, n - half);
        s.pos0 = r.c.first + j0;
        s.last = s.pos0 + n - 1;
        s.lo = p.window > 0 ? max(0, max(0, s.pos0 + 1) - p.window) : 0;
        s.sink = min(p.n_sink, s.lo);
        s.lead = min((s.sink + kBlk - 1) / kBlk, s.lo / kBlk);
        s.tiles = r.tiles(i);
        const int last0 = s.pos0 + s.tokens[0] - 1;
        s.count[0] = last0 < 0 ? 1 : s.lead + last0 / kBlk + 1 - s.lo / kBlk;
        s.count[1] = s.tokens[1] > 0 ? s.tiles : 0;
        fresh = false;
      }
      s.kvh = kvh;
      s.real = at + cost;
      int64_t a = max((int64_t)0, plan.x0 - s.real), e = min((int64_t)s.tiles, plan.x1 - s.real);
      if (s.tiles + cost <= plan.whole) {
        a = 0;
        e = at >= plan.x0 ? s.tiles : 0;  // at < x1 here
      }
      s.a = (int)a;
      s.e = (int)e;
      at += s.tiles + cost;
      if (++kvh == p.Hkv) {
        kvh = 0;
        fresh = true;
        if (++i == r.units) {
          i = 0;
          if (at < plan.x1)
            do r.set(p, ++b); while (r.units == 0);
        }
      }
      if (a < e) return true;
    }
    return false;
  }
};

// ---------------------------------------------------------------- roles

// K boxes (warps 0, 1) or V boxes (warps 2, 3) of every tile.
template <int D>
__device__ __forceinline__ void run_producer(const ChunkParams& p, const Plan& plan, int cost, const Maps& maps, Bars& bars,
                                             uint32_t base, int warp, int lane) {
  using C = Cfg<D>;
  const int v = warp / 2;
  const int bs = p.block_size, br = min(kBlk, bs & -bs);
  const int sub_n = kBlk / br;
  const int j = lane * 2 + (warp & 1);  // box: sub-block j / halves, column half j % halves
  const int sub = j / (D / 64), h = j % (D / 64);
  const bool has_box = sub < sub_n;
  const int64_t rows_total = p.num_blocks * p.Hkv * bs;
  const CUtensorMap* map = v ? &maps.v : &maps.k;
  const uint32_t dst0 = base + (v ? C::kOffV : C::kOffK) + h * kHalf + sub * br * 128;
  uint32_t g = 0;  // tiles so far
  bool ok = true;
  Walk walk(p, plan, cost);
  Piece s;
  while (ok && walk.next(s)) {
    const int32_t* trow = p.table + (int64_t)s.b * p.max_blocks;
    // where this lane's box of tile t comes from: the first row, or past the end for zeros
    auto row_of = [&](int t) -> int {
      const int pos = s.key(t) + sub * br;
      if (!has_box || !(pos <= s.last && (pos + br > s.lo || pos < s.sink))) return (int)rows_total;
      const int col = pos / bs;
      const int64_t blk = __ldg(trow + col);
      if (blk < 0 || blk >= p.num_blocks) {
        if (p.status) atomicOr(p.status, TV_DEV_BAD_BLOCK);
        return (int)rows_total;
      }
      return (int)((blk * p.Hkv + s.kvh) * bs + (pos - col * bs));
    };
    int row = row_of(s.a);
    for (int t = s.a; t < s.e; ++t, ++g) {
      const int now = row;
      if (t + 1 < s.e) row = row_of(t + 1);
      const uint32_t slot = g % C::kSlots, use = g / C::kSlots;
      if (use > 0) ok = mbar_wait_warp(&bars.empty[v][slot], (use - 1) & 1, &bars.abort, p.status, limit_ns());
      if (!ok) break;
      if (withhold(2 * g + v)) continue;
      if ((warp & 1) == 0 && lane == 0) mbar_expect_tx(&bars.full[v][slot], C::kTile);
      __syncwarp();
      if (has_box) tma_2d(dst0 + slot * C::kTile, map, h * 64, now, &bars.full[v][slot]);
      __syncwarp();
    }
  }
  // what was asked for lands before the CTA ends
  if (!ok && lane == 0)
    for (uint32_t i = g > C::kSlots ? g - C::kSlots : 0; i < g; ++i)
      mbar_wait(&bars.full[v][i % C::kSlots], (i / C::kSlots) & 1, &bars.abort, nullptr, limit_ns(), false);
}

// The end of an issuing thread: nothing that it asked for still runs, or arrives, when the CTA frees its TMEM and ends.
__device__ __forceinline__ void drain(Bars& bars, int i) {
  mma_commit(&bars.drain[i]);
  mbar_wait(&bars.drain[i], 0, &bars.abort, nullptr, limit_ns(), false);
}

// A slot is released by both M tiles, by a commit behind the products that read it or, where none do, by an arrival once
// it has landed: so every waiting thread sees every phase of its barriers, and parities tell them apart.

// Loads M tile m's Q of each unit, once the unit before it has no more products with its own, and issues S = Q K^T of
// its tiles.  Tile j takes the columns of tile j - 2, whose P V has to be done.
template <int D>
__device__ __forceinline__ void issue_scores(const ChunkParams& p, const Plan& plan, int cost, const Maps& maps, Bars& bars,
                                             uint32_t base, uint32_t tmem, int m) {
  using C = Cfg<D>;
  constexpr uint32_t id = idesc_bf16(128, kBlk, false);
  constexpr uint32_t hi = desc_hi(1024);
  const uint32_t sQ = base + m * C::kQTile;
  const uint32_t q_lo = desc_lo(sQ, 0);
  uint32_t g = 0, units = 0, n_s = 0;  // ring's tiles, this M tile's units and tiles
  bool ok = true;
  Walk walk(p, plan, cost);
  Piece s;
  auto wait = [&](uint64_t* bar, uint32_t parity) { return mbar_wait(bar, parity, &bars.abort, p.status, limit_ns()); };
  while (ok && walk.next(s)) {
    const int n_mine = s.computed(m);
    if (n_mine > 0) {
      if (units > 0) ok = wait(&bars.q_free[m], (units - 1) & 1);
      if (!ok) break;
      mbar_expect_tx(&bars.q_full[m], D / 64 * p.G * (128 / p.G) * 128);
#pragma unroll
      for (int h = 0; h < D / 64; ++h)
        tma_3d(sQ + h * kQHalf, &maps.q, h * 64, s.kvh * p.G, s.s0 + m * (128 / p.G), &bars.q_full[m]);
      ++units;
      ok = wait(&bars.q_full[m], (units - 1) & 1);
    }
    for (int k = 0; ok && k < s.e - s.a; ++k, ++g) {
      const uint32_t slot = g % C::kSlots;
      ok = wait(&bars.full[0][slot], (g / C::kSlots) & 1);
      if (!ok) break;
      if (k >= n_mine) {
        mbar_arrive(&bars.empty[0][slot]);
        continue;
      }
      if (n_s >= 2) ok = wait(&bars.pv_done[m][n_s & 1], ((n_s - 2) >> 1) & 1);
      if (!ok) break;
      fence_after();
      const uint32_t k_lo = desc_lo(base + C::kOffK + slot * C::kTile, 0);
      const uint32_t dS = tmem + kColS(m, n_s);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t in = (kk % 4) * 2;  // 16 columns further in a 64-column half
        mma_bf16(dS, (uint64_t)hi << 32 | (q_lo + (kk / 4) * (kQHalf >> 4) + in),
                 (uint64_t)hi << 32 | (k_lo + (kk / 4) * (kHalf >> 4) + in), id, kk > 0);
      }
      mma_commit(&bars.s_full[m][n_s & 1]);
      mma_commit(&bars.empty[0][slot]);
      if (k == 0 && s.kvh + 1 < p.Hkv) {  // the next unit's Q, most likely, on its way to L2
#pragma unroll
        for (int h = 0; h < D / 64; ++h)
          tma_prefetch_3d(&maps.q, h * 64, (s.kvh + 1) * p.G, s.s0 + m * (128 / p.G));
      }
      if (k == n_mine - 1) mma_commit(&bars.q_free[m]);
      ++n_s;
    }
  }
  if (units) mbar_wait(&bars.q_full[m], (units - 1) & 1, &bars.abort, nullptr, limit_ns(), false);  // no load is left
  drain(bars, m);
}

// Issues O_m += P_m V of its tiles.
template <int D>
__device__ __forceinline__ void issue_outputs(const ChunkParams& p, const Plan& plan, int cost, Bars& bars, uint32_t base,
                                              uint32_t tmem, int m) {
  using C = Cfg<D>;
  constexpr uint32_t id = idesc_bf16(128, D, true);
  constexpr uint32_t hi = desc_hi(1024);
  const uint32_t dO = tmem + kColO(m);
  uint32_t g = 0, n_pv = 0;  // ring's tiles, this M tile's tiles
  bool ok = true;
  Walk walk(p, plan, cost);
  Piece s;
  auto wait = [&](uint64_t* bar, uint32_t parity) { return mbar_wait(bar, parity, &bars.abort, p.status, limit_ns()); };
  while (ok && walk.next(s)) {
    const int n_mine = s.computed(m);
    for (int k = 0; ok && k < s.e - s.a; ++k, ++g) {
      const uint32_t slot = g % C::kSlots;
      ok = wait(&bars.full[1][slot], (g / C::kSlots) & 1);
      if (!ok) break;
      if (k >= n_mine) {
        mbar_arrive(&bars.empty[1][slot]);
        continue;
      }
      if (s.ragged(s.key(s.a + k))) mbar_arrive(&bars.v_seen[m]);  // the softmax threads clear those keys
      ok = wait(&bars.p_full[m][n_pv & 1], (n_pv >> 1) & 1);
      if (!ok) break;
      fence_after();
      const uint32_t aP = tmem + kColS(m, n_pv);
      const uint32_t lo = desc_lo(base + C::kOffV + slot * C::kTile, kHalf);  // MN-major V: the next 64 columns
      if (k > 0) mma_ts<true>(dO, aP, lo, hi, id);
      else mma_ts<false>(dO, aP, lo, hi, id);
#pragma unroll
      for (int kk = 1; kk < kBlk / 16; ++kk) mma_ts<true>(dO, aP + kk * 8, lo + kk * (2048 >> 4), hi, id);
      mma_commit(&bars.pv_done[m][n_pv & 1]);
      mma_commit(&bars.empty[1][slot]);
      ++n_pv;
    }
  }
  drain(bars, 2 + m);
}

__device__ __forceinline__ float max64(const float (&v)[64]) {
  float a[22];
#pragma unroll
  for (int i = 0; i < 21; ++i) a[i] = max3(v[3 * i], v[3 * i + 1], v[3 * i + 2]);
  a[21] = v[63];
  float b[8];
#pragma unroll
  for (int i = 0; i < 7; ++i) b[i] = max3(a[3 * i], a[3 * i + 1], a[3 * i + 2]);
  b[7] = a[21];
  return max3(max3(b[0], b[1], b[2]), max3(b[3], b[4], b[5]), fmaxf(b[6], b[7]));
}

__device__ __forceinline__ void store32(void* dst, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

__device__ __forceinline__ void store16(void* dst, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  *reinterpret_cast<uint4*>(dst) = make_uint4(a, b, c, d);
}

__device__ __forceinline__ uint32_t count_arrival(uint32_t* counter) {
  uint32_t before;
  asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], %2;" : "=r"(before) : "l"(counter), "r"(1u) : "memory");
  return before;
}

// Joins a split unit's pieces, in order, by the 8 softmax warps: 8 neighbouring rows at a time, the lanes sharing their
// outputs, the next piece on its way meanwhile.  (A row at a time, every trip to memory waited for: 45 us for 256 rows.)
template <int D>
__device__ __noinline__ void join(const ChunkParams& p, const Plan& plan, const Piece& s, int warp, int lane) {
  constexpr int kW = D == 64 ? 64 : 128, kCols = D / kW, kE = kW / 32, kRows = 8;  // columns at a time
  constexpr int kSlot = 128 * Cfg<D>::kM, kWarps = 4 * Cfg<D>::kM;
  using Part = typename std::conditional<kE == 4, float4, float2>::type;
  const int c0 = (int)run_of(s.real, plan.total, plan.ctas), c1 = (int)run_of(s.real + s.tiles - 1, plan.total, plan.ctas);
  const int n = c1 - c0 + 1, per = 128 / p.G;
  const int blocks0 = (s.tokens[0] * p.G + kRows - 1) / kRows, blocks = blocks0 + (s.tokens[1] * p.G + kRows - 1) / kRows;
  // piece 0 lies in its CTA's second slot, the others in the first
  const int64_t first = ((int64_t)c0 * 2 + 1) * kSlot, then = ((int64_t)c0 * 2 + 2) * kSlot;
  auto load = [&](int q, int i, float2& ml, Part (&v)[kRows]) {
    const int blk = q / kCols;
    const int at_row = blk < blocks0 ? blk * kRows : 128 + (blk - blocks0) * kRows;
    const int64_t at = (i == 0 ? first : then + (int64_t)(i - 1) * (2 * kSlot)) + at_row;
    ml = __ldcg(reinterpret_cast<const float2*>(p.part_ml) + at + lane % kRows);
    const Part* src = reinterpret_cast<const Part*>(p.part_o + at * D + q % kCols * kW) + lane;
#pragma unroll
    for (int r = 0; r < kRows; ++r) v[r] = __ldcg(src + r * (D / kE));
  };
  float2 ml;
  Part v[kRows];
  if (warp < blocks * kCols) load(warp, 0, ml, v);
#pragma unroll 1
  for (int q = warp; q < blocks * kCols; q += kWarps) {
    const int blk = q / kCols;
    const int m = blk >= blocks0, row = (blk - (m ? blocks0 : 0)) * kRows;  // of the M tile
    float top = kNoScore, sum = 0.f, o[kRows][kE] = {};
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      float2 ml_next = ml;
      Part v_next[kRows];
#pragma unroll
      for (int r = 0; r < kRows; ++r) v_next[r] = v[r];
      if (i + 1 < n) load(q, i + 1, ml_next, v_next);
      else if (q + kWarps < blocks * kCols) load(q + kWarps, 0, ml_next, v_next);
      const float now = fmaxf(top, ml.x), keep = exp2_approx(top - now);
      const float w = ml.y == 0.f ? 0.f : exp2_approx(ml.x - now);
      sum = fmaf(sum, keep, w * ml.y);
      top = now;
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        const float kr = __shfl_sync(0xffffffffu, keep, r), wr = __shfl_sync(0xffffffffu, w, r);
        const float* x = reinterpret_cast<const float*>(&v[r]);
#pragma unroll
        for (int e = 0; e < kE; ++e) o[r][e] = fmaf(o[r][e], kr, wr == 0.f ? 0.f : wr * x[e]);  // else x may be anything
        v[r] = v_next[r];
      }
      ml = ml_next;
    }
    const float f = inverse(sum);
    const int rows = s.tokens[m] * p.G - row;  // that are the unit's
    auto out_row = [&](int r) {
      return ((int64_t)s.s0 + m * per + (row + r) / p.G) * p.Hq + s.kvh * p.G + (row + r) % p.G;
    };
    if (lane < min(rows, kRows) && p.lse && q % kCols == 0) p.lse[out_row(lane)] = (top + log2f(sum)) * kLn2;
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const float fr = __shfl_sync(0xffffffffu, f, r);
      if (r >= rows) continue;
      char* dst = p.out + (out_row(r) * D + q % kCols * kW + lane * kE) * 2;
      if constexpr (kE == 4)
        *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16(o[r][0] * fr, o[r][1] * fr), pack_bf16(o[r][2] * fr, o[r][3] * fr));
      else
        *reinterpret_cast<uint32_t*>(dst) = pack_bf16(o[r][0] * fr, o[r][1] * fr);
    }
  }
}

// Softmax and results of M tile m's rows, one a thread.  kAny: a cap, a bias or a scale that is not positive.
template <int D, bool kAny>
__device__ __forceinline__ void run_softmax(const ChunkParams& p, const Plan& plan, int cost, const Maps& maps, Bars& bars,
                                            uint8_t* sV, uint32_t stage, uint32_t tmem, int m, int warp, int lane) {
  using C = Cfg<D>;
  const int rl = (warp % 4) * 32 + lane;  // row of the M tile = TMEM lane
  const uint32_t lane_at = tmem + ((uint32_t)(warp % 4 * 32) << 16);
  const uint32_t tO = lane_at + kColO(m);
  const float mul = p.scale * kLog2e;
  const bool wide = reinterpret_cast<uintptr_t>(p.out) % 32 == 0;  // else 16-byte stores
  const Scorer score(p);
  // factor of the cap's exponential where the cap is small enough for that form, else 0
  const float cap_in = kAny && score.cap2 > 0.f && score.cap2 <= 128.f ? fminf(fmaxf(score.cap_mul, -0x1p100f), 0x1p100f) * (2.f * kLog2e) : 0.f;
  uint32_t g = 0, done = 0, posts = 0, cleared = 0;  // ring's tiles, this M tile's tiles
  bool ok = true;
  Walk walk(p, plan, cost);
  Piece s;
  while (ok && walk.next(s)) {
    const int n_mine = s.computed(m);
    const int tok = rl / p.G, head = s.kvh * p.G + rl % p.G;
    const bool valid = tok < s.tokens[m];
    const int first = s.pos0 + m * (128 / p.G);      // position of the M tile's first token
    const int last = first + s.tokens[m] - 1;
    const int pos = valid ? first + tok : -1;
    const float slope = kAny && p.slopes && valid ? slope_of(p.slopes, head) : 0.f;
    float top = kNoScore, sum = 0.f;
    // The M tiles' softmaxes share the issue slots, their products the tensor pipe: out of step with each other they
    // share better where the tiles are many.  Not at all | from 16 tiles on | from 4: 8192 tokens behind 24576 5.51 | 5.48 |
    // 5.48 ms, 64 turns 740 | 739 | 738 us, 32 prompts of 512 tokens 119 | 118 | 128 us.
    if (m == 1 && n_mine >= 16) {
      const long long from = clock64();
      while (clock64() - from < 600) {
      }
    }
    for (int k = 0; k < n_mine; ++k, ++done) {
      const int t0 = s.key(s.a + k);
      const uint32_t tS = lane_at + kColS(m, done);
      ok = mbar_wait_warp(&bars.s_full[m][done & 1], (done >> 1) & 1, &bars.abort, p.status, limit_ns());
      if (!ok) break;
      fence_after();
      // rows that do not see all of the tile's keys
      const bool cut = t0 + kBlk - 1 > first || (p.window > 0 && last - t0 >= p.window);
      uint64_t seen = ~0ull;
      if (cut) {
        auto below = [](int n) -> uint64_t { return n <= 0 ? 0 : n >= 64 ? ~0ull : (1ull << n) - 1; };
        seen = below(min(pos - t0, 63) + 1);
        if (p.window > 0 && pos - t0 >= p.window)  // not below the window, but for the kept first keys
          seen &= ~below(min(pos - t0 - p.window, 63) + 1) | below(min(p.n_sink - t0, 64));
      }
      float sv[64];
      {
        uint32_t r0[32], r1[32];
        tmem_ld32(tS, r0);
        tmem_ld32(tS + 32, r1);
        tmem_ld_wait(r0);
        tmem_loaded(r1);
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          sv[c] = __uint_as_float(r0[c]);
          sv[32 + c] = __uint_as_float(r1[c]);
        }
      }
      if constexpr (kAny) {
        if (cap_in > 0.f || cap_in < 0.f) {
          // tanh y = 1 - 2 / (1 + e^2y): off by 2^-21 of the cap at most, 4e-5 here, small scores as much as large ones.  In
          // units of 2^-24 around y = -0.8, where the sum is largest: the argument's factors and product 1.5, the exponential
          // (2^-22) 1.2, 1 + e^2y 1.4, the reciprocal (a step) 2, the cap's factor and the last product 1.7.  (Scorer's form
          // keeps small scores' bits: 16 windows of 1024 with a cap of 30 take 1070 us with it, 620 this way.)
#pragma unroll
          for (int c = 0; c < 64; ++c) sv[c] = fmaf(rcp_approx(1.f + exp2_approx(sv[c] * cap_in)), -2.f * score.cap2, score.cap2);
        } else {
#pragma unroll
          for (int c = 0; c < 64; c += 16) {
            float y[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) y[e] = sv[c + e];
            score(y);
#pragma unroll
            for (int e = 0; e < 16; ++e) sv[c + e] = y[e];
          }
        }
        if (p.slopes) {
#pragma unroll
          for (int c = 0; c < 64; ++c) sv[c] = fmaf(slope, (float)(t0 + c - pos), sv[c]);
        }
      }
      if (cut) {
        const uint32_t lo = (uint32_t)seen, hi = (uint32_t)(seen >> 32);
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          if (!(lo & 1u << c)) sv[c] = -INFINITY;
          if (!(hi & 1u << c)) sv[32 + c] = -INFINITY;
        }
      }
      // keys that no row of the unit sees leave V
      if (s.ragged(t0)) {
        const uint32_t slot = (g + k) % C::kSlots;
        ok = mbar_wait_warp(&bars.v_seen[m], cleared & 1, &bars.abort, p.status, limit_ns());
        if (!ok) break;
        ++cleared;
        const int t = t0 + rl % kBlk;
        if (t > s.last || (t < s.lo && t >= s.sink)) {
          for (int h = rl / kBlk; h < D / 64; h += 2) {
            uint4* row = reinterpret_cast<uint4*>(sV + slot * C::kTile + h * kHalf + rl % kBlk * 128);
#pragma unroll
            for (int y = 0; y < 8; ++y) row[y] = make_uint4(0, 0, 0, 0);
          }
        }
        fence_proxy_async();
        __syncwarp();
      }
      // Weights against the reference as it is.  It may lie below the maximum as long as their sum stays below 2^20:
      // floats do not mind.  Past that, and in a unit's first tile, it becomes the maximum and the weights are taken again.
      // (Without a bias it seldom moves.  A slope above 0.22 moves it in every tile, as the far keys come first: 8 x 1000
      // tokens, 32/8 heads of 128, 195 us with the usual slopes, 95 without.)
      const float f = kAny ? 1.f : mul;
      const uint64_t sc2 = pack_f32x2(f, f);
      uint32_t pk[32];
      float tile_sum;
      auto weigh = [&]() {
        const uint64_t neg2 = pack_f32x2(-top, -top);
        uint64_t acc0 = 0, acc1 = 0;
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          float e0, e1;
          exp2_pair(sv[2 * c], sv[2 * c + 1], sc2, neg2, e0, e1);
          if (c & 1) acc1 = add_f32x2(acc1, pack_f32x2(e0, e1)); else acc0 = add_f32x2(acc0, pack_f32x2(e0, e1));
          pk[c] = pack_bf16(e0, e1);
        }
        tile_sum = sum_f32x2(add_f32x2(acc0, acc1));
      };
      if (k == 0) top = fmaxf(top, max64(sv) * f);
      weigh();
      const bool grow = valid && k > 0 && tile_sum > kMost;
      if (__any_sync(0xffffffffu, grow)) {
        const float now = grow ? fmaxf(top, max64(sv) * f) : top;
        const float alpha = exp2_approx(top - now);  // 0 without a score before
        ok = mbar_wait_warp(&bars.pv_done[m][(done - 1) & 1], ((done - 1) >> 1) & 1, &bars.abort, p.status, limit_ns());
        if (!ok) break;
        fence_after();
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t r[32];
          tmem_ld32(tO + c, r);
          tmem_ld_wait(r);
#pragma unroll
          for (int j = 0; j < 32; ++j) r[j] = __float_as_uint(__uint_as_float(r[j]) * alpha);
          tmem_st32(tO + c, r);
        }
        sum *= alpha;
        top = now;
        weigh();
      }
      tmem_st32(tS, pk);
      sum += tile_sum;
      tmem_st_wait();
      fence_before();
      mbar_arrive(&bars.p_full[m][done & 1]);
    }
    if (!ok) break;
    g += s.e - s.a;
    if (n_mine > 0) {
      ok = mbar_wait_warp(&bars.pv_done[m][(done - 1) & 1], ((done - 1) >> 1) & 1, &bars.abort, p.status, limit_ns());
      if (!ok) break;
      fence_after();
    }
    if (!s.split()) {
      if (n_mine > 0) {
        const int64_t at = ((int64_t)s.s0 + m * (128 / p.G) + tok) * p.Hq + head;
        const float f = inverse(sum);
        char* dst = p.out + at * D * 2;
        if (maps.out_tokens && __all_sync(0xffffffffu, valid)) {
          // whole warps: 64 columns at a time through shared memory, stored by TMA (rows of their own, stored directly,
          // touch 32 lines an instruction: 3600 cycles a unit, 1500 this way)
          const uint32_t mine = stage + (warp - 8) * 4096;
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            uint32_t r[32];
            tmem_ld32(tO + c, r);
            tmem_ld_wait(r);
            if (c % 64 == 0) {
              if (lane == 0) tma_store_read_wait();  // the last box has left
              __syncwarp();
            }
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              uint32_t w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                w[e] = pack_bf16(__uint_as_float(r[8 * x + 2 * e]) * f, __uint_as_float(r[8 * x + 2 * e + 1]) * f);
              sts16(mine + lane * 128 + (((c % 64 / 8 + x) ^ (lane & 7)) << 4), w[0], w[1], w[2], w[3]);
            }
            if (c % 64 == 32) {
              fence_proxy_async();
              __syncwarp();
              if (lane == 0) {
                const int row = (warp % 4) * 32;  // of the M tile
                tma_store_3d(&maps.out, mine, c - 32, s.kvh * p.G + row % p.G, s.s0 + m * (128 / p.G) + row / p.G);
              }
            }
          }
          if (p.lse) p.lse[at] = (top + log2f(sum)) * kLn2;
          fence_before();
          continue;
        }
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t r[32];
          tmem_ld32(tO + c, r);
          tmem_ld_wait(r);
          if (valid) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              uint32_t w[8];
#pragma unroll
              for (int e = 0; e < 8; ++e)
                w[e] = pack_bf16(__uint_as_float(r[16 * x + 2 * e]) * f, __uint_as_float(r[16 * x + 2 * e + 1]) * f);
              if (wide) {
                store32(dst + (c + 16 * x) * 2, w);
              } else {
                store16(dst + (c + 16 * x) * 2, w[0], w[1], w[2], w[3]);
                store16(dst + (c + 16 * x) * 2 + 16, w[4], w[5], w[6], w[7]);
              }
            }
          }
          __syncwarp();
        }
        if (valid && p.lse) p.lse[at] = (top + log2f(sum)) * kLn2;
        fence_before();
      }
      continue;
    }
    // a piece: its rows to the workspace; the unit's last arrival joins them
    {
      const int64_t slot = (int64_t)blockIdx.x * 2 + (s.a == 0);
      const int64_t row = slot * (128 * C::kM) + m * 128 + rl;
      if (valid) {
        reinterpret_cast<float2*>(p.part_ml)[row] = make_float2(top, sum);
        if (n_mine == 0) {
          const uint32_t zero[8] = {};
#pragma unroll 1
          for (int c = 0; c < D; c += 8) store32(p.part_o + row * D + c, zero);
        }
      }
      __syncwarp();
      if (n_mine > 0) {
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t r[32];
          tmem_ld32(tO + c, r);
          tmem_ld_wait(r);
          if (valid) {
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              uint32_t w[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) w[e] = r[8 * x + e];
              store32(p.part_o + row * D + c + 8 * x, w);
            }
          }
          __syncwarp();
        }
        fence_before();
      }
      __threadfence();
      mbar_arrive(&bars.posted);
      ok = mbar_wait_warp(&bars.posted, posts & 1, &bars.abort, p.status, limit_ns());
      if (!ok) break;
      if (warp == 8 && lane == 0) {
        const int c0 = (int)run_of(s.real, plan.total, plan.ctas);
        const uint32_t n = (uint32_t)(run_of(s.real + s.tiles - 1, plan.total, plan.ctas) - c0 + 1);
        const bool all = count_arrival(p.arrive + c0) == n - 1;
        if (all) p.arrive[c0] = 0;
        bars.last = all;
        mbar_arrive(&bars.decided);
      }
      ok = mbar_wait_warp(&bars.decided, posts & 1, &bars.abort, p.status, limit_ns());
      if (!ok) break;
      ++posts;
      if (*(volatile int*)&bars.last) {
        __threadfence();
        join<D>(p, plan, s, warp - 8, lane);
      }
    }
  }
  if (lane == 0) tma_store_wait();  // outputs are written when the CTA ends
  __syncwarp();
}

template <int D, bool kAny>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_tc_kernel(const __grid_constant__ ChunkParams p, const __grid_constant__ Maps maps,
                    const __grid_constant__ Residues res, int cost, int least, float join_cost) {
  using C = Cfg<D>;
  extern __shared__ uint8_t raw[];
  __shared__ Bars bars;
  __shared__ Plan plan;
  const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
  uint8_t* sV = raw + (base - smem_u32(raw)) + C::kOffV;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (p.cu && p.status && blockIdx.x == 0) {
    ChunkOf c;
    for (int b = threadIdx.x; b < p.B; b += kThreads)
      if (!chunk_of(p, b, c)) atomicOr(p.status, TV_DEV_BAD_OFFSETS);
  }
  make_plan(p, res, cost, least, join_cost, plan);
  if (plan.x0 >= plan.x1) return;  // all threads, before anything is set up
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kSlots; ++i) {
      for (int v = 0; v < 2; ++v) {
        mbar_init(&bars.full[v][i], 1);
        mbar_init(&bars.empty[v][i], C::kM);
      }
    }
    for (int m = 0; m < 2; ++m) {
      mbar_init(&bars.q_full[m], 1);
      mbar_init(&bars.q_free[m], 1);
      for (int x = 0; x < 2; ++x) {
        mbar_init(&bars.s_full[m][x], 1);
        mbar_init(&bars.p_full[m][x], 128);
        mbar_init(&bars.pv_done[m][x], 1);
      }
      mbar_init(&bars.v_seen[m], 1);
      mbar_init(&bars.drain[m], 1);
      mbar_init(&bars.drain[2 + m], 1);
    }
    mbar_init(&bars.posted, 128 * C::kM);
    mbar_init(&bars.decided, 1);
    bars.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 6) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&bars.tmem)), "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = bars.tmem;
  // registers: 256 threads x 72 + 256 x 184 = 512 x 128, what the block was launched with
  if (warp < 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp < 4) {
      run_producer<D>(p, plan, cost, maps, bars, base, warp, lane);
    } else if (warp < 6) {
      if (lane == 0 && warp - 4 < C::kM) issue_scores<D>(p, plan, cost, maps, bars, base, tmem, warp - 4);
    } else {
      if (lane == 0 && warp - 6 < C::kM) issue_outputs<D>(p, plan, cost, bars, base, tmem, warp - 6);
    }
    __syncwarp();
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
    if (warp < 8 + 4 * C::kM)
      run_softmax<D, kAny>(p, plan, cost, maps, bars, sV, base + C::kOffOut, tmem, (warp - 8) / 4, warp, lane);
  }
  fence_before();
  __syncthreads();
  if (warp == 6) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
  }
}

// ---------------------------------------------------------------- host side

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

int get_encoder(EncodeTiled* fn) {
  static std::once_flag once;
  static EncodeTiled cached = nullptr;
  static cudaError_t err = cudaSuccess;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    err = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q);
    if (err == cudaSuccess && q == cudaDriverEntryPointSuccess) cached = reinterpret_cast<EncodeTiled>(f);
  });
  if (!cached) return fail(TV_ERR_CUDA, "cuTensorMapEncodeTiled unavailable (%s)", cudaGetErrorName(err));
  *fn = cached;
  return TV_OK;
}

int encode(EncodeTiled fn, CUtensorMap* map, const void* ptr, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
           const cuuint32_t* box, const char* what) {
  const cuuint32_t one[3] = {1, 1, 1};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(ptr), dims, strides, box, one,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(TV_ERR_CUDA, "cuTensorMapEncodeTiled(%s) failed with %d", what, (int)r);
  return TV_OK;
}

// Boxes of a softmax warp's 32 rows, where rows of one token fill them: 32 / G tokens, or 32 heads of one.
int encode_out(EncodeTiled fn, Maps* maps, const ChunkParams& p, int D) {
  maps->out_tokens = p.G <= 32 && 32 % p.G == 0 ? 32 / p.G : p.G % 32 == 0 ? 1 : 0;
  if (!maps->out_tokens) {
    maps->out = maps->q;
    return TV_OK;
  }
  const cuuint64_t row = (cuuint64_t)D * 2;
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)p.Hq, (cuuint64_t)p.T}, strides[2] = {row, row * p.Hq};
  const cuuint32_t box[3] = {64, (cuuint32_t)std::min(p.G, 32), (cuuint32_t)maps->out_tokens};
  return encode(fn, &maps->out, p.out, 3, dims, strides, box, "out");
}

template <int D, bool kAny>
int launch(const ChunkParams& p, const Maps& maps, cudaStream_t stream) {
  constexpr int smem = Cfg<D>::kSmem;
  const cudaError_t e =
      cudaFuncSetAttribute(chunk_tc_kernel<D, kAny>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(chunk_tc_kernel)");
  // join of one piece in tiles, over the number of units (about): 1500 cycles of 1900 for 64 rows
  const int step = Cfg<D>::kM * (128 / p.G);
  const int64_t units = (int64_t)p.Hkv * std::max<int64_t>(ceil_div(p.T, step), std::min(p.T, p.B));
  const int64_t rows = std::min<int64_t>(step, ceil_div(p.T, p.B)) * p.G;
  const float join_cost = 0.8f * (float)ceil_div(rows, 64) / (float)units;
  chunk_tc_kernel<D, kAny><<<p.ctas, kThreads, smem, stream>>>(p, maps, residues_of(step), 4, 8, join_cost);
  TV_LAUNCH_CHECK("chunk_tc_kernel");
  return TV_OK;
}

}  // namespace

const char* chunk_tc_unsupported(const DeviceInfo& dev, const ChunkParams& p, int dtype, int head_dim) {
  if (dev.cc_major != 10) return "device is not sm_10x";
  if (dtype != TV_BF16) return "dtype is not bf16";
  if (p.G > 128) return "more than 128 query heads per KV head";
  if (p.block_size % 8) return "block_size is not a multiple of 8";
  if (p.num_blocks >= INT32_MAX / ((int64_t)p.Hkv * p.block_size)) return "the cache has 2^31 rows";
  if (p.T > 1 && (p.q_stride < (int64_t)p.Hq * head_dim * 2 || p.q_stride >= (int64_t)1 << 40))
    return "queries of neighbouring tokens overlap, or lie 2^40 bytes apart";
  if (dev.max_smem_optin < (size_t)Cfg<128>::kSmem + sizeof(Bars) + sizeof(Plan) + 256) return "not enough shared memory";
  return nullptr;
}

int chunk_tc_m_tiles(int head_dim) { return head_dim == 256 ? Cfg<256>::kM : Cfg<128>::kM; }

size_t chunk_tc_workspace(int head_dim, int ctas) {
  return (size_t)ctas * 2 * 128 * chunk_tc_m_tiles(head_dim) * (head_dim + 2) * 4;
}

int launch_chunk_tc(const ChunkParams& p, int D, cudaStream_t stream) {
  EncodeTiled fn;
  if (int rc = get_encoder(&fn)) return rc;
  Maps maps;
  const int br = std::min(kBlk, p.block_size & -p.block_size);
  const cuuint64_t row = (cuuint64_t)D * 2;
  {
    const cuuint64_t dims[2] = {(cuuint64_t)D, (cuuint64_t)p.num_blocks * p.Hkv * p.block_size}, strides[1] = {row};
    const cuuint32_t box[2] = {64, (cuuint32_t)br};
    if (int rc = encode(fn, &maps.k, p.k_cache, 2, dims, strides, box, "k_cache")) return rc;
    if (int rc = encode(fn, &maps.v, p.v_cache, 2, dims, strides, box, "v_cache")) return rc;
  }
  {
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)p.Hq, (cuuint64_t)p.T};
    const cuuint64_t strides[2] = {row, p.T > 1 ? (cuuint64_t)p.q_stride : row * p.Hq};
    const cuuint32_t box[3] = {64, (cuuint32_t)p.G, (cuuint32_t)(128 / p.G)};
    if (int rc = encode(fn, &maps.q, p.q, 3, dims, strides, box, "q")) return rc;
  }
  if (int rc = encode_out(fn, &maps, p, D)) return rc;
  // the plain form masks before it scales: its factor has to keep -inf what it is
  const bool any = p.softcap > 0.f || p.slopes || !(p.scale * kLog2e >= FLT_MIN);
  if (D == 256) return any ? launch<256, true>(p, maps, stream) : launch<256, false>(p, maps, stream);
  if (D == 64) return any ? launch<64, true>(p, maps, stream) : launch<64, false>(p, maps, stream);
  return any ? launch<128, true>(p, maps, stream) : launch<128, false>(p, maps, stream);
}

}  // namespace tv

#ifdef TV_TEST_HOOKS
// Development builds only: the wait limit, and the ring entry of CTA 0 that gets no loads (-1: none).
extern "C" int tv_test_set_chunk_hooks(unsigned long long limit_ns, int withhold_entry) {
  if (cudaMemcpyToSymbol(tv::g_chunk_limit_ns, &limit_ns, sizeof(limit_ns)) != cudaSuccess) return -6;
  if (cudaMemcpyToSymbol(tv::g_chunk_withhold, &withhold_entry, sizeof(withhold_entry)) != cudaSuccess) return -6;
  return cudaDeviceSynchronize() == cudaSuccess ? 0 : -6;
}
#endif
