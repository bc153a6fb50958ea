// Attention of a chunk of new tokens over the paged cache: what the CUDA-core
// kernel (chunk.cu) and the tcgen05 kernel (chunk_tc.cu) share.
#pragma once

#include <climits>
#include <cstdint>

#include "common.h"

namespace tv {

struct ChunkParams {
  const char* q;
  int64_t q_stride;  // bytes between tokens
  const char* k_cache;
  const char* v_cache;
  int64_t num_blocks;
  int block_size;
  const int32_t* table;
  int max_blocks;
  const int32_t* seq_lens;
  const int32_t* cu;  // nullable: T / B tokens each
  int T, B, Hq, Hkv, G;
  float scale, softcap;
  int window, n_sink;
  const float* slopes;
  char* out;
  float* lse;
  int32_t* status;
  uint32_t* arrive;  // tcgen05 kernel: arrivals of split units, by their first CTA
  int m_tiles;       // ... 128-row M tiles of a unit
  float* part_o;     // [CTAs][2][rows][D]
  float* part_ml;    // [CTAs][2][rows][2]
  int ctas;
};

// A request's chunk: packed rows s0 .. s0 + n - 1, the first at position first (below 0 where the chunk is longer than
// the sequence), L keys.
struct ChunkOf {
  int s0, n, L, first;
};

#ifdef __CUDACC__
// False (and no tokens) where its offsets decrease or leave [0, T].
__device__ __forceinline__ bool chunk_of(const ChunkParams& p, int b, ChunkOf& c) {
  bool ok = true;
  if (p.cu) {
    c.s0 = __ldg(p.cu + b);
    const int s1 = __ldg(p.cu + b + 1);
    ok = c.s0 >= 0 && s1 >= c.s0 && s1 <= p.T;
    c.n = ok ? s1 - c.s0 : 0;
  } else {
    c.n = p.T / p.B;
    c.s0 = b * c.n;
  }
  const int64_t cap = min((int64_t)p.max_blocks * p.block_size, (int64_t)INT32_MAX - 1023);  // a tile's end is an int
  c.L = (int)max((int64_t)0, min((int64_t)__ldg(p.seq_lens + b), cap));
  c.first = c.L - c.n;
  return ok;
}
#endif

// The tcgen05 kernel: why it cannot run a shape (nullptr: it can), its workspace, its launch.
const char* chunk_tc_unsupported(const DeviceInfo& dev, const ChunkParams& p, int dtype, int head_dim);
int chunk_tc_m_tiles(int head_dim);
size_t chunk_tc_workspace(int head_dim, int ctas);
int launch_chunk_tc(const ChunkParams& p, int head_dim, cudaStream_t stream);

}  // namespace tv
