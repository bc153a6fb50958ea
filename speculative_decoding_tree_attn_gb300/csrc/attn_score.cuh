// Scores of the attention kernels over the paged cache (one token or a chunk):
// scale, cap and distance bias in the log2 domain.
#pragma once

#include <cfloat>
#include <cmath>

#include "common.h"

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNoScore = -FLT_MAX;  // maximum of no scores, and of -inf alone: finite, so that -inf weighs 0 against it

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// What a row is multiplied with: 1 over its weights' sum, which is 1 at least where there are any.  Without (no visible
// key, or only scores of -inf) the row is zero, and its m + log2 of the sum is -inf by itself; NaN outputs stay NaN.
__device__ __forceinline__ float inverse(float sum) { return 1.f / fmaxf(sum, FLT_MIN); }

// Score of one (head, key) in the log2 domain from its raw product.
struct Scorer {
  float mul, cap2, cap_mul;  // mul: scale log2 e;  cap2: softcap log2 e, 0 without
  template <class P>
  __device__ __forceinline__ explicit Scorer(const P& p)
      : mul(p.scale * kLog2e), cap2(p.softcap * kLog2e), cap_mul(0.f) {
    // a finite factor for the smallest caps too: 0 has to stay 0
    if (p.softcap > 0.f) cap_mul = fmaxf(fminf(p.scale / p.softcap, FLT_MAX), -FLT_MAX);
  }
  // tanh y within 6 2^-24 of itself: up to 1.25 the seventh convergent of Lambert's continued fraction
  // y / (1 + y^2 / (3 + y^2 / (5 + ..))), beyond 1 - 2 / (1 + e^2y), which loses its last bits only for small y.
  // (Both forms for a warp only where one of its scores needs the second.)
  template <int N>
  __device__ __forceinline__ void operator()(float (&x)[N]) const {
    if (cap2 > 0.f) {
      float z[N], most = 0.f;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        x[i] *= cap_mul;
        z[i] = x[i] * x[i];
        most = fmaxf(most, z[i]);
      }
      const bool far = __any_sync(0xffffffffu, most > 1.5625f);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float n = fmaf(fmaf(z[i] + 378.f, z[i], 17325.f), z[i], 135135.f);
        const float d = fmaf(fmaf(fmaf(28.f, z[i], 3150.f), z[i], 62370.f), z[i], 135135.f);
        float t = x[i] * (n * rcp_approx(d));
        if (far && !(z[i] <= 1.5625f)) t = 1.f - 2.f * rcp_approx(1.f + exp2_approx(x[i] * (2.f * kLog2e)));
        x[i] = cap2 * t;
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] *= mul;
    }
  }
};

// A head's bias in the log2 domain, held within float32: the last key's distance is 0 and has to give 0.
__device__ __forceinline__ float slope_of(const float* slopes, int head) {
  float x = __ldg(slopes + head) * kLog2e;
  asm("{\n\tmin.NaN.f32 %0, %0, 0f7f7fffff;\n\tmax.NaN.f32 %0, %0, 0fff7fffff;\n\t}" : "+f"(x));
  return x;
}

// tanh x is x to float32 for |x| < 2^-12: a factor below the normal numbers would lose bits of it, and caps nothing as
// long as q . k is below 2^114.
inline float cap_that_matters(float scale, float softcap) {
  return softcap > 0.f && std::fabs(scale / softcap) < FLT_MIN ? 0.f : softcap;
}

// Scores are kept in the log2 domain: their factors are held there too.
inline bool factors_fit(float scale, float softcap) {
  return std::isfinite(scale * kLog2e) && softcap >= 0.f && std::isfinite(softcap * kLog2e);
}

}  // namespace
