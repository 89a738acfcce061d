// Decay per head of the linear attention recurrence.
//
//   S_t = lam S_{t-1} + k_t v_t^T,   o_t = q_t S_t,   lam = exp(g), g <= 0
//
// For a chunk of R tokens with local index l = 0 .. R-1 entered with state S:
//   o_l = sum_{m <= l} lam^(l-m) (q_l . k_m) v_m + lam^(l+1) q_l S
//   S'  = lam^R S + sum_m lam^(R-1-m) k_m v_m^T
// In reverse order (the backward's sums over later tokens, G_t = lam G_{t+1} +
// q_t^T do_t) the state is held already decayed, Ghat = lam G, so that it
// starts from dL/dS_N and ends as dL/dS_0:
//   o_l   = sum_{m >= l} lam^(m-l) (q_l . k_m) v_m + lam^(R-1-l) q_l Ghat
//   Ghat' = lam^R Ghat + sum_m lam^(m+1) k_m v_m^T
// Every exponent is >= 0, so no factor exceeds 1 and none overflows; g = -inf
// (lam = 0) is a valid decay.
#pragma once
#include <cuda_runtime.h>

namespace lcl {
namespace decay {

// lam^n = exp(n g) for n >= 0, correctly rounded up to fp32 (lam^0 = 1 for
// every g).  Evaluated in double, once per item and table entry: the fp32
// exponential of a rounded product is up to n |g| 2^-24 off, and an error in
// lam^C repeats at every chunk.
__device__ __forceinline__ float power(double g, int n) { return n == 0 ? 1.f : static_cast<float>(exp(g * n)); }

// lam^n as the sum of two fp32 values.  A state lives through thousands of
// chunks: with slow decay one fp32 factor, 3e-8 off at worst, would repeat its
// error as often (1024 chunks: 3e-5).
//
// Both values are positive (as long as lam^n is above 2^-126): hi is below lam^n,
// never equal to it (1 is 1 - 2^-24 and 2^-24), so that an infinite state stays
// infinite: x hi + x lo with a lo of zero would be infinity times zero, with a
// negative one infinity minus infinity.  For a finite x the sum is as good: the
// fused x hi + (x lo) is rounded once, and for lam^n = 1 it is x.
__device__ __forceinline__ void power2(double g, int n, float& hi, float& lo) {
    const double f = n == 0 ? 1.0 : exp(g * n);
    hi = __double2float_rz(f);
    if (hi > 0.f && hi == f) hi = __uint_as_float(__float_as_uint(hi) - 1u);
    lo = static_cast<float>(f - hi);
}

}  // namespace decay
}  // namespace lcl
