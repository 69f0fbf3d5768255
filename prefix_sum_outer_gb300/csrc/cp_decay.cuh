// Pieces shared by the kernels of linear attention with a decay for each head:
//     S_t = a S_{t-1} + k_t v_t^T,   out_t = s S_t^T q_t,   a = e^{g_h}.
// Over a piece of rows 0 .. n-1 that starts from S (the state after the row
// before it):
//     out_i = s sum_{j<=i} a^{i-j} (q_i . k_j) v_j + s a^{i+1} S^T q_i,
//     S'    = a^n S + sum_j a^{n-1-j} k_j v_j^T,
// and backward, from R (the gradient of the state after the piece's last row,
// scale and all, seen from the row behind it; z = 1 where it is seen from that
// last row itself, as the gradient of S_N is, else 0):
//     dv_j  = s sum_{i>=j} a^{i-j} (k_j . q_i) go_i + a^{n-j-z} R^T k_j,
//     dk_j  = s sum_{i>=j} a^{i-j} (v_j . go_i) q_i + a^{n-j-z} R v_j,
//     dq_i  = s sum_{j<=i} a^{i-j} (go_i . v_j) k_j + s a^{i+1} S go_i,
//     R'    = a^{n-z} R + s sum_i a^i q_i go_i^T,
// so every result is one product of three row arrays (a, b, c) with a state,
// in forward or reverse order.
#pragma once
#include "cp_delta.cuh"

namespace cp {
namespace decay {

using namespace delta;  // element loads and stores, packed fp32, decay_parts

// A head's log decay as the kernels use it: in [-120, 0], e^-120 being 0 in fp32
// (so that 0 times -inf never occurs); a positive one, whose powers overflow,
// and NaN make the head's results NaN.
__device__ __forceinline__ float head_decay(float g) {
  return g <= 0.f ? fmaxf(g, kMinLogDecay) : __int_as_float(0x7fffffff);
}
// a^n as one number and, for a state's decay over a step, as hi + lo: g n is
// formed exactly, for its rounding alone would leave |g n| 2^-24
__device__ __forceinline__ float power(float g, int n) {
  const float x = g * (float)n;
  return fmaf(expf(x), fmaf(g, (float)n, -x), expf(x));
}
__device__ __forceinline__ float2 power_parts(float g, int n) {
  float x = g * (float)n, f = fmaf(g, (float)n, -x);
  // decay_parts knows its lo for |x| < 0.34; a state of more than that a step
  // still remembers a few steps, so its power is squared up from a smaller one
  int k = 0;
  while (x < -0.3f && k < 8) {
    x *= 0.5f;
    f *= 0.5f;
    ++k;
  }
  float2 p = decay_parts(x, f);
  for (; k > 0; --k) {
    const float h = p.x * p.x;
    p = make_float2(h, fmaf(p.x, p.x, -h) + 2.f * p.x * p.y);
  }
  return p;
}
// rows of sequence b
__device__ __forceinline__ int64_t rows_of(const int* lengths, int64_t b, int64_t N) {
  if (lengths == nullptr) return N;
  const int64_t n = lengths[b];
  return n < 0 ? 0 : (n > N ? N : n);
}

}  // namespace decay
}  // namespace cp
