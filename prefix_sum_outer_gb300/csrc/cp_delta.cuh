// Pieces shared by the gated delta rule's kernels.
//
// The rule, per head (S: D x M state, fp32):
//     S_t = a_t S_{t-1} + k_t u_t^T,   u_t = b_t (v_t - a_t S_{t-1}^T k_t),
//     out_t = s S_t^T q_t,             a_t = e^{g_t}.
// Over a chunk of C rows that starts from S, with G the running sum of g,
// Gam_ij = e^{G_i - G_j} (j <= i), gam_i = e^{G_i}, del_j = e^{G_C - G_j}:
//     A_ij = b_i Gam_ij k_i.k_j (j < i),     P_ij = s Gam_ij q_i.k_j (j <= i),
//     R = V - gam K S,   U = (I + A)^-1 (b R),
//     out = s gam Q S + P U,   S' = gam_C S + K^T (del U).
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "cp_internal.h"

namespace cp {
namespace delta {

template <typename T>
__device__ __forceinline__ float ld_f32(const T* p);
template <>
__device__ __forceinline__ float ld_f32<float>(const float* p) { return *p; }
template <>
__device__ __forceinline__ float ld_f32<__nv_bfloat16>(const __nv_bfloat16* p) {
  return __bfloat162float(*p);
}
template <>
__device__ __forceinline__ float ld_f32<__half>(const __half* p) { return __half2float(*p); }

template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }

// pairs of fp32 in one instruction
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "add.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 sub2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "sub.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mul.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mov.b64 z, {%6, %7};\n\tfma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// A log decay, in powers of two, as two parts whose running sums over a chunk
// stay exact to fp32: a multiple of 2^-10 (sums of up to 64 of them at |g| <= 120
// are exact) and the rest (|f| <= 2^-11, with what rounding g log2(e) left over).
// With one fp32 sum, a decay near e^-100 (a cleared state) would leave every
// later difference G_i - G_j of its chunk 1e-5 off.  Below -120 the decay is 0
// in fp32, and -inf becomes finite, so that differences of sums are never inf -
// inf.  NaN stays NaN.
constexpr float kMinLogDecay = -120.f;
__device__ __forceinline__ float2 split_decay(float g) {
  constexpr double kLog2e = 1.4426950408889634;
  constexpr float kHi = (float)kLog2e, kLo = (float)(kLog2e - (double)kHi);
  g = g < kMinLogDecay ? kMinLogDecay : g;
  const float l = g * kHi, c = rintf(l * 1024.f) * 0x1p-10f;
  return make_float2(c, (l - c) + fmaf(g, kLo, fmaf(g, kHi, -l)));
}
// e^{G_i - G_j} from the two-part running sums
__device__ __forceinline__ float decay_between(float2 gi, float2 gj) {
  return exp2f((gi.x - gj.x) + (gi.y - gj.y));
}
// The decay of a state over a step, e^{g + f} with f below g's rounding, as hi +
// lo.  One fp32 number is up to 2^-25 off, the same way at every step where the
// decay is the same, and a state that remembers n steps would be n times as far
// off (4e-4 after 8,000 tokens at g = -1e-4, one by one).  lo is what rounding
// e^g left over: e^g - 1 is g (exact) and the rest of the series, which for |g| <
// 0.34 is below 0.07 and so good to 4e-9 in fp32; g - (hi - 1) has no rounding.
// Past that the state forgets within a few steps, and lo is 0.
__device__ __forceinline__ float2 decay_parts(float g, float f) {
  const float hi = expf(g);
  if (!(fabsf(g) < 0.34f)) return make_float2(hi, 0.f);
  float q = 1.f / 40320.f;
  q = fmaf(q, g, 1.f / 5040.f);
  q = fmaf(q, g, 1.f / 720.f);
  q = fmaf(q, g, 1.f / 120.f);
  q = fmaf(q, g, 1.f / 24.f);
  q = fmaf(q, g, 1.f / 6.f);
  q = fmaf(q, g, 0.5f);
  const float left = (g - (hi - 1.f)) + q * (g * g);
  return make_float2(hi, fmaf(hi, f, left));
}
__device__ __forceinline__ float2 decay_parts(float2 G) {  // from a two-part sum
  constexpr double kLn2 = 0.6931471805599453;
  constexpr float kHi = (float)kLn2, kLo = (float)(kLn2 - (double)kHi);
  const float x = G.x * kHi, y = fmaf(G.y, kHi, fmaf(G.x, kLo, fmaf(G.x, kHi, -x)));
  const float g = x + y, z = g - x;  // x + y = g + f exactly
  return decay_parts(g, (x - (g - z)) + (y - z));
}
// inclusive running sums of one pair per lane over a warp
__device__ __forceinline__ float2 warp_scan(float2 x, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const float cx = __shfl_up_sync(0xffffffffu, x.x, o), cy = __shfl_up_sync(0xffffffffu, x.y, o);
    if (lane >= o) {
      x.x += cx;
      x.y += cy;
    }
  }
  return x;
}

// Launched as a programmatic dependent, as the product kernels are: a kernel's
// launch (and, in the chains, its set-up) runs under the end of the one before
// it in the stream, and it touches no global memory before that one has
// completed; a CTA lets the next kernel be scheduled only when its own work is
// done.
template <class K, class... A>
inline cudaError_t launch_dependent(K kern, dim3 grid, unsigned threads, size_t smem,
                                    cudaStream_t stream, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

}  // namespace delta
}  // namespace cp
