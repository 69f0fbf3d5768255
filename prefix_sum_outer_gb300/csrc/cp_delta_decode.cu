// One token of the gated delta rule for every head, the state in place:
//     S <- a S + k u^T,   u = b (v - a S^T k),   out = s S^T q.
// The update needs S^T k before it, and the readout of the updated state is
//     S'^T q = a S^T q + (k . q) u,
// so both sums over the rows of S run while S is in registers and the state is
// read and written once: 8 D M bytes per head, which bound the step.  The state's
// decay is applied as hi + lo, for it is applied token after token (cp_delta.cuh).
// A CTA takes 32 value columns of one head, as 8 groups of four or, where rows
// are not whole 16-byte pieces, one by one; its threads hold every row of them,
// ROWS each (64 rows, one by one at D > 64, take 255 registers and spill 16 bytes).
//
// bf16, B = 512, H = 16, D = M = 64: 48.5 us a step back to back, 5.6 TB/s; every
// store of a head waits for all of its loads, which the plain step's do not
// (42.8 us for the same state).
//
// A state of a pool is addressed by the sequence's slot; a slot outside the
// pool is an idle row: out is zero and no state is touched.
#include <algorithm>

#include "cp_delta.cuh"

namespace cp {
namespace {

using namespace delta;

// A CTA has one barrier between its loads and its stores, so an SM wants many
// small ones out of step: bf16, B = 512, H = 16, D = M = 64, back to back, 47.5
// us with ten CTAs of 32 columns, 51.7 with five of 64.
constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kCols = 32;  // value columns of a CTA

template <int V>
struct Vec;
template <>
struct Vec<4> {
  float4 x;
  __device__ __forceinline__ float& operator[](int i) { return (&x.x)[i]; }
};
template <>
struct Vec<1> {
  float x;
  __device__ __forceinline__ float& operator[](int) { return x; }
};

template <bool STREAM, int V>
__device__ __forceinline__ Vec<V> ld_state(const float* p) {
  Vec<V> r;
  if constexpr (V == 4) {
    r.x = STREAM ? __ldcs(reinterpret_cast<const float4*>(p)) : *reinterpret_cast<const float4*>(p);
  } else {
    r.x = STREAM ? __ldcs(p) : *p;
  }
  return r;
}
template <bool STREAM, int V>
__device__ __forceinline__ void st_state(float* p, Vec<V> v) {
  if constexpr (V == 4) {
    if constexpr (STREAM) __stcs(reinterpret_cast<float4*>(p), v.x);
    else *reinterpret_cast<float4*>(p) = v.x;
  } else {
    if constexpr (STREAM) __stcs(p, v.x);
    else *p = v.x;
  }
}

// V: columns a thread owns; ROWS: rows of S it holds (D <= ROWS * row groups).
// Consecutive threads take consecutive columns, so a warp reads whole pieces of
// state rows.
template <typename T, int V, int ROWS, bool STREAM>
__global__ void __launch_bounds__(kThreads, ROWS <= 4 ? 10 : 1)
    delta_decode_kernel(const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v,
                        const float* __restrict__ g, const float* __restrict__ beta,
                        const int* __restrict__ slots, T* __restrict__ out,
                        float* __restrict__ state, int64_t pool, int H, int group, int D, int M,
                        float scale) {
  constexpr int CG = kCols / V;         // column groups (8 or 32: a warp has whole row groups)
  constexpr int RG = kThreads / CG;     // row groups
  __shared__ float part[2][kWarps][kCols];   // per-warp sums: a S^T k and a S^T q, unscaled
  __shared__ float kq_part[kWarps];
  const int64_t p = blockIdx.x;         // b * H + h
  const int64_t b = p / H;
  const int h = (int)(p % H), c0 = blockIdx.y * kCols;
  const int64_t pk = b * (H / group) + h / group;
  const int cg = threadIdx.x % CG, rg = threadIdx.x / CG, w = threadIdx.x / 32;
  const int lane = threadIdx.x % 32, c = c0 + cg * V;
  const int64_t slot = slots != nullptr ? slots[b] : b;
  if (slot < 0 || slot >= pool) {
    for (int i = threadIdx.x; i < kCols && c0 + i < M; i += kThreads)
      out[p * M + c0 + i] = from_f32<T>(0.f);
    return;
  }
  float* S = state + (slot * H + h) * (int64_t)D * M;
  const bool on = c < M;
  Vec<V> st[ROWS];
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    const int d = rg + r * RG;
    if (on && d < D) st[r] = ld_state<STREAM, V>(S + (int64_t)d * M + c);
  }
  // everything else the step reads goes out behind the state, before any use
  float vv[V];
#pragma unroll
  for (int i = 0; i < V; ++i) vv[i] = on ? ld_f32<T>(v + p * M + c + i) : 0.f;
  const float2 decay = decay_parts(g[p], 0.f);
  const float a = decay.x, bt = beta[p];
  float sk[V] = {}, sq[V] = {}, kq = 0.f, kd[ROWS];
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    const int d = rg + r * RG;
    kd[r] = 0.f;
    if (d < D) {
      kd[r] = ld_f32<T>(k + pk * D + d);
      const float qd = ld_f32<T>(q + pk * D + d);
      kq = fmaf(kd[r], qd, kq);
      if (on)
#pragma unroll
        for (int i = 0; i < V; ++i) {
          sk[i] = fmaf(kd[r], st[r][i], sk[i]);
          sq[i] = fmaf(qd, st[r][i], sq[i]);
        }
    }
  }
  // row groups of a warp, then of the CTA
#pragma unroll
  for (int o = CG; o < 32; o *= 2) {
    kq += __shfl_xor_sync(0xffffffffu, kq, o);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      sk[i] += __shfl_xor_sync(0xffffffffu, sk[i], o);
      sq[i] += __shfl_xor_sync(0xffffffffu, sq[i], o);
    }
  }
  if (lane < CG)
#pragma unroll
    for (int i = 0; i < V; ++i) {
      part[0][w][cg * V + i] = sk[i];
      part[1][w][cg * V + i] = sq[i];
    }
  if (lane == 0 && cg == 0) kq_part[w] = kq;
  __syncthreads();
  float u[V], o[V], dot = 0.f;
#pragma unroll
  for (int s = 0; s < kWarps; ++s) dot += kq_part[s];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    float x = 0.f, y = 0.f;
#pragma unroll
    for (int s = 0; s < kWarps; ++s) {
      x += part[0][s][cg * V + i];
      y += part[1][s][cg * V + i];
    }
    u[i] = bt * (vv[i] - a * x);
    o[i] = scale * fmaf(dot, u[i], a * y);
  }
  if (!on) return;
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    const int d = rg + r * RG;
    if (d < D) {
#pragma unroll
      for (int i = 0; i < V; ++i) st[r][i] = fmaf(a, st[r][i], fmaf(kd[r], u[i], decay.y * st[r][i]));
      st_state<STREAM, V>(S + (int64_t)d * M + c, st[r]);
    }
  }
  if (rg == 0)
#pragma unroll
    for (int i = 0; i < V; ++i) out[p * M + c + i] = from_f32<T>(o[i]);
}

template <typename T, int V, int ROWS>
cudaError_t launch(const DeltaShape& s, const DeltaDecode& f, cudaStream_t stream) {
  const dim3 grid((unsigned)(s.B * s.H), (unsigned)((s.M + kCols - 1) / kCols));
  // a state larger than half the L2 is gone before the next step, as in the
  // plain decoding step
  const bool st = (size_t)s.B * s.H * s.D * s.M * sizeof(float) > device_l2_bytes() / 2;
  auto kern = st ? delta_decode_kernel<T, V, ROWS, true> : delta_decode_kernel<T, V, ROWS, false>;
  kern<<<grid, kThreads, 0, stream>>>(
      static_cast<const T*>(f.q), static_cast<const T*>(f.k), static_cast<const T*>(f.v), f.g,
      f.beta, f.slots, static_cast<T*>(f.out), f.state, f.pool, (int)s.H, (int)(s.H / s.Hk),
      (int)s.D, (int)s.M, s.scale);
  return cudaGetLastError();
}

template <typename T>
cudaError_t run(const DeltaShape& s, const DeltaDecode& f, cudaStream_t stream) {
  if (s.M % 4 != 0) {  // 4 row groups
    if (s.D <= 64) return launch<T, 1, 16>(s, f, stream);
    return launch<T, 1, 64>(s, f, stream);
  }
  // 16 row groups
  if (s.D <= 64) return launch<T, 4, 4>(s, f, stream);
  if (s.D <= 128) return launch<T, 4, 8>(s, f, stream);
  return launch<T, 4, 16>(s, f, stream);
}

}  // namespace

cudaError_t delta_decode_launch(const DeltaShape& s, const DeltaDecode& f, cudaStream_t stream) {
  if (s.dtype == CP_DTYPE_BF16) return run<__nv_bfloat16>(s, f, stream);
  if (s.dtype == CP_DTYPE_F16) return run<__half>(s, f, stream);
  return run<float>(s, f, stream);
}

}  // namespace cp
