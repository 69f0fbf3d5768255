// One token of linear attention with a decay for each head, the state in place:
//     S <- a S + k v^T,   out = s S^T q.
// The state is read and written once, 8 D M bytes a head, which bound the step;
// an element needs nothing but its own row's k and column's v, so every store
// follows its own load.  The state's decay is applied as hi + lo, for it is
// applied token after token (cp_delta.cuh).  A CTA takes 64 or 32 value columns of
// one head, four to a thread or, where rows are not whole 16-byte pieces, one; a
// thread holds ROWS rows of them, next to one another, so that its part of q and k
// comes in one load each.
//
// bf16, B = 512, H = 16, D = M = 64: 41.3 us a step back to back, 6.6 TB/s, 99% of
// the copy rate; with 128 columns to a CTA 57 us, with 32 (128 threads) 43, with
// rows 16 apart and q and k element by element 49.
//
// A state of a pool is addressed by the sequence's slot; a slot outside the
// pool is an idle row: out is zero and no state is touched.
#include "cp_decay.cuh"

namespace cp {
namespace {

using namespace decay;

// N dense elements as fp32, in one load where they are a whole piece of memory
template <typename T, int N, bool WHOLE>
__device__ __forceinline__ void ld_row(float (&x)[N], const T* p, int left) {
  if constexpr (WHOLE) {
    struct alignas(sizeof(T) * (N > 8 ? 8 : N) > 16 ? 16 : sizeof(T) * (N > 8 ? 8 : N)) Piece {
      T t[sizeof(T) * (N > 8 ? 8 : N) > 16 ? 16 / sizeof(T) : (N > 8 ? 8 : N)];
    };
    constexpr int K = sizeof(Piece) / sizeof(T);
#pragma unroll
    for (int i = 0; i < N / K; ++i) {
      Piece q{};
      if (i * K < left) q = reinterpret_cast<const Piece*>(p)[i];
#pragma unroll
      for (int j = 0; j < K; ++j) x[i * K + j] = i * K < left ? ld_f32<T>(&q.t[j]) : 0.f;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = i < left ? ld_f32<T>(p + i) : 0.f;
  }
}

template <typename T, int V, int ROWS, bool WHOLE, bool STREAM, int kCols, int kThreads, int kMin>
__global__ void __launch_bounds__(kThreads, kMin)
    decay_decode_kernel(const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v,
                        const float* __restrict__ g, const int* __restrict__ slots,
                        T* __restrict__ out, float* __restrict__ state, int64_t pool, int H,
                        int group, int D, int M, float scale) {
  constexpr int kWarps = kThreads / 32;
  constexpr int CG = kCols / V;         // column groups (8 to 32: a warp has whole row groups)
  __shared__ float part[kWarps][kCols];
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
  float st[ROWS][V];
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    const int d = rg * ROWS + r;
    if (on && d < D) {
      const float* at = S + (int64_t)d * M + c;
      if constexpr (V == 4) {
        const float4 x = STREAM ? __ldcs(reinterpret_cast<const float4*>(at))
                                : *reinterpret_cast<const float4*>(at);
        st[r][0] = x.x; st[r][1] = x.y; st[r][2] = x.z; st[r][3] = x.w;
      } else {
        st[r][0] = STREAM ? __ldcs(at) : *at;
      }
    }
  }
  // everything else the step reads goes out behind the state, before any use
  float vv[V], kd[ROWS], qd[ROWS];
  ld_row<T, V, V == 4>(vv, v + p * M + c, M - c);
  ld_row<T, ROWS, WHOLE>(kd, k + pk * D + rg * ROWS, D - rg * ROWS);
  ld_row<T, ROWS, WHOLE>(qd, q + pk * D + rg * ROWS, D - rg * ROWS);
  const float2 a = decay_parts(head_decay(g[h]), 0.f);
  float o[V] = {};
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    const int d = rg * ROWS + r;
    if (on && d < D) {
      float* at = S + (int64_t)d * M + c;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        st[r][i] = fmaf(a.x, st[r][i], fmaf(kd[r], vv[i], a.y * st[r][i]));
        o[i] = fmaf(qd[r], st[r][i], o[i]);
      }
      if constexpr (V == 4) {
        const float4 x = make_float4(st[r][0], st[r][1], st[r][2], st[r][3]);
        if constexpr (STREAM) __stcs(reinterpret_cast<float4*>(at), x);
        else *reinterpret_cast<float4*>(at) = x;
      } else {
        if constexpr (STREAM) __stcs(at, st[r][0]);
        else *at = st[r][0];
      }
    }
  }
  // row groups of a warp, then of the CTA
#pragma unroll
  for (int m = CG; m < 32; m *= 2)
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] += __shfl_xor_sync(0xffffffffu, o[i], m);
  if (lane < CG)
#pragma unroll
    for (int i = 0; i < V; ++i) part[w][cg * V + i] = o[i];
  __syncthreads();
  if (threadIdx.x < kCols && c0 + threadIdx.x < M) {
    float x = 0.f;
#pragma unroll
    for (int s = 0; s < kWarps; ++s) x += part[s][threadIdx.x];
    out[p * M + c0 + threadIdx.x] = from_f32<T>(scale * x);
  }
}

template <typename T, int V, int ROWS, bool WHOLE, int kCols, int kThreads, int kMin>
cudaError_t launch(const DecayShape& s, const DecayDecode& f, cudaStream_t stream) {
  const dim3 grid((unsigned)(s.B * s.H), (unsigned)((s.M + kCols - 1) / kCols));
  // a state larger than half the L2 is gone before the next step, as in the
  // plain decoding step
  const bool st = (size_t)s.B * s.H * s.D * s.M * sizeof(float) > device_l2_bytes() / 2;
  auto kern = st ? decay_decode_kernel<T, V, ROWS, WHOLE, true, kCols, kThreads, kMin>
                 : decay_decode_kernel<T, V, ROWS, WHOLE, false, kCols, kThreads, kMin>;
  kern<<<grid, kThreads, 0, stream>>>(
      static_cast<const T*>(f.q), static_cast<const T*>(f.k), static_cast<const T*>(f.v), f.g,
      f.slots, static_cast<T*>(f.out), f.state, f.pool, (int)s.H, (int)(s.H / s.Hk), (int)s.D,
      (int)s.M, s.scale);
  return cudaGetLastError();
}

template <typename T>
cudaError_t run(const DecayShape& s, const DecayDecode& f, cudaStream_t stream) {
  if (s.M % 4 != 0) {  // 4 row groups
    if (s.D <= 64) return launch<T, 1, 16, false, 32, 128, 1>(s, f, stream);
    return launch<T, 1, 64, false, 32, 128, 1>(s, f, stream);
  }
  // 16 row groups of four, eight or sixteen rows
  if (s.D % 8 != 0) {
    if (s.D <= 64) return launch<T, 4, 4, false, 32, 128, 1>(s, f, stream);
    return launch<T, 4, 16, false, 32, 128, 1>(s, f, stream);
  }
  if (s.M <= 32) {
    if (s.D <= 64) return launch<T, 4, 4, true, 32, 128, 8>(s, f, stream);
    if (s.D <= 128) return launch<T, 4, 8, true, 32, 128, 4>(s, f, stream);
  } else {
    if (s.D <= 64) return launch<T, 4, 4, true, 64, 256, 4>(s, f, stream);
    if (s.D <= 128) return launch<T, 4, 8, true, 64, 256, 2>(s, f, stream);
  }
  return launch<T, 4, 16, true, 32, 128, 1>(s, f, stream);
}

}  // namespace

cudaError_t decay_decode_launch(const DecayShape& s, const DecayDecode& f, cudaStream_t stream) {
  if (s.dtype == CP_DTYPE_BF16) return run<__nv_bfloat16>(s, f, stream);
  if (s.dtype == CP_DTYPE_F16) return run<__half>(s, f, stream);
  return run<float>(s, f, stream);
}

}  // namespace cp
