// The norm of queries and keys per head with the position rotation, in one
// pass over the rows:
//     y = w o x r,   r = (c sum x^2 + eps)^-1/2,   c = 1/D (rms) or 1 (l2),
// then features (i, i + R/2), i < R/2, of the first R turned by the token's
// angles: (y1 cos - y2 sin, y2 cos + y1 sin).  Backward, with d the output's
// gradient turned back:
//     dw = sum over rows of d o x r,   t = w o d,   dx = r (t - c r^2 x (x . t)).
//
// Input rows may have any strides (the projection's token-major rows, read in
// place); output rows are head-major and dense, as the products take them, so
// the transposition costs nothing beside the norm.  The pass is bound by its
// reads and writes.  A row is held by D/8 lanes, eight features each (16 bytes
// of bf16 or fp16), as many rows to a warp as fit; the partner of a feature
// under the rotation comes from its lane by shuffle.  Everything between the
// load and the store is fp32 and rounded once.
#include <algorithm>

#include "cp_delta.cuh"

namespace cp {
namespace {

using namespace delta;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

struct Side {          // queries or keys
  const void* x;
  const void* w;       // [D], or null
  const void* gy;      // [B][H][N][D]
  void* y;             // [B][H][N][D]: the output, or dx
  int64_t sb, sh, sn;  // strides of x, elements
  int64_t rows;        // B * H * N
  int H;
};

struct Args {
  Side side[2];
  const float *cos, *sin;  // [B or 1][N][R/2]
  int64_t cs_batch;        // elements between batches (0: shared)
  float* dw_part;          // [2][blocks][D]
  int64_t N;
  int D, R, lanes;         // lanes of a row: D / 8 rounded up to a power of two
  float c, eps;
};

template <typename T>
__device__ __forceinline__ void load8(float (&r)[8], const T* p, bool wide) {
  if constexpr (sizeof(T) == 4) {
    if (wide) {
      const float4 a = *reinterpret_cast<const float4*>(p);
      const float4 b = *reinterpret_cast<const float4*>(p + 4);
      r[0] = a.x; r[1] = a.y; r[2] = a.z; r[3] = a.w;
      r[4] = b.x; r[5] = b.y; r[6] = b.z; r[7] = b.w;
      return;
    }
  } else {
    if (wide) {
      const uint4 a = *reinterpret_cast<const uint4*>(p);
      const T* e = reinterpret_cast<const T*>(&a);
#pragma unroll
      for (int i = 0; i < 8; ++i) r[i] = ld_f32<T>(e + i);
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = ld_f32<T>(p + i);
}

template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&r)[8]) {
  if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<float4*>(p) = make_float4(r[0], r[1], r[2], r[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(r[4], r[5], r[6], r[7]);
  } else {
    uint4 a;
    T* e = reinterpret_cast<T*>(&a);
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = from_f32<T>(r[i]);
    *reinterpret_cast<uint4*>(p) = a;
  }
}

// Turn a row spread over `lanes` lanes (lane l: features 8 l ..) by the angles
// at cs, sn; dir = -1 turns back.  A feature i < R has its partner R/2 away.
// With R/2 a multiple of 8 the partners are whole lanes; otherwise they are
// fetched one by one.
__device__ __forceinline__ void rotate8(float (&y)[8], const float* cs, const float* sn, int R,
                                        int l, int lanes, float dir) {
  const int half = R / 2, f0 = 8 * l;
  if (half == 0) return;
  float z[8];
  if (half % 8 == 0) {
    const bool low = f0 < half, in = f0 < R;
    const int src = in ? (low ? l + half / 8 : l - half / 8) : l;
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = __shfl_sync(0xffffffffu, y[i], src, lanes);
    if (in) {
      const int a0 = low ? f0 : f0 - half;
      const float s = low ? -dir : dir;
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = fmaf(y[i], cs[a0 + i], s * z[i] * sn[a0 + i]);
    }
    return;
  }
  // partner of feature f0 + i: which lane, and which of its eight
#pragma unroll
  for (int i = 0; i < 8; ++i) z[i] = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int f = f0 + i, want = f < half ? f + half : (f < R ? f - half : f);
    // every lane asks for slot j of lane want / 8 in turn
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float t = __shfl_sync(0xffffffffu, y[j], want / 8, lanes);
      if (want % 8 == j) z[i] = t;
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int f = f0 + i;
    if (f < R) {
      const int a = f < half ? f : f - half;
      const float s = f < half ? -dir : dir;
      y[i] = fmaf(y[i], cs[a], s * z[i] * sn[a]);
    }
  }
}

// Rows are taken token by token (all heads of a token, then the next), so the
// lanes of a warp share a token's angles and read neighbouring input rows.
template <typename T, bool BWD>
__global__ void __launch_bounds__(kThreads) qk_rope_kernel(Args a) {
  extern __shared__ float sm[];  // BWD: [kWarps][D] partial weight gradients
  const Side& s = a.side[blockIdx.y];
  const int lanes = a.lanes, per_warp = 32 / lanes;
  const int lane = threadIdx.x % 32, w = threadIdx.x / 32, l = lane % lanes;
  const bool on = 8 * l < a.D;
  const T* x = static_cast<const T*>(s.x);
  T* y = static_cast<T*>(s.y);
  const T* gy = static_cast<const T*>(s.gy);
  // strided rows of 16-byte pieces at 16-byte addresses, or element loads
  const int64_t piece = 16 / sizeof(T);
  const bool wide = (reinterpret_cast<uintptr_t>(x) & 15) == 0 && s.sb % piece == 0 &&
                    s.sh % piece == 0 && s.sn % piece == 0;
  float wt[8], dw[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    wt[i] = s.w != nullptr && on ? ld_f32<T>(static_cast<const T*>(s.w) + 8 * l + i) : 1.f;
    dw[i] = 0.f;
  }
  const int64_t step = (int64_t)gridDim.x * kWarps * per_warp;
  // every lane of a warp walks the same number of rows: the shuffles need all
  for (int64_t r0 = ((int64_t)blockIdx.x * kWarps + w) * per_warp; r0 < s.rows; r0 += step) {
    const int64_t r = r0 + lane / lanes;
    const bool live = r < s.rows && on;
    const int64_t rr = min(r, s.rows - 1), tok = rr / s.H;
    const int h = (int)(rr % s.H);
    const int64_t b = tok / a.N, n = tok % a.N;
    const float* cs = a.cos + b * a.cs_batch + n * (a.R / 2);
    const float* sn = a.sin + b * a.cs_batch + n * (a.R / 2);
    const int64_t to = ((b * s.H + h) * a.N + n) * a.D + 8 * l;
    float v[8] = {};
    if (live) load8<T>(v, x + b * s.sb + h * s.sh + n * s.sn + 8 * l, wide);
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(v[i], v[i], ss);
    for (int o = lanes / 2; o > 0; o /= 2) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float inv = 1.f / sqrtf(fmaf(a.c, ss, a.eps));
    if constexpr (!BWD) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = v[i] * inv * wt[i];
      rotate8(v, cs, sn, a.R, l, lanes, 1.f);
      if (live) store8<T>(y + to, v);
    } else {
      float d[8] = {};
      if (live) load8<T>(d, gy + to, true);
      rotate8(d, cs, sn, a.R, l, lanes, -1.f);
      float xt = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (live) dw[i] = fmaf(d[i], v[i] * inv, dw[i]);
        d[i] *= wt[i];
        xt = fmaf(v[i], d[i], xt);
      }
      for (int o = lanes / 2; o > 0; o /= 2) xt += __shfl_xor_sync(0xffffffffu, xt, o);
      const float m = a.c * inv * inv * xt;
#pragma unroll
      for (int i = 0; i < 8; ++i) d[i] = inv * fmaf(-m, v[i], d[i]);
      if (live) store8<T>(y + to, d);
    }
  }
  if constexpr (BWD) {
    if (s.w == nullptr) return;
    // rows of a warp, then the warps, in a fixed order
#pragma unroll
    for (int i = 0; i < 8; ++i)
      for (int o = lanes; o < 32; o *= 2) dw[i] += __shfl_xor_sync(0xffffffffu, dw[i], o);
    if (lane < lanes && on)
#pragma unroll
      for (int i = 0; i < 8; ++i) sm[w * a.D + 8 * l + i] = dw[i];
    __syncthreads();
    for (int d = threadIdx.x; d < a.D; d += kThreads) {
      float t = 0.f;
      for (int i = 0; i < kWarps; ++i) t += sm[i * a.D + d];
      a.dw_part[((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * a.D + d] = t;
    }
  }
}

// dw[d] = sum over the blocks of dw_part[side][block][d]: one CTA per side and
// feature
template <typename T>
__global__ void __launch_bounds__(128)
    qk_rope_join_kernel(const float* __restrict__ part, T* dwq, T* dwk, int blocks, int D) {
  __shared__ float red[4];
  T* out = blockIdx.y == 0 ? dwq : dwk;
  if (out == nullptr) return;
  const float* p = part + (int64_t)blockIdx.y * blocks * D + blockIdx.x;
  float s = 0.f;
  for (int i = threadIdx.x; i < blocks; i += 128) s += p[(int64_t)i * D];
  for (int o = 16; o > 0; o /= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = s;
  __syncthreads();
  if (threadIdx.x == 0) out[blockIdx.x] = from_f32<T>(red[0] + red[1] + red[2] + red[3]);
}

int row_lanes(int64_t D) {
  int l = 1;
  while (8 * l < D) l *= 2;
  return l;
}

// four CTAs to an SM, fewer when the rows do not fill them
int n_blocks(const QkRope& f) {
  const int64_t per = kWarps * (32 / row_lanes(f.D));
  const int64_t rows = f.B * f.N * std::max(f.Hq, f.Hk);
  return (int)std::min<int64_t>((rows + per - 1) / per, 4 * kPlanSMs);
}

template <typename T>
cudaError_t run(const QkRope& f, float* scratch, bool backward, cudaStream_t stream) {
  Args a{};
  for (int i = 0; i < 2; ++i) {
    Side& s = a.side[i];
    s.x = i ? f.xk : f.xq;
    s.w = i ? f.wk : f.wq;
    s.gy = i ? f.gk : f.gq;
    s.y = i ? f.yk : f.yq;
    s.H = (int)(i ? f.Hk : f.Hq);
    s.rows = f.B * f.N * s.H;
    const int64_t* st = i ? f.stride_k : f.stride_q;
    s.sb = st[0]; s.sh = st[1]; s.sn = st[2];
  }
  a.cos = f.cos; a.sin = f.sin; a.cs_batch = f.cs_batch;
  a.dw_part = scratch;
  a.N = f.N; a.D = (int)f.D; a.R = (int)f.R; a.lanes = row_lanes(f.D);
  a.c = f.rms ? 1.f / (float)f.D : 1.f;
  a.eps = f.eps;
  const dim3 grid((unsigned)n_blocks(f), 2);
  if (!backward) {
    qk_rope_kernel<T, false><<<grid, kThreads, 0, stream>>>(a);
    return cudaGetLastError();
  }
  qk_rope_kernel<T, true><<<grid, kThreads, kWarps * f.D * sizeof(float), stream>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || (f.dwq == nullptr && f.dwk == nullptr)) return e;
  qk_rope_join_kernel<T><<<dim3((unsigned)f.D, 2), 128, 0, stream>>>(
      scratch, static_cast<T*>(f.dwq), static_cast<T*>(f.dwk), (int)grid.x, (int)f.D);
  return cudaGetLastError();
}

}  // namespace

size_t qk_rope_scratch(const QkRope& f) {
  return f.B * f.N == 0 ? 0 : sizeof(float) * 2 * (size_t)n_blocks(f) * f.D;
}

cudaError_t qk_rope_launch(const QkRope& f, void* scratch, bool backward, cudaStream_t stream) {
  float* s = static_cast<float*>(scratch);
  if (f.dtype == CP_DTYPE_BF16) return run<__nv_bfloat16>(f, s, backward, stream);
  if (f.dtype == CP_DTYPE_F16) return run<__half>(f, s, backward, stream);
  return run<float>(f, s, backward, stream);
}

}  // namespace cp
