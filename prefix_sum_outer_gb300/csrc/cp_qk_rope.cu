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
// reads and writes, so what counts is loads in flight: a row is held by D/8
// lanes, eight features each (16 bytes of bf16 or fp16), as many rows to a warp
// as fit, a warp takes four rows to a lane group (backward: two) at once and
// loads the next four before it works on them.  The partner of a feature under the rotation comes from its
// lane by shuffle.  Everything between the load and the store is fp32 and
// rounded once.
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

// Eight features as they lie in memory.
template <typename T>
struct Raw8 {
  uint4 x[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ void load8(Raw8<T>& r, const T* p, bool wide) {
  if (wide) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.x[i] = reinterpret_cast<const uint4*>(p)[i];
  } else {
    T* e = reinterpret_cast<T*>(&r);
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = p[i];
  }
}
template <typename T>
__device__ __forceinline__ void unpack8(float2 (&v)[4], const Raw8<T>& r) {
  const T* e = reinterpret_cast<const T*>(&r);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = make_float2(ld_f32<T>(e + 2 * i), ld_f32<T>(e + 2 * i + 1));
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float2 (&v)[4]) {
  Raw8<T> r;
  T* e = reinterpret_cast<T*>(&r);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    e[2 * i] = from_f32<T>(v[i].x);
    e[2 * i + 1] = from_f32<T>(v[i].y);
  }
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) reinterpret_cast<uint4*>(p)[i] = r.x[i];
}
__device__ __forceinline__ float dot8(const float2 (&x)[4], const float2 (&y)[4]) {
  float2 s = mul2(x[0], y[0]);
#pragma unroll
  for (int i = 1; i < 4; ++i) s = fma2(x[i], y[i], s);
  return s.x + s.y;
}

// The cosines of a lane's eight features and their sines with the rotation's
// sign (dir = -1 turns back); features from R on stand still.  FAST: R/2 is a
// multiple of 8, so the lane's features all lie in one half.
template <bool FAST>
__device__ __forceinline__ void load_angles(float2 (&c)[4], float2 (&s)[4], const float* cs,
                                            const float* sn, int R, int f0, bool wide, float dir) {
  const int half = R / 2;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    c[i] = both(1.f);
    s[i] = both(0.f);
  }
  if constexpr (FAST) {
    if (f0 >= R) return;
    const int a = f0 < half ? f0 : f0 - half;
    const float2 d = both(f0 < half ? -dir : dir);
    if (wide) {
#pragma unroll
      for (int i = 0; i < 4; i += 2) {
        const float4 x = *reinterpret_cast<const float4*>(cs + a + 2 * i);
        const float4 y = *reinterpret_cast<const float4*>(sn + a + 2 * i);
        c[i] = make_float2(x.x, x.y);
        c[i + 1] = make_float2(x.z, x.w);
        s[i] = mul2(d, make_float2(y.x, y.y));
        s[i + 1] = mul2(d, make_float2(y.z, y.w));
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        c[i] = make_float2(cs[a + 2 * i], cs[a + 2 * i + 1]);
        s[i] = mul2(d, make_float2(sn[a + 2 * i], sn[a + 2 * i + 1]));
      }
    }
  } else {
    float* cf = reinterpret_cast<float*>(c);
    float* sf = reinterpret_cast<float*>(s);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int f = f0 + i;
      if (f < R) {
        cf[i] = cs[f < half ? f : f - half];
        sf[i] = (f < half ? -dir : dir) * sn[f < half ? f : f - half];
      }
    }
  }
}

// Turn a row spread over `lanes` lanes (lane l: features 8 l ..).  A feature f <
// R has its partner R/2 away: with FAST the whole lanes trade, otherwise every
// feature asks for its partner's lane in turn.
template <bool FAST>
__device__ __forceinline__ void rotate8(float2 (&y)[4], const float2 (&c)[4], const float2 (&s)[4],
                                        int R, int l, int lanes) {
  const int half = R / 2, f0 = 8 * l;
  if (half == 0) return;
  if constexpr (FAST) {
    const int src = f0 >= R ? l : (f0 < half ? l + half / 8 : l - half / 8);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 z = make_float2(__shfl_sync(0xffffffffu, y[i].x, src, lanes),
                                   __shfl_sync(0xffffffffu, y[i].y, src, lanes));
      y[i] = fma2(z, s[i], mul2(y[i], c[i]));
    }
  } else {
    float* yf = reinterpret_cast<float*>(y);
    float z[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int f = f0 + i, want = f < half ? f + half : (f < R ? f - half : f);
      z[i] = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float t = __shfl_sync(0xffffffffu, yf[j], want / 8, lanes);
        if (want % 8 == j) z[i] = t;
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = fma2(make_float2(z[2 * i], z[2 * i + 1]), s[i], mul2(y[i], c[i]));
  }
}

// A row's place: token (batch b, position n) and head, advanced by a fixed
// number of rows without a division.
struct Place {
  uint32_t b, h, n;
};

// Rows are taken token by token (all heads of a token, then the next), so the
// lanes of a warp share a token's angles and read neighbouring input rows.
template <typename T, bool BWD, bool FAST>
__global__ void __launch_bounds__(kThreads, 2) qk_rope_kernel(Args a) {
  extern __shared__ float sm[];  // BWD: [kWarps][D] partial weight gradients
  constexpr int U = FAST ? (BWD ? 2 : 4) : 1;  // turns in flight
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
  const int half = a.R / 2;
  const bool wide_cs = ((reinterpret_cast<uintptr_t>(a.cos) | reinterpret_cast<uintptr_t>(a.sin)) & 15) == 0 &&
                       half % 4 == 0 && a.cs_batch % 4 == 0;
  float2 wt[4], dw[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    wt[i] = both(1.f);
    if (s.w != nullptr && on)
      wt[i] = make_float2(ld_f32<T>(static_cast<const T*>(s.w) + 8 * l + 2 * i),
                          ld_f32<T>(static_cast<const T*>(s.w) + 8 * l + 2 * i + 1));
    dw[i] = both(0.f);
  }
  // a warp takes U x per_warp consecutive rows, then jumps by `step`
  const uint32_t step = gridDim.x * kWarps * per_warp * U;  // (at most 152 x 8 x 32 x 4)
  const uint32_t H = (uint32_t)s.H, N = (uint32_t)a.N;
  const bool per_batch = a.cs_batch != 0;
  const uint32_t step_tok = step / H, step_h = step % H;
  int64_t r_warp = ((int64_t)blockIdx.x * kWarps + w) * per_warp * U;
  Place base;
  {
    const int64_t r = r_warp + lane / lanes, tok = r / s.H;
    base.h = (uint32_t)(r % s.H);
    base.b = (uint32_t)(tok / a.N);
    base.n = (uint32_t)(tok % a.N);
  }
  // a turn's rows, as loaded
  struct Turn {
    Raw8<T> x[U], g[BWD ? U : 1];
    uint32_t out_row[U], tok[U];  // rows of the output, of the angles
    bool live[U];
  };
  auto load_turn = [&](Turn& q) {
    Place at = base;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      q.live[u] = r_warp + u * per_warp + lane / lanes < s.rows && on;
      q.out_row[u] = (at.b * H + at.h) * N + at.n;
      q.tok[u] = (per_batch ? at.b * N : 0) + at.n;
      q.x[u] = Raw8<T>{};
      if constexpr (BWD) q.g[u] = Raw8<T>{};
      if (q.live[u]) {
        load8<T>(q.x[u], x + at.b * s.sb + at.h * s.sh + at.n * s.sn + 8 * l, wide);
        if constexpr (BWD) load8<T>(q.g[u], gy + (int64_t)q.out_row[u] * a.D + 8 * l, true);
      }
      at.h += per_warp;
      while (at.h >= H) {
        at.h -= H;
        if (++at.n == N) {
          at.n = 0;
          ++at.b;
        }
      }
    }
    base.h += step_h;
    base.n += step_tok;
    if (base.h >= H) {
      base.h -= H;
      ++base.n;
    }
    if (base.n >= N) {
      base.b += base.n / N;
      base.n %= N;
    }
    r_warp += step;
  };
  // every lane of a warp walks the same number of turns: the shuffles need all
  bool more = r_warp < s.rows;
  Turn next;
  if (more) load_turn(next);
  while (more) {
    const Turn q = next;
    more = r_warp < s.rows;
    if (more) load_turn(next);  // under this turn's arithmetic
    float2 c[4], si[4];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      // a token's heads share its angles
      if (u == 0 || q.tok[u] != q.tok[u - 1]) {
        const int64_t cs = per_batch ? q.tok[u] / N * a.cs_batch + (int64_t)(q.tok[u] % N) * half
                                     : (int64_t)q.tok[u] * half;
        load_angles<FAST>(c, si, a.cos + cs, a.sin + cs, q.live[u] ? a.R : 0, 8 * l, wide_cs,
                          BWD ? -1.f : 1.f);
      }
      T* to = y + (int64_t)q.out_row[u] * a.D + 8 * l;
      float2 v[4];
      unpack8<T>(v, q.x[u]);
      float ss = dot8(v, v);
      for (int o = lanes / 2; o > 0; o /= 2) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const float inv = rsqrtf(fmaf(a.c, ss, a.eps));  // 2 ulp
      if constexpr (!BWD) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = mul2(v[i], mul2(both(inv), wt[i]));
        rotate8<FAST>(v, c, si, a.R, l, lanes);
        if (q.live[u]) store8<T>(to, v);
      } else {
        float2 d[4];
        unpack8<T>(d, q.g[u]);
        rotate8<FAST>(d, c, si, a.R, l, lanes);
        if (q.live[u])
#pragma unroll
          for (int i = 0; i < 4; ++i) dw[i] = fma2(d[i], mul2(v[i], both(inv)), dw[i]);
#pragma unroll
        for (int i = 0; i < 4; ++i) d[i] = mul2(d[i], wt[i]);
        float xt = dot8(v, d);
        for (int o = lanes / 2; o > 0; o /= 2) xt += __shfl_xor_sync(0xffffffffu, xt, o);
        const float2 m = both(-a.c * inv * inv * xt);
#pragma unroll
        for (int i = 0; i < 4; ++i) d[i] = mul2(both(inv), fma2(m, v[i], d[i]));
        if (q.live[u]) store8<T>(to, d);
      }
    }
  }
  if constexpr (BWD) {
    if (s.w == nullptr) return;
    // rows of a warp, then the warps, in a fixed order
#pragma unroll
    for (int i = 0; i < 4; ++i)
      for (int o = lanes; o < 32; o *= 2) {
        dw[i].x += __shfl_xor_sync(0xffffffffu, dw[i].x, o);
        dw[i].y += __shfl_xor_sync(0xffffffffu, dw[i].y, o);
      }
    if (lane < lanes && on)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        sm[w * a.D + 8 * l + 2 * i] = dw[i].x;
        sm[w * a.D + 8 * l + 2 * i + 1] = dw[i].y;
      }
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

// one CTA of each side to an SM, two resident; fewer when the rows do not fill
// them
int n_blocks(const QkRope& f) {
  // (a CTA's turn; the kernel takes up to four of them at once)
  const int64_t per = kWarps * (32 / row_lanes(f.D));
  const int64_t rows = f.B * f.N * std::max(f.Hq, f.Hk);
  return (int)std::min<int64_t>((rows + per - 1) / per, kPlanSMs);
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
  const bool fast = f.R % 16 == 0;
  if (!backward) {
    (fast ? qk_rope_kernel<T, false, true> : qk_rope_kernel<T, false, false>)<<<grid, kThreads, 0, stream>>>(a);
    return cudaGetLastError();
  }
  (fast ? qk_rope_kernel<T, true, true> : qk_rope_kernel<T, true, false>)<<<grid, kThreads, kWarps * f.D * sizeof(float), stream>>>(a);
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
