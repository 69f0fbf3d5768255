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
// reads and writes, so what counts is loads in flight and few instructions
// beside them: a row is held by D / 16 lanes, each with eight features and the
// eight they turn with (two 16-byte pieces of bf16 or fp16), so that the turn
// stays within a lane and a sum over the row takes few shuffles; as many rows
// to a warp as fit, two turns of them at once (backward: one), and the next
// ones loaded before these are worked on.  Where R or D is not a multiple of 16
// a lane has eight features, asks for their partners by shuffle and takes twice
// the turns (bf16, B = 8, H = 16, N = 2048, D = 64, cold: 33 + 54 us at R = 32, by
// pairs, 78 + 120 us at R = 40, by shuffles).  Everything between the load and the
// store is fp32 and rounded once.  bf16, B = 8, H = 16, N = 4096, D = 64, with
// weights, cold: at R = 16 forward 60 us, backward 105 us, at R = 64 62 and 102 us,
// 4.3 to 4.5 and 3.8 to 3.9 TB/s, and 5 us to join the weights' gradients.
// Registers hold the loads in flight, two CTAs to an SM, and not all of them: rows
// of fp32 take twice the registers of 16-bit ones at as many turns and spill 40
// bytes a thread forward, 60 backward (B = 8, H = 16, N = 2048, D = R = 64: 49 + 81
// us, 5.5 and 4.9 TB/s); the shuffles' copies spill 40 to 70 bytes for 16-bit rows,
// 184 and 236 for fp32 ones.
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
  int D, R, lanes;         // lanes of a row, a power of two
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

// FAST (R and D multiples of 16): the cosines and sines of a lane's eight
// features f0 .. of the turned ones' first half, dir = -1 turning back; the rest
// stands still.
__device__ __forceinline__ void load_angles(float2 (&c)[4], float2 (&s)[4], const float* cs,
                                            const float* sn, bool turned, int f0, bool wide,
                                            float dir) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    c[i] = both(1.f);
    s[i] = both(0.f);
  }
  if (!turned) return;
  const float2 d = both(dir);
  if (wide) {
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      const float4 x = *reinterpret_cast<const float4*>(cs + f0 + 2 * i);
      const float4 y = *reinterpret_cast<const float4*>(sn + f0 + 2 * i);
      c[i] = make_float2(x.x, x.y);
      c[i + 1] = make_float2(x.z, x.w);
      s[i] = mul2(d, make_float2(y.x, y.y));
      s[i + 1] = mul2(d, make_float2(y.z, y.w));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      c[i] = make_float2(cs[f0 + 2 * i], cs[f0 + 2 * i + 1]);
      s[i] = mul2(d, make_float2(sn[f0 + 2 * i], sn[f0 + 2 * i + 1]));
    }
  }
}
// the turn of the lane's two pieces
__device__ __forceinline__ void rotate8(float2 (&y)[2][4], const float2 (&c)[4],
                                        const float2 (&s)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 lo = y[0][i], hi = y[1][i];
    y[0][i] = fma2(hi, mul2(s[i], both(-1.f)), mul2(lo, c[i]));
    y[1][i] = fma2(lo, s[i], mul2(hi, c[i]));
  }
}

// Otherwise: those of the lane's eight features f0 .., wherever they lie, the
// sines with the rotation's sign, features from R on standing still ..
__device__ __forceinline__ void load_angles_any(float2 (&c)[4], float2 (&s)[4], const float* cs,
                                                const float* sn, int R, int f0, float dir) {
  const int half = R / 2;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    c[i] = both(1.f);
    s[i] = both(0.f);
  }
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
// .. and the turn of a row spread over `lanes` lanes (lane l: features 8 l ..):
// a feature f < R has its partner half = R / 2 away, in the lane half / 8 away or
// the next, at an offset that is the same for every lane: with the registers
// turned by half % 8 (three rounds of selects), each feature takes one shuffle
// from above and one from below.
__device__ __forceinline__ void rotate8_any(float2 (&y)[4], const float2 (&c)[4],
                                            const float2 (&s)[4], int R, int l, int lanes) {
  const int half = R / 2, f0 = 8 * l, o = half % 8;
  if (half == 0) return;
  const float* yf = reinterpret_cast<const float*>(y);
  float up[8], down[8];  // elements (i + o) % 8 and (i - o) % 8
#pragma unroll
  for (int i = 0; i < 8; ++i) up[i] = down[i] = yf[i];
#pragma unroll
  for (int n = 4; n > 0; n /= 2) {
    float u[8], d[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      u[i] = o & n ? up[(i + n) % 8] : up[i];
      d[i] = o & n ? down[(i + 8 - n) % 8] : down[i];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      up[i] = u[i];
      down[i] = d[i];
    }
  }
  float z[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float a = __shfl_sync(0xffffffffu, up[i], l + half / 8 + (i + o >= 8), lanes);
    const float b = __shfl_sync(0xffffffffu, down[i], l - half / 8 - (i < o), lanes);
    z[i] = f0 + i < half ? a : (f0 + i < R ? b : 0.f);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) y[i] = fma2(make_float2(z[2 * i], z[2 * i + 1]), s[i], mul2(y[i], c[i]));
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
  constexpr int P = FAST ? 2 : 1;         // a lane's pieces of eight features
  constexpr int U = (BWD ? 2 : 4) / P;    // turns in flight
  const Side& s = a.side[blockIdx.y];
  const int lanes = a.lanes, per_warp = 32 / lanes;
  const int lane = threadIdx.x % 32, w = threadIdx.x / 32, l = lane % lanes;
  const bool on = 8 * P * l < a.D;
  const T* x = static_cast<const T*>(s.x);
  T* y = static_cast<T*>(s.y);
  const T* gy = static_cast<const T*>(s.gy);
  // strided rows of 16-byte pieces at 16-byte addresses, or element loads
  const int64_t piece = 16 / sizeof(T);
  const bool wide = (reinterpret_cast<uintptr_t>(x) & 15) == 0 && s.sb % piece == 0 &&
                    s.sh % piece == 0 && s.sn % piece == 0;
  const int half = a.R / 2;
  // the pieces' first features: FAST pairs the turned features' halves, and
  // those of the rest
  int f[P];
  f[0] = 8 * l;
  const bool turned = 8 * l < half;  // (FAST)
  if constexpr (FAST) {
    f[1] = f[0] + half;
    if (!turned) {
      f[0] += half;
      f[1] = f[0] + (a.D - a.R) / 2;
    }
  }
  const bool wide_cs = ((reinterpret_cast<uintptr_t>(a.cos) | reinterpret_cast<uintptr_t>(a.sin)) & 15) == 0 &&
                       half % 4 == 0 && a.cs_batch % 4 == 0;
  float2 wt[P][4], dw[P][4];
#pragma unroll
  for (int e = 0; e < P; ++e)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      wt[e][i] = both(1.f);
      if (s.w != nullptr && on)
        wt[e][i] = make_float2(ld_f32<T>(static_cast<const T*>(s.w) + f[e] + 2 * i),
                               ld_f32<T>(static_cast<const T*>(s.w) + f[e] + 2 * i + 1));
      dw[e][i] = both(0.f);
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
    Raw8<T> x[U][P], g[BWD ? U : 1][P];
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
      const T* xr = x + at.b * s.sb + at.h * s.sh + at.n * s.sn;
      const T* gr = gy + (int64_t)q.out_row[u] * a.D;
#pragma unroll
      for (int e = 0; e < P; ++e) {
        q.x[u][e] = Raw8<T>{};
        if (q.live[u]) load8<T>(q.x[u][e], xr + f[e], wide);
        if constexpr (BWD) {
          q.g[u][e] = Raw8<T>{};
          if (q.live[u]) load8<T>(q.g[u][e], gr + f[e], true);
        }
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
        if constexpr (FAST)
          load_angles(c, si, a.cos + cs, a.sin + cs, q.live[u] && turned, 8 * l, wide_cs,
                      BWD ? -1.f : 1.f);
        else
          load_angles_any(c, si, a.cos + cs, a.sin + cs, q.live[u] ? a.R : 0, 8 * l,
                          BWD ? -1.f : 1.f);
      }
      const auto turn = [&](float2(&y8)[P][4]) {
        if constexpr (FAST) {
          // (what stands still is left alone: by a sine of 0, an infinite
          // feature would make its neighbour in the lane NaN)
          if (turned) rotate8(y8, c, si);
        } else
          rotate8_any(y8[0], c, si, a.R, l, lanes);
      };
      T* to = y + (int64_t)q.out_row[u] * a.D;
      float2 v[P][4];
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < P; ++e) {
        unpack8<T>(v[e], q.x[u][e]);
        ss += dot8(v[e], v[e]);
      }
      for (int o = lanes / 2; o > 0; o /= 2) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const float inv = rsqrtf(fmaf(a.c, ss, a.eps));  // 2 ulp
      if constexpr (!BWD) {
#pragma unroll
        for (int e = 0; e < P; ++e)
#pragma unroll
          for (int i = 0; i < 4; ++i) v[e][i] = mul2(v[e][i], mul2(both(inv), wt[e][i]));
        turn(v);
        if (q.live[u])
#pragma unroll
          for (int e = 0; e < P; ++e) store8<T>(to + f[e], v[e]);
      } else {
        float2 d[P][4];
#pragma unroll
        for (int e = 0; e < P; ++e) unpack8<T>(d[e], q.g[u][e]);
        turn(d);
        float xt = 0.f;
#pragma unroll
        for (int e = 0; e < P; ++e) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (q.live[u]) dw[e][i] = fma2(d[e][i], mul2(v[e][i], both(inv)), dw[e][i]);
            d[e][i] = mul2(d[e][i], wt[e][i]);
          }
          xt += dot8(v[e], d[e]);
        }
        for (int o = lanes / 2; o > 0; o /= 2) xt += __shfl_xor_sync(0xffffffffu, xt, o);
        const float2 m = both(-a.c * inv * inv * xt);
#pragma unroll
        for (int e = 0; e < P; ++e) {
#pragma unroll
          for (int i = 0; i < 4; ++i) d[e][i] = mul2(both(inv), fma2(m, v[e][i], d[e][i]));
          if (q.live[u]) store8<T>(to + f[e], d[e]);
        }
      }
    }
  }
  if constexpr (BWD) {
    if (s.w == nullptr) return;
    // rows of a warp, then the warps, in a fixed order
#pragma unroll
    for (int e = 0; e < P; ++e) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        for (int o = lanes; o < 32; o *= 2) {
          dw[e][i].x += __shfl_xor_sync(0xffffffffu, dw[e][i].x, o);
          dw[e][i].y += __shfl_xor_sync(0xffffffffu, dw[e][i].y, o);
        }
      if (lane < lanes && on)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          sm[w * a.D + f[e] + 2 * i] = dw[e][i].x;
          sm[w * a.D + f[e] + 2 * i + 1] = dw[e][i].y;
        }
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

int row_lanes(int64_t D, int features) {
  int l = 1;
  while (features * l < D) l *= 2;
  return l;
}

// one CTA of each side to an SM, two resident; fewer when the rows do not fill
// them
int n_blocks(const QkRope& f) {
  // (the smallest turn that a CTA takes: rows of eight features a lane)
  const int64_t per = kWarps * (32 / row_lanes(f.D, 8));
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
  const bool fast = f.R % 16 == 0 && f.D % 16 == 0;
  a.N = f.N; a.D = (int)f.D; a.R = (int)f.R; a.lanes = row_lanes(f.D, fast ? 16 : 8);
  a.c = f.rms ? 1.f / (float)f.D : 1.f;
  a.eps = f.eps;
  const dim3 grid((unsigned)n_blocks(f), 2);
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
