// Layer norm of rows of C features, with its gradients: for a row x of mean mu,
// r = (mean (x - mu)^2 + eps)^-1/2 and xh = (x - mu) r,
//     y  = xh w + b;      t = gy w,   dx = r (t - mean t - xh mean (t xh)),
//     dw = sum over rows of gy xh,    db = sum over rows of gy.
// A row is held in registers by a group of threads (4 lanes to a whole CTA), so
// it is read once in each pass, and the variance is taken of x - mu, in fp32.
// The traffic bounds both passes: x and y, or x, gy and dx.  bf16 B=8 H=16 N=4096
// C=64 by heads: forward 28 us (4.8 TB/s), backward 42 (4.8) and its join 5, 74 back to
// back; 32,768 rows of 1,024 73.
//
// Backward, a group takes every so-many-th row of one head and keeps the sums of
// the weight's and the bias's gradient for its columns in fp32 registers; a CTA's
// groups join them in shared memory, the CTAs' parts go to the workspace and are
// summed in order by a second launch, so results are the same every time.  No
// statistics are kept from the forward: the row is in registers anyway.
#include <algorithm>
#include <atomic>

#include "cp_delta.cuh"
#include "sm103_ptx.cuh"

namespace cp {
namespace {

using namespace delta;  // element loads and stores

constexpr int kBwdThreads = 128;  // of a backward CTA whose rows take a warp or less

struct Args {
  const void *x, *w, *b, *gy;
  void *y, *dx;
  float* part;             // [H][gridDim.x][2][C]
  int64_t sb, sh, sn;      // strides of x
  int64_t yb, yh, yn;      // of y and gy
  int64_t N;
  unsigned rows, n;        // rows of a head; N as 32 bits (rows < 2^31)
  int H, C, G;
  int64_t w_head;          // elements between heads' weights
  float eps;
};

// VEC dense elements as they lie in memory
template <typename T, int VEC>
struct Raw;
template <typename T>
struct Raw<T, 1> {
  T x;
  __device__ __forceinline__ float get(int) const { return ld_f32<T>(&x); }
  __device__ __forceinline__ void set(int, float f) { x = from_f32<T>(f); }
};
template <>
struct Raw<float, 4> {
  float4 x;
  __device__ __forceinline__ float get(int i) const { return (&x.x)[i]; }
  __device__ __forceinline__ void set(int i, float f) { (&x.x)[i] = f; }
};
template <typename T>
struct Raw<T, 8> {
  uint4 x;
  __device__ __forceinline__ float get(int i) const {
    const uint32_t w = (&x.x)[i / 2];
    const unsigned short s = (unsigned short)(i % 2 ? w >> 16 : w);
    return ld_f32<T>(reinterpret_cast<const T*>(&s));
  }
  __device__ __forceinline__ void set(int i, float f) {
    const T t = from_f32<T>(f);
    const uint32_t s = *reinterpret_cast<const unsigned short*>(&t);
    uint32_t& w = (&x.x)[i / 2];
    w = i % 2 ? (w & 0xffffu) | (s << 16) : s;  // (the even one goes first)
  }
};

// Arithmetic on a vector's elements in fp32.  16-bit elements enter it by the
// mixed-precision instructions, two of a word at a time: shifts and masks that
// widen them, done at each of their three uses, would take half of the backward's
// time.
#define CP_MIXED_OPS(TYPE, NAME)                                                              \
  __device__ __forceinline__ float2 plus(TYPE, uint32_t a, float2 c) { /* a + c */            \
    float2 r;                                                                                 \
    asm("{\n\t.reg .b16 x, y;\n\tmov.b32 {x, y}, %2;\n\tadd.rn.f32." NAME " %0, x, %3;\n\t"     \
        "add.rn.f32." NAME " %1, y, %4;\n\t}"                                                 \
        : "=f"(r.x), "=f"(r.y) : "r"(a), "f"(c.x), "f"(c.y));                                 \
    return r;                                                                                 \
  }                                                                                           \
  __device__ __forceinline__ float2 minus(TYPE, uint32_t a, float c) { /* a - c */            \
    float2 r;                                                                                 \
    asm("{\n\t.reg .b16 x, y;\n\tmov.b32 {x, y}, %2;\n\tsub.rn.f32." NAME " %0, x, %3;\n\t"     \
        "sub.rn.f32." NAME " %1, y, %3;\n\t}"                                                 \
        : "=f"(r.x), "=f"(r.y) : "r"(a), "f"(c));                                             \
    return r;                                                                                 \
  }                                                                                           \
  __device__ __forceinline__ float2 times(TYPE, uint32_t a, uint32_t b, float2 c) { /* ab + c */ \
    float2 r;                                                                                 \
    asm("{\n\t.reg .b16 x, y, u, v;\n\tmov.b32 {x, y}, %2;\n\tmov.b32 {u, v}, %3;\n\t"          \
        "fma.rn.f32." NAME " %0, x, u, %4;\n\tfma.rn.f32." NAME " %1, y, v, %5;\n\t}"         \
        : "=f"(r.x), "=f"(r.y) : "r"(a), "r"(b), "f"(c.x), "f"(c.y));                         \
    return r;                                                                                 \
  }
CP_MIXED_OPS(__nv_bfloat16, "bf16")
CP_MIXED_OPS(__half, "f16")
#undef CP_MIXED_OPS
constexpr float2 kZero2 = {0.f, 0.f};

// s += x (two running sums)
template <typename T, int VEC>
__device__ __forceinline__ void sum_into(float2& s, const Raw<T, VEC>& x) {
  if constexpr (VEC == 8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) s = plus(T(), (&x.x.x)[i], s);
  } else if constexpr (VEC == 4) {
    s = add2(add2(s, make_float2(x.x.x, x.x.y)), make_float2(x.x.z, x.x.w));
  } else {
    s.x += x.get(0);
  }
}
// x - c
template <typename T, int VEC>
__device__ __forceinline__ void diff(float (&d)[VEC], const Raw<T, VEC>& x, float c) {
  if constexpr (VEC == 8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 r = minus(T(), (&x.x.x)[i], c);
      d[2 * i] = r.x;
      d[2 * i + 1] = r.y;
    }
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e) d[e] = x.get(e) - c;
  }
}
// g w, or without W g
template <bool W, typename T, int VEC>
__device__ __forceinline__ void product(float (&t)[VEC], const Raw<T, VEC>& g, const Raw<T, VEC>& w) {
  if constexpr (VEC == 8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float2 r;
      if constexpr (W) r = times(T(), (&g.x.x)[i], (&w.x.x)[i], kZero2);
      else r = plus(T(), (&g.x.x)[i], kZero2);
      t[2 * i] = r.x;
      t[2 * i + 1] = r.y;
    }
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e) t[e] = W ? g.get(e) * w.get(e) : g.get(e);
  }
}
// s += g w, or without W g (two running sums)
template <bool W, typename T, int VEC>
__device__ __forceinline__ void sum_product_into(float2& s, const Raw<T, VEC>& g, const Raw<T, VEC>& w) {
  if constexpr (!W) {
    sum_into(s, g);
  } else if constexpr (VEC == 8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) s = times(T(), (&g.x.x)[i], (&w.x.x)[i], s);
  } else if constexpr (VEC == 4) {
    s = fma2(make_float2(g.x.x, g.x.y), make_float2(w.x.x, w.x.y), s);
    s = fma2(make_float2(g.x.z, g.x.w), make_float2(w.x.z, w.x.w), s);
  } else {
    s.x = fmaf(g.get(0), w.get(0), s.x);
  }
}

template <typename T, int VEC>
__device__ __forceinline__ Raw<T, VEC> load(const T* p) {
  return *reinterpret_cast<const Raw<T, VEC>*>(p);
}
template <typename T, int VEC>
__device__ __forceinline__ Raw<T, VEC> zero() {
  Raw<T, VEC> r;
#pragma unroll
  for (int i = 0; i < VEC; ++i) r.set(i, 0.f);
  return r;
}

// Sums of NS values over a row's group: GL lanes, or a CTA of whole warps, whose
// parts meet in `red`.  (A row's two sums have a `red` each, so the barrier of the
// one keeps the next row's from the other's readers.)
template <int GL, bool MULTI, int NS>
__device__ __forceinline__ void group_sum(float (&v)[NS], float (*red)[33]) {
#pragma unroll
  for (int o = GL / 2; o > 0; o /= 2)
#pragma unroll
    for (int i = 0; i < NS; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  if constexpr (MULTI) {
    const int w = threadIdx.x / 32, lane = threadIdx.x % 32, nw = blockDim.x / 32;
    if (lane == 0)
#pragma unroll
      for (int i = 0; i < NS; ++i) red[i][w] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      v[i] = lane < nw ? red[i][lane] : 0.f;
#pragma unroll
      for (int o = 16; o > 0; o /= 2) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    }
  }
}

// KV vectors of a row to a thread, RPT rows at a time
template <int VEC, int KV, int MT>
constexpr int kRpt = MT > 0 || KV * VEC >= 32 ? 1 : 32 / (KV * VEC) > 4 ? 4 : 32 / (KV * VEC);

// MT: a row takes a CTA of at most so many threads; 0: a warp or less
template <typename T, int VEC, int GL, int KV, int MT>
__global__ void __launch_bounds__(MT > 0 ? MT : 256) layer_norm_fwd_kernel(const Args a) {
  constexpr bool MULTI = MT > 0;
  constexpr int RPT = kRpt<VEC, KV, MT>;
  __shared__ float red[2][1][33];
  const int G = MULTI ? blockDim.x : GL;
  const int t = threadIdx.x % G, grp = threadIdx.x / G, groups = blockDim.x / G;
  const int h = blockIdx.y;
  const T* x = static_cast<const T*>(a.x) + h * a.sh;
  T* y = static_cast<T*>(a.y) + h * a.yh;
  ptx::grid_dep_wait();
  Raw<T, VEC> raw[RPT][KV];
  int64_t at[RPT];
#pragma unroll
  for (int r = 0; r < RPT; ++r) {
    const unsigned row = (blockIdx.x * RPT + r) * groups + grp;
    at[r] = -1;
    if (row < a.rows) {
      const unsigned b = row / a.n, n = row - b * a.n;
      const T* p = x + b * a.sb + n * a.sn;
      at[r] = b * a.yb + n * a.yn;
#pragma unroll
      for (int i = 0; i < KV; ++i) {
        const int c = (i * G + t) * VEC;
        raw[r][i] = c < a.C ? load<T, VEC>(p + c) : zero<T, VEC>();
      }
    } else {
#pragma unroll
      for (int i = 0; i < KV; ++i) raw[r][i] = zero<T, VEC>();
    }
  }
  const float inv = 1.f / (float)a.C;
#pragma unroll
  for (int r = 0; r < RPT; ++r) {
    float2 two = kZero2;
#pragma unroll
    for (int i = 0; i < KV; ++i) sum_into(two, raw[r][i]);
    float s[1] = {two.x + two.y};
    group_sum<GL, MULTI, 1>(s, red[0]);
    const float mu = s[0] * inv;
    s[0] = 0.f;
#pragma unroll
    for (int i = 0; i < KV; ++i)
      if ((i * G + t) * VEC < a.C) {
        float d[VEC];
        diff(d, raw[r][i], mu);
#pragma unroll
        for (int e = 0; e < VEC; ++e) s[0] = fmaf(d[e], d[e], s[0]);
      }
    group_sum<GL, MULTI, 1>(s, red[1]);
    const float rs = rsqrtf(fmaf(s[0], inv, a.eps));
    if (at[r] >= 0) {
      const T* w = a.w == nullptr ? nullptr : static_cast<const T*>(a.w) + h * a.w_head;
      const T* b = a.b == nullptr ? nullptr : static_cast<const T*>(a.b) + h * a.w_head;
#pragma unroll
      for (int i = 0; i < KV; ++i) {
        const int c = (i * G + t) * VEC;
        if (c < a.C) {
          Raw<T, VEC> o, ww, bb;
          float d[VEC], fw[VEC], fb[VEC];
          diff(d, raw[r][i], mu);
          if (w != nullptr) {
            ww = load<T, VEC>(w + c);
            product<false>(fw, ww, ww);
          }
          if (b != nullptr) {
            bb = load<T, VEC>(b + c);
            product<false>(fb, bb, bb);
          }
#pragma unroll
          for (int e = 0; e < VEC; ++e)
            o.set(e, fmaf(d[e] * rs, w != nullptr ? fw[e] : 1.f, b != nullptr ? fb[e] : 0.f));
          *reinterpret_cast<Raw<T, VEC>*>(y + at[r] + c) = o;
        }
      }
    }
  }
}

// CTAs to an SM: with 16 elements to a thread four, which leave it 128 registers (two:
// 90 against 80 us forward and backward, bf16 B=8 H=16 N=4096 C=64); with 32 the sums
// and the rows at hand and ahead fill those by themselves: two.
template <int VEC, int KV, int MT>
constexpr int kBwdMin = MT > 0 ? (MT <= 512 ? 512 / MT : 1) : KV * VEC <= 8 ? 8 : KV * VEC <= 16 ? 4 : 2;

// Rows first, first + step, ... of a head's B * N: a row's offset in a tensor goes
// by steps, without a division a row.
struct Walk {
  int64_t at, by, wrap;  // elements
  __device__ __forceinline__ Walk(const Args& a, unsigned row, unsigned sb, unsigned sn, int64_t b,
                                  int64_t n)
      : at((row / a.n) * b + (row % a.n) * n), by(sb * b + sn * n), wrap(b - a.n * n) {}
};

// WEIGHTED: there is a w.  SUMS: where the weight's and the bias's gradients
// gather: shared memory (a CTA to a row, whose threads would not hold them beside
// the row) or registers
template <typename T, int VEC, int GL, int KV, int MT, bool SUMS, bool WEIGHTED>
__global__ void __launch_bounds__(MT > 0 ? MT : kBwdThreads, kBwdMin<VEC, KV, MT>)
    layer_norm_bwd_kernel(const Args a) {
  constexpr bool MULTI = MT > 0, AHEAD = VEC > 1;
  constexpr int E = KV * VEC;
  constexpr int W = VEC > 1 ? 4 : 1;  // floats to an access of the sums
  extern __shared__ __align__(16) float sums[];  // SUMS: [2][E / W][G][W]; else [2][groups][G * E]
  __shared__ float red[2][2][33];
  const int G = MULTI ? blockDim.x : GL;
  const int t = threadIdx.x % G, grp = threadIdx.x / G, groups = blockDim.x / G;
  const int h = blockIdx.y;
  const T* w = static_cast<const T*>(a.w) + (WEIGHTED ? h * a.w_head + t * VEC : 0);
  const float inv = 1.f / (float)a.C;
  float dw[SUMS ? 1 : E] = {}, db[SUMS ? 1 : E] = {};
  auto place = [&](int which, int e) { return sums + ((which * (E / W) + e / W) * G + t) * W; };
  ptx::grid_dep_wait();
  if constexpr (SUMS) {
    for (int i = threadIdx.x; i < 2 * E * G; i += blockDim.x) sums[i] = 0.f;
    __syncthreads();
  }
  const unsigned step = gridDim.x * groups, sb = step / a.n, sn = step % a.n;
  unsigned row = blockIdx.x * groups + grp;
  unsigned n_now = row % a.n, n_next = n_now;
  // x and gy of the row to load, dx of the row at hand
  Walk wx(a, row, sb, sn, a.sb, a.sn), wg(a, row, sb, sn, a.yb, a.yn);
  Walk wd(a, row, sb, sn, (int64_t)a.H * a.N * a.C, a.C);
  const T* x = static_cast<const T*>(a.x) + h * a.sh + t * VEC;
  const T* gy = static_cast<const T*>(a.gy) + h * a.yh + t * VEC;
  T* dx = static_cast<T*>(a.dx) + (int64_t)h * a.N * a.C + t * VEC;
  bool in[KV];
#pragma unroll
  for (int i = 0; i < KV; ++i) in[i] = (i * G + t) * VEC < a.C;
  Raw<T, VEC> nx[KV], ng[KV];
  unsigned left = row < a.rows ? (a.rows - 1 - row) / step + 1 : 0;  // rows of this group
  unsigned to_load = left;
  auto fetch = [&]() {
#pragma unroll
    for (int i = 0; i < KV; ++i) {
      if (to_load > 0 && in[i]) {
        nx[i] = load<T, VEC>(x + wx.at + i * G * VEC);
        ng[i] = load<T, VEC>(gy + wg.at + i * G * VEC);
      } else {
        nx[i] = ng[i] = zero<T, VEC>();
      }
    }
    if (to_load > 0) --to_load;
    n_next += sn;
    const bool over = n_next >= a.n;
    n_next -= over ? a.n : 0;
    wx.at += wx.by + (over ? wx.wrap : 0);
    wg.at += wg.by + (over ? wg.wrap : 0);
  };
  if constexpr (AHEAD) fetch();
  // every group of a warp makes as many turns (shuffles span the warp)
  const unsigned first = blockIdx.x * groups;
  unsigned turns = first < a.rows ? (a.rows - 1 - first) / step + 1 : 0;
#pragma unroll 1
  for (; turns > 0; --turns) {
    Raw<T, VEC> xr[KV], g[KV];
    if constexpr (!AHEAD) fetch();
#pragma unroll
    for (int i = 0; i < KV; ++i) {
      xr[i] = nx[i];
      g[i] = ng[i];
    }
    // a row's loads go out under the arithmetic of the row before it
    if constexpr (AHEAD) fetch();
    // sums of x and of t = gy w
    float2 sx = kZero2, st = kZero2;
    Raw<T, VEC> ww[KV];
#pragma unroll
    for (int i = 0; i < KV; ++i) {
      if constexpr (WEIGHTED) ww[i] = in[i] ? load<T, VEC>(w + i * G * VEC) : zero<T, VEC>();
      sum_into(sx, xr[i]);
      sum_product_into<WEIGHTED>(st, g[i], ww[i]);
    }
    float s[2] = {sx.x + sx.y, st.x + st.y};
    group_sum<GL, MULTI, 2>(s, red[0]);
    const float mu = s[0] * inv, s0 = s[1] * inv;
    // of d = x - mu squared and of t d
    sx = st = kZero2;
#pragma unroll
    for (int i = 0; i < KV; ++i) {
      if (!in[i]) continue;
      float tt[VEC], d[VEC];
      product<WEIGHTED>(tt, g[i], ww[i]);
      diff(d, xr[i], mu);
      if constexpr (VEC > 1) {
#pragma unroll
        for (int e = 0; e < VEC; e += 2) {
          const float2 dd = make_float2(d[e], d[e + 1]);
          sx = fma2(dd, dd, sx);
          st = fma2(dd, make_float2(tt[e], tt[e + 1]), st);
        }
      } else {
        sx.x = fmaf(d[0], d[0], sx.x);
        st.x = fmaf(d[0], tt[0], st.x);
      }
    }
    s[0] = sx.x + sx.y;
    s[1] = st.x + st.y;
    group_sum<GL, MULTI, 2>(s, red[1]);
    const float rs = rsqrtf(fmaf(s[0], inv, a.eps)), s1 = s[1] * rs * inv;
    if (left > 0) {
      --left;
#pragma unroll
      for (int i = 0; i < KV; ++i) {
        if (!in[i]) continue;
        float tt[VEC], gg[VEC], out[VEC], d[VEC];
        product<WEIGHTED>(tt, g[i], ww[i]);
        product<false>(gg, g[i], g[i]);
        diff(d, xr[i], mu);
        if constexpr (VEC > 1) {
#pragma unroll
          for (int e = 0; e < VEC; e += 2) {
            const float2 xx = mul2(make_float2(d[e], d[e + 1]), both(rs));
            // rs (tt - s0 - xx s1)
            const float2 y = mul2(both(rs), fma2(xx, both(-s1), add2(make_float2(tt[e], tt[e + 1]), both(-s0))));
            d[e] = xx.x;
            d[e + 1] = xx.y;
            out[e] = y.x;
            out[e + 1] = y.y;
          }
        } else {
          d[0] *= rs;
          out[0] = rs * fmaf(d[0], -s1, tt[0] - s0);
        }
        Raw<T, VEC> o;
#pragma unroll
        for (int e = 0; e < VEC; ++e) o.set(e, out[e]);
        *reinterpret_cast<Raw<T, VEC>*>(dx + wd.at + i * G * VEC) = o;
#pragma unroll
        for (int e0 = 0; e0 < VEC; e0 += W) {
          if constexpr (SUMS) {
            float *qw = place(0, i * VEC + e0), *qb = place(1, i * VEC + e0);
            if constexpr (W == 4) {
              float4 z = *reinterpret_cast<float4*>(qw), y = *reinterpret_cast<float4*>(qb);
              z.x = fmaf(gg[e0], d[e0], z.x);
              z.y = fmaf(gg[e0 + 1], d[e0 + 1], z.y);
              z.z = fmaf(gg[e0 + 2], d[e0 + 2], z.z);
              z.w = fmaf(gg[e0 + 3], d[e0 + 3], z.w);
              y.x += gg[e0]; y.y += gg[e0 + 1]; y.z += gg[e0 + 2]; y.w += gg[e0 + 3];
              *reinterpret_cast<float4*>(qw) = z;
              *reinterpret_cast<float4*>(qb) = y;
            } else {
              *qw = fmaf(gg[e0], d[e0], *qw);
              *qb += gg[e0];
            }
          } else if constexpr (W == 4) {
#pragma unroll
            for (int e = e0; e < e0 + 4; e += 2) {
              const int j = SUMS ? 0 : i * VEC + e, k = SUMS ? 0 : j + 1;
              const float2 z = fma2(make_float2(gg[e], gg[e + 1]), make_float2(d[e], d[e + 1]),
                                    make_float2(dw[j], dw[k]));
              const float2 y = add2(make_float2(gg[e], gg[e + 1]), make_float2(db[j], db[k]));
              dw[j] = z.x; dw[k] = z.y; db[j] = y.x; db[k] = y.y;
            }
          } else {
            const int j = SUMS ? 0 : i * VEC + e0;
            dw[j] = fmaf(gg[e0], d[e0], dw[j]);
            db[j] += gg[e0];
          }
        }
      }
      n_now += sn;
      const bool over = n_now >= a.n;
      n_now -= over ? a.n : 0;
      wd.at += wd.by + (over ? wd.wrap : 0);
    }
  }
  if (a.part == nullptr) return;
  float* part = a.part + ((int64_t)h * gridDim.x + blockIdx.x) * 2 * a.C;
  if constexpr (MULTI) {
#pragma unroll
    for (int i = 0; i < KV; ++i)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const int c = (i * G + t) * VEC + e;
        if (c < a.C) {
          part[c] = SUMS ? place(0, i * VEC + e)[e % W] : dw[SUMS ? 0 : i * VEC + e];
          part[a.C + c] = SUMS ? place(1, i * VEC + e)[e % W] : db[SUMS ? 0 : i * VEC + e];
        }
      }
  } else {
    const int width = G * E;
#pragma unroll
    for (int i = 0; i < KV; ++i)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const int c = (i * G + t) * VEC + e;
        sums[grp * width + c] = dw[SUMS ? 0 : i * VEC + e];
        sums[(groups + grp) * width + c] = db[SUMS ? 0 : i * VEC + e];
      }
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * width; c += blockDim.x) {
      const int which = c / width, col = c % width;
      if (col >= a.C) continue;
      float s = 0.f;
      for (int i = 0; i < groups; ++i) s += sums[(which * groups + i) * width + col];
      part[which * a.C + col] = s;
    }
  }
}

// The parts [P][2][C] of blockIdx.y's weights, summed in order: 32 columns to a
// CTA, 32 lines of parts
constexpr int kLines = 32;
template <typename T>
__global__ void __launch_bounds__(32 * kLines)
    layer_norm_join_kernel(const float* part, T* dw, T* db, int P, int C) {
  __shared__ float s[2][kLines][33];
  const int lane = threadIdx.x % 32, line = threadIdx.x / 32, c = blockIdx.x * 32 + lane;
  const float* p = part + (int64_t)blockIdx.y * P * 2 * C;
  float x = 0.f, y = 0.f;
  ptx::grid_dep_wait();
  if (c < C)
#pragma unroll 4
    for (int i = line; i < P; i += kLines) {
      x += p[(int64_t)i * 2 * C + c];
      y += p[(int64_t)i * 2 * C + C + c];
    }
  s[0][line][lane] = x;
  s[1][line][lane] = y;
  __syncthreads();
  if (line < 2 && c < C) {
    T* to = line == 0 ? dw : db;
    if (to != nullptr) {
      float z = 0.f;
#pragma unroll
      for (int i = 0; i < kLines; ++i) z += s[line][i][lane];
      to[(int64_t)blockIdx.y * C + c] = from_f32<T>(z);
    }
  }
}

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// How a row is shared out: vectors of 16 bytes where every row starts on such a
// boundary, else elements; G threads of KV of them.
// In the backward a thread of several warps' rows takes half as many, so that the
// sums of its columns stay in registers, up to rows of 1024 vectors.
struct Split {
  bool vec;
  int G, KV;
};
Split split(int64_t n, bool vec, bool backward) {  // n: vectors or elements of a row
  if (vec) {
    if (n <= 4) return {true, 4, 1};
    for (int G = 4; G <= 32; G *= 2)
      if (n <= 2 * G) return {true, G, 2};
    if (n <= 128) return {true, 32, 4};
    if (backward)
      for (int G = 128; G <= 512; G *= 2)
        if (n <= 2 * G) return {true, G, 2};
    for (int G = 64; G <= 1024; G *= 2)
      if (n <= 4 * G) return {true, G, 4};
    return {true, 1024, 8};
  }
  if (n <= 128) return {false, 32, 4};
  for (int G = 32; G <= 1024; G *= 2)
    if (n <= 16 * G) return {false, G, 16};
  return {false, 1024, 32};
}

// CTAs to a head in the backward: as many as an SM holds, and no more than there
// are rows.  Of the sizes alone, as the workspace is.
int64_t bwd_ctas(const LayerNorm& f, const Split& s, int64_t V) {
  const int64_t E = s.KV * (s.vec ? V : 1), groups = s.G > 32 ? 1 : kBwdThreads / s.G;
  const int64_t per_sm = s.G > 32 ? std::max(1, 512 / s.G) : E <= 8 ? 8 : E <= 16 ? 4 : 2;
  const int64_t rows = (f.B * f.N + groups - 1) / groups;
  return std::max<int64_t>(1, std::min<int64_t>(rows, (kPlanSMs * per_sm + f.H - 1) / f.H));
}

template <typename T, int VEC, int GL, int KV, int MT>
cudaError_t forward(const LayerNorm& f, const Args& a, cudaStream_t stream) {
  const int threads = MT > 0 ? a.G : 256;
  const int64_t per = (int64_t)kRpt<VEC, KV, MT> * (threads / (MT > 0 ? a.G : GL));
  const dim3 grid((unsigned)((a.rows + per - 1) / per), (unsigned)f.H);
  return launch_dependent(layer_norm_fwd_kernel<T, VEC, GL, KV, MT>, grid, threads, 0, stream, a);
}

template <typename T, int VEC, int GL, int KV, int MT, bool SUMS = false>
cudaError_t backward(const LayerNorm& f, const Args& a, const Split& s, cudaStream_t stream) {
  const int threads = MT > 0 ? a.G : kBwdThreads;
  const unsigned ctas = (unsigned)bwd_ctas(f, s, 16 / sizeof(T));
  const size_t smem = SUMS || (MT == 0 && a.part != nullptr)
                          ? (size_t)2 * threads * KV * VEC * sizeof(float) : 0;
  auto kern = f.w != nullptr ? layer_norm_bwd_kernel<T, VEC, GL, KV, MT, SUMS, true>
                             : layer_norm_bwd_kernel<T, VEC, GL, KV, MT, SUMS, false>;
  if constexpr (SUMS) {
    // more than 48 KB wants asking for, once per device
    static std::atomic<uint64_t> asked_with{0}, asked_without{0};
    std::atomic<uint64_t>& asked = f.w != nullptr ? asked_with : asked_without;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if ((asked.load(std::memory_order_acquire) & bit) == 0) {
      e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               2 * MT * KV * VEC * (int)sizeof(float));
      if (e != cudaSuccess) return e;
      asked.fetch_or(bit, std::memory_order_release);
    }
  }
  cudaError_t e = launch_dependent(kern, dim3(ctas, (unsigned)f.H), threads, smem, stream, a);
  if (e != cudaSuccess || a.part == nullptr) return e;
  const int heads = f.per_head ? (int)f.H : 1;
  return launch_dependent(layer_norm_join_kernel<T>, dim3((unsigned)((f.C + 31) / 32), heads),
                          32 * kLines, 0, stream, a.part, static_cast<T*>(f.dw),
                          static_cast<T*>(f.db), (int)(ctas * f.H / heads), a.C);
}

template <typename T>
cudaError_t run(const LayerNorm& f, void* scratch, bool back, cudaStream_t stream) {
  constexpr int V = 16 / sizeof(T);
  Args a{};
  a.x = f.x; a.w = f.w; a.b = f.b; a.gy = f.gy; a.y = f.y; a.dx = f.dx;
  a.sb = f.stride[0]; a.sh = f.stride[1]; a.sn = f.stride[2];
  a.N = f.N; a.rows = (unsigned)(f.B * f.N); a.n = (unsigned)f.N;
  a.H = (int)f.H; a.C = (int)f.C; a.eps = f.eps;
  a.w_head = f.per_head ? f.C : 0;
  a.yb = f.H * f.N * f.C;
  a.yh = f.token_major ? f.C : f.N * f.C;
  a.yn = f.token_major ? f.H * f.C : f.C;
  bool vec = f.C % V == 0;
  for (const void* p : {f.x, f.w, f.b}) vec = vec && aligned(p, 16);
  for (int64_t s : {a.sb, a.sh, a.sn}) vec = vec && s % V == 0;
  const Split s = split(vec ? f.C / V : f.C, vec, back);
  a.G = s.G;
  if (!back) {
    if (!vec) {
      if (s.KV == 32) return forward<T, 1, 32, 32, 1024>(f, a, stream);
      if (s.G > 32) return forward<T, 1, 32, 16, 1024>(f, a, stream);
      return s.KV == 4 ? forward<T, 1, 32, 4, 0>(f, a, stream)
                       : forward<T, 1, 32, 16, 0>(f, a, stream);
    }
    if constexpr (V == 4)
      if (s.KV == 8) return forward<T, V, 32, 8, 1024>(f, a, stream);
    if (s.G > 512) return forward<T, V, 32, 4, 1024>(f, a, stream);
    if (s.G > 32) return forward<T, V, 32, 4, 512>(f, a, stream);
    if (s.KV == 1) return forward<T, V, 4, 1, 0>(f, a, stream);
    if (s.G == 4) return forward<T, V, 4, 2, 0>(f, a, stream);
    if (s.G == 8) return forward<T, V, 8, 2, 0>(f, a, stream);
    if (s.G == 16) return forward<T, V, 16, 2, 0>(f, a, stream);
    if (s.KV == 2) return forward<T, V, 32, 2, 0>(f, a, stream);
    return forward<T, V, 32, 4, 0>(f, a, stream);
  }
  a.part = f.dw != nullptr || f.db != nullptr ? static_cast<float*>(scratch) : nullptr;
  // (2 E fp32 sums a thread: 128 KB of shared memory for 16,384 features; past
  // that they stay in registers, and some of them in local memory)
  if (!vec) {
    if (s.KV == 32) return backward<T, 1, 32, 32, 1024>(f, a, s, stream);
    if (s.G > 512) return backward<T, 1, 32, 16, 1024, true>(f, a, s, stream);
    if (s.G > 32) return backward<T, 1, 32, 16, 512, true>(f, a, s, stream);
    return s.KV == 4 ? backward<T, 1, 32, 4, 0>(f, a, s, stream)
                     : backward<T, 1, 32, 16, 0>(f, a, s, stream);
  }
  if constexpr (V == 4)
    if (s.KV == 8) return backward<T, V, 32, 8, 1024>(f, a, s, stream);
  if (s.G > 512) return backward<T, V, 32, 4, 1024, V == 4>(f, a, s, stream);
  if (s.KV == 4 && s.G > 32) return backward<T, V, 32, 4, 512, true>(f, a, s, stream);
  if (s.G > 256) return backward<T, V, 32, 2, 512>(f, a, s, stream);
  if (s.G > 128) return backward<T, V, 32, 2, 256>(f, a, s, stream);
  if (s.G > 32) return backward<T, V, 32, 2, 128>(f, a, s, stream);
  if (s.KV == 1) return backward<T, V, 4, 1, 0>(f, a, s, stream);
  if (s.G == 4) return backward<T, V, 4, 2, 0>(f, a, s, stream);
  if (s.G == 8) return backward<T, V, 8, 2, 0>(f, a, s, stream);
  if (s.G == 16) return backward<T, V, 16, 2, 0>(f, a, s, stream);
  if (s.KV == 2) return backward<T, V, 32, 2, 0>(f, a, s, stream);
  return backward<T, V, 32, 4, 0>(f, a, s, stream);
}

}  // namespace

// Whether rows move as vectors is known at the call alone: room for either.
size_t layer_norm_scratch(const LayerNorm& f) {
  const int64_t V = f.dtype == CP_DTYPE_F32 ? 4 : 8;
  int64_t ctas = bwd_ctas(f, split(f.C, false, true), V);
  if (f.C % V == 0) ctas = std::max(ctas, bwd_ctas(f, split(f.C / V, true, true), V));
  return (size_t)ctas * f.H * 2 * f.C * sizeof(float);
}

cudaError_t layer_norm_launch(const LayerNorm& f, void* scratch, bool backward,
                              cudaStream_t stream) {
  if (f.dtype == CP_DTYPE_BF16) return run<__nv_bfloat16>(f, scratch, backward, stream);
  if (f.dtype == CP_DTYPE_F16) return run<__half>(f, scratch, backward, stream);
  return run<float>(f, scratch, backward, stream);
}

}  // namespace cp
