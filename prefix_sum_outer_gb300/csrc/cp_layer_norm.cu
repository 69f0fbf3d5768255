// Layer norm of rows of C features, with its gradients: for a row x of mean mu,
// r = (mean (x - mu)^2 + eps)^-1/2 and xh = (x - mu) r,
//     y  = xh w + b;      t = gy w,   dx = r (t - mean t - xh mean (t xh)),
//     dw = sum over rows of gy xh,    db = sum over rows of gy.
// A row is held in registers by a group of threads (4 lanes to a whole CTA), so
// it is read once in each pass, and the variance is taken of x - mu, in fp32.
// The traffic bounds both passes: x and y, or x, gy and dx.
//
// Backward, a group takes every so-many-th row of one head and keeps the sums of
// the weight's and the bias's gradient for its columns in fp32 registers; a CTA's
// groups join them in shared memory, the CTAs' parts go to the workspace and are
// summed in order by a second launch, so results are the same every time.  No
// statistics are kept from the forward: the row is in registers anyway.
#include <algorithm>

#include "cp_delta.cuh"

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
    w = i % 2 ? (w & 0xffffu) | (s << 16) : (w & 0xffff0000u) | s;
  }
};

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

// Sums of NS values over a row's group: GL lanes, or a CTA of whole warps
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
    __syncthreads();
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
  __shared__ float red[1][33];
  const int G = MULTI ? blockDim.x : GL;
  const int t = threadIdx.x % G, grp = threadIdx.x / G, groups = blockDim.x / G;
  const int h = blockIdx.y;
  const T* x = static_cast<const T*>(a.x) + h * a.sh;
  T* y = static_cast<T*>(a.y) + h * a.yh;
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
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < KV; ++i)
#pragma unroll
      for (int e = 0; e < VEC; ++e) s[0] += raw[r][i].get(e);
    group_sum<GL, MULTI, 1>(s, red);
    const float mu = s[0] * inv;
    s[0] = 0.f;
#pragma unroll
    for (int i = 0; i < KV; ++i)
      if ((i * G + t) * VEC < a.C)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float d = raw[r][i].get(e) - mu;
          s[0] = fmaf(d, d, s[0]);
        }
    group_sum<GL, MULTI, 1>(s, red);
    const float rs = rsqrtf(fmaf(s[0], inv, a.eps));
    if (at[r] >= 0) {
      const T* w = a.w == nullptr ? nullptr : static_cast<const T*>(a.w) + h * a.w_head;
      const T* b = a.b == nullptr ? nullptr : static_cast<const T*>(a.b) + h * a.w_head;
#pragma unroll
      for (int i = 0; i < KV; ++i) {
        const int c = (i * G + t) * VEC;
        if (c < a.C) {
          Raw<T, VEC> o, ww, bb;
          if (w != nullptr) ww = load<T, VEC>(w + c);
          if (b != nullptr) bb = load<T, VEC>(b + c);
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            const float xh = (raw[r][i].get(e) - mu) * rs;
            o.set(e, fmaf(xh, w != nullptr ? ww.get(e) : 1.f, b != nullptr ? bb.get(e) : 0.f));
          }
          *reinterpret_cast<Raw<T, VEC>*>(y + at[r] + c) = o;
        }
      }
    }
  }
}

template <typename T, int VEC, int GL, int KV, int MT>
__global__ void __launch_bounds__(MT > 0 ? MT : kBwdThreads) layer_norm_bwd_kernel(const Args a) {
  constexpr bool MULTI = MT > 0;
  constexpr int E = KV * VEC;
  extern __shared__ float sums[];  // [2][groups][G * E], unless MULTI
  __shared__ float red[2][33];
  const int G = MULTI ? blockDim.x : GL;
  const int t = threadIdx.x % G, grp = threadIdx.x / G, groups = blockDim.x / G;
  const int h = blockIdx.y;
  const T* x = static_cast<const T*>(a.x) + h * a.sh;
  const T* gy = static_cast<const T*>(a.gy) + h * a.yh;
  T* dx = static_cast<T*>(a.dx) + (int64_t)h * a.N * a.C;
  const T* w = a.w == nullptr ? nullptr : static_cast<const T*>(a.w) + h * a.w_head;
  const float inv = 1.f / (float)a.C;
  float dw[E] = {}, db[E] = {};
  Raw<T, VEC> nx[KV], ng[KV];
  // a row's loads go out under the arithmetic of the row before it
  auto fetch = [&](unsigned row) {
    if (row < a.rows) {
      const unsigned b = row / a.n, n = row - b * a.n;
      const T *px = x + b * a.sb + n * a.sn, *pg = gy + b * a.yb + n * a.yn;
#pragma unroll
      for (int i = 0; i < KV; ++i) {
        const int c = (i * G + t) * VEC;
        if (c < a.C) {
          nx[i] = load<T, VEC>(px + c);
          ng[i] = load<T, VEC>(pg + c);
        } else {
          nx[i] = ng[i] = zero<T, VEC>();
        }
      }
    }
  };
  const unsigned step = gridDim.x * groups;
  unsigned row = blockIdx.x * groups + grp;
  fetch(row);
  // every group of a warp makes as many turns (shuffles span the warp)
  for (unsigned first = blockIdx.x * groups; first < a.rows; first += step, row += step) {
    const bool on = row < a.rows;
    float xh[E];
    Raw<T, VEC> g[KV];
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < KV; ++i) {
      g[i] = ng[i];
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        xh[i * VEC + e] = on ? nx[i].get(e) : 0.f;
        s[0] += xh[i * VEC + e];
      }
    }
    if (row + step > row) fetch(row + step);
    float m[1] = {s[0]};
    group_sum<GL, MULTI, 1>(m, red);
    const float mu = m[0] * inv;
    m[0] = 0.f;
#pragma unroll
    for (int i = 0; i < KV; ++i)
      if ((i * G + t) * VEC < a.C)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          float& d = xh[i * VEC + e];
          d -= mu;
          m[0] = fmaf(d, d, m[0]);
        }
    group_sum<GL, MULTI, 1>(m, red);
    const float rs = rsqrtf(fmaf(m[0], inv, a.eps));
    s[0] = 0.f;
#pragma unroll
    for (int i = 0; i < KV; ++i) {
      const int c = (i * G + t) * VEC;
      Raw<T, VEC> ww;
      if (w != nullptr && c < a.C) ww = load<T, VEC>(w + c);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        float& xx = xh[i * VEC + e];
        xx *= rs;
        const float gg = on && c < a.C ? g[i].get(e) : 0.f;
        const float tt = w != nullptr && c < a.C ? gg * ww.get(e) : gg;
        s[0] += tt;
        s[1] = fmaf(tt, xx, s[1]);
        if (on) {
          dw[i * VEC + e] = fmaf(gg, xx, dw[i * VEC + e]);
          db[i * VEC + e] += gg;
        }
      }
    }
    group_sum<GL, MULTI, 2>(s, red);
    const float s0 = s[0] * inv, s1 = s[1] * inv;
    if (on) {
      const unsigned b = row / a.n, n = row - b * a.n;
      T* p = dx + ((int64_t)b * a.H * a.N + n) * a.C;
#pragma unroll
      for (int i = 0; i < KV; ++i) {
        const int c = (i * G + t) * VEC;
        if (c < a.C) {
          Raw<T, VEC> o, ww;
          if (w != nullptr) ww = load<T, VEC>(w + c);
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            const float gg = g[i].get(e), tt = w != nullptr ? gg * ww.get(e) : gg;
            o.set(e, rs * (tt - s0 - xh[i * VEC + e] * s1));
          }
          *reinterpret_cast<Raw<T, VEC>*>(p + c) = o;
        }
      }
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
          part[c] = dw[i * VEC + e];
          part[a.C + c] = db[i * VEC + e];
        }
      }
  } else {
    const int width = G * E;
#pragma unroll
    for (int i = 0; i < KV; ++i)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const int c = (i * G + t) * VEC + e;
        sums[grp * width + c] = dw[i * VEC + e];
        sums[(groups + grp) * width + c] = db[i * VEC + e];
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
// CTA, eight lines of parts
template <typename T>
__global__ void __launch_bounds__(256)
    layer_norm_join_kernel(const float* __restrict__ part, T* dw, T* db, int P, int C) {
  __shared__ float s[2][8][33];
  const int lane = threadIdx.x % 32, line = threadIdx.x / 32, c = blockIdx.x * 32 + lane;
  const float* p = part + (int64_t)blockIdx.y * P * 2 * C;
  float x = 0.f, y = 0.f;
  if (c < C)
#pragma unroll 4
    for (int i = line; i < P; i += 8) {
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
      for (int i = 0; i < 8; ++i) z += s[line][i][lane];
      to[(int64_t)blockIdx.y * C + c] = from_f32<T>(z);
    }
  }
}

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// How a row is shared out: vectors of 16 bytes where every row starts on such a
// boundary, else elements; G threads of KV of them.  The backward holds three
// more numbers to an element, so a thread of it takes half as many.
struct Split {
  bool vec;
  int G, KV;
};
Split split(int64_t n, bool vec, bool backward) {  // n: vectors or elements of a row
  if (vec) {
    for (int G = 4; G <= 32; G *= 2)
      if (n <= G) return {true, G, 1};
    if (n <= 64) return {true, 32, 2};
    if (n <= 128) return {true, 32, 4};
    for (int G = 64; G <= 512; G *= 2)
      if (n <= (backward ? 2 : 4) * G) return {true, G, backward ? 2 : 4};
    if (n <= 2048) return {true, 512, 4};
    return {true, 1024, n <= 4096 ? 4 : 8};
  }
  if (n <= 128) return {false, 32, 4};
  if (n <= 512) return {false, 32, 16};
  for (int G = 64; G <= 1024; G *= 2)
    if (n <= 16 * G) return {false, G, 16};
  return {false, 1024, 32};
}

// CTAs to a head in the backward: a few rounds of warps to an SM, and no more
// than there are rows.  Of the sizes alone, as the workspace is.
int64_t bwd_ctas(const LayerNorm& f, int G) {
  const int64_t groups = G > 32 ? 1 : kBwdThreads / G;
  const int64_t want = (int64_t)kPlanSMs * std::max<int64_t>(1, 16 * 32 / std::max(G, kBwdThreads));
  const int64_t rows = (f.B * f.N + groups - 1) / groups;
  return std::max<int64_t>(1, std::min<int64_t>(rows, (want + f.H - 1) / f.H));
}

template <typename T, int VEC, int GL, int KV, int MT>
cudaError_t forward(const LayerNorm& f, const Args& a, cudaStream_t stream) {
  const int threads = MT > 0 ? a.G : 256;
  const int64_t per = (int64_t)kRpt<VEC, KV, MT> * (threads / (MT > 0 ? a.G : GL));
  const dim3 grid((unsigned)((a.rows + per - 1) / per), (unsigned)f.H);
  layer_norm_fwd_kernel<T, VEC, GL, KV, MT><<<grid, threads, 0, stream>>>(a);
  return cudaGetLastError();
}

template <typename T, int VEC, int GL, int KV, int MT>
cudaError_t backward(const LayerNorm& f, const Args& a, cudaStream_t stream) {
  const int threads = MT > 0 ? a.G : kBwdThreads;
  const unsigned ctas = (unsigned)bwd_ctas(f, a.G);
  const size_t smem =
      MT > 0 || a.part == nullptr ? 0 : (size_t)2 * threads * KV * VEC * sizeof(float);
  layer_norm_bwd_kernel<T, VEC, GL, KV, MT>
      <<<dim3(ctas, (unsigned)f.H), threads, smem, stream>>>(a);
  if (a.part != nullptr) {
    const int heads = f.per_head ? (int)f.H : 1;
    layer_norm_join_kernel<T><<<dim3((unsigned)((f.C + 31) / 32), heads), 256, 0, stream>>>(
        a.part, static_cast<T*>(f.dw), static_cast<T*>(f.db), (int)(ctas * f.H / heads), a.C);
  }
  return cudaGetLastError();
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
    if (s.G == 4) return forward<T, V, 4, 1, 0>(f, a, stream);
    if (s.G == 8) return forward<T, V, 8, 1, 0>(f, a, stream);
    if (s.G == 16) return forward<T, V, 16, 1, 0>(f, a, stream);
    if (s.KV == 1) return forward<T, V, 32, 1, 0>(f, a, stream);
    if (s.KV == 2) return forward<T, V, 32, 2, 0>(f, a, stream);
    return forward<T, V, 32, 4, 0>(f, a, stream);
  }
  a.part = f.dw != nullptr || f.db != nullptr ? static_cast<float*>(scratch) : nullptr;
  if (!vec) {
    if (s.KV == 32) return backward<T, 1, 32, 32, 1024>(f, a, stream);
    if (s.G > 512) return backward<T, 1, 32, 16, 1024>(f, a, stream);
    if (s.G > 32) return backward<T, 1, 32, 16, 512>(f, a, stream);
    return s.KV == 4 ? backward<T, 1, 32, 4, 0>(f, a, stream)
                     : backward<T, 1, 32, 16, 0>(f, a, stream);
  }
  if constexpr (V == 4)
    if (s.KV == 8) return backward<T, V, 32, 8, 1024>(f, a, stream);
  if (s.G > 512) return backward<T, V, 32, 4, 1024>(f, a, stream);
  if (s.G > 32)
    return s.KV == 2 ? backward<T, V, 32, 2, 512>(f, a, stream)
                     : backward<T, V, 32, 4, 512>(f, a, stream);
  if (s.G == 4) return backward<T, V, 4, 1, 0>(f, a, stream);
  if (s.G == 8) return backward<T, V, 8, 1, 0>(f, a, stream);
  if (s.G == 16) return backward<T, V, 16, 1, 0>(f, a, stream);
  if (s.KV == 1) return backward<T, V, 32, 1, 0>(f, a, stream);
  if (s.KV == 2) return backward<T, V, 32, 2, 0>(f, a, stream);
  return backward<T, V, 32, 4, 0>(f, a, stream);
}

}  // namespace

// Whether rows move as vectors is known at the call alone: room for either.
size_t layer_norm_scratch(const LayerNorm& f) {
  const int64_t V = f.dtype == CP_DTYPE_F32 ? 4 : 8;
  int64_t ctas = bwd_ctas(f, split(f.C, false, true).G);
  if (f.C % V == 0) ctas = std::max(ctas, bwd_ctas(f, split(f.C / V, true, true).G));
  return (size_t)ctas * f.H * 2 * f.C * sizeof(float);
}

cudaError_t layer_norm_launch(const LayerNorm& f, void* scratch, bool backward,
                              cudaStream_t stream) {
  if (f.dtype == CP_DTYPE_BF16) return run<__nv_bfloat16>(f, scratch, backward, stream);
  if (f.dtype == CP_DTYPE_F16) return run<__half>(f, scratch, backward, stream);
  return run<float>(f, scratch, backward, stream);
}

}  // namespace cp
