// Linear attention with a decay for each head on the CUDA cores, any dtype, fp32
// throughout (formulas in cp_decay.cuh): chunks of 64 rows in three launches,
//   sums    each chunk's sum_j a^{n-1-j} k_j v_j^T (backward: and sum_i a^i q_i
//           go_i^T), a CTA per chunk and 64 x 64 block of the state;
//   prefix  the states before the chunks, in place, a thread per element of the
//           state (one fma a chunk, the decay as hi + lo);
//   out     the chunks' rows from their decayed scores and the state, a CTA per
//           chunk and 64 columns.
// A sequence of one chunk needs no prefix: out reads the given states, and sums,
// launched where a state is wanted, writes it.
//
// Backward, the two directions' sums and prefixes and the three products (dq, dk,
// dv) share the launches; dq and dk of a key head walk its value heads inside
// the CTA, in order.  Only the prefix is sequential, so short calls of few heads
// still fill the card.
//
// A CTA has 128 threads of 8 rows x 4 columns, on pairs of fp32 (fma.f32x2).
// The fma pipes and the shared-memory reads that feed them bound it: B=8 H=16 N=4096
// D=M=64 in fp32, forward 510 us (34 TFLOP/s, scores counted whole), backward 1,334.
#include <algorithm>

#include "cp_decay.cuh"
#include "sm103_ptx.cuh"

namespace cp {
namespace {

using namespace decay;

constexpr int kC = 64;        // rows of a chunk, columns of a block
constexpr int kK = 32;        // contraction block
constexpr int kLd = kC + 4;   // padded row of a shared tile (16-byte rows)
constexpr int kThreads = 128;

struct Args {
  const void *q, *k, *v, *go;
  const float* g;
  const int* lengths;
  const float *s0, *gs;          // S_0 and dL/dS_N, may be null
  float *s_end, *ds0;            // S_N and dL/dS_0, may be null
  void *out, *dq, *dk, *dv;
  float *fwd, *rev;              // states before the chunks, in either order
  int64_t N, n, B;
  int H, Hk, group, D, M;
  float scale;
  bool backward;
};

struct Tile {
  float x[kC][kLd];
};

// acc(8 x 4) += x^T y over rows k0 .. k1 - 1 of two shared tiles
__device__ __forceinline__ void gemm(float2 (&acc)[4][4], const float (*x)[kLd],
                                     const float (*y)[kLd], int k0, int k1, int rg, int cg) {
#pragma unroll 4
  for (int k = k0; k < k1; ++k) {
    const float4 a0 = *reinterpret_cast<const float4*>(&x[k][rg * 8]);
    const float4 a1 = *reinterpret_cast<const float4*>(&x[k][rg * 8 + 4]);
    const float4 b = *reinterpret_cast<const float4*>(&y[k][cg * 4]);
    const float2 a[4] = {make_float2(a0.x, a0.y), make_float2(a0.z, a0.w), make_float2(a1.x, a1.y),
                         make_float2(a1.z, a1.w)};
    const float bb[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[r][c] = fma2(a[r], both(bb[c]), acc[r][c]);
  }
}

__device__ __forceinline__ void clear(float2 (&acc)[4][4]) {
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int c = 0; c < 4; ++c) acc[r][c] = make_float2(0.f, 0.f);
}

// A block on its way from global to shared memory, in registers: its loads go out
// together, and under the products on the block before it.  A thread moves four
// neighbours at a time, by one load where rows are whole fours.
constexpr int kTurned = kC * kK / kThreads / 4, kWhole = kC * kC / kThreads / 4;  // fours to a thread

template <typename T>
__device__ __forceinline__ float4 ld4(const T* p, int left, bool vec) {
  if (left <= 0) return make_float4(0.f, 0.f, 0.f, 0.f);
  if (vec) {
    if constexpr (sizeof(T) == 4) {
      return *reinterpret_cast<const float4*>(p);
    } else {
      const uint2 w = *reinterpret_cast<const uint2*>(p);
      const T* t = reinterpret_cast<const T*>(&w);
      return make_float4(ld_f32<T>(t), ld_f32<T>(t + 1), ld_f32<T>(t + 2), ld_f32<T>(t + 3));
    }
  }
  return make_float4(ld_f32<T>(p), left > 1 ? ld_f32<T>(p + 1) : 0.f, left > 2 ? ld_f32<T>(p + 2) : 0.f,
                     left > 3 ? ld_f32<T>(p + 3) : 0.f);
}

template <typename T>
__device__ __forceinline__ void st4(T* p, const float (&v)[4], int left, bool vec) {
  if (vec) {
    if constexpr (sizeof(T) == 4) {
      *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
      uint2 w;
      T* t = reinterpret_cast<T*>(&w);
#pragma unroll
      for (int i = 0; i < 4; ++i) t[i] = from_f32<T>(v[i]);
      *reinterpret_cast<uint2*>(p) = w;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < left) p[i] = from_f32<T>(v[i]);
}

// columns c0 .. c0 + kK - 1 of 64 rows, rows past nv and columns past C as zero, to
// tile[col][row], a row's factor f[row] applied where given
template <typename T>
__device__ __forceinline__ void fetch_turned(float4 (&v)[kTurned], const T* p, int C, int c0, int nv) {
  const int c = 4 * (threadIdx.x % (kK / 4));
#pragma unroll
  for (int i = 0; i < kTurned; ++i) {
    const int r = threadIdx.x / (kK / 4) + i * (kThreads / (kK / 4));
    v[i] = ld4<T>(p + (int64_t)r * C + c0 + c, r < nv ? C - c0 - c : 0, C % 4 == 0);
  }
}
__device__ __forceinline__ void put_turned(float (*t)[kLd], const float4 (&v)[kTurned], const float* f) {
  const int c = 4 * (threadIdx.x % (kK / 4));
#pragma unroll
  for (int i = 0; i < kTurned; ++i) {
    const int r = threadIdx.x / (kK / 4) + i * (kThreads / (kK / 4));
    const float by = f != nullptr ? f[r] : 1.f;
    t[c][r] = v[i].x * by;
    t[c + 1][r] = v[i].y * by;
    t[c + 2][r] = v[i].z * by;
    t[c + 3][r] = v[i].w * by;
  }
}
// 64 columns from c0 of 64 rows, to tile[row][col]
template <typename T>
__device__ __forceinline__ void fetch_rows(float4 (&v)[kWhole], const T* p, int C, int c0, int nv) {
  const int c = 4 * (threadIdx.x % (kC / 4));
#pragma unroll
  for (int i = 0; i < kWhole; ++i) {
    const int r = threadIdx.x / (kC / 4) + i * (kThreads / (kC / 4));
    v[i] = ld4<T>(p + (int64_t)r * C + c0 + c, r < nv ? C - c0 - c : 0, C % 4 == 0);
  }
}
__device__ __forceinline__ void put_rows(float (*t)[kLd], const float4 (&v)[kWhole], const float* f) {
  const int c = 4 * (threadIdx.x % (kC / 4));
#pragma unroll
  for (int i = 0; i < kWhole; ++i) {
    const int r = threadIdx.x / (kC / 4) + i * (kThreads / (kC / 4));
    const float by = f != nullptr ? f[r] : 1.f;
    *reinterpret_cast<float4*>(&t[r][c]) =
        make_float4(v[i].x * by, v[i].y * by, v[i].z * by, v[i].w * by);
  }
}
// rows k0 .. k0 + kK - 1 of 64 columns from c0 of a state [.][M], or of its
// transpose, to tile[row][col]
__device__ __forceinline__ void fetch_state(float4 (&v)[kTurned], const float* s, int M, bool turned,
                                            int DA, int DC, int k0, int c0) {
#pragma unroll
  for (int i = 0; i < kTurned; ++i) {
    const int j = threadIdx.x + i * kThreads;
    if (turned) {
      const int k = k0 + 4 * (j % (kK / 4)), c = c0 + j / (kK / 4);
      v[i] = ld4<float>(s + (int64_t)c * M + k, c < DC ? DA - k : 0, M % 4 == 0);
    } else {
      const int k = k0 + j / (kC / 4), c = c0 + 4 * (j % (kC / 4));
      v[i] = ld4<float>(s + (int64_t)k * M + c, k < DA ? DC - c : 0, M % 4 == 0);
    }
  }
}
__device__ __forceinline__ void put_state(float (*t)[kLd], const float4 (&v)[kTurned], bool turned) {
#pragma unroll
  for (int i = 0; i < kTurned; ++i) {
    const int j = threadIdx.x + i * kThreads;
    if (turned) {
      const int k = 4 * (j % (kK / 4)), c = j / (kK / 4);
      t[k][c] = v[i].x;
      t[k + 1][c] = v[i].y;
      t[k + 2][c] = v[i].z;
      t[k + 3][c] = v[i].w;
    } else {
      *reinterpret_cast<float4*>(&t[j / (kC / 4)][4 * (j % (kC / 4))]) = v[i];
    }
  }
}

// sums: blockIdx.y = 64 x 64 block of the state, z = direction
template <typename T>
__global__ void __launch_bounds__(kThreads) decay_sums_kernel(const Args a) {
  __shared__ __align__(16) Tile x, y;
  __shared__ float f[kC];
  ptx::grid_dep_wait();
  const bool rev = blockIdx.z != 0;
  const int64_t bh = blockIdx.x / a.n, c = blockIdx.x % a.n, b = bh / a.H;
  const int h = (int)(bh % a.H);
  const int64_t rows = rows_of(a.lengths, b, a.N);
  const int nv = (int)max((int64_t)0, min((int64_t)kC, rows - c * kC));
  if (nv == 0 && a.n > 1) return;
  const bool end = a.n == 1;  // the state after the only chunk, itself
  float* s = end ? (rev ? a.ds0 : a.s_end) : (rev ? a.rev : a.fwd);
  if (s == nullptr) return;   // (the backward of one chunk has no S_N to write)
  const int mb = (a.M + kC - 1) / kC;
  const int d0 = (blockIdx.y / mb) * kC, m0 = (blockIdx.y % mb) * kC;
  const int64_t row0 = bh * a.N + c * kC, krow0 = (b * a.Hk + h / a.group) * a.N + c * kC;
  const float g = head_decay(a.g[h]);
  float4 vx[kWhole], vy[kWhole];
  fetch_rows<T>(vx, static_cast<const T*>(rev ? a.q : a.k) + krow0 * a.D, a.D, d0, nv);
  fetch_rows<T>(vy, static_cast<const T*>(rev ? a.go : a.v) + row0 * a.M, a.M, m0, nv);
  if (threadIdx.x < kC) {
    const int r = threadIdx.x;
    f[r] = r < nv ? (rev ? a.scale * power(g, r) : power(g, nv - 1 - r)) : 0.f;
  }
  __syncthreads();
  put_rows(x.x, vx, f);
  put_rows(y.x, vy, nullptr);
  __syncthreads();
  const int cg = threadIdx.x % 16, rg = threadIdx.x / 16;
  float2 acc[4][4];
  clear(acc);
  gemm(acc, x.x, y.x, 0, nv, rg, cg);
  s += (bh * a.n + c) * (int64_t)a.D * a.M;
  const float* from = !end || (rev ? a.gs : a.s0) == nullptr
                          ? nullptr : (rev ? a.gs : a.s0) + bh * (int64_t)a.D * a.M;
  // (dL/dS_0 is a times the gradient seen from the first row)
  const float2 keep = power_parts(g, nv);
  const float by = rev && nv > 0 ? power(g, 1) : 1.f;
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    const int d = d0 + rg * 8 + r, m = m0 + cg * 4;
    if (d >= a.D || m >= a.M) continue;
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = r % 2 ? acc[r / 2][i].y : acc[r / 2][i].x;
      if (end) {
        const float S = from == nullptr || m + i >= a.M ? 0.f : from[(int64_t)d * a.M + m + i];
        v[i] = fmaf(keep.x, S, fmaf(keep.y, S, by * v[i]));
      }
    }
    st4<float>(s + (int64_t)d * a.M + m, v, a.M - m, a.M % 4 == 0);
  }
}

// prefix: a thread walks one element of a head's state over the chunks
__global__ void __launch_bounds__(256) decay_prefix_kernel(const Args a, int blocks) {
  ptx::grid_dep_wait();
  const bool rev = blockIdx.y != 0;
  const int64_t bh = blockIdx.x / blocks, b = bh / a.H;
  const int64_t DM = (int64_t)a.D * a.M, e = (int64_t)(blockIdx.x % blocks) * 256 + threadIdx.x;
  if (e >= DM) return;
  const float g = head_decay(a.g[bh % a.H]);
  const int64_t rows = rows_of(a.lengths, b, a.N);
  const int64_t live = (rows + kC - 1) / kC;   // chunks that hold rows
  const int last = (int)(rows - (live - 1) * kC);
  float* s = (rev ? a.rev : a.fwd) + bh * a.n * DM + e;
  const float2 full = power_parts(g, kC);
  const float* from = rev ? a.gs : a.s0;
  float* to = rev ? a.ds0 : a.s_end;
  float S = from != nullptr ? from[bh * DM + e] : 0.f;
  constexpr int kAhead = 8;
  float next[kAhead];
  auto place = [&](int64_t i) { return rev ? live - 1 - i : i; };
#pragma unroll
  for (int i = 0; i < kAhead; ++i) next[i] = i < live ? s[place(i) * DM] : 0.f;
  for (int64_t i0 = 0; i0 < live; i0 += kAhead) {
    float now[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      now[i] = next[i];
      next[i] = i0 + kAhead + i < live ? s[place(i0 + kAhead + i) * DM] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (i0 + i >= live) break;
      const int64_t c = place(i0 + i);
      // the last chunk's rows; the gradient of S_N is seen from its last row
      const float2 f = c != live - 1 ? full : power_parts(g, rev ? last - 1 : last);
      s[c * DM] = S;
      S = fmaf(f.x, S, fmaf(f.y, S, now[i]));
    }
  }
  if (to != nullptr) {
    if (rev && live > 0) {
      const float2 f = power_parts(g, 1);
      S = fmaf(f.x, S, f.y * S);
    }
    to[bh * DM + e] = S;
  }
}

// out: blockIdx.y = 64 columns of the result, z = product
template <typename T>
__global__ void __launch_bounds__(kThreads, 3) decay_out_kernel(const Args a) {
  __shared__ __align__(16) float x[kK][kLd];
  __shared__ __align__(16) Tile y, P;
  __shared__ float pw[kC + 1], f[kC];
  ptx::grid_dep_wait();
  // 0: the forward's out or dq, 1: dv, 2: dk
  const int kind = a.backward ? (int)blockIdx.z : -1;
  const bool rev = kind > 0;              // order, and which states
  const bool key_out = kind == 0 || kind == 2, turned = key_out;
  const int DA = key_out ? a.M : a.D, DC = key_out ? a.D : a.M;
  const int heads = key_out ? a.Hk : a.H;
  const int c0 = blockIdx.y * kC;
  const int64_t oh = blockIdx.x / a.n, c = blockIdx.x % a.n;  // result's head, over the batch
  if (oh >= a.B * heads || c0 >= DC) return;
  const int64_t b = oh / heads;
  const int64_t rows = rows_of(a.lengths, b, a.N);
  const int nv = (int)max((int64_t)0, min((int64_t)kC, rows - c * kC));
  const bool last = rows > c * kC && rows <= (c + 1) * kC;
  const int cg = threadIdx.x % 16, rg = threadIdx.x / 16;
  float2 acc[4][4];
  clear(acc);
  const int h0 = (int)(oh % heads) * (key_out ? a.group : 1);
  for (int h = h0; nv > 0 && h < h0 + (key_out ? a.group : 1); ++h) {
    const int64_t vrow = (b * a.H + h) * a.N + c * kC;
    const int64_t krow = (b * a.Hk + h / a.group) * a.N + c * kC;
    const T *pa, *pb, *pc;
    const T *q = static_cast<const T*>(a.q) + krow * a.D, *k = static_cast<const T*>(a.k) + krow * a.D;
    const T* v = static_cast<const T*>(a.v) + vrow * a.M;
    const T* go = static_cast<const T*>(a.go) + (kind >= 0 ? vrow * a.M : 0);
    if (kind < 0) { pa = q; pb = k; pc = v; }
    else if (kind == 0) { pa = go; pb = v; pc = k; }
    else if (kind == 1) { pa = k; pb = q; pc = go; }
    else { pa = v; pb = go; pc = q; }
    const float g = head_decay(a.g[h]);
    __syncthreads();
    if (threadIdx.x <= kC) {
      const int r = threadIdx.x;
      pw[r] = power(g, r);
      // the gradient of S_N is seen from the last row
      if (r < kC)
        f[r] = r >= nv ? 0.f
               : rev   ? power(g, nv - r - (last ? 1 : 0))
                       : a.scale * power(g, r + 1);
    }
    // scores
    float4 va[kTurned], vb[kTurned], vc[kWhole];
    fetch_turned<T>(va, pa, DA, 0, nv);
    fetch_turned<T>(vb, pb, DA, 0, nv);
    float2 p[4][4];
    clear(p);
    for (int k0 = 0; k0 < DA; k0 += kK) {
      __syncthreads();
      put_turned(x, va, nullptr);
      put_turned(y.x, vb, nullptr);
      __syncthreads();
      if (k0 + kK < DA) {
        fetch_turned<T>(va, pa, DA, k0 + kK, nv);
        fetch_turned<T>(vb, pb, DA, k0 + kK, nv);
      } else {
        fetch_rows<T>(vc, pc, DC, c0, nv);
      }
      gemm(p, x, y.x, 0, min(kK, DA - k0), rg, cg);
    }
#pragma unroll
    for (int r = 0; r < 8; ++r)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = rg * 8 + r, j = cg * 4 + i;
        const bool on = rev ? j >= row : j <= row;
        const float w = a.scale * pw[on ? (rev ? j - row : row - j) : 0];
        P.x[j][row] = on ? w * (r % 2 ? p[r / 2][i].y : p[r / 2][i].x) : 0.f;
      }
    __syncthreads();
    put_rows(y.x, vc, nullptr);
    __syncthreads();
    const float* s = a.n > 1 ? (rev ? a.rev : a.fwd) : (rev ? a.gs : a.s0);
    if (s != nullptr) {
      s += ((b * a.H + h) * a.n + c) * (int64_t)a.D * a.M;
      fetch_turned<T>(va, pa, DA, 0, nv);
      fetch_state(vb, s, a.M, turned, DA, DC, 0, c0);
    }
    // (a warp has 16 rows, whose scores past the diagonal are 0)
    gemm(acc, P.x, y.x, rev ? (rg & ~1) * 8 : 0, rev ? nv : min(nv, (rg & ~1) * 8 + 16), rg, cg);
    // the state's part
    for (int k0 = 0; s != nullptr && k0 < DA; k0 += kK) {
      __syncthreads();
      put_turned(x, va, f);
      put_state(y.x, vb, turned);
      __syncthreads();
      if (k0 + kK < DA) {
        fetch_turned<T>(va, pa, DA, k0 + kK, nv);
        fetch_state(vb, s, a.M, turned, DA, DC, k0 + kK, c0);
      }
      gemm(acc, x, y.x, 0, min(kK, DA - k0), rg, cg);
    }
  }
  T* out = static_cast<T*>(kind < 0 ? a.out : kind == 0 ? a.dq : kind == 1 ? a.dv : a.dk) +
           (oh * a.N + c * kC) * DC;
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    const int row = rg * 8 + r, col = c0 + cg * 4;
    if (c * kC + row >= a.N || col >= DC) continue;
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = row < nv ? (r % 2 ? acc[r / 2][i].y : acc[r / 2][i].x) : 0.f;
    st4<T>(out + (int64_t)row * DC + col, v, DC - col, DC % 4 == 0);
  }
}

int64_t chunks(const DecayShape& s) { return (s.N + kC - 1) / kC; }

size_t states_bytes(const DecayShape& s) {
  if (chunks(s) == 1) return 0;
  return (size_t)chunks(s) * s.B * s.H * s.D * s.M * sizeof(float);
}

template <typename T>
cudaError_t launch(const Args& a, cudaStream_t stream) {
  const int64_t BH = a.B * a.H;
  const unsigned dirs = a.backward ? 2 : 1;
  const unsigned db = (a.D + kC - 1) / kC, mb = (a.M + kC - 1) / kC;
  if (BH * a.n > (int64_t)INT32_MAX) return cudaErrorInvalidValue;
  cudaError_t e = cudaSuccess;
  if (a.n > 1 || (a.backward ? a.ds0 : a.s_end) != nullptr)
    e = launch_dependent(decay_sums_kernel<T>, dim3((unsigned)(BH * a.n), db * mb, dirs), kThreads,
                         0, stream, a);
  if (e == cudaSuccess && a.n > 1) {
    const int blocks = (a.D * a.M + 255) / 256;
    e = launch_dependent(decay_prefix_kernel, dim3((unsigned)(BH * blocks), dirs), 256, 0, stream, a,
                         blocks);
  }
  if (e != cudaSuccess) return e;
  return launch_dependent(
      decay_out_kernel<T>,
      dim3((unsigned)(BH * a.n), a.backward ? std::max(db, mb) : mb, a.backward ? 3 : 1), kThreads, 0,
      stream, a);
}

cudaError_t run(const DecayShape& s, Args& a, cudaStream_t stream) {
  a.lengths = s.lengths;
  a.N = s.N; a.n = chunks(s); a.B = s.B;
  a.H = (int)s.H; a.Hk = (int)s.Hk; a.group = (int)(s.H / s.Hk);
  a.D = (int)s.D; a.M = (int)s.M; a.scale = s.scale;
  if (s.dtype == CP_DTYPE_BF16) return launch<__nv_bfloat16>(a, stream);
  if (s.dtype == CP_DTYPE_F16) return launch<__half>(a, stream);
  return launch<float>(a, stream);
}

}  // namespace

size_t decay_simt_scratch(const DecayShape& s, bool backward) {
  return states_bytes(s) * (backward ? 2 : 1);
}

cudaError_t decay_simt_fwd(const DecayShape& s, const DecayFwd& f, void* scratch,
                           cudaStream_t stream) {
  Args a{};
  a.q = f.q; a.k = f.k; a.v = f.v; a.g = f.g;
  a.s0 = f.state_in; a.s_end = f.state_out; a.out = f.out;
  a.fwd = static_cast<float*>(scratch);
  return run(s, a, stream);
}

cudaError_t decay_simt_bwd(const DecayShape& s, const DecayBwd& f, void* scratch,
                           cudaStream_t stream) {
  Args a{};
  a.q = f.q; a.k = f.k; a.v = f.v; a.go = f.grad_out; a.g = f.g;
  a.s0 = f.state_in; a.gs = f.grad_state_out; a.ds0 = f.grad_state_in;
  a.dq = f.dq; a.dk = f.dk; a.dv = f.dv;
  a.fwd = static_cast<float*>(scratch);
  a.rev = a.fwd + states_bytes(s) / sizeof(float);
  a.backward = true;
  return run(s, a, stream);
}

}  // namespace cp
