// The gated delta rule on the CUDA cores in fp32: the path of fp32 and fp16
// inputs (widened on load) and of the bf16 shapes the tensor-core kernels do
// not take (D > 128).  The formulas are in cp_delta.cuh.
//
// Forward: one CTA per (head, block of MB value columns) walks the sequence in
// chunks of 32 rows with the MB x D state, transposed, in shared memory; the
// value columns of a head never meet, so a block of them is a problem of its
// own.  A chunk is six small products on shared-memory tiles and a triangular
// solve by substitution, a lane to a row.  Tiles lie so that both operands of a
// product run along its contraction and load 16 bytes at a time; the rows of
// the next chunk are loaded under the solve.  What bounds the walk is the
// latency of its steps on the SMs that its heads fill: about 14,000 cycles a
// chunk, half of those SMs' issue slots in use (fp32, D = M = 64, 8 heads, N = 509,
// cold: 108 us on 32 SMs; 128 heads, N = 4096: 1.26 ms for a floor of 80 us).
//
// Backward: the same walk in reverse with the state's gradient in shared
// memory, from the states the forward left before each chunk:
//     dU = P^T dO + del K dS',   (I + A)^T dX = dU,   dR = b dX = dV,
//     dP = tril(dO U^T),   dA = -stril(dX U^T),
//     dS = gam_C dS' + Q^T (s gam dO) - K^T (gam dR),
//     dQ = s gam dO S^T + Mq K,                  Mq = s dP o Gam,
//     dK = Mq^T Q + del U dS'^T - gam dR S^T + Ma K + Ma^T K,  Ma = b dA o Gam,
//     db_i = dX_i . R_i + sum_j dA_ij Gam_ij k_i.k_j,
//     dg_t = sum over pairs i >= t > j of (Mq q.k + Ma k.k)_ij
//            + sum_{i>=t} (row i's part with S) + sum_{j<t} (row j's with dS')
//            + gam_C <S, dS'>.
// dg's sums run over the pairs that straddle t, never as a difference of
// running totals, which would cancel.  Every gradient of q, k, b and g is a
// sum over value columns, so the column blocks (and the value heads that share
// a key head) leave fp32 parts that one more launch adds in a fixed order.
// Bound as the forward is: fp32, D = M = 64, 8 heads, N = 509, cold: 235 us, and 9
// us for the parts' sums.
#include <algorithm>

#include "cp_delta.cuh"

namespace cp {
namespace {

using namespace delta;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kC = 32;        // rows of a chunk
constexpr int kLdc = kC + 4;  // pitch of a tile with a chunk's rows along its columns

// Pitch of a tile row of n floats: a multiple of 16 bytes whose number of
// 16-byte words is odd, so that eight rows' words fall in different banks.
__host__ __device__ __forceinline__ int pitch(int n) { return 4 * (((n + 3) / 4) | 1); }

// Where a thread's outputs of a [kC] x [MB] product lie: LC lanes along the
// columns, RT consecutive rows and CT columns LC apart to a thread.
template <int MB>
struct Place {
  static constexpr int LC = MB < 32 ? MB : 32, CT = MB / LC, RT = LC / 16;
  int row, col;
  __device__ __forceinline__ Place() {
    const int w = threadIdx.x / 32, l = threadIdx.x % 32;
    row = (w * (32 / LC) + l / LC) * RT;
    col = l % LC;
  }
};

__device__ __forceinline__ void fma4(float& acc, float4 a, float4 b) {
  acc = fmaf(a.x, b.x, acc);
  acc = fmaf(a.y, b.y, acc);
  acc = fmaf(a.z, b.z, acc);
  acc = fmaf(a.w, b.w, acc);
}
__device__ __forceinline__ float4 at4(const float* p) { return *reinterpret_cast<const float4*>(p); }

// acc[r][c] += sum_k a[row + r][k] b[col + LC c][k], k < n (a multiple of 4):
// both operands run along the contraction in 16-byte loads.
template <int MB>
__device__ __forceinline__ void dot(float (&acc)[Place<MB>::RT][Place<MB>::CT], const Place<MB>& at,
                                    const float* a, int lda, const float* b, int ldb, int n) {
  constexpr int RT = Place<MB>::RT, CT = Place<MB>::CT, LC = Place<MB>::LC;
  a += at.row * lda;
  b += at.col * ldb;
#pragma unroll 4
  for (int k = 0; k < n; k += 4) {
    float4 av[RT], bv[CT];
#pragma unroll
    for (int r = 0; r < RT; ++r) av[r] = at4(a + r * lda + k);
#pragma unroll
    for (int c = 0; c < CT; ++c) bv[c] = at4(b + c * LC * ldb + k);
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int c = 0; c < CT; ++c) fma4(acc[r][c], av[r], bv[c]);
  }
}
// the same for two left operands over one right one
template <int MB>
__device__ __forceinline__ void dot2(float (&acc)[Place<MB>::RT][Place<MB>::CT],
                                     float (&acc2)[Place<MB>::RT][Place<MB>::CT],
                                     const Place<MB>& at, const float* a, const float* a2, int lda,
                                     const float* b, int ldb, int n) {
  constexpr int RT = Place<MB>::RT, CT = Place<MB>::CT, LC = Place<MB>::LC;
  a += at.row * lda;
  a2 += at.row * lda;
  b += at.col * ldb;
#pragma unroll 4
  for (int k = 0; k < n; k += 4) {
    float4 av[RT], aw[RT], bv[CT];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      av[r] = at4(a + r * lda + k);
      aw[r] = at4(a2 + r * lda + k);
    }
#pragma unroll
    for (int c = 0; c < CT; ++c) bv[c] = at4(b + c * LC * ldb + k);
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int c = 0; c < CT; ++c) {
        fma4(acc[r][c], av[r], bv[c]);
        fma4(acc2[r][c], aw[r], bv[c]);
      }
  }
}

struct Args {
  const void *q, *k, *v, *go;
  const float *g, *beta, *state_in, *grad_state_out;
  void *out, *dq, *dk, *dv;
  float *state_out, *ckpt, *dg, *dbeta, *grad_state_in;
  float *dq_part, *dk_part, *dg_part, *db_part;  // [n_mb][BH][N][..], or null: written whole
  int64_t N;
  int D, M, H, group;
  float scale;
};

// A chunk's rows of q or k on their way to shared memory: the first 128
// columns wait in registers, loaded while the chunk before is worked on.
template <typename T>
struct Rows {
  T x[2][4];
  __device__ __forceinline__ void fetch(const T* src, int64_t i0, int64_t N, int D) {
    const int i = threadIdx.x / 32 * 2, l = threadIdx.x % 32;
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int c = 0; c < 4; ++c)
        x[r][c] = i0 + i + r < N && l + 32 * c < D ? src[(i0 + i + r) * D + l + 32 * c]
                                                   : from_f32<T>(0.f);
  }
  // rows past N and columns from D to the next multiple of 4 are zero
  __device__ __forceinline__ void put(float* dst, int ld, const T* src, int64_t i0, int64_t N,
                                      int D) {
    const int i = threadIdx.x / 32 * 2, l = threadIdx.x % 32, Dp = (D + 3) & ~3;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (l + 32 * c < Dp) dst[(i + r) * ld + l + 32 * c] = ld_f32<T>(&x[r][c]);
#pragma unroll 1
      for (int c = l + 128; c < Dp; c += 32)
        dst[(i + r) * ld + c] =
            i0 + i + r < N && c < D ? ld_f32<T>(src + (i0 + i + r) * D + c) : 0.f;
    }
  }
};
// A chunk's rows of a block of MB value columns, kept transposed: [MB][kLdc].
template <typename T, int MB>
struct Cols {
  static constexpr int kN = kC * MB / kThreads;
  T x[kN];
  __device__ __forceinline__ void fetch(const T* src, int64_t i0, int64_t N, int M, int c0) {
    const int c = threadIdx.x % MB;
#pragma unroll
    for (int u = 0; u < kN; ++u) {
      const int64_t i = i0 + threadIdx.x / MB + u * (kThreads / MB);
      x[u] = i < N && c0 + c < M ? src[i * M + c0 + c] : from_f32<T>(0.f);
    }
  }
  __device__ __forceinline__ void put(float* dst) {
#pragma unroll
    for (int u = 0; u < kN; ++u)
      dst[threadIdx.x % MB * kLdc + threadIdx.x / MB + u * (kThreads / MB)] = ld_f32<T>(&x[u]);
  }
};

struct alignas(16) Gates {
  float2 G[kC];   // running sums of the log decay
  float b[kC], gam[kC], del[kC];
  float2 last;    // gam of the last row, hi + lo
};

// by one warp
__device__ __forceinline__ void load_gates(Gates& s, const float* g, const float* beta, int64_t i0,
                                           int64_t N) {
  const int i = threadIdx.x % 32;
  const bool on = i0 + i < N;
  const float2 G = warp_scan(split_decay(on ? g[i0 + i] : 0.f), i);
  const float2 E = make_float2(__shfl_sync(0xffffffffu, G.x, 31), __shfl_sync(0xffffffffu, G.y, 31));
  const float2 zero = make_float2(0.f, 0.f);
  s.G[i] = G;
  s.b[i] = on ? beta[i0 + i] : 0.f;
  s.gam[i] = decay_between(G, zero);
  s.del[i] = decay_between(E, G);
  if (i == 0) s.last = decay_parts(E);
}

// (I + A) u = x in place for a warp's columns of x [MB][kLdc], at[j][i] = A_ij;
// a lane holds a row, and each solved row leaves the rows below it at once.
template <int MB>
__device__ __forceinline__ void solve_down(float* x, const float* at) {
  const int w = threadIdx.x / 32, l = threadIdx.x % 32;
  float u[MB / kWarps];
#pragma unroll
  for (int c = 0; c < MB / kWarps; ++c) u[c] = x[(w + kWarps * c) * kLdc + l];
#pragma unroll 8
  for (int j = 0; j < kC - 1; ++j) {
    const float a = at[j * kLdc + l];
#pragma unroll
    for (int c = 0; c < MB / kWarps; ++c) {
      const float s = __shfl_sync(0xffffffffu, u[c], j);
      if (l > j) u[c] = fmaf(-a, s, u[c]);
    }
  }
#pragma unroll
  for (int c = 0; c < MB / kWarps; ++c) x[(w + kWarps * c) * kLdc + l] = u[c];
}
// and beside it (I + A)^T v = y from the last row up, a[j][i] = A_ji: two
// chains of steps that do not wait for one another
template <int MB>
__device__ __forceinline__ void solve_both(float* x, const float* at, float* y, const float* a) {
  const int w = threadIdx.x / 32, l = threadIdx.x % 32;
  float u[MB / kWarps], v[MB / kWarps];
#pragma unroll
  for (int c = 0; c < MB / kWarps; ++c) {
    u[c] = x[(w + kWarps * c) * kLdc + l];
    v[c] = y[(w + kWarps * c) * kLdc + l];
  }
#pragma unroll 4
  for (int j = 0; j < kC - 1; ++j) {
    const int i = kC - 1 - j;
    const float ad = at[j * kLdc + l], au = a[i * kLdc + l];
#pragma unroll
    for (int c = 0; c < MB / kWarps; ++c) {
      const float s = __shfl_sync(0xffffffffu, u[c], j), t = __shfl_sync(0xffffffffu, v[c], i);
      if (l > j) u[c] = fmaf(-ad, s, u[c]);
      if (l < i) v[c] = fmaf(-au, t, v[c]);
    }
  }
#pragma unroll
  for (int c = 0; c < MB / kWarps; ++c) {
    x[(w + kWarps * c) * kLdc + l] = u[c];
    y[(w + kWarps * c) * kLdc + l] = v[c];
  }
}

// s[c][d] = D x MB block of a state, or zero; the padding of both is zero
template <int MB>
__device__ __forceinline__ void load_state(float* s, int ldd, const float* src, int D, int M,
                                           int c0) {
  const int Dp = (D + 3) & ~3, c = threadIdx.x % MB;
  for (int d = threadIdx.x / MB; d < Dp; d += kThreads / MB)
    s[c * ldd + d] = src != nullptr && d < D && c0 + c < M ? src[(int64_t)d * M + c0 + c] : 0.f;
}
template <int MB>
__device__ __forceinline__ void store_state(float* dst, const float* s, int ldd, int D, int M,
                                            int c0) {
  const int c = threadIdx.x % MB;
  if (c0 + c < M)
    for (int d = threadIdx.x / MB; d < D; d += kThreads / MB)
      dst[(int64_t)d * M + c0 + c] = s[c * ldd + d];
}

template <typename T, int MB>
__global__ void __launch_bounds__(kThreads) delta_fwd_kernel(Args p) {
  extern __shared__ __align__(16) float sm[];
  using PM = Place<MB>;
  using PC = Place<kC>;
  const int D = p.D, M = p.M, ldd = pitch(D), Dp = (D + 3) & ~3;
  float* S = sm;                 // [MB][ldd]
  float* K = S + MB * ldd;       // [kC][ldd]
  float* Q = K + kC * ldd;       // [kC][ldd]
  float* U = Q + kC * ldd;       // [MB][kLdc]  V, then b R, then U
  float* At = U + MB * kLdc;     // [kC][kLdc]  A transposed
  float* P = At + kC * kLdc;     // [kC][kLdc]
  __shared__ Gates gates[2];
  const int w = threadIdx.x / 32, l = threadIdx.x % 32;
  const int64_t p_ = blockIdx.x;
  const int c0 = blockIdx.y * MB;
  const int64_t N = p.N, pk = (p_ / p.H) * (p.H / p.group) + (p_ % p.H) / p.group;
  const T* q = static_cast<const T*>(p.q) + pk * N * D;
  const T* k = static_cast<const T*>(p.k) + pk * N * D;
  const T* v = static_cast<const T*>(p.v) + p_ * N * M;
  const float *g = p.g + p_ * N, *beta = p.beta + p_ * N;
  T* out = static_cast<T*>(p.out) + p_ * N * M;
  const int64_t n_chunks = (N + kC - 1) / kC;
  const PM at;
  const PC pair;
  Rows<T> kr, qr;
  Cols<T, MB> vr;
  load_state<MB>(S, ldd, p.state_in != nullptr ? p.state_in + p_ * D * M : nullptr, D, M, c0);
  kr.fetch(k, 0, N, D);
  qr.fetch(q, 0, N, D);
  vr.fetch(v, 0, N, M, c0);
  if (w == kWarps - 1) load_gates(gates[0], g, beta, 0, N);
  for (int64_t ch = 0; ch < n_chunks; ++ch) {
    const int64_t i0 = ch * kC;
    const Gates& gt = gates[ch & 1];
    __syncthreads();
    kr.put(K, ldd, k, i0, N, D);
    qr.put(Q, ldd, q, i0, N, D);
    vr.put(U);
    if (p.ckpt != nullptr) store_state<MB>(p.ckpt + (p_ * n_chunks + ch) * D * M, S, ldd, D, M, c0);
    __syncthreads();
    {
      float kk[PC::RT][1] = {}, qk[PC::RT][1] = {};
      dot2<kC>(kk, qk, pair, K, Q, ldd, K, ldd, Dp);
#pragma unroll
      for (int r = 0; r < PC::RT; ++r) {
        const int i = pair.row + r, j = pair.col;
        const float e = j <= i ? decay_between(gt.G[i], gt.G[j]) : 0.f;
        At[j * kLdc + i] = j < i ? gt.b[i] * e * kk[r][0] : 0.f;
        P[i * kLdc + j] = j <= i ? p.scale * e * qk[r][0] : 0.f;
      }
    }
    float o[PM::RT][PM::CT] = {};
    {
      float ks[PM::RT][PM::CT] = {};
      dot2<MB>(ks, o, at, K, Q, ldd, S, ldd, Dp);
#pragma unroll
      for (int r = 0; r < PM::RT; ++r)
#pragma unroll
        for (int c = 0; c < PM::CT; ++c) {
          const int i = at.row + r;
          float* x = U + (at.col + PM::LC * c) * kLdc + i;
          *x = gt.b[i] * (*x - gt.gam[i] * ks[r][c]);
          o[r][c] *= p.scale * gt.gam[i];
        }
    }
    __syncthreads();
    if (ch + 1 < n_chunks) {
      kr.fetch(k, i0 + kC, N, D);
      qr.fetch(q, i0 + kC, N, D);
      vr.fetch(v, i0 + kC, N, M, c0);
      if (w == kWarps - 1) load_gates(gates[(ch + 1) & 1], g, beta, i0 + kC, N);
    }
    solve_down<MB>(U, At);
    __syncthreads();
    dot<MB>(o, at, P, kLdc, U, kLdc, kC);
#pragma unroll
    for (int r = 0; r < PM::RT; ++r)
#pragma unroll
      for (int c = 0; c < PM::CT; ++c) {
        const int64_t i = i0 + at.row + r;
        const int j = c0 + at.col + PM::LC * c;
        if (i < N && j < M) out[i * M + j] = from_f32<T>(o[r][c]);
      }
    // the state: lanes along its rows d, a warp's columns 16 apart
#pragma unroll 1
    for (int d = l; d < Dp; d += 32) {
      float acc[MB / kWarps] = {};
#pragma unroll
      for (int x = 0; x < kC; x += 4) {
        const float4 del = at4(gt.del + x);
        const float4 kd = make_float4(K[x * ldd + d] * del.x, K[(x + 1) * ldd + d] * del.y,
                                      K[(x + 2) * ldd + d] * del.z, K[(x + 3) * ldd + d] * del.w);
#pragma unroll
        for (int c = 0; c < MB / kWarps; ++c) fma4(acc[c], kd, at4(U + (w + kWarps * c) * kLdc + x));
      }
#pragma unroll
      for (int c = 0; c < MB / kWarps; ++c) {
        float* s = S + (w + kWarps * c) * ldd + d;
        *s = fmaf(gt.last.x, *s, fmaf(gt.last.y, *s, acc[c]));
      }
    }
  }
  __syncthreads();
  if (p.state_out != nullptr) store_state<MB>(p.state_out + p_ * D * M, S, ldd, D, M, c0);
}

template <typename T, int MB>
__global__ void __launch_bounds__(kThreads) delta_bwd_kernel(Args p) {
  extern __shared__ __align__(16) float sm[];
  using PM = Place<MB>;
  using PC = Place<kC>;
  constexpr int RT = PM::RT, CT = PM::CT, LC = PM::LC;
  const int D = p.D, M = p.M, ldd = pitch(D), Dp = (D + 3) & ~3;
  float* S = sm;                   // [MB][ldd]  state before the chunk
  float* dS = S + MB * ldd;        // [MB][ldd]  gradient of the state after it
  float* K = dS + MB * ldd;        // [kC][ldd]
  float* Q = K + kC * ldd;         // [kC][ldd]
  float* dO = Q + kC * ldd;        // [MB][kLdc]  then s gam dO
  float* U = dO + MB * kLdc;       // [MB][kLdc]  V, b R, U, then del U
  float* dX = U + MB * kLdc;       // [MB][kLdc]  dU, dX, then gam dR
  float* A = dX + MB * kLdc;       // [kC][kLdc]  A, then the pairs' weights in dg
  float* At = A + kC * kLdc;       // [kC][kLdc]  A transposed, then Mq
  float* Pt = At + kC * kLdc;      // [kC][kLdc]  P transposed, then Mq transposed
  float* Ms = Pt + kC * kLdc;      // [kC][kLdc]  Ma + Ma^T
  __shared__ Gates gates[2];
  __shared__ float red[kWarps], rows[2][kC];  // of dg: row i's part with S, row j's with dS'
  const int64_t p_ = blockIdx.x;
  const int c0 = blockIdx.y * MB;
  const int64_t N = p.N, pk = (p_ / p.H) * (p.H / p.group) + (p_ % p.H) / p.group;
  const T* q = static_cast<const T*>(p.q) + pk * N * D;
  const T* k = static_cast<const T*>(p.k) + pk * N * D;
  const T* v = static_cast<const T*>(p.v) + p_ * N * M;
  const T* go = static_cast<const T*>(p.go) + p_ * N * M;
  const float *g = p.g + p_ * N, *beta = p.beta + p_ * N;
  T* dv = static_cast<T*>(p.dv) + p_ * N * M;
  const int64_t part = ((int64_t)blockIdx.y * gridDim.x + p_) * N;
  const int64_t n_chunks = (N + kC - 1) / kC;
  const float* ckpt = p.ckpt + p_ * n_chunks * D * M;
  const int w = threadIdx.x / 32, l = threadIdx.x % 32;
  const PM at;
  const PC pair;
  Rows<T> kr, qr;
  Cols<T, MB> vr, gr;
  load_state<MB>(dS, ldd, p.grad_state_out != nullptr ? p.grad_state_out + p_ * D * M : nullptr, D,
                 M, c0);
  if (n_chunks > 0) {
    const int64_t i0 = (n_chunks - 1) * kC;
    load_state<MB>(S, ldd, ckpt + (n_chunks - 1) * D * M, D, M, c0);
    kr.fetch(k, i0, N, D);
    qr.fetch(q, i0, N, D);
    vr.fetch(v, i0, N, M, c0);
    gr.fetch(go, i0, N, M, c0);
    if (w == kWarps - 1) load_gates(gates[(n_chunks - 1) & 1], g, beta, i0, N);
  }
  for (int64_t ch = n_chunks - 1; ch >= 0; --ch) {
    const int64_t i0 = ch * kC;
    const Gates& gt = gates[ch & 1];
    __syncthreads();
    kr.put(K, ldd, k, i0, N, D);
    qr.put(Q, ldd, q, i0, N, D);
    vr.put(U);
    gr.put(dO);
    __syncthreads();
    // a thread's pairs (i, j) of the chunk: k.k, q.k and the decay between them
    float kk[PC::RT][1] = {}, qk[PC::RT][1] = {}, gm[PC::RT];
    dot2<kC>(kk, qk, pair, K, Q, ldd, K, ldd, Dp);
#pragma unroll
    for (int r = 0; r < PC::RT; ++r) {
      const int i = pair.row + r, j = pair.col;
      gm[r] = j <= i ? decay_between(gt.G[i], gt.G[j]) : 0.f;
      const float a = j < i ? gt.b[i] * gm[r] * kk[r][0] : 0.f;
      A[i * kLdc + j] = a;
      At[j * kLdc + i] = a;
      Pt[j * kLdc + i] = j <= i ? p.scale * gm[r] * qk[r][0] : 0.f;
    }
    // and its entries (i, c) of the products with S and dS'
    float ks[RT][CT] = {}, qs[RT][CT] = {}, kd[RT][CT] = {}, rr[RT][CT];
    dot2<MB>(ks, qs, at, K, Q, ldd, S, ldd, Dp);
    dot<MB>(kd, at, K, ldd, dS, ldd, Dp);
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int c = 0; c < CT; ++c) {
        const int i = at.row + r;
        float* x = U + (at.col + LC * c) * kLdc + i;
        rr[r][c] = *x - gt.gam[i] * ks[r][c];
        *x = gt.b[i] * rr[r][c];
      }
    float z = 0.f;
#pragma unroll 2
    for (int d = l; d < D; d += 32)
#pragma unroll
      for (int c = w; c < MB; c += kWarps) z = fmaf(S[c * ldd + d], dS[c * ldd + d], z);
    for (int o = 16; o > 0; o /= 2) z += __shfl_xor_sync(0xffffffffu, z, o);
    if (l == 0) red[w] = z;
    __syncthreads();
    {
      float du[RT][CT] = {};
      dot<MB>(du, at, Pt, kLdc, dO, kLdc, kC);
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int c = 0; c < CT; ++c)
          dX[(at.col + LC * c) * kLdc + at.row + r] = du[r][c] + gt.del[at.row + r] * kd[r][c];
    }
    __syncthreads();
    if (ch > 0) {
      kr.fetch(k, i0 - kC, N, D);
      qr.fetch(q, i0 - kC, N, D);
      vr.fetch(v, i0 - kC, N, M, c0);
      gr.fetch(go, i0 - kC, N, M, c0);
      if (w == kWarps - 1) load_gates(gates[(ch - 1) & 1], g, beta, i0 - kC, N);
    }
    solve_both<MB>(U, At, dX, A);
    __syncthreads();
    // dP and dA of the pairs: the sums over the columns, weighted
    float db[PC::RT], wt[PC::RT], mq[PC::RT], ma[PC::RT];
    {
      float dp[PC::RT] = {}, da[PC::RT] = {};
      static_assert(PC::RT == 2, "a pair's two rows are read as one word");
#pragma unroll 8
      for (int c = 0; c < MB; ++c) {
        const float u = U[c * kLdc + pair.col];
        const float2 o = *reinterpret_cast<const float2*>(dO + c * kLdc + pair.row);
        const float2 x = *reinterpret_cast<const float2*>(dX + c * kLdc + pair.row);
        dp[0] = fmaf(o.x, u, dp[0]);
        dp[1] = fmaf(o.y, u, dp[1]);
        da[0] = fmaf(x.x, u, da[0]);
        da[1] = fmaf(x.y, u, da[1]);
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int i = pair.row + r, j = pair.col;
        mq[r] = p.scale * gm[r] * dp[r];
        const float t = j < i ? -gm[r] * da[r] : 0.f;  // without b: db needs it so
        db[r] = t * kk[r][0];
        ma[r] = gt.b[i] * t;
        wt[r] = mq[r] * qk[r][0] + ma[r] * kk[r][0];
      }
    }
    // the rows' sums: of db, and of dg's parts with S and with dS'
#pragma unroll
    for (int r = 0; r < 2; ++r)
      for (int o = 16; o > 0; o /= 2) db[r] += __shfl_xor_sync(0xffffffffu, db[r], o);
    float dbr[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      const int i = at.row + r;
      float b = 0.f, s = 0.f, t = 0.f;
#pragma unroll
      for (int c = 0; c < CT; ++c) {
        const int e = (at.col + LC * c) * kLdc + i;
        const float x = dX[e];
        b = fmaf(x, rr[r][c], b);
        s += p.scale * dO[e] * qs[r][c] - gt.b[i] * x * ks[r][c];
        t = fmaf(U[e], kd[r][c], t);
      }
      for (int o = LC / 2; o > 0; o /= 2) {
        b += __shfl_xor_sync(0xffffffffu, b, o);
        s += __shfl_xor_sync(0xffffffffu, s, o);
        t += __shfl_xor_sync(0xffffffffu, t, o);
      }
      dbr[r] = b;
      if (at.col == 0) {
        rows[0][i] = gt.gam[i] * s;
        rows[1][i] = gt.del[i] * t;
      }
    }
    // a warp's two rows are 2w and 2w + 1 in both placements
    if (at.col == 0)
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const int i = at.row + r;
        if (i0 + i < N) {
          const float s = dbr[r] + (i % 2 == 0 ? db[0] : db[1]);
          if (p.db_part != nullptr)
            p.db_part[part + i0 + i] = s;
          else
            p.dbeta[p_ * N + i0 + i] = s;
        }
      }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int i = pair.row + r, j = pair.col;
      A[i * kLdc + j] = wt[r];
      At[i * kLdc + j] = mq[r];
      Pt[j * kLdc + i] = mq[r];
      if (j <= i) {
        Ms[i * kLdc + j] = ma[r];
        Ms[j * kLdc + i] = ma[r];
      }
    }
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int c = 0; c < CT; ++c) {
        const int i = at.row + r, j = c0 + at.col + LC * c;
        const int e = (at.col + LC * c) * kLdc + i;
        const float x = gt.b[i] * dX[e];
        if (i0 + i < N && j < M) dv[(i0 + i) * M + j] = from_f32<T>(x);
        dX[e] = gt.gam[i] * x;
        dO[e] *= p.scale * gt.gam[i];
        U[e] *= gt.del[i];
      }
    __syncthreads();
    // dg_t: warp w takes t = w and w + 16: lane j < t sums its column from row
    // t on; lane l >= t adds row l's part
    {
      float zs = 0.f;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) zs += red[i];
      zs *= gt.last.x;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int t = w + kWarps * u;
        float s = 0.f;
        if (l < t) {
#pragma unroll 8
          for (int i = t; i < kC; ++i) s += A[i * kLdc + l];
          s += rows[1][l];
        } else {
          s = rows[0][l];
        }
        for (int o = 16; o > 0; o /= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
        s += zs;
        if (l == 0 && i0 + t < N) {
          if (p.dg_part != nullptr)
            p.dg_part[part + i0 + t] = s;
          else
            p.dg[p_ * N + i0 + t] = s;
        }
      }
    }
    // dQ and dK of rows 2w and 2w + 1: lanes along d
#pragma unroll 1
    for (int j0 = l; j0 < Dp; j0 += 64) {
      const bool two = j0 + 32 < Dp;
      const int j1 = two ? j0 + 32 : j0;
      float aq[2][2] = {}, ak[2][2] = {};
#pragma unroll 4
      for (int x = 0; x < MB; ++x) {
        const float s0 = S[x * ldd + j0], s1 = S[x * ldd + j1];
        const float t0 = dS[x * ldd + j0], t1 = dS[x * ldd + j1];
        const float2 a = *reinterpret_cast<const float2*>(dO + x * kLdc + 2 * w);
        const float2 b = *reinterpret_cast<const float2*>(dX + x * kLdc + 2 * w);
        const float2 u = *reinterpret_cast<const float2*>(U + x * kLdc + 2 * w);
        aq[0][0] = fmaf(a.x, s0, aq[0][0]);
        aq[0][1] = fmaf(a.x, s1, aq[0][1]);
        aq[1][0] = fmaf(a.y, s0, aq[1][0]);
        aq[1][1] = fmaf(a.y, s1, aq[1][1]);
        ak[0][0] = fmaf(u.x, t0, fmaf(-b.x, s0, ak[0][0]));
        ak[0][1] = fmaf(u.x, t1, fmaf(-b.x, s1, ak[0][1]));
        ak[1][0] = fmaf(u.y, t0, fmaf(-b.y, s0, ak[1][0]));
        ak[1][1] = fmaf(u.y, t1, fmaf(-b.y, s1, ak[1][1]));
      }
#pragma unroll 4
      for (int x = 0; x < kC; ++x) {
        const float k0 = K[x * ldd + j0], k1 = K[x * ldd + j1];
        const float q0 = Q[x * ldd + j0], q1 = Q[x * ldd + j1];
        const float2 a = *reinterpret_cast<const float2*>(Pt + x * kLdc + 2 * w);
        const float2 t = *reinterpret_cast<const float2*>(At + x * kLdc + 2 * w);
        const float2 m = *reinterpret_cast<const float2*>(Ms + x * kLdc + 2 * w);
        aq[0][0] = fmaf(a.x, k0, aq[0][0]);
        aq[0][1] = fmaf(a.x, k1, aq[0][1]);
        aq[1][0] = fmaf(a.y, k0, aq[1][0]);
        aq[1][1] = fmaf(a.y, k1, aq[1][1]);
        ak[0][0] = fmaf(t.x, q0, fmaf(m.x, k0, ak[0][0]));
        ak[0][1] = fmaf(t.x, q1, fmaf(m.x, k1, ak[0][1]));
        ak[1][0] = fmaf(t.y, q0, fmaf(m.y, k0, ak[1][0]));
        ak[1][1] = fmaf(t.y, q1, fmaf(m.y, k1, ak[1][1]));
      }
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int64_t i = i0 + 2 * w + r;
          const int d = j0 + 32 * c;
          if (i >= N || d >= D) continue;
          if (p.dq_part != nullptr) {
            p.dq_part[(part + i) * D + d] = aq[r][c];
            p.dk_part[(part + i) * D + d] = ak[r][c];
          } else {
            static_cast<T*>(p.dq)[(p_ * N + i) * D + d] = from_f32<T>(aq[r][c]);
            static_cast<T*>(p.dk)[(p_ * N + i) * D + d] = from_f32<T>(ak[r][c]);
          }
        }
    }
    __syncthreads();
    // the states of the chunk before: S from memory, dS from this chunk
    if (ch > 0) load_state<MB>(S, ldd, ckpt + (ch - 1) * D * M, D, M, c0);
#pragma unroll 1
    for (int d = l; d < Dp; d += 32) {
      float acc[MB / kWarps] = {};
#pragma unroll
      for (int x = 0; x < kC; x += 4) {
        const float4 qv = make_float4(Q[x * ldd + d], Q[(x + 1) * ldd + d], Q[(x + 2) * ldd + d],
                                      Q[(x + 3) * ldd + d]);
        const float4 kv = make_float4(-K[x * ldd + d], -K[(x + 1) * ldd + d],
                                      -K[(x + 2) * ldd + d], -K[(x + 3) * ldd + d]);
#pragma unroll
        for (int c = 0; c < MB / kWarps; ++c) {
          fma4(acc[c], qv, at4(dO + (w + kWarps * c) * kLdc + x));
          fma4(acc[c], kv, at4(dX + (w + kWarps * c) * kLdc + x));
        }
      }
#pragma unroll
      for (int c = 0; c < MB / kWarps; ++c) {
        float* s = dS + (w + kWarps * c) * ldd + d;
        *s = fmaf(gt.last.x, *s, fmaf(gt.last.y, *s, acc[c]));
      }
    }
  }
  __syncthreads();
  if (p.grad_state_in != nullptr) store_state<MB>(p.grad_state_in + p_ * D * M, dS, ldd, D, M, c0);
}

// out[head][row] = sum over the column blocks and the group's heads of parts
// [n_mb][heads][group][rows], in that order; the launch's rows of blocks are
// dq, dk and, where they have parts, dg and db
template <typename T>
__device__ __forceinline__ void join(const float* __restrict__ part, T* __restrict__ out,
                                     int64_t rows, int64_t heads, int group, int n_mb) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, n = rows * heads;
  if (i >= n) return;
  const int64_t h = i / rows, r = i % rows;
  float s = 0.f;
  for (int m = 0; m < n_mb; ++m)
    for (int g = 0; g < group; ++g) s += part[((int64_t)m * heads * group + h * group + g) * rows + r];
  out[i] = from_f32<T>(s);
}
template <typename T>
__global__ void __launch_bounds__(256) delta_join_kernel(DeltaJoin x) {
  switch (blockIdx.y) {
    case 0: return join(x.dq_part, static_cast<T*>(x.dq), x.N * x.D, x.heads, x.group, x.n_mb);
    case 1: return join(x.dk_part, static_cast<T*>(x.dk), x.N * x.D, x.heads, x.group, x.n_mb);
    case 2: return join(x.dg_part, x.dg, x.N, x.heads * x.group, 1, x.n_mb);
    default: return join(x.db_part, x.db, x.N, x.heads * x.group, 1, x.n_mb);
  }
}

// Value columns of a CTA: 64 while the state's tiles and the row tiles fit the
// shared memory (D <= 128), else 32; halved while the halves still get an SM
// each: the walk's time is its own latency then, and the columns lengthen it.
// (fp32, D = M = 64, N = 512, forward and backward calls back to back, the parts'
// sums with the latter: 8 heads 102 + 233 us with 16 columns, 122 + 294 with 32,
// 163 + 408 with 64; 64 heads 122 + 332 with 32, 163 + 410 with 64, 198 + 522 with
// 16, two turns of the SMs.  The 64-column backward spills 72 to 76 bytes a thread,
// the 64- and 32-column forward 4 to 16.)
int block_cols(int64_t BH, int64_t D, int64_t M) {
  int mb = D <= 128 && M > 32 ? 64 : 32;
  while (mb > 16 && BH * ((M + mb / 2 - 1) / (mb / 2)) <= kPlanSMs) mb /= 2;
  return mb;
}

size_t fwd_smem(int D, int mb) {
  return sizeof(float) * (size_t)((mb + 2 * kC) * pitch(D) + (mb + 2 * kC) * kLdc);
}
size_t bwd_smem(int D, int mb) {
  return sizeof(float) * (size_t)((2 * mb + 2 * kC) * pitch(D) + (3 * mb + 4 * kC) * kLdc);
}

template <typename T, int MB>
cudaError_t launch(const Args& a, int64_t BH, bool backward, cudaStream_t stream) {
  const dim3 grid((unsigned)BH, (unsigned)((a.M + MB - 1) / MB));
  const size_t smem = backward ? bwd_smem(a.D, MB) : fwd_smem(a.D, MB);
  void (*kern)(Args) = backward ? delta_bwd_kernel<T, MB> : delta_fwd_kernel<T, MB>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  kern<<<grid, kThreads, smem, stream>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t run(const Args& a, int64_t BH, bool backward, cudaStream_t stream) {
  switch (block_cols(BH, a.D, a.M)) {
    case 64: return launch<T, 64>(a, BH, backward, stream);
    case 32: return launch<T, 32>(a, BH, backward, stream);
    default: return launch<T, 16>(a, BH, backward, stream);
  }
}

cudaError_t run(const Args& a, int64_t BH, cp_dtype_t dtype, bool backward, cudaStream_t stream) {
  if (dtype == CP_DTYPE_BF16) return run<__nv_bfloat16>(a, BH, backward, stream);
  if (dtype == CP_DTYPE_F16) return run<__half>(a, BH, backward, stream);
  return run<float>(a, BH, backward, stream);
}

int n_blocks(const DeltaShape& s) {
  const int mb = block_cols(s.B * s.H, s.D, s.M);
  return (int)((s.M + mb - 1) / mb);
}
bool has_parts(const DeltaShape& s) { return s.H != s.Hk || n_blocks(s) > 1; }

}  // namespace

cudaError_t delta_join_launch(const DeltaJoin& x, cp_dtype_t dtype, cudaStream_t stream) {
  const int64_t n = std::max(x.N * x.D * x.heads, x.dg == nullptr ? 0 : x.N * x.heads * x.group);
  const dim3 grid((unsigned)((n + 255) / 256), x.dg == nullptr ? 2 : 4);
  if (dtype == CP_DTYPE_BF16)
    delta_join_kernel<__nv_bfloat16><<<grid, 256, 0, stream>>>(x);
  else if (dtype == CP_DTYPE_F16)
    delta_join_kernel<__half><<<grid, 256, 0, stream>>>(x);
  else
    delta_join_kernel<float><<<grid, 256, 0, stream>>>(x);
  return cudaGetLastError();
}

int delta_simt_chunk() { return kC; }

size_t delta_simt_scratch(const DeltaShape& s, bool backward) {
  if (!backward || !has_parts(s)) return 0;
  return sizeof(float) * (size_t)n_blocks(s) * s.B * s.H * s.N * (2 * s.D + 2);
}

cudaError_t delta_simt_fwd(const DeltaShape& s, const DeltaFwd& f, cudaStream_t stream) {
  Args a{};
  a.q = f.q; a.k = f.k; a.v = f.v; a.g = f.g; a.beta = f.beta;
  a.state_in = f.state_in; a.out = f.out; a.state_out = f.state_out; a.ckpt = f.ckpt;
  a.N = s.N; a.D = (int)s.D; a.M = (int)s.M; a.H = (int)s.H; a.group = (int)(s.H / s.Hk);
  a.scale = s.scale;
  return run(a, s.B * s.H, s.dtype, false, stream);
}

cudaError_t delta_simt_bwd(const DeltaShape& s, const DeltaBwd& f, void* scratch,
                           cudaStream_t stream) {
  Args a{};
  a.q = f.q; a.k = f.k; a.v = f.v; a.g = f.g; a.beta = f.beta; a.go = f.grad_out;
  a.ckpt = const_cast<float*>(f.ckpt); a.grad_state_out = f.grad_state_out;
  a.dq = f.dq; a.dk = f.dk; a.dv = f.dv; a.dg = f.dg; a.dbeta = f.dbeta;
  a.grad_state_in = f.grad_state_in;
  a.N = s.N; a.D = (int)s.D; a.M = (int)s.M; a.H = (int)s.H; a.group = (int)(s.H / s.Hk);
  a.scale = s.scale;
  const int64_t BH = s.B * s.H;
  if (!has_parts(s)) return run(a, BH, s.dtype, true, stream);
  const int n_mb = n_blocks(s);
  const int64_t rows = n_mb * BH * s.N;
  a.dq_part = static_cast<float*>(scratch);
  a.dk_part = a.dq_part + rows * s.D;
  a.dg_part = a.dk_part + rows * s.D;
  a.db_part = a.dg_part + rows;
  cudaError_t e = run(a, BH, s.dtype, true, stream);
  if (e != cudaSuccess) return e;
  return delta_join_launch({a.dq_part, a.dk_part, a.dg_part, a.db_part, f.dq, f.dk, f.dg, f.dbeta,
                            s.N, s.D, s.B * s.Hk, a.group, n_mb},
                           s.dtype, stream);
}

}  // namespace cp
