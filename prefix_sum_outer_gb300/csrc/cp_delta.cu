// The gated delta rule on the CUDA cores in fp32: the path of fp32 and fp16
// inputs (widened on load) and of the bf16 shapes the tensor-core kernels do
// not take (D > 128).  The formulas are in cp_delta.cuh.
//
// Forward: one CTA per (head, block of MB value columns) walks the sequence in
// chunks of 32 rows with the D x MB state in shared memory; the value columns
// of a head never meet, so a block of them is a problem of its own.  A chunk is
// six small products on shared-memory tiles and a triangular solve by
// substitution, one thread per value column.
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
#include <algorithm>

#include "cp_delta.cuh"

namespace cp {
namespace {

using namespace delta;

constexpr int kThreads = 256;
constexpr int kC = 32;  // rows of a chunk

// out(i, j) = sum_k a(i, k) b(k, j) for i < R, j < N over the CTA: warp w takes
// rows w, w + 8, .., lane l columns l, l + 32, ..; a is read as a broadcast and
// b by consecutive lanes (rows of odd pitch keep either orientation free of
// bank conflicts).
template <int RT, int CT, class FA, class FB, class FE>
__device__ __forceinline__ void mm(int R, int N, int K, FA a, FB b, FE e) {
  const int w = threadIdx.x / 32, l = threadIdx.x % 32;
  for (int i0 = w; i0 < R; i0 += 8 * RT) {
    for (int j0 = l; j0 < N; j0 += 32 * CT) {
      float acc[RT][CT] = {};
      int ii[RT], jj[CT];
#pragma unroll
      for (int r = 0; r < RT; ++r) ii[r] = min(i0 + 8 * r, R - 1);
#pragma unroll
      for (int c = 0; c < CT; ++c) jj[c] = min(j0 + 32 * c, N - 1);
#pragma unroll 4
      for (int k = 0; k < K; ++k) {
        float av[RT], bv[CT];
#pragma unroll
        for (int r = 0; r < RT; ++r) av[r] = a(ii[r], k);
#pragma unroll
        for (int c = 0; c < CT; ++c) bv[c] = b(k, jj[c]);
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
          for (int c = 0; c < CT; ++c) acc[r][c] = fmaf(av[r], bv[c], acc[r][c]);
      }
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int c = 0; c < CT; ++c)
          if (i0 + 8 * r < R && j0 + 32 * c < N) e(ii[r], jj[c], acc[r][c]);
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

// rows [i0, i0 + 32) of a [N][ncol] matrix (columns [c0, c0 + nc)) as fp32
// rows of pitch ld; rows past N are zero
template <typename T>
__device__ __forceinline__ void load_rows(float* dst, int ld, const T* src, int64_t i0, int64_t N,
                                          int ncol, int c0, int nc) {
  for (int e = threadIdx.x; e < kC * nc; e += kThreads) {
    const int i = e / nc, c = e % nc;
    dst[i * ld + c] = i0 + i < N ? ld_f32<T>(src + (i0 + i) * ncol + c0 + c) : 0.f;
  }
}

struct Gates {
  float2 G[kC];   // running sums of the log decay
  float b[kC], gam[kC], del[kC];
  float last;     // gam of the last row
};

__device__ __forceinline__ void load_gates(Gates& s, const float* g, const float* beta, int64_t i0,
                                           int64_t N) {
  if (threadIdx.x < 32) {
    const int i = threadIdx.x;
    const bool on = i0 + i < N;
    const float2 G = warp_scan(split_decay(on ? g[i0 + i] : 0.f), i);
    const float2 E = make_float2(__shfl_sync(0xffffffffu, G.x, 31), __shfl_sync(0xffffffffu, G.y, 31));
    const float2 zero = make_float2(0.f, 0.f);
    s.G[i] = G;
    s.b[i] = on ? beta[i0 + i] : 0.f;
    s.gam[i] = decay_between(G, zero);
    s.del[i] = decay_between(E, G);
    if (i == 0) s.last = decay_between(E, zero);
  }
}

template <typename T, int MB>
__global__ void __launch_bounds__(kThreads) delta_fwd_kernel(Args p) {
  extern __shared__ float sm[];
  const int D = p.D, M = p.M, ldd = D + 1;
  constexpr int ldm = MB + 1, ldc = kC + 1;
  float* S = sm;                 // [D][ldm]
  float* K = S + D * ldm;        // [kC][ldd]
  float* Q = K + kC * ldd;       // [kC][ldd]
  float* U = Q + kC * ldd;       // [kC][ldm]  V, then b R, then U
  float* O = U + kC * ldm;       // [kC][ldm]
  float* A = O + kC * ldm;       // [kC][ldc]
  float* P = A + kC * ldc;       // [kC][ldc]
  __shared__ Gates gt;
  const int64_t p_ = blockIdx.x;
  const int c0 = blockIdx.y * MB, nc = min(MB, M - c0);
  const int64_t N = p.N, pk = (p_ / p.H) * (p.H / p.group) + (p_ % p.H) / p.group;
  const T* q = static_cast<const T*>(p.q) + pk * N * D;
  const T* k = static_cast<const T*>(p.k) + pk * N * D;
  const T* v = static_cast<const T*>(p.v) + p_ * N * M;
  T* out = static_cast<T*>(p.out) + p_ * N * M;
  const int64_t n_chunks = (N + kC - 1) / kC;
  for (int e = threadIdx.x; e < D * nc; e += kThreads) {
    const int d = e / nc, c = e % nc;
    S[d * ldm + c] = p.state_in != nullptr ? p.state_in[(p_ * D + d) * M + c0 + c] : 0.f;
  }
  for (int64_t ch = 0; ch < n_chunks; ++ch) {
    const int64_t i0 = ch * kC;
    __syncthreads();
    load_rows<T>(K, ldd, k, i0, N, D, 0, D);
    load_rows<T>(Q, ldd, q, i0, N, D, 0, D);
    load_rows<T>(U, ldm, v, i0, N, M, c0, nc);
    load_gates(gt, p.g + p_ * N, p.beta + p_ * N, i0, N);
    if (p.ckpt != nullptr)
      for (int e = threadIdx.x; e < D * nc; e += kThreads) {
        const int d = e / nc, c = e % nc;
        p.ckpt[((p_ * n_chunks + ch) * D + d) * M + c0 + c] = S[d * ldm + c];
      }
    __syncthreads();
    mm<4, 1>(kC, kC, D, [&](int i, int x) { return K[i * ldd + x]; },
             [&](int x, int j) { return K[j * ldd + x]; }, [&](int i, int j, float a) {
               A[i * ldc + j] = j < i ? gt.b[i] * decay_between(gt.G[i], gt.G[j]) * a : 0.f;
             });
    mm<4, 1>(kC, kC, D, [&](int i, int x) { return Q[i * ldd + x]; },
             [&](int x, int j) { return K[j * ldd + x]; }, [&](int i, int j, float a) {
               P[i * ldc + j] = j <= i ? p.scale * decay_between(gt.G[i], gt.G[j]) * a : 0.f;
             });
    mm<4, 2>(kC, nc, D, [&](int i, int x) { return K[i * ldd + x]; },
             [&](int x, int j) { return S[x * ldm + j]; }, [&](int i, int j, float a) {
               U[i * ldm + j] = gt.b[i] * (U[i * ldm + j] - gt.gam[i] * a);
             });
    mm<4, 2>(kC, nc, D, [&](int i, int x) { return Q[i * ldd + x]; },
             [&](int x, int j) { return S[x * ldm + j]; },
             [&](int i, int j, float a) { O[i * ldm + j] = p.scale * gt.gam[i] * a; });
    __syncthreads();
    if (threadIdx.x < nc) {
      const int c = threadIdx.x;
      float u[kC];
#pragma unroll
      for (int i = 0; i < kC; ++i) {
        float x = U[i * ldm + c];
#pragma unroll
        for (int j = 0; j < i; ++j) x = fmaf(-A[i * ldc + j], u[j], x);
        u[i] = x;
        U[i * ldm + c] = x;
      }
    }
    __syncthreads();
    mm<4, 2>(kC, nc, kC, [&](int i, int x) { return P[i * ldc + x]; },
             [&](int x, int j) { return U[x * ldm + j]; }, [&](int i, int j, float a) {
               if (i0 + i < N) out[(i0 + i) * M + c0 + j] = from_f32<T>(O[i * ldm + j] + a);
             });
    mm<4, 2>(D, nc, kC, [&](int d, int x) { return K[x * ldd + d] * gt.del[x]; },
             [&](int x, int j) { return U[x * ldm + j]; },
             [&](int d, int j, float a) { S[d * ldm + j] = fmaf(gt.last, S[d * ldm + j], a); });
  }
  __syncthreads();
  if (p.state_out != nullptr)
    for (int e = threadIdx.x; e < D * nc; e += kThreads) {
      const int d = e / nc, c = e % nc;
      p.state_out[(p_ * D + d) * M + c0 + c] = S[d * ldm + c];
    }
}

template <typename T, int MB>
__global__ void __launch_bounds__(kThreads) delta_bwd_kernel(Args p) {
  extern __shared__ float sm[];
  const int D = p.D, M = p.M, ldd = D + 1;
  constexpr int ldm = MB + 1, ldc = kC + 1;
  float* S = sm;                   // [D][ldm]  state before the chunk
  float* dS = S + D * ldm;         // [D][ldm]  gradient of the state after it
  float* K = dS + D * ldm;         // [kC][ldd]
  float* Q = K + kC * ldd;         // [kC][ldd]
  float* R = Q + kC * ldd;         // [kC][ldm]  V, then R
  float* dO = R + kC * ldm;        // [kC][ldm]
  float* U = dO + kC * ldm;        // [kC][ldm]
  float* dX = U + kC * ldm;        // [kC][ldm]  dU, then dX
  float* QS = dX + kC * ldm;       // [kC][ldm]
  float* KS = QS + kC * ldm;       // [kC][ldm]
  float* KD = KS + kC * ldm;       // [kC][ldm]  K dS'
  float* KK = KD + kC * ldm;       // [kC][ldc]
  float* QK = KK + kC * ldc;       // [kC][ldc]
  float* Gm = QK + kC * ldc;       // [kC][ldc]  Gam
  float* Mq = Gm + kC * ldc;       // [kC][ldc]
  float* Ma = Mq + kC * ldc;       // [kC][ldc]
  float* row = Ma + kC * ldc;      // [kC] r_i, [kC] c_j
  __shared__ Gates gt;
  __shared__ float red[8], zdot;
  const int64_t p_ = blockIdx.x;
  const int c0 = blockIdx.y * MB, nc = min(MB, M - c0);
  const int64_t N = p.N, pk = (p_ / p.H) * (p.H / p.group) + (p_ % p.H) / p.group;
  const T* q = static_cast<const T*>(p.q) + pk * N * D;
  const T* k = static_cast<const T*>(p.k) + pk * N * D;
  const T* v = static_cast<const T*>(p.v) + p_ * N * M;
  const T* go = static_cast<const T*>(p.go) + p_ * N * M;
  T* dv = static_cast<T*>(p.dv) + p_ * N * M;
  const int64_t part = ((int64_t)blockIdx.y * gridDim.x + p_) * N;
  const int64_t n_chunks = (N + kC - 1) / kC;
  const int w = threadIdx.x / 32, l = threadIdx.x % 32;
  for (int e = threadIdx.x; e < D * nc; e += kThreads) {
    const int d = e / nc, c = e % nc;
    dS[d * ldm + c] = p.grad_state_out != nullptr ? p.grad_state_out[(p_ * D + d) * M + c0 + c] : 0.f;
  }
  for (int64_t ch = n_chunks - 1; ch >= 0; --ch) {
    const int64_t i0 = ch * kC;
    __syncthreads();
    load_rows<T>(K, ldd, k, i0, N, D, 0, D);
    load_rows<T>(Q, ldd, q, i0, N, D, 0, D);
    load_rows<T>(R, ldm, v, i0, N, M, c0, nc);
    load_rows<T>(dO, ldm, go, i0, N, M, c0, nc);
    load_gates(gt, p.g + p_ * N, p.beta + p_ * N, i0, N);
    for (int e = threadIdx.x; e < D * nc; e += kThreads) {
      const int d = e / nc, c = e % nc;
      S[d * ldm + c] = p.ckpt[((p_ * n_chunks + ch) * D + d) * M + c0 + c];
    }
    __syncthreads();
    mm<4, 1>(kC, kC, D, [&](int i, int x) { return K[i * ldd + x]; },
             [&](int x, int j) { return K[j * ldd + x]; }, [&](int i, int j, float a) {
               KK[i * ldc + j] = a;
               Gm[i * ldc + j] = j <= i ? decay_between(gt.G[i], gt.G[j]) : 0.f;
             });
    mm<4, 1>(kC, kC, D, [&](int i, int x) { return Q[i * ldd + x]; },
             [&](int x, int j) { return K[j * ldd + x]; },
             [&](int i, int j, float a) { QK[i * ldc + j] = a; });
    mm<4, 2>(kC, nc, D, [&](int i, int x) { return K[i * ldd + x]; },
             [&](int x, int j) { return S[x * ldm + j]; }, [&](int i, int j, float a) {
               KS[i * ldm + j] = a;
               R[i * ldm + j] -= gt.gam[i] * a;
               U[i * ldm + j] = gt.b[i] * R[i * ldm + j];
             });
    mm<4, 2>(kC, nc, D, [&](int i, int x) { return Q[i * ldd + x]; },
             [&](int x, int j) { return S[x * ldm + j]; },
             [&](int i, int j, float a) { QS[i * ldm + j] = a; });
    mm<4, 2>(kC, nc, D, [&](int i, int x) { return K[i * ldd + x]; },
             [&](int x, int j) { return dS[x * ldm + j]; },
             [&](int i, int j, float a) { KD[i * ldm + j] = a; });
    __syncthreads();
    // dU, and <S, dS'>
    mm<4, 2>(kC, nc, kC, [&](int i, int x) { return QK[x * ldc + i] * Gm[x * ldc + i]; },
             [&](int x, int j) { return dO[x * ldm + j]; }, [&](int i, int j, float a) {
               dX[i * ldm + j] = p.scale * a + gt.del[i] * KD[i * ldm + j];
             });
    float z = 0.f;
    for (int d = w; d < D; d += 8)
      for (int c = l; c < nc; c += 32) z = fmaf(S[d * ldm + c], dS[d * ldm + c], z);
    for (int o = 16; o > 0; o /= 2) z += __shfl_xor_sync(0xffffffffu, z, o);
    if (l == 0) red[w] = z;
    __syncthreads();
    if (threadIdx.x < nc) {
      const int c = threadIdx.x;
      float u[kC];
#pragma unroll
      for (int i = 0; i < kC; ++i) {
        float x = 0.f;
#pragma unroll
        for (int j = 0; j < i; ++j) x = fmaf(KK[i * ldc + j] * Gm[i * ldc + j], u[j], x);
        u[i] = U[i * ldm + c] - gt.b[i] * x;
        U[i * ldm + c] = u[i];
      }
    } else if (threadIdx.x >= 128 && threadIdx.x < 128 + nc) {
      const int c = threadIdx.x - 128;
      float x[kC];
#pragma unroll
      for (int i = kC - 1; i >= 0; --i) {
        float y = dX[i * ldm + c];
#pragma unroll
        for (int j = i + 1; j < kC; ++j)
          y = fmaf(-gt.b[j] * KK[j * ldc + i] * Gm[j * ldc + i], x[j], y);
        x[i] = y;
        dX[i * ldm + c] = y;
        if (i0 + i < N) dv[(i0 + i) * M + c0 + c] = from_f32<T>(gt.b[i] * y);
      }
    }
    if (threadIdx.x == 255) {
      float s = 0.f;
      for (int i = 0; i < 8; ++i) s += red[i];
      zdot = gt.last * s;
    }
    __syncthreads();
    // dP and dA, weighted
    mm<4, 1>(kC, kC, nc, [&](int i, int x) { return dO[i * ldm + x]; },
             [&](int x, int j) { return U[j * ldm + x]; },
             [&](int i, int j, float a) { Mq[i * ldc + j] = p.scale * Gm[i * ldc + j] * a; });
    mm<4, 1>(kC, kC, nc, [&](int i, int x) { return dX[i * ldm + x]; },
             [&](int x, int j) { return U[j * ldm + x]; }, [&](int i, int j, float a) {
               // without b: db needs it so, and b enters below
               Ma[i * ldc + j] = j < i ? -Gm[i * ldc + j] * a : 0.f;
             });
    __syncthreads();
    // row sums: db, the parts of dg with S and with dS'
    for (int i = w; i < kC; i += 8) {
      float db = 0.f, r = 0.f, cc = 0.f;
      for (int c = l; c < nc; c += 32) {
        const float x = dX[i * ldm + c];
        db = fmaf(x, R[i * ldm + c], db);
        r += p.scale * dO[i * ldm + c] * QS[i * ldm + c] - gt.b[i] * x * KS[i * ldm + c];
        cc = fmaf(U[i * ldm + c], KD[i * ldm + c], cc);
      }
      db = fmaf(Ma[i * ldc + l], KK[i * ldc + l], db);
      for (int o = 16; o > 0; o /= 2) {
        db += __shfl_xor_sync(0xffffffffu, db, o);
        r += __shfl_xor_sync(0xffffffffu, r, o);
        cc += __shfl_xor_sync(0xffffffffu, cc, o);
      }
      if (l == 0) {
        row[i] = gt.gam[i] * r;
        row[kC + i] = gt.del[i] * cc;
        if (i0 + i < N) {
          if (p.db_part != nullptr)
            p.db_part[part + i0 + i] = db;
          else
            p.dbeta[p_ * N + i0 + i] = db;
        }
      }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < kC * kC; e += kThreads) {
      const int i = e / kC, j = e % kC;
      Ma[i * ldc + j] *= gt.b[i];
      // the pair's weight in dg takes the place of q.k, which it is made from
      QK[i * ldc + j] = Mq[i * ldc + j] * QK[i * ldc + j] + Ma[i * ldc + j] * KK[i * ldc + j];
    }
    __syncthreads();
    // dg_t: warp w takes t = w, w + 8, ..: lane j < t sums its column from row
    // t on; lane l >= t adds row l's part
    for (int t = w; t < kC; t += 8) {
      float s = 0.f;
      if (l < t) {
        for (int i = t; i < kC; ++i) s += QK[i * ldc + l];
        s += row[kC + l];
      } else {
        s = row[l];
      }
      for (int o = 16; o > 0; o /= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
      s += zdot;
      if (l == 0 && i0 + t < N) {
        if (p.dg_part != nullptr)
          p.dg_part[part + i0 + t] = s;
        else
          p.dg[p_ * N + i0 + t] = s;
      }
    }
    // dQ and dK, two products each into registers by way of shared memory:
    // KS and QS become s gam dO and gam dR
    __syncthreads();
    for (int e = threadIdx.x; e < kC * nc; e += kThreads) {
      const int i = e / nc, c = e % nc;
      QS[i * ldm + c] = p.scale * gt.gam[i] * dO[i * ldm + c];
      KS[i * ldm + c] = gt.gam[i] * gt.b[i] * dX[i * ldm + c];
      KD[i * ldm + c] = gt.del[i] * U[i * ldm + c];
    }
    __syncthreads();
    {
      constexpr int RT = 4, CT = 2;
      for (int j0 = l; j0 < D; j0 += 32 * CT) {
        float aq[RT][CT] = {}, ak[RT][CT] = {};
        int jj[CT];
#pragma unroll
        for (int c = 0; c < CT; ++c) jj[c] = min(j0 + 32 * c, D - 1);
        for (int x = 0; x < nc; ++x) {
          float sv[CT], dsv[CT];
#pragma unroll
          for (int c = 0; c < CT; ++c) {
            sv[c] = S[jj[c] * ldm + x];
            dsv[c] = dS[jj[c] * ldm + x];
          }
#pragma unroll
          for (int r = 0; r < RT; ++r) {
            const int i = w + 8 * r;
            const float a = QS[i * ldm + x], b = KS[i * ldm + x], u = KD[i * ldm + x];
#pragma unroll
            for (int c = 0; c < CT; ++c) {
              aq[r][c] = fmaf(a, sv[c], aq[r][c]);
              ak[r][c] = fmaf(u, dsv[c], fmaf(-b, sv[c], ak[r][c]));
            }
          }
        }
        for (int x = 0; x < kC; ++x) {
          float kv[CT], qv[CT];
#pragma unroll
          for (int c = 0; c < CT; ++c) {
            kv[c] = K[x * ldd + jj[c]];
            qv[c] = Q[x * ldd + jj[c]];
          }
#pragma unroll
          for (int r = 0; r < RT; ++r) {
            const int i = w + 8 * r;
            const float a = Mq[i * ldc + x], at = Mq[x * ldc + i];
            const float m = Ma[i * ldc + x] + Ma[x * ldc + i];
#pragma unroll
            for (int c = 0; c < CT; ++c) {
              aq[r][c] = fmaf(a, kv[c], aq[r][c]);
              ak[r][c] = fmaf(at, qv[c], fmaf(m, kv[c], ak[r][c]));
            }
          }
        }
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
          for (int c = 0; c < CT; ++c) {
            const int64_t i = i0 + w + 8 * r;
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
    }
    __syncthreads();
    mm<4, 2>(D, nc, kC, [&](int d, int x) { return Q[x * ldd + d]; },
             [&](int x, int j) { return QS[x * ldm + j]; },
             [&](int d, int j, float a) { dS[d * ldm + j] = fmaf(gt.last, dS[d * ldm + j], a); });
    mm<4, 2>(D, nc, kC, [&](int d, int x) { return K[x * ldd + d]; },
             [&](int x, int j) { return KS[x * ldm + j]; },
             [&](int d, int j, float a) { dS[d * ldm + j] -= a; });
  }
  __syncthreads();
  if (p.grad_state_in != nullptr)
    for (int e = threadIdx.x; e < D * nc; e += kThreads) {
      const int d = e / nc, c = e % nc;
      p.grad_state_in[(p_ * D + d) * M + c0 + c] = dS[d * ldm + c];
    }
}

// out[b][hk][i] = sum over the column blocks and the group's heads of parts
// [n_mb][B][Hk][group][rows], in that order
template <typename T>
__global__ void __launch_bounds__(256)
    delta_join_kernel(const float* __restrict__ part, T* __restrict__ out, int64_t rows,
                      int64_t heads, int group, int n_mb) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, n = rows * heads;
  if (i >= n) return;
  const int64_t h = i / rows, r = i % rows;
  float s = 0.f;
  for (int m = 0; m < n_mb; ++m)
    for (int g = 0; g < group; ++g) s += part[((int64_t)m * heads * group + h * group + g) * rows + r];
  out[i] = from_f32<T>(s);
}

// Value columns of a CTA: 64 while two D x 64 fp32 tiles and the row tiles fit
// the shared memory (D <= 128), else 32.
int block_cols(int64_t D, int64_t M) { return D <= 128 && M > 32 ? 64 : 32; }

size_t fwd_smem(int64_t D, int mb) {
  return sizeof(float) * (size_t)(D * (mb + 1) + 2 * kC * (D + 1) + 2 * kC * (mb + 1) + 2 * kC * (kC + 1));
}
size_t bwd_smem(int64_t D, int mb) {
  return sizeof(float) *
         (size_t)(2 * D * (mb + 1) + 2 * kC * (D + 1) + 7 * kC * (mb + 1) + 5 * kC * (kC + 1) + 2 * kC);
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
  return block_cols(a.D, a.M) == 64 ? launch<T, 64>(a, BH, backward, stream)
                                    : launch<T, 32>(a, BH, backward, stream);
}

cudaError_t run(const Args& a, int64_t BH, cp_dtype_t dtype, bool backward, cudaStream_t stream) {
  if (dtype == CP_DTYPE_BF16) return run<__nv_bfloat16>(a, BH, backward, stream);
  if (dtype == CP_DTYPE_F16) return run<__half>(a, BH, backward, stream);
  return run<float>(a, BH, backward, stream);
}

int n_blocks(int64_t D, int64_t M) {
  const int mb = block_cols(D, M);
  return (int)((M + mb - 1) / mb);
}
bool has_parts(const DeltaShape& s) { return s.H != s.Hk || n_blocks(s.D, s.M) > 1; }

}  // namespace

cudaError_t delta_join_launch(const float* part, void* out, int64_t rows, int64_t heads, int group,
                              int n_mb, cp_dtype_t dtype, cudaStream_t stream) {
  const unsigned grid = (unsigned)((rows * heads + 255) / 256);
  if (dtype == CP_DTYPE_BF16)
    delta_join_kernel<<<grid, 256, 0, stream>>>(part, static_cast<__nv_bfloat16*>(out), rows, heads,
                                                group, n_mb);
  else if (dtype == CP_DTYPE_F16)
    delta_join_kernel<<<grid, 256, 0, stream>>>(part, static_cast<__half*>(out), rows, heads, group,
                                                n_mb);
  else
    delta_join_kernel<<<grid, 256, 0, stream>>>(part, static_cast<float*>(out), rows, heads, group,
                                                n_mb);
  return cudaGetLastError();
}

int delta_simt_chunk() { return kC; }

size_t delta_simt_scratch(const DeltaShape& s, bool backward) {
  if (!backward || !has_parts(s)) return 0;
  return sizeof(float) * (size_t)n_blocks(s.D, s.M) * s.B * s.H * s.N * (2 * s.D + 2);
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
  const int n_mb = n_blocks(s.D, s.M);
  const int64_t rows = n_mb * BH * s.N;
  a.dq_part = static_cast<float*>(scratch);
  a.dk_part = a.dq_part + rows * s.D;
  a.dg_part = a.dk_part + rows * s.D;
  a.db_part = a.dg_part + rows;
  cudaError_t e = run(a, BH, s.dtype, true, stream);
  if (e != cudaSuccess) return e;
  const int64_t heads = s.B * s.Hk;
  e = delta_join_launch(a.dq_part, f.dq, s.N * s.D, heads, a.group, n_mb, s.dtype, stream);
  if (e == cudaSuccess)
    e = delta_join_launch(a.dk_part, f.dk, s.N * s.D, heads, a.group, n_mb, s.dtype, stream);
  if (e == cudaSuccess)
    e = delta_join_launch(a.dg_part, f.dg, s.N, BH, 1, n_mb, CP_DTYPE_F32, stream);
  if (e == cudaSuccess)
    e = delta_join_launch(a.db_part, f.dbeta, s.N, BH, 1, n_mb, CP_DTYPE_F32, stream);
  return e;
}

}  // namespace cp
