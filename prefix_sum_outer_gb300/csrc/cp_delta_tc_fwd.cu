// Forward of the gated delta rule on the tensor cores (bf16, D <= 128), two
// launches for the sequence or for each of a few pieces of it:
//
// 1. What a chunk needs of its own keys, queries and gates, one CTA per value
//    head and chunk: [K; Q] K^T by MMA, A and P from it by the decays, T = (I +
//    A)^-1 by blocks, P T by MMA; the tiles of T, P T (and, for a backward, P)
//    go to memory as they lie in shared memory.  A CTA's steps wait for one
//    another, so what counts is CTAs to an SM: T lies over what it is made from
//    and P T over P, in both memories, and four fit.  B = 8, H = 16, N = 4096, D =
//    64, with P kept: 158 us, 4.3 TB/s.
//
// 2. The chain.  A CTA walks one head's chunks of 64 rows for 32 value columns
//    (columns never meet), two warpgroups of 16 columns each; lane d holds row
//    d of the fp32 state in registers.  A chunk is three MMAs:
//        [K; Q] S          -> KS (lanes 0-63), QS (lanes 64-127)
//        R = b (V - gam KS) -> shared memory
//        [T; P T] R        -> U (lanes 0-63), P U (lanes 64-127)
//        out = s gam QS + P U;   del U -> shared memory
//        K^T (del U)       -> S = gam_C S + it, -> shared memory
//    P T in place of P takes a fourth dependent step (P U) off the chain and
//    gives both products one 128-lane MMA.  The chain is bound by its own
//    latency, 400 to 700 cycles to a product and 300 to 700 to a conversion of 16
//    columns, so it is cut into few columns a CTA (64 columns took 4.6k cycles a
//    chunk where 32 took 3.4k, with factors in two parts).  Past 32 KB of
//    instructions every one of them takes 3.1 cycles to fetch (measured): the two
//    launches' work in one kernel, with a chunk's matrices made two ahead by
//    warps beside the chain, took 7.4k cycles a chunk.  B = 8, H = 16, N = 4096, D =
//    M = 64, two CTAs to an SM: 204 us with what a backward needs kept, 5.5 TB/s.
//    B = 4, H = 8, N = 8229, D = 128, M = 64, 64 CTAs: 297 us in four pieces, 4.5k
//    cycles a chunk (4.0k where the copies' source is in L2).
#include <algorithm>

#include "cp_delta_tc.cuh"

namespace cp {
namespace {

using namespace delta;

// ------------------------------------------------------- a chunk's matrices
struct PrepArgs {
  const float *g, *beta;
  uint8_t *t, *pt, *p;  // [BH][chunks] x 24 KB each (three parts); p may be null
  int* status;
  int64_t N;
  int n_chunks, chunk0, span, H, group;  // of n_chunks: span chunks from chunk0 on
  bool beside;                           // beside the chain over the piece before
  float scale;
};

template <int DP>
struct PrepLayout {
  static constexpr int kBoxes = DP / 64;
  static constexpr int kKQBox = 2 * kBox;
  static constexpr int kKQ = kBoxes * kKQBox;
  // K and Q are done with before A and P are written: T (three parts) lies over
  // the blocks that it is made from and these over K and Q, P and then P T behind
  // them.  A product with a part of T reads 64 rows past it, of the next.
  static constexpr int oKQ = 0;
  static constexpr int oInv = 0;
  static constexpr int oT = 0;
  static constexpr int oP = kTTile;
  static constexpr int oG = 2 * kTTile;
  static constexpr int oBar = oG + (int)sizeof(GateSlot);
  static constexpr int kBytes = oBar + 64 + 1024;
  static constexpr int kPerSM = 4;
  static_assert(kKQ <= oG && sizeof(InvTiles) <= kTTile, "places");
  static_assert(kPerSM * (kBytes + 1024) <= 233472, "shared memory");
  static_assert(sizeof(InvTiles) % 16 == 0 && sizeof(GateSlot) % 16 == 0, "alignment");
};

template <int DP>
__global__ void __launch_bounds__(128, PrepLayout<DP>::kPerSM)
    delta_tc_prep_kernel(const __grid_constant__ CUtensorMap tm_q,
                         const __grid_constant__ CUtensorMap tm_k, const PrepArgs a) {
  using L = PrepLayout<DP>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = align_tiles(smem_raw);
  GateSlot* gs = reinterpret_cast<GateSlot*>(sm + L::oG);
  InvTiles* it = reinterpret_cast<InvTiles*>(sm + L::oInv);
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + L::oBar);
  uint64_t* done = full + 1;  // [2]
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(full + 3);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  const int w = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0);  // (uniform to the compiler)
  const int lane = threadIdx.x % 32, t = threadIdx.x;
  const int64_t p = blockIdx.x / a.span;
  const int chunk = a.chunk0 + blockIdx.x % a.span, i0 = chunk * kCh;
  const int pk = (int)((p / a.H) * (a.H / a.group) + (p % a.H) / a.group);
  if (!a.beside) grid_dep_wait();
  float4 gb = make_float4(0.f, 0.f, 0.f, 0.f);
  if (w == 3) {
    const int64_t i = i0 + lane, at = p * a.N;
    gb = make_float4(i < a.N ? a.g[at + i] : 0.f, i + 32 < a.N ? a.g[at + i + 32] : 0.f,
                     i < a.N ? a.beta[at + i] : 0.f, i + 32 < a.N ? a.beta[at + i + 32] : 0.f);
  }
  if (t == 0) {
    for (int i = 0; i < 3; ++i) mbar_init(full + i, 1);
    *abort_flag = 0;
    fence_mbar_init();
    mbar_arrive_expect_tx(full, L::kKQ);
    const uint64_t keep = policy_evict_last();  // the chain reads K and Q again
    for (int x = 0; x < L::kBoxes; ++x) {
      tma_load_3d(sm + L::oKQ + x * L::kKQBox, &tm_k, full, 64 * x, i0, pk, keep);
      tma_load_3d(sm + L::oKQ + x * L::kKQBox + kBox, &tm_q, full, 64 * x, i0, pk, keep);
    }
  }
  if (w == 0) {
    tmem_alloc(tmem_holder, 64);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_holder, 0), t_pt = tmem;  // one after the other
  const uint32_t s_base = smem_u32(sm), lane_base = (uint32_t)w << 21;
  const uint32_t T_addr = s_base + L::oT, P_addr = s_base + L::oP;
  constexpr uint32_t id_nn64 = idesc_bf16_f32(128, 64, 0, 0);  // A [rows x K], B [cols x K]
  if (w == 0) {
    wait_or_abort(full, 0, a.status, abort_flag);
    __syncwarp();
    const uint32_t el = elect_one();
    mma_tile<DP / 16, false, false>(el, tmem, s_base + L::oKQ, s_base + L::oKQ, id_nn64, 16, 16,
                                    L::kKQBox, L::kKQBox, true);
    if (el) mma_commit(done);
  }
  if (w == 3) {  // under the product
    write_gates(gs, lane, gb.x, gb.y, gb.z, gb.w);
  }
  __syncthreads();
  wait_or_abort(done, 0, a.status, abort_flag);
  tc_fence_after();
  // A by the lanes of K, P by those of Q
  const int i = t & 63;
  decayed_row(tmem + lane_base, gs, i, w >= 2, w & 1, w < 2 ? gs->b[i] : a.scale,
              [&](int cb, const float2(&v)[8]) {
                if (w < 2)
                  put_a16(it, i, cb, v);
                else
                  store16_split(sm + L::oP, kBox, i, 2 * cb, v);
              });
  __syncthreads();
  uint4 xw[2], xw3[2];
  uint32_t z[4][3][4];
  invert_diag(it, w, lane, xw, xw3);
  __syncthreads();
  invert_below(it, w, lane, z);
  __syncthreads();
  put_t_transposed(sm + L::oT, kBox, w, lane, xw, xw3, z);
  tc_fence_before();
  fence_proxy_async_smem();
  __syncthreads();
  const int64_t tile = (p * a.n_chunks + chunk) * (int64_t)kTTile;
  if (w == 0) {
    tc_fence_after();
    const uint32_t el = elect_one();
    // (P T)^T = T^T P^T; lanes 0-63 are read
#pragma unroll 1
    for (int x = 2; x >= 0; --x)
#pragma unroll 1
      for (int y = x; y >= 0; --y)
        mma_tile<4, false, false>(el, t_pt, T_addr + y * kBox, P_addr + (x - y) * kBox, id_nn64, 16, 16,
                                  0, 0, x == 2 && y == 2);
    if (el) mma_commit(done + 1);
  }
  if (t == 0) {
    bulk_store(a.t + tile, sm + L::oT, kTTile);
    if (a.p != nullptr) bulk_store(a.p + tile, sm + L::oP, kTTile);
    tma_store_commit();
    if (a.p != nullptr) tma_store_wait_read_all();
  }
  wait_or_abort(done + 1, 0, a.status, abort_flag);
  tc_fence_after();
  if (a.p != nullptr) __syncthreads();  // P has been read
  if (w < 2) {
#pragma unroll 1
    for (int h = 0; h < 4; ++h) {
      float2 v[8];
      tmem_ld16(t_pt + lane_base + 16 * h, v);
      store16_split(sm + L::oP, kBox, t, 2 * h, v);
    }
  }
  tc_fence_before();
  fence_proxy_async_smem();
  __syncthreads();
  if (t == 0) {
    bulk_store(a.pt + tile, sm + L::oP, kTTile);
    tma_store_commit();
    tma_store_wait_read_all();
    if (*abort_flag) linger();
  }
  __syncthreads();
  grid_dep_launch_dependents();
  if (w == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 64);
  }
  // this grid ends after the chain beside it, so that the next one follows both
  if (a.beside && blockIdx.x == 0) grid_dep_wait();
}

// ------------------------------------------------------------------- chain
struct FwdArgs {
  const __nv_bfloat16* v;
  const float *g, *beta, *state_in;
  const uint8_t *t, *pt;             // of the first launch
  __nv_bfloat16* out;
  uint8_t *keep_s, *keep_u;          // see Saved
  float* state_out;
  int* status;
  int64_t N;
  int n_chunks, chunk0, span, H, group, D, M;
  bool lead;  // the next piece's matrices run beside this chain
  float scale;
};

template <int DP, bool KEEP>
struct FwdLayout {
  static constexpr int kBoxes = DP / 64;
  static constexpr int kKQBox = 2 * kBox;               // 64 columns of K over Q: [128 x 64]
  static constexpr int kKQ = kBoxes * kKQBox;
  static constexpr int kT = 2 * kBox;                   // [T; P T] transposed, one part
  static constexpr int oT = 2 * kKQ;                    // three (after two stages of K, Q)
  static constexpr int oS = oT + 3 * kT;                // [DP x (first | second part)]
  static constexpr int oR = oS + DP * 128;              // [64 x (first | second part)]
  static constexpr int oX = oR + kBox;                  // [DP x (S's third | R's third)]
  // fp32 copies on their way to memory (KEEP): U's may lie over S, done with when
  // it is made, and at D <= 64 S's over R
  static constexpr int oKeepU = oS;
  static constexpr int oKeepS = DP == 64 ? oR : oX + DP * 128;
  static constexpr int oG = KEEP && DP > 64 ? oKeepS + DP * 128 : oX + DP * 128;
  static constexpr int oBar = oG + 2 * (int)sizeof(GateSlot);
  static constexpr int kBytes = oBar + 128 + 1024;
  static constexpr int kPerSM = DP == 64 ? 2 : 1;
  static_assert(kPerSM * (kBytes + 1024) <= 233472, "shared memory");
};

// KEEP: leave what the backward needs (Saved).
template <int DP, bool KEEP>
__global__ void __launch_bounds__(kChainThreads, FwdLayout<DP, KEEP>::kPerSM)
    delta_tc_fwd_kernel(const __grid_constant__ CUtensorMap tm_q,
                        const __grid_constant__ CUtensorMap tm_k, const FwdArgs a) {
  using L = FwdLayout<DP, KEEP>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = align_tiles(smem_raw);
  GateSlot* gates = reinterpret_cast<GateSlot*>(sm + L::oG);
  uint64_t* kq_full = reinterpret_cast<uint64_t*>(sm + L::oBar);  // [2]
  uint64_t* t_full = kq_full + 2;
  uint64_t* done = kq_full + 3;  // [3]
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(done + 3);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0);  // (uniform to the compiler)
  const int lane = threadIdx.x % 32, sub = warp / 4, t = threadIdx.x % 128;
  const int64_t p = blockIdx.x;  // b * H + h
  const int pk = (int)((p / a.H) * (a.H / a.group) + (p % a.H) / a.group);
  const int n = a.span, c0 = blockIdx.y * kCB + 16 * sub, nc = a.M - c0;  // 16 columns
  const int64_t tile0 = p * a.n_chunks + a.chunk0, row0 = (int64_t)a.chunk0 * kCh;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 6; ++i) mbar_init(kq_full + i, 1);
    if (KEEP) {  // the first and last products, and the copies out of S and U
      mbar_init(done, 2);
      mbar_init(done + 2, 2);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(tmem_holder, 128);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_holder, 0), s_base = smem_u32(sm);
  const uint32_t lane_col = ((uint32_t)(warp % 4) << 21) + 16 * sub;
  const uint32_t T_addr = s_base + L::oT, S_addr = s_base + L::oS, R_addr = s_base + L::oR;
  const uint32_t S_third = s_base + L::oX, R_third = S_third + 64;
  uint8_t *S_tile = sm + L::oS, *R_tile = sm + L::oR, *X_tile = sm + L::oX;
  constexpr uint32_t id_nt = idesc_bf16_f32(128, 96, 0, 1);  // A [rows x K], B [K x cols]
  constexpr uint32_t id_tt = idesc_bf16_f32(128, 96, 1, 1);  // A [K x rows], B [K x cols]
  const uint64_t once = policy_evict_first();
  auto load_kq = [&](int c) {
    uint64_t* bar = kq_full + (c & 1);
    uint8_t* dst = sm + (c & 1) * L::kKQ;
    mbar_arrive_expect_tx(bar, L::kKQ);
    for (int x = 0; x < L::kBoxes; ++x) {
      tma_load_3d(dst + x * L::kKQBox, &tm_k, bar, 64 * x, (int)row0 + c * kCh, pk, once);
      tma_load_3d(dst + x * L::kKQBox + kBox, &tm_q, bar, 64 * x, (int)row0 + c * kCh, pk, once);
    }
  };
  auto load_t = [&](int c) {
    const int64_t tile = (tile0 + c) * kTTile;
    mbar_arrive_expect_tx(t_full, 2 * kTTile);
#pragma unroll 1
    for (int h = 0; h < 3; ++h) {
      bulk_load(sm + L::oT + h * L::kT, a.t + tile + h * kBox, kBox, t_full);
      bulk_load(sm + L::oT + h * L::kT + kBox, a.pt + tile + h * kBox, kBox, t_full);
    }
  };
  // one warp: the gates, loaded a chunk before they are written
  float4 gb;
  auto load_gates = [&](int c) {
    const int64_t i = row0 + (int64_t)c * kCh + lane;
    const float* g = a.g + p * a.N;
    const float* b = a.beta + p * a.N;
    gb = make_float4(i < a.N ? g[i] : 0.f, i + 32 < a.N ? g[i + 32] : 0.f, i < a.N ? b[i] : 0.f,
                     i + 32 < a.N ? b[i + 32] : 0.f);
  };
  auto put_gates = [&](int c) {
    write_gates(gates + (c & 1), lane, gb.x, gb.y, gb.z, gb.w);
    load_gates(c + 1);
  };
  // lanes 0-63: the row of V, loaded a chunk ahead
  const int64_t at = p * a.N * a.M + c0;
  uint4 vv[2];
  auto load_v = [&](int c) {
    const int64_t row = row0 + (int64_t)c * kCh + t;
    read16(a.v + at + row * a.M, nc, t < 64 && row < a.N, vv);
  };
  const bool row_on = t < a.D;
  float2 S[8];
  grid_dep_wait();
  if (a.lead) grid_dep_launch_dependents();

  if (warp == 8) {  // the copies and the gates, a chunk ahead
    if (lane == 0) {
      load_kq(0);
      load_t(0);
      if (n > 1) load_kq(1);
    }
    __syncwarp();
    load_gates(0);
    put_gates(0);
    for (int c = 0; c < n; ++c) {
      __syncthreads();
      if (c + 1 < n) put_gates(c + 1);
      wait_or_abort(done + 1, c & 1, a.status, abort_flag);
      if (lane == 0 && c + 1 < n) load_t(c + 1);
      __syncwarp();
      wait_or_abort(done + 2, c & 1, a.status, abort_flag);
      if (lane == 0 && c + 2 < n) load_kq(c + 2);
      __syncwarp();
    }
  } else {
  read16(a.state_in + (p * a.D + t) * a.M + c0, nc, a.state_in != nullptr && row_on, S);
  load_v(0);
  for (int c = 0; c < n; ++c) {
    const uint32_t kq = s_base + (c & 1) * L::kKQ, phase = c & 1;
    const GateSlot* gs = gates + (c & 1);
    if (t < DP) {
      store_parts(S_tile, X_tile, 0, t, sub, S);
      if (KEEP) put_f32(sm + L::oKeepS, t, sub, S);
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
      wait_or_abort(kq_full + (c & 1), (c >> 1) & 1, a.status, abort_flag);
      __syncwarp();
      tc_fence_after();
      const uint32_t el = elect_one();
      mma_tile<DP / 16, false, true>(el, tmem, kq, S_addr, id_nt, 16, S_third - S_addr, L::kKQBox, 0,
                                     true);
      if (el) mma_commit(done);
    }
    const int64_t kept = (tile0 + c) * gridDim.y + blockIdx.y;
    if (KEEP && threadIdx.x == 128) {
      bulk_store(a.keep_s + kept * (DP * 128), sm + L::oKeepS, DP * 128);
      tma_store_commit();
      tma_store_wait_read_all();
      mbar_arrive(done);
    }
    wait_or_abort(done, phase, a.status, abort_flag);
    tc_fence_after();
    float2 x[8];
    load16_sum(tmem + lane_col, x);
    if (t < 64) {
      const float2 b = both(gs->b[t]), bg = both(-gs->b[t] * gs->gam[t]);
      float2 v[8];
      unpack16(vv, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = fma2(bg, x[j], mul2(b, v[j]));
      store_parts(R_tile, X_tile, 4, t, sub, x);
      if (c + 1 < n) load_v(c + 1);
    } else {
      const float2 gam = both(a.scale * gs->gam[t - 64]);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = mul2(gam, x[j]);  // waits for P U
    }
    fence_proxy_async_smem();
    tc_fence_before();
    named_barrier_sync(1, 256);
    if (warp == 0) {
      wait_or_abort(t_full, phase, a.status, abort_flag);
      __syncwarp();
      tc_fence_after();
      const uint32_t el = elect_one();
      mma_parts<true>(el, tmem, T_addr, L::kT, kBox, R_addr, R_third);
      if (el) mma_commit(done + 1);
    }
    wait_or_abort(done + 1, phase, a.status, abort_flag);
    tc_fence_after();
    {
      const int64_t row = row0 + (int64_t)c * kCh + (t & 63);
      float2 r[8];
      load16_sum(tmem + lane_col, r);
      if (t < 64) {
        if (KEEP) put_f32(sm + L::oKeepU, t, sub, r);
        const float2 del = both(gs->del[t]);
#pragma unroll
        for (int j = 0; j < 8; ++j) r[j] = mul2(del, r[j]);
        store_parts(R_tile, X_tile, 4, t, sub, r);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) r[j] = add2(x[j], r[j]);
        uint4 w[2];
        pack16(r, w);
        if (row < a.N) write16(a.out + at + row * a.M, nc, w);
      }
    }
    fence_proxy_async_smem();
    tc_fence_before();
    named_barrier_sync(1, 256);
    if (warp == 0) {
      tc_fence_after();
      const uint32_t el = elect_one();
      // K^T: 64 columns of K to a 64-lane block; with one such block the
      // lanes past 64 take Q's, and are not read
      constexpr uint32_t lbo = DP == 128 ? L::kKQBox : kBox;
      mma_tile<4, true, true>(el, tmem, kq, R_addr, id_tt, lbo, R_third - R_addr, 0, 0, true);
      if (el) mma_commit(done + 2);
    }
    if (KEEP && threadIdx.x == 128) {
      bulk_store(a.keep_u + kept * kBox, sm + L::oKeepU, kBox);
      tma_store_commit();
      tma_store_wait_read_all();
      mbar_arrive(done + 2);
    }
    wait_or_abort(done + 2, phase, a.status, abort_flag);
    tc_fence_after();
    const float2 last = both(gs->last.x), last_lo = both(gs->last.y);
    load16_sum(tmem + lane_col, x);
#pragma unroll
    for (int j = 0; j < 8; ++j) S[j] = fma2(last, S[j], fma2(last_lo, S[j], x[j]));
  }
  if (a.state_out != nullptr && row_on) write16(a.state_out + (p * a.D + t) * a.M + c0, nc, S);
  if (KEEP && threadIdx.x == 128) tma_store_wait_read_all();
  }
  // every load and MMA has been waited for by the loop that used it
  if (*abort_flag) linger();
  tc_fence_before();
  __syncthreads();
  grid_dep_launch_dependents();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 128);
  }
}

// Device scratch of a forward: P T, T when it is not kept, and the state
// between pieces.
size_t tiles_bytes(const DeltaShape& s) {
  return (size_t)(s.B * s.H * ((s.N + kCh - 1) / kCh)) * kTTile;
}

// Pieces of the sequence: where the chain leaves half of the SMs idle, a
// piece's matrices are made under the chain over the piece before, at a few
// microseconds a piece (with factors in two parts, B = 4, H = 8, N = 8229, D =
// 128, M = 64: 254 us in four pieces, 274 whole; B = 2, H = 8, N = 32768, D = M =
// 128: 896 in six, 969; in three parts 302 and 1079, in as many pieces).
int n_pieces(const DeltaShape& s) {
  const int64_t ctas = s.B * s.H * ((s.M + kCB - 1) / kCB), n = (s.N + kCh - 1) / kCh;
  if (ctas > kPlanSMs / 2) return 1;
  return (int)std::max<int64_t>(1, std::min<int64_t>(n / 32, 6));
}

template <int DP, bool KEEP>
cp_status_t launch(const DeltaShape& s, const DeltaFwd& f, void* scratch, int* status,
                   cudaStream_t stream) {
  using LP = PrepLayout<DP>;
  using L = FwdLayout<DP, KEEP>;
  auto prep = delta_tc_prep_kernel<DP>;
  auto chain = delta_tc_fwd_kernel<DP, KEEP>;
  if (cudaFuncSetAttribute(prep, cudaFuncAttributeMaxDynamicSharedMemorySize, LP::kBytes) != cudaSuccess ||
      cudaFuncSetAttribute(chain, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kBytes) != cudaSuccess)
    return CP_ERR_CUDA;
  const Saved k(s);
  const int64_t BH = s.B * s.H;
  uint8_t* kept = reinterpret_cast<uint8_t*>(f.ckpt);
  uint8_t* area = static_cast<uint8_t*>(scratch);
  PrepArgs a{};
  a.g = f.g; a.beta = f.beta;
  a.pt = area;
  a.t = KEEP ? kept + k.s_bytes + k.u_bytes : area + tiles_bytes(s);
  a.p = KEEP ? a.t + k.t_bytes : nullptr;
  a.status = status;
  a.N = s.N; a.n_chunks = (int)k.n; a.H = (int)s.H; a.group = (int)(s.H / s.Hk); a.scale = s.scale;
  const int pieces = n_pieces(s);
  float* between = reinterpret_cast<float*>(area + 2 * tiles_bytes(s));
  FwdArgs c{};
  c.v = static_cast<const __nv_bfloat16*>(f.v);
  c.out = static_cast<__nv_bfloat16*>(f.out);
  if (KEEP) {
    c.keep_s = kept;
    c.keep_u = kept + k.s_bytes;
  }
  c.g = f.g; c.beta = f.beta; c.t = a.t; c.pt = a.pt; c.status = status;
  c.N = s.N; c.n_chunks = (int)k.n; c.H = a.H; c.group = a.group;
  c.D = (int)s.D; c.M = (int)s.M; c.scale = s.scale;
  // (encoding a map needs the device's context current in this thread: the
  // calls above see to that)
  CUtensorMap mq, mk;
  if (!make_chunk_map(&mq, f.q, s.B * s.Hk, s.N, s.D) || !make_chunk_map(&mk, f.k, s.B * s.Hk, s.N, s.D))
    return CP_ERR_CUDA;
  const dim3 grid((unsigned)BH, (unsigned)((s.M + kCB - 1) / kCB));
  for (int i = 0; i < pieces; ++i) {
    const bool last = i + 1 == pieces;
    // the first piece, under whose matrices nothing runs, is half as long
    const auto start = [&](int x) { return (int)(k.n * std::max(2 * x - 1, 0) / (2 * pieces - 1)); };
    a.chunk0 = c.chunk0 = start(i);
    a.span = c.span = start(i + 1) - a.chunk0;
    a.beside = i > 0;
    c.lead = !last;
    // (a chain's CTA reads only what it wrote itself)
    c.state_in = i > 0 ? between : f.state_in;
    c.state_out = last ? f.state_out : between;
    if (launch_dependent(prep, dim3((unsigned)(BH * a.span)), 128, LP::kBytes, stream, mq, mk, a) != cudaSuccess ||
        launch_dependent(chain, grid, kChainThreads, L::kBytes, stream, mq, mk, c) != cudaSuccess)
      return CP_ERR_CUDA;
  }
  return CP_OK;
}

}  // namespace

bool delta_tc_supported(const DeltaShape& s) {
  return s.dtype == CP_DTYPE_BF16 && s.D <= 128 && s.D % 8 == 0 && s.M % 8 == 0 &&
         s.B * s.H * ((s.N + kCh - 1) / kCh) < (int64_t)1 << 30;  // tensor-map and grid indexes
}

size_t delta_tc_ckpt_bytes(const DeltaShape& s) { return (size_t)Saved(s).bytes(); }

size_t delta_tc_fwd_scratch(const DeltaShape& s) {
  return 2 * tiles_bytes(s) + (n_pieces(s) > 1 ? sizeof(float) * (size_t)(s.B * s.H * s.D * s.M) : 0);
}

cp_status_t delta_tc_fwd(const DeltaShape& s, const DeltaFwd& f, void* scratch, int* status,
                         cudaStream_t stream) {
  if (f.ckpt != nullptr)
    return s.D <= 64 ? launch<64, true>(s, f, scratch, status, stream)
                     : launch<128, true>(s, f, scratch, status, stream);
  return s.D <= 64 ? launch<64, false>(s, f, scratch, status, stream)
                   : launch<128, false>(s, f, scratch, status, stream);
}

}  // namespace cp
