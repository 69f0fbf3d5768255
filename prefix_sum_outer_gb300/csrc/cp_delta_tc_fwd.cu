// Forward of the gated delta rule on the tensor cores (bf16, D <= 128).
//
// A CTA walks one head's chunks of 64 rows with the fp32 state of up to 128
// value columns in registers.  Value columns never meet, so each 64 of them (a
// "half") are a chain of their own, run by two warpgroups of 32 columns each;
// lane d holds row d of the state.  A chunk is three MMAs on the chain:
//     [K; Q] S          -> KS (lanes 0-63), QS (lanes 64-127)
//     R = b (V - gam KS) -> shared memory
//     [T; P T] R        -> U (lanes 0-63), P U (lanes 64-127)
//     out = s gam QS + P U;   del U -> shared memory
//     K^T (del U)       -> S = gam_C S + it, -> shared memory
// T = (I + A)^-1.  P T in place of P takes a fourth dependent step
// (P U) off the chain and gives both products one 128-lane MMA.  The chain is
// bound by its own latency: the conversions between the products, the MMAs'
// operand reads and the round trips through tensor memory.  So the conversions
// are spread over 256 threads, and a factor's hi and lo parts enter as one
// 128-column operand: an MMA of 64 columns takes as long as its 128 x 16 left
// operand takes to read (62 cycles measured), one of 128 columns little more.
//
// The last warpgroup makes T and P T one chunk ahead: [K; Q] K^T by MMA, A and
// P from it by the decays, the inverse by blocks, P T by MMA; one of its
// threads keeps the K, Q ring full by TMA.
#include <algorithm>

#include "cp_delta_tc.cuh"

namespace cp {
namespace {

using namespace delta;

// Gate slots: the last group writes chunk c's once the halves have issued [T; P
// T] R of chunk c - 2, whose slot they still read.
constexpr int kSlots = 3;

struct TcFwdArgs {
  const __nv_bfloat16* v;
  const float *g, *beta, *state_in;
  __nv_bfloat16* out;
  float* state_out;
  // kept for the backward (see Saved); null: not kept
  __nv_bfloat16 *keep_s, *keep_u;
  uint8_t* keep_tp;
  int64_t u_part;  // elements between U's parts
  int* status;
  int64_t N;
  int n_chunks, H, group, D, M;
  float scale;
};

template <int DP, int NH>
struct FwdLayout {
  static constexpr int kBoxes = DP / 64;
  static constexpr int kKQBox = 2 * kBox;               // 64 columns of K over Q: [128 x 64]
  static constexpr int kKQ = kBoxes * kKQBox;
  static constexpr int kT = 2 * kBox;                   // [T; P T] transposed, one part
  static constexpr int kS = DP * 128;                   // [DP x 64], one part
  static constexpr int kFixed = 2 * kT + NH * 2 * (kS + kBox) + 2 * kBox + (int)sizeof(InvTiles) +
                                kSlots * (int)sizeof(GateSlot) + 256 + 1024;
  static constexpr int NST = (tc::kSmemLimit - kFixed) / kKQ < 4 ? (tc::kSmemLimit - kFixed) / kKQ : 4;
  static constexpr int oT = NST * kKQ;                  // hi, lo
  static constexpr int oS = oT + 2 * kT;                // per half: hi, lo
  static constexpr int oR = oS + NH * 2 * kS;           // per half: hi, lo
  static constexpr int oP = oR + NH * 2 * kBox;         // hi, lo
  static constexpr int oInv = oP + 2 * kBox;
  static constexpr int oG = oInv + (int)sizeof(InvTiles);
  static constexpr int oBar = oG + kSlots * (int)sizeof(GateSlot);
  static constexpr int kBytes = oBar + 256 + 1024;
  static constexpr int kThreads = 128 * (2 * NH + 1);
  static constexpr int cPrep = NH * 128;                // tensor-memory columns of the last group
  static_assert(NST >= 2 && kBytes <= tc::kSmemLimit, "shared memory");
  static_assert(sizeof(InvTiles) % 16 == 0 && sizeof(GateSlot) % 16 == 0, "alignment");
};

template <int DP, int NH>
__global__ void __launch_bounds__(FwdLayout<DP, NH>::kThreads, 1)
    delta_tc_fwd_kernel(const __grid_constant__ CUtensorMap tm_q,
                        const __grid_constant__ CUtensorMap tm_k, const TcFwdArgs a) {
  using L = FwdLayout<DP, NH>;
  constexpr int NST = L::NST;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                           ~static_cast<uintptr_t>(1023));
  GateSlot* gates = reinterpret_cast<GateSlot*>(sm + L::oG);
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::oBar);
  uint64_t* kq_full = bars;            // [NST] loader -> all
  uint64_t* kq_empty = kq_full + NST;  // [NST] halves -> loader
  uint64_t* t_full = kq_empty + NST;   // last group -> halves: T, P T and the gates
  uint64_t* t_empty = t_full + 1;      // halves -> last group
  uint64_t* p_done = t_empty + 1;      // [2] the last group's MMAs
  uint64_t* h_done = p_done + 2;       // [NH][3] the halves' MMAs
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(h_done + 3 * NH);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int64_t p = blockIdx.x;  // b * H + h
  const int pk = (int)((p / a.H) * (a.H / a.group) + (p % a.H) / a.group);
  const int n = a.n_chunks;

  if (threadIdx.x == 0) {
    for (int i = 0; i < NST; ++i) {
      mbar_init(kq_full + i, 1);
      mbar_init(kq_empty + i, NH);
    }
    mbar_init(t_full, 128);
    mbar_init(t_empty, NH);
    mbar_init(p_done, 1);
    mbar_init(p_done + 1, 1);
    for (int i = 0; i < 3 * NH; ++i) mbar_init(h_done + i, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(tmem_holder, 512);
    tmem_relinquish();
  }
  // the blocks of T and P above the diagonal are never written
  for (int i = threadIdx.x; i < 2 * L::kT / 16; i += L::kThreads)
    reinterpret_cast<uint4*>(sm + L::oT)[i] = make_uint4(0, 0, 0, 0);
  for (int i = threadIdx.x; i < 2 * kBox / 16; i += L::kThreads)
    reinterpret_cast<uint4*>(sm + L::oP)[i] = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const uint32_t lane_base = (uint32_t)(warp % 4) << 21;  // this warp's 32 lanes
  const uint32_t s_base = smem_u32(sm);
  constexpr uint32_t id_nn64 = idesc_bf16_f32(128, 64, 0, 0);    // A [rows x K], B [cols x K]
  constexpr uint32_t id_nn128 = idesc_bf16_f32(128, 128, 0, 0);
  constexpr uint32_t id_nt128 = idesc_bf16_f32(128, 128, 0, 1);  // B [K x cols]
  constexpr uint32_t id_tt128 = idesc_bf16_f32(128, 128, 1, 1);  // A [K x rows], B [K x cols]
  const uint32_t T_addr = s_base + L::oT;

  if (warp >= 8 * NH) {
    // ------------------------------------------------- T and P T, one ahead
    const int w = warp - 8 * NH, t = threadIdx.x - 256 * NH;
    const uint32_t t_kk = tmem + L::cPrep, t_pt = t_kk + 64;
    InvTiles* it = reinterpret_cast<InvTiles*>(sm + L::oInv);
    uint8_t* T_hi = sm + L::oT;             // transposed: rows j of T, then rows j of P T
    uint8_t* T_lo = T_hi + L::kT;
    uint8_t* P_hi = sm + L::oP;
    uint8_t* P_lo = P_hi + kBox;
    const uint32_t P_addr = s_base + L::oP;
    float g0 = 0.f, g1 = 0.f, b0 = 0.f, b1 = 0.f;
    auto load_gates = [&](int c) {
      const int64_t i = (int64_t)c * kCh + lane;
      const float* g = a.g + p * a.N;
      const float* b = a.beta + p * a.N;
      g0 = i < a.N ? g[i] : 0.f;
      b0 = i < a.N ? b[i] : 0.f;
      g1 = i + 32 < a.N ? g[i + 32] : 0.f;
      b1 = i + 32 < a.N ? b[i + 32] : 0.f;
    };
    const uint64_t keep = policy_evict_first();
    // chunk c into its stage, once the halves are done with chunk c - NST
    auto load_chunk = [&](int c) {
      const int st = c % NST;
      if (c >= NST) wait_or_abort(kq_empty + st, ((c / NST) - 1) & 1, a.status, abort_flag);
      if (*abort_flag) return;
      uint8_t* dst = sm + st * L::kKQ;
      mbar_arrive_expect_tx(kq_full + st, L::kKQ);
      for (int x = 0; x < L::kBoxes; ++x) {
        tma_load_3d(dst + x * L::kKQBox, &tm_k, kq_full + st, 64 * x, c * kCh, pk, keep);
        tma_load_3d(dst + x * L::kKQBox + kBox, &tm_q, kq_full + st, 64 * x, c * kCh, pk, keep);
      }
    };
    if (t == 96) {
      tma_prefetch_desc(&tm_q);
      tma_prefetch_desc(&tm_k);
      for (int c = 0; c < min(n, NST); ++c) load_chunk(c);
    }
    if (w == 3) load_gates(0);
    for (int c = 0; c < n; ++c) {
      const int st = c % NST;
      const uint32_t kq = s_base + st * L::kKQ;
      GateSlot* gs = gates + c % kSlots;
      if (t == 0) {
        wait_or_abort(kq_full + st, (c / NST) & 1, a.status, abort_flag);
        if (!*abort_flag) {
          mma_tile<DP / 16, false, false>(t_kk, kq, kq, id_nn64, 16, 16, L::kKQBox, L::kKQBox, true);
          mma_commit(p_done);
        }
      }
      if (w == 3) {
        write_gates(gs, lane, g0, g1, b0, b1);
        if (c + 1 < n) load_gates(c + 1);
      }
      named_barrier_sync(1, 128);
      wait_or_abort(p_done, c & 1, a.status, abort_flag);
      tc_fence_after();
      // A by the lanes of K, P by those of Q
      if (w < 2) {
        decayed_row(t_kk + lane_base, gs, t, false, w, gs->b[t],
                    [&](int cb, const float2(&v)[8]) { put_a16(it, t, cb, v); });
      } else {
        decayed_row(t_kk + lane_base, gs, t - 64, true, w - 2, a.scale,
                    [&](int cb, const float2(&v)[8]) {
                      store16_split(P_hi, P_lo, t - 64, 2 * cb, v);
                    });
      }
      tc_fence_before();
      named_barrier_sync(1, 128);
      float x[16], z[3][2][4];
      invert_diag(it, w, lane, x);
      named_barrier_sync(1, 128);
      invert_below(it, w, lane, z);
      if (c > 0) wait_or_abort(t_empty, (c - 1) & 1, a.status, abort_flag);
      put_t_transposed(T_hi, T_lo, w, lane, x, z);
      fence_proxy_async_smem();
      named_barrier_sync(1, 128);
      if (t == 0 && !*abort_flag) {
        tc_fence_after();
        // (P T)^T = T^T P^T, P^T's parts side by side; lanes 0-63 are read
        mma_tile<4, false, false>(t_pt, T_addr, P_addr, id_nn128, 16, 16, 0, 0, true);
        mma_tile<4, false, false>(t_pt, T_addr + L::kT, P_addr, id_nn128, 16, 16, 0, 0, false);
        mma_commit(p_done + 1);
      }
      if (t == 64 && a.keep_tp != nullptr && blockIdx.y == 0) {
        uint8_t* to = a.keep_tp + (p * n + c) * (int64_t)(4 * kBox);
        bulk_store(to, T_hi, kBox);
        bulk_store(to + kBox, T_lo, kBox);
        bulk_store(to + 2 * kBox, P_hi, 2 * kBox);
        tma_store_commit();
      }
      wait_or_abort(p_done + 1, c & 1, a.status, abort_flag);
      tc_fence_after();
      if (w < 2) {
#pragma unroll 1
        for (int h = 0; h < 4; ++h) {
          float2 v[8];
          load16_sum(t_pt + lane_base + 16 * h, v);
          store16_split(T_hi + kBox, T_lo + kBox, t, 2 * h, v);
        }
      }
      tc_fence_before();
      fence_proxy_async_smem();
      // the copies out of this chunk's tiles have read them (the next chunk's
      // writes come after a barrier)
      if (t == 64) tma_store_wait_read_all();
      mbar_arrive(t_full);
      if (t == 96 && c > 0 && c - 1 + NST < n) load_chunk(c - 1 + NST);
    }
    if (t == 64) tma_store_wait_all();
  } else {
    // ---------------------------------------------------------- the chain
    const int half = warp / 8, sub = (warp / 4) % 2, t = threadIdx.x % 128;
    const bool issuer = threadIdx.x == 256 * half;
    const int bar_id = 2 + half;
    const int c0 = (blockIdx.y * NH + half) * 64 + 32 * sub;  // this thread's 32 value columns
    const int nc = max(0, min(32, a.M - c0));
    const uint32_t t_acc = tmem + 128 * half;           // every product's accumulators
    const uint32_t t_mine = t_acc + lane_base + 32 * sub;
    uint8_t* S_hi = sm + L::oS + half * 2 * L::kS;
    uint8_t* S_lo = S_hi + L::kS;
    uint8_t* R_hi = sm + L::oR + half * 2 * kBox;
    uint8_t* R_lo = R_hi + kBox;
    const uint32_t S_addr = smem_u32(S_hi), R_addr = smem_u32(R_hi);
    uint64_t* done = h_done + 3 * half;
    const bool row_on = t < a.D;
    float2 S[16];
    {
      const float* src = a.state_in == nullptr ? nullptr : a.state_in + (p * a.D + t) * a.M + c0;
#pragma unroll
      for (int j = 0; j < 32; j += 4) {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (src != nullptr && row_on && j < nc) v = *reinterpret_cast<const float4*>(src + j);
        S[j / 2] = make_float2(v.x, v.y);
        S[j / 2 + 1] = make_float2(v.z, v.w);
      }
    }
    const __nv_bfloat16* v_src = a.v + p * a.N * a.M + c0;
    __nv_bfloat16* o_dst = a.out + p * a.N * a.M + c0;
    uint4 vv[4];  // lanes 0-63: the row's 32 values, loaded a chunk ahead
    auto load_v = [&](int c) {
      const int64_t row = (int64_t)c * kCh + t;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        vv[j] = make_uint4(0, 0, 0, 0);
        if (t < 64 && row < a.N && 8 * j < nc)
          vv[j] = *reinterpret_cast<const uint4*>(v_src + row * a.M + 8 * j);
      }
    };
    load_v(0);
    for (int c = 0; c < n; ++c) {
      const int st = c % NST;
      const uint32_t kq = s_base + st * L::kKQ;
      const GateSlot* gs = gates + c % kSlots;
      if (t < DP) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint4 hi[2], lo[2];
          split16(*reinterpret_cast<const float2(*)[8]>(S + 8 * h), hi, lo);
          put16(S_hi, t, 4 * sub + 2 * h, hi);
          put16(S_lo, t, 4 * sub + 2 * h, lo);
          if (a.keep_s != nullptr && row_on) {
            __nv_bfloat16* to = a.keep_s + (((p * n + c) * 2) * (int64_t)a.D + t) * a.M + c0 + 16 * h;
            write16(to, nc - 16 * h, hi);
            write16(to + (int64_t)a.D * a.M, nc - 16 * h, lo);
          }
        }
      }
      fence_proxy_async_smem();
      tc_fence_before();
      named_barrier_sync(bar_id, 256);
      if (issuer) {
        wait_or_abort(kq_full + st, (c / NST) & 1, a.status, abort_flag);
        if (!*abort_flag) {
          tc_fence_after();
          mma_tile<DP / 16, false, true>(t_acc, kq, S_addr, id_nt128, 16, L::kS, L::kKQBox, 0, true);
          mma_commit(done);
        }
      }
      wait_or_abort(t_full, c & 1, a.status, abort_flag);
      wait_or_abort(done, c & 1, a.status, abort_flag);
      tc_fence_after();
      float2 qs[16];  // lanes 64-127: s gam QS
      if (t < 64) {
        const float2 b = both(gs->b[t]), bg = both(-gs->b[t] * gs->gam[t]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float2 r[8];
          load16_sum(t_mine + 16 * h, r);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint4 u4 = vv[2 * h + j];
            const uint32_t u[4] = {u4.x, u4.y, u4.z, u4.w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
              r[4 * j + e] = fma2(bg, r[4 * j + e],
                                  mul2(b, make_float2(__uint_as_float(u[e] << 16),
                                                      __uint_as_float(u[e] & 0xffff0000u))));
          }
          store16_split(R_hi, R_lo, t, 4 * sub + 2 * h, r);
        }
        if (c + 1 < n) load_v(c + 1);
      } else {
        const float2 gam = both(a.scale * gs->gam[t - 64]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float2 r[8];
          load16_sum(t_mine + 16 * h, r);
#pragma unroll
          for (int j = 0; j < 8; ++j) qs[8 * h + j] = mul2(gam, r[j]);
        }
      }
      fence_proxy_async_smem();
      tc_fence_before();
      named_barrier_sync(bar_id, 256);
      if (issuer && !*abort_flag) {
        tc_fence_after();
        mma_tile<4, true, true>(t_acc, T_addr, R_addr, id_tt128, kBox, kBox, 0, 0, true);
        mma_tile<4, true, true>(t_acc, T_addr + L::kT, R_addr, id_tt128, kBox, kBox, 0, 0, false);
        mma_commit(done + 1);
        mma_commit(t_empty);
      }
      wait_or_abort(done + 1, c & 1, a.status, abort_flag);
      tc_fence_after();
      if (t < 64) {
        const float2 del = both(gs->del[t]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float2 r[8];
          load16_sum(t_mine + 16 * h, r);
          if (a.keep_u != nullptr && (int64_t)c * kCh + t < a.N) {
            uint4 hi[2], lo[2];
            split16(r, hi, lo);
            __nv_bfloat16* to = a.keep_u + (p * a.N + (int64_t)c * kCh + t) * a.M + c0 + 16 * h;
            write16(to, nc - 16 * h, hi);
            write16(to + a.u_part, nc - 16 * h, lo);
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) r[j] = mul2(del, r[j]);
          store16_split(R_hi, R_lo, t, 4 * sub + 2 * h, r);
        }
      } else {
        const int64_t row = (int64_t)c * kCh + t - 64;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float2 r[8];
          load16_sum(t_mine + 16 * h, r);
          uint32_t w[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            r[j] = add2(qs[8 * h + j], r[j]);
            w[j] = tc::pack_bf16x2(r[j].x, r[j].y);
          }
#pragma unroll
          for (int j = 0; j < 2; ++j)
            if (row < a.N && 16 * h + 8 * j < nc)
              *reinterpret_cast<uint4*>(o_dst + row * a.M + 16 * h + 8 * j) =
                  make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
        }
      }
      fence_proxy_async_smem();
      tc_fence_before();
      named_barrier_sync(bar_id, 256);
      if (issuer && !*abort_flag) {
        tc_fence_after();
        // K^T: 64 columns of K to a 64-lane block; with one such block the
        // lanes past 64 take Q's, and are not read
        constexpr uint32_t lbo = DP == 128 ? L::kKQBox : kBox;
        mma_tile<4, true, true>(t_acc, kq, R_addr, id_tt128, lbo, kBox, 0, 0, true);
        mma_commit(done + 2);
        mma_commit(kq_empty + st);
      }
      wait_or_abort(done + 2, c & 1, a.status, abort_flag);
      tc_fence_after();
      const float2 last = both(gs->gam[kCh - 1]);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float2 r[8];
        load16_sum(t_mine + 16 * h, r);
#pragma unroll
        for (int j = 0; j < 8; ++j) S[8 * h + j] = fma2(last, S[8 * h + j], r[j]);
      }
    }
    if (a.state_out != nullptr && row_on) {
      float* dst = a.state_out + (p * a.D + t) * a.M + c0;
#pragma unroll
      for (int j = 0; j < 32; j += 4)
        if (j < nc)
          *reinterpret_cast<float4*>(dst + j) =
                make_float4(S[j / 2].x, S[j / 2].y, S[j / 2 + 1].x, S[j / 2 + 1].y);
    }
  }
  // every load and MMA has been waited for by the loop that used it; after an
  // abort, give what is in flight time to land before the memory goes
  tc_fence_before();
  __syncthreads();
  if (*abort_flag) {
    const uint64_t t0 = globaltimer();
    while (globaltimer() - t0 < 1000000ull) {
    }
  }
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int DP, int NH>
cp_status_t launch(const DeltaShape& s, const DeltaFwd& f, const TcFwdArgs& a, cudaStream_t stream) {
  using L = FwdLayout<DP, NH>;
  auto kern = delta_tc_fwd_kernel<DP, NH>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kBytes) != cudaSuccess)
    return CP_ERR_CUDA;
  // (encoding a map needs the device's context current in this thread: the
  // call above sees to that)
  CUtensorMap mq, mk;
  if (!make_chunk_map(&mq, f.q, s.B * s.Hk, s.N, s.D) || !make_chunk_map(&mk, f.k, s.B * s.Hk, s.N, s.D))
    return CP_ERR_CUDA;
  const dim3 grid((unsigned)(s.B * s.H), (unsigned)((s.M + 64 * NH - 1) / (64 * NH)));
  kern<<<grid, L::kThreads, L::kBytes, stream>>>(mq, mk, a);
  return cudaGetLastError() == cudaSuccess ? CP_OK : CP_ERR_CUDA;
}

}  // namespace

bool delta_tc_supported(const DeltaShape& s) {
  return s.dtype == CP_DTYPE_BF16 && s.D <= 128 && s.D % 8 == 0 && s.M % 8 == 0 &&
         s.B * s.H * ((s.N + kCh - 1) / kCh) < (int64_t)1 << 30;  // tensor-map and grid indexes
}


size_t delta_tc_ckpt_bytes(const DeltaShape& s) { return (size_t)Saved(s).bytes(); }

cp_status_t delta_tc_fwd(const DeltaShape& s, const DeltaFwd& f, int* status, cudaStream_t stream) {
  TcFwdArgs a{};
  a.v = static_cast<const __nv_bfloat16*>(f.v);
  a.g = f.g; a.beta = f.beta; a.state_in = f.state_in;
  a.out = static_cast<__nv_bfloat16*>(f.out);
  a.state_out = f.state_out; a.status = status;
  if (f.ckpt != nullptr) {
    const Saved k(s);
    uint8_t* at = reinterpret_cast<uint8_t*>(f.ckpt);
    a.keep_s = reinterpret_cast<__nv_bfloat16*>(at);
    a.keep_u = reinterpret_cast<__nv_bfloat16*>(at + k.s_bytes);
    a.keep_tp = at + k.s_bytes + k.u_bytes;
    a.u_part = s.B * s.H * s.N * s.M;
  }
  a.N = s.N; a.n_chunks = (int)((s.N + kCh - 1) / kCh);
  a.H = (int)s.H; a.group = (int)(s.H / s.Hk); a.D = (int)s.D; a.M = (int)s.M; a.scale = s.scale;
  if (s.D <= 64) return s.M <= 64 ? launch<64, 1>(s, f, a, stream) : launch<64, 2>(s, f, a, stream);
  return s.M <= 64 ? launch<128, 1>(s, f, a, stream) : launch<128, 2>(s, f, a, stream);
}

}  // namespace cp
