// Backward of the gated delta rule on the tensor cores (bf16, D <= 128), from
// what the forward kept (Saved: the states before the chunks, U, the inverse
// T = (I + A)^-1 and P).  Two launches:
//
// 1. The reverse chain, as sequential as the forward's and laid out like it: a
//    CTA per head and 64 value columns, two warpgroups of 32 columns, lane d
//    holding row d of the state's gradient dS' in tensor memory.  A chunk is
//        K dS'                          (lanes 0-63)
//        dU = P^T dO + del K dS'         -> shared memory
//        T^T dU                         -> dX
//        [K; Q]^T [-gam b dX; s gam dO]  -> dS = gam_C dS' + it, -> shared memory
//    P^T dO of the next chunk is issued behind the last product; while that
//    one runs, dX is read out a second time for what the chain does not wait
//    for (dX itself, dV = b dX, dX . V).  dU enters in three parts: P^T dO sums
//    up to 64 rows, of which T^T leaves the differences when keys repeat, so
//    dU's rounding is the largest error of dX.  It leaves dX and the dS' of
//    every chunk as hi and lo parts.
//
// 2. The gradients, one CTA per head and chunk, all chunks at once: with every
//    factor already in hi and lo parts in global memory, TMA puts them straight
//    into operand tiles.  Lanes 0-63 are the rows of K, 64-127 those of Q:
//        [dX; dO] U^T  -> Ma (A's part), Mq (P's part), by the decays
//        [dX; dO] S^T,  U dS'^T,  [Ma; Mq] K,  Ma^T K + Mq^T Q
//        dK = -gam b dX S^T + del U dS'^T + Ma K + Ma^T K + Mq^T Q
//        dQ = s gam dO S^T + Mq K
//    and the sums for the gates (cp_delta.cu has the formulas):
//        db_i = dX_i . U_i / b_i,                        where b_i is not 0,
//             = dX_i . V_i - gam_i k_i . (S dX_i) + sum_j Ma_ij / b_i k_i.k_j
//    (Ma / b is what is at hand), with dX . V from the chain.  The first is the
//    diagonal of dX U^T; the second, its value at b_i = 0 too, is a difference
//    of terms that nearly cancel when keys repeat.
#include <algorithm>

#include "cp_delta_tc.cuh"

namespace cp {
namespace {

using namespace delta;

// ------------------------------------------------------------ reverse chain
struct ChainArgs {
  const float *g, *beta, *grad_state_out;
  const uint8_t *t, *pm;        // tiles of T and P
  float *xv, *grad_state_in;    // xv [M / 32 blocks][BH][N]: dX . V over the block
  int* status;
  int64_t N;
  int n_chunks, BH, H, group, D, M;
  float scale;
};

template <int DP>
struct ChainLayout {
  static constexpr int kBoxes = DP / 64;
  static constexpr int kKQBox = 2 * kBox;
  static constexpr int kKQ = kBoxes * kKQBox;
  static constexpr int kS = DP * 128;
  static constexpr int oT = 2 * kKQ;           // hi, lo
  static constexpr int oP = oT + 2 * kBox;     // hi, lo
  static constexpr int oS = oP + 2 * kBox;     // hi, lo
  static constexpr int oB = oS + 2 * kS;       // [128 x 64]: dU, then -gam b dX; s gam dO; hi, lo
  static constexpr int oB3 = oB + 4 * kBox;    // [64 x 64]: dU's third part
  static constexpr int oO = oB3 + kBox;        // dO
  static constexpr int oV = oO + kBox;
  static constexpr int oX = oV + kBox;         // dX: hi, lo
  static constexpr int oDV = oX + 2 * kBox;
  static constexpr int oG = oDV + kBox;
  static constexpr int oBar = oG + 2 * (int)sizeof(GateSlot);
  static constexpr int kBytes = oBar + 128 + 1024;
  static_assert(kBytes <= tc::kSmemLimit, "shared memory");
};

template <int DP>
__global__ void __launch_bounds__(256, 1)
    delta_tc_chain_kernel(const __grid_constant__ CUtensorMap tm_q,
                          const __grid_constant__ CUtensorMap tm_k,
                          const __grid_constant__ CUtensorMap tm_v,
                          const __grid_constant__ CUtensorMap tm_do,
                          const __grid_constant__ CUtensorMap tm_dv,
                          const __grid_constant__ CUtensorMap tm_x,
                          const __grid_constant__ CUtensorMap tm_ds, const ChainArgs a) {
  using L = ChainLayout<DP>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                           ~static_cast<uintptr_t>(1023));
  GateSlot* gates = reinterpret_cast<GateSlot*>(sm + L::oG);
  uint64_t* kq_full = reinterpret_cast<uint64_t*>(sm + L::oBar);  // [2]
  uint64_t *t_full = kq_full + 2, *p_full = kq_full + 3, *v_full = kq_full + 4, *o_full = kq_full + 5;
  uint64_t* done = kq_full + 6;  // [3]
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(done + 3);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0);  // (uniform to the compiler)
  const int lane = threadIdx.x % 32, sub = warp / 4, t = threadIdx.x % 128;
  const int p = blockIdx.x;  // b * H + h
  const int pk = (p / a.H) * (a.H / a.group) + (p % a.H) / a.group;
  const int n = a.n_chunks, c64 = blockIdx.y * 64;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 9; ++i) mbar_init(kq_full + i, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(tmem_holder, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_holder, 0), s_base = smem_u32(sm);
  const uint32_t lane_col = ((uint32_t)(warp % 4) << 21) + 32 * sub;  // this thread's columns
  // K dS', then dX; P^T dO, then dX's third accumulator; the update; dS
  const uint32_t t_acc = tmem, t_e0 = tmem + 128, t_up = tmem + 192, t_s = tmem + 320;
  const uint32_t T_addr = s_base + L::oT, P_addr = s_base + L::oP, S_addr = s_base + L::oS;
  const uint32_t B_addr = s_base + L::oB, O_addr = s_base + L::oO;
  uint8_t *S_hi = sm + L::oS, *S_lo = S_hi + L::kS;
  uint8_t *B_hi = sm + L::oB, *B_lo = B_hi + 2 * kBox;
  constexpr uint32_t id_nt128 = idesc_bf16_f32(128, 128, 0, 1);
  constexpr uint32_t id_nt192 = idesc_bf16_f32(128, 192, 0, 1);
  constexpr uint32_t id_tt64 = idesc_bf16_f32(128, 64, 1, 1);
  constexpr uint32_t id_tt128 = idesc_bf16_f32(128, 128, 1, 1);
  const uint64_t once = policy_evict_first();
  // step s of the walk is chunk n - 1 - s
  auto load_kq = [&](int s) {
    uint64_t* bar = kq_full + (s & 1);
    uint8_t* dst = sm + (s & 1) * L::kKQ;
    mbar_arrive_expect_tx(bar, L::kKQ);
    for (int x = 0; x < L::kBoxes; ++x) {
      tma_load_3d(dst + x * L::kKQBox, &tm_k, bar, 64 * x, (n - 1 - s) * kCh, pk, once);
      tma_load_3d(dst + x * L::kKQBox + kBox, &tm_q, bar, 64 * x, (n - 1 - s) * kCh, pk, once);
    }
  };
  auto load_tile = [&](int at, const uint8_t* src, uint64_t* bar, int s) {
    mbar_arrive_expect_tx(bar, 2 * kBox);
    bulk_load(sm + at, src + ((int64_t)p * n + n - 1 - s) * (2 * kBox), 2 * kBox, bar);
  };
  auto load_rows = [&](int at, const CUtensorMap* map, uint64_t* bar, int s) {
    mbar_arrive_expect_tx(bar, kBox);
    tma_load_3d(sm + at, map, bar, c64, (n - 1 - s) * kCh, p, once);
  };
  auto issue_e0 = [&](int s) {  // warp 0: P^T dO of step s
    wait_or_abort(p_full, s & 1, a.status, abort_flag);
    wait_or_abort(o_full, s & 1, a.status, abort_flag);
    __syncwarp();
    const uint32_t el = elect_one();
    mma_tile<4, true, true>(el, t_e0, P_addr, O_addr, id_tt64, kBox, 16, 0, 0, true);
    mma_tile<4, true, true>(el, t_e0, P_addr + kBox, O_addr, id_tt64, kBox, 16, 0, 0, false);
  };
  // one warp: the gates, loaded a step before they are written
  float4 gb;
  auto load_gates = [&](int s) {
    const int64_t i = (int64_t)(n - 1 - s) * kCh + lane;
    const float* g = a.g + p * a.N;
    const float* b = a.beta + p * a.N;
    gb = make_float4(i < a.N ? g[i] : 0.f, i + 32 < a.N ? g[i + 32] : 0.f, i < a.N ? b[i] : 0.f,
                     i + 32 < a.N ? b[i + 32] : 0.f);
  };
  auto put_gates = [&](int s) {
    write_gates(gates + (s & 1), lane, gb.x, gb.y, gb.z, gb.w);
    if (s + 1 < n) load_gates(s + 1);
  };

  if (threadIdx.x == 96) {
    load_kq(0);
    load_tile(L::oP, a.pm, p_full, 0);
    load_rows(L::oO, &tm_do, o_full, 0);
    load_tile(L::oT, a.t, t_full, 0);
    load_rows(L::oV, &tm_v, v_full, 0);
    if (n > 1) load_kq(1);
  }
  const bool row_on = t < a.D;
#pragma unroll 1
  for (int h = 0; h < 2; ++h) {
    const int c0 = c64 + 32 * sub + 16 * h;
    float2 s[8];
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (a.grad_state_out != nullptr && row_on && c0 + 2 * j < a.M)
        v = *reinterpret_cast<const float4*>(a.grad_state_out + ((int64_t)p * a.D + t) * a.M + c0 + 2 * j);
      s[j] = make_float2(v.x, v.y);
      s[j + 1] = make_float2(v.z, v.w);
    }
    tmem_st16(t_s + lane_col + 16 * h, s);
    if (t < DP) store16_split(S_hi, S_lo, t, 4 * sub + 2 * h, s);
  }
  tmem_st_wait();
  if (warp == 7) {
    load_gates(0);
    put_gates(0);
  }
  if (warp == 0) issue_e0(0);

  for (int s = 0; s < n; ++s) {
    const uint32_t kq = s_base + (s & 1) * L::kKQ, phase = s & 1;
    const GateSlot* gs = gates + (s & 1);
    const int chunk = n - 1 - s;
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
      wait_or_abort(kq_full + (s & 1), (s >> 1) & 1, a.status, abort_flag);
      __syncwarp();
      tc_fence_after();
      const uint32_t el = elect_one();
      mma_tile<DP / 16, false, true>(el, t_acc, kq, S_addr, id_nt128, 16, L::kS, L::kKQBox, 0, true);
      if (el) mma_commit(done);
    }
    if (threadIdx.x == 128) {
      const int at = (p * n + chunk) * 2;
      tma_store_3d(&tm_ds, S_hi, c64, 0, at);
      tma_store_3d(&tm_ds, S_lo, c64, 0, at + 1);
      if (s > 0) {  // the step before's dX and dV
        tma_store_3d(&tm_x, sm + L::oX, c64, (chunk + 1) * kCh, p);
        tma_store_3d(&tm_x, sm + L::oX + kBox, c64, (chunk + 1) * kCh, a.BH + p);
        tma_store_3d(&tm_dv, sm + L::oDV, c64, (chunk + 1) * kCh, p);
      }
      tma_store_commit();
    }
    if (t >= 64) {  // s gam dO, under the product
      const float2 w = both(a.scale * gs->gam[t - 64]);
      wait_or_abort(o_full, phase, a.status, abort_flag);
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        float2 x[8];
        get16(sm + L::oO, t - 64, 4 * sub + 2 * h, x);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = mul2(w, x[j]);
        store16_split(B_hi, B_lo, t, 4 * sub + 2 * h, x);
      }
    }
    wait_or_abort(done, phase, a.status, abort_flag);
    tc_fence_after();
    if (t < 64) {
      const float2 del = both(gs->del[t]);
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        uint32_t e0[16];
        tmem_ld16(t_e0 + lane_col + 16 * h, e0);
        float2 r[8];
        load16_sum(t_acc + lane_col + 16 * h, r);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          r[j] = fma2(del, r[j], make_float2(__uint_as_float(e0[2 * j]), __uint_as_float(e0[2 * j + 1])));
        uint4 x0[2], x1[2], x2[2];
        split16_3(r, x0, x1, x2);
        put16(B_hi, t, 4 * sub + 2 * h, x0);
        put16(B_lo, t, 4 * sub + 2 * h, x1);
        put16(sm + L::oB3, t, 4 * sub + 2 * h, x2);
      }
    }
    // the stores out of the S, dX and dV tiles have read them
    if (threadIdx.x == 128) tma_store_wait_read_all();
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
      wait_or_abort(t_full, phase, a.status, abort_flag);
      __syncwarp();
      tc_fence_after();
      const uint32_t el = elect_one();
      // T^T hi with dU's three parts (the third's accumulator takes P^T dO's
      // place, which has been read), T^T lo with two
      mma_tile<4, false, true>(el, t_acc, T_addr, B_addr, id_nt192, 16, 2 * kBox, 0, 0, true);
      mma_tile<4, false, true>(el, t_acc, T_addr + kBox, B_addr, id_nt128, 16, 2 * kBox, 0, 0, false);
      if (el) mma_commit(done + 1);
    }
    if (threadIdx.x == 96 && s + 1 < n) {  // P^T dO and s gam dO have read them
      load_tile(L::oP, a.pm, p_full, s + 1);
      load_rows(L::oO, &tm_do, o_full, s + 1);
    }
    if (warp == 7 && s + 1 < n) put_gates(s + 1);
    wait_or_abort(done + 1, phase, a.status, abort_flag);
    tc_fence_after();
    float2 r3[8];
    const float2 w = both(t < 64 ? -gs->b[t] * gs->gam[t] : 0.f);
    if (t < 64) {
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        float2 r[8];
        tmem_ld16(t_e0 + lane_col + 16 * h, r3);
        load16_sum(t_acc + lane_col + 16 * h, r);
#pragma unroll
        for (int j = 0; j < 8; ++j) r[j] = mul2(w, add2(r[j], r3[j]));
        store16_split(B_hi, B_lo, t, 4 * sub + 2 * h, r);
      }
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
      tc_fence_after();
      const uint32_t el = elect_one();
      // [K; Q]^T: 128 rows along K; with one 64-column block the lanes past 64
      // read on into the tiles behind, and are not used
      constexpr uint32_t lbo = DP == 128 ? L::kKQBox : kBox;
      mma_tile<8, true, true>(el, t_up, kq, B_addr, id_tt128, lbo, 2 * kBox, 0, 0, true);
      if (el) mma_commit(done + 2);
    }
    if (threadIdx.x == 96 && s + 1 < n) load_tile(L::oT, a.t, t_full, s + 1);
    if (t < 64) {  // under the product
      const int64_t i = (int64_t)chunk * kCh + t;
      const float2 b = both(gs->b[t]);
      float2 dot = both(0.f);
      wait_or_abort(v_full, phase, a.status, abort_flag);
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        float2 r[8], v[8];
        tmem_ld16(t_e0 + lane_col + 16 * h, r3);
        load16_sum(t_acc + lane_col + 16 * h, r);
        get16(sm + L::oV, t, 4 * sub + 2 * h, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          r[j] = add2(r[j], r3[j]);
          dot = fma2(r[j], v[j], dot);
        }
        store16_split(sm + L::oX, sm + L::oX + kBox, t, 4 * sub + 2 * h, r);
#pragma unroll
        for (int j = 0; j < 8; ++j) r[j] = mul2(b, r[j]);
        uint4 dv[2];
        pack16(r, dv);
        put16(sm + L::oDV, t, 4 * sub + 2 * h, dv);
      }
      if (i < a.N && c64 + 32 * sub < a.M)
        a.xv[((int64_t)(c64 / 32 + sub) * a.BH + p) * a.N + i] = dot.x + dot.y;
    }
    tc_fence_before();
    __syncthreads();  // dX has been read, and V
    if (warp == 0 && s + 1 < n) {
      tc_fence_after();
      issue_e0(s + 1);
    }
    if (threadIdx.x == 96 && s + 1 < n) load_rows(L::oV, &tm_v, v_full, s + 1);
    wait_or_abort(done + 2, phase, a.status, abort_flag);
    tc_fence_after();
    if (threadIdx.x == 96 && s + 2 < n) load_kq(s + 2);
    const float2 last = both(gs->gam[kCh - 1]);
#pragma unroll 1
    for (int h = 0; h < 2; ++h) {
      float2 r[8], x[8];
      load16_sum(t_up + lane_col + 16 * h, r);
      tmem_ld16(t_s + lane_col + 16 * h, x);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = fma2(last, x[j], r[j]);
      tmem_st16(t_s + lane_col + 16 * h, x);
      if (t < DP) store16_split(S_hi, S_lo, t, 4 * sub + 2 * h, x);
    }
    tmem_st_wait();
  }
  if (a.grad_state_in != nullptr) {
#pragma unroll 1
    for (int h = 0; h < 2; ++h) {
      const int c0 = c64 + 32 * sub + 16 * h;
      float2 s[8];
      tmem_ld16(t_s + lane_col + 16 * h, s);
#pragma unroll
      for (int j = 0; j < 8; j += 2)
        if (row_on && c0 + 2 * j < a.M)
          *reinterpret_cast<float4*>(a.grad_state_in + ((int64_t)p * a.D + t) * a.M + c0 + 2 * j) =
              make_float4(s[j].x, s[j].y, s[j + 1].x, s[j + 1].y);
    }
  }
  fence_proxy_async_smem();
  __syncthreads();
  if (threadIdx.x == 128) {  // the last step's (chunk 0) dX and dV
    tma_store_3d(&tm_x, sm + L::oX, c64, 0, p);
    tma_store_3d(&tm_x, sm + L::oX + kBox, c64, 0, a.BH + p);
    tma_store_3d(&tm_dv, sm + L::oDV, c64, 0, p);
    tma_store_commit();
    tma_store_wait_all();
    if (*abort_flag) linger();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------- gradients
struct GradArgs {
  const float *g, *beta, *xv;
  __nv_bfloat16 *dq, *dk;       // written whole (one value head to a key head) ..
  float *dq_part, *dk_part;     // .. or [BH][N][D] fp32 parts
  float *dg, *dbeta;
  int* status;
  int64_t N;
  int n_chunks, BH, H, group, D, M;
  float scale;
};

template <int DP>
struct GradLayout {
  static constexpr int kBoxes = DP / 64;
  static constexpr int kKQBox = 2 * kBox;
  static constexpr int kKQ = kBoxes * kKQBox;
  static constexpr int kS = DP * 128;
  static constexpr int oA = kKQ;              // [dX; dO] hi, [dX lo; 0]; then [Ma; Mq] hi, lo
  static constexpr int oU = oA + 4 * kBox;    // hi, lo
  static constexpr int oS = oU + 2 * kBox;    // hi, lo
  static constexpr int oD = oS + 2 * kS;      // dS' hi, lo
  static constexpr int oG = oD + 2 * kS;
  static constexpr int oX = oG + (int)sizeof(GateSlot);  // sums for the gates
  static constexpr int kXFloats = 8 * 64 + 2 * 64 * 6 + 16;
  static constexpr int oBar = oX + kXFloats * 4;
  static constexpr int kBytes = oBar + 64 + 1024;
  static constexpr int kStage = 3 * kBox + 2 * kBox + 4 * kS;  // bytes TMA brings per 64 value columns
  static constexpr int kCols = DP == 64 ? 256 : 512;           // tensor memory
  static constexpr int kPerSM = DP == 64 ? 2 : 1;
  static_assert(kPerSM * (kBytes + 1024) <= 233472, "shared memory");
};

// The 32 columns 32 ch .. of the row's decayed products, as decayed_row gives
// them; f(c, v, r): v the weights alone (0 where masked), r the accumulator.
template <class F>
__device__ __forceinline__ void decayed_half(uint32_t t_acc, const GateSlot* gs, int i, bool diag,
                                             int row32, int ch, float w, F f) {
  const int last = diag ? i : i - 1;
  float p = w;
  if (ch < row32) p *= gs->half[i - 32];
#pragma unroll 1
  for (int c = 2 * ch + 1; c >= 2 * ch; --c) {
    float2 v[8];
    if (ch == row32) {
      float x[17];
#pragma unroll
      for (int e = 0; e < 16; e += 4) {
        const float4 t = *reinterpret_cast<const float4*>(gs->a + 16 * c + e);
        x[e] = t.x; x[e + 1] = t.y; x[e + 2] = t.z; x[e + 3] = t.w;
      }
      x[16] = gs->a[16 * c + 16];
      float u[16];
#pragma unroll
      for (int e = 15; e >= 0; --e) {
        if (16 * c + e < i) p *= x[e + 1];
        u[e] = 16 * c + e <= last ? p : 0.f;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = make_float2(u[2 * e], u[2 * e + 1]);
    } else if (ch < row32) {
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const float4 t = *reinterpret_cast<const float4*>(gs->e + 16 * c + 2 * e);
        v[e] = mul2(both(p), make_float2(t.x, t.y));
        v[e + 1] = mul2(both(p), make_float2(t.z, t.w));
      }
      p *= gs->piece[c];
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = both(0.f);
    }
    f(c, v);
  }
}

template <int DP>
__global__ void __launch_bounds__(256, GradLayout<DP>::kPerSM)
    delta_tc_grad_kernel(const __grid_constant__ CUtensorMap tm_q,
                         const __grid_constant__ CUtensorMap tm_k,
                         const __grid_constant__ CUtensorMap tm_do,
                         const __grid_constant__ CUtensorMap tm_x,
                         const __grid_constant__ CUtensorMap tm_u,
                         const __grid_constant__ CUtensorMap tm_s,
                         const __grid_constant__ CUtensorMap tm_ds, const GradArgs a) {
  using L = GradLayout<DP>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                           ~static_cast<uintptr_t>(1023));
  GateSlot* gs = reinterpret_cast<GateSlot*>(sm + L::oG);
  float* e_sum = reinterpret_cast<float*>(sm + L::oX);  // [8 warps][64]: pairs' part of dg
  float* dots = e_sum + 512;     // [2 column halves][6][64]: rows' sums, as written below
  float* z_sum = dots + 768;     // [8]
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::oBar);
  uint64_t *kq_full = bars, *full = bars + 1, *done = bars + 2;  // done [2]
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + 4);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0);  // (uniform to the compiler)
  const int lane = threadIdx.x % 32, wg = warp / 4, t = threadIdx.x % 128;
  const bool issuer = threadIdx.x == 0;
  const int64_t p = blockIdx.x / a.n_chunks;
  const int chunk = blockIdx.x % a.n_chunks, i0 = chunk * kCh;
  const int pk = (int)((p / a.H) * (a.H / a.group) + (p % a.H) / a.group);
  const int n_mb = (a.M + 63) / 64;

  if (issuer) {
    for (int i = 0; i < 4; ++i) mbar_init(bars + i, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(tmem_holder, L::kCols);
    tmem_relinquish();
  }
  if (warp == 1) {
    const int64_t i = i0 + lane, at = p * a.N;
    write_gates(gs, lane, i < a.N ? a.g[at + i] : 0.f, i + 32 < a.N ? a.g[at + i + 32] : 0.f,
                i < a.N ? a.beta[at + i] : 0.f, i + 32 < a.N ? a.beta[at + i + 32] : 0.f);
  }
  // no lo part under dO
  for (int i = threadIdx.x; i < kBox / 16; i += 256)
    reinterpret_cast<uint4*>(sm + L::oA + 3 * kBox)[i] = make_uint4(0, 0, 0, 0);
  for (int i = threadIdx.x; i < 512; i += 256) e_sum[i] = 0.f;
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_holder, 0), s_base = smem_u32(sm);
  const uint32_t t_kk = tmem, t_p2 = tmem + 64, t_in = tmem + 128, t_u = t_in + DP;
  const uint32_t lane_base = (uint32_t)(warp % 4) << 21;
  const uint32_t A_addr = s_base + L::oA, U_addr = s_base + L::oU, S_addr = s_base + L::oS;
  const uint32_t D_addr = s_base + L::oD;
  constexpr uint32_t id_nn64 = idesc_bf16_f32(128, 64, 0, 0);
  constexpr uint32_t id_nnD = idesc_bf16_f32(128, DP, 0, 0);
  constexpr uint32_t id_ntD = idesc_bf16_f32(128, DP, 0, 1);
  constexpr uint32_t id_ttD = idesc_bf16_f32(128, DP, 1, 1);
  const uint64_t keep = policy_evict_first();
  auto load_mb = [&](int m) {
    mbar_arrive_expect_tx(full, L::kStage);
    const int c = 64 * m, s0 = (int)((p * a.n_chunks + chunk) * 2);
    tma_load_3d(sm + L::oA, &tm_x, full, c, i0, (int)p, keep);
    tma_load_3d(sm + L::oA + kBox, &tm_do, full, c, i0, (int)p, keep);
    tma_load_3d(sm + L::oA + 2 * kBox, &tm_x, full, c, i0, a.BH + (int)p, keep);
    tma_load_3d(sm + L::oU, &tm_u, full, c, i0, (int)p, keep);
    tma_load_3d(sm + L::oU + kBox, &tm_u, full, c, i0, a.BH + (int)p, keep);
    for (int h = 0; h < 2; ++h) {
      tma_load_3d(sm + L::oS + h * L::kS, &tm_s, full, c, 0, s0 + h, keep);
      tma_load_3d(sm + L::oD + h * L::kS, &tm_ds, full, c, 0, s0 + h, keep);
    }
  };
  if (issuer) {
    mbar_arrive_expect_tx(kq_full, L::kKQ);
    for (int x = 0; x < L::kBoxes; ++x) {
      tma_load_3d(sm + x * L::kKQBox, &tm_k, kq_full, 64 * x, i0, pk, keep);
      tma_load_3d(sm + x * L::kKQBox + kBox, &tm_q, kq_full, 64 * x, i0, pk, keep);
    }
    load_mb(0);
  }
  if (warp == 0) {
    wait_or_abort(kq_full, 0, a.status, abort_flag);
    __syncwarp();
    mma_tile<DP / 16, false, false>(elect_one(), t_kk, s_base, s_base, id_nn64, 16, 16, L::kKQBox, L::kKQBox, true);
  }
  float z = 0.f;  // <S, dS'>, this thread's share
  for (int m = 0; m < n_mb; ++m) {
    if (warp == 0) {
      wait_or_abort(full, m & 1, a.status, abort_flag);
      __syncwarp();
      const uint32_t el = elect_one();
#pragma unroll 1
      for (int x = 0; x < 4; ++x) {
        // (A hi, B hi), (A lo, B hi), (A hi, B lo), (A lo, B lo)
        const uint32_t ap = (x & 1) * 2 * kBox, up = (x & 1) * kBox, b = x >> 1;
        const bool fresh = m == 0 && x == 0;
        mma_tile<4, false, false>(el, t_p2, A_addr + ap, U_addr + b * kBox, id_nn64, 16, 16, 0, 0, fresh);
        mma_tile<4, false, false>(el, t_in, A_addr + ap, S_addr + b * L::kS, id_nnD, 16, 16, 0, 0, fresh);
        // lanes past 64 read on behind U and are not used
        mma_tile<4, false, false>(el, t_u, U_addr + up, D_addr + b * L::kS, id_nnD, 16, 16, 0, 0, fresh);
      }
      if (el) mma_commit(done);
    }
    wait_or_abort(full, m & 1, a.status, abort_flag);
    // the MMAs read the tiles at the same time
    for (int e = threadIdx.x; e < DP * 8; e += 256) {
      const uint4 sh = *reinterpret_cast<const uint4*>(sm + L::oS + 16 * e);
      const uint4 sl = *reinterpret_cast<const uint4*>(sm + L::oS + L::kS + 16 * e);
      const uint4 dh = *reinterpret_cast<const uint4*>(sm + L::oD + 16 * e);
      const uint4 dl = *reinterpret_cast<const uint4*>(sm + L::oD + L::kS + 16 * e);
      const uint32_t w[4][4] = {{sh.x, sh.y, sh.z, sh.w}, {sl.x, sl.y, sl.z, sl.w},
                                {dh.x, dh.y, dh.z, dh.w}, {dl.x, dl.y, dl.z, dl.w}};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float s0 = __uint_as_float(w[0][i] << 16) + __uint_as_float(w[1][i] << 16);
        const float s1 = __uint_as_float(w[0][i] & 0xffff0000u) + __uint_as_float(w[1][i] & 0xffff0000u);
        const float d0 = __uint_as_float(w[2][i] << 16) + __uint_as_float(w[3][i] << 16);
        const float d1 = __uint_as_float(w[2][i] & 0xffff0000u) + __uint_as_float(w[3][i] & 0xffff0000u);
        z = fmaf(s1, d1, fmaf(s0, d0, z));
      }
    }
    wait_or_abort(done, m & 1, a.status, abort_flag);
    if (m + 1 < n_mb) {
      fence_proxy_async_smem();
      __syncthreads();  // every thread has read the tiles
      if (issuer) load_mb(m + 1);
    }
  }
  tc_fence_after();
  for (int o = 16; o > 0; o /= 2) z += __shfl_xor_sync(0xffffffffu, z, o);
  if (lane == 0) z_sum[warp] = z;

  // lanes 0-63 ("K rows"): i = t; lanes 64-127 ("Q rows"): i = t - 64
  const bool is_k = t < 64;
  const int i = t & 63, row32 = i / 32;
  const float gam = gs->gam[i], del = gs->del[i], bt = gs->b[i];
  // the products with the state: a half of D's columns a thread
  constexpr int HC = DP / 2;
  float2 g2[HC / 2];
  {
    const uint8_t* xr = sm;  // the row of k or q
    const float w = is_k ? -gam * bt : a.scale * gam;
    float2 din = both(0.f), du = both(0.f);
#pragma unroll
    for (int h = 0; h < HC / 16; ++h) {
      const int c = wg * HC + 16 * h;
      uint32_t r[16], u[16];
      tmem_ld16(t_in + lane_base + c, r);
      tmem_ld16(t_u + lane_base + c, u);
      tmem_ld_wait();
      const uint8_t* src = xr + (c / 64) * L::kKQBox + t * 128;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint4 x4 = *reinterpret_cast<const uint4*>(src + ((((c & 63) / 8 + j) ^ (t & 7)) << 4));
        const uint32_t xw[4] = {x4.x, x4.y, x4.z, x4.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int k = 8 * j + 2 * e;
          const float2 x = make_float2(__uint_as_float(xw[e] << 16), __uint_as_float(xw[e] & 0xffff0000u));
          const float2 in = make_float2(__uint_as_float(r[k]), __uint_as_float(r[k + 1]));
          din = fma2(x, in, din);
          float2 o = mul2(both(w), in);
          if (is_k) {
            const float2 uu = make_float2(__uint_as_float(u[k]), __uint_as_float(u[k + 1]));
            du = fma2(x, uu, du);
            o = fma2(both(del), uu, o);
          }
          g2[8 * h + k / 2] = o;
        }
      }
    }
    // [0] k . (dX S^T), [1] q . (dO S^T), [2] k . (U dS'^T)
    float* d = dots + wg * 384;
    if (is_k) {
      d[i] = din.x + din.y;
      d[128 + i] = du.x + du.y;
    } else {
      d[64 + i] = din.x + din.y;
    }
  }
  // Ma and Mq, their tiles, and the pairs' sums
  uint8_t *M_hi = sm + L::oA, *M_lo = M_hi + 2 * kBox;
  float part[32];    // columns 32 wg ..: the pair's weight in dg, then its running sum
  float db = 0.f, own = 0.f;  // own: dX_i . U_i
  decayed_half(t_p2, gs, i, !is_k, row32, wg, is_k ? -1.f : a.scale, [&](int c, float2(&v)[8]) {
    uint32_t r[16], kk[16];
    tmem_ld16(t_p2 + lane_base + 16 * c, r);
    tmem_ld16(t_kk + lane_base + 16 * c, kk);
    tmem_ld_wait();
    const float wm = is_k ? bt : 1.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      // masked places stay 0 whatever the accumulators hold
      float2 m = mul2(v[e], make_float2(__uint_as_float(r[2 * e]), __uint_as_float(r[2 * e + 1])));
      const int j = 16 * c + 2 * e, last = is_k ? i - 1 : i;
      if (j > last) m.x = 0.f;
      if (j + 1 > last) m.y = 0.f;
      float2 x = mul2(m, make_float2(__uint_as_float(kk[2 * e]), __uint_as_float(kk[2 * e + 1])));
      if (j > last) x.x = 0.f;
      if (j + 1 > last) x.y = 0.f;
      db += x.x + x.y;
      if (j == i) own = __uint_as_float(r[2 * e]);
      if (j + 1 == i) own = __uint_as_float(r[2 * e + 1]);
      v[e] = mul2(both(wm), m);
      x = mul2(both(wm), x);
      if ((c & 1) == 0) {
        part[2 * e] = x.x;
        part[2 * e + 1] = x.y;
      } else {
        part[16 + 2 * e] = x.x;
        part[16 + 2 * e + 1] = x.y;
      }
    }
    store16_split(M_hi, M_lo, t, 2 * c, v);
  });
  tc_fence_before();
  fence_proxy_async_smem();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    const uint32_t el = elect_one();
#pragma unroll 1
    for (int x = 0; x < 2; ++x) {  // the tile's hi and lo parts
      const uint32_t ap = A_addr + x * 2 * kBox;
      // [Ma; Mq] K
      mma_tile<4, false, true>(el, t_in, ap, s_base, id_ntD, 16, L::kKQBox, 0, 0, x == 0);
      // Ma^T K + Mq^T Q; lanes past 64 read on and are not used
      mma_tile<8, true, true>(el, t_u, ap, s_base, id_ttD, kBox, L::kKQBox, 0, 0, x == 0);
    }
    if (el) mma_commit(done + 1);
  }
  // under the products: dg_t's pairs, sum over rows i >= t of the row's columns
  // before t.  Running sums along the row first; column 32 wg + k of `part`
  // then belongs to t = 32 wg + k + 1.
  float run = 0.f;
#pragma unroll
  for (int k = 0; k < 32; ++k) {
    run += part[k];
    part[k] = run;
  }
#pragma unroll
  for (int k = 0; k < 32; ++k)
    if (32 * wg + k + 1 > i) part[k] = 0.f;
  // sum over the warp's 32 rows: lane l ends with column l
#pragma unroll
  for (int o = 16; o > 0; o /= 2) {
    const bool up = (lane & o) != 0;
#pragma unroll
    for (int k = 0; k < o; ++k) {
      const float give = up ? part[k] : part[k + o];
      const float get = __shfl_xor_sync(0xffffffffu, give, o);
      part[k] = (up ? part[k + o] : part[k]) + get;
    }
  }
  if (32 * wg + lane + 1 < 64) e_sum[warp * 64 + 32 * wg + lane + 1] = part[0];
  if (wg == 0 && row32 == 1) {
    // rows 32-63, columns 0-31: their whole sum for every t in 33 .. i
    float x = run;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const float y = __shfl_down_sync(0xffffffffu, x, o);
      if (lane + o < 32) x += y;
    }
    if (lane > 0) e_sum[warp * 64 + 32 + lane] = x;
  }
  if (is_k) {
    dots[wg * 384 + 192 + i] = db;
    if (row32 == wg) dots[256 + i] = own;
  }
  __syncthreads();
  if (warp == 7) {
    // the gates' gradients: lane l has rows l and l + 32
    const float zt = gs->gam[kCh - 1] * (((z_sum[0] + z_sum[1]) + (z_sum[2] + z_sum[3])) +
                                         ((z_sum[4] + z_sum[5]) + (z_sum[6] + z_sum[7])));
    float r[2], c[2], own[2], kx[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int j = lane + 32 * h;
      kx[h] = dots[j] + dots[384 + j];
      const float qo = dots[64 + j] + dots[448 + j], ku = dots[128 + j] + dots[512 + j];
      r[h] = gs->gam[j] * (a.scale * qo - gs->b[j] * kx[h]);
      own[h] = c[h] = gs->del[j] * ku;
    }
    // sums of r from the row on, of c before it
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float x = __shfl_down_sync(0xffffffffu, r[h], o), y = __shfl_up_sync(0xffffffffu, c[h], o);
        if (lane + o < 32) r[h] += x;
        if (lane >= o) c[h] += y;
      }
    }
    const float r_hi = __shfl_sync(0xffffffffu, r[1], 0), c_lo = __shfl_sync(0xffffffffu, c[0], 31);
    c[0] -= own[0];
    c[1] -= own[1];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int j = lane + 32 * h;
      if (i0 + j < a.N) {
        float s = zt + r[h] + c[h] + (h ? c_lo : r_hi);
        for (int x = 0; x < 8; ++x) s += e_sum[x * 64 + j];
        const int64_t at = p * a.N + i0 + j;
        a.dg[at] = s;
        float d = dots[192 + j] + dots[576 + j] - gs->gam[j] * kx[h];
        for (int x = 0; x < (a.M + 31) / 32; ++x) d += a.xv[(int64_t)x * a.BH * a.N + at];
        // U carries b as a factor, far above the smallest number down to 2^-80
        const float b = gs->b[j];
        a.dbeta[at] = fabsf(b) < 0x1p-80f ? d : dots[256 + j] / b;
      }
    }
  }
  wait_or_abort(done + 1, 0, a.status, abort_flag);
  tc_fence_after();
  const int64_t orow = p * a.N + i0 + i;
  const bool live = i0 + i < a.N;
#pragma unroll
  for (int h = 0; h < HC / 16; ++h) {
    const int c = wg * HC + 16 * h;
    uint32_t r[16], u[16];
    tmem_ld16(t_in + lane_base + c, r);
    tmem_ld16(t_u + lane_base + c, u);
    tmem_ld_wait();
    float2 o[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      o[e] = add2(g2[8 * h + e], make_float2(__uint_as_float(r[2 * e]), __uint_as_float(r[2 * e + 1])));
      if (is_k)
        o[e] = add2(o[e], make_float2(__uint_as_float(u[2 * e]), __uint_as_float(u[2 * e + 1])));
    }
    if (a.dq_part != nullptr) {
      float* to = (is_k ? a.dk_part : a.dq_part) + orow * a.D + c;
#pragma unroll
      for (int e = 0; e < 8; e += 2)
        if (live && c + 2 * e < a.D)
          *reinterpret_cast<float4*>(to + 2 * e) = make_float4(o[e].x, o[e].y, o[e + 1].x, o[e + 1].y);
    } else {
      __nv_bfloat16* to = (is_k ? a.dk : a.dq) + orow * a.D + c;
      uint4 w[2];
#pragma unroll
      for (int j = 0; j < 2; ++j)
        w[j] = make_uint4(tc::pack_bf16x2(o[4 * j].x, o[4 * j].y), tc::pack_bf16x2(o[4 * j + 1].x, o[4 * j + 1].y),
                          tc::pack_bf16x2(o[4 * j + 2].x, o[4 * j + 2].y),
                          tc::pack_bf16x2(o[4 * j + 3].x, o[4 * j + 3].y));
      if (live) write16(to, a.D - c, w);
    }
  }
  if (*abort_flag) linger();
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, L::kCols);
  }
}

// What the chain leaves for the gradients.
struct Scratch {
  int64_t ds, dx, xv, part;  // bytes
  uint8_t *ds_at, *dx_at, *xv_at, *part_at;
  explicit Scratch(const DeltaShape& s, void* at = nullptr) {
    auto up = [](int64_t x) { return (x + 255) / 256 * 256; };
    const int64_t BH = s.B * s.H, n = (s.N + kCh - 1) / kCh;
    ds = up(4 * BH * n * s.D * s.M);
    dx = up(4 * BH * s.N * s.M);
    xv = up(4 * ((s.M + 31) / 32) * BH * s.N);
    part = s.H == s.Hk ? 0 : up(4 * BH * s.N * s.D);
    ds_at = static_cast<uint8_t*>(at);
    dx_at = ds_at + ds;
    xv_at = dx_at + dx;
    part_at = xv_at + xv;
  }
  int64_t bytes() const { return ds + dx + xv + 2 * part; }
};

template <int DP>
cp_status_t launch(const DeltaShape& s, const DeltaBwd& f, const Scratch& w, const ChainArgs& c,
                   const GradArgs& g, cudaStream_t stream) {
  const uint8_t* kept = reinterpret_cast<const uint8_t*>(f.ckpt);
  using LC = ChainLayout<DP>;
  using LG = GradLayout<DP>;
  auto chain = delta_tc_chain_kernel<DP>;
  auto grad = delta_tc_grad_kernel<DP>;
  if (cudaFuncSetAttribute(chain, cudaFuncAttributeMaxDynamicSharedMemorySize, LC::kBytes) != cudaSuccess ||
      cudaFuncSetAttribute(grad, cudaFuncAttributeMaxDynamicSharedMemorySize, LG::kBytes) != cudaSuccess)
    return CP_ERR_CUDA;
  // (encoding a map needs the device's context current in this thread: the
  // calls above see to that)
  const Saved k(s);
  const int64_t heads = s.B * s.H;
  CUtensorMap q, kk, v, go, dv, x, u, st, ds;
  if (!make_chunk_map(&q, f.q, s.B * s.Hk, s.N, s.D) || !make_chunk_map(&kk, f.k, s.B * s.Hk, s.N, s.D) ||
      !make_chunk_map(&v, f.v, heads, s.N, s.M) || !make_chunk_map(&go, f.grad_out, heads, s.N, s.M) ||
      !make_chunk_map(&dv, f.dv, heads, s.N, s.M) || !make_chunk_map(&x, w.dx_at, 2 * heads, s.N, s.M) ||
      !make_chunk_map(&u, kept + k.s_bytes, 2 * heads, s.N, s.M) ||
      !make_chunk_map(&st, kept, heads * k.n * 2, s.D, s.M, DP) ||
      !make_chunk_map(&ds, w.ds_at, heads * k.n * 2, s.D, s.M, DP))
    return CP_ERR_CUDA;
  const unsigned BH = (unsigned)heads;
  chain<<<dim3(BH, (unsigned)((s.M + 63) / 64)), 256, LC::kBytes, stream>>>(q, kk, v, go, dv, x, ds, c);
  if (cudaGetLastError() != cudaSuccess) return CP_ERR_CUDA;
  grad<<<BH * (unsigned)c.n_chunks, 256, LG::kBytes, stream>>>(q, kk, go, x, u, st, ds, g);
  return cudaGetLastError() == cudaSuccess ? CP_OK : CP_ERR_CUDA;
}

}  // namespace

size_t delta_tc_scratch(const DeltaShape& s) { return (size_t)Scratch(s).bytes(); }

cp_status_t delta_tc_bwd(const DeltaShape& s, const DeltaBwd& f, void* scratch, int* status,
                         cudaStream_t stream) {
  const Saved k(s);
  const Scratch w(s, scratch);
  const int64_t BH = s.B * s.H;
  ChainArgs c{};
  c.g = f.g; c.beta = f.beta; c.grad_state_out = f.grad_state_out;
  c.t = reinterpret_cast<const uint8_t*>(f.ckpt) + k.s_bytes + k.u_bytes;
  c.pm = c.t + k.t_bytes;
  c.xv = reinterpret_cast<float*>(w.xv_at);
  c.grad_state_in = f.grad_state_in;
  c.status = status;
  c.N = s.N; c.n_chunks = (int)k.n; c.BH = (int)BH;
  c.H = (int)s.H; c.group = (int)(s.H / s.Hk); c.D = (int)s.D; c.M = (int)s.M; c.scale = s.scale;
  GradArgs g{};
  g.g = f.g; g.beta = f.beta; g.xv = c.xv;
  g.dq = static_cast<__nv_bfloat16*>(f.dq);
  g.dk = static_cast<__nv_bfloat16*>(f.dk);
  if (w.part != 0) {
    g.dq_part = reinterpret_cast<float*>(w.part_at);
    g.dk_part = reinterpret_cast<float*>(w.part_at + w.part);
  }
  g.dg = f.dg; g.dbeta = f.dbeta; g.status = status;
  g.N = s.N; g.n_chunks = (int)k.n; g.BH = (int)BH; g.H = c.H; g.group = c.group; g.D = c.D;
  g.M = c.M; g.scale = s.scale;
  cp_status_t st = s.D <= 64 ? launch<64>(s, f, w, c, g, stream) : launch<128>(s, f, w, c, g, stream);
  if (st != CP_OK || w.part == 0) return st;
  const int64_t heads = s.B * s.Hk;
  cudaError_t e = delta_join_launch(g.dq_part, f.dq, s.N * s.D, heads, c.group, 1, s.dtype, stream);
  if (e == cudaSuccess)
    e = delta_join_launch(g.dk_part, f.dk, s.N * s.D, heads, c.group, 1, s.dtype, stream);
  return e == cudaSuccess ? CP_OK : CP_ERR_CUDA;
}

}  // namespace cp
