// Backward of the gated delta rule on the tensor cores (bf16, D <= 128), from
// what the forward kept (Saved: the states before the chunks, U, the inverse
// T = (I + A)^-1 and P).  Two launches:
//
// 1. The reverse chain, as sequential as the forward's and laid out like it: a
//    CTA per head and 32 value columns, two warpgroups of 16 columns, lane d
//    holding row d of the state's gradient dS' in registers.  A chunk is
//        K dS'                          (lanes 0-63)
//        dU = P^T dO + del K dS'         -> shared memory
//        T^T dU                         -> dX
//        [K; Q]^T [-gam b dX; s gam dO]  -> dS = gam_C dS' + it, -> shared memory
//    P^T dO of the next chunk is issued behind the last product; while that
//    one runs, dX, dV = b dX and dX . V go out.  It leaves dX and the dS' of
//    every chunk in fp32.  T, P, the states and their third parts take 152 KB, one
//    CTA to an SM.  Bound by its latency as the forward's is: B = 8, H = 16, N =
//    4096, D = M = 64, 256 CTAs, two turns of the SMs, 350 us, 4.4 TB/s; B = 4, H =
//    8, N = 1024, 64 CTAs, 41 us, 5.1k cycles a chunk.
//
// 2. The gradients, one CTA per head and chunk, all chunks at once: the chains'
//    fp32 tiles come by plain loads, a block of 32 value columns ahead, and are
//    split into operand tiles here.  Lanes 0-63 are the rows of K, 64-127 those of
//    Q:
//        [dX; dO] U^T  -> Ma (A's part), Mq (P's part), by the decays
//        [dX; dO] S^T,  U dS'^T,  [Ma; Mq] K,  Ma^T K + Mq^T Q
//        dK = -gam b dX S^T + del U dS'^T + Ma K + Ma^T K + Mq^T Q
//        dQ = s gam dO S^T + Mq K
//    and the sums for the gates (cp_delta.cu has the formulas):
//        db_i = dX_i . U_i / b_i,                        where b_i is not 0,
//             = dX_i . V_i - gam_i k_i . (S dX_i) + sum_j Ma_ij / b_i k_i.k_j
//    (Ma / b is what is at hand), with dX . V from the chain.  The first is summed
//    in fp32 where the tiles are split; the second, its value at b_i = 0 too, is a
//    difference of terms that nearly cancel when keys repeat.  Two CTAs fill an
//    SM's tensor memory (one at D > 64, and where M > 64 leaves sums to hold in
//    registers, 255 a thread and 4 bytes spilled), and a CTA is a line of stages,
//    of which whatever can runs under the products.  B = 8, H = 16, N = 4096, D = M
//    = 64: 318 us, 2.6 TB/s, 41 % of the issue slots, the tensor pipe 31 % active.
#include <algorithm>

#include "cp_delta_tc.cuh"

namespace cp {
namespace {

using namespace delta;

// ------------------------------------------------------------ reverse chain
struct ChainArgs {
  const __nv_bfloat16 *v, *go;
  const float *g, *beta, *grad_state_out;
  const uint8_t *t, *pm;        // tiles of T and P
  __nv_bfloat16* dv;
  uint8_t *ds, *dx;             // dS' and dX, fp32, as Saved's S and U
  float *xv, *grad_state_in;    // xv [M / 16 blocks][BH][N]: dX . V over the block
  int* status;
  int64_t N;
  int n_chunks, H, group, D, M;
  float scale;
};

template <int DP>
struct ChainLayout {
  static constexpr int kBoxes = DP / 64;
  static constexpr int kKQBox = 2 * kBox;
  static constexpr int kKQ = kBoxes * kKQBox;
  static constexpr int oT = 2 * kKQ;           // three parts (after two stages of K, Q)
  static constexpr int oP = oT + kTTile;       // three parts
  static constexpr int oS = oP + kTTile;       // [DP x (first | second part)]
  static constexpr int oB = oS + DP * 128;     // [128 x (first | second)]: dU, then -gam b dX; s gam dO
  static constexpr int oX = oB + 2 * kBox;     // [128 x (dS's third | B's third)]
  static constexpr int oO = oX + 2 * kBox;     // [64 x dO]
  static constexpr int oKeepS = oO + kBox;     // fp32 copies of dS' and dX on their way to memory
  static constexpr int oKeepX = oKeepS + DP * 128;
  static constexpr int oG = oKeepX + kBox;
  static constexpr int oBar = oG + 2 * (int)sizeof(GateSlot);
  static constexpr int kBytes = oBar + 128 + 1024;
  static constexpr int kPerSM = 1;
  static_assert(kPerSM * (kBytes + 1024) <= 233472, "shared memory");
};

template <int DP>
__global__ void __launch_bounds__(kChainThreads, ChainLayout<DP>::kPerSM)
    delta_tc_chain_kernel(const __grid_constant__ CUtensorMap tm_q,
                          const __grid_constant__ CUtensorMap tm_k, const ChainArgs a) {
  using L = ChainLayout<DP>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = align_tiles(smem_raw);
  GateSlot* gates = reinterpret_cast<GateSlot*>(sm + L::oG);
  uint64_t* kq_full = reinterpret_cast<uint64_t*>(sm + L::oBar);  // [2]
  uint64_t *t_full = kq_full + 2, *p_full = kq_full + 3;
  uint64_t* done = kq_full + 4;  // [3]
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(done + 3);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0);  // (uniform to the compiler)
  const int lane = threadIdx.x % 32, sub = warp / 4, t = threadIdx.x % 128;
  const int64_t p = blockIdx.x;  // b * H + h
  const int pk = (int)((p / a.H) * (a.H / a.group) + (p % a.H) / a.group);
  const int n = a.n_chunks, c0 = blockIdx.y * kCB + 16 * sub, nc = a.M - c0;  // 16 columns

  if (threadIdx.x == 0) {
    for (int i = 0; i < 7; ++i) mbar_init(kq_full + i, 1);
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
  // K dS', T^T dU and the update, one after the other (96 columns); P^T dO (32)
  const uint32_t t_acc = tmem, t_e0 = tmem + 96;
  const uint32_t T_addr = s_base + L::oT, P_addr = s_base + L::oP, S_addr = s_base + L::oS;
  const uint32_t B_addr = s_base + L::oB, S_third = s_base + L::oX, B_third = S_third + 64;
  const uint32_t O_addr = s_base + L::oO;
  uint8_t *S_tile = sm + L::oS, *B_tile = sm + L::oB, *X_tile = sm + L::oX, *O_tile = sm + L::oO;
  constexpr uint32_t id_nt96 = idesc_bf16_f32(128, 96, 0, 1);
  constexpr uint32_t id_tt32 = idesc_bf16_f32(128, 32, 1, 1);
  constexpr uint32_t id_tt96 = idesc_bf16_f32(128, 96, 1, 1);
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
    mbar_arrive_expect_tx(bar, kTTile);
    bulk_load(sm + at, src + (p * n + n - 1 - s) * (int64_t)kTTile, kTTile, bar);
  };
  auto issue_e0 = [&](int s) {  // warp 0: P^T dO of step s
    wait_or_abort(p_full, s & 1, a.status, abort_flag);
    __syncwarp();
    const uint32_t el = elect_one();
#pragma unroll 1
    for (int x = 2; x >= 0; --x)
      mma_tile<4, true, true>(el, t_e0, P_addr + x * kBox, O_addr, id_tt32, kBox, 16, 0, 0, x == 2);
  };
  // lanes 0-63: the row of V, loaded a step ahead; lanes 64-127: that of dO
  const int64_t at = p * a.N * a.M + c0;
  uint4 row[2];
  auto load_row = [&](int s) {
    const int64_t i = (int64_t)(n - 1 - s) * kCh + (t & 63);
    read16((t < 64 ? a.v : a.go) + at + i * a.M, nc, i < a.N, row);
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

  const bool row_on = t < a.D;
  float2 dS[8];
  grid_dep_wait();

  if (warp == 8) {  // the copies and the gates, a step ahead
    if (lane == 0) {
      load_kq(0);
      load_tile(L::oP, a.pm, p_full, 0);
      load_tile(L::oT, a.t, t_full, 0);
      if (n > 1) load_kq(1);
    }
    __syncwarp();
    load_gates(0);
    put_gates(0);
    __syncthreads();
    for (int s = 0; s < n; ++s) {
      __syncthreads();
      const bool more = s + 1 < n;
      wait_or_abort(done, s & 1, a.status, abort_flag);
      if (lane == 0 && more) load_tile(L::oP, a.pm, p_full, s + 1);  // P^T dO has read P
      __syncwarp();
      if (more) put_gates(s + 1);
      wait_or_abort(done + 1, s & 1, a.status, abort_flag);
      if (lane == 0 && more) load_tile(L::oT, a.t, t_full, s + 1);
      __syncwarp();
      wait_or_abort(done + 2, s & 1, a.status, abort_flag);
      if (lane == 0 && s + 2 < n) load_kq(s + 2);
      __syncwarp();
    }
  } else {
  read16(a.grad_state_out + (p * a.D + t) * a.M + c0, nc, a.grad_state_out != nullptr && row_on, dS);
  load_row(0);
  if (t >= 64) put16(O_tile, t - 64, 2 * sub, row);
  fence_proxy_async_smem();
  __syncthreads();
  if (warp == 0) issue_e0(0);
  for (int s = 0; s < n; ++s) {
    const uint32_t kq = s_base + (s & 1) * L::kKQ, phase = s & 1;
    const GateSlot* gs = gates + (s & 1);
    const int chunk = n - 1 - s;
    const int64_t tile = (p * n + chunk) * gridDim.y + blockIdx.y;
    if (t < DP) {
      store_parts(S_tile, X_tile, 0, t, sub, dS);
      put_f32(sm + L::oKeepS, t, sub, dS);
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
      wait_or_abort(kq_full + (s & 1), (s >> 1) & 1, a.status, abort_flag);
      __syncwarp();
      tc_fence_after();
      const uint32_t el = elect_one();
      mma_tile<DP / 16, false, true>(el, t_acc, kq, S_addr, id_nt96, 16, S_third - S_addr, L::kKQBox, 0,
                                     true);
      if (el) mma_commit(done);
    }
    if (threadIdx.x == 128) {
      bulk_store(a.ds + tile * (DP * 128), sm + L::oKeepS, DP * 128);
      if (s > 0) bulk_store(a.dx + (tile + gridDim.y) * kBox, sm + L::oKeepX, kBox);  // the step before's
      tma_store_commit();
    }
    float2 x[8];
    if (t >= 64) {  // s gam dO, under the product
      const float2 w = both(a.scale * gs->gam[t - 64]);
      unpack16(row, x);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = mul2(w, x[j]);
      store_parts(B_tile, X_tile, 4, t, sub, x);
      if (s + 1 < n) load_row(s + 1);
    }
    wait_or_abort(done, phase, a.status, abort_flag);
    tc_fence_after();
    if (t < 64) {
      const float2 del = both(gs->del[t]);
      float2 e0[8];
      tmem_ld16(t_e0 + lane_col, e0);
      load16_sum(t_acc + lane_col, x);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = fma2(del, x[j], e0[j]);
      store_parts(B_tile, X_tile, 4, t, sub, x);
    }
    // the copies out of dS' and dX have read them
    if (threadIdx.x == 128) tma_store_wait_read_all();
    fence_proxy_async_smem();
    tc_fence_before();
    named_barrier_sync(1, 256);
    if (warp == 0) {
      wait_or_abort(t_full, phase, a.status, abort_flag);
      __syncwarp();
      tc_fence_after();
      const uint32_t el = elect_one();
      mma_parts<false>(el, t_acc, T_addr, kBox, 16, B_addr, B_third);
      if (el) mma_commit(done + 1);
    }
    if (t >= 64 && s + 1 < n) put16(O_tile, t - 64, 2 * sub, row);  // P^T dO has read dO
    wait_or_abort(done + 1, phase, a.status, abort_flag);
    tc_fence_after();
    if (t < 64) {
      float2 r[8];
      load16_sum(t_acc + lane_col, x);
      const float2 w = both(-gs->b[t] * gs->gam[t]);
#pragma unroll
      for (int j = 0; j < 8; ++j) r[j] = mul2(w, x[j]);
      store_parts(B_tile, X_tile, 4, t, sub, r);
    }
    fence_proxy_async_smem();
    tc_fence_before();
    named_barrier_sync(1, 256);
    if (warp == 0) {
      tc_fence_after();
      const uint32_t el = elect_one();
      // [K; Q]^T: 128 rows along K; with one 64-column block the lanes past 64
      // read on into the tiles behind, and are not used
      constexpr uint32_t lbo = DP == 128 ? L::kKQBox : kBox;
      mma_tile<8, true, true>(el, t_acc, kq, B_addr, id_tt96, lbo, B_third - B_addr, 0, 0, true);
      if (el) mma_commit(done + 2);
      if (s + 1 < n) issue_e0(s + 1);
    }
    if (t < 64) {  // under the product: x is dX
      const int64_t i = (int64_t)chunk * kCh + t;
      const float2 b = both(gs->b[t]);
      float2 dot = both(0.f), v[8];
      unpack16(row, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) dot = fma2(x[j], v[j], dot);
      put_f32(sm + L::oKeepX, t, sub, x);
      uint4 dv[2];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = mul2(b, x[j]);
      pack16(v, dv);
      if (i < a.N) {
        write16(a.dv + at + i * a.M, nc, dv);
        if (nc > 0) a.xv[((int64_t)(c0 / 16) * gridDim.x + p) * a.N + i] = dot.x + dot.y;
      }
      if (s + 1 < n) load_row(s + 1);
    }
    wait_or_abort(done + 2, phase, a.status, abort_flag);
    tc_fence_after();
    const float2 last = both(gs->last.x), last_lo = both(gs->last.y);
    load16_sum(t_acc + lane_col, x);
#pragma unroll
    for (int j = 0; j < 8; ++j) dS[j] = fma2(last, dS[j], fma2(last_lo, dS[j], x[j]));
  }
  if (a.grad_state_in != nullptr && row_on)
    write16(a.grad_state_in + (p * a.D + t) * a.M + c0, nc, dS);
  }
  fence_proxy_async_smem();
  __syncthreads();
  if (threadIdx.x == 128) {  // the last step's, chunk 0
    bulk_store(a.dx + (p * n * gridDim.y + blockIdx.y) * kBox, sm + L::oKeepX, kBox);
    tma_store_commit();
    tma_store_wait_read_all();
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

// ---------------------------------------------------------------- gradients
struct GradArgs {
  const __nv_bfloat16* go;
  const float *g, *beta, *xv;
  const float4 *s, *u, *ds, *dx;   // fp32 tiles, in their 16-byte pieces
  __nv_bfloat16 *dq, *dk;
  float *dq_part, *dk_part;     // [BH][N][D] fp32, where value heads share a key head; else null
  float *dg, *dbeta;
  int* status;
  int64_t N;
  int n_chunks, BH, H, group, D, M;
  float scale;
};

// WIDE: more than 64 value columns.
template <int DP, bool WIDE>
struct GradLayout {
  static constexpr int kBoxes = DP / 64;
  static constexpr int kKQBox = 2 * kBox;
  static constexpr int kKQ = kBoxes * kKQBox;
  // a block of 32 value columns: tiles of (first | second part), the third
  // parts two to a tile; then [Ma; Mq] in three parts over the first 48 KB
  static constexpr int kRows = DP == 64 ? 64 : 128;
  static constexpr int oA = kKQ;              // [dX; dO]
  static constexpr int oA3 = oA + 2 * kBox;   // [128 x ([dX; dO]'s third | dS's)]
  static constexpr int oU3 = oA3 + 2 * kBox;  // [(U's third | S's)]
  static constexpr int oU = oU3 + kRows * 128;
  static constexpr int oS = oU + kBox;
  static constexpr int oD = oS + DP * 128;    // dS'
  static constexpr int oG = oD + DP * 128;
  static constexpr int oX = oG + (int)sizeof(GateSlot);  // sums for the gates
  static constexpr int kXFloats = 8 * 64 + 2 * 64 * 6 + 16;
  static constexpr int oBar = oX + kXFloats * 4;
  static constexpr int kBytes = oBar + 64 + 1024;
  static constexpr int kCols = DP == 64 ? 256 : 512;           // tensor memory
  static constexpr int kPerSM = DP == 64 && !WIDE ? 2 : 1;
  static_assert(oA + 6 * kBox <= oG, "[Ma; Mq]");
  static_assert(kPerSM * (kBytes + 1024) <= 233472, "shared memory");
};

// Four fp32 values, columns 4 c .. of a block's row, into its factor's parts.
__device__ __forceinline__ void put4(uint8_t* tile, uint8_t* third, int third_ch, int row, int c,
                                     float4 v) {
  uint2 a, b, d;
  split_pair3(make_float2(v.x, v.y), a.x, b.x, d.x);
  split_pair3(make_float2(v.z, v.w), a.y, b.y, d.y);
  const int at = row * 128 + 8 * (c & 1), x = row & 7, ch = c / 2;
  *reinterpret_cast<uint2*>(tile + at + ((ch ^ x) << 4)) = a;
  *reinterpret_cast<uint2*>(tile + at + (((4 + ch) ^ x) << 4)) = b;
  *reinterpret_cast<uint2*>(third + at + (((third_ch + ch) ^ x) << 4)) = d;
}

template <int DP, bool WIDE>
__global__ void __launch_bounds__(256, GradLayout<DP, WIDE>::kPerSM)
    delta_tc_grad_kernel(const __grid_constant__ CUtensorMap tm_q,
                         const __grid_constant__ CUtensorMap tm_k, const GradArgs a) {
  using L = GradLayout<DP, WIDE>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = align_tiles(smem_raw);
  GateSlot* gs = reinterpret_cast<GateSlot*>(sm + L::oG);
  float* e_sum = reinterpret_cast<float*>(sm + L::oX);  // [8 warps][64]: pairs' part of dg
  float* dots = e_sum + 512;     // [2 column halves][6][64]: rows' sums, as written below
  float* z_sum = dots + 768;     // [8]
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::oBar);
  uint64_t *kq_full = bars, *done = bars + 1;  // done [2]
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + 3);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0);  // (uniform to the compiler)
  const int lane = threadIdx.x % 32, wg = warp / 4, t = threadIdx.x % 128;
  const bool issuer = threadIdx.x == 0;
  const int64_t p = blockIdx.x / a.n_chunks;
  const int chunk = blockIdx.x % a.n_chunks, i0 = chunk * kCh;
  const int pk = (int)((p / a.H) * (a.H / a.group) + (p % a.H) / a.group);
  const int blocks = (a.M + kCB - 1) / kCB;

  const uint64_t keep = policy_evict_first();
  const int64_t tile0 = (p * a.n_chunks + chunk) * blocks;
  // What comes by plain loads sets out first, beside the copies, and then a
  // block ahead under the products: a thread's 16-byte pieces of the block's fp32
  // tiles, of dO eight columns of a row, and the gates of one warp's rows.
  constexpr int kUP = 64 * 8 / 256, kSP = DP * 8 / 256;  // pieces of a 64-row tile, of a state
  float4 xu[kUP], xx[kUP], xs[kSP], xd[kSP];
  uint4 dov;
  const int do_row = threadIdx.x / 4, do_ch = threadIdx.x % 4;
  auto load_block = [&](int m) {
    const int64_t u = (tile0 + m) * (64 * 8) + threadIdx.x, s = (tile0 + m) * (DP * 8) + threadIdx.x;
#pragma unroll
    for (int e = 0; e < kUP; ++e) {
      xx[e] = __ldcs(a.dx + u + 256 * e);
      xu[e] = __ldcs(a.u + u + 256 * e);
    }
#pragma unroll
    for (int e = 0; e < kSP; ++e) {
      xs[e] = __ldcs(a.s + s + 256 * e);
      xd[e] = __ldcs(a.ds + s + 256 * e);
    }
    const int col = kCB * m + 8 * do_ch;
    dov = i0 + do_row < a.N && col < a.M
              ? *reinterpret_cast<const uint4*>(a.go + (p * a.N + i0 + do_row) * a.M + col)
              : make_uint4(0, 0, 0, 0);
  };
  grid_dep_wait();
  if (issuer) {
    for (int i = 0; i < 3; ++i) mbar_init(bars + i, 1);
    *abort_flag = 0;
    fence_mbar_init();
    mbar_arrive_expect_tx(kq_full, L::kKQ);
    for (int x = 0; x < L::kBoxes; ++x) {
      tma_load_3d(sm + x * L::kKQBox, &tm_k, kq_full, 64 * x, i0, pk, keep);
      tma_load_3d(sm + x * L::kKQBox + kBox, &tm_q, kq_full, 64 * x, i0, pk, keep);
    }
  }
  if (warp == 0) {
    __syncwarp();
    tmem_alloc(tmem_holder, L::kCols);
    tmem_relinquish();
  }
  float4 gb = make_float4(0.f, 0.f, 0.f, 0.f);
  if (warp == 1) {
    const int64_t i = i0 + lane, at = p * a.N;
    gb = make_float4(i < a.N ? a.g[at + i] : 0.f, i + 32 < a.N ? a.g[at + i + 32] : 0.f,
                     i < a.N ? a.beta[at + i] : 0.f, i + 32 < a.N ? a.beta[at + i + 32] : 0.f);
  }
  load_block(0);
  {  // dO has no second and third part
    const uint4 zero = make_uint4(0, 0, 0, 0);
    const int at = (64 + do_row) * 128, x = do_row & 7;
    *reinterpret_cast<uint4*>(sm + L::oA + at + (((4 + do_ch) ^ x) << 4)) = zero;
    *reinterpret_cast<uint4*>(sm + L::oA3 + at + ((do_ch ^ x) << 4)) = zero;
  }
  for (int i = threadIdx.x; i < 512; i += 256) e_sum[i] = 0.f;
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_holder, 0), s_base = smem_u32(sm);
  const uint32_t t_kk = tmem, t_p2 = tmem + 64, t_in = tmem + 128, t_u = t_in + DP;
  const uint32_t lane_base = (uint32_t)(warp % 4) << 21;
  const uint32_t A_addr = s_base + L::oA;
  constexpr uint32_t id_nn64 = idesc_bf16_f32(128, 64, 0, 0);
  constexpr uint32_t id_nnD = idesc_bf16_f32(128, DP, 0, 0);
  constexpr uint32_t id_ntD = idesc_bf16_f32(128, DP, 0, 1);
  constexpr uint32_t id_ttD = idesc_bf16_f32(128, DP, 1, 1);
  if (warp == 0) {
    wait_or_abort(kq_full, 0, a.status, abort_flag);
    __syncwarp();
    mma_tile<DP / 16, false, false>(elect_one(), t_kk, s_base, s_base, id_nn64, 16, 16, L::kKQBox, L::kKQBox, true);
  }
  float z = 0.f;           // <S, dS'>, this thread's share
  float own[kUP] = {};     // dX . U of the thread's rows
  // lanes 0-63 ("K rows"): i = t; lanes 64-127 ("Q rows"): i = t - 64
  const bool is_k = t < 64;
  const int i = t & 63, row32 = i / 32;
  // The products with the states and the pairs are read out every two blocks, and
  // summed here: an MMA rounds its sum toward zero, and six a step of 16 columns,
  // all into one accumulator, would leave 1.6e-6 of dg at 200 columns.
  constexpr int HC = DP / 2;  // a half of D's columns a thread
  float2 g2[HC / 2], din = both(0.f), du = both(0.f), p2[2][8];
  if (WIDE) {
#pragma unroll
    for (int e = 0; e < HC / 2; ++e) g2[e] = both(0.f);
#pragma unroll
    for (int e = 0; e < 16; ++e) p2[e / 8][e % 8] = both(0.f);
  }
  const auto read_states = [&]() {
    const float w = is_k ? -gs->gam[i] * gs->b[i] : a.scale * gs->gam[i], del = gs->del[i];
#pragma unroll
    for (int h = 0; h < HC / 16; ++h) {
      const int c = wg * HC + 16 * h;
      uint32_t r[16], u[16];
      tmem_ld16(t_in + lane_base + c, r);
      tmem_ld16(t_u + lane_base + c, u);
      tmem_ld_wait();
      const uint8_t* src = sm + (c / 64) * L::kKQBox + t * 128;  // the row of k or q
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
          g2[8 * h + k / 2] = WIDE ? add2(g2[8 * h + k / 2], o) : o;
        }
      }
    }
  };
  for (int m = 0; m < blocks; ++m) {
    if (m > 0) wait_or_abort(done, (m - 1) & 1, a.status, abort_flag);  // the tiles have been read
    if (WIDE && m > 0 && m % 2 == 0) {
      tc_fence_after();
      read_states();
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float2 r[8];
        tmem_ld16(t_p2 + lane_base + 16 * (2 * wg + h), r);
#pragma unroll
        for (int e = 0; e < 8; ++e) p2[h][e] = add2(p2[h][e], r[e]);
      }
    }
#pragma unroll
    for (int e = 0; e < kUP; ++e) {
      const int i = threadIdx.x + 256 * e, row = i / 8, c = (i % 8) ^ (row & 7);
      put4(sm + L::oA, sm + L::oA3, 0, row, c, xx[e]);
      put4(sm + L::oU, sm + L::oU3, 0, row, c, xu[e]);
      own[e] = fmaf(xx[e].x, xu[e].x, own[e]);
      own[e] = fmaf(xx[e].y, xu[e].y, own[e]);
      own[e] = fmaf(xx[e].z, xu[e].z, own[e]);
      own[e] = fmaf(xx[e].w, xu[e].w, own[e]);
    }
#pragma unroll
    for (int e = 0; e < kSP; ++e) {
      const int i = threadIdx.x + 256 * e, row = i / 8, c = (i % 8) ^ (row & 7);
      put4(sm + L::oS, sm + L::oU3, 4, row, c, xs[e]);
      put4(sm + L::oD, sm + L::oA3, 4, row, c, xd[e]);
      z = fmaf(xs[e].x, xd[e].x, z);
      z = fmaf(xs[e].y, xd[e].y, z);
      z = fmaf(xs[e].z, xd[e].z, z);
      z = fmaf(xs[e].w, xd[e].w, z);
    }
    *reinterpret_cast<uint4*>(sm + L::oA + (64 + do_row) * 128 + ((do_ch ^ (do_row & 7)) << 4)) = dov;
    tc_fence_before();
    fence_proxy_async_smem();
    __syncthreads();
    if (warp == 0) {
      tc_fence_after();
      const uint32_t el = elect_one();
      // part x of a factor: 64 bytes on for the second, another tile for the third
      const auto part = [&](uint32_t first, uint32_t third, int x) {
        return x == 2 ? third : first + 64 * x;
      };
#pragma unroll 1
      for (int x = 2; x >= 0; --x)
#pragma unroll 1
        for (int y = x; y >= 0; --y) {
          const bool fresh = m % 2 == 0 && x == 2 && y == 2;
          const uint32_t dx = part(A_addr, s_base + L::oA3, y), u = part(s_base + L::oU, s_base + L::oU3, y);
          mma_tile<2, false, false>(el, t_p2, dx, part(s_base + L::oU, s_base + L::oU3, x - y), id_nn64, 16,
                                    16, 0, 0, fresh);
          mma_tile<2, false, false>(el, t_in, dx, part(s_base + L::oS, s_base + L::oU3 + 64, x - y), id_nnD,
                                    16, 16, 0, 0, fresh);
          // lanes past 64 read on behind U and are not used
          mma_tile<2, false, false>(el, t_u, u, part(s_base + L::oD, s_base + L::oA3 + 64, x - y), id_nnD, 16,
                                    16, 0, 0, fresh);
        }
      if (el) mma_commit(done);
    }
    if (m + 1 < blocks) load_block(m + 1);
    if (warp == 1 && m == 0) write_gates(gs, lane, gb.x, gb.y, gb.z, gb.w);
    if (warp >= 6 && m == 0) {  // dX . V of the rows, from the chain's blocks
      const int i = threadIdx.x - 192;
      float d = 0.f;
      if (i0 + i < a.N)
#pragma unroll 4
        for (int x = 0; x < (a.M + 15) / 16; ++x) d += a.xv[((int64_t)x * a.BH + p) * a.N + i0 + i];
      dots[640 + i] = d;
    }
  }
  wait_or_abort(done, (blocks - 1) & 1, a.status, abort_flag);
  tc_fence_after();
  for (int o = 16; o > 0; o /= 2) z += __shfl_xor_sync(0xffffffffu, z, o);
  if (lane == 0) z_sum[warp] = z;
#pragma unroll
  for (int e = 0; e < kUP; ++e) {  // a row's eight pieces lie side by side
    for (int o = 4; o > 0; o /= 2) own[e] += __shfl_xor_sync(0xffffffffu, own[e], o);
    if (lane % 8 == 0) dots[256 + threadIdx.x / 8 + 32 * e] = own[e];
  }
  __syncthreads();  // the gates
  const float bt = gs->b[i];
  read_states();
  {
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
  float part[32];    // columns 32 wg ..: the pair's weight in dg, then its running sum
  float db = 0.f;
  const int last = is_k ? i - 1 : i;
  const float wm = is_k ? bt : 1.f;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int c = 2 * wg + h;
    uint32_t r[16], kk[16];
    tmem_ld16(t_p2 + lane_base + 16 * c, r);
    tmem_ld16(t_kk + lane_base + 16 * c, kk);
    float2 v[8];
    decays16(gs, i, row32, c, last, is_k ? -1.f : a.scale, v);
    tmem_ld_wait();
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float2 m = make_float2(__uint_as_float(r[2 * e]), __uint_as_float(r[2 * e + 1]));
      if (WIDE) m = add2(m, p2[h][e]);
      // masked places stay 0 whatever the accumulators hold
      m = mul2(v[e], m);
      const int j = 16 * c + 2 * e;
      if (j > last) m.x = 0.f;
      if (j + 1 > last) m.y = 0.f;
      float2 x = mul2(m, make_float2(__uint_as_float(kk[2 * e]), __uint_as_float(kk[2 * e + 1])));
      if (j > last) x.x = 0.f;
      if (j + 1 > last) x.y = 0.f;
      db += x.x + x.y;
      v[e] = mul2(both(wm), m);
      x = mul2(both(wm), x);
      part[16 * h + 2 * e] = x.x;
      part[16 * h + 2 * e + 1] = x.y;
    }
    store16_split(sm + L::oA, 2 * kBox, t, 2 * c, v);
  }
  tc_fence_before();
  fence_proxy_async_smem();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    const uint32_t el = elect_one();
#pragma unroll 1
    for (int x = 2; x >= 0; --x) {  // the tile's parts
      const uint32_t ap = A_addr + x * 2 * kBox;
      // [Ma; Mq] K
      mma_tile<4, false, true>(el, t_in, ap, s_base, id_ntD, 16, L::kKQBox, 0, 0, x == 2);
      // Ma^T K + Mq^T Q; lanes past 64 read on and are not used
      mma_tile<8, true, true>(el, t_u, ap, s_base, id_ttD, kBox, L::kKQBox, 0, 0, x == 2);
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
  }
  __syncthreads();
  if (warp >= 6) {
    // the gates' gradients, a warp to a half of the rows: lane l has row l of it
    const int h = warp - 6, j = lane + 32 * h, far = lane + 32 * (1 - h);
    const float zt = gs->gam[kCh - 1] * (((z_sum[0] + z_sum[1]) + (z_sum[2] + z_sum[3])) +
                                         ((z_sum[4] + z_sum[5]) + (z_sum[6] + z_sum[7])));
    const auto kx = [&](int x) { return dots[x] + dots[384 + x]; };
    const auto with_s = [&](int x) {   // row x's part with S
      return gs->gam[x] * (a.scale * (dots[64 + x] + dots[448 + x]) - gs->b[x] * kx(x));
    };
    const auto with_ds = [&](int x) {  // and with dS'
      return gs->del[x] * (dots[128 + x] + dots[512 + x]);
    };
    // sums of the first from the row on, of the second before it; the other
    // half gives one of them whole
    float r = with_s(j), c = with_ds(j), rest = h ? with_ds(far) : with_s(far);
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const float x = __shfl_down_sync(0xffffffffu, r, o), y = __shfl_up_sync(0xffffffffu, c, o);
      rest += __shfl_xor_sync(0xffffffffu, rest, o);
      if (lane + o < 32) r += x;
      if (lane >= o) c += y;
    }
    c = __shfl_up_sync(0xffffffffu, c, 1);
    if (lane == 0) c = 0.f;
    float pairs = 0.f;
#pragma unroll
    for (int x = 0; x < 8; ++x) pairs += e_sum[x * 64 + j];
    if (i0 + j < a.N) {
      const int64_t at = p * a.N + i0 + j;
      a.dg[at] = zt + r + c + rest + pairs;
      const float d = dots[192 + j] + dots[576 + j] + dots[640 + j] - gs->gam[j] * kx(j);
      // U carries b as a factor, far above the smallest number down to 2^-80
      const float b = gs->b[j];
      a.dbeta[at] = fabsf(b) < 0x1p-80f ? d : dots[256 + j] / b;
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
      // over k and q, which the last products have read
      uint4 w[2];
      pack16(o, w);
      put16(sm + (c / 64) * L::kKQBox, t, (c % 64) / 8, w);
    }
  }
  if (a.dq_part == nullptr) {
    // the warp's 32 rows, its half of the columns, in whole sectors
    __syncwarp();
    constexpr int kPieces = HC / 8;
#pragma unroll
    for (int x = 0; x < kPieces; ++x) {
      const int row = 32 * (warp % 4) + (32 * x + lane) / kPieces;
      const int col = wg * HC + 8 * (lane % kPieces);
      const uint4 w = *reinterpret_cast<const uint4*>(
          sm + (col / 64) * L::kKQBox + row * 128 + (((col % 64) / 8 ^ (row & 7)) << 4));
      const int64_t at = p * a.N + i0 + (row & 63);
      if (i0 + (row & 63) < a.N && col < a.D)
        *reinterpret_cast<uint4*>((row < 64 ? a.dk : a.dq) + at * a.D + col) = w;
    }
  }
  if (*abort_flag) linger();
  tc_fence_before();
  __syncthreads();
  grid_dep_launch_dependents();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, L::kCols);
  }
}

// What the chain leaves for the gradients.
struct Scratch {
  int64_t ds, dx, xv, part;  // bytes; dS' and dX in tiles
  uint8_t *ds_at, *dx_at, *xv_at, *part_at;
  explicit Scratch(const DeltaShape& s, void* at = nullptr) {
    auto up = [](int64_t x) { return (x + 255) / 256 * 256; };
    const int64_t BH = s.B * s.H;
    const Saved k(s);
    ds = k.s_bytes;
    dx = k.u_bytes;
    xv = up(4 * ((s.M + 15) / 16) * BH * s.N);
    part = s.H == s.Hk ? 0 : up(4 * BH * s.N * s.D);
    ds_at = static_cast<uint8_t*>(at);
    dx_at = ds_at + ds;
    xv_at = dx_at + dx;
    part_at = xv_at + xv;
  }
  int64_t bytes() const { return ds + dx + xv + 2 * part; }
};

template <int DP, bool WIDE>
cp_status_t launch(const DeltaShape& s, const DeltaBwd& f, const ChainArgs& c, const GradArgs& g,
                   cudaStream_t stream) {
  using LC = ChainLayout<DP>;
  using LG = GradLayout<DP, WIDE>;
  auto chain = delta_tc_chain_kernel<DP>;
  auto grad = delta_tc_grad_kernel<DP, WIDE>;
  if (cudaFuncSetAttribute(chain, cudaFuncAttributeMaxDynamicSharedMemorySize, LC::kBytes) != cudaSuccess ||
      cudaFuncSetAttribute(grad, cudaFuncAttributeMaxDynamicSharedMemorySize, LG::kBytes) != cudaSuccess)
    return CP_ERR_CUDA;
  // (encoding a map needs the device's context current in this thread: the
  // calls above see to that)
  CUtensorMap q, kk;
  if (!make_chunk_map(&q, f.q, s.B * s.Hk, s.N, s.D) || !make_chunk_map(&kk, f.k, s.B * s.Hk, s.N, s.D))
    return CP_ERR_CUDA;
  const unsigned BH = (unsigned)(s.B * s.H);
  const dim3 grid(BH, (unsigned)((s.M + kCB - 1) / kCB));
  if (launch_dependent(chain, grid, kChainThreads, LC::kBytes, stream, q, kk, c) != cudaSuccess ||
      launch_dependent(grad, dim3(BH * (unsigned)c.n_chunks), 256, LG::kBytes, stream, q, kk, g) != cudaSuccess)
    return CP_ERR_CUDA;
  return CP_OK;
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
  c.v = static_cast<const __nv_bfloat16*>(f.v);
  c.go = static_cast<const __nv_bfloat16*>(f.grad_out);
  c.dv = static_cast<__nv_bfloat16*>(f.dv);
  c.ds = w.ds_at;
  c.dx = w.dx_at;
  c.xv = reinterpret_cast<float*>(w.xv_at);
  c.grad_state_in = f.grad_state_in;
  c.status = status;
  c.N = s.N; c.n_chunks = (int)k.n;
  c.H = (int)s.H; c.group = (int)(s.H / s.Hk); c.D = (int)s.D; c.M = (int)s.M; c.scale = s.scale;
  GradArgs g{};
  g.go = c.go; g.g = f.g; g.beta = f.beta; g.xv = c.xv;
  g.s = reinterpret_cast<const float4*>(f.ckpt);
  g.u = g.s + k.s_bytes / 16;
  g.ds = reinterpret_cast<const float4*>(w.ds_at);
  g.dx = reinterpret_cast<const float4*>(w.dx_at);
  if (w.part != 0) {
    g.dq_part = reinterpret_cast<float*>(w.part_at);
    g.dk_part = reinterpret_cast<float*>(w.part_at + w.part);
  }
  g.dq = static_cast<__nv_bfloat16*>(f.dq); g.dk = static_cast<__nv_bfloat16*>(f.dk);
  g.dg = f.dg; g.dbeta = f.dbeta; g.status = status;
  g.N = s.N; g.n_chunks = (int)k.n; g.BH = (int)BH; g.H = c.H; g.group = c.group; g.D = c.D;
  g.M = c.M; g.scale = s.scale;
  cp_status_t st = s.D <= 64 ? (s.M <= 64 ? launch<64, false> : launch<64, true>)(s, f, c, g, stream)
                             : (s.M <= 64 ? launch<128, false> : launch<128, true>)(s, f, c, g, stream);
  if (st != CP_OK || w.part == 0) return st;
  const cudaError_t e = delta_join_launch({g.dq_part, g.dk_part, nullptr, nullptr, f.dq, f.dk, nullptr,
                                           nullptr, s.N, s.D, s.B * s.Hk, c.group, 1},
                                          s.dtype, stream);
  return e == cudaSuccess ? CP_OK : CP_ERR_CUDA;
}

}  // namespace cp
