// Linear attention with a decay for each head on the 5th-generation tensor cores
// (bf16, D and M at most 128; formulas in cp_decay.cuh).
//
// Forward, and each of the backward's dq, dv and dk, is one product of three row
// arrays a, b, c with a state (DA x DC), walked in tiles of 128 rows, forward or
// in reverse.  With S the fp32 state before tile t and w_ij = e^{g |i - j|}:
//     P   = w o A_t B_t^T           masked to the tile's causal triangle
//     C'  = (e^{g (127 - r)} c_r)   the tile's rows as the state takes them
//     O_t = P C_t + (e^{g (r + 1)}) o (A_t S)
//     S   = e^{128 g} S + B_t^T C'
// Nothing in a tile but A S waits for the state, and the state's update is one
// fma, so the tiles stream through a pipeline of warps:
//   warp 0        TMA producer: A, B and C tiles into a ring each, whichever has room
//   warps 1..3    MMA issuers: B^T C'; A B^T and A S; P C
//   warps 4..7    state group: fp32 S in registers (thread = row); its copy as three
//                 bf16 numbers, the operand of A S
//   warps 8..15   P groups: P times its powers, masked, hi + lo, back into TMEM
//   warps 16..19  O group: O from its two accumulators, to bf16, TMA store
//   warps 20..27  C' groups: a row times its power, as three bf16 numbers
// A CTA walks one piece of one head's sequence for 64 columns of c.
//
// Precision.  S lives in registers in fp32 and takes each tile's B^T C' by an fma
// that rounds to nearest, its decay as hi + lo: an accumulator kept in tensor
// memory would be rounded toward zero at every MMA and lose 1e-5 of a state that
// remembers thousands of rows.  C' and the copy of S enter their products as three bf16
// numbers, all 24 bits, whether or not a state is asked for, so that asking changes no
// other result.  P has two (17 bits): its rounding, 2e-6 of a score, is a thousandth
// of a bf16 result's own, 2^-9, and moves one result in a thousand or two to the next
// bf16 number.  A third part of P would need 64 columns more of a tensor memory that is
// full, a second accumulator for B^T C' given up for them: 96 against 66 us (B=8 H=16
// N=4096 D=M=64), with the results 4.8e-5 from the rounded 64-bit ones instead of 5.4e-5
// (two parts of everything: 1.1e-4).  A call of one tile, whose results are P's alone
// but for a carried state's part, has a buffer of P free for its third parts: 6e-5 and
// less with three, 1e-4 with two, 43 against 40 us for B=64 H=16 N=128 D=M=64, and 17
// either way, the call's, for B=8.
//
// Powers come from a table of e^{g n}, n <= 128, of products in shared memory: a
// 32-column chunk of P left of the diagonal one has w_ij = e^{g (i - j0 - 31)}
// e^{g (31 - (j - j0))}, two numbers at most 1, one per row and one per column.
//
// No memory or matrix rate bounds it: when every factor had two parts, leaving out any
// one of the products, or of the groups' stores, gave at most 4 %, the P groups' work
// 10 %.  The roles share four schedulers, and a tile takes about 3,400 cycles with
// 64-wide A (1,900 of them the tensor core's, for the bf16 parts) and 4,900 with 128,
// where C's two boxes, which wait for O, hold up the next.  Forward: B=8 H=16 N=4096
// D=M=64 66 us, 61 % of the copy rate on 128 SMs; B=2 H=8 N=32768 D=M=128 231; forward
// and backward of the first 245 to 252.  O straight from the registers, 32 bytes of a row to a
// store, frees C sooner: 215 against 220 us for the second as it was then, but 232
// against 224 for the last.
//
// Sequences of few heads are cut into pieces: the same kernel with the output
// left out (AGG) sums each piece's B^T C', a prefix launch turns the sums into
// the states the pieces start from, and the pieces run side by side.
#include <algorithm>
#include <atomic>

#include "cp_decay.cuh"
#include "cp_delta_tc.cuh"

namespace cp {
namespace {

using namespace decay;
using namespace cp::ptx;
using tc::kBoxBytes;
using tc::kSmemLimit;
using tc::kTile;
using tc::record_timeout;
using tc::sw128_offset;

constexpr int kMB = 64;   // columns of c to a CTA
constexpr int kBarBytes = 768, kTableBytes = 1280;
constexpr int kNP = 2;    // buffers of P
constexpr uint32_t kHi = desc_hi(1024);

// What the products of a launch share, and what is each one's own.
struct Common {
  const float* g;
  const int* lengths;
  int* status;
  int64_t N;
  int H, Hk, group, BH, n_mb, n_tiles, seg_tiles, G;
  int sub, sub_tiles;      // parts of a piece in the summing launch, and their tiles
  int products;
};
struct Own {
  const float* state_in;   // may be null (zero)
  float* state_out;        // may be null
  float* slots;            // [problems][G][sub][DP][64]: sums, then the pieces' first states
  float* out_f32;          // not null: the result goes here in fp32, [BH][N][DC]
  int64_t st_r, st_c;      // strides of a state's rows and columns
  int DA, DC;
  int a_key, b_key, c_key, o_key;   // whether an array has key heads
  int reverse;
  float s_p, s_o, s_c;     // factors of P, of A S and of C'
};
template <int MAX>
struct Set {
  Common all;
  Own own[MAX];
};
template <int MAX>
struct Maps {
  CUtensorMap a[MAX], b[MAX], c[MAX], o[MAX];
};

// The bf16 numbers that an element of C', and of the copy of S, enters its products as:
// all of its 24 bits.
constexpr int kParts = 3;

template <int DP, bool AGG>
struct Layout {
  static constexpr int kABoxes = DP / 64;
  static constexpr int kBStage = kABoxes * kBoxBytes;
  static constexpr int kSOne = DP * 128;                       // a bf16 copy of the state
  static constexpr int kSBytes = AGG ? 0 : kParts * kSOne;
  // C' goes a few rows at a time through NV buffers: with 128-wide A the copies of S
  // leave room for two of 16 rows
  static constexpr int kVRows = !AGG && DP == 128 ? 16 : 32;
  static constexpr int kVOne = kVRows * 128;                   // a part of them
  static constexpr int NV = AGG || DP == 128 ? 2 : 4;
  static constexpr int kPieces = kTile / kVRows;               // to a tile
  static constexpr int kVBytes = NV * kParts * kVOne;
  static constexpr int kRoom = kSmemLimit - 1024 - kBarBytes - kTableBytes;
  static constexpr int NB = AGG && DP == 128 ? 1 : 2;          // stages of the B ring
  // tiles of A, which wait for the state, and of C, whose boxes take O: what is left.
  // In one ring, C before A, a 128-wide A waited for the O two tiles back: 235 against
  // 220 us (B=2 H=8 N=32768 D=M=128, with two parts to every factor)
  static constexpr int RA = AGG ? 0 : DP == 128 ? 2 : 3;
  static constexpr int RC = AGG ? 3 : (kRoom - (NB + RA) * kBStage - kSBytes - kVBytes) / kBoxBytes;
  static constexpr int kBoxes = (NB + RA) * kABoxes + RC;
  static constexpr int kSmem =
      kBoxes * kBoxBytes + kSBytes + kVBytes + kBarBytes + kTableBytes + 1024;
  static constexpr int kVGroup = AGG ? 8 : 20;                 // first warp of the C' groups
  static constexpr int kThreads = 32 * (kVGroup + 8);
  static constexpr int SC = DP / 2;                            // columns of S to a thread
  // tensor memory: P, A S, P C, and B^T C' as [first part | rest]
  static constexpr int kColO1 = kNP * 128, kColO2 = kColO1 + kMB;
  static constexpr int kColS = AGG ? 0 : kColO2 + kMB;
  static constexpr int kCols = AGG ? 128 : 512;
  static_assert(RC >= 2, "a tile does not fit");
  static_assert((2 * NB + 2 * RA + 3 * RC + 34) * 8 <= kBarBytes, "barriers");
  static_assert(kSmem <= kSmemLimit && kColS + 128 <= kCols, "no room");
};

// hi = bf16(x), and x - hi: the differences by mixed fma, whose bf16 operand needs
// no widening (shifts and masks go to the pipe that has the least to spare here:
// 19 cycles a pair and scheduler with them in three parts, 16 without)
__device__ __forceinline__ uint32_t split_hi(float2& x) {
  const uint32_t h = tc::pack_bf16x2(x.x, x.y);
  asm("{\n\t.reg .b16 a, b, m;\n\tmov.b32 {a, b}, %2;\n\tmov.b16 m, 0xBF80;\n\t"
      "fma.rn.f32.bf16 %0, a, m, %3;\n\tfma.rn.f32.bf16 %1, b, m, %4;\n\t}"
      : "=f"(x.x), "=f"(x.y)
      : "r"(h), "f"(x.x), "f"(x.y));
  return h;
}
// two bf16 numbers as fp32
__device__ __forceinline__ float2 widen(uint32_t h) {
  float2 r;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
      "add.rn.f32.bf16 %0, a, %3;\n\tadd.rn.f32.bf16 %1, b, %3;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "r"(h), "f"(0.f));
  return r;
}

// Twenty-eight warps walk eight different pieces of code, so what stalls them first is
// the instruction cache: loops stay rolled, and a wait is a few instructions, its
// limit a count (a try takes tens of nanoseconds to a microsecond, so a third of a
// second at least) and not a clock's.  A warp's lanes wait together and agree, so that
// the code behind a wait is uniform: its addresses and descriptors stay in uniform
// registers, where one lane alone in a branch moves each there first (forward and
// backward of B=8 H=16 N=4096 D=M=64: 249 us with the issuers and the producer as
// single lanes, 219 so, when every factor had two parts).
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  uint32_t tries = 0;
  bool there = true;
  while (!mbar_try_wait(bar, parity))
    if (*abort_flag != 0 || ++tries > (1u << 24)) {
      there = false;
      break;
    }
  return __all_sync(~0u, there);
}
__device__ __forceinline__ bool test(uint64_t* bar, uint32_t parity) {
  return __all_sync(~0u, mbar_test_wait(bar, parity));
}

template <int REGS>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS));
}
template <int REGS>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS));
}

// MAX: products that share a launch, at most (their CTAs in turn, so that those of
// one head, which read the same rows, run side by side).  ONE: a sequence is one tile,
// and P has three parts
template <int DP, bool AGG, bool ONE, int MAX>
__global__ void __launch_bounds__(Layout<DP, AGG>::kThreads, AGG ? 2 : 1)
    decay_tc_kernel(const __grid_constant__ Maps<MAX> maps, const __grid_constant__ Set<MAX> set) {
  using L = Layout<DP, AGG>;
  constexpr int NB = L::NB, RA = L::RA, RC = L::RC;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align_tiles(smem_raw);
  uint8_t* b_ring = smem;                            // [NB] B tiles
  uint8_t* a_ring = b_ring + NB * L::kBStage;        // [RA] A tiles
  uint8_t* ring = a_ring + RA * L::kBStage;          // [RC] C boxes
  uint8_t* vp = ring + RC * kBoxBytes;               // [NV][kParts] a piece's rows of C'
  uint8_t* s_tile = vp + L::kVBytes;                 // [kParts] the copy of S
  uint64_t* full_b = reinterpret_cast<uint64_t*>(s_tile + L::kSBytes);
  uint64_t* empty_b = full_b + NB;
  uint64_t* full_a = empty_b + NB;     // [RA]
  uint64_t* empty_a = full_a + RA;     // [RA]
  uint64_t* full_c = empty_a + RA;     // [RC]
  uint64_t* empty_c = full_c + RC;     // [RC]
  uint64_t* c_read = empty_c + RC;     // [RC] read by the C' groups
  uint64_t* p_done = c_read + RC;      // [kNP] A B^T in TMEM
  uint64_t* p_ready = p_done + kNP;    // [kNP] P packed
  uint64_t* pc_done = p_ready + kNP;   // [kNP] P C done: the buffer is free
  uint64_t* s_ready = pc_done + kNP;   // copy of S written
  uint64_t* as_done = s_ready + 1;     // A S done: the copy is free
  uint64_t* o1_done = as_done + 1;     // A S
  uint64_t* o2_done = o1_done + 1;     // P C
  uint64_t* o1_free = o2_done + 1;     // read
  uint64_t* o2_free = o1_free + 1;
  uint64_t* vp_ready = o2_free + 1;    // [4] a piece of C' written
  uint64_t* vp_free = vp_ready + 4;    // [4] their products done
  uint64_t* kv_done = vp_free + 4;     // B^T C' in TMEM
  uint64_t* kv_free = kv_done + 1;     // B^T C' read
  uint64_t* fixed = kv_free + 1;       // rows past the sequence's end cleared
  uint64_t* fin = fixed + 1;           // [3]
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(fin + 3);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(fin + 4);
  float* pw = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(full_b) + kBarBytes);  // [129]
  float* cf = pw + 132;                // [32] a chunk's column powers

  // (a shuffle's result is the warp's own)
  const int warp = __shfl_sync(~0u, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const Common& a = set.all;
  const int which = MAX == 1 ? 0 : blockIdx.x % a.products;
  const Own& own = set.own[which];
  const CUtensorMap &tm_a = maps.a[which], &tm_b = maps.b[which], &tm_c = maps.c[which],
                    &tm_o = maps.o[which];
  int idx = MAX == 1 ? blockIdx.x : blockIdx.x / a.products;
  const int mb = idx % a.n_mb;
  idx /= a.n_mb;
  const int bh = idx % a.BH;
  int seg = idx / a.BH, part = 0;
  if (AGG) {
    part = seg % a.sub;
    seg = seg / a.sub + (own.reverse ? 1 : 0);  // (nothing follows the last in scan order)
  }
  const int b = bh / a.H, h = bh % a.H;
  const bool rev = own.reverse != 0;
  const float s_p = own.s_p, s_o = own.s_o, s_c = own.s_c;
  float* const out_f32 = own.out_f32;

  if (threadIdx.x == 0) {
    for (int i = 0; i < NB; ++i) {
      mbar_init(&full_b[i], 1);
      mbar_init(&empty_b[i], AGG ? 1 : 2);
    }
    for (int i = 0; i < RA; ++i) {
      mbar_init(&full_a[i], 1);
      mbar_init(&empty_a[i], 2);         // A B^T, A S
    }
    for (int i = 0; i < RC; ++i) {
      mbar_init(&full_c[i], 1);
      mbar_init(&empty_c[i], AGG ? 8 : 4);  // the C' warps; the O warps
      mbar_init(&c_read[i], 8);
    }
    for (int i = 0; i < kNP; ++i) {
      mbar_init(&p_done[i], 1);
      mbar_init(&p_ready[i], 8);
      mbar_init(&pc_done[i], 1);
    }
    mbar_init(s_ready, 4);
    mbar_init(as_done, 1);
    mbar_init(o1_done, 1);
    mbar_init(o2_done, 1);
    mbar_init(o1_free, 4);
    mbar_init(o2_free, 4);
    for (int i = 0; i < 4; ++i) {
      mbar_init(&vp_ready[i], 4);
      mbar_init(&vp_free[i], 1);
    }
    mbar_init(kv_done, 1);
    mbar_init(kv_free, 4);
    mbar_init(fixed, 4);
    for (int i = 0; i < 3; ++i) mbar_init(&fin[i], 1);
    *abort_flag = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
    tma_prefetch_desc(&tm_b);
    tma_prefetch_desc(&tm_c);
    if (!AGG) {
      tma_prefetch_desc(&tm_a);
      tma_prefetch_desc(&tm_o);
    }
  }
  if (warp == 1) {
    tmem_alloc(tmem_holder, L::kCols);
    tmem_relinquish();
  }
  grid_dep_wait();  // what the kernel before this one wrote is visible from here
  const float g = head_decay(a.g[h]);
  if (threadIdx.x <= kTile) pw[threadIdx.x] = power(g, threadIdx.x);
  if (threadIdx.x >= 160 && threadIdx.x < 192) {
    const int c = threadIdx.x - 160;
    cf[c] = power(g, rev ? c : 31 - c);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(~0u, *tmem_holder, 0);
  const int wq = warp & 3, row = wq * 32 + lane;
  const uint32_t lane_base = tmem + (static_cast<uint32_t>(wq * 32) << 16);

  // ---- the piece's tiles: those that hold rows, in scan order
  const int64_t rows = __shfl_sync(~0u, rows_of(a.lengths, b, a.N), 0);
  const int live = (int)((rows + kTile - 1) / kTile);
  const int t_first = seg * a.seg_tiles + (AGG ? part * a.sub_tiles : 0);
  const int t_stop = min(a.n_tiles, min((seg + 1) * a.seg_tiles, t_first + (AGG ? a.sub_tiles : a.seg_tiles)));
  const int t_end = max(t_first, min(t_stop, live));
  const int n_it = t_end - t_first;
  auto tile_of = [&](int it) { return rev ? t_end - 1 - it : t_first + it; };
  auto rows_in = [&](int tile) { return tile == live - 1 ? (int)(rows - (int64_t)tile * kTile) : kTile; };
  // the gradient of S_N is seen from the last row itself, other states from the
  // row behind the tile
  auto shift = [&](int tile) { return rev && tile == live - 1 ? 1 : 0; };
  // tiles whose B^T C' is wanted: not the last of a piece that hands nothing on
  const bool last_seg = rev ? seg == 0 : seg == a.G - 1;
  const bool hands_on = AGG || (last_seg && own.state_out != nullptr);
  const int n_kv = hands_on ? n_it : n_it - 1;

  if (warp < 4) {
    fewer_registers<40>();
    if (warp == 0) {
      // ---------------------------------------------------------- producer
      {
        const uint32_t el = elect_one();
        const uint64_t pol = AGG ? policy_evict_last() : policy_evict_first();
        const int hk = b * a.Hk + h / a.group;
        const int ia = own.a_key ? hk : bh, ib = own.b_key ? hk : bh, ic = own.c_key ? hk : bh;
        bool ok = true;
        int nA = AGG ? n_it : 0, nB = 0, nC = 0;
        uint32_t idle = 0;
#pragma unroll 1
        while (nA < n_it || nB < n_it || nC < n_it) {
          ++idle;
          if (nC < n_it && (nC < RC || test(&empty_c[nC % RC], (nC / RC - 1) & 1))) {
            const int st = nC % RC;
            if (el) {
              mbar_arrive_expect_tx(&full_c[st], kBoxBytes);
              tma_load_3d(ring + st * kBoxBytes, &tm_c, &full_c[st], mb * kMB, tile_of(nC) * kTile,
                          ic, pol);
            }
            ++nC;
            idle = 0;
          }
          if (nB < n_it && (nB < NB || test(&empty_b[nB % NB], (nB / NB - 1) & 1))) {
            const int st = nB % NB;
            if (el) {
              mbar_arrive_expect_tx(&full_b[st], L::kBStage);
#pragma unroll
              for (int y = 0; y < L::kABoxes; ++y)
                tma_load_3d(b_ring + st * L::kBStage + y * kBoxBytes, &tm_b, &full_b[st], y * 64,
                            tile_of(nB) * kTile, ib, pol);
            }
            ++nB;
            idle = 0;
          }
          if constexpr (!AGG)
            if (nA < n_it && (nA < RA || test(&empty_a[nA % RA], (nA / RA - 1) & 1))) {
              const int st = nA % RA;
              if (el) {
                mbar_arrive_expect_tx(&full_a[st], L::kBStage);
#pragma unroll
                for (int y = 0; y < L::kABoxes; ++y)
                  tma_load_3d(a_ring + st * L::kBStage + y * kBoxBytes, &tm_a, &full_a[st], y * 64,
                              tile_of(nA) * kTile, ia, pol);
              }
              ++nA;
              idle = 0;
            }
          if (idle > 0) __nanosleep(20);
          if (__any_sync(~0u, *abort_flag != 0) || idle > (1u << 24)) {
            ok = false;
            break;
          }
        }
        if (!ok && el) record_timeout(a.status, abort_flag);
        if (!ok || *abort_flag) {
          // let the copies already issued land before the CTA's memory goes
          // away: all but the last of a ring's were waited for by their users
          // or land with it
          for (int i = max(0, nB - NB); i < nB; ++i)
            mbar_wait_timeout(&full_b[i % NB], (i / NB) & 1, CP_WAIT_TIMEOUT_NS / 64);
          for (int i = max(0, nC - RC); i < nC; ++i)
            mbar_wait_timeout(&full_c[i % RC], (i / RC) & 1, CP_WAIT_TIMEOUT_NS / 64);
          if constexpr (!AGG)
            for (int i = max(0, nA - RA); i < nA; ++i)
              mbar_wait_timeout(&full_a[i % RA], (i / RA) & 1, CP_WAIT_TIMEOUT_NS / 64);
        }
      }
    } else if (warp == 1 || !AGG) {
      // ------------------------------------------------------- MMA issuers
      constexpr uint32_t idesc_p = idesc_bf16_f32(128, 128, 0, 0);   // A . B^T
      constexpr uint32_t idesc_s2 = idesc_bf16_f32(128, 128, 1, 1);  // B^T . [C'_1 | C'_2]
      constexpr uint32_t idesc_s1 = idesc_bf16_f32(128, kMB, 1, 1);  // B^T . C'_3
      constexpr uint32_t idesc_o = idesc_bf16_f32(128, kMB, 0, 1);   // A . S, P . C
      auto b_addr = [&](int it) { return smem_u32(b_ring + (it % NB) * L::kBStage); };
      [[maybe_unused]] auto a_addr = [&](int it) { return smem_u32(a_ring + (it % max(RA, 1)) * L::kBStage); };
      auto tail = [&](int it) { return rows_in(tile_of(it)) < kTile; };
      bool ok = true;
      const uint32_t el = elect_one();
      // (A S is issued by the warp of A B^T: by that of P C it would take 234 against 232
      // us with 128-wide A, B=2 H=8 N=32768, and more with 64-wide)
      // (these loops stay rolled: with four MMAs to a turn the backward of B=8 H=16
      // N=4096 D=M=64 takes the same 184 us)
      [[maybe_unused]] auto issue_p = [&](int it) {
        tc_fence_after();
        const uint32_t t_p = tmem + (it % kNP) * 128;
        const uint32_t k_lo = desc_lo(b_addr(it), 16), q_lo = desc_lo(a_addr(it), 16);
#pragma unroll 1
        for (int kk = 0; kk < DP / 16; ++kk) {
          const uint32_t in = ((kk >> 2) * kBoxBytes + (kk & 3) * 32) >> 4;
          mma_ss_lo_elect<kHi, kHi>(t_p, q_lo + in, k_lo + in, idesc_p, kk > 0, el);
        }
        mma_commit_elect(&p_done[it % kNP], el);
        mma_commit_elect(&empty_b[it % NB], el);
        mma_commit_elect(&empty_a[it % max(RA, 1)], el);
      };
      [[maybe_unused]] auto issue_as = [&](int it) {
        tc_fence_after();
        const uint32_t s_lo = desc_lo(smem_u32(s_tile), L::kSOne);
        const uint32_t q_lo = desc_lo(a_addr(it), 16);
        // (the small parts first: an MMA rounds its sum toward zero)
#pragma unroll 1
        for (int part = kParts - 1; part >= 0; --part)
#pragma unroll 2
          for (int kk = 0; kk < DP / 16; ++kk)
            mma_ss_lo_elect<kHi, kHi>(
                tmem + L::kColO1, q_lo + (((kk >> 2) * kBoxBytes + (kk & 3) * 32) >> 4),
                s_lo + ((part * L::kSOne + kk * 2048) >> 4), idesc_o, part < kParts - 1 || kk > 0, el);
        mma_commit_elect(as_done, el);
        mma_commit_elect(o1_done, el);
        mma_commit_elect(&empty_a[it % max(RA, 1)], el);
      };
      if (warp == 1) {
        // B^T C', a piece at a time, from either C' group in turn
#pragma unroll 1
        for (int it = 0; it < n_kv && ok; ++it) {
          ok = wait(&full_b[it % NB], (it / NB) & 1, abort_flag) &&
               (it == 0 || wait(kv_free, (it - 1) & 1, abort_flag)) &&
               (!tail(it) || wait(fixed, 0, abort_flag));
          // (A = B^T, 128 rows of it: a 64-wide B's own twice over, so that both
          // halves of the lanes hold the state's rows)
          const uint32_t bt_lo = desc_lo(b_addr(it), DP == 64 ? 0 : kBoxBytes);
#pragma unroll 1
          for (int x = 0; x < L::kPieces; ++x) {
            const uint32_t parity = L::NV == 4 ? it & 1 : x >> 1 & 1;
            if (!ok || !wait(&vp_ready[x % L::NV], parity, abort_flag)) { ok = false; break; }
            tc_fence_after();
            const uint32_t v_lo = desc_lo(smem_u32(vp + x % L::NV * kParts * L::kVOne), L::kVOne);
#pragma unroll
            for (int kk = 0; kk < L::kVRows / 16; ++kk)
              mma_ss_lo_elect<kHi, kHi>(tmem + L::kColS, bt_lo + ((x * L::kVOne + kk * 2048) >> 4),
                                  v_lo + ((kk * 2048) >> 4), idesc_s2, (x | kk) > 0, el);
#pragma unroll
            for (int kk = 0; kk < L::kVRows / 16; ++kk)
              mma_ss_lo_elect<kHi, kHi>(tmem + L::kColS + kMB, bt_lo + ((x * L::kVOne + kk * 2048) >> 4),
                                  v_lo + ((2 * L::kVOne + kk * 2048) >> 4), idesc_s1, 1u, el);
            mma_commit_elect(&vp_free[x % L::NV], el);
          }
          if (!ok) break;
          mma_commit_elect(kv_done, el);
          mma_commit_elect(&empty_b[it % NB], el);
        }
      } else if (warp == 2) {
        // A B^T, as far ahead as there are buffers, and A S, whichever can go
        int nP = 0, nQ = 0;
        uint32_t idle = 0;
#pragma unroll 1
        while (nP < n_it || nQ < n_it) {
          ++idle;
          if (nP < n_it && test(&full_a[nP % max(RA, 1)], (nP / max(RA, 1)) & 1) &&
              test(&full_b[nP % NB], (nP / NB) & 1) &&
              (nP < kNP || test(&pc_done[nP % kNP], ((nP - kNP) / kNP) & 1)) &&
              (!tail(nP) || test(fixed, 0))) {
            issue_p(nP);
            ++nP;
            idle = 0;
          }
          if (nQ < nP && test(s_ready, nQ & 1) &&
              (nQ == 0 || test(o1_free, (nQ - 1) & 1))) {
            issue_as(nQ);
            ++nQ;
            idle = 0;
          }
          if (idle > 0) __nanosleep(20);
          if (__any_sync(~0u, *abort_flag != 0) || idle > (1u << 24)) {
            ok = false;
            break;
          }
        }
      } else {
        // P C
#pragma unroll 1
        for (int it = 0; it < n_it && ok; ++it) {
          const int bf = it % kNP, x = it % RC;
          ok = wait(&p_ready[bf], (it / kNP) & 1, abort_flag) &&
               wait(&full_c[x], (it / RC) & 1, abort_flag) &&
               (it == 0 || wait(o2_free, (it - 1) & 1, abort_flag)) &&
               (!tail(it) || wait(fixed, 0, abort_flag));
          if (!ok) break;
          tc_fence_after();
          const uint32_t c_lo = desc_lo(smem_u32(ring + x * kBoxBytes), kBoxBytes);
          // 32 columns of P: the first parts in their first 16 TMEM columns, the second
          // in the next, two j to a column; the third parts of an only tile in the other
          // buffer (the small parts first, as in A S)
          constexpr int parts = ONE ? 3 : 2;
#pragma unroll 1
          for (int part = parts - 1; part >= 0; --part) {
            const uint32_t p = tmem + (part == 2 ? 128 : bf * 128 + part * 16);
            const int step = part == 2 ? 16 : 32;
#pragma unroll 2
            for (int kk = 0; kk < kTile / 16; ++kk)
              mma_ts_lo_elect<kHi>(tmem + L::kColO2, p + (kk >> 1) * step + (kk & 1) * 8,
                             c_lo + ((kk * 2048) >> 4), idesc_o, part < parts - 1 || kk > 0, el);
          }
          mma_commit_elect(&pc_done[bf], el);
          mma_commit_elect(o2_done, el);
        }
      }
      if (!ok && el) record_timeout(a.status, abort_flag);
      // every MMA this thread issued completes before TMEM is released
      mma_commit_elect(&fin[warp - 1], el);
      mbar_wait_timeout(&fin[warp - 1], 0, CP_WAIT_TIMEOUT_NS);
    }
  } else if (warp < 8) {
    // ---------------------------------------------------------- state group
    more_registers<(AGG ? 104 : 88) + (DP == 64 ? 0 : AGG ? 16 : 48)>();
    {
      // thread: a row of S; with 64 rows two threads share one, half of its
      // columns each
      constexpr int SC = L::SC;
      const int d = DP == 64 ? row & 63 : row, c0 = DP == 64 ? (row >> 6) * SC : 0;
      const int pidx = bh * a.n_mb + mb, m0 = mb * kMB + c0;
      const int at = AGG ? part : rev ? a.sub - 1 : 0;  // where the prefix launch leaves a piece's first state
      float* slot = own.slots + ((((int64_t)pidx * a.G + seg) * a.sub + at) * DP + d) * kMB + c0;
      float2 S[SC / 2];
      const bool first_seg = rev ? seg == a.G - 1 : seg == 0;
      if (!AGG && !first_seg) {
#pragma unroll
        for (int x = 0; x < SC / 4; ++x) {
          const float4 f = reinterpret_cast<const float4*>(slot)[x];
          S[2 * x] = make_float2(f.x, f.y);
          S[2 * x + 1] = make_float2(f.z, f.w);
        }
      } else {
        const bool on = !AGG && own.state_in != nullptr && d < own.DA;
        const float* s = own.state_in + (int64_t)bh * own.DA * own.DC + d * own.st_r;
#pragma unroll
        for (int x = 0; x < SC / 2; ++x) {
          S[x].x = on && m0 + 2 * x < own.DC ? s[(m0 + 2 * x) * own.st_c] : 0.f;
          S[x].y = on && m0 + 2 * x + 1 < own.DC ? s[(m0 + 2 * x + 1) * own.st_c] : 0.f;
        }
      }
      const float2 full_step = power_parts(g, kTile);
      bool ok = true;
#pragma unroll 1
      for (int it = 0; it < n_it; ++it) {
        if constexpr (!AGG) {
          // the A S that last read the copy has completed
          if (it > 0 && !wait(as_done, (it - 1) & 1, abort_flag)) {
            ok = false;
            break;
          }
#pragma unroll
          for (int c = 0; c < SC / 8; ++c) {
            uint32_t p[kParts][4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              float2 s = S[4 * c + x];
#pragma unroll
              for (int y = 0; y < kParts - 1; ++y) p[y][x] = split_hi(s);
              p[kParts - 1][x] = tc::pack_bf16x2(s.x, s.y);
            }
            const uint32_t off = sw128_offset(d, c0 + 8 * c, 0);
#pragma unroll
            for (int y = 0; y < kParts; ++y)
              *reinterpret_cast<uint4*>(s_tile + y * L::kSOne + off) =
                  make_uint4(p[y][0], p[y][1], p[y][2], p[y][3]);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(s_ready);
        }
        if (it < n_kv) {
          const int tile = tile_of(it), nv = rows_in(tile);
          const float2 f = nv == kTile && shift(tile) == 0 ? full_step : power_parts(g, nv - shift(tile));
          if (!wait(kv_done, it & 1, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < SC / 16; ++c) {
            uint32_t p[16], q[16];
            tmem_ld16(lane_base + L::kColS + c0 + 16 * c, p);
            tmem_ld16(lane_base + L::kColS + kMB + c0 + 16 * c, q);
            tmem_ld_wait();
#pragma unroll
            for (int x = 0; x < 8; ++x) {
              float2& s = S[8 * c + x];
              const float2 t = add2(make_float2(__uint_as_float(p[2 * x]), __uint_as_float(p[2 * x + 1])),
                                    make_float2(__uint_as_float(q[2 * x]), __uint_as_float(q[2 * x + 1])));
              s = fma2(both(f.x), s, fma2(both(f.y), s, t));
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(kv_free);
        }
      }
      if (!ok) record_timeout(a.status, abort_flag);
      if (AGG && ok && n_it > 0) {
#pragma unroll
        for (int x = 0; x < SC / 4; ++x)
          reinterpret_cast<float4*>(slot)[x] =
              make_float4(S[2 * x].x, S[2 * x].y, S[2 * x + 1].x, S[2 * x + 1].y);
      }
      if (!AGG && ok && hands_on && d < own.DA) {
        if (rev && live > 0) {
          const float2 f = power_parts(g, 1);
#pragma unroll
          for (int x = 0; x < SC / 2; ++x) S[x] = fma2(both(f.x), S[x], mul2(both(f.y), S[x]));
        }
        float* s = own.state_out + (int64_t)bh * own.DA * own.DC + d * own.st_r;
#pragma unroll
        for (int x = 0; x < SC / 2; ++x) {
          if (m0 + 2 * x < own.DC) s[(m0 + 2 * x) * own.st_c] = S[x].x;
          if (m0 + 2 * x + 1 < own.DC) s[(m0 + 2 * x + 1) * own.st_c] = S[x].y;
        }
      }
    }
  } else if (warp >= L::kVGroup) {
    // -------------------------------- C' groups: every other piece of a tile
    fewer_registers<DP == 64 ? 56 : AGG ? 48 : 40>();
    const int half = (warp - L::kVGroup) / 4;
    const int tid = threadIdx.x - 32 * L::kVGroup - 128 * half;
    bool ok = true;
#pragma unroll 1
    for (int it = 0; it < n_it; ++it) {
      const int tile = tile_of(it), nv = rows_in(tile);
      const int st = it % RC;
      uint8_t* c_s = ring + st * kBoxBytes;
      ok = wait(&full_c[st], (it / RC) & 1, abort_flag);
      if (nv < kTile) {
        // rows of B and C past the sequence's end, which a shorter sequence of
        // a batch finds filled, are cleared before any product reads them
        if (half == 0) {
          ok = ok && wait(&full_b[it % NB], (it / NB) & 1, abort_flag);
          uint8_t* b_s = b_ring + (it % NB) * L::kBStage;
#pragma unroll 1
          for (int i = nv * 8 + tid; ok && i < kTile * 8; i += 128) {
            reinterpret_cast<uint4*>(c_s)[i] = make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int x = 0; x < L::kABoxes; ++x)
              reinterpret_cast<uint4*>(b_s + x * kBoxBytes)[i] = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0 && ok) mbar_arrive(fixed);
        }
        ok = ok && wait(fixed, 0, abort_flag);
      }
      if (it < n_kv) {
        constexpr int kEach = L::kVRows / 16;   // pieces of 8 columns to a thread, 16 rows apart
#pragma unroll 1
        for (int x = 0; x < L::kPieces / 2 && ok; ++x) {
          const int first = L::kVRows * (2 * x + half);  // row
          const int bf = (2 * x + half) % L::NV;
          uint8_t* to = vp + bf * kParts * L::kVOne;
          uint4 v[kEach];
          float w[kEach];
#pragma unroll
          for (int y = 0; y < kEach; ++y) {
            const int r = first + tid / 8 + 16 * y;
            v[y] = reinterpret_cast<const uint4*>(c_s)[8 * first + tid + 128 * y];
            w[y] = r < nv ? s_c * pw[rev ? r : nv - 1 - r] : 0.f;
          }
          if (L::NV == 4 ? it > 0 : it + x > 0)
            ok = wait(&vp_free[bf], (L::NV == 4 ? it + 1 : x + 1) & 1, abort_flag);
#pragma unroll
          for (int y = 0; y < kEach; ++y) {
            const uint32_t in[4] = {v[y].x, v[y].y, v[y].z, v[y].w};
            uint32_t out[kParts][4];
#pragma unroll
            for (int z = 0; z < 4; ++z) {
              float2 f = mul2(both(w[y]), widen(in[z]));
#pragma unroll
              for (int p = 0; p < kParts - 1; ++p) out[p][z] = split_hi(f);
              out[kParts - 1][z] = tc::pack_bf16x2(f.x, f.y);
            }
            if (ok)
#pragma unroll
              for (int p = 0; p < kParts; ++p)
                reinterpret_cast<uint4*>(to + p * L::kVOne)[tid + 128 * y] =
                    make_uint4(out[p][0], out[p][1], out[p][2], out[p][3]);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0 && ok) mbar_arrive(&vp_ready[bf]);
        }
      }
      if (!ok) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(AGG ? &empty_c[st] : &c_read[st]);
    }
    if (!ok) record_timeout(a.status, abort_flag);
  } else if (warp < 16) {
    // ------------------------- P groups: columns 0 .. 63 and 64 .. 127 of a tile
    if constexpr (!AGG && DP == 64) more_registers<80>();
    const int c_first = warp < 12 ? 0 : 2;
    bool ok = true;
    for (int it = 0; it < n_it; ++it) {
      const int bf = it % kNP;
      if (!wait(&p_done[bf], (it / kNP) & 1, abort_flag)) { ok = false; break; }
      tc_fence_after();
      const uint32_t pc = lane_base + bf * 128;
#pragma unroll 1
      for (int c = c_first; c < c_first + 2; ++c) {
        uint32_t r[32];               // then hi in the first 16, lo in the next
        if (rev ? c < wq : c > wq) {  // masked as a whole
#pragma unroll
          for (int x = 0; x < 32; ++x) r[x] = 0u;
          tmem_st32(pc + 32 * c, r);
          if constexpr (ONE) tmem_st16(pc + 128 + 16 * c, r);
          continue;
        }
        tmem_ld32(pc + 32 * c, r);
        uint32_t lo[16], third[ONE ? 16 : 1];
        auto put = [&](int x, float2 p) {
          r[x] = split_hi(p);
          if constexpr (ONE) {
            lo[x] = split_hi(p);
            third[x] = tc::pack_bf16x2(p.x, p.y);
          } else {
            lo[x] = tc::pack_bf16x2(p.x, p.y);
          }
        };
        if (c == wq) {
          // the diagonal chunk: a power per element, masked places 0 whatever
          // the accumulators hold
          const float* w = rev ? pw - lane : pw + lane;
          tmem_ld_wait();
#pragma unroll
          for (int x = 0; x < 16; ++x) {
            float2 p;
            const bool k0 = rev ? 2 * x >= lane : 2 * x <= lane;
            const bool k1 = rev ? 2 * x + 1 >= lane : 2 * x + 1 <= lane;
            p.x = k0 ? __uint_as_float(r[2 * x]) * (s_p * w[rev ? 2 * x : -2 * x]) : 0.f;
            p.y = k1 ? __uint_as_float(r[2 * x + 1]) * (s_p * w[rev ? 2 * x + 1 : -2 * x - 1]) : 0.f;
            put(x, p);
          }
        } else {
          const float2 rf = both(s_p * pw[rev ? 32 * c - row : row - 32 * c - 31]);
          const float4* f = reinterpret_cast<const float4*>(cf);
          tmem_ld_wait();
#pragma unroll
          for (int x = 0; x < 16; ++x) {
            const float2 w = x % 2 ? make_float2(f[x / 2].z, f[x / 2].w) : make_float2(f[x / 2].x, f[x / 2].y);
            float2 p = mul2(mul2(rf, w),
                            make_float2(__uint_as_float(r[2 * x]), __uint_as_float(r[2 * x + 1])));
            put(x, p);
          }
        }
#pragma unroll
        for (int x = 0; x < 16; ++x) r[16 + x] = lo[x];
        tmem_st32(pc + 32 * c, r);
        // (the only tile is buffer 0's: buffer 1 takes the third parts)
        if constexpr (ONE) tmem_st16(pc + 128 + 16 * c, third);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_ready[bf]);
    }
    if (!ok) record_timeout(a.status, abort_flag);
  } else {
    // -------------------------------------------------------------- O group
    if constexpr (!AGG) more_registers<104>();
    const int o_tid = threadIdx.x - 32 * 16;
    const int oh = own.o_key ? b * a.Hk + h / a.group : bh;
    const float full_row = s_o * pw[rev ? kTile - row : row + 1];
    bool ok = true;
    for (int it = 0; it < n_it; ++it) {
      const int tile = tile_of(it), nv = rows_in(tile);
      const float rf = !rev || (nv == kTile && shift(tile) == 0) ? full_row
                       : row < nv ? s_o * pw[nv - row - shift(tile)] : 0.f;
      // A S, scaled, waits in registers for P C, whose accumulator is given back
      // as soon as it is read: the next tile's P C waits for it
      float2 o[kMB / 2];
      ok = wait(&c_read[it % RC], (it / RC) & 1, abort_flag);
      ok = ok && wait(o1_done, it & 1, abort_flag);
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < kMB / 16; ++c) {
        uint32_t p[16];
        tmem_ld16(lane_base + L::kColO1 + 16 * c, p);
        tmem_ld_wait();
#pragma unroll
        for (int x = 0; x < 8; ++x)
          o[8 * c + x] = mul2(both(rf), make_float2(__uint_as_float(p[2 * x]), __uint_as_float(p[2 * x + 1])));
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(o1_free);
      ok = ok && wait(o2_done, it & 1, abort_flag);
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < kMB / 16; ++c) {
        uint32_t p[16];
        tmem_ld16(lane_base + L::kColO2 + 16 * c, p);
        tmem_ld_wait();
#pragma unroll
        for (int x = 0; x < 8; ++x)
          o[8 * c + x] = add2(o[8 * c + x], make_float2(__uint_as_float(p[2 * x]), __uint_as_float(p[2 * x + 1])));
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(o2_free);
      if (nv < kTile && row >= nv)
#pragma unroll
        for (int x = 0; x < kMB / 2; ++x) o[x] = make_float2(0.f, 0.f);
      // (this tile's C has been read, by the C' groups and P C: its box takes O)
      const int st = it % RC;
      uint8_t* o_tile = ring + st * kBoxBytes;
      if (!ok) break;
      if (out_f32 == nullptr) {
#pragma unroll
        for (int c = 0; c < kMB / 8; ++c)
          *reinterpret_cast<uint4*>(o_tile + sw128_offset(row, 8 * c, 0)) =
              make_uint4(tc::pack_bf16x2(o[4 * c].x, o[4 * c].y),
                         tc::pack_bf16x2(o[4 * c + 1].x, o[4 * c + 1].y),
                         tc::pack_bf16x2(o[4 * c + 2].x, o[4 * c + 2].y),
                         tc::pack_bf16x2(o[4 * c + 3].x, o[4 * c + 3].y));
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          if ((int64_t)tile * kTile + 32 * wq < a.N) {
            tma_store_3d(&tm_o, o_tile + 32 * wq * 128, mb * kMB, tile * kTile + 32 * wq, oh);
            tma_store_commit();
            tma_store_wait_read_all();
          }
          mbar_arrive(&empty_c[st]);
        }
      } else {
        // fp32 parts, which a later launch sums over the heads of a group
        float* to = out_f32 + ((int64_t)bh * a.N + (int64_t)tile * kTile + row) * own.DC + mb * kMB;
        if ((int64_t)tile * kTile + row < a.N)
#pragma unroll
          for (int x = 0; x < kMB / 4; ++x)
            if (mb * kMB + 4 * x < own.DC)
              reinterpret_cast<float4*>(to)[x] =
                  make_float4(o[2 * x].x, o[2 * x].y, o[2 * x + 1].x, o[2 * x + 1].y);
        if (lane == 0) mbar_arrive(&empty_c[st]);
      }
    }
    if (!ok) record_timeout(a.status, abort_flag);
    // tiles behind the sequence's end: zeros
    if (ok && max(t_first, live) < t_stop) {
      if (out_f32 == nullptr) {
        // (the rows that took the last O are this warp's alone by now)
        __syncwarp();
        uint8_t* o_tile = ring + max(0, n_it - 1) % RC * kBoxBytes;
#pragma unroll
        for (int c = 0; c < kMB / 8; ++c)
          *reinterpret_cast<uint4*>(o_tile + sw128_offset(row, 8 * c, 0)) = make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          for (int tile = max(t_first, live); tile < t_stop; ++tile)
            if ((int64_t)tile * kTile + 32 * wq < a.N)
              tma_store_3d(&tm_o, o_tile + 32 * wq * 128, mb * kMB, tile * kTile + 32 * wq, oh);
          tma_store_commit();
        }
      } else {
        const int64_t r0 = (int64_t)max(t_first, live) * kTile, r1 = min(a.N, (int64_t)t_stop * kTile);
        const int cols = min(kMB, own.DC - mb * kMB) / 4;
        float* to = out_f32 + (int64_t)bh * a.N * own.DC + mb * kMB;
        for (int64_t i = o_tid; i < (r1 - r0) * cols; i += 128)
          *reinterpret_cast<float4*>(to + (r0 + i / cols) * own.DC + i % cols * 4) =
              make_float4(0.f, 0.f, 0.f, 0.f);
      }
    }
    if (lane == 0) tma_store_wait_all();
  }

  tc_fence_before();
  __syncthreads();
  grid_dep_launch_dependents();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, L::kCols);
  }
}

// power_parts of a part that is not whole, out of line
static __device__ __noinline__ float2 short_part(float g, int n) { return power_parts(g, n); }

// Sums [problems][G][sub][E] of the pieces' parts give the states the pieces start
// from, each in the place of its piece's first part in scan order: a thread walks
// four elements over the parts, whose loads go out ahead.
constexpr int kPrefixThreads = 128;
template <int MAX>
__global__ void __launch_bounds__(kPrefixThreads)
    decay_tc_prefix_kernel(const __grid_constant__ Set<MAX> set, int DP) {
  const Common& a = set.all;
  const Own& own = set.own[MAX == 1 ? 0 : blockIdx.y];
  const int E4 = DP * kMB / 4, per = E4 / kPrefixThreads;
  const int problem = blockIdx.x / per, e = (blockIdx.x % per) * kPrefixThreads + threadIdx.x;
  const int bh = problem / a.n_mb, mb = problem % a.n_mb;
  float4* s = reinterpret_cast<float4*>(own.slots) + (int64_t)problem * a.G * a.sub * E4 + e;
  const int n = (a.G - 1) * a.sub;  // parts that were summed, in scan order
  grid_dep_wait();
  auto slot = [&](int i) { return (int64_t)(own.reverse ? a.G * a.sub - 1 - i : i); };
  constexpr int kAhead = 8;
  float4 next[kAhead];
#pragma unroll
  for (int i = 0; i < kAhead; ++i) next[i] = i < n ? s[slot(i) * E4] : float4{};
  const float g = head_decay(a.g[bh % a.H]);
  const int64_t rows = rows_of(a.lengths, bh / a.H, a.N);
  const int r = 4 * e / kMB, c = mb * kMB + 4 * e % kMB;
  float4 S{};
  if (own.state_in != nullptr && r < own.DA && c < own.DC) {  // (columns come in eights)
    const float* p = own.state_in + (int64_t)bh * own.DA * own.DC + r * own.st_r + c * own.st_c;
    S = make_float4(p[0], p[own.st_c], p[2 * own.st_c], p[3 * own.st_c]);
  }
  const float2 whole = power_parts(g, a.sub_tiles * kTile);
  // the part at hand, and where the sum behind a piece's last part goes
  int seg = own.reverse ? a.G - 1 : 0, part = own.reverse ? a.sub - 1 : 0;
  const int last = own.reverse ? 0 : a.sub - 1;
#pragma unroll 1
  for (int i0 = 0; i0 < n; i0 += kAhead) {
    float4 now[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      now[i] = next[i];
      next[i] = i0 + kAhead + i < n ? s[slot(i0 + kAhead + i) * E4] : float4{};
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (i0 + i >= n) break;
      const int64_t t0 = (int64_t)seg * a.seg_tiles + part * a.sub_tiles;
      const int64_t t1 = min((int64_t)a.n_tiles, min((int64_t)(seg + 1) * a.seg_tiles, t0 + a.sub_tiles));
      const int64_t lo = t0 * kTile, hi = min(rows, t1 * kTile);  // the part's rows
      if (hi > lo) {
        const int m = (int)(hi - lo) - (own.reverse && rows == hi ? 1 : 0);
        const float2 f = m == a.sub_tiles * kTile ? whole : short_part(g, m);
        S.x = fmaf(f.x, S.x, fmaf(f.y, S.x, now[i].x));
        S.y = fmaf(f.x, S.y, fmaf(f.y, S.y, now[i].y));
        S.z = fmaf(f.x, S.z, fmaf(f.y, S.z, now[i].z));
        S.w = fmaf(f.x, S.w, fmaf(f.y, S.w, now[i].w));
      }
      // (the next piece's first sum has been read, being among those ahead)
      const int at = seg * a.sub + part;
      if (part == last) {
        s[(int64_t)(own.reverse ? at - 1 : at + 1) * E4] = S;
        part = own.reverse ? a.sub : -1;
        seg += own.reverse ? -1 : 1;
      }
      part += own.reverse ? -1 : 1;
    }
  }
}

// ---------------------------------------------------------------- host
struct Plan {
  int DP, n_mb, n_tiles, seg_tiles, G, sub, sub_tiles;
  int64_t problems;    // of one product
  size_t slot_bytes;   // of one product
  double tiles;        // in line, as estimated
};
// G, the pieces to a sequence, is the one with the least tiles in line: rounds of
// CTAs on the SMs times the tiles of a piece, a round's start and end worth
// four; and with G > 1 the summing launch, which reads all pieces but one at
// three times that rate, and the two launches more, worth four.  (A tile is 1.6 to
// 2.4 us.)  At most 64 pieces: the prefix walks them one after the other, which this
// estimate leaves out.  With up to 152 B=1 H=2 N=65536 D=M=64 takes 71 us, not 47,
// H=1 D=M=128 79, not 57; H=1 D=M=64 alone gains, 51 for 56, at N=262144 84 for 105.
Plan plan(const DecayShape& s, int64_t DA, int64_t DC, int products) {
  Plan p;
  p.DP = DA <= 64 ? 64 : 128;
  p.n_mb = (int)((DC + kMB - 1) / kMB);
  p.n_tiles = (int)((s.N + kTile - 1) / kTile);
  p.problems = s.B * s.H * p.n_mb;
  const int64_t all = p.problems * products;
  int64_t G = 1;
  double best = 0;
  for (int64_t g = 1; g <= std::min<int64_t>(p.n_tiles, 64) && (g == 1 || all < 4 * kPlanSMs); ++g) {
    const int64_t rounds = (all * g + kPlanSMs - 1) / kPlanSMs, tiles = (p.n_tiles + g - 1) / g;
    double t = rounds * (tiles + 4.0);
    if (g > 1) t += 4 + 0.33 * all * (g - 1) / g * p.n_tiles / kPlanSMs;
    if (g == 1 || t < best) {
      best = t;
      G = g;
    }
  }
  p.tiles = best;
  p.seg_tiles = (int)((p.n_tiles + G - 1) / G);
  p.G = (p.n_tiles + p.seg_tiles - 1) / p.seg_tiles;
  // the summing launch has two CTAs to an SM
  const int64_t sums = all * (p.G - 1);
  const int64_t sub = sums > 0 ? std::max<int64_t>(1, 2 * kPlanSMs / sums) : 1;
  p.sub_tiles = (int)std::max<int64_t>(1, (p.seg_tiles + sub - 1) / sub);
  p.sub = (p.seg_tiles + p.sub_tiles - 1) / p.sub_tiles;
  p.slot_bytes = p.G > 1 ? sizeof(float) * (size_t)p.problems * p.G * p.sub * p.DP * kMB : 0;
  return p;
}

template <int DP, bool AGG, bool ONE, int MAX>
cudaError_t launch(const Maps<MAX>& maps, const Set<MAX>& set, unsigned grid, cudaStream_t stream) {
  using L = Layout<DP, AGG>;
  auto kern = decay_tc_kernel<DP, AGG, ONE, MAX>;
  // the shared-memory opt-in is set once per device for each instantiation
  static std::atomic<uint64_t> configured{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if ((configured.load(std::memory_order_acquire) & bit) == 0) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmem);
    if (e != cudaSuccess) return e;
    configured.fetch_or(bit, std::memory_order_release);
  }
  return launch_dependent(kern, dim3(grid), L::kThreads, L::kSmem, stream, maps, set);
}

template <int DP, int MAX>
cudaError_t launch_all(const Plan& pl, const Maps<MAX>& maps, const Set<MAX>& set,
                       cudaStream_t stream) {
  const unsigned n = (unsigned)(pl.problems * set.all.products);
  if (pl.G > 1) {
    cudaError_t e = launch<DP, true, false, MAX>(maps, set, n * (pl.G - 1) * pl.sub, stream);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)(pl.problems * DP * kMB / 4 / kPrefixThreads), set.all.products);
    e = launch_dependent(decay_tc_prefix_kernel<MAX>, grid, kPrefixThreads, 0, stream, set, DP);
    if (e != cudaSuccess) return e;
  }
  return pl.n_tiles == 1 ? launch<DP, false, true, MAX>(maps, set, n, stream)
                         : launch<DP, false, false, MAX>(maps, set, n * pl.G, stream);
}

struct RowProduct {
  const void *a, *b, *c;
  void* out;
  bool a_key, b_key, c_key, o_key, turned, reverse;  // turned: the state is held [DC][DA]
  int64_t DA, DC;
  const float* state_in;
  float *state_out, *out_f32;
  float s_p, s_o, s_c;
};

// The products of one launch: of one class of widths, DA and DC each at most 64 or
// above
template <int MAX>
cp_status_t run(const DecayShape& s, const float* g, const RowProduct* products, int n, float* slots,
                int* status, cudaStream_t stream) {
  // the maps are made by the driver, which wants a context bound to this thread:
  // a thread that autograd starts may not have called the runtime yet
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaSetDevice(dev) != cudaSuccess) return CP_ERR_CUDA;
  const Plan pl = plan(s, products[0].DA, products[0].DC, n);
  const int64_t vh = s.B * s.H, kh = s.B * s.Hk;
  Maps<MAX> maps;
  Set<MAX> set{};
  Common& a = set.all;
  a.g = g;
  a.lengths = s.lengths;
  a.status = status;
  a.N = s.N;
  a.H = (int)s.H; a.Hk = (int)s.Hk; a.group = (int)(s.H / s.Hk); a.BH = (int)vh;
  a.n_mb = pl.n_mb; a.n_tiles = pl.n_tiles; a.seg_tiles = pl.seg_tiles; a.G = pl.G;
  a.sub = pl.sub; a.sub_tiles = pl.sub_tiles;
  a.products = n;
  for (int i = 0; i < n; ++i) {
    const RowProduct& p = products[i];
    if (!tc::make_map(&maps.a[i], p.a, p.a_key ? kh : vh, s.N, p.DA) ||
        !tc::make_map(&maps.b[i], p.b, p.b_key ? kh : vh, s.N, p.DA) ||
        !tc::make_map(&maps.c[i], p.c, p.c_key ? kh : vh, s.N, p.DC) ||
        !tc::make_map(&maps.o[i], p.out, p.o_key ? kh : vh, s.N, p.DC, 0, 32))
      return CP_ERR_UNSUPPORTED_SHAPE;
    Own& o = set.own[i];
    o.state_in = p.state_in;
    o.state_out = p.state_out;
    o.slots = slots + i * (pl.slot_bytes / sizeof(float));
    o.out_f32 = p.out_f32;
    o.st_r = p.turned ? 1 : p.DC;
    o.st_c = p.turned ? p.DA : 1;
    o.DA = (int)p.DA; o.DC = (int)p.DC;
    o.a_key = p.a_key; o.b_key = p.b_key; o.c_key = p.c_key; o.o_key = p.o_key;
    o.reverse = p.reverse;
    o.s_p = p.s_p; o.s_o = p.s_o; o.s_c = p.s_c;
  }
  const cudaError_t e = pl.DP == 64 ? launch_all<64>(pl, maps, set, stream)
                                    : launch_all<128>(pl, maps, set, stream);
  return e == cudaSuccess ? CP_OK : CP_ERR_CUDA;
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

size_t part_bytes(const DecayShape& s) {
  return s.H == s.Hk ? 0 : round256(sizeof(float) * (size_t)s.B * s.H * s.N * s.D);
}

}  // namespace

bool decay_tc_supported(const DecayShape& s) {
  return s.dtype == CP_DTYPE_BF16 && s.D <= 128 && s.M <= 128;
}

// Products of one class of widths may share a launch: where that saves rounds of
// CTAs or launches, for a CTA whose product is chosen as it runs is a tenth slower.
// The backward, three products in one launch against three launches: B=2 H=8 N=1000
// D=M=64 34 against 50 us, D=M=128 27 against 63, B=3 H=10 N=3000 D=M=64 54 against
// 82, and B=8 H=16 N=4096 D=M=64, three rounds either way, 213 against 184.
static int in_one_launch(const DecayShape& s) {
  const double dq = plan(s, s.M, s.D, 1).tiles;
  auto pays = [&](int n) { return 1.1 * plan(s, s.M, s.D, n).tiles < n * (dq + 1); };
  if ((s.D <= 64) == (s.M <= 64) && pays(3)) return 3;  // dq, dk, dv
  return pays(2) ? 2 : 1;                               // dq, dk
}

size_t decay_tc_scratch(const DecayShape& s, bool backward) {
  if (!backward) return plan(s, s.D, s.M, 1).slot_bytes;
  const int n = in_one_launch(s);
  const size_t slots = std::max(n * plan(s, s.M, s.D, n).slot_bytes,
                                n < 3 ? plan(s, s.D, s.M, 1).slot_bytes : 0);
  return round256(slots) + 2 * part_bytes(s);
}

cp_status_t decay_tc_fwd(const DecayShape& s, const DecayFwd& f, void* scratch, int* status,
                         cudaStream_t stream) {
  const RowProduct p{f.q, f.k, f.v, f.out, true, true, false, false, false, false, s.D, s.M,
                  f.state_in, f.state_out, nullptr, s.scale, s.scale, 1.f};
  return run<1>(s, f.g, &p, 1, static_cast<float*>(scratch), status, stream);
}

cp_status_t decay_tc_bwd(const DecayShape& s, const DecayBwd& f, void* scratch, int* status,
                         cudaStream_t stream) {
  const bool grouped = s.H != s.Hk;
  float* slots = static_cast<float*>(scratch);
  float* parts = reinterpret_cast<float*>(static_cast<char*>(scratch) +
                                          (decay_tc_scratch(s, true) - 2 * part_bytes(s)));
  float* dq_part = grouped ? parts : nullptr;
  float* dk_part = grouped ? parts + part_bytes(s) / sizeof(float) : nullptr;
  const RowProduct p[3] = {
      {f.grad_out, f.v, f.k, f.dq, false, false, true, true, true, false, s.M, s.D, f.state_in,
       nullptr, dq_part, s.scale, s.scale, 1.f},
      {f.v, f.grad_out, f.q, f.dk, false, false, true, true, true, true, s.M, s.D,
       f.grad_state_out, nullptr, dk_part, s.scale, 1.f, s.scale},
      {f.k, f.q, f.grad_out, f.dv, true, true, false, false, false, true, s.D, s.M,
       f.grad_state_out, f.grad_state_in, nullptr, s.scale, 1.f, s.scale}};
  const int n = in_one_launch(s);
  cp_status_t st = CP_OK;
  if (n > 1) st = run<3>(s, f.g, p, n, slots, status, stream);
  for (int i = n > 1 ? n : 0; i < 3 && st == CP_OK; ++i)
    st = run<1>(s, f.g, p + i, 1, slots, status, stream);
  if (st != CP_OK || !grouped) return st;
  return delta_join_launch({dq_part, dk_part, nullptr, nullptr, f.dq, f.dk, nullptr, nullptr, s.N,
                            s.D, s.B * s.Hk, (int)(s.H / s.Hk), 1},
                           s.dtype, stream) == cudaSuccess
             ? CP_OK
             : CP_ERR_CUDA;
}

}  // namespace cp
