// The gated delta rule on the 5th-generation tensor cores: what its forward
// and backward kernels share (formulas in cp_delta.cuh).
//
// Every contraction is a tcgen05.mma with bf16 operands in shared memory and
// an fp32 accumulator of 128 lanes in tensor memory.  q, k, v and the output's
// gradient are bf16 as they come; what is computed (S, R, U, P, the inverse and
// the gradients' factors) is fp32 and enters a product as three bf16 numbers, all
// of its 24 bits, so a product with an input is three MMAs and one of two such
// factors six (the terms left out are 2^-27 of it).  With two numbers each (16
// bits) the carried state and the gates' gradients, which are fp32, were 3e-6 to
// 7e-6 off; with three they are where fp32 arithmetic leaves them, at 2e-7 to
// 5e-7.  Terms of one size share an accumulator where there is room, and elsewhere
// the small ones go first: an MMA rounds its sum toward zero.
//
// An operand tile is 64 columns wide (128 bytes, 128-byte swizzle), so it can
// enter as [rows x K] or transposed, by its descriptor alone.
#pragma once
#include "cp_delta.cuh"
#include "cp_tc_common.cuh"

namespace cp {
namespace delta {

using namespace cp::ptx;

constexpr int kCh = 64;               // rows of a chunk
constexpr int kBox = kCh * 128;       // bytes of a [64 x 64] bf16 tile
constexpr uint32_t kDescHi = desc_hi(1024);

// The first 1024-byte boundary of the shared memory, as an offset from its
// array: the compiler then knows what follows for shared memory and addresses
// it with 32 bits.
__device__ __forceinline__ uint8_t* align_tiles(uint8_t* smem) {
  return smem + (-smem_u32(smem) & 1023u);
}

// The gates of a chunk.  Every decay between two rows is the exponential of a
// difference of running sums (in two parts, cp_delta.cuh), of which the sums'
// rounding leaves 1e-7; a product of up to 64 factors e^g would leave each one's
// rounding, the same way at every row where the decay is constant.  A cleared
// state's decay stays an exact zero.
struct alignas(16) GateSlot {
  float2 G[kCh];                      // running sums of the log decay
  float b[kCh];
  float gam[kCh], del[kCh];           // decay up to row i, after row j
  float tail[32], half[32];           // decay after row j up to row 31, from row 32 to row 32 + i
  float2 last;                        // decay over the chunk, hi + lo
};

// 2^x for x <= 0, to 2^-22; 0 below 2^-126
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// One warp: the slot from the lane's two rows' (lane, lane + 32) log decays and
// strengths.
__device__ __forceinline__ void write_gates(GateSlot* s, int lane, float g0, float g1, float b0,
                                            float b1) {
  const float2 zero = make_float2(0.f, 0.f);
  const auto total = [](float2 x) {
    return make_float2(__shfl_sync(0xffffffffu, x.x, 31), __shfl_sync(0xffffffffu, x.y, 31));
  };
  const float2 G0 = warp_scan(split_decay(g0), lane), mid = total(G0);
  const float2 H1 = warp_scan(split_decay(g1), lane), G1 = add2(mid, H1), end = total(G1);
  s->G[lane] = G0;
  s->G[lane + 32] = G1;
  s->b[lane] = b0;
  s->b[lane + 32] = b1;
  s->gam[lane] = decay_between(G0, zero);
  s->gam[lane + 32] = decay_between(G1, zero);
  s->del[lane] = decay_between(end, G0);
  s->del[lane + 32] = decay_between(end, G1);
  s->tail[lane] = decay_between(mid, G0);
  s->half[lane] = decay_between(H1, zero);
  if (lane == 0) s->last = decay_parts(end);
}

// w times the decay from row j to row i of the chunk for the 16 columns j = 16
// c .. of row i (own: with those of the row's half, row32), 0 past column last.
__device__ __forceinline__ void decays16(const GateSlot* gs, int i, int row32, int c, int last,
                                         float w, float2 (&v)[8]) {
  if (c >= 2 * row32 + 2) {
#pragma unroll
    for (int x = 0; x < 8; ++x) v[x] = both(0.f);
  } else if (c >= 2 * row32) {
    const float2 Gi = gs->G[i];
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      const float4 g = *reinterpret_cast<const float4*>(gs->G + 16 * c + 2 * x);
      const float2 d0 = sub2(Gi, make_float2(g.x, g.y)), d1 = sub2(Gi, make_float2(g.z, g.w));
      v[x].x = 16 * c + 2 * x <= last ? w * exp2_fast(d0.x + d0.y) : 0.f;
      v[x].y = 16 * c + 2 * x + 1 <= last ? w * exp2_fast(d1.x + d1.y) : 0.f;
    }
  } else {
    const float2 p = both(w * gs->half[i - 32]);
#pragma unroll
    for (int x = 0; x < 8; x += 2) {
      const float4 t = *reinterpret_cast<const float4*>(gs->tail + 16 * c + 2 * x);
      v[x] = mul2(p, make_float2(t.x, t.y));
      v[x + 1] = mul2(p, make_float2(t.z, t.w));
    }
  }
}

// x as two bf16 numbers; each packed as pairs
__device__ __forceinline__ void split_pair(float2 x, uint32_t& hi, uint32_t& lo) {
  hi = tc::pack_bf16x2(x.x, x.y);
  const float2 d =
      sub2(x, make_float2(__uint_as_float(hi << 16), __uint_as_float(hi & 0xffff0000u)));
  lo = tc::pack_bf16x2(d.x, d.y);
}

// x as three bf16 numbers (all of fp32's bits)
__device__ __forceinline__ void split_pair3(float2 x, uint32_t& a, uint32_t& b, uint32_t& c) {
  a = tc::pack_bf16x2(x.x, x.y);
  const float2 d = sub2(x, make_float2(__uint_as_float(a << 16), __uint_as_float(a & 0xffff0000u)));
  split_pair(d, b, c);
}
__device__ __forceinline__ void split16_3(const float2 (&x)[8], uint4 (&a)[2], uint4 (&b)[2],
                                          uint4 (&c)[2]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    split_pair3(x[4 * i], a[i].x, b[i].x, c[i].x);
    split_pair3(x[4 * i + 1], a[i].y, b[i].y, c[i].y);
    split_pair3(x[4 * i + 2], a[i].z, b[i].z, c[i].z);
    split_pair3(x[4 * i + 3], a[i].w, b[i].w, c[i].w);
  }
}
// columns [8 ch, 8 ch + 16) of row `row` of a 64-column tile
__device__ __forceinline__ void put16(uint8_t* tile, int row, int ch, const uint4 (&v)[2]) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
    *reinterpret_cast<uint4*>(tile + row * 128 + (((ch + i) ^ (row & 7)) << 4)) = v[i];
}
__device__ __forceinline__ void pack16(const float2 (&x)[8], uint4 (&w)[2]) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
    w[i] = make_uint4(tc::pack_bf16x2(x[4 * i].x, x[4 * i].y), tc::pack_bf16x2(x[4 * i + 1].x, x[4 * i + 1].y),
                      tc::pack_bf16x2(x[4 * i + 2].x, x[4 * i + 2].y),
                      tc::pack_bf16x2(x[4 * i + 3].x, x[4 * i + 3].y));
}
// 16 fp32 values into a matrix's three parts, `part` bytes apart
__device__ __forceinline__ void store16_split(uint8_t* tile, int part, int row, int ch,
                                              const float2 (&x)[8]) {
  uint4 a[2], b[2], c[2];
  split16_3(x, a, b, c);
  put16(tile, row, ch, a);
  put16(tile + part, row, ch, b);
  put16(tile + 2 * part, row, ch, c);
}
// .. and into a tile of fp32 rows of 32 columns, as it goes to memory (16-byte
// pieces of a row in an order of its own, so that rows fall in different banks)
__device__ __forceinline__ void put_f32(uint8_t* tile, int row, int sub, const float2 (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    *reinterpret_cast<float4*>(tile + row * 128 + (((4 * sub + i) ^ (row & 7)) << 4)) =
        make_float4(x[2 * i].x, x[2 * i].y, x[2 * i + 1].x, x[2 * i + 1].y);
}
// the same 16 columns to global memory, of which `nc` are inside the matrix
__device__ __forceinline__ void write16(__nv_bfloat16* dst, int nc, const uint4 (&v)[2]) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (8 * i < nc) *reinterpret_cast<uint4*>(dst + 8 * i) = v[i];
}

// acc (128 lanes at tmem d) (+)= A B over K, with A and B at shared addresses
// a, b and their tiles' K steps of 16.  Run by a whole converged warp, issued by
// its elected lane: with one thread in the branch every MMA took 125 cycles to
// issue, its descriptors going from vector to uniform registers; so it takes 62.
//   KA / KB: the operand's rows run along K (transposed use): a step is 16
//   rows (2048 bytes); otherwise 16 columns (32 bytes), and every fourth step
//   moves to the next 64-column tile, `box` bytes on.
// lbo: distance of the second 64-lane block of a transposed A (or of the
// second 64 columns of a transposed B).
template <int STEPS, bool KA, bool KB>
__device__ __forceinline__ void mma_tile(uint32_t el, uint32_t d, uint32_t a, uint32_t b,
                                         uint32_t idesc, uint32_t a_lbo, uint32_t b_lbo,
                                         uint32_t a_box, uint32_t b_box, bool fresh) {
  const uint32_t a_lo = desc_lo(a, a_lbo), b_lo = desc_lo(b, b_lbo);
#pragma unroll
  for (int k = 0; k < STEPS; ++k) {
    const uint32_t ao = KA ? k * 2048 : (k / 4) * a_box + (k % 4) * 32;
    const uint32_t bo = KB ? k * 2048 : (k / 4) * b_box + (k % 4) * 32;
    mma_ss_lo_elect<kDescHi, kDescHi>(d, a_lo + (ao >> 4), b_lo + (bo >> 4), idesc,
                                      (fresh && k == 0) ? 0u : 1u, el);
  }
}

// Wait; a wait that gives up records the timeout and sets the CTA's abort
// flag, after which every other wait of the CTA gives up at once: the CTA runs
// to its end on whatever it holds (every address stays the same), and its
// results are undefined.
// The polling is out of line: these kernels' instruction stream is long and
// mostly straight, and its fetch is the first stall when it grows (with the
// loops below unrolled, 118 KB, a third of all stalls).
static __device__ __noinline__ void wait_slow(uint64_t* bar, uint32_t parity, int* status,
                                              volatile int* abort_flag) {
  if (!mbar_wait(bar, parity, abort_flag)) tc::record_timeout(status, abort_flag);
}
__device__ __forceinline__ void wait_or_abort(uint64_t* bar, uint32_t parity, int* status,
                                              volatile int* abort_flag) {
  if (!mbar_try_wait(bar, parity)) wait_slow(bar, parity, status, abort_flag);
}

// After an abort, a millisecond for the copies and MMAs in flight to land
// before the CTA gives its memory back.
static __device__ __noinline__ void linger() {
  const uint64_t t0 = globaltimer();
  while (globaltimer() - t0 < 1000000ull) {
  }
}

// 16 consecutive 32-bit columns of the warp's lanes
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float2 (&x)[8]) {
  uint32_t r[16];
  tmem_ld16(taddr, r);
  tmem_ld_wait();
#pragma unroll
  for (int i = 0; i < 8; ++i)
    x[i] = make_float2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
}

// The chains run 32 value columns to a CTA, 16 to a thread: a factor's first part
// is columns 0-31 of a 64-column tile and its second columns 32-63; the third
// parts of two factors share another.  One MMA of 96 columns takes all three.
constexpr int kCB = 32;
// .. by two warpgroups, and a ninth warp for the copies and the gates: written
// by one of the eight, they kept the others at a barrier for 340 to 440 cycles
// of a chunk's 3,600 to 3,900.
constexpr int kChainThreads = 256 + 32;

// 16 columns of such a product: the sum of its three accumulators, the small
// ones first (and in turn, for the registers)
__device__ __forceinline__ void load16_sum(uint32_t taddr, float2 (&x)[8]) {
  uint32_t h[16], l[16];
  tmem_ld16(taddr + kCB, h);
  tmem_ld16(taddr + 2 * kCB, l);
  tmem_ld_wait();
#pragma unroll
  for (int i = 0; i < 8; ++i)
    x[i] = add2(make_float2(__uint_as_float(h[2 * i]), __uint_as_float(h[2 * i + 1])),
                make_float2(__uint_as_float(l[2 * i]), __uint_as_float(l[2 * i + 1])));
  tmem_ld16(taddr, h);
  tmem_ld_wait();
#pragma unroll
  for (int i = 0; i < 8; ++i)
    x[i] = add2(make_float2(__uint_as_float(h[2 * i]), __uint_as_float(h[2 * i + 1])), x[i]);
}
// .. and 16 fp32 values into such a factor's tiles, the thread's columns being 16
// sub ..; third: the third parts' tile, the factor's columns beginning at 8 ch
__device__ __forceinline__ void store_parts(uint8_t* tile, uint8_t* third, int ch, int row, int sub,
                                            const float2 (&x)[8]) {
  uint4 a[2], b[2], c[2];
  split16_3(x, a, b, c);
  put16(tile, row, 2 * sub, a);
  put16(tile, row, 4 + 2 * sub, b);
  put16(third, row, ch + 2 * sub, c);
}
// T B of two computed factors at acc, whose columns then hold the products' terms
// by size: A's first part with all three of B's, its second with two, its third
// with one.  A's parts are a_part bytes apart.
template <bool KA>
__device__ __forceinline__ void mma_parts(uint32_t el, uint32_t acc, uint32_t a, uint32_t a_part,
                                          uint32_t a_lbo, uint32_t b, uint32_t b_third) {
  mma_tile<4, KA, true>(el, acc, a, b, idesc_bf16_f32(128, 3 * kCB, KA, 1), a_lbo, b_third - b, 0, 0,
                        true);
  mma_tile<4, KA, true>(el, acc + kCB, a + a_part, b, idesc_bf16_f32(128, 2 * kCB, KA, 1), a_lbo, 16,
                        0, 0, false);
  mma_tile<4, KA, true>(el, acc + 2 * kCB, a + 2 * a_part, b, idesc_bf16_f32(128, kCB, KA, 1), a_lbo,
                        16, 0, 0, false);
}
// 16 columns of a row of inputs, of which nc are inside the matrix
__device__ __forceinline__ void read16(const __nv_bfloat16* src, int nc, bool on, uint4 (&v)[2]) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
    v[i] = on && 8 * i < nc ? *reinterpret_cast<const uint4*>(src + 8 * i) : make_uint4(0, 0, 0, 0);
}
__device__ __forceinline__ void unpack16(const uint4 (&v)[2], float2 (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
    for (int e = 0; e < 4; ++e)
      x[4 * i + e] = make_float2(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xffff0000u));
  }
}
// 16 columns of a row of fp32 (zero outside)
__device__ __forceinline__ void read16(const float* src, int nc, bool on, float2 (&x)[8]) {
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (on && 2 * j < nc) v = *reinterpret_cast<const float4*>(src + 2 * j);
    x[j] = make_float2(v.x, v.y);
    x[j + 1] = make_float2(v.z, v.w);
  }
}
__device__ __forceinline__ void write16(float* dst, int nc, const float2 (&x)[8]) {
#pragma unroll
  for (int j = 0; j < 8; j += 2)
    if (2 * j < nc)
      *reinterpret_cast<float4*>(dst + 2 * j) = make_float4(x[j].x, x[j].y, x[j + 1].x, x[j + 1].y);
}

// ------------------------------------------------ the inverse of I + A
// T = (I + A)^-1 for a 64 x 64 strictly lower triangular A, by four warps, warp
// a the columns of block a (16 columns).  The four diagonal blocks are inverted
// by substitution, a lane to a column; the blocks below follow from
//     X_ba = -X_bb sum_{a <= c < b} A_bc X_ca,
// transposed (Z_ab = X_ba^T = -(sum_c Z_ac A_bc^T) X_bb^T) so that a result
// tile is the next product's left factor without leaving its registers.  These
// are 16 x 16 products of a few hundred cycles' latency in all: mma.sync, each
// factor in three parts; a tcgen05 product's way through tensor memory costs more
// than the product.  Blockwise substitution keeps the inverse to about the
// factors' precision whatever A is; the doubling product (I - A)(I + A^2) ..
// loses everything to cancellation when keys repeat.
constexpr int kDiagPitch = 16 * 24 + 16;   // floats between diagonal blocks
struct InvTiles {
  // diagonal blocks of A, fp32, transposed: [block][column l][row i]; then,
  // in its place, the block's inverse, transposed, three bf16 parts
  float diag[4 * kDiagPitch];
  // blocks below the diagonal, bf16, row major, at index b (b - 1) / 2 + c for
  // block (b, c), in three parts
  __nv_bfloat16 low[6][3][16 * 16];
  __device__ __forceinline__ __nv_bfloat16* xt(int b, int part) {
    return reinterpret_cast<__nv_bfloat16*>(diag + b * kDiagPitch) + part * 256;
  }
};

__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                          uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}

// Block column c (16 columns) of row i of A, into the tiles.
__device__ __forceinline__ void put_a16(InvTiles* it, int i, int c, const float2 (&v)[8]) {
  const int b = i / 16;
  if (c == b) {
    float* d = it->diag + b * kDiagPitch + i % 16;
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      d[32 * x] = v[x].x;
      d[32 * x + 16] = v[x].y;
    }
  } else if (c < b) {
    const int idx = b * (b - 1) / 2 + c;
    uint4 part[3][2];
    split16_3(v, part[0], part[1], part[2]);
#pragma unroll
    for (int x = 0; x < 3; ++x) {
      uint4* to = reinterpret_cast<uint4*>(it->low[idx][x] + (i % 16) * 16);
      to[0] = part[x][0];
      to[1] = part[x][1];
    }
  }
}

// Warp b: the inverse of diagonal block b, column l % 16 by lane l, to xt and
// packed in w (lanes 0-15 the first part, 16-31 the second) and w3 (the third).
__device__ __forceinline__ void invert_diag(InvTiles* it, int b, int lane, uint4 (&w)[2],
                                            uint4 (&w3)[2]) {
  const int c = lane & 15;
  float x[16];
  const float* d = it->diag + b * kDiagPitch;
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] = i == c ? 1.f : 0.f;
#pragma unroll
  for (int l = 0; l < 15; ++l) {
#pragma unroll
    for (int i = (l + 1) / 4 * 4; i < 16; i += 4) {
      const float4 a = *reinterpret_cast<const float4*>(d + 16 * l + i);
      if (i > l) x[i] = fmaf(-a.x, x[l], x[i]);
      if (i + 1 > l) x[i + 1] = fmaf(-a.y, x[l], x[i + 1]);
      if (i + 2 > l) x[i + 2] = fmaf(-a.z, x[l], x[i + 2]);
      if (i + 3 > l) x[i + 3] = fmaf(-a.w, x[l], x[i + 3]);
    }
  }
  uint32_t p[8], p3[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    uint32_t h, l;
    split_pair3(make_float2(x[2 * i], x[2 * i + 1]), h, l, p3[i]);
    p[i] = lane < 16 ? h : l;
  }
  w[0] = make_uint4(p[0], p[1], p[2], p[3]);
  w[1] = make_uint4(p[4], p[5], p[6], p[7]);
  w3[0] = make_uint4(p3[0], p3[1], p3[2], p3[3]);
  w3[1] = make_uint4(p3[4], p3[5], p3[6], p3[7]);
  __syncwarp();  // the block has been read by every lane
  uint4* to = reinterpret_cast<uint4*>(it->xt(b, lane >> 4) + c * 16);
  to[0] = w[0];
  to[1] = w[1];
  if (lane < 16) {
    to = reinterpret_cast<uint4*>(it->xt(b, 2) + c * 16);
    to[0] = w3[0];
    to[1] = w3[1];
  }
}

// big, small [n tile] += a b, both in three parts, small taking all but the first
// parts' product; b fragments as {tile 0: k low, k high, tile 1: k low, k high}
__device__ __forceinline__ void mma_split(float (&big)[2][4], float (&small)[2][4],
                                          const uint32_t (&a)[3][4], const uint32_t (&b)[3][4]) {
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    mma_16816(big[n], a[0], b[0][2 * n], b[0][2 * n + 1]);
#pragma unroll
    for (int x = 2; x > 0; --x)
#pragma unroll
      for (int y = x; y >= 0; --y) mma_16816(small[n], a[y], b[x - y][2 * n], b[x - y][2 * n + 1]);
  }
}
// sign (big + small) as the next product's left factor
__device__ __forceinline__ void next_factor(uint32_t (&z)[3][4], const float (&big)[2][4],
                                            const float (&small)[2][4], float sign) {
#pragma unroll
  for (int n = 0; n < 2; ++n)
#pragma unroll
    for (int r = 0; r < 2; ++r)
      split_pair3(make_float2(sign * (big[n][2 * r] + small[n][2 * r]),
                              sign * (big[n][2 * r + 1] + small[n][2 * r + 1])),
                  z[0][2 * n + r], z[1][2 * n + r], z[2][2 * n + r]);
}

// Warp a: Z_ab = X_ba^T for b = a + s, packed in z[s], three parts: word 2 n + r
// is columns (rows of X) 16 b + 8 n + 2 (lane % 4) and the next, row (column of X)
// 16 a + lane / 4 + 8 r.  After invert_diag and a barrier.
__device__ __forceinline__ void invert_below(InvTiles* it, int a, int lane, uint32_t (&z)[4][3][4]) {
  const int g = lane / 4, t = lane % 4;
  {
    const int at[4] = {g * 8 + t, (g + 8) * 8 + t, g * 8 + t + 4, (g + 8) * 8 + t + 4};
#pragma unroll
    for (int x = 0; x < 3; ++x)
#pragma unroll
      for (int i = 0; i < 4; ++i) z[0][x][i] = reinterpret_cast<const uint32_t*>(it->xt(a, x))[at[i]];
  }
#pragma unroll
  for (int s = 1; s < 4; ++s) {  // b = a + s
    const int b = a + s;
    if (b > 3) break;
    float big[2][4] = {}, small[2][4] = {};
    uint32_t f[3][4];
#pragma unroll
    for (int c = 0; c < s; ++c) {
      const int idx = b * (b - 1) / 2 + a + c;
#pragma unroll
      for (int x = 0; x < 3; ++x)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int k = 0; k < 2; ++k)
            f[x][2 * n + k] =
                reinterpret_cast<const uint32_t*>(it->low[idx][x])[(8 * n + g) * 8 + 4 * k + t];
      mma_split(big, small, z[c], f);
    }
    uint32_t y[3][4];
    next_factor(y, big, small, -1.f);
    // X_bb^T as a right factor: rows k of xt, transposed on load; lane -> row
    // lane % 16, column half lane / 16
    const uint32_t row = (uint32_t)((lane % 16) * 32 + (lane / 16) * 16);
#pragma unroll
    for (int x = 0; x < 3; ++x) ldmatrix_x4_trans(f[x], smem_u32(it->xt(b, x)) + row);
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) big[n][i] = small[n][i] = 0.f;
    mma_split(big, small, y, f);
    next_factor(z[s], big, small, 1.f);
  }
}

// Warp a's columns of the inverse X, as rows of the transposed tile (row j,
// column i: element (i, j)), the three parts `part` bytes apart: the diagonal
// block from w and w3, those below from z, those above zero.
__device__ __forceinline__ void put_t_transposed(uint8_t* tile, int part, int a, int lane,
                                                 const uint4 (&w)[2], const uint4 (&w3)[2],
                                                 const uint32_t (&z)[4][3][4]) {
  uint8_t* own = tile + (lane < 16 ? 0 : part);
  const int own_row = 16 * a + (lane & 15);
  put16(own, own_row, 2 * a, w);
  if (lane < 16) put16(tile + 2 * part, own_row, 2 * a, w3);
  const uint4 zero[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
#pragma unroll 1
  for (int b = 0; b < a; ++b) {
    put16(own, own_row, 2 * b, zero);
    if (lane < 16) put16(tile + 2 * part, own_row, 2 * b, zero);
  }
  const int g = lane / 4;
  uint8_t* row = tile + (16 * a + g) * 128 + 4 * (lane % 4);
#pragma unroll
  for (int s = 1; s < 4; ++s) {
    if (a + s > 3) break;
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      uint8_t* to = row + (((2 * (a + s) + n) ^ g) << 4);
#pragma unroll
      for (int x = 0; x < 3; ++x)
#pragma unroll
        for (int r = 0; r < 2; ++r)
          *reinterpret_cast<uint32_t*>(to + 1024 * r + x * part) = z[s][x][2 * n + r];
    }
  }
}

// Row i of the chunk's k.k or q.k (lane of the accumulator at t_kk), weighted
// by the decays: w times the decay from row j to row i, for j < i (and for j =
// i, where it is w, with `diag`), 0 elsewhere; f(c, v) takes columns 16 c .. 16 c
// + 15.  row32: the row's half of the chunk, uniform over the warp.
template <class F>
__device__ __forceinline__ void decayed_row(uint32_t t_kk, const GateSlot* gs, int i, bool diag,
                                            int row32, float w, F f) {
  const int last = diag ? i : i - 1;
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    uint32_t r[16];
    tmem_ld16(t_kk + 16 * c, r);
    float2 v[8];
    decays16(gs, i, row32, c, last, w, v);
    tmem_ld_wait();
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      // masked places stay 0 whatever the accumulators hold
      const float2 y =
          mul2(v[x], make_float2(__uint_as_float(r[2 * x]), __uint_as_float(r[2 * x + 1])));
      v[x].x = 16 * c + 2 * x <= last ? y.x : 0.f;
      v[x].y = 16 * c + 2 * x + 1 <= last ? y.y : 0.f;
    }
    f(c, v);
  }
}

// Launched as a programmatic dependent, as the product kernels are: a kernel's
// launch (and, in the chains, its set-up) runs under the end of the one before
// it in the stream, and it touches no global memory before that one has
// completed; a CTA lets the next kernel be scheduled only when its own work is
// done.
template <class K, class... A>
inline cudaError_t launch_dependent(K kern, dim3 grid, unsigned threads, size_t smem,
                                    cudaStream_t stream, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

// one contiguous shared -> global copy (16-byte aligned, a multiple of 16)
__device__ __forceinline__ void bulk_store(void* gdst, const void* smem_src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(gdst),
               "r"(smem_u32(smem_src)), "r"(bytes)
               : "memory");
}

// What the forward keeps for the backward:
//   S  [BH][chunks][blocks of 32 columns]  the state before every chunk, fp32
//   U  [BH][chunks][blocks of 32 columns]  what every row wrote, fp32
//   T  [BH][chunks]                        the inverse (transposed), 24 KB
//   P  [BH][chunks]                        24 KB
// S and U as put_f32 lays them out; T and P as operand tiles, as they lie in
// shared memory (fp32 values in three bf16 parts, swizzled), so that the reverse
// chain's copies bring them ready for the tensor cores.  With them neither of the
// backward's kernels recomputes a chunk's inverse.
constexpr int kTTile = 3 * kBox;
struct Saved {
  int64_t n, blocks, s_tile, s_bytes, u_bytes, t_bytes;  // t_bytes: of T, and of P
  Saved(const DeltaShape& s)
      : n((s.N + kCh - 1) / kCh),
        blocks((s.M + kCB - 1) / kCB),
        s_tile(s.D <= 64 ? 64 * 128 : 128 * 128),
        s_bytes(s.B * s.H * n * blocks * s_tile),
        u_bytes(s.B * s.H * n * blocks * kBox),
        t_bytes(s.B * s.H * n * kTTile) {}
  int64_t bytes() const { return s_bytes + u_bytes + 2 * t_bytes; }
};

// [heads][N][cols] bf16, boxes of 64 columns x 64 rows, 128-byte swizzle
inline bool make_chunk_map(CUtensorMap* m, const void* ptr, int64_t heads, int64_t N, int64_t cols) {
  auto enc = tc::get_encode();
  if (enc == nullptr) return false;
  cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)N, (cuuint64_t)heads};
  cuuint64_t strides[2] = {(cuuint64_t)cols * 2, (cuuint64_t)(N * cols * 2)};
  cuuint32_t box[3] = {64, (cuuint32_t)kCh, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(ptr), dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace delta
}  // namespace cp
