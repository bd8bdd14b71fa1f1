// decode.cuh -- the whole sparse MoE block for a few tokens in two kernels.
//
// With T <= kDecodeMaxT tokens the block reads every active expert's weights
// for one or two rows each: the time is the weight bytes over the HBM rate plus
// whatever latency the launches and barriers add.
//   k_decode_route: the RMSNorm, the shared expert's gate, the router's logits
//     (split over 16 experts x slices of d, fp32 partials) and, for E4M3 and mx4
//     weights, x as their products take it (below);
//   k_decode, cooperative, one CTA per SM:
//   1. every CTA adds the partials in slice order and selects each token's top k
//      (one warp per token; the same code and inputs, so the same result in every
//      CTA), and lists the active experts;
//   2. gate/up: h[t, slot, f] = w * SiLU(W_g[f] x_t) * (W_u[f] x_t), units of 16
//      features of one expert.  The routing weight w is applied here, so that
//   -- grid barrier (E4M3, mx4: h is scaled to f16 like x, and another barrier) --
//   3. the down projection is ONE sum per output: y[t, n] = sum over the active
//      experts and their features of W_d[n, f] h[t, slot, f], units of 16 outputs
//      over all experts; fp32 throughout, rounded once, no atomics: reproducible.
//
// The products run on mma.sync with the 16 weight rows as M and the tokens (8
// columns, two blocks of them above 8 tokens) as N; at these sizes the tensor core
// is idle most of the time and what counts is the bytes in flight and the
// instructions per weight byte.
//   bytes: every warp streams its pieces (16 rows x 64 bytes) through a ring of its own
//     in shared memory by cp.async, kDecStages stages of two pieces deep, over unit
//     boundaries and, for the down projection's first pieces, from before the barrier:
//     no block-wide step waits for memory.
//   instructions: bf16 weights go to m16n8k16 as they are, E4M3 and mx4 codes are
//     converted to f16 (exactly) two at a time.  For those the tokens' values are f16
//     under a power of two per 128 columns, the largest in [2^14, 2^15), which holds a
//     bf16 exactly down to 2^-31 of it: a channel far above the others costs them nothing.
//     (E4M3 codes as they are, with x and h as two E4M3 terms under one scale, held the
//     others to 2^-18 of it, and were slower too: 4 tokens at d = 4096, I = 1536, E = 64,
//     k = 6 103 us against 97, 16 tokens 195 against 181.)
//     8 tokens at d = 8192, I = 2048, E = 512, k = 10, mx4: with the codes converted to
//     bf16 by bit moves (20 operations per 8 codes at half rate) and fragments loaded
//     straight into registers 852 us.
// An expert's product has one column per token that chose it, so that the second block
// of eight is computed only where more than eight did (16 tokens at d = 4096, I = 1536,
// E = 64, k = 6, both kernels: E4M3 187 us, mx4 157; with a column per token 265 and
// 211); the down projection
// adds an expert's columns to its tokens' sums in shared memory.
//
// A team of kw warps shares a unit, splitting its K pieces, and adds its parts
// through shared memory in warp order; kw is picked per phase from the unit and
// piece counts (team_warps).
#pragma once
#include "common.cuh"
#include "mx4.cuh"
#include "ptx.cuh"

namespace moe {

constexpr int kDecodeMaxT = 16;
constexpr int kDecodeThreads = 512;
constexpr int kDecodeWarps = kDecodeThreads / 32;
constexpr int kDecodeMaxSplit = 16;  // slices of d in the router's partial logits
constexpr int kDecStages = 3;        // ring stages of a warp
constexpr int kDecPiece = 16 * 64;   // bytes of a piece
constexpr int kDecScales = 64;       // bytes of its scales
constexpr int kDecStage = 2 * (kDecPiece + kDecScales);
enum : unsigned { kKernDecode = 4 };

// Dynamic shared memory with nb blocks of 8 token columns: the rings, and a
// buffer of every warp's partial sums.
constexpr int decode_smem(int nb) { return kDecodeWarps * (kDecStages * kDecStage + 2 * nb * 4 * 32 * 4); }

struct DecodeArgs {
  int T, d, E, k, I, I_s;
  const bf16* x;        // [T, d] the block's input
  const bf16* gamma;    // [d] RMSNorm weight, or NULL
  float eps;
  double inv_d;         // 1 / d
  const bf16* gate_w;   // [d] shared expert's gate, or NULL
  const bf16* w_router; // [E, d]
  const float* bias;    // [E] or NULL
  const uint8_t *wg, *wu, *wd, *sg, *su, *sd;
  const uint8_t* sc[6]; // scale parts: gate, up, down, shared gate, up, down
  float* gate;          // [T] weight of the shared expert, or NULL (1)
  bf16* xn;             // [T, d] the normalised input (bf16 weights with a norm)
  uint8_t* xq;          // [T][d / 32][64] x as scaled f16 (dec_split)
  float* xsc;           // [d / 128][kDecodeMaxT] its scales
  float* logits;        // [splits][T][E] partial logits
  int splits;
  void* h;              // [T, k + 1, ldh] bf16, or fp32 where h is scaled before the down projection
  uint8_t* hq;          // [T * (k + 1)][ldh / 32][64] h, scaled likewise
  float* hsc;           // [T * (k + 1)][ldh / 128] its scales
  int ldh;
  int32_t* ids;         // [T, k] or NULL
  float* tw;            // [T, k] or NULL
  bf16* y;              // [T, d]
  unsigned* bar;        // grid-barrier counter, zeroed by k_decode_route
  unsigned* status;
};

// -------------------------------------------------------------- weight types
// PC: K columns of a piece (64 bytes of a row); BV: 16-byte vectors of token data
// a lane holds per piece.
enum { kDecBf16 = 0, kDecFp8 = 1, kDecMx4 = 2 };
template <int W>
struct DecW {
  static constexpr int PC = W == kDecBf16 ? 32 : W == kDecFp8 ? 64 : 128;
  static constexpr int BV = W == kDecBf16 ? 1 : W == kDecFp8 ? 2 : 4;
  static constexpr bool SCALED = W != kDecBf16;  // token values under a scale per 128 columns
  static __device__ __forceinline__ int64_t bytes(int64_t n) { return W == kDecBf16 ? 2 * n : W == kDecFp8 ? n : n >> 1; }
};

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {  // d = A * B
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// Four 8x8 tiles of 16-bit elements, one row address a lane: word c of row g of each.
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ uint32_t lds32(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ void lds128(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
// 16 bytes global -> shared past L1 (zeros where ok is false), the rest of a 256-byte
// piece of the row to L2 with them (four tokens on E4M3 weights 117 -> 111 us); 4 bytes.
__device__ __forceinline__ void dec_copy16(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16u : 0u) : "memory");
}
__device__ __forceinline__ void dec_copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void dec_copy4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

// -------------------------------------------------------------- pieces
// A piece's rows are 64 bytes apart in shared memory, its 16-byte units swizzled
// so that a fragment load meets every bank once.
__device__ __forceinline__ uint32_t dec_unit(int row, int u) { return row * 64 + ((u ^ ((row >> 1) & 3)) << 4); }

// Bytes from the start of a matrix of K columns to row r, lane unit c, of piece 0.
template <int W>
__device__ __forceinline__ int64_t dec_row_at(int r, int K, int c) {
  return DecW<W>::bytes((int64_t)r * K) + c * 16;
}
// Copy 16 rows x 64 bytes at q (row g, this lane's unit) to slot `at`; step8: bytes of
// eight rows.  Only bf16 matrices end inside a piece: ok0, ok8 (rows g, g + 8 and the
// lane's columns exist).
template <int W>
__device__ __forceinline__ void dec_issue(uint32_t at, const uint8_t* q, int64_t step8, bool ok0, bool ok8) {
  if (W == kDecBf16) {
    dec_copy16(at, q, ok0);
    dec_copy16(at + 512, ok8 ? q + step8 : q, ok8);
  } else {
    dec_copy16(at, q);
    dec_copy16(at + 512, q + step8);
  }
}

// A piece's fragment: rows g (lo) and g + 8 (hi).  bf16: the lane's own 16 bytes (the
// K order inside a fragment is free as long as both operands share it); else word c of
// each 16-byte unit.  s0, s8: mx4, the scale bytes of the rows; E4M3, s0 the scale.
struct DecFrag {
  uint32_t lo[4], hi[4], s0, s8;
};
template <int W>
__device__ __forceinline__ void dec_read(DecFrag& f, uint32_t at, uint32_t sc_at, int lane) {
  if (W == kDecBf16) {
    const uint32_t d = at + dec_unit(lane >> 2, lane & 3);
    lds128(f.lo, d);
    lds128(f.hi, d + 512);
    f.s0 = f.s8 = 0;
  } else {
    const uint32_t d = at + dec_unit(lane & 7, lane >> 3);
    ldmatrix4(f.lo, d);
    ldmatrix4(f.hi, d + 512);
    f.s0 = lds32(sc_at + (W == kDecMx4 ? (lane >> 2) * 4 : 0));
    f.s8 = W == kDecMx4 ? lds32(sc_at + (lane >> 2) * 4 + 32) : 0u;
  }
}

// Eight mx4 codes -> four f16 pairs of consecutive values.
__device__ __forceinline__ void mx4_to_f16(uint32_t q, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(q));
}
// Four E4M3 codes -> two f16 pairs of consecutive values.
__device__ __forceinline__ void e4m3_to_f16(uint32_t q, uint32_t (&h)[2]) {
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(h[0]), "=r"(h[1])
      : "r"(q));
}
// Some byte of w is 0 or 255.
__device__ __forceinline__ bool has_edge_byte(uint32_t w) {
  return (((w - 0x01010101u) & ~w) | ((~w - 0x01010101u) & w)) & 0x80808080u;
}

// acc[nb] += A * B over one piece.  bw[nb]: the lane's token data; xs[nb]: scales of
// its two token columns.
template <int W, int NB>
__device__ __forceinline__ void dec_mma(float (&acc)[NB][4], const DecFrag& f, const uint4 (&bw)[NB][DecW<W>::BV],
                                        const float2 (&xs)[NB]) {
  if (W == kDecBf16) {
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
        mma_bf16(acc[nb], f.lo[0], f.hi[0], f.lo[1], f.hi[1], bw[nb][0].x, bw[nb][0].y);
        mma_bf16(acc[nb], f.lo[2], f.hi[2], f.lo[3], f.hi[3], bw[nb][0].z, bw[nb][0].w);
      }
  } else if (W == kDecFp8) {
    const float sc = __uint_as_float(f.s0);
    float p[NB][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // 16 columns
      uint32_t l[2], h[2];
      e4m3_to_f16(f.lo[i], l);
      e4m3_to_f16(f.hi[i], h);
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const uint4 b = bw[nb][(i >> 1) % DecW<W>::BV];
        if (i == 0) mma_f16_first(p[nb], l[0], h[0], l[1], h[1], b.x, b.y);
        else mma_f16(p[nb], l[0], h[0], l[1], h[1], i & 1 ? b.z : b.x, i & 1 ? b.w : b.y);
      }
    }
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const float s0 = sc * xs[nb].x, s1 = sc * xs[nb].y;
      acc[nb][0] = fmaf(s0, p[nb][0], acc[nb][0]);
      acc[nb][1] = fmaf(s1, p[nb][1], acc[nb][1]);
      acc[nb][2] = fmaf(s0, p[nb][2], acc[nb][2]);
      acc[nb][3] = fmaf(s1, p[nb][3], acc[nb][3]);
    }
  } else {
    float s0[4], s8[4];
    if (__any_sync(0xffffffffu, has_edge_byte(f.s0) || has_edge_byte(f.s8))) {
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        s0[b] = __uint_as_float(mx4_scale_bits(f.s0 >> (8 * b) & 255u));
        s8[b] = __uint_as_float(mx4_scale_bits(f.s8 >> (8 * b) & 255u));
      }
    } else {
#pragma unroll
      for (int b = 0; b < 4; ++b) {  // the byte at the top, under the sign
        s0[b] = __uint_as_float(__byte_perm(f.s0, 0, b << 12 | 0x444) >> 1);
        s8[b] = __uint_as_float(__byte_perm(f.s8, 0, b << 12 | 0x444) >> 1);
      }
    }
    float sum[NB][4];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int i = 0; i < 4; ++i) sum[nb][i] = 0.f;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      uint32_t l[4], h[4];
      mx4_to_f16(f.lo[b], l);
      mx4_to_f16(f.hi[b], h);
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
          const uint4 t = bw[nb][b % DecW<W>::BV];
          float p[4];
          mma_f16_first(p, l[0], h[0], l[1], h[1], t.x, t.y);
          mma_f16(p, l[2], h[2], l[3], h[3], t.z, t.w);
          sum[nb][0] = fmaf(s0[b], p[0], sum[nb][0]);
          sum[nb][1] = fmaf(s0[b], p[1], sum[nb][1]);
          sum[nb][2] = fmaf(s8[b], p[2], sum[nb][2]);
          sum[nb][3] = fmaf(s8[b], p[3], sum[nb][3]);
        }
    }
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[nb][i] = fmaf(i & 1 ? xs[nb].y : xs[nb].x, sum[nb][i], acc[nb][i]);
  }
}

// Token data of piece kc for the lane's token column (p: its row).
template <int W>
__device__ __forceinline__ void dec_tok(uint4 (&bw)[DecW<W>::BV], const uint8_t* p, int kc, int K, int c) {
  // bf16: 8 columns a lane, zeros past the last (they meet the weights' zeros); scaled:
  // 16 bytes a lane and 32-column block
#pragma unroll
  for (int i = 0; i < DecW<W>::BV; ++i) {
    const uint4* q = reinterpret_cast<const uint4*>(p + (kc * DecW<W>::BV + i) * 64 + c * 16);
    if (W != kDecBf16 || kc * 32 + c * 8 < K) bw[i] = *q;
    else bw[i] = make_uint4(0u, 0u, 0u, 0u);
  }
}

// -------------------------------------------------------------- scaled tokens
// Four consecutive values a lane, 128 columns a warp: as f16 to q (the 128 columns'
// 256 bytes), the scale to *sc.  A block holding an infinity or a NaN becomes NaN.
// A lane c of a product takes 16 bytes of each 32 columns: mx4 columns 8c .. 8c + 7 (the
// codes of a 32-bit word), E4M3 4c .. 4c + 3 and 16 + 4c .. (a word each).
template <int W>
__device__ __forceinline__ void dec_split(const float (&v)[4], uint8_t* q, float* sc, int lane) {
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) amax = max(amax, __float_as_uint(v[i]) & 0x7fffffffu);
  amax = __reduce_max_sync(0xffffffffu, amax);
  const float nan = __uint_as_float(0x7fffffffu);
  const uint32_t e = max(amax >> 23, 15u);
  const float inv = e == 255u ? nan : __uint_as_float((268u - e) << 23);  // 2^(14 - exponent)
  const __half2 a = __floats2half2_rn(v[0] * inv, v[1] * inv), b = __floats2half2_rn(v[2] * inv, v[3] * inv);
  const int at = W == kDecMx4 ? lane * 8 : (lane >> 3) * 64 + (lane & 3) * 16 + (lane >> 2 & 1) * 8;
  *reinterpret_cast<uint2*>(q + at) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  if (lane == 0) *sc = e == 255u ? nan : __uint_as_float((e - 14u) << 23);
}

// Barrier of the cooperative grid, in two halves: writes before a CTA's arrival are
// visible to every thread after the wait.  What a CTA can do without the others' writes
// (starting the next copies) goes between; before the arrival it would hold up the
// release.  Bounded as every wait of the library; false: a CTA did not come.
__device__ __forceinline__ void dec_grid_arrive(unsigned* bar) {
  __syncthreads();
  if (threadIdx.x == 0) asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(bar) : "memory");
}
__device__ __forceinline__ bool dec_grid_wait(unsigned* bar, unsigned n, unsigned* status, int* s_ok) {
  if (threadIdx.x == 0) {
    const unsigned want = n * gridDim.x;
    const long long t0 = clock64();
    int ok = 1;
    for (unsigned i = 1;; ++i) {
      unsigned v;
      asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(bar) : "memory");
      if (v >= want) break;
      if ((i & 15u) == 0 && clock64() - t0 > wait_limit()) {
        atomicCAS(status, 0u, kStatusTimeoutBase | (kKernDecode << 8) | n);
        ok = 0;
        break;
      }
    }
    *s_ok = ok;
  }
  __syncthreads();
  return *s_ok != 0;
}

// Warps per team for `units` units of `chunks` K chunks: the fewest rounds of
// chunks, a split costing about one chunk for the reduction.
// One warp; every lane returns it (lane i weighs 2^i warps).
__device__ __forceinline__ int team_warps(unsigned units, unsigned chunks, unsigned grid) {
  const unsigned lane = threadIdx.x & 31;
  unsigned key = ~0u;
  if (1u << lane <= (unsigned)kDecodeWarps) {
    const unsigned teams = grid * (kDecodeWarps >> lane);
    const unsigned cost = (units + teams - 1) / teams * (((chunks + (1u << lane) - 1) >> lane) + (lane > 0 ? 1 : 0));
    key = min(cost, ~0u >> 3) << 3 | lane;  // (of equal costs the fewest warps)
  }
  return 1 << (__reduce_min_sync(0xffffffffu, key) & 7u);
}

// f<1>() or f<2>(): a block of columns is computed only where an expert has them (NB: the
// most there can be), with registers for as many.
template <int NB, typename F>
__device__ __forceinline__ void dec_blocks(int cols, F f) {
  if (NB == 1 || cols <= 8) f.template operator()<1>();
  else f.template operator()<NB>();
}

__device__ __forceinline__ void team_sync(int team, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "r"(threads) : "memory");
}

struct DecShared {
  int32_t ids[kDecodeMaxT][kMaxK];
  float w[kDecodeMaxT][kMaxK];
  int32_t act[kDecodeMaxT * kMaxK];                // active experts, ascending
  uint8_t col[kDecodeMaxT * kMaxK][kDecodeMaxT];   // its columns: token | slot << 4, tokens ascending
  uint32_t mask[kDecodeMaxT * kMaxK];              // tokens of an active expert, one bit each
  int32_t flag[512];
  int32_t rank[512];
  int32_t wsum[kDecodeWarps];
  // down projection: the active experts' (then the shared expert's) matrices and scales
  const uint8_t* wd[kDecodeMaxT * kMaxK + 1];
  const uint8_t* sc[kDecodeMaxT * kMaxK + 1];
  int n_act, ok;
};

__device__ __forceinline__ float dec_warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Top k of one token's logits by one warp: k rounds of (largest key, lowest
// expert holding it).  Keys order as the logits; NaN sorts below every number.
template <int NPL>
__device__ __forceinline__ void dec_topk(const float* logits, int E, int k, int t, DecShared& s) {
  const int lane = threadIdx.x & 31;
  float l[NPL];
  uint32_t key[NPL];
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    const int e = lane + 32 * i;
    l[i] = e < E ? logits[e] : 0.f;
    const uint32_t u = __float_as_uint(l[i]);
    // order-preserving map, kept above 0 (taken or absent) and 1 (NaN)
    uint32_t q = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
    if (l[i] != l[i]) q = 1u;
    key[i] = e < E ? q : 0u;
  }
  // the lane's best and its lowest holder; only the lane that loses it looks again
  uint32_t best;
  unsigned at;
  auto look = [&]() {
    best = key[0];
    at = lane;
#pragma unroll
    for (int i = 1; i < NPL; ++i)
      if (key[i] > best) {
        best = key[i];
        at = lane + 32 * i;
      }
  };
  look();
  unsigned my_e = 0;
  for (int j = 0; j < k; ++j) {
    const uint32_t top = __reduce_max_sync(0xffffffffu, best);
    const unsigned e = __reduce_min_sync(0xffffffffu, best == top && at < (unsigned)E ? at : 0xffffffffu);
    if (lane == j) my_e = e;
    if (e == at) {
#pragma unroll
      for (int i = 0; i < NPL; ++i)
        if (e == (unsigned)(lane + 32 * i)) key[i] = 0u;
      look();
    }
  }
  const float mine = lane < k ? logits[my_e] : 0.f, top = __shfl_sync(0xffffffffu, mine, 0);
  const float p = lane < k ? expf(mine - top) : 0.f;
  const float den = dec_warp_sum(p);
  if (lane < k) {
    s.ids[t][lane] = (int)my_e;
    s.w[t][lane] = p / den;
  }
}

// -------------------------------------------------------------- norm, gate, logits
// v * (r.x + r.y) * (1 + gamma), what each operation rounds off carried along: a value
// that fp32 puts on the other side of the middle of two bf16 moves a logit by 2^-8 of
// its term, and so which experts are taken.
__device__ __forceinline__ float dec_norm(float v, float gamma, float2 r) {
  const float t = 1.0f + gamma, tl = gamma - (t - 1.0f);
  const float p = v * r.x, pl = fmaf(v, r.y, fmaf(v, r.x, -p));
  const float q = p * t, s = q + fmaf(p, tl, fmaf(pl, t, fmaf(p, t, -q)));
  return isfinite(q) ? s : q;
}
// Eight values of x, normalised and rounded to bf16.
__device__ __forceinline__ uint4 dec_norm8(uint4 x, uint4 gamma, float2 r) {
  const uint32_t a[4] = {x.x, x.y, x.z, x.w}, g[4] = {gamma.x, gamma.y, gamma.z, gamma.w};
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    o[i] = pack_bf16x2(dec_norm(__uint_as_float(a[i] << 16), __uint_as_float(g[i] << 16), r),
                       dec_norm(__uint_as_float(a[i] & 0xffff0000u), __uint_as_float(g[i] & 0xffff0000u), r));
  return make_uint4(o[0], o[1], o[2], o[3]);
}
template <int W, int NB>
__global__ void __launch_bounds__(kDecodeThreads, 1) k_decode_route(const DecodeArgs a) {
  pdl_begin();  // after the previous kernel in the stream (programmatic launch)
  __shared__ float2 s_r[kDecodeMaxT];  // 1 / rms and what its rounding to fp32 took off
  __shared__ double s_sq[kDecodeWarps];
  __shared__ float s_part[kDecodeWarps];
  __shared__ float red[kDecodeWarps][NB * 128];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, c = lane & 3;
  if (blockIdx.x == 0 && tid == 0) *a.bar = 0;
  const uint4* gam = reinterpret_cast<const uint4*>(a.gamma);
  if (a.gamma) {  // 1 / rms of every token, in every CTA alike: the warps share the tokens out
    int wpt = 16;  // warps of a token
    while (wpt * a.T > kDecodeWarps) wpt >>= 1;
    const int t = warp / wpt;
    float ss = 0.f, sl = 0.f;  // the sum of squares, and what its additions rounded off
    if (t < a.T) {
      const uint4* row = reinterpret_cast<const uint4*>(a.x + (int64_t)t * a.d);
#pragma unroll 4
      for (int j = warp % wpt * 32 + lane; j < a.d / 8; j += wpt * 32) {
        const uint4 v = __ldg(row + j);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        float s8 = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float p = __uint_as_float(w[i] << 16), q = __uint_as_float(w[i] & 0xffff0000u);
          s8 = fmaf(p, p, s8);
          s8 = fmaf(q, q, s8);
        }
        const float sum = ss + s8, back = sum - ss;
        sl += (ss - (sum - back)) + (s8 - back);
        ss = sum;
      }
    }
    double sq = isfinite(ss) ? (double)ss + sl : ss;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
    if (lane == 0) s_sq[warp] = sq;
    __syncthreads();
    if (tid < a.T) {
      double v = 0.0;
      for (int w = 0; w < wpt; ++w) v += s_sq[tid * wpt + w];
      const double m = v * a.inv_d + a.eps;
      const float r = 1.0f / sqrtf((float)m);
      // (one Newton step from r, whose second term is what r lacks)
      s_r[tid] = make_float2(r, r > 0.f && isfinite(r) ? (float)(0.5 * r * (1.0 - m * r * r)) : 0.f);
    }
    __syncthreads();
  }
  auto input8 = [&](int t, int v) {  // vector v of token t's (normalised) row
    const uint4 x = __ldg(reinterpret_cast<const uint4*>(a.x + (int64_t)t * a.d) + v);
    return a.gamma ? dec_norm8(x, __ldg(gam + v), s_r[t]) : x;
  };
  // partial logits: units of 16 experts and a slice of d
  const int tiles = (a.E + 15) >> 4;
  const int nch = (a.d + 31) >> 5;
  const int per = (nch + a.splits - 1) / a.splits;
  for (int u = blockIdx.x; u < tiles * a.splits; u += gridDim.x) {
    const int et = u % tiles, sp = u / tiles;
    const bool ok0 = et * 16 + g < a.E, ok8 = et * 16 + g + 8 < a.E;
    const uint4* w0 = reinterpret_cast<const uint4*>(a.w_router + (int64_t)(et * 16 + g) * a.d);
    const uint4* w8 = w0 + a.d;  // eight rows of d / 8 vectors
    float acc[NB][4];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[nb][i] = 0.f;
    const int k1 = min(nch, (sp + 1) * per);
    const uint4 z = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll 2
    for (int kc = sp * per + warp; kc < k1; kc += kDecodeWarps) {
      const int v = kc * 4 + c;
      const bool kok = v * 8 < a.d;
      const uint4 l = kok && ok0 ? __ldg(w0 + v) : z, h = kok && ok8 ? __ldg(w8 + v) : z;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const int t = nb * 8 + g;
        const uint4 b = t < a.T && kok ? input8(t, v) : z;
        mma_bf16(acc[nb], l.x, h.x, l.y, h.y, b.x, b.y);
        mma_bf16(acc[nb], l.z, h.z, l.w, h.w, b.z, b.w);
      }
    }
    __syncthreads();  // the previous unit's sums have been read
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int i = 0; i < 4; ++i) red[warp][(nb * 4 + i) * 32 + lane] = acc[nb][i];
    __syncthreads();
    for (int q = tid; q < NB * 128; q += kDecodeThreads) {
      float v = 0.f;
      for (int w = 0; w < kDecodeWarps; ++w) v += red[w][q];
      const int ln = q & 31, i = (q >> 5) & 3, nb = q >> 7;
      const int e = et * 16 + (ln >> 2) + (i >> 1) * 8, t = nb * 8 + (ln & 3) * 2 + (i & 1);
      if (e < a.E && t < a.T) a.logits[((int64_t)sp * a.T + t) * a.E + e] = v;
    }
  }
  // the products' input, and the shared expert's gate; the last warps of the grid first
  const int gw = (gridDim.x - 1 - blockIdx.x) * kDecodeWarps + warp, gn = gridDim.x * kDecodeWarps;
  if (DecW<W>::SCALED) {
    const int nk = a.d >> 7;
    for (int i = gw; i < a.T * nk; i += gn) {
      const int t = i / nk, kb = i % nk;
      const int at = kb * 128 + lane * 4;
      const uint2 x = __ldg(reinterpret_cast<const uint2*>(a.x + (int64_t)t * a.d + at));
      uint32_t w[2] = {x.x, x.y};
      if (a.gamma) {
        const uint2 gm = __ldg(reinterpret_cast<const uint2*>(a.gamma + at));
        const uint4 n = dec_norm8(make_uint4(x.x, x.y, 0u, 0u), make_uint4(gm.x, gm.y, 0u, 0u), s_r[t]);
        w[0] = n.x;
        w[1] = n.y;
      }
      const float v[4] = {__uint_as_float(w[0] << 16), __uint_as_float(w[0] & 0xffff0000u), __uint_as_float(w[1] << 16),
                          __uint_as_float(w[1] & 0xffff0000u)};
      dec_split<W>(v, a.xq + (int64_t)i * 256, a.xsc + kb * kDecodeMaxT + t, lane);
    }
  } else if (a.gamma) {
    const int n8 = a.d >> 3;
    for (int i = gw * 32 + lane; i < a.T * n8; i += gn * 32)
      reinterpret_cast<uint4*>(a.xn)[i] = input8(i / n8, i % n8);
  }
  if (a.gate)  // a CTA per token, from the grid's end
    for (int t = gridDim.x - 1 - blockIdx.x; t < a.T; t += gridDim.x) {
      float z = 0.f;
      for (int j = tid; j < a.d / 8; j += kDecodeThreads) {
        const uint4 x = input8(t, j), w = __ldg(reinterpret_cast<const uint4*>(a.gate_w) + j);
        const uint32_t p[4] = {x.x, x.y, x.z, x.w}, q[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          z = fmaf(__uint_as_float(p[i] << 16), __uint_as_float(q[i] << 16), z);
          z = fmaf(__uint_as_float(p[i] & 0xffff0000u), __uint_as_float(q[i] & 0xffff0000u), z);
        }
      }
      z = dec_warp_sum(z);
      __syncthreads();  // s_part has been read
      if (lane == 0) s_part[warp] = z;
      __syncthreads();
      if (tid == 0) {
        float v = 0.f;
        for (int w = 0; w < kDecodeWarps; ++w) v += s_part[w];
        a.gate[t] = 1.0f / (1.0f + expf(-v));
      }
    }
}

// -------------------------------------------------------------- experts
// NB: blocks of 8 token columns (1 for T <= 8, 2 up to kDecodeMaxT).
template <int W, int NB>
__global__ void __launch_bounds__(kDecodeThreads, 1) k_decode(const DecodeArgs a) {
  constexpr int PC = DecW<W>::PC, BV = DecW<W>::BV, D = kDecStages;
  constexpr int RED = 2 * NB * 4 * 32;  // floats a warp hands to its team
  extern __shared__ __align__(128) uint8_t dyn[];
  __shared__ DecShared s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, c = lane & 3;
  float* red_all = reinterpret_cast<float*>(dyn + kDecodeWarps * D * kDecStage);

  // ---- 1. routing, in every CTA alike (the logits in the rings' place)
  {
    float* lg = reinterpret_cast<float*>(dyn);
    static_assert(kDecodeMaxT * 512 * 4 <= kDecodeWarps * D * kDecStage, "logits");
    const int n = a.T * a.E;
    for (int i = tid; i < n; i += kDecodeThreads) {
      float v = a.bias ? __ldg(a.bias + i % a.E) : 0.f;
      for (int p0 = 0; p0 < a.splits; p0 += 8) {  // eight in flight, added in order
        float part[8];
#pragma unroll
        for (int p = 0; p < 8; ++p) part[p] = p0 + p < a.splits ? __ldcg(a.logits + (p0 + p) * n + i) : 0.f;
#pragma unroll
        for (int p = 0; p < 8; ++p)
          if (p0 + p < a.splits) v += part[p];
      }
      lg[i] = v;
    }
    s.flag[tid] = 0;
    if (tid < kDecodeMaxT * kMaxK) s.mask[tid] = 0;
    __syncthreads();
    if (warp < a.T) {
      const float* l = lg + warp * a.E;
      if (a.E <= 128) dec_topk<4>(l, a.E, a.k, warp, s);
      else if (a.E <= 256) dec_topk<8>(l, a.E, a.k, warp, s);
      else dec_topk<16>(l, a.E, a.k, warp, s);
      __syncwarp();
      if (lane < a.k) s.flag[s.ids[warp][lane]] = 1;
    }
    __syncthreads();
    const int f = s.flag[tid];
    const unsigned m = __ballot_sync(0xffffffffu, f);
    if (lane == 0) s.wsum[warp] = __popc(m);
    __syncthreads();
    int before = __popc(m & ((1u << lane) - 1u));
    for (int w = 0; w < warp; ++w) before += s.wsum[w];
    if (f) {
      s.act[before] = tid;
      s.rank[tid] = before;
    }
    if (tid == kDecodeThreads - 1) s.n_act = before + f;
    __syncthreads();
    if (tid < a.T * a.k) atomicOr(&s.mask[s.rank[s.ids[tid / a.k][tid % a.k]]], 1u << (tid / a.k));
    __syncthreads();
  }
  const int f_r = (a.I + 15) >> 4, f_s = (a.I_s + 15) >> 4;  // units of 16 features per expert
  const int nch_d = (a.d + PC - 1) / PC;
  const int nch_i = (a.I + PC - 1) / PC, nch_s = (a.I_s + PC - 1) / PC;
  const int nst_i = (nch_i + 1) >> 1, nst_s = (nch_s + 1) >> 1;  // down projection: stages of two pieces
  const int n_act = s.n_act;
  if (tid < a.T * a.k) {
    const int t = tid / a.k, j = tid % a.k, e = s.ids[t][j];
    s.col[s.rank[e]][__popc(s.mask[s.rank[e]] & ((1u << t) - 1u))] = (uint8_t)(t | j << 4);
    if (blockIdx.x == 0) {
      if (a.ids) a.ids[tid] = e;
      if (a.tw) a.tw[tid] = s.w[t][j];
    }
  }
  for (int i = tid; i <= n_act; i += kDecodeThreads) {
    const int64_t m = i < n_act ? s.act[i] : 0, block = (int64_t)(a.d >> 7) * (a.I >> 7);
    s.wd[i] = i < n_act ? a.wd + DecW<W>::bytes(m * a.d * a.I) : a.sd;
    s.sc[i] = i < n_act ? a.sc[2] + m * block * (W == kDecMx4 ? kMxTileBytes : 4) : a.sc[5];
  }
  const int kw1 = team_warps(n_act * f_r + f_s, nch_d, gridDim.x);
  const int kw2 = team_warps((a.d + 15) >> 4, n_act * nst_i + nst_s, gridDim.x);
  __syncthreads();
  const uint32_t ring = smem_u32(dyn) + warp * (D * kDecStage);
  int in_slot = 0, out_slot = 0;  // the stage to copy into, the stage to read

  // ---- 2. gate/up and SwiGLU: units of 16 features, the shared expert's first
  {
    const int kw = kw1, team = warp / kw, tw = warp % kw, tpc = kDecodeWarps / kw;
    const int units = f_s + n_act * f_r, step = gridDim.x * tpc;
    const uint8_t* xin = DecW<W>::SCALED ? a.xq : reinterpret_cast<const uint8_t*>(a.gamma ? a.xn : a.x);
    const int64_t xrow = (int64_t)a.d * 2;  // bytes of a token's row, bf16 or f16
    const int64_t step8 = DecW<W>::bytes((int64_t)8 * a.d);
    const uint32_t lane_at = dec_unit(g, c);
    int iu = tw < nch_d ? blockIdx.x + gridDim.x * team : units, ik = tw;
    const uint8_t *wg = nullptr, *wu = nullptr, *sp = nullptr;  // this lane's places in the next pieces
    bool ok0 = true, ok8 = true;
    auto enter = [&]() {
      if (iu >= units) return;
      const bool sh = iu < f_s;
      const int n0 = (sh ? iu : (iu - f_s) % f_r) * 16, N = sh ? a.I_s : a.I;
      const int64_t m = sh ? 0 : s.act[(iu - f_s) / f_r];
      ok0 = W != kDecBf16 || n0 + g < N;
      ok8 = W != kDecBf16 || n0 + g + 8 < N;
      const int64_t at = DecW<W>::bytes(m * N * a.d) + dec_row_at<W>(n0 + (ok0 ? g : 0), a.d, c) + (int64_t)tw * 64;
      wg = (sh ? a.sg : a.wg) + at;
      wu = (sh ? a.su : a.wu) + at;
      // lanes 0..15: gate's scales, 16..31: up's
      const int64_t kt = a.d >> 7, mt = m * (N >> 7) * kt;
      const uint8_t* sc = lane < 16 ? (sh ? a.sc[3] : a.sc[0]) : (sh ? a.sc[4] : a.sc[1]);
      if (W == kDecMx4) sp = sc + mt * kMxTileBytes + mx4_scale_at(n0 + (lane & 15), (int64_t)tw * 4, kt);
      if (W == kDecFp8) sp = sc + 4 * (mt + (n0 >> 7) * kt);
    };
    auto issue = [&]() {
      if (iu < units) {
        const uint32_t at = ring + in_slot * kDecStage;
        const bool kok = W != kDecBf16 || ik * 32 + c * 8 < a.d;
        dec_issue<W>(at + lane_at, wg, step8, kok && ok0, kok && ok8);
        dec_issue<W>(at + kDecPiece + lane_at, wu, step8, kok && ok0, kok && ok8);
        if (W == kDecMx4) dec_copy4(at + 2 * kDecPiece + lane * 4, sp);
        if (W == kDecFp8 && (lane & 15) == 0) dec_copy4(at + 2 * kDecPiece + lane * 4, sp + (ik >> 1) * 4);
        ik += kw;
        wg += kw * 64;
        wu += kw * 64;
        if (W == kDecMx4) sp += kw * kMxTileBytes;
        if (ik >= nch_d) {
          ik = tw;
          iu += step;
          enter();
        }
      }
      cp_async_commit();
      in_slot = in_slot + 1 == D ? 0 : in_slot + 1;
    };
    enter();
#pragma unroll 1
    for (int i = 0; i < D; ++i) issue();
    float* red = red_all + team * kw * RED;
    for (int u = blockIdx.x + gridDim.x * team; u < units; u += step) {
      const bool sh = u < f_s;
      const int ga = sh ? 0 : (u - f_s) / f_r;
      const int n0 = (sh ? u : (u - f_s) % f_r) * 16;
      const int N = sh ? a.I_s : a.I;
      const int cols = sh ? a.T : __popc(s.mask[ga]);  // tokens of the expert
      dec_blocks<NB>(cols, [&]<int NU>() {
        const uint8_t* tok[NU];
        const float *sc0[NU], *sc1[NU];  // scales of the lane's product columns 2c, 2c + 1 of the block
        // of column q; of one that does not exist the first's (the product's column is not used)
        auto token = [&](int q) { return sh ? (q < cols ? q : 0) : s.col[ga][q < cols ? q : 0] & 15; };
#pragma unroll
        for (int nb = 0; nb < NU; ++nb) {
          const int q = nb * 8 + g;
          tok[nb] = xin + token(q) * xrow;
          sc0[nb] = a.xsc + token(nb * 8 + 2 * c);
          sc1[nb] = a.xsc + token(nb * 8 + 2 * c + 1);
        }
        float ag[NU][4], au[NU][4];
#pragma unroll
        for (int nb = 0; nb < NU; ++nb)
#pragma unroll
          for (int i = 0; i < 4; ++i) ag[nb][i] = au[nb][i] = 0.f;
        for (int kc = tw; kc < nch_d; kc += kw) {
          uint4 bw[NU][BV];
          float2 xs[NU];
#pragma unroll
          for (int nb = 0; nb < NU; ++nb) {
            dec_tok<W>(bw[nb], tok[nb], kc, a.d, c);
            if (DecW<W>::SCALED) {
              const int at = (kc * PC >> 7) * kDecodeMaxT;
              xs[nb] = make_float2(__ldg(sc0[nb] + at), __ldg(sc1[nb] + at));
            }
          }
          cp_async_wait<D - 1>();
          __syncwarp();
          DecFrag fg, fu;
          const uint32_t at = ring + out_slot * kDecStage;
          dec_read<W>(fg, at, at + 2 * kDecPiece, lane);
          dec_read<W>(fu, at + kDecPiece, at + 2 * kDecPiece + kDecScales, lane);
          out_slot = out_slot + 1 == D ? 0 : out_slot + 1;
          __syncwarp();  // the stage has been read
          issue();
          dec_mma<W, NU>(ag, fg, bw, xs);
          dec_mma<W, NU>(au, fu, bw, xs);
        }
#pragma unroll
        for (int nb = 0; nb < NU; ++nb)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            red[tw * RED + (nb * 4 + i) * 32 + lane] = ag[nb][i];
            red[tw * RED + (NB * 4 + nb * 4 + i) * 32 + lane] = au[nb][i];
          }
      });
      if (kw > 1) team_sync(team, kw * 32);
      else __syncwarp();
      for (int q = tw * 32 + lane; q < (cols > 8 ? NB : 1) * 128; q += kw * 32) {
        float vg = 0.f, vu = 0.f;
        for (int w = 0; w < kw; ++w) {
          vg += red[w * RED + q];
          vu += red[w * RED + NB * 128 + q];
        }
        const int ln = q & 31, i = (q >> 5) & 3, nb = q >> 7;
        const int f = n0 + (ln >> 2) + (i >> 1) * 8, col = nb * 8 + (ln & 3) * 2 + (i & 1);
        if (f >= N || col >= cols) continue;
        const int t = sh ? col : s.col[ga][col] & 15, j = sh ? a.k : s.col[ga][col] >> 4;
        const float w = sh ? (a.gate ? __ldg(a.gate + t) : 1.f) : s.w[t][j];
        const float hv = w * (vg / (1.f + __expf(-vg)) * vu);
        const int64_t at = ((int64_t)t * (a.k + 1) + j) * a.ldh + f;
        // bf16 weights: h rounded to bf16, as the products of the fused forward take it.
        // (As the sum of two bf16 terms the outputs were off by 0.0017 of their norm, their
        // own rounding, in place of 0.0024, and 8 tokens at d = 4096, I = 1536, E = 64,
        // k = 6 took 244 us in place of 234.)
        if (DecW<W>::SCALED) static_cast<float*>(a.h)[at] = hv;
        else static_cast<bf16*>(a.h)[at] = __float2bfloat16_rn(hv);
      }
      if (kw > 1) team_sync(team, kw * 32);
      else __syncwarp();
    }
  }

  dec_grid_arrive(a.bar);

  // ---- 3. down projection: units of 16 outputs, K runs over every active expert,
  // two consecutive pieces of one expert a stage; a warp of a team takes a contiguous
  // range of the stages.  The first stages are copied before the barrier.
  {
    const int kw = kw2, team = warp / kw, tw = warp % kw, tpc = kDecodeWarps / kw;
    const int units = (a.d + 15) >> 4, step = gridDim.x * tpc;
    const int total = n_act * nst_i + nst_s, per = (total + kw - 1) / kw;
    const int p0 = tw * per, count = min(per, total - p0);  // this warp's stages of a unit (none: count <= 0)
    const int ga0 = min(p0 / nst_i, n_act), ks0 = p0 - ga0 * nst_i;
    const uint32_t lane_at = dec_unit(g, c);
    // the next stage to copy: unit, expert (n_act: the shared one), stage in the expert
    int iu = count > 0 ? blockIdx.x + gridDim.x * team : units, iga = 0, iks = 0, ileft = 0;
    const uint8_t *wp = nullptr, *sp = nullptr;  // this lane's places
    int64_t step8 = 0;
    bool ok0 = true, ok8 = true;
    auto expert = [&]() {
      const int K = iga < n_act ? a.I : a.I_s, n0 = iu * 16;
      step8 = DecW<W>::bytes((int64_t)8 * K);
      wp = s.wd[iga] + DecW<W>::bytes((int64_t)(n0 + (ok0 ? g : 0)) * K) + c * 16 + iks * 128;
      if (W == kDecMx4) sp = s.sc[iga] + mx4_scale_at(n0 + (lane & 15), (int64_t)(2 * iks + (lane >> 4)) * 4, K >> 7);
      if (W == kDecFp8) sp = s.sc[iga] + 4 * ((int64_t)(n0 >> 7) * (K >> 7) + iks);
    };
    auto enter = [&]() {
      if (iu >= units) return;
      ok0 = W != kDecBf16 || iu * 16 + g < a.d;
      ok8 = W != kDecBf16 || iu * 16 + g + 8 < a.d;
      iga = ga0;
      iks = ks0;
      ileft = count;
      expert();
    };
    auto issue = [&]() {
      if (iu < units) {
        const uint32_t at = ring + in_slot * kDecStage;
        const int K = iga < n_act ? a.I : a.I_s, nch = iga < n_act ? nch_i : nch_s;
        const bool two = 2 * iks + 1 < nch;
        const bool k0 = W != kDecBf16 || iks * 64 + c * 8 < K, k1 = W != kDecBf16 || iks * 64 + 32 + c * 8 < K;
        dec_issue<W>(at + lane_at, wp, step8, k0 && ok0, k0 && ok8);
        if (two) dec_issue<W>(at + kDecPiece + lane_at, wp + 64, step8, k1 && ok0, k1 && ok8);
        if (W == kDecMx4 && (two || lane < 16)) dec_copy4(at + 2 * kDecPiece + lane * 4, sp);
        if (W == kDecFp8 && (lane & 15) == 0) dec_copy4(at + 2 * kDecPiece + lane * 4, sp);
        wp += 128;
        sp += W == kDecMx4 ? 2 * kMxTileBytes : 4;
        if (--ileft == 0) {
          iu += step;
          enter();
        } else if (iga < n_act && ++iks == nst_i) {
          ++iga;
          iks = 0;
          expert();
        } else if (iga == n_act) {
          ++iks;
        }
      }
      cp_async_commit();
      in_slot = in_slot + 1 == D ? 0 : in_slot + 1;
    };
    enter();
#pragma unroll 1
    for (int i = 0; i < D; ++i) issue();
    if (!dec_grid_wait(a.bar, 1, a.status, &s.ok)) {
      cp_async_wait<0>();
      return;
    }
    const int ldt = a.ldh >> 7;
    if (DecW<W>::SCALED) {
      const int n = a.T * (a.k + 1) * ldt;
      for (int i = blockIdx.x * kDecodeWarps + warp; i < n; i += gridDim.x * kDecodeWarps) {
        const int r = i / ldt, kb = i % ldt;
        if (kb * 128 >= (r % (a.k + 1) == a.k ? a.I_s : a.I)) continue;
        const float4 x =
            __ldcg(reinterpret_cast<const float4*>(static_cast<const float*>(a.h) + (int64_t)r * a.ldh + kb * 128) + lane);
        const float v[4] = {x.x, x.y, x.z, x.w};
        dec_split<W>(v, a.hq + (int64_t)i * 256, a.hsc + i, lane);
      }
      dec_grid_arrive(a.bar);
      if (!dec_grid_wait(a.bar, 2, a.status, &s.ok)) {
        cp_async_wait<0>();
        return;
      }
    }
    const uint8_t* hin = DecW<W>::SCALED ? a.hq : reinterpret_cast<const uint8_t*>(a.h);
    const int64_t hrow = (int64_t)a.ldh * 2;
    float* red = red_all + team * kw * RED;
    for (int u = blockIdx.x + gridDim.x * team; u < units; u += step) {
      const int n0 = u * 16;
      float* sum = red + tw * RED;  // [token][16 outputs]
      for (int i = lane; i < NB * 128; i += 32) sum[i] = 0.f;
      __syncwarp();
      int ga = ga0, ks = ks0, left = count;
      while (left > 0) {  // an expert's stages
        const bool sh = ga >= n_act;
        const int K = sh ? a.I_s : a.I, nch = sh ? nch_s : nch_i;
        const int k1 = min(ks + left, sh ? nst_s : nst_i);
        const int cols = sh ? a.T : __popc(s.mask[ga]);  // tokens of the expert
        dec_blocks<NB>(cols, [&]<int NU>() {
          const uint8_t* tok[NU];
          const float *sc0[NU], *sc1[NU];  // scales of the lane's product columns 2c, 2c + 1 of the block
          auto row = [&](int q) {  // of h; a column that does not exist: the first column's
            const int v = sh ? (q < cols ? q : 0) | a.k << 4 : s.col[ga][q < cols ? q : 0];
            return (v & 15) * (a.k + 1) + (v >> 4);
          };
#pragma unroll
          for (int nb = 0; nb < NU; ++nb) {
            const int q = nb * 8 + g;
            tok[nb] = hin + row(q) * hrow;
            sc0[nb] = a.hsc + row(nb * 8 + 2 * c) * ldt;
            sc1[nb] = a.hsc + row(nb * 8 + 2 * c + 1) * ldt;
          }
          left -= k1 - ks;
          // an expert's part reaches only its own tokens' sums, an infinity or a NaN in its
          // weights too
          float part[NU][4];
#pragma unroll
          for (int nb = 0; nb < NU; ++nb)
#pragma unroll
            for (int r = 0; r < 4; ++r) part[nb][r] = 0.f;
          for (; ks < k1; ++ks) {
            uint4 bw[2][NU][BV];
            float2 xs[2][NU];
            const bool two = 2 * ks + 1 < nch;
#pragma unroll
            for (int nb = 0; nb < NU; ++nb) {
              dec_tok<W>(bw[0][nb], tok[nb], 2 * ks, K, c);
              dec_tok<W>(bw[1][nb], tok[nb], two ? 2 * ks + 1 : 2 * ks, K, c);
              if (DecW<W>::SCALED) {
                const int kb = 2 * ks * PC >> 7;  // (E4M3: both pieces are in it)
                xs[0][nb] = xs[1][nb] = make_float2(sc0[nb][kb], sc1[nb][kb]);
                if (W == kDecMx4 && two) xs[1][nb] = make_float2(sc0[nb][kb + 1], sc1[nb][kb + 1]);
              }
            }
            cp_async_wait<D - 1>();
            __syncwarp();
            DecFrag f0, f1;
            const uint32_t at = ring + out_slot * kDecStage;
            dec_read<W>(f0, at, at + 2 * kDecPiece, lane);
            dec_read<W>(f1, at + kDecPiece, at + 2 * kDecPiece + kDecScales, lane);
            out_slot = out_slot + 1 == D ? 0 : out_slot + 1;
            __syncwarp();  // the stage has been read
            issue();
            dec_mma<W, NU>(part, f0, bw[0], xs[0]);
            if (two) dec_mma<W, NU>(part, f1, bw[1], xs[1]);
          }
#pragma unroll
          for (int nb = 0; nb < NU; ++nb)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const int q = nb * 8 + 2 * c + (r & 1);
              if (q < cols) sum[(sh ? q : s.col[ga][q] & 15) * 16 + g + (r >> 1) * 8] += part[nb][r];
            }
        });
        __syncwarp();  // (the next expert's columns are other lanes' tokens)
        ++ga;
        ks = 0;
      }
      if (kw > 1) team_sync(team, kw * 32);
      else __syncwarp();
      for (int q = tw * 32 + lane; q < NB * 128; q += kw * 32) {
        float v = 0.f;
        for (int w2 = 0; w2 < kw; ++w2) v += red[w2 * RED + q];
        const int n = n0 + (q & 15), t = q >> 4;
        if (n < a.d && t < a.T) a.y[(int64_t)t * a.d + n] = __float2bfloat16_rn(v);
      }
      if (kw > 1) team_sync(team, kw * 32);
      else __syncwarp();
    }
  }
}

}  // namespace moe
