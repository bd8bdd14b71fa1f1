// decode.cuh -- the whole sparse MoE block for a few tokens in one kernel.
//
// With T <= kDecodeMaxT tokens the block reads every active expert's weights
// for one or two rows each: the time is the weight bytes over the HBM rate plus
// whatever latency the launches add, so one cooperative kernel (one CTA per SM)
// runs all of it, with two grid barriers:
//   1. router logits, split over (16 experts) x (slices of d): fp32 partials;
//   -- barrier --
//   2. every CTA adds the partials in slice order and selects each token's top k
//      (one warp per token; the same code and inputs, so the same result in every
//      CTA), and lists the active experts;
//   3. gate/up: h[t, slot, f] = w * SiLU(W_g[f] x_t) * (W_u[f] x_t) in bf16, units of 16
//      features of one expert.  The routing weight w is applied here, so that
//   -- barrier --
//   4. the down projection is ONE sum per output: y[t, n] = sum over the active
//      experts and their features of W_d[n, f] h[t, slot, f], units of 16 outputs
//      over all experts; fp32 throughout, rounded once, no atomics: reproducible.
//
// The products run on mma.sync.m16n8k16 (bf16, fp32 accumulate) with the 16
// weight rows as M and the tokens (8 columns, two blocks of them above 8 tokens)
// as N.  Weight fragments are loaded straight from global memory in 16-byte
// pieces, one row per lane group and four adjacent pieces per row: the K order
// inside a fragment is free as long as both operands share it, so lane c simply
// takes the c-th 16 bytes of the row's chunk.  At these sizes the kernel is bound by the bytes it
// keeps in flight, not by the tensor core (one m16n8k16 per 512 weight bytes), and
// registers as the landing place need no shared-memory round trip.
// E4M3 and mx4 codes become bf16 in registers by moving the code's exponent and
// mantissa bits under bf16's (exact) and one bf16 multiply by a power of two;
// E4M3 block scales multiply the fp32 sums of each 128-column block.
// Tokens an expert was not chosen for are zero columns of its product.
//
// A team of kw warps shares a unit, splitting its K chunks, and adds its parts
// through shared memory in warp order; kw is picked per phase from the unit and
// chunk counts (team_warps).
#pragma once
#include "common.cuh"
#include "mx4.cuh"
#include "ptx.cuh"

namespace moe {

constexpr int kDecodeMaxT = 16;
constexpr int kDecodeThreads = 512;
constexpr int kDecodeWarps = kDecodeThreads / 32;
constexpr int kDecodeMaxSplit = 16;  // slices of d in the router's partial logits
enum : unsigned { kKernDecode = 4 };

struct DecodeArgs {
  int T, d, E, k, I, I_s;
  const bf16* x;        // [T, d] the block's (normalised) input
  const bf16* w_router; // [E, d]
  const float* bias;    // [E] or NULL
  const uint8_t *wg, *wu, *wd, *sg, *su, *sd;
  const uint8_t* sc[6]; // scale parts: gate, up, down, shared gate, up, down
  const float* gate;    // [T] weight of the shared expert, or NULL (1)
  bf16* xs;             // [T, d] x in the weight type's K order (E4M3, mx4)
  float* logits;        // [splits][T][E] partial logits
  int splits;
  bf16* h;              // [T, k + 1, ldh]
  int ldh;
  int32_t* ids;         // [T, k] or NULL
  float* tw;            // [T, k] or NULL
  bf16* y;              // [T, d]
  unsigned* bar;        // grid-barrier counter, zero at launch
  unsigned* status;
};

// -------------------------------------------------------------- weight types
// LD: 16-byte pieces a lane loads per row and chunk; CH: K columns of a chunk;
// MM: mma steps per chunk; BW: 32-bit words of token data a lane holds per chunk.
enum { kDecBf16 = 0, kDecFp8 = 1, kDecMx4 = 2 };
template <int W>
struct DecW;
template <>
struct DecW<kDecBf16> {
  static constexpr int CH = 32, LD = 1, MM = 2, BW = 4;
  static __device__ __forceinline__ int64_t bytes(int64_t n) { return 2 * n; }
};
template <>
struct DecW<kDecFp8> {
  static constexpr int CH = 128, LD = 2, MM = 8, BW = 16;
  static __device__ __forceinline__ int64_t bytes(int64_t n) { return n; }
};
template <>
struct DecW<kDecMx4> {
  static constexpr int CH = 128, LD = 1, MM = 8, BW = 16;
  static __device__ __forceinline__ int64_t bytes(int64_t n) { return n >> 1; }
};

// Where element e of a row goes in the K order the converters below produce:
// E4M3 pairs codes (0, 2) and (1, 3) of a word, mx4 codes (i, i + 4).
template <int W>
__device__ __forceinline__ int dec_place(int e) {
  if (W == kDecFp8) return (e & ~3) | ((e & 1) << 1) | ((e >> 1) & 1);
  if (W == kDecMx4) return (e & ~7) | ((e & 3) << 1) | ((e >> 2) & 1);
  return e;
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// Four E4M3 codes -> bf16 pairs (codes 0, 2) and (codes 1, 3).  The seven low
// bits of a code, four places up in a bf16, read as code * 2^-120 (also for
// subnormal codes), so one multiply by 2^120 gives the value.
__device__ __forceinline__ void dec_e4m3x4(uint32_t q, uint32_t& p02, uint32_t& p13) {
  const uint32_t l = q << 8;
  const uint32_t a = (l & 0x80008000u) | ((l >> 4) & 0x07f007f0u);
  const uint32_t b = (q & 0x80008000u) | ((q >> 4) & 0x07f007f0u);
  p02 = mul_bf16x2(a, 0x7b807b80u);
  p13 = mul_bf16x2(b, 0x7b807b80u);
}
// Eight mx4 codes -> four bf16 pairs (i, i + 4), scaled: exponent and mantissa
// bits six places up read as code * 2^-126; m1 (and m2) make up 2^126 * scale.
__device__ __forceinline__ void dec_mx4x8(uint32_t q, uint32_t m1, uint32_t (&p)[4]) {
  p[0] = ((q << 12) & 0x80008000u) | ((q << 6) & 0x01c001c0u);
  p[1] = ((q << 8) & 0x80008000u) | ((q << 2) & 0x01c001c0u);
  p[2] = ((q << 4) & 0x80008000u) | ((q >> 2) & 0x01c001c0u);
  p[3] = (q & 0x80008000u) | ((q >> 6) & 0x01c001c0u);
#pragma unroll
  for (int i = 0; i < 4; ++i) p[i] = mul_bf16x2(p[i], m1);
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Weight bytes pass through once: no L1 allocation.
__device__ __forceinline__ uint4 ld_stream(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// One 16-row weight operand of a unit: this lane's rows are g and g + 8.
template <int W>
struct DecRows {
  const uint8_t* p;   // row g, this lane's piece of chunk 0
  int64_t step8;      // bytes from row g to row g + 8
  const uint8_t* sc;  // E4M3: fp32 scales of the row block; mx4: scale byte of row g, this lane's block, chunk 0
  bool ok0, ok8;      // rows inside the matrix
};
template <int W>
struct DecFrag {
  uint4 lo[DecW<W>::LD], hi[DecW<W>::LD];
  uint32_t s0, s8;  // E4M3: fp32 scale bits (s0); mx4: scale bytes of the two rows
};

// rows n0 .. n0 + 15 of matrix `m` [N, K] of the stack at w (scales sc)
template <int W>
__device__ __forceinline__ DecRows<W> dec_rows(const uint8_t* w, const uint8_t* sc, int64_t m, int N, int K, int n0,
                                               int g, int c) {
  DecRows<W> r;
  const int64_t row = m * N + n0 + g;
  r.p = w + DecW<W>::bytes(row * K) + c * 16;
  r.step8 = DecW<W>::bytes((int64_t)8 * K);
  r.ok0 = n0 + g < N;
  r.ok8 = n0 + g + 8 < N;
  if (W == kDecFp8)
    r.sc = sc + 4 * ((m * (N >> 7) + (n0 >> 7)) * (int64_t)(K >> 7));
  else if (W == kDecMx4)
    r.sc = sc + (m * (N >> 7)) * (int64_t)(K >> 7) * kMxTileBytes + mx4_scale_at(n0 + g, c, K >> 7);
  else
    r.sc = nullptr;
  return r;
}

// Chunk kc of the operand (kpiece: columns of this lane's piece that exist).
template <int W>
__device__ __forceinline__ void dec_load(DecFrag<W>& f, const DecRows<W>& r, int kc, bool kok) {
  const uint4 z = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
  for (int i = 0; i < DecW<W>::LD; ++i) {
    const uint8_t* q = r.p + (int64_t)kc * (64 * DecW<W>::LD) + i * 64;
    f.lo[i] = kok && r.ok0 ? ld_stream(q) : z;
    f.hi[i] = kok && r.ok8 ? ld_stream(q + r.step8) : z;
  }
  f.s0 = f.s8 = 0;
  if (W == kDecFp8) f.s0 = kok ? __ldg(reinterpret_cast<const uint32_t*>(r.sc) + kc) : 0u;
  if (W == kDecMx4 && kok) {
    f.s0 = __ldg(r.sc + (int64_t)kc * kMxTileBytes);
    f.s8 = __ldg(r.sc + (int64_t)kc * kMxTileBytes + 8 * 16);
  }
}

// acc[nb] += A * B over one chunk.  bw[nb]: the lane's token words.
template <int W, int NB>
__device__ __forceinline__ void dec_mma(float (&acc)[NB][4], const DecFrag<W>& f, const uint32_t (&bw)[NB][DecW<W>::BW],
                                        unsigned nbmask) {
  if (W == kDecBf16) {
    const uint32_t l[4] = {f.lo[0].x, f.lo[0].y, f.lo[0].z, f.lo[0].w};
    const uint32_t h[4] = {f.hi[0].x, f.hi[0].y, f.hi[0].z, f.hi[0].w};
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
      if (nbmask >> nb & 1u)
#pragma unroll
        for (int s = 0; s < 2; ++s)
          mma_bf16(acc[nb], l[2 * s], h[2 * s], l[2 * s + 1], h[2 * s + 1], bw[nb][2 * s], bw[nb][2 * s + 1]);
  } else if (W == kDecFp8) {
    float part[NB][4];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int i = 0; i < 4; ++i) part[nb][i] = 0.f;
    uint32_t nan_l = 0, nan_h = 0;  // bit 7 of a byte: a NaN code (0x7f, 0xff) was there
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t l[4] = {f.lo[i % DecW<W>::LD].x, f.lo[i % DecW<W>::LD].y, f.lo[i % DecW<W>::LD].z,
                             f.lo[i % DecW<W>::LD].w};
      const uint32_t h[4] = {f.hi[i % DecW<W>::LD].x, f.hi[i % DecW<W>::LD].y, f.hi[i % DecW<W>::LD].z,
                             f.hi[i % DecW<W>::LD].w};
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        uint32_t a0, a2, a1, a3;
        dec_e4m3x4(l[s], a0, a2);
        dec_e4m3x4(h[s], a1, a3);
        nan_l |= (l[s] & 0x7f7f7f7fu) + 0x01010101u;
        nan_h |= (h[s] & 0x7f7f7f7fu) + 0x01010101u;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
          if (nbmask >> nb & 1u)
            mma_bf16(part[nb], a0, a1, a2, a3, bw[nb][(i * 8 + 2 * s) % DecW<W>::BW],
                     bw[nb][(i * 8 + 2 * s + 1) % DecW<W>::BW]);
      }
    }
    const float sc = __uint_as_float(f.s0);
    const unsigned bad = ((nan_l & 0x80808080u) ? 1u : 0u) | ((nan_h & 0x80808080u) ? 2u : 0u);
    if (__any_sync(0xffffffffu, bad)) {  // the bit move reads them as 480: a row holding one is NaN
      unsigned row = bad | __shfl_xor_sync(0xffffffffu, bad, 1);
      row |= __shfl_xor_sync(0xffffffffu, row, 2);
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (row >> (i >> 1) & 1u) part[nb][i] = __int_as_float(0x7fffffff);
    }
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[nb][i] = fmaf(sc, part[nb][i], acc[nb][i]);
  } else {
    // 2^126 * scale as one bf16 factor while it is one (scale <= 2), else as two
    const bool big = f.s0 > 128u || f.s8 > 128u;
    uint32_t m0 = (min(f.s0, 128u) + 126u) << 7, m8 = (min(f.s8, 128u) + 126u) << 7;
    m0 |= m0 << 16;
    m8 |= m8 << 16;
    const bool any_big = __any_sync(0xffffffffu, big);
    const uint32_t l[4] = {f.lo[0].x, f.lo[0].y, f.lo[0].z, f.lo[0].w};
    const uint32_t h[4] = {f.hi[0].x, f.hi[0].y, f.hi[0].z, f.hi[0].w};
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      uint32_t a[4], b[4];
      dec_mx4x8(l[w], m0, a);
      dec_mx4x8(h[w], m8, b);
      if (any_big) {
        uint32_t e0 = f.s0 == 255u ? 0x7fffu : (max(f.s0, 128u) - 1u) << 7;
        uint32_t e8 = f.s8 == 255u ? 0x7fffu : (max(f.s8, 128u) - 1u) << 7;
        e0 |= e0 << 16;
        e8 |= e8 << 16;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          a[i] = mul_bf16x2(a[i], e0);
          b[i] = mul_bf16x2(b[i], e8);
        }
      }
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
          if (nbmask >> nb & 1u)
            mma_bf16(acc[nb], a[2 * s], b[2 * s], a[2 * s + 1], b[2 * s + 1],
                     bw[nb][(4 * w + 2 * s) % DecW<W>::BW], bw[nb][(4 * w + 2 * s + 1) % DecW<W>::BW]);
    }
  }
}

// Token words of one chunk for the lane's token (p: its row at this lane's
// piece of chunk 0, NULL: a zero column).  E4M3 pieces are 32 bf16 apart twice.
template <int W>
__device__ __forceinline__ void dec_tok(uint32_t (&bw)[DecW<W>::BW], const bf16* p, int kc, bool kok) {
  const uint4* q = reinterpret_cast<const uint4*>(p + (int64_t)kc * DecW<W>::CH);
#pragma unroll
  for (int i = 0; i < DecW<W>::BW / 4; ++i) {
    // bf16: 8 columns a lane; E4M3: 16 at c * 16 and 16 at 64 + c * 16; mx4: 32 at c * 32
    const int at = W == kDecFp8 ? (i & 1) + (i >> 1) * 8 : i;
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (p && kok) v = *(q + at);
    bw[4 * i] = v.x;
    bw[4 * i + 1] = v.y;
    bw[4 * i + 2] = v.z;
    bw[4 * i + 3] = v.w;
  }
}
// columns of a lane's first piece: the offset of its token data in a chunk
template <int W>
__device__ __forceinline__ int dec_tok_off(int c) {
  return c * (W == kDecMx4 ? 32 : W == kDecFp8 ? 16 : 8);
}

// All CTAs of the cooperative grid have reached round `n` (1, 2, ..) of the
// barrier.  Writes before it are visible to every thread after it.  Bounded as
// every wait of the library; false: a CTA did not come.
__device__ __forceinline__ bool dec_grid_barrier(unsigned* bar, unsigned n, unsigned* status, int* s_ok) {
  __syncthreads();
  if (threadIdx.x == 0) {
    const unsigned want = n * gridDim.x;
    __threadfence();
    atomicAdd(bar, 1u);
    const long long t0 = clock64(), lim = wait_limit();
    int ok = 1;
    for (;;) {
      unsigned v;
      asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(bar) : "memory");
      if (v >= want) break;
      if (clock64() - t0 > lim) {
        atomicCAS(status, 0u, kStatusTimeoutBase | (kKernDecode << 8) | n);
        ok = 0;
        break;
      }
    }
    __threadfence();
    *s_ok = ok;
  }
  __syncthreads();
  return *s_ok != 0;
}

// Warps per team for `units` units of `chunks` K chunks: the fewest rounds of
// chunks, a split costing about one chunk for the reduction.
__device__ __forceinline__ int team_warps(int units, int chunks, int grid) {
  int best = 1;
  int64_t cost = INT64_MAX;
  for (int kw = 1; kw <= kDecodeWarps; kw *= 2) {
    const int64_t teams = (int64_t)grid * (kDecodeWarps / kw);
    const int64_t c = cdiv(units, teams) * (cdiv(chunks, kw) + (kw > 1 ? 1 : 0));
    if (c < cost) {
      cost = c;
      best = kw;
    }
  }
  return best;
}

__device__ __forceinline__ void team_sync(int team, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "r"(threads) : "memory");
}

struct DecShared {
  int32_t ids[kDecodeMaxT][kMaxK];
  float w[kDecodeMaxT][kMaxK];
  int32_t act[kDecodeMaxT * kMaxK];                // active experts, ascending
  int8_t slot[kDecodeMaxT * kMaxK][kDecodeMaxT];   // slot of a token at an active expert, or -1
  uint32_t mask[kDecodeMaxT * kMaxK];              // tokens of an active expert, one bit each
  int32_t flag[512];
  int32_t rank[512];
  int32_t wsum[kDecodeWarps];
  int n_act, kw1, kw2, ok;
};

// Top k of one token's logits by one warp: k rounds of (largest key, lowest
// expert holding it).  Keys order as the logits; NaN sorts below every number.
template <int NPL>
__device__ __forceinline__ void dec_topk(const DecodeArgs& a, int t, DecShared& s) {
  const int lane = threadIdx.x & 31;
  float l[NPL];
  uint32_t key[NPL];
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    const int e = lane + 32 * i;
    l[i] = e < a.E && a.bias ? __ldg(a.bias + e) : 0.f;
  }
  for (int p = 0; p < a.splits; ++p) {
    const float* row = a.logits + ((int64_t)p * a.T + t) * a.E;
#pragma unroll
    for (int i = 0; i < NPL; ++i)
      if (lane + 32 * i < a.E) l[i] += __ldcg(row + lane + 32 * i);
  }
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    const uint32_t u = __float_as_uint(l[i]);
    // order-preserving map, kept above 0 (taken or absent) and 1 (NaN)
    uint32_t q = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
    if (l[i] != l[i]) q = 1u;
    key[i] = lane + 32 * i < a.E ? q : 0u;
  }
  float v0 = 0.f, den = 0.f, my_v = 0.f;
  int my_e = 0;
  for (int j = 0; j < a.k; ++j) {
    uint32_t best = 0;
#pragma unroll
    for (int i = 0; i < NPL; ++i) best = max(best, key[i]);
    const uint32_t top = __reduce_max_sync(0xffffffffu, best);
    unsigned cand = 0xffffffffu;
    float cv = 0.f;
#pragma unroll
    for (int i = NPL - 1; i >= 0; --i)
      if (key[i] == top && lane + 32 * i < a.E) {
        cand = lane + 32 * i;
        cv = l[i];
      }
    const unsigned e = __reduce_min_sync(0xffffffffu, cand);
    const float v = __shfl_sync(0xffffffffu, cv, e & 31);
#pragma unroll
    for (int i = 0; i < NPL; ++i)
      if (e == (unsigned)(lane + 32 * i)) key[i] = 0u;
    if (j == 0) v0 = v;
    den += expf(v - v0);
    if (lane == j) {
      my_v = v;
      my_e = (int)e;
    }
  }
  if (lane < a.k) {
    s.ids[t][lane] = my_e;
    s.w[t][lane] = expf(my_v - v0) / den;
  }
}

// -------------------------------------------------------------- the kernel
// NB: blocks of 8 token columns (1 for T <= 8, 2 up to kDecodeMaxT).
template <int W, int NB>
__global__ void __launch_bounds__(kDecodeThreads, 1) k_decode(const DecodeArgs a) {
  constexpr int CH = DecW<W>::CH, BW = DecW<W>::BW;
  constexpr int RED = 2 * NB * 4 * 32;  // floats a warp hands to its team
  extern __shared__ float red_all[];    // two buffers of kDecodeWarps * RED
  __shared__ DecShared s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, c = lane & 3;

  // ---- 1. partial logits; x in the weights' K order
  {
    const int tiles = (a.E + 15) >> 4;
    const int nch = (a.d + 31) >> 5;
    const int per = (nch + a.splits - 1) / a.splits;
    for (int u = blockIdx.x; u < tiles * a.splits; u += gridDim.x) {
      const int et = u % tiles, sp = u / tiles;
      const DecRows<kDecBf16> r =
          dec_rows<kDecBf16>(reinterpret_cast<const uint8_t*>(a.w_router), nullptr, 0, a.E, a.d, et * 16, g, c);
      float acc[NB][4];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[nb][i] = 0.f;
      const int k1 = min(nch, (sp + 1) * per);
      for (int kc = sp * per + warp; kc < k1; kc += kDecodeWarps) {
        const bool kok = kc * 32 + c * 8 < a.d;
        DecFrag<kDecBf16> f;
        uint32_t bw[NB][4];
        dec_load<kDecBf16>(f, r, kc, kok);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          const int t = nb * 8 + g;
          dec_tok<kDecBf16>(bw[nb], t < a.T ? a.x + (int64_t)t * a.d + c * 8 : nullptr, kc, kok);
        }
        dec_mma<kDecBf16, NB>(acc, f, bw, ~0u);
      }
      __syncthreads();  // the previous unit's sums have been read
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int i = 0; i < 4; ++i) red_all[warp * RED + (nb * 4 + i) * 32 + lane] = acc[nb][i];
      __syncthreads();
      for (int q = tid; q < NB * 128; q += kDecodeThreads) {
        float v = 0.f;
        for (int w = 0; w < kDecodeWarps; ++w) v += red_all[w * RED + q];
        const int ln = q & 31, i = (q >> 5) & 3, nb = q >> 7;
        const int e = et * 16 + (ln >> 2) + (i >> 1) * 8, t = nb * 8 + (ln & 3) * 2 + (i & 1);
        if (e < a.E && t < a.T) a.logits[((int64_t)sp * a.T + t) * a.E + e] = v;
      }
    }
    if (W != kDecBf16) {
      const int n8 = a.T * (a.d >> 3);
      for (int v = blockIdx.x * kDecodeThreads + tid; v < n8; v += gridDim.x * kDecodeThreads) {
        const uint4 q = __ldg(reinterpret_cast<const uint4*>(a.x) + v);
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
        uint16_t o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) o[dec_place<W>(e)] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
        reinterpret_cast<uint4*>(a.xs)[v] = make_uint4(o[0] | (uint32_t)o[1] << 16, o[2] | (uint32_t)o[3] << 16,
                                                       o[4] | (uint32_t)o[5] << 16, o[6] | (uint32_t)o[7] << 16);
      }
    }
  }
  if (!dec_grid_barrier(a.bar, 1, a.status, &s.ok)) return;

  // ---- 2. routing, in every CTA alike
  if (warp < a.T) {
    if (a.E <= 128) dec_topk<4>(a, warp, s);
    else if (a.E <= 256) dec_topk<8>(a, warp, s);
    else dec_topk<16>(a, warp, s);
  }
  s.flag[tid] = 0;
  if (tid < kDecodeMaxT * kMaxK) s.mask[tid] = 0;
  for (int i = tid; i < kDecodeMaxT * kMaxK * kDecodeMaxT / 4; i += kDecodeThreads)
    reinterpret_cast<uint32_t*>(&s.slot[0][0])[i] = 0xffffffffu;
  __syncthreads();
  const int npair = a.T * a.k;
  if (tid < npair) s.flag[s.ids[tid / a.k][tid % a.k]] = 1;
  __syncthreads();
  {
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
  }
  __syncthreads();
  if (tid < npair) {
    const int t = tid / a.k, j = tid % a.k, e = s.ids[t][j];
    s.slot[s.rank[e]][t] = (int8_t)j;
    atomicOr(&s.mask[s.rank[e]], 1u << t);
    if (blockIdx.x == 0) {
      if (a.ids) a.ids[tid] = e;
      if (a.tw) a.tw[tid] = s.w[t][j];
    }
  }
  const int f_r = (a.I + 15) >> 4, f_s = (a.I_s + 15) >> 4;  // units of 16 features per expert
  const int nch_d = (a.d + CH - 1) / CH;
  const int nch_i = (a.I + CH - 1) / CH, nch_s = (a.I_s + CH - 1) / CH;
  if (tid == 0) {
    s.kw1 = team_warps(s.n_act * f_r + f_s, nch_d, gridDim.x);
    s.kw2 = team_warps((a.d + 15) >> 4, s.n_act * nch_i + nch_s, gridDim.x);
  }
  __syncthreads();
  const int n_act = s.n_act;
  const bf16* xin = W == kDecBf16 ? a.x : a.xs;

  // ---- 3. gate/up and SwiGLU: units of 16 features, the shared expert's first
  {
    const int kw = s.kw1, team = warp / kw, tw = warp % kw, tpc = kDecodeWarps / kw;
    const int units = f_s + n_act * f_r;
    int buf = 0;
    for (int u = blockIdx.x + gridDim.x * team; u < units; u += gridDim.x * tpc) {
      const bool sh = u < f_s;
      const int ga = sh ? 0 : (u - f_s) / f_r;
      const int n0 = (sh ? u : (u - f_s) % f_r) * 16;
      const int N = sh ? a.I_s : a.I;
      const int64_t m = sh ? 0 : s.act[ga];
      const DecRows<W> rg = dec_rows<W>(sh ? a.sg : a.wg, sh ? a.sc[3] : a.sc[0], m, N, a.d, n0, g, c);
      const DecRows<W> ru = dec_rows<W>(sh ? a.su : a.wu, sh ? a.sc[4] : a.sc[1], m, N, a.d, n0, g, c);
      const bf16* tok[NB];
      unsigned nbmask = 0;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const int t = nb * 8 + g;
        const bool in = t < a.T && (sh || s.slot[ga][t] >= 0);
        tok[nb] = in ? xin + (int64_t)t * a.d + dec_tok_off<W>(c) : nullptr;
        nbmask |= (__any_sync(0xffffffffu, in) ? 1u : 0u) << nb;
      }
      float ag[NB][4], au[NB][4];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int i = 0; i < 4; ++i) ag[nb][i] = au[nb][i] = 0.f;
      constexpr int U = W == kDecBf16 ? (NB == 1 ? 4 : 3) : (W == kDecMx4 && NB == 1 ? 2 : 1);
      for (int kc = tw; kc < nch_d; kc += kw * U) {
        DecFrag<W> fg[U], fu[U];
        uint32_t bw[U][NB][BW];
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const int q = kc + i * kw;
          const bool kok = q < nch_d && (W != kDecBf16 || q * CH + c * 8 < a.d);
          dec_load<W>(fg[i], rg, q, kok);
          dec_load<W>(fu[i], ru, q, kok);
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const int q = kc + i * kw;
          const bool kok = q < nch_d && (W != kDecBf16 || q * CH + c * 8 < a.d);
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) dec_tok<W>(bw[i][nb], tok[nb], q, kok);
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
          dec_mma<W, NB>(ag, fg[i], bw[i], nbmask);
          dec_mma<W, NB>(au, fu[i], bw[i], nbmask);
        }
      }
      float* red = red_all + buf * (kDecodeWarps * RED) + (team * kw) * RED;
      buf ^= 1;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          red[tw * RED + (nb * 4 + i) * 32 + lane] = ag[nb][i];
          red[tw * RED + (NB * 4 + nb * 4 + i) * 32 + lane] = au[nb][i];
        }
      if (kw > 1) team_sync(team, kw * 32);
      else __syncwarp();
      for (int q = tw * 32 + lane; q < NB * 128; q += kw * 32) {
        float vg = 0.f, vu = 0.f;
        for (int w = 0; w < kw; ++w) {
          vg += red[w * RED + q];
          vu += red[w * RED + NB * 128 + q];
        }
        const int ln = q & 31, i = (q >> 5) & 3, nb = q >> 7;
        const int f = n0 + (ln >> 2) + (i >> 1) * 8, t = nb * 8 + (ln & 3) * 2 + (i & 1);
        if (f >= N || t >= a.T) continue;
        const int j = sh ? a.k : s.slot[ga][t];
        if (j < 0) continue;
        const float w = sh ? (a.gate ? __ldg(a.gate + t) : 1.f) : s.w[t][j];
        const float hv = w * (vg / (1.f + __expf(-vg)) * vu);
        a.h[((int64_t)t * (a.k + 1) + j) * a.ldh + dec_place<W>(f)] = __float2bfloat16_rn(hv);
      }
    }
  }
  if (!dec_grid_barrier(a.bar, 2, a.status, &s.ok)) return;

  // ---- 4. down projection: units of 16 outputs, K runs over every active expert
  {
    const int kw = s.kw2, team = warp / kw, tw = warp % kw, tpc = kDecodeWarps / kw;
    const int units = (a.d + 15) >> 4;
    const int total = n_act * nch_i + nch_s;
    int buf = 0;
    for (int u = blockIdx.x + gridDim.x * team; u < units; u += gridDim.x * tpc) {
      const int n0 = u * 16;
      float acc[NB][4];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[nb][i] = 0.f;
      constexpr int U = W == kDecBf16 ? 4 : (W == kDecMx4 && NB == 1 ? 2 : 1);
      for (int p = tw; p < total; p += kw * U) {
        DecFrag<W> f[U];
        uint32_t bw[U][NB][BW], member[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const int q = p + i * kw;
          const bool in = q < total;
          const int ga = in ? q / nch_i : 0;
          const bool sh = in && ga >= n_act;
          const int kc = sh ? q - n_act * nch_i : q - ga * nch_i;
          const int K = sh ? a.I_s : a.I;
          const bool kok = in && (W != kDecBf16 || kc * CH + c * 8 < K);
          const DecRows<W> r = dec_rows<W>(sh ? a.sd : a.wd, sh ? a.sc[5] : a.sc[2], sh ? 0 : s.act[min(ga, n_act - 1)],
                                           a.d, K, n0, g, c);
          dec_load<W>(f[i], r, kc, kok);
          member[i] = !in ? 0u : sh ? 0xffffu : s.mask[ga];
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            const int t = nb * 8 + g;
            const int j = !kok || t >= a.T ? -1 : sh ? a.k : s.slot[ga][t];
            const bf16* hp =
                j >= 0 ? a.h + ((int64_t)t * (a.k + 1) + j) * a.ldh + dec_tok_off<W>(c) : nullptr;
            dec_tok<W>(bw[i][nb], hp, kc, kok);
          }
        }
        // the sum over experts takes an expert's part only for its own tokens: an
        // infinity or a NaN in its weights reaches no other token
#pragma unroll
        for (int i = 0; i < U; ++i) {
          float part[NB][4];
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int r = 0; r < 4; ++r) part[nb][r] = 0.f;
          dec_mma<W, NB>(part, f[i], bw[i], ~0u);
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int r = 0; r < 4; ++r)
              if (member[i] >> (nb * 8 + 2 * c + (r & 1)) & 1u) acc[nb][r] += part[nb][r];
        }
      }
      float* red = red_all + buf * (kDecodeWarps * RED) + (team * kw) * RED;
      buf ^= 1;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int i = 0; i < 4; ++i) red[tw * RED + (nb * 4 + i) * 32 + lane] = acc[nb][i];
      if (kw > 1) team_sync(team, kw * 32);
      else __syncwarp();
      for (int q = tw * 32 + lane; q < NB * 128; q += kw * 32) {
        float v = 0.f;
        for (int w = 0; w < kw; ++w) v += red[w * RED + q];
        const int ln = q & 31, i = (q >> 5) & 3, nb = q >> 7;
        const int n = n0 + (ln >> 2) + (i >> 1) * 8, t = nb * 8 + (ln & 3) * 2 + (i & 1);
        if (n < a.d && t < a.T) a.y[(int64_t)t * a.d + n] = __float2bfloat16_rn(v);
      }
    }
  }
}

}  // namespace moe
