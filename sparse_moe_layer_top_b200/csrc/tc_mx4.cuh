// tc_mx4.cuh -- the expert GEMMs on microscaled 4-bit weights (mx4.cuh), with
// bf16 activations, on the block-scaled tensor cores.
//
// tcgen05.mma.kind::mxf8f6f4 multiplies 4-bit weights as they are stored by 8-bit
// activations, each with its power-of-two scale per 32 values, so no weight is
// converted.  A bf16 activation is given to it as the sum of two E4M3 terms,
//     x = s (hi + lo / 16),   s a power of two per 32 values,
// hi = x / s rounded to four significant bits, lo the rest: bf16 has eight, so the
// two terms hold x exactly down to about 2^-10 of the block's largest value and to
// 2^-21 of that value below (k_mx_split).  Two MMAs per 32 columns add both into
// one fp32 accumulator, lo under a scale byte smaller by four.  Per weight
// that is the work of one bf16 MMA (the 8-bit rate is twice as high), while HBM and
// the shared-memory fill carry a quarter and a half of the bytes.
//
// The tokens are the MMA's M, the weights its N: A holds the 2 x 64 plane rows of a
// chunk of kNCH = 64 tokens (row 2j the hi terms of token j, row 2j + 1 its lo terms),
// B 256 weight rows (128 of gate, 128 of up; or 256 rows of the down matrix).  Shared
// memory bounds the loop: per 32 columns A and B are read once (32 + 64 wavefronts of
// 128 bytes) and filled once (32 + 64), against 128 cycles of MMA.  The form with the
// weights as M and 64 tokens as N, a separate MMA per plane and matrix, reads 192
// and measured 3.32 ms on the gate/up product of 2048 tokens x 10 experts at
// d = 8192, I = 2048, E = 512.
// A K block is 128 columns: TMA unpacks the 4-bit rows into the 8-bit containers the
// MMA reads (16 codes per 16 bytes, 128-byte swizzle).  Four warps bring the scale
// tiles of the weights (one 512-byte tile per 128 rows: its layout in memory is the
// tensor core's) and of the tokens into TMEM from registers, ahead of the MMAs that
// read them; copied there from shared memory by the MMA thread (tcgen05.cp), three
// tiles cost the tensor pipe about 220 cycles per 512 cycles of MMA.
// Other ways to bring the codes, measured on the gate/up product of 2048 tokens x 10
// experts at d = 8192, I = 2048, E = 512 (this one: 2.14 ms; its loads alone 1.64, its
// MMAs and scales alone 1.37): 8-byte cp.async by eight warps 2.86 ms; 16-byte loads to
// registers, stored by eight warps, 3.1 ms; weights and token rows in rings of their own,
// 5 and 3 stages, 2.30 ms; TMA prefetches to L2 eight K blocks ahead 2.81 ms.
//
// The tile list is the one of tc_swap.cuh: the chunks of one weight tile are adjacent.
// TMEM: one accumulator of 256 columns, then 16 groups of 16 scale columns (tokens 4,
// weights 8).  Two accumulators and the scales do not fit 512 columns; the epilogue
// warps instead take the whole accumulator into registers (128 a thread) and hand it
// back before they compute or store, while the loads run on.
//
// Warps: 0 producer; 1 TMEM owner and MMA issuer; 2..9 epilogue; 10..13 scales.
#pragma once
#include "mx4.cuh"
#include "tc_swap.cuh"

namespace moe {

enum : unsigned { kKernGemmMx4 = 5 };

struct Mx4Cfg {
  static constexpr int KB = 128;                 // columns per K block
  static constexpr int A_BYTES = 2 * kNCH * KB;  // hi and lo rows of the token chunk
  static constexpr int B_BYTES = 256 * KB;       // weight rows, unpacked
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int SMALL = 16;               // chunks of at most this many tokens load 2 * SMALL rows of A
  // Bytes the barrier counts: the unpacking loads count the packed codes they read
  static constexpr int TX_BYTES = A_BYTES + B_BYTES / 2;
  static constexpr int TX_SMALL = TX_BYTES - A_BYTES + 2 * SMALL * KB;
  static constexpr int STAGES = 4;
  static constexpr int RING_BYTES = STAGES * STAGE_BYTES;
  static constexpr int EPI_WARPS = 8;
  static constexpr int SF_WARPS = 4;
  static constexpr int THREADS = 64 + 32 * (EPI_WARPS + SF_WARPS);
  // scale columns: SF_GROUPS groups of SF_KB K blocks of 16 columns (tokens 4, weights 8)
  static constexpr int SF_COL = 256, SF_COLS = 16, SF_KB = 4, SF_GROUPS = 4;
  static constexpr int TMEM_COLS = 512;
  static constexpr int BAR_BYTES = (2 * STAGES + 2 * SF_GROUPS + 3) * 8 + 8;
  static constexpr int SCHED_INTS = 2 * (512 + 2);
  static constexpr int SMEM_BYTES = 1024 + RING_BYTES + BAR_BYTES + SCHED_INTS * 4;
  static_assert(SF_COL + SF_GROUPS * SF_KB * SF_COLS <= TMEM_COLS, "TMEM columns");
  static_assert(A_BYTES % 1024 == 0 && B_BYTES % 1024 == 0, "swizzled tiles need 1024-byte alignment");
  static_assert(SMEM_BYTES <= 232448, "shared memory");
};

// ---------------------------------------------------------------- activations
// Row r of the activations (row_tok ? x[row_tok[r]] : x[r], d elements) as two
// rows of E4M3 terms, hl[2 r] (hi) and hl[2 r + 1] (lo), and scale tiles
// sf[chunk][d / 128][512], chunk = the kNCH-row chunk of the row's group,
// numbered over the groups as the GEMM's tile list numbers them (prefix[g] /
// col_tiles; prefix of the routed groups' column tiles), tile rows as the MMA's A
// rows.  Rows in no group are left alone.
//
// Scale: mx_split_byte; at least 2^-123, so that lo's byte (four less) exists.  A
// block holding an infinity or a NaN becomes NaN.
// One warp per row, 8 values a lane (4 lanes a scale block), four loads in flight.
struct MxSplitArgs {
  const bf16* x;
  const int32_t* row_tok;  // NULL: row r itself
  const int32_t* offs;
  const int32_t* prefix;
  int E, col_tiles;
  int max_chunk;           // last chunk the scale buffer holds
  int64_t rows, x_rows;
  int d;
  uint8_t* hl;
  uint8_t* sf;
  unsigned* status;
};
constexpr int kMxSplitRows = 8;  // rows per block, one warp each

__device__ __forceinline__ uint32_t mx_lo_byte(uint32_t b) { return b == 255u ? 255u : b - 4u; }
// Two values under scale byte b -> their hi codes (low half) and lo codes (high half).
__device__ __forceinline__ uint32_t mx_split2(float v0, float v1, float inv) {
  const float a0 = v0 * inv, a1 = v1 * inv;
  const uint32_t h = e4m3x2(a0, a1);
  const float2 w = e4m3x2_value(h);
  return h | e4m3x2((a0 - w.x) * 16.f, (a1 - w.y) * 16.f) << 16;
}
__global__ void __launch_bounds__(32 * kMxSplitRows) k_mx_split(MxSplitArgs p) {
  pdl_begin();  // after the previous kernel in the stream (programmatic launch)
  const int64_t r = (int64_t)blockIdx.x * kMxSplitRows + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (r >= p.rows || r < __ldg(p.offs) || r >= __ldg(p.offs + p.E + 1)) return;
  // the row's group: the last g with offs[g] <= r, 32 candidates a step
  const int step = (p.E + 32) / 32;  // E + 1 groups
  const int g0 = (__popc(__ballot_sync(0xffffffffu, lane * step <= p.E && __ldg(p.offs + min(lane * step, p.E)) <= r)) - 1) * step;
  const int g = g0 + __popc(__ballot_sync(0xffffffffu, lane < step && g0 + lane <= p.E && __ldg(p.offs + min(g0 + lane, p.E)) <= r)) - 1;
  const int j = (int)(r - __ldg(p.offs + g));
  const int64_t chunk = __ldg(p.prefix + g) / p.col_tiles + j / kNCH;
  if (j < 0 || chunk > p.max_chunk) return;  // group offsets that claim more rows than there are
  const int i = 2 * (j % kNCH);  // the MMA's A row of the hi terms
  int64_t src = r;
  if (p.row_tok) {
    src = __ldg(p.row_tok + r);
    if (!in_range(src, p.x_rows, p.status, kSiteGatherToken)) return;
  }
  const bf16* x = p.x + src * p.d;
  uint8_t* hrow = p.hl + 2 * r * p.d;
  uint8_t* lrow = hrow + p.d;
  uint8_t* sf = p.sf + chunk * (p.d / 128) * kMxTileBytes + (i & 31) * 16 + (i >> 5) * 4;
  constexpr int U = 4;
  for (int c0 = lane * 8; c0 < p.d; c0 += U * 256) {  // d is a multiple of 128: half warps agree
    uint4 q[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      q[u] = c0 + u * 256 < p.d ? __ldg(reinterpret_cast<const uint4*>(x + c0 + u * 256)) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = c0 + u * 256;
      if (c >= p.d) break;
      const unsigned half = 0xffffu << (lane & 16);
      const uint32_t w[4] = {q[u].x, q[u].y, q[u].z, q[u].w};
      uint32_t amax = 0;
#pragma unroll
      for (int t = 0; t < 4; ++t) amax = max(amax, max(w[t] << 16 & 0x7fff0000u, w[t] & 0x7fff0000u));
      amax = max(amax, __shfl_xor_sync(half, amax, 1));
      amax = max(amax, __shfl_xor_sync(half, amax, 2));
      const uint32_t b = mx_split_byte(amax);
      const float inv = mx_split_inv(b);
      uint32_t s[4];
#pragma unroll
      for (int t = 0; t < 4; ++t)
        s[t] = mx_split2(__uint_as_float(w[t] << 16), __uint_as_float(w[t] & 0xffff0000u), inv);
      *reinterpret_cast<uint2*>(hrow + c) = make_uint2(__byte_perm(s[0], s[1], 0x5410), __byte_perm(s[2], s[3], 0x5410));
      *reinterpret_cast<uint2*>(lrow + c) = make_uint2(__byte_perm(s[0], s[1], 0x7632), __byte_perm(s[2], s[3], 0x7632));
      // the four bytes of a 128-column block meet in its first lane
      const int base = lane & 16;
      const uint32_t b1 = __shfl_sync(half, b, base + 4), b2 = __shfl_sync(half, b, base + 8),
                     b3 = __shfl_sync(half, b, base + 12);
      if ((lane & 15) == 0) {
        uint8_t* t = sf + (int64_t)(c >> 7) * kMxTileBytes;
        *reinterpret_cast<uint32_t*>(t) = b | b1 << 8 | b2 << 16 | b3 << 24;
        *reinterpret_cast<uint32_t*>(t + 16) =
            mx_lo_byte(b) | mx_lo_byte(b1) << 8 | mx_lo_byte(b2) << 16 | mx_lo_byte(b3) << 24;
      }
    }
  }
}

// ---------------------------------------------------------------- PTX
// D[tmem] (+)= (A * scale_A) (B * scale_B)^T: A E4M3, B 4-bit (E2M1 in 8-bit
// containers), one scale byte per row and 32 columns from TMEM, fp32 accumulate.
__device__ __forceinline__ void umma_mxf8f6f4(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                              uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
          d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}
// 32 lanes x 4 / 8 consecutive 32-bit columns into TMEM (one row per thread).
__device__ __forceinline__ void tmem_st4(uint32_t taddr, uint4 v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "r"(v.x), "r"(v.y),
               "r"(v.z), "r"(v.w)
               : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, uint4 v, uint4 w) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(v.x),
               "r"(v.y), "r"(v.z), "r"(v.w), "r"(w.x), "r"(w.y), "r"(w.z), "r"(w.w)
               : "memory");
}
// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok));
  return ok != 0;
}
// Instruction descriptor, .kind::mxf8f6f4: A E4M3, B E2M1, both K-major, M = 128,
// UE8M0 scales; `id` selects the byte of each scale word (the 32-column step).
__device__ __forceinline__ uint32_t idesc_mx4(int N, int id) {
  return ((uint32_t)id << 4) | (0u << 7) | (5u << 10) | ((uint32_t)(N >> 3) << 17) | (1u << 23) | (1u << 27) |
         ((uint32_t)id << 29);
}
// The accumulator's hi rows (even lanes) and lo rows (odd lanes) of 32 columns summed:
// of every 2 G columns the even lane gets the first G, the odd lane the others, so
// that a 16-byte store of the two fills a 32-byte sector.
template <int G>
__device__ __forceinline__ void mx_sum_planes(const uint32_t (&a)[32], uint32_t* out, bool odd) {
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const uint32_t e = a[j / G * 2 * G + j % G], o = a[j / G * 2 * G + G + j % G];
    const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? e : o, 1);
    out[j] = __float_as_uint(__uint_as_float(odd ? o : e) + __uint_as_float(got));
  }
}
__device__ __forceinline__ uint4 mx_bf16x8(const uint32_t* v, float w) {
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = pack_bf16x2(w * __uint_as_float(v[2 * i]), w * __uint_as_float(v[2 * i + 1]));
  return make_uint4(r[0], r[1], r[2], r[3]);
}

// tmX / tmXs: the hi / lo rows (box 128 columns x 128 rows / 2 * SMALL rows);
// tmB / tmC: 4-bit weight maps (box 128 codes x 128 rows), gate (or the down
// matrix) and up; _r [E, N, K], _s [N, K].
struct Mx4Args {
  TcGemmArgs g;
  const uint8_t *sb_r, *sb_s, *sc_r, *sc_s;  // weight scale tiles of B and C
  const uint8_t* sf;                         // token scale tiles
  int ld;                                    // columns of the token rows
  int col_tiles;                             // column tiles of a routed group
  int max_chunk;                             // last chunk sf (and sf_out) holds
  uint8_t* hl_out;                           // SwiGLU: the activations as hi / lo rows of ldh columns
  uint8_t* sf_out;                           // and their scale tiles
};

template <int EPI>
__global__ void __launch_bounds__(Mx4Cfg::THREADS, 1)
    k_gemm_mx4(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmXs,
               const __grid_constant__ CUtensorMap tmB_r, const __grid_constant__ CUtensorMap tmB_s,
               const __grid_constant__ CUtensorMap tmC_r, const __grid_constant__ CUtensorMap tmC_s, Mx4Args a) {
  using Cfg = Mx4Cfg;
  constexpr int S = Cfg::STAGES;
  constexpr bool HALVES = EPI != kTcSwiGLU;  // two halves of 256 rows of one matrix
  constexpr int TILE_ROWS = HALVES ? 256 : 128;
  constexpr int C_ROW = HALVES ? 128 : 0;
  const TcGemmArgs& p = a.g;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + Cfg::RING_BYTES);
  uint64_t* empty = full + S;
  uint64_t* sfull = empty + S;
  uint64_t* sempty = sfull + Cfg::SF_GROUPS;
  uint64_t* tfull = sempty + Cfg::SF_GROUPS;
  uint64_t* tempty = tfull + 1;
  uint64_t* drain = tempty + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int32_t* s_pre = reinterpret_cast<int32_t*>(smem + Cfg::RING_BYTES + Cfg::BAR_BYTES);
  int32_t* s_offs = s_pre + 514;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned tcode = kStatusTimeoutBase | (kKernGemmMx4 << 8);
  const long long lim = wait_limit();
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full + s, 1);
      mbar_init(empty + s, 1);
    }
    for (int s = 0; s < Cfg::SF_GROUPS; ++s) {
      mbar_init(sfull + s, Cfg::SF_WARPS);
      mbar_init(sempty + s, 1);
    }
    mbar_init(tfull, 1);
    mbar_init(tempty, Cfg::EPI_WARPS);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tmX);
    prefetch_tmap(&tmXs);
    prefetch_tmap(&tmB_r);
    prefetch_tmap(&tmB_s);
    prefetch_tmap(&tmC_r);
    prefetch_tmap(&tmC_s);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, Cfg::TMEM_COLS);
    tmem_relinquish();
  }
  pdl_begin();  // the schedule and the token rows come from earlier kernels
  for (int i = threadIdx.x; i < p.E + 2; i += blockDim.x) {
    s_pre[i] = __ldg(p.prefix + i);
    s_offs[i] = __ldg(p.offs + i);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int total = s_pre[p.E + 1];

  if (warp == 0) {
    if (lane == 0) {
      // ------------------------------------------------ producer
      const uint64_t pol_w = policy_evict_first();
      const uint64_t pol_x = policy_evict_last();
      int stage = 0;
      uint32_t phase = 0, issued = 0, last_par = 0;
      bool ok = true;
      for (int tile = blockIdx.x; tile < total && ok; tile += gridDim.x) {
        const SwapTile t = decode_swap<TILE_ROWS>(p, s_pre, s_offs, tile);
        const bool sh = t.g == p.E;
        const int nkb = (sh ? p.K_s : p.K_r) / Cfg::KB;
        const bool small = t.rows - t.c0 <= Cfg::SMALL;
        for (int kb = 0; kb < nkb; ++kb) {
          if (!mbar_wait(empty + stage, phase ^ 1, abort_flag, p.status, tcode | 1, lim)) {
            ok = false;
            break;
          }
          uint64_t* land = full + stage;
          uint8_t* base = smem + stage * Cfg::STAGE_BYTES;
          uint8_t* wb = base + Cfg::A_BYTES;
          const int k0 = kb * Cfg::KB;
          mbar_arrive_expect_tx(land, small ? Cfg::TX_SMALL : Cfg::TX_BYTES);
          if (sh) {
            tma_load_2d(wb, &tmB_s, land, k0, t.n0, pol_w);
            tma_load_2d(wb + Cfg::B_BYTES / 2, &tmC_s, land, k0, t.n0 + C_ROW, pol_w);
          } else {
            tma_load_3d(wb, &tmB_r, land, k0, t.n0, t.g, pol_w);
            tma_load_3d(wb + Cfg::B_BYTES / 2, &tmC_r, land, k0, t.n0 + C_ROW, t.g, pol_w);
          }
          tma_load_2d(base, small ? &tmXs : &tmX, land, k0, 2 * (int)t.row0, pol_x);
          issued |= 1u << stage;
          last_par = (last_par & ~(1u << stage)) | (phase << stage);
          if (++stage == S) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      if (*abort_flag)
        for (int s = 0; s < S; ++s)
          if (issued >> s & 1u) drain_wait(full + s, last_par >> s & 1u);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------ MMA issuer: the warp waits, one lane issues
    const bool leader = elect_one();
    int stage = 0, sg = 0;
    uint32_t phase = 0, sphase = 0, acc_phase = 0;
    const uint64_t desc0 = sdesc_sw128(smem_u32(smem));
    bool ok = true;
    for (int tile = blockIdx.x; tile < total && ok; tile += gridDim.x) {
      const SwapTile t = decode_swap<TILE_ROWS>(p, s_pre, s_offs, tile);
      const int n = t.n0 + C_ROW < t.N ? 256 : 128;  // weight rows that exist
      const int nkb = (t.g == p.E ? p.K_s : p.K_r) / Cfg::KB;
      if (!__all_sync(0xffffffffu, mbar_wait(tempty, acc_phase ^ 1, abort_flag, p.status, tcode | 2, lim))) break;
      tc_fence_after();
      for (int kb = 0; kb < nkb; ++kb) {
        const int sk = kb % Cfg::SF_KB;
        const bool got = (sk != 0 || mbar_wait(sfull + sg, sphase, abort_flag, p.status, tcode | 5, lim)) &&
                         mbar_wait(full + stage, phase, abort_flag, p.status, tcode | 3, lim);
        if (!__all_sync(0xffffffffu, got)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint64_t dx = desc0 + (uint32_t)(stage * (Cfg::STAGE_BYTES >> 4));
        const uint32_t sf = tmem_base + Cfg::SF_COL + (sg * Cfg::SF_KB + sk) * Cfg::SF_COLS;
        const bool group_end = sk == Cfg::SF_KB - 1 || kb + 1 == nkb;
        if (leader) {
#pragma unroll
          for (int kk = 0; kk < Cfg::KB / 32; ++kk)
            umma_mxf8f6f4(tmem_base, dx + 2 * kk, dx + (Cfg::A_BYTES >> 4) + 2 * kk, idesc_mx4(n, kk), sf, sf + 4,
                          (kb | kk) != 0);
          umma_commit(empty + stage);
          if (group_end) umma_commit(sempty + sg);
          if (kb + 1 == nkb) umma_commit(tfull);
        }
        __syncwarp();
        if (group_end && ++sg == Cfg::SF_GROUPS) {
          sg = 0;
          sphase ^= 1;
        }
        if (++stage == S) {
          stage = 0;
          phase ^= 1;
        }
      }
      acc_phase ^= 1;
    }
    if (leader) {
      umma_commit(drain);
      drain_wait(drain, 0);
    }
    __syncwarp();
  } else if (warp >= 2 + Cfg::EPI_WARPS) {
    // ------------------------------------------------ scales into TMEM
    // A scale tile is 32 rows of 16 bytes: row l goes to lane l of every lane quarter,
    // its four words to four columns.  Each warp fills the quarter it can reach, a
    // group of SF_KB K blocks at a time; the next group waits in registers.
    constexpr int U = Cfg::SF_KB;
    const uint32_t tq = tmem_base + Cfg::SF_COL + ((uint32_t)((warp & 3) * 32) << 16);
    // the next group to load
    int ft = blockIdx.x, fk = 0, fn = 0;
    const uint4 *sx = nullptr, *sb = nullptr, *sc = nullptr;
    uint4 x[U], b[U], c[U];
    auto fetch = [&]() {  // false: no group is left
      if (ft >= total) return false;
      if (fk == 0) {
        const SwapTile t = decode_swap<TILE_ROWS>(p, s_pre, s_offs, ft);
        const bool sh = t.g == p.E;
        fn = (sh ? p.K_s : p.K_r) / Cfg::KB;
        // tiles: [group][row tile][K block]; a second half past the matrix takes the
        // first half's (the MMA does not read it)
        const int64_t rt = (int64_t)(sh ? 0 : t.g) * (t.N / 128) + t.n0 / 128;
        const int64_t ct = rt + (t.n0 + C_ROW < t.N ? C_ROW / 128 : 0);
        sx = reinterpret_cast<const uint4*>(a.sf + (int64_t)min(s_pre[t.g] / a.col_tiles + t.c0 / kNCH, a.max_chunk) *
                                                       (a.ld / Cfg::KB) * kMxTileBytes) + lane;
        sb = reinterpret_cast<const uint4*>((sh ? a.sb_s : a.sb_r) + rt * fn * kMxTileBytes) + lane;
        sc = reinterpret_cast<const uint4*>((sh ? a.sc_s : a.sc_r) + ct * fn * kMxTileBytes) + lane;
      }
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int at = min(fk + i, fn - 1) * (kMxTileBytes / 16);  // (past the end: not read)
        x[i] = __ldcg(sx + at);
        b[i] = __ldg(sb + at);
        c[i] = __ldg(sc + at);
      }
      fk += U;
      if (fk >= fn) {
        fk = 0;
        ft += gridDim.x;
      }
      return true;
    };
    int sg = 0;
    uint32_t sphase = 0;
    while (fetch()) {
      // (the MMAs that read these columns last have completed)
      if (!__all_sync(0xffffffffu, mbar_wait(sempty + sg, sphase ^ 1, abort_flag, p.status, tcode | 6, lim))) break;
      tc_fence_after();
#pragma unroll
      for (int i = 0; i < U; ++i) {
        tmem_st4(tq + (sg * U + i) * Cfg::SF_COLS, x[i]);
        tmem_st8(tq + (sg * U + i) * Cfg::SF_COLS + 4, b[i], c[i]);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(sfull + sg);
      if (++sg == Cfg::SF_GROUPS) {
        sg = 0;
        sphase ^= 1;
      }
    }
  } else {
    // ------------------------------------------------ epilogue
    // Warps of lane quarter q = warp % 4 hold tokens 16 q .. 16 q + 15 (lane pairs);
    // the two of a quarter take half of the weight rows each.  After the planes are
    // summed a lane has one token and 32 features (SwiGLU) or 64 outputs.
    const int q = warp & 3, eg = (warp - 2) >> 2;
    const bool odd = lane & 1;
    const int i = q * 32 + lane, jj = i >> 1;
    uint32_t acc_phase = 0;
    for (int tile = blockIdx.x; tile < total; tile += gridDim.x) {
      const SwapTile t = decode_swap<TILE_ROWS>(p, s_pre, s_offs, tile);
      const int64_t row = t.row0 + jj;
      bool in = jj < t.rows - t.c0 && row < p.rows_cap;
      int64_t dst = row;
      float w = 1.f;
      if (EPI == kTcSlotStore && in) {
        dst = __ldg(p.row_dst + row);
        w = __ldg(p.row_w + row);
        in = dst >= 0 && in_range(dst, p.ys_rows, p.status, kSiteSlotRow);
      }
      if (!__all_sync(0xffffffffu, mbar_wait(tfull, acc_phase, abort_flag, p.status, tcode | 4, lim)))
        break;  // the warp stops as one: its TMEM loads are warp-collective
      acc_phase ^= 1;
      tc_fence_after();
      const bool work = q * 16 < t.rows - t.c0 && (!HALVES || t.n0 + eg * 128 < t.N);  // (uniform in the warp)
      // the lane's sums.  SwiGLU: v the gate of 2 x 16 of 64 features, w2 their up; else
      // v and w2 64 of 128 outputs, 8 of every 16
      constexpr int G = HALVES ? 8 : 16;
      uint32_t v[32], w2[32];
      if (work) {
        const uint32_t tb = tmem_base + ((uint32_t)(q * 32) << 16) + (HALVES ? eg * 128 : eg * 64);
        uint32_t t0[32], t1[32];
        tmem_ld32(tb, t0);
        tmem_ld32(tb + 32, t1);
        tmem_wait_regs(t0);
        tmem_wait_regs(t1);
        mx_sum_planes<G>(t0, v, odd);
        mx_sum_planes<G>(t1, v + 16, odd);
        tmem_ld32(tb + (HALVES ? 64 : 128), t0);
        tmem_ld32(tb + (HALVES ? 96 : 160), t1);
        tmem_wait_regs(t0);
        tmem_wait_regs(t1);
        mx_sum_planes<G>(t0, w2, odd);
        mx_sum_planes<G>(t1, w2 + 16, odd);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(tempty);
      if (!work) continue;
      if (EPI == kTcSwiGLU) {
        // 16 features each of two 32-feature blocks; the pair holds both blocks' other halves
        uint32_t amax[2] = {0, 0};
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          // (the fast division, good to two steps of fp32: with the exact one this epilogue
          // held up the products of short K, 4096 tokens 205 us against 164)
          const float z = __uint_as_float(v[j]);
          v[j] = __float_as_uint(__fdividef(z, 1.f + __expf(-z)) * __uint_as_float(w2[j]));
          amax[j >> 4] = max(amax[j >> 4], v[j] & 0x7fffffffu);
        }
        // the activation enters the down product as two E4M3 terms, with no bf16
        // in between: hi and lo / 16 hold it to 2^-8 of its value, as bf16 would
        uint32_t b[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          b[k] = mx_split_byte(max(amax[k], __shfl_xor_sync(0xffffffffu, amax[k], 1)));
          const float inv = mx_split_inv(b[k]);
#pragma unroll
          for (int j = 0; j < 16; j += 4) {
            const uint32_t* x = v + 16 * k + j;
            const uint32_t s0 = mx_split2(__uint_as_float(x[0]), __uint_as_float(x[1]), inv);
            const uint32_t s1 = mx_split2(__uint_as_float(x[2]), __uint_as_float(x[3]), inv);
            w2[4 * k + j / 4] = __byte_perm(s0, s1, 0x5410);
            w2[8 + 4 * k + j / 4] = __byte_perm(s0, s1, 0x7632);
          }
        }
        const int chunk = s_pre[t.g] / a.col_tiles + t.c0 / kNCH;
        if (!in || chunk > a.max_chunk) continue;
        const int n = t.n0 + eg * 64;
        uint8_t* h = a.hl_out + 2 * row * p.ldh + n + (odd ? 16 : 0);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          *reinterpret_cast<uint4*>(h + 32 * k) = make_uint4(w2[4 * k], w2[4 * k + 1], w2[4 * k + 2], w2[4 * k + 3]);
          *reinterpret_cast<uint4*>(h + p.ldh + 32 * k) =
              make_uint4(w2[8 + 4 * k], w2[9 + 4 * k], w2[10 + 4 * k], w2[11 + 4 * k]);
        }
        // the two blocks' scale bytes: the even lane writes hi's (A row i), the odd lane lo's
        uint8_t* sf = a.sf_out + ((int64_t)chunk * (p.ldh / 128) + (n >> 7)) * kMxTileBytes + (i & 31) * 16 +
                      (i >> 5) * 4 + ((n & 127) >> 5);
        *reinterpret_cast<uint16_t*>(sf) =
            (uint16_t)(odd ? mx_lo_byte(b[0]) | mx_lo_byte(b[1]) << 8 : b[0] | b[1] << 8);
      } else {
        if (!in) continue;
        const int n = t.n0 + eg * 128 + (odd ? 8 : 0);
        bf16* o = EPI == kTcSlotStore ? p.ys + dst * p.ldy + n : p.out + row * p.ldo + n;
#pragma unroll
        for (int j = 0; j < 4; ++j) *reinterpret_cast<uint4*>(o + 16 * j) = mx_bf16x8(v + 8 * j, w);
#pragma unroll
        for (int j = 0; j < 4; ++j) *reinterpret_cast<uint4*>(o + 64 + 16 * j) = mx_bf16x8(w2 + 8 * j, w);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem_base, Cfg::TMEM_COLS);
  }
}

}  // namespace moe
