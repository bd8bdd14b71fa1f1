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
// The shape is the weight-row form of tc_swap.cuh: weight rows are the MMA's M,
// up to kNCH tokens of a group its N; a tile is two 128-row weight matrices, gate
// and up, or the two halves of 256 rows of the down matrix; the tile list and the
// epilogue are the ones defined there.
// A K block is 128 columns: TMA unpacks the 4-bit rows into the 8-bit containers the
// MMA reads (16 codes per 16 bytes, 128-byte swizzle), brings both planes of the
// token tile in one box, and the scale tiles of the weights (one 512-byte tile per
// matrix: their layout in memory is the tensor core's) and of the tokens as plain
// bulk copies.  The MMA thread moves the scale tiles into TMEM
// (tcgen05.cp.32x128b.warpx4) ahead of the MMAs that read them.
//
// TMEM: two accumulator buffers of 2 kNCH columns, then 16 scale columns per
// stage (gate 4, up 4, tokens 4: rows 0..63 of the hi plane, then of the lo plane).
//
// Warps: 0 producer; 1 TMEM owner and MMA issuer; 2..9 epilogue.
#pragma once
#include "mx4.cuh"
#include "tc_swap.cuh"

namespace moe {

enum : unsigned { kKernGemmMx4 = 5 };

struct Mx4Cfg {
  static constexpr int KB = 128;                   // columns per K block
  static constexpr int W_BYTES = 128 * KB;         // one matrix, unpacked
  static constexpr int X_BYTES = 2 * kNCH * KB;    // hi and lo planes
  static constexpr int SF_AT = 2 * W_BYTES + X_BYTES;
  // bytes the barrier counts: the unpacking load counts the packed codes it reads
  static constexpr int TX_BYTES = 2 * (W_BYTES / 2) + X_BYTES + 3 * kMxTileBytes;
  static constexpr int STAGE_BYTES = (SF_AT + 3 * kMxTileBytes + 1023) / 1024 * 1024;
  static constexpr int STAGES = 4;
  static constexpr int RING_BYTES = STAGES * STAGE_BYTES;
  static constexpr int EPI_WARPS = 8;
  static constexpr int THREADS = 64 + 32 * EPI_WARPS;
  static constexpr int ACC_COLS = 2 * kNCH;
  static constexpr int SF_COL = 2 * ACC_COLS, SF_COLS = 16;
  static constexpr int TMEM_COLS = 512;
  static constexpr int BAR_BYTES = (2 * STAGES + 5) * 8 + 16;
  static constexpr int SCHED_INTS = 2 * (512 + 2);
  static constexpr int SMEM_BYTES = 1024 + RING_BYTES + BAR_BYTES + SCHED_INTS * 4;
  static_assert(SF_COL + STAGES * SF_COLS <= TMEM_COLS, "TMEM columns");
  static_assert(W_BYTES % 1024 == 0 && X_BYTES % 1024 == 0, "swizzled tiles need 1024-byte alignment");
  static_assert(SMEM_BYTES <= 232448, "shared memory");
};

// ---------------------------------------------------------------- activations
// Row r of the activations (row_tok ? x[row_tok[r]] : x[r], ld elements wide, the
// first K_r or K_s of them used) as two E4M3 planes hl[2][rows_cap][ld] and
// scale tiles sf[chunk][ld / 128][512], chunk = the kNCH-row chunk of the row's
// group, numbered over the groups as the GEMM's tile list numbers them
// (prefix[g] / col_tiles; prefix of the routed groups' column tiles).  Rows in
// no group are left alone.
//
// Scale: the power of two that puts the block's largest value in (224, 448], the
// top of E4M3's range; at least 2^-123, so that lo's byte (four less) exists.  A
// block holding an infinity or a NaN becomes NaN.
// One block of 256 threads per row, 8 values a thread, 4 threads a scale block.
struct MxSplitArgs {
  const bf16* x;
  const int32_t* row_tok;  // NULL: row r itself
  const int32_t* offs;
  const int32_t* prefix;
  int E, col_tiles;
  int max_chunk;           // last chunk the scale buffer holds
  int64_t rows_cap, x_rows;
  int ld, K_r, K_s;
  uint8_t* hl;
  uint8_t* sf;
  unsigned* status;
};

__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {  // a in the low byte
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 e4m3x2_value(uint32_t q) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)q, __NV_E4M3);
  return __half22float2(__half2(h));
}

__global__ void __launch_bounds__(256) k_mx_split(MxSplitArgs p) {
  pdl_begin();  // after the previous kernel in the stream (programmatic launch)
  const int64_t r = blockIdx.x;
  if (r < __ldg(p.offs) || r >= __ldg(p.offs + p.E + 1)) return;
  int lo = 0, hi = p.E + 1;  // offs[lo] <= r < offs[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(p.offs + mid) <= r) lo = mid; else hi = mid;
  }
  const int g = lo, j = (int)(r - __ldg(p.offs + g));
  const int K = g < p.E ? p.K_r : p.K_s;
  const int64_t chunk = __ldg(p.prefix + g) / p.col_tiles + j / kNCH;
  if (chunk > p.max_chunk) return;  // group offsets that claim more rows than there are
  const int jj = j % kNCH;
  int64_t src = r;
  if (p.row_tok) {
    src = __ldg(p.row_tok + r);
    if (!in_range(src, p.x_rows, p.status, kSiteGatherToken)) return;
  }
  const bf16* x = p.x + src * p.ld;
  uint8_t* hrow = p.hl + r * p.ld;
  uint8_t* lrow = hrow + p.rows_cap * p.ld;
  uint8_t* sf = p.sf + chunk * (p.ld / 128) * kMxTileBytes + (jj & 31) * 16 + (jj >> 5) * 4;
  const int lane = threadIdx.x & 31;
  for (int c0 = 0; c0 < K; c0 += 256 * 8) {  // uniform: K is a multiple of 128, a warp's 256 columns may end half way
    const int c = c0 + threadIdx.x * 8;
    const bool ok = c < K;
    float v[8];
    if (ok) {
      load8<bf16>(x + c, v);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 0.f;
    }
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = max(amax, __float_as_uint(v[i]) & 0x7fffffffu);
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    // amax = m * 2^(e - 127): m <= 1.75 fits 448 = 1.75 * 2^8 under 2^(e - 127 - 8)
    const uint32_t e = amax >> 23;
    uint32_t b = e + ((amax & 0x7fffffu) > 0x600000u ? 1u : 0u);
    b = b < 12u ? 4u : b - 8u;
    const bool bad = e == 255u;
    const float inv = __uint_as_float((254u - b) << 23);
    uint32_t h[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a0 = v[2 * i] * inv, a1 = v[2 * i + 1] * inv;
      h[i] = e4m3x2(a0, a1);
      const float2 w = e4m3x2_value(h[i]);
      l[i] = e4m3x2((a0 - w.x) * 16.f, (a1 - w.y) * 16.f);
      if (bad) h[i] = l[i] = 0x7f7fu;
    }
    if (bad) b = 255u;
    if (ok) {
      *reinterpret_cast<uint2*>(hrow + c) = make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
      *reinterpret_cast<uint2*>(lrow + c) = make_uint2(l[0] | l[1] << 16, l[2] | l[3] << 16);
    }
    // the four bytes of a 128-column block meet in its first lane
    const int base = lane & 16;
    const uint32_t b1 = __shfl_sync(0xffffffffu, b, base + 4), b2 = __shfl_sync(0xffffffffu, b, base + 8),
                   b3 = __shfl_sync(0xffffffffu, b, base + 12);
    if ((lane & 15) == 0 && ok) {
      uint8_t* d = sf + (int64_t)(c >> 7) * kMxTileBytes;
      const uint32_t w = b | b1 << 8 | b2 << 16 | b3 << 24;
      const uint32_t lw = (b == 255u ? b : b - 4u) | (b1 == 255u ? b1 : b1 - 4u) << 8 |
                          (b2 == 255u ? b2 : b2 - 4u) << 16 | (b3 == 255u ? b3 : b3 - 4u) << 24;
      *reinterpret_cast<uint32_t*>(d) = w;       // hi plane: rows 0..63 of the tile
      *reinterpret_cast<uint32_t*>(d + 8) = lw;  // lo plane: rows 64..127
    }
  }
}

// ---------------------------------------------------------------- PTX
// D[tmem] (+)= (A * scale_A) (B * scale_B)^T: A 4-bit (E2M1 in 8-bit containers),
// B E4M3, one scale byte per row and 32 columns from TMEM, fp32 accumulate.
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
// A 512-byte scale tile (32 rows of 16 bytes) into 4 TMEM columns, the same 32
// lanes repeated in every lane quarter; in order with this thread's MMAs.
__device__ __forceinline__ void tmem_cp_scales(uint32_t taddr, uint64_t sdesc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc) : "memory");
}
// Unswizzled descriptor of a scale tile: 8-row core groups of 128 bytes.
__device__ __forceinline__ uint64_t sdesc_scales(uint32_t saddr) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)1 << 16;
  d |= (uint64_t)(128 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  return d;
}
// Instruction descriptor, .kind::mxf8f6f4: A E2M1, B E4M3, both K-major, UE8M0
// scales; `id` selects the byte of each scale word (the 32-column step).
__device__ __forceinline__ uint32_t idesc_mx4(int N, int id) {
  return ((uint32_t)id << 4) | (5u << 7) | (0u << 10) | ((uint32_t)(N >> 3) << 17) | (1u << 23) | (1u << 27) |
         ((uint32_t)id << 29);
}
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(
          smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}

// tmX: token planes (box 128 x kNCH x 2); tmB / tmC: 4-bit weight maps (box 128
// codes x 128 rows), gate (or the down matrix) and up; _r [E, N, K], _s [N, K].
struct Mx4Args {
  TcGemmArgs g;
  const uint8_t *sb_r, *sb_s, *sc_r, *sc_s;  // weight scale tiles of B and C
  const uint8_t* sf;                         // token scale tiles
  int ld;                                    // columns of the token planes
  int col_tiles;                             // column tiles of a routed group
  int max_chunk;                             // last chunk sf holds
};

template <int EPI>
__global__ void __launch_bounds__(Mx4Cfg::THREADS, 1)
    k_gemm_mx4(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmB_r,
               const __grid_constant__ CUtensorMap tmB_s, const __grid_constant__ CUtensorMap tmC_r,
               const __grid_constant__ CUtensorMap tmC_s, Mx4Args a) {
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
  uint64_t* tfull = empty + S;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int32_t* s_pre = reinterpret_cast<int32_t*>(smem + Cfg::RING_BYTES + Cfg::BAR_BYTES);
  int32_t* s_offs = s_pre + 514;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned tcode = kStatusTimeoutBase | (kKernGemmMx4 << 8);
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full + s, 1);
      mbar_init(empty + s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull + b, 1);
      mbar_init(tempty + b, Cfg::EPI_WARPS);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tmX);
    prefetch_tmap(&tmB_r);
    prefetch_tmap(&tmB_s);
    prefetch_tmap(&tmC_r);
    prefetch_tmap(&tmC_s);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, Cfg::TMEM_COLS);
    tmem_relinquish();
  }
  pdl_begin();  // the schedule and the token planes come from earlier kernels
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
        // scale tiles: [group][row tile][K block]; a second half past the matrix
        // re-reads the first half's (its codes read as zero and its rows are not stored)
        const int64_t rt = (int64_t)(sh ? 0 : t.g) * (t.N / 128) + t.n0 / 128;
        const bool c_in = t.n0 + C_ROW < t.N;
        const uint8_t* sb = (sh ? a.sb_s : a.sb_r) + rt * nkb * kMxTileBytes;
        const uint8_t* sc = (sh ? a.sc_s : a.sc_r) + (rt + (c_in ? C_ROW / 128 : 0)) * nkb * kMxTileBytes;
        const uint8_t* sx =
            a.sf + (int64_t)min(s_pre[t.g] / a.col_tiles + t.c0 / kNCH, a.max_chunk) * (a.ld / Cfg::KB) * kMxTileBytes;
        for (int kb = 0; kb < nkb; ++kb) {
          if (!mbar_wait(empty + stage, phase ^ 1, abort_flag, p.status, tcode | 1)) {
            ok = false;
            break;
          }
          uint64_t* land = full + stage;
          uint8_t* base = smem + stage * Cfg::STAGE_BYTES;
          const int k0 = kb * Cfg::KB;
          mbar_arrive_expect_tx(land, Cfg::TX_BYTES);
          if (sh) {
            tma_load_2d(base, &tmB_s, land, k0, t.n0, pol_w);
            tma_load_2d(base + Cfg::W_BYTES, &tmC_s, land, k0, t.n0 + C_ROW, pol_w);
          } else {
            tma_load_3d(base, &tmB_r, land, k0, t.n0, t.g, pol_w);
            tma_load_3d(base + Cfg::W_BYTES, &tmC_r, land, k0, t.n0 + C_ROW, t.g, pol_w);
          }
          tma_load_3d(base + 2 * Cfg::W_BYTES, &tmX, land, k0, (int)t.row0, 0, pol_x);
          bulk_load(base + Cfg::SF_AT, sb + (int64_t)kb * kMxTileBytes, kMxTileBytes, land, pol_w);
          bulk_load(base + Cfg::SF_AT + kMxTileBytes, sc + (int64_t)kb * kMxTileBytes, kMxTileBytes, land, pol_w);
          bulk_load(base + Cfg::SF_AT + 2 * kMxTileBytes, sx + (int64_t)kb * kMxTileBytes, kMxTileBytes, land, pol_x);
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
    if (lane == 0) {
      // ------------------------------------------------ MMA issuer
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      for (int tile = blockIdx.x; tile < total && ok; tile += gridDim.x) {
        const SwapTile t = decode_swap<TILE_ROWS>(p, s_pre, s_offs, tile);
        const int n = min(kNCH, (t.rows - t.c0 + 15) & ~15);  // the MMA's N: the chunk's tokens rounded up to 16
        const int nkb = (t.g == p.E ? p.K_s : p.K_r) / Cfg::KB;
        if (!mbar_wait(tempty + acc, acc_phase ^ 1, abort_flag, p.status, tcode | 2)) break;
        tc_fence_after();
        const uint32_t d0 = tmem_base + acc * Cfg::ACC_COLS;
        for (int kb = 0; kb < nkb; ++kb) {
          if (!mbar_wait(full + stage, phase, abort_flag, p.status, tcode | 3)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sw = smem_u32(smem + stage * Cfg::STAGE_BYTES);
          const uint32_t sx = sw + 2 * Cfg::W_BYTES, ss = sw + Cfg::SF_AT;
          // this stage's scale columns: the MMAs that read them last time have
          // completed (the producer waited for their commit before refilling the stage)
          const uint32_t sf = tmem_base + Cfg::SF_COL + stage * Cfg::SF_COLS;
#pragma unroll
          for (int i = 0; i < 3; ++i) tmem_cp_scales(sf + 4 * i, sdesc_scales(ss + i * kMxTileBytes));
#pragma unroll
          for (int kk = 0; kk < Cfg::KB / 32; ++kk) {
            const uint32_t id = idesc_mx4(n, kk);
            const uint64_t hi = sdesc_sw128(sx + kk * 32), lo = sdesc_sw128(sx + kNCH * Cfg::KB + kk * 32);
            const uint64_t wb = sdesc_sw128(sw + kk * 32), wc = sdesc_sw128(sw + Cfg::W_BYTES + kk * 32);
            umma_mxf8f6f4(d0, wb, hi, id, sf, sf + 8, (kb | kk) != 0);
            umma_mxf8f6f4(d0, wb, lo, id, sf, sf + 10, 1);
            umma_mxf8f6f4(d0 + kNCH, wc, hi, id, sf + 4, sf + 8, (kb | kk) != 0);
            umma_mxf8f6f4(d0 + kNCH, wc, lo, id, sf + 4, sf + 10, 1);
          }
          umma_commit(empty + stage);
          if (++stage == S) {
            stage = 0;
            phase ^= 1;
          }
        }
        if (!ok) break;
        umma_commit(tfull + acc);
        if (++acc == 2) {
          acc = 0;
          acc_phase ^= 1;
        }
      }
      umma_commit(drain);
      drain_wait(drain, 0);
    }
    __syncwarp();
  } else {
    swap_epilogue<true, EPI, Cfg::EPI_WARPS>(p, s_pre, s_offs, total, tmem_base, tfull, tempty, abort_flag, tcode, warp,
                                             lane);
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
