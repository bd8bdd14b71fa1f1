// mx4.cuh -- the microscaled 4-bit format (MX E2M1, "mx4"): conversions, the
// address of a scale byte, and the quantisation kernels ("quantification" to 4
// bits is one of the formats named on the Fondations page, chapter 06).
//
// A value is code * 2^(b - 127): the code has a sign, two exponent bits and one
// mantissa bit (0, 0.5, 1, 1.5, 2, 3, 4, 6), the scale byte b is shared by 32
// consecutive values of a row; b = 255 stands for a block of NaN.  Codes are
// packed two per byte, the lower-indexed value in the low half.  Scale bytes
// are kept per tile of 128 rows x 128 columns, 512 contiguous bytes: byte
// (r % 32) * 16 + (r / 32) * 4 + c / 32, which is the order in which the tensor
// core's scale columns are filled; tiles run along the columns, then down the
// rows, then over the matrices.  Rows and columns past a matrix's end hold 127.
#pragma once
#include "common.cuh"

namespace moe {

struct mx4 {  // weight element type of the kernels that take mx4 weights (two values)
  uint8_t pair;
};

constexpr int kMxTile = 128;       // rows and columns of a scale tile
constexpr int kMxTileBytes = 512;  // its scale bytes

// 2^(b - 127) as fp32: subnormal for b = 0, NaN for b = 255.
__host__ __device__ __forceinline__ uint32_t mx4_scale_bits(uint32_t b) {
  return b == 0 ? 0x00400000u : b == 255 ? 0x7fffffffu : b << 23;
}

// Byte of (row r, column block cb = c / 32) in a matrix of kt column tiles.
__host__ __device__ __forceinline__ int64_t mx4_scale_at(int64_t r, int64_t cb, int64_t kt) {
  return ((r >> 7) * kt + (cb >> 2)) * kMxTileBytes + (r & 31) * 16 + ((r & 127) >> 5) * 4 + (cb & 3);
}

// Eight fp32 values -> eight codes, value 0 in the lowest half-byte (round to
// nearest, ties to the even code, saturating at 6).
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// Eight codes -> eight fp32 values (unscaled).
__device__ __forceinline__ void e2m1x8_to_f32(uint32_t q, float (&v)[8]) {
  uint32_t h[4];
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(q));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}

// One value of a matrix of K columns (scalar kernels).
__device__ __forceinline__ float mx4_value(const mx4* codes, const uint8_t* scales, int64_t n, int64_t c, int64_t K) {
  const uint32_t q = (codes[(n * K + c) >> 1].pair >> ((c & 1) * 4)) & 15u;
  const uint32_t m = q & 7u;
  const float a = m < 2 ? 0.5f * m : (1.0f + 0.5f * (m & 1)) * (float)(1u << ((m >> 1) - 1));
  const float s = __uint_as_float(mx4_scale_bits(scales[mx4_scale_at(n, c >> 5, K >> 7)]));
  return (q & 8u ? -a : a) * s;
}

// ---------------------------------------------------------------- E4M3 terms
// The expert GEMMs on 4-bit weights take a bf16 value as the sum of two E4M3 terms
// under one power-of-two scale per block of columns (tc_mx4.cuh).
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {  // a in the low byte
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 e4m3x2_value(uint32_t q) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)q, __NV_E4M3);
  return __half22float2(__half2(h));
}

// Scale byte of a block whose largest magnitude has the bits amax: the power of two
// that puts it in (224, 448], the top of E4M3's range; at least 4, 255 for a NaN block.
// amax = m * 2^(e - 127), and m <= 1.75 fits 448 = 1.75 * 2^8 under 2^(e - 127 - 8).
__device__ __forceinline__ uint32_t mx_split_byte(uint32_t amax) {
  const uint32_t e = amax >> 23;
  if (e == 255u) return 255u;
  const uint32_t b = e + ((amax & 0x7fffffu) > 0x600000u ? 1u : 0u);
  return b < 12u ? 4u : b - 8u;
}
__device__ __forceinline__ float mx_split_inv(uint32_t b) {  // a NaN block multiplies by NaN: codes of NaN
  return b == 255u ? __uint_as_float(0x7fffffffu) : __uint_as_float((254u - b) << 23);
}

// ---------------------------------------------------------------- quantise
// Block scale of 32 values: with amax = m * 2^e, 1 <= m < 2, the scale is
// 2^(e - 2), so that the largest value lands in [4, 8) and saturates above 6 (the
// conversion of the OCP MX specification); 2^0 for a block of zeros; a block
// holding an infinity or a NaN becomes a NaN block (codes 0).  The division
// by a power of two is exact, so the only rounding is the code's.
//
// One block of 256 threads per 128 x 128 tile: 16 threads a row, 8 values a
// thread, 4 threads a scale block (two shuffles), 8 row passes whose loads are
// all issued before the first is used.  Memory bound: 2 (4) bytes read and 17/32
// written per value.  256 x 2048 x 512 bf16 values quantised and read back 260 us
// (207 at the copy rate); with 128, 512, 1024 threads a tile 287, 258, 337 us, 2048 x
// 8192 values 22.8 us (26.7, 24.6, 26.8); a block per two tiles, a warp a row, 288.
template <typename TA>
__device__ __forceinline__ void load8(const TA* p, float (&v)[8]);
template <>
__device__ __forceinline__ void load8<bf16>(const bf16* p, float (&v)[8]) {
  const uint4 a = __ldg(reinterpret_cast<const uint4*>(p));
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
template <>
__device__ __forceinline__ void load8<float>(const float* p, float (&v)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

struct MxTileIndex {
  int64_t m, rt, ct;  // matrix, row tile, column tile
};
__device__ __forceinline__ MxTileIndex mx4_tile(int64_t b, int64_t row_tiles, int64_t col_tiles) {
  MxTileIndex t;
  t.ct = b % col_tiles;
  b /= col_tiles;
  t.rt = b % row_tiles;
  t.m = b / row_tiles;
  return t;
}

template <typename TA>
__global__ void __launch_bounds__(256) k_mx4_quantize(const TA* __restrict__ x, int64_t rows, int64_t cols,
                                                      int64_t row_tiles, int64_t col_tiles,
                                                      uint32_t* __restrict__ codes, uint4* __restrict__ scales) {
  pdl_begin();  // after the previous kernel in the stream (programmatic launch)
  __shared__ __align__(16) uint8_t s_sc[kMxTileBytes];
  const MxTileIndex t = mx4_tile(blockIdx.x, row_tiles, col_tiles);
  const int tr = threadIdx.x >> 4, tc = threadIdx.x & 15;
  const int64_t c = t.ct * kMxTile + tc * 8;
  const int64_t r0 = t.rt * kMxTile + tr;
  const bool cok = c < cols;  // cols is a multiple of 32: the 4 threads of a block agree
  const int64_t at0 = (t.m * rows + r0) * cols + c;
  float v[8][8];
#pragma unroll
  for (int p = 0; p < 8; ++p) {
    if (cok && r0 + p * 16 < rows) {
      load8<TA>(x + at0 + (int64_t)p * 16 * cols, v[p]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[p][i] = 0.f;
    }
  }
#pragma unroll
  for (int p = 0; p < 8; ++p) {
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = max(amax, __float_as_uint(v[p][i]) & 0x7fffffffu);
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    const uint32_t e = amax >> 23;  // biased exponent of the largest magnitude (255: not finite)
    const uint32_t b = amax == 0 ? 127u : e == 255u ? 255u : e < 2u ? 0u : e - 2u;
    const float inv = __uint_as_float((254u - min(b, 253u)) << 23);
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = b == 255u ? 0.f : v[p][i] * inv;
    const int row = tr + p * 16;
    const bool ok = cok && r0 + p * 16 < rows;
    if (ok) codes[(at0 + (int64_t)p * 16 * cols) >> 3] = e2m1x8(q);
    if ((tc & 3) == 0) s_sc[(row & 31) * 16 + (row >> 5) * 4 + (tc >> 2)] = (uint8_t)(ok ? b : 127u);
  }
  __syncthreads();
  if (threadIdx.x < kMxTileBytes / 16)
    scales[(int64_t)blockIdx.x * (kMxTileBytes / 16) + threadIdx.x] =
        *reinterpret_cast<const uint4*>(s_sc + threadIdx.x * 16);
}

// ---------------------------------------------------------------- read back
// codes * scale in bf16 or fp32: exact in both (two significant bits), except
// that a scale byte above 252 can pass the largest finite value (infinity).
template <typename TA>
__global__ void __launch_bounds__(256) k_mx4_dequantize(const uint32_t* __restrict__ codes,
                                                        const uint4* __restrict__ scales, int64_t rows, int64_t cols,
                                                        int64_t row_tiles, int64_t col_tiles, TA* __restrict__ out) {
  pdl_begin();  // after the previous kernel in the stream (programmatic launch)
  __shared__ __align__(16) uint8_t s_sc[kMxTileBytes];
  const MxTileIndex t = mx4_tile(blockIdx.x, row_tiles, col_tiles);
  const int tr = threadIdx.x >> 4, tc = threadIdx.x & 15;
  const int64_t c = t.ct * kMxTile + tc * 8;
  const int64_t r0 = t.rt * kMxTile + tr;
  const int64_t at0 = (t.m * rows + r0) * cols + c;
  uint32_t q[8];
#pragma unroll
  for (int p = 0; p < 8; ++p)
    q[p] = c < cols && r0 + p * 16 < rows ? __ldg(codes + ((at0 + (int64_t)p * 16 * cols) >> 3)) : 0u;
  if (threadIdx.x < kMxTileBytes / 16)
    *reinterpret_cast<uint4*>(s_sc + threadIdx.x * 16) =
        __ldg(scales + (int64_t)blockIdx.x * (kMxTileBytes / 16) + threadIdx.x);
  __syncthreads();
  if (c >= cols) return;
#pragma unroll
  for (int p = 0; p < 8; ++p) {
    if (r0 + p * 16 >= rows) continue;
    const int row = tr + p * 16;
    const float s = __uint_as_float(mx4_scale_bits(s_sc[(row & 31) * 16 + (row >> 5) * 4 + (tc >> 2)]));
    float v[8];
    e2m1x8_to_f32(q[p], v);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= s;
    TA* dst = out + at0 + (int64_t)p * 16 * cols;
    if (sizeof(TA) == 2) {
      *reinterpret_cast<uint4*>(dst) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                  pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
    } else {
      reinterpret_cast<float4*>(dst)[0] = make_float4(v[0], v[1], v[2], v[3]);
      reinterpret_cast<float4*>(dst)[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
  }
}

}  // namespace moe
