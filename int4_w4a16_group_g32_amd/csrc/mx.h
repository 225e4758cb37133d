// MXFP4 matrices: format helpers and the launch arguments of the products
// (internal).
//
// A value is E2M1 (codes 0 .. 7: 0, 1/2, 1, 3/2, 2, 3, 4, 6; bit 3 the sign)
// times 2^(scale byte - 127), one byte per block of 32 values along K; byte 255
// makes its whole block NaN.
#pragma once

#include "common.h"
#include "dispatch.h"
#include "mfma_ops.h"

namespace w4 {

constexpr int kMxBlock = 32;    // values of one scale
constexpr int kMxStep = 128;    // K of one tiled step: one v_mfma_scale_f32_16x16x128_f8f6f4
constexpr int kMxTileRows = 64; // weight rows (output columns) of one tile
constexpr int kMxTileCodes = kMxTileRows * kMxStep / 2;          // bytes of a tile's codes, one step
constexpr int kMxTileScales = kMxTileRows * kMxStep / kMxBlock;  // bytes of its scales
constexpr int kMxMaxK = 1 << 20;  // offsets inside one tile, or 256 activation rows, stay below 2^31
constexpr int kMxMaxRows = 1 << 24;
constexpr size_t kMxMaxValues = static_cast<size_t>(1) << 33;  // a launch's threads are counted in 32 bits

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

inline size_t mx_codes_bytes(size_t rows, size_t K, bool tiled) {
  return tiled ? (rows + 63) / 64 * ((K + 127) / 128) * kMxTileCodes : rows * (K / 2);
}
inline size_t mx_scales_bytes(size_t rows, size_t K, bool tiled) {
  return tiled ? (rows + 63) / 64 * ((K + 127) / 128) * kMxTileScales : rows * (K / kMxBlock);
}

inline w4a16_status_t check_mx_shape(int32_t rows, int32_t K) {
  if (rows < 0 || K < 0) return W4A16_ERR_INVALID_ARG;
  if (K % kMxBlock != 0 || K > kMxMaxK || rows > kMxMaxRows) return W4A16_ERR_UNSUPPORTED;
  if (static_cast<size_t>(rows) * K > kMxMaxValues) return W4A16_ERR_UNSUPPORTED;
  return W4A16_OK;
}

inline w4a16_status_t check_mx(const w4a16_mx_t* m) {
  if (m == nullptr || !aligned16(m->codes) || !aligned16(m->scales)) return W4A16_ERR_INVALID_ARG;
  const w4a16_status_t st = check_mx_shape(m->rows, m->K);
  if (st != W4A16_OK) return st;
  if (m->rows != 0 && m->K != 0 && (m->codes == nullptr || m->scales == nullptr)) return W4A16_ERR_INVALID_ARG;
  if (m->layout != W4A16_MX_ROWS && m->layout != W4A16_MX_TILED) return W4A16_ERR_UNSUPPORTED;
  if (m->layout == W4A16_MX_TILED && m->rows % 16 != 0) return W4A16_ERR_UNSUPPORTED;
  return W4A16_OK;
}

// ---------------------------------------------------------------- device helpers

// Scale byte of a block whose largest magnitude has these bits (sign cleared):
// floor(log2) - 2, at least -127; 255 where it is not finite.  Bits below the
// smallest normal float (exponent 0) end at byte 0 as well: 2^-126 / 4 is below
// 2^-127 already.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax_bits) {
  const uint32_t e = amax_bits >> 23;
  return e == 255 ? 255 : (e > 2 ? e - 2 : 0);
}

// 2^(127 - byte): what brings a block of this scale byte to E2M1's range
// (exact: bytes are at most 252, or 255, where the codes are 0).
__device__ __forceinline__ float mx_scale_inverse(uint32_t byte) {
  return byte == 255 ? 0.0f : __uint_as_float((254 - byte) << 23);
}

// Eight scaled values to eight codes, the first in the lowest nibble: nearest,
// ties to the even code, at most 6, in hardware.
__device__ __forceinline__ uint32_t mx_codes8(const float v[8]) {
  uint32_t r = 0;
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[0], v[1], 1.0f, 0);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[2], v[3], 1.0f, 1);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[4], v[5], 1.0f, 2);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[6], v[7], 1.0f, 3);
  return r;
}

// Eight codes as exact bf16 values times the power of two `scale` (a float with
// only an exponent; bits 0 stand for 2^-127, an infinity for NaN).  E2M1 has two
// significant bits and bf16 float's exponents, subnormals included, so this is
// exact up to 1.5 * 2^127, and an infinity above.
__device__ __forceinline__ bf16x8 mx_bf16(uint32_t codes, float scale) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3);
  return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// Four adjacent outputs from element `at`.
__device__ __forceinline__ void mx_store4(void* y, size_t at, int bf16, const f32x4& v) {
  if (bf16) {
    uint2 b;
    b.x = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{v[0], v[1]}, bf16x2));
    b.y = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{v[2], v[3]}, bf16x2));
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(y) + at) = b;
  } else {
    *reinterpret_cast<f32x4*>(static_cast<float*>(y) + at) = v;
  }
}

// 32 columns of h from column n as MXFP4: the lane's 4 columns of each half
// (row `row`, k block kb), the other three lanes of the row 16 lanes apart.
__device__ __forceinline__ void mx_store_h(void* codes, uint8_t* scales, int row, int N, int n, int kb, bool row_ok,
                                           const f32x4& lo, const f32x4& hi) {
  uint32_t m = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    m = max(m, max(__float_as_uint(lo[e]) & 0x7fffffffu, __float_as_uint(hi[e]) & 0x7fffffffu));
  m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 16)));
  m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 32)));
  const uint32_t byte = mx_scale_byte(m);
  const float inv = mx_scale_inverse(byte);
  float v[8];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    v[e] = byte == 255 ? 0.0f : lo[e] * inv;
    v[4 + e] = byte == 255 ? 0.0f : hi[e] * inv;
  }
  const uint32_t q = mx_codes8(v);
  if (!row_ok || n >= N) return;
  const size_t r = static_cast<size_t>(row);
  uint16_t* o = reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(codes) + r * (N / 2) + n / 2);
  o[kb] = static_cast<uint16_t>(q);
  o[4 + kb] = static_cast<uint16_t>(q >> 16);
  if (kb == 0) scales[r * (N / kMxBlock) + n / kMxBlock] = static_cast<uint8_t>(byte);
}

// Four adjacent values as kN bf16 planes of `plane` elements: 8 significant
// bits each, cut off, the last rounded to nearest (of three it is exact, down to
// 2^-110: below, its lowest bits are under bf16's smallest step, 2^-133).
template <int kN>
__device__ __forceinline__ void mx_store_pieces(void* planes, size_t at, size_t plane, f32x4 v) {
#pragma unroll
  for (int p = 0; p < kN; ++p) {
    if (p + 1 < kN) {
      f32x4 cut;
#pragma unroll
      for (int e = 0; e < 4; ++e) cut[e] = __uint_as_float(__float_as_uint(v[e]) & 0xffff0000u);
      uint2 b;
      b.x = __builtin_amdgcn_perm(__float_as_uint(v[1]), __float_as_uint(v[0]), 0x07060302);
      b.y = __builtin_amdgcn_perm(__float_as_uint(v[3]), __float_as_uint(v[2]), 0x07060302);
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(planes) + p * plane + at) = b;
      v -= cut;
    } else {
      mx_store4(planes, p * plane + at, 1, v);
    }
  }
}

// h as the down product takes it: float32, or two or three bf16 planes.
__device__ __forceinline__ void mx_store_hidden(void* h, size_t at, size_t plane, int pieces, const f32x4& v) {
  if (pieces == 0) mx_store4(h, at, 0, v);
  else if (pieces == 2) mx_store_pieces<2>(h, at, plane, v);
  else mx_store_pieces<3>(h, at, plane, v);
}

// ---------------------------------------------------------------- products

// What the activations of a product are.
enum MxX {
  kMxXf32 = 0,   // float32, as three bf16 pieces: exact (from 2^-110 on)
  kMxXf32h = 1,  // float32, as two bf16 pieces: 2^-17 (the intermediate of a bf16 layer)
  kMxXbf16 = 2,
  kMxXfp4 = 3    // MXFP4 rows
};

struct MxArgs {
  const void* x;          // [M][K] values, or the codes of MXFP4 rows
  const uint8_t* xs;      // MXFP4: their scales
  const uint8_t* wc[2];   // TILED codes (two matrices: gate and up)
  const uint8_t* ws[2];
  int M, N, K, S;         // S: steps of 128 k
  void* y;                // [M][N], or the codes of h
  uint8_t* ys;            // MXFP4 h: its scales
  int y_bf16;
  int h_pieces;           // other h: 0 float32, else bf16 planes of M * N
};

// Rows in blocks of 16, the whole K inside a workgroup (mx_stream.hip).
hipError_t launch_mx_stream(MxX xk, bool glu, const MxArgs& a, hipStream_t stream);
constexpr int kMxStreamRows = 16;
constexpr int kMxStreamCols = 32;  // of a workgroup (of each matrix) with more rows

// More rows, tiles of them in LDS (mx_tile.hip).  x: [M][K] bf16, or float32
// rows as bf16 planes [pieces][M][K], or MXFP4 rows; y as in MxArgs, or with glu
// h as bf16 planes or MXFP4 rows.
struct MxTileArgs : MxArgs {
  float* planes;  // sums of shared tiles: [workgroup of a tile][matrices][M][N]
  int tiles, row_tiles, band, bm, cols, tile0;  // tile0: the first column tile of the launch
  int unit_steps, per, quota;  // steps of a unit of K; units of a tile, and of a workgroup
};
struct MxTilePlan {
  int bm = 0, cols = 0, tiles = 0, unit_steps = 0, per = 0, quota = 0;
  size_t plane_bytes = 0;  // 0: every tile is one workgroup's
  // tiles of other sizes from column rest_from on (0: none)
  int rest_from = 0, rest_bm = 0, rest_cols = 0;
};
// (bm 0: the streamed form)
MxTilePlan plan_mx_product(int M, int N, int K, MxX xk, bool glu);
hipError_t launch_mx_tile(MxX xk, bool glu, const MxTilePlan& p, MxTileArgs& a, hipStream_t stream);
// float32 values as three bf16 planes of n values
hipError_t launch_mx_pieces(const float* x, size_t n, void* out, hipStream_t stream);

}  // namespace w4
