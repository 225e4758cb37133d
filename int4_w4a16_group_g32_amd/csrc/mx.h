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
constexpr size_t kMxMaxValues = static_cast<size_t>(1) << 34;  // a launch's threads are counted in 32 bits

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

// Byte c of a dword of scale bytes as the float power of two.
template <int c>
__device__ __forceinline__ float mx_scale(uint32_t dword) {
  return __uint_as_float(c == 3 ? (dword >> 24) << 23 : ((dword >> (8 * c)) & 0xffu) << 23);
}

// ---------------------------------------------------------------- products

// What the activations of a product are.
enum MxX {
  kMxXf32 = 0,   // float32, as three bf16 pieces: exact
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
};

// Rows in blocks of 16, the whole K inside a workgroup (mx_stream.hip).
hipError_t launch_mx_stream(MxX xk, bool glu, const MxArgs& a, hipStream_t stream);

}  // namespace w4
