// MXFP4 format kernels: quantisers, the ROWS -> TILED prepack and dequantize.
//
// Rule (OCP microscaling, E2M1 elements and E8M0 scales): per block of 32
// values along K, scale 2^(floor(log2 max|x|) - 2), codes the nearest value of
// x / scale, ties to the even code, saturating at 6.
#include "mx.h"

namespace w4 {
namespace {

// Eight values of a row of type T (bf16 as uint16_t).
template <typename T>
__device__ __forceinline__ void load8(const T* p, float v[8]);
template <>
__device__ __forceinline__ void load8<float>(const float* p, float v[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
template <>
__device__ __forceinline__ void load8<uint16_t>(const uint16_t* p, float v[8]) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

// Four threads a block, eight values each: their loads and code stores are
// contiguous over a wave, and the block's largest magnitude takes two lane
// exchanges.  Bound by memory: 4.53 B (f32) or 2.53 B (bf16) a value.
template <typename T>
__global__ __launch_bounds__(256) void mx_quantize_kernel(const T* __restrict__ x, size_t n8,
                                                          uint32_t* __restrict__ codes,
                                                          uint8_t* __restrict__ scales) {
  const size_t i = blockIdx.x * static_cast<size_t>(256) + threadIdx.x;
  if (i >= n8) return;  // (n8 is a multiple of 4: a block's four threads stay together)
  float v[8];
  load8(x + 8 * i, v);
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[j]) & 0x7fffffffu);
  m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 1)));
  m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 2)));
  const uint32_t byte = mx_scale_byte(m);
  const float inv = mx_scale_inverse(byte);
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = byte == 255 ? 0.0f : v[j] * inv;
  codes[i] = mx_codes8(v);
  if ((i & 3) == 0) scales[i >> 2] = static_cast<uint8_t>(byte);
}

// One thread per (row block of 32 k, column) of w[K][N]: its 32 values are one
// block of the transposed matrix's row n.  A load step: reads are contiguous
// over the columns, the 16-byte code stores are not.
template <typename T>
__global__ __launch_bounds__(256) void mx_quantize_weight_kernel(const T* __restrict__ w, int K, int N,
                                                                 uint4* __restrict__ codes,
                                                                 uint8_t* __restrict__ scales) {
  const size_t i = blockIdx.x * static_cast<size_t>(256) + threadIdx.x;
  const int G = K / kMxBlock;
  if (i >= static_cast<size_t>(G) * N) return;
  const size_t g = i / N, n = i % N;
  const T* p = w + g * kMxBlock * N + n;
  float v[kMxBlock];
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < kMxBlock; ++j) {
    v[j] = load_act<T>(p, static_cast<size_t>(j) * N);
    m = max(m, __float_as_uint(v[j]) & 0x7fffffffu);
  }
  const uint32_t byte = mx_scale_byte(m);
  const float inv = mx_scale_inverse(byte);
#pragma unroll
  for (int j = 0; j < kMxBlock; ++j) v[j] = byte == 255 ? 0.0f : v[j] * inv;
  codes[n * G + g] = make_uint4(mx_codes8(v), mx_codes8(v + 8), mx_codes8(v + 16), mx_codes8(v + 24));
  scales[n * G + g] = static_cast<uint8_t>(byte);
}

// Where row r's block g (of 32 values) sits in the TILED layout, in 16-byte
// units of codes and bytes of scales; S = ceil(K / 128) steps.
__device__ __forceinline__ size_t tiled_unit(size_t r, int g, int S) {
  return ((r / 64 * S + g / 4) * 4 + (r / 16) % 4) * 64 + 16 * (g % 4) + r % 16;
}
__device__ __forceinline__ size_t tiled_scale(size_t r, int g, int S) {
  return ((r / 64 * S + g / 4) * 64 + 16 * (g % 4) + r % 16) * 4 + (r / 16) % 4;
}

// One thread per block of the padded matrix: blocks past the last row or K are
// zeros with scale 1.
__global__ __launch_bounds__(256) void mx_prepack_kernel(const uint4* __restrict__ codes,
                                                         const uint8_t* __restrict__ scales, int rows, int G, int S,
                                                         size_t total, uint4* __restrict__ dst_codes,
                                                         uint8_t* __restrict__ dst_scales) {
  const size_t i = blockIdx.x * static_cast<size_t>(256) + threadIdx.x;
  if (i >= total) return;
  const size_t r = i / (4 * S);
  const int g = static_cast<int>(i % (4 * S));
  const bool in = r < static_cast<size_t>(rows) && g < G;
  dst_codes[tiled_unit(r, g, S)] = in ? codes[r * G + g] : make_uint4(0, 0, 0, 0);
  dst_scales[tiled_scale(r, g, S)] = in ? scales[r * G + g] : 127;
}

// One thread per kE times eight values, a block's threads side by side: wave
// stores of 1 KiB (bf16) or 2 KiB.
constexpr int kE = 4;
template <typename T, bool kTiled>
__global__ __launch_bounds__(256) void mx_dequantize_kernel(const uint32_t* __restrict__ codes,
                                                            const uint8_t* __restrict__ scales, size_t n8, int G,
                                                            int S, T* __restrict__ out) {
  const size_t i0 = blockIdx.x * static_cast<size_t>(256 * kE) + threadIdx.x;
  uint32_t c[kE], byte[kE];
#pragma unroll
  for (int e = 0; e < kE; ++e) {
    const size_t i = i0 + 256 * e;
    if (i >= n8) break;
    size_t word = i, sc = i >> 2;
    if constexpr (kTiled) {
      const size_t r = (i >> 2) / G;
      const int g = static_cast<int>((i >> 2) % G);
      word = tiled_unit(r, g, S) * 4 + (i & 3);
      sc = tiled_scale(r, g, S);
    }
    c[e] = codes[word];
    byte[e] = scales[sc];
  }
#pragma unroll
  for (int e = 0; e < kE; ++e) {
    const size_t i = i0 + 256 * e;
    if (i >= n8) break;
    // (byte 0 is 2^-127, a subnormal float; 255 is NaN)
    const float s = __uint_as_float(byte[e] == 255 ? 0x7fc00000u : (byte[e] == 0 ? 0x00400000u : byte[e] << 23));
    float v[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      // exact: a code has two significant bits
      const f32x2 p = j == 0   ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[e], 1.0f, 0)
                      : j == 1 ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[e], 1.0f, 1)
                      : j == 2 ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[e], 1.0f, 2)
                               : __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[e], 1.0f, 3);
      v[2 * j] = p[0] * s;
      v[2 * j + 1] = p[1] * s;
    }
    if constexpr (sizeof(T) == 4) {
      float4* o = reinterpret_cast<float4*>(out + 8 * i);
      o[0] = make_float4(v[0], v[1], v[2], v[3]);
      o[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      uint32_t b[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        b[j] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{v[2 * j], v[2 * j + 1]}, bf16x2));
      *reinterpret_cast<uint4*>(out + 8 * i) = make_uint4(b[0], b[1], b[2], b[3]);
    }
  }
}

inline unsigned blocks_for(size_t n) { return static_cast<unsigned>((n + 255) / 256); }

// Output buffers of the quantisers and the prepack, apart from each other and
// from `in`.
w4a16_status_t check_out(const void* codes, size_t codes_bytes, const void* scales, size_t scales_bytes, size_t need_c,
                         size_t need_s, const void* in, size_t in_bytes) {
  if (codes == nullptr || scales == nullptr || !aligned16(codes) || !aligned16(scales)) return W4A16_ERR_INVALID_ARG;
  if (codes_bytes < need_c || scales_bytes < need_s) return W4A16_ERR_WORKSPACE;
  if (ranges_overlap(codes, need_c, scales, need_s) || ranges_overlap(in, in_bytes, codes, need_c) ||
      ranges_overlap(in, in_bytes, scales, need_s))
    return W4A16_ERR_INVALID_ARG;
  return W4A16_OK;
}

}  // namespace
}  // namespace w4

using namespace w4;

extern "C" size_t w4a16_mx_codes_bytes(int32_t rows, int32_t K, w4a16_mx_layout_t layout) {
  if (check_mx_shape(rows, K) != W4A16_OK) return 0;
  if (layout != W4A16_MX_ROWS && layout != W4A16_MX_TILED) return 0;
  if (layout == W4A16_MX_TILED && rows % 16 != 0) return 0;
  return mx_codes_bytes(rows, K, layout == W4A16_MX_TILED);
}

extern "C" size_t w4a16_mx_scales_bytes(int32_t rows, int32_t K, w4a16_mx_layout_t layout) {
  if (w4a16_mx_codes_bytes(rows, K, layout) == 0) return 0;
  return mx_scales_bytes(rows, K, layout == W4A16_MX_TILED);
}

extern "C" w4a16_status_t w4a16_mx_quantize(const void* x, w4a16_dtype_t xt, int32_t rows, int32_t K, uint8_t* codes,
                                            size_t codes_bytes, uint8_t* scales, size_t scales_bytes,
                                            hipStream_t stream) {
  if (xt != W4A16_F32 && xt != W4A16_BF16) return W4A16_ERR_INVALID_ARG;
  w4a16_status_t st = check_mx_shape(rows, K);
  if (st != W4A16_OK) return st;
  const size_t n = static_cast<size_t>(rows) * K;
  if (n == 0) return W4A16_OK;
  if (x == nullptr || !aligned16(x)) return W4A16_ERR_INVALID_ARG;
  st = check_out(codes, codes_bytes, scales, scales_bytes, n / 2, n / kMxBlock, x, n * dtype_bytes(xt));
  if (st != W4A16_OK) return st;
  uint32_t* c = reinterpret_cast<uint32_t*>(codes);
  if (xt == W4A16_F32)
    mx_quantize_kernel<<<blocks_for(n / 8), 256, 0, stream>>>(static_cast<const float*>(x), n / 8, c, scales);
  else
    mx_quantize_kernel<<<blocks_for(n / 8), 256, 0, stream>>>(static_cast<const uint16_t*>(x), n / 8, c, scales);
  return launch_status();
}

extern "C" w4a16_status_t w4a16_mx_quantize_weight(const void* w, w4a16_dtype_t wt, int32_t K, int32_t N,
                                                   uint8_t* codes, size_t codes_bytes, uint8_t* scales,
                                                   size_t scales_bytes, hipStream_t stream) {
  if (wt != W4A16_F32 && wt != W4A16_BF16) return W4A16_ERR_INVALID_ARG;
  w4a16_status_t st = check_mx_shape(N, K);
  if (st != W4A16_OK) return st;
  const size_t n = static_cast<size_t>(N) * K;
  if (n == 0) return W4A16_OK;
  if (w == nullptr || !aligned16(w)) return W4A16_ERR_INVALID_ARG;
  st = check_out(codes, codes_bytes, scales, scales_bytes, n / 2, n / kMxBlock, w, n * dtype_bytes(wt));
  if (st != W4A16_OK) return st;
  uint4* c = reinterpret_cast<uint4*>(codes);
  if (wt == W4A16_F32)
    mx_quantize_weight_kernel<<<blocks_for(n / kMxBlock), 256, 0, stream>>>(static_cast<const float*>(w), K, N, c,
                                                                           scales);
  else
    mx_quantize_weight_kernel<<<blocks_for(n / kMxBlock), 256, 0, stream>>>(static_cast<const uint16_t*>(w), K, N, c,
                                                                           scales);
  return launch_status();
}

extern "C" w4a16_status_t w4a16_mx_prepack(const w4a16_mx_t* src, uint8_t* dst_codes, size_t dst_codes_bytes,
                                           uint8_t* dst_scales, size_t dst_scales_bytes, w4a16_mx_t* out,
                                           hipStream_t stream) {
  w4a16_status_t st = check_mx(src);
  if (st != W4A16_OK) return st;
  if (out == nullptr) return W4A16_ERR_INVALID_ARG;
  if (src->layout != W4A16_MX_ROWS || src->rows % 16 != 0) return W4A16_ERR_UNSUPPORTED;
  const size_t cb = mx_codes_bytes(src->rows, src->K, true), sb = mx_scales_bytes(src->rows, src->K, true);
  if (cb != 0) {
    st = check_out(dst_codes, dst_codes_bytes, dst_scales, dst_scales_bytes, cb, sb, src->codes,
                   mx_codes_bytes(src->rows, src->K, false));
    if (st != W4A16_OK) return st;
    const size_t ib = mx_scales_bytes(src->rows, src->K, false);
    if (ranges_overlap(src->scales, ib, dst_codes, cb) || ranges_overlap(src->scales, ib, dst_scales, sb))
      return W4A16_ERR_INVALID_ARG;
  }
  const w4a16_mx_t m = *src;  // (out may be src)
  *out = m;
  out->codes = dst_codes;
  out->scales = dst_scales;
  out->layout = W4A16_MX_TILED;
  if (cb == 0) return W4A16_OK;
  mx_prepack_kernel<<<blocks_for(sb), 256, 0, stream>>>(
      reinterpret_cast<const uint4*>(m.codes), m.scales, m.rows, m.K / kMxBlock, (m.K + kMxStep - 1) / kMxStep, sb,
      reinterpret_cast<uint4*>(dst_codes), dst_scales);
  return launch_status();
}

extern "C" w4a16_status_t w4a16_mx_dequantize(const w4a16_mx_t* m, void* out, w4a16_dtype_t ot, size_t out_bytes,
                                              hipStream_t stream) {
  const w4a16_status_t st = check_mx(m);
  if (st != W4A16_OK) return st;
  if (ot != W4A16_F32 && ot != W4A16_BF16) return W4A16_ERR_INVALID_ARG;
  const size_t n = static_cast<size_t>(m->rows) * m->K, need = n * dtype_bytes(ot);
  if (n == 0) return W4A16_OK;
  if (out == nullptr || !aligned16(out)) return W4A16_ERR_INVALID_ARG;
  if (out_bytes < need) return W4A16_ERR_WORKSPACE;
  const uint32_t* c = reinterpret_cast<const uint32_t*>(m->codes);
  const int G = m->K / kMxBlock, S = (m->K + kMxStep - 1) / kMxStep;
  const bool tiled = m->layout == W4A16_MX_TILED;
  if (ranges_overlap(m->codes, mx_codes_bytes(m->rows, m->K, tiled), out, need) ||
      ranges_overlap(m->scales, mx_scales_bytes(m->rows, m->K, tiled), out, need))
    return W4A16_ERR_INVALID_ARG;
  const unsigned blocks = blocks_for((n / 8 + kE - 1) / kE);
  auto run = [&](auto kernel, auto* o) { kernel<<<blocks, 256, 0, stream>>>(c, m->scales, n / 8, G, S, o); };
  if (ot == W4A16_F32) {
    float* o = static_cast<float*>(out);
    tiled ? run(mx_dequantize_kernel<float, true>, o) : run(mx_dequantize_kernel<float, false>, o);
  } else {
    uint16_t* o = static_cast<uint16_t*>(out);
    tiled ? run(mx_dequantize_kernel<uint16_t, true>, o) : run(mx_dequantize_kernel<uint16_t, false>, o);
  }
  return launch_status();
}
