// Products of up to 16 rows with MXFP4 weights, streamed.
//
// y[m][n] = sum_k x[m][k] e2m1(W[n][k]) 2^(s[n][k / 32] - 127)
//
// The weights are the matrix cores' first operand (16 output columns), the
// rows of x the second, so a lane ends with four adjacent columns of one row.
// A TILED step holds 128 k of 64 columns: lane l of a load has row l % 16 of a
// 16-column block and its k block l / 16, 32 codes in 16 bytes, and one dword
// with the scales of the lane's blocks of all four 16-column blocks.
//  - MXFP4 rows: one v_mfma_scale_f32_16x16x128_f8f6f4 a step and block, which
//    applies both scales; products and their sum are good to 2^-21 of the
//    largest (fp8 operands only to 2^-11, so wider rows do not go that way).
//  - bf16 and float32 rows: codes and scale become exact bf16 values in one
//    conversion per pair, and v_mfma_f32_16x16x32_bf16 takes codes 8j .. 8j+7 of
//    every lane as its j-th 32 k, the rows of x in the same order.  float32
//    values enter as three bf16 pieces whose sum they are exactly.
//
// Bound by the weights' bytes.  A workgroup owns the columns of one tile and
// all of K: its waves take every kW-th step, so nothing is summed across
// workgroups and one launch is the whole product; the waves' sums meet in LDS
// in wave order.  The rows come straight from the L2: few of them are there.
#include "mx.h"

namespace w4 {
namespace {

constexpr int kW = 8;        // waves of a workgroup
constexpr int kRows = 16;    // rows of x in a launch's row block
constexpr int kRing = 2;     // steps in flight per wave
constexpr int kOob = 0x7fffffff;  // an offset past every buffer: the load gives 0

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* base, size_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, static_cast<int>(bytes), 0x00020000);
}

template <int kX, int kNB, int kMats>
struct Step {
  static constexpr int kXv = kX == kMxXfp4 ? 1 : (kX == kMxXbf16 ? 4 : 8);
  u32x4 w[kMats][kNB];
  uint32_t ws[kMats];
  u32x4 x[kXv];
  uint32_t xs;
};

// bf16 piece number p of eight float32 values: 8 significant bits each, cut off
// (the last of two pieces rounded to nearest); r holds what is left.
template <int kLeft>
__device__ __forceinline__ bf16x8 next_piece(float r[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (kLeft == 0) {
      const bf16x2 b = __builtin_convertvector(f32x2{r[2 * i], r[2 * i + 1]}, bf16x2);
      w[i] = __builtin_bit_cast(uint32_t, b);
    } else {
      const uint32_t a = __float_as_uint(r[2 * i]), b = __float_as_uint(r[2 * i + 1]);
      w[i] = __builtin_amdgcn_perm(b, a, 0x07060302);
      r[2 * i] -= __uint_as_float(a & 0xffff0000u);
      r[2 * i + 1] -= __uint_as_float(b & 0xffff0000u);
    }
  }
  return __builtin_bit_cast(bf16x8, u32x4{w[0], w[1], w[2], w[3]});
}

__device__ __forceinline__ i32x8 widen(const u32x4& v) {
  return i32x8{static_cast<int>(v[0]), static_cast<int>(v[1]), static_cast<int>(v[2]), static_cast<int>(v[3]), 0, 0, 0, 0};
}

// One tile: kNB 16-column blocks of each of kMats matrices, one block of 16 rows.
template <int kX, int kNB, bool kGlu>
__global__ __launch_bounds__(kW * 64) void mx_stream_kernel(const MxArgs a) {
  constexpr int kMats = kGlu ? 2 : 1;
  using St = Step<kX, kNB, kMats>;
  const int tiles = (a.N + 16 * kNB - 1) / (16 * kNB);
  const int tile = blockIdx.x % tiles, r0 = blockIdx.x / tiles * kRows;
  const int nrows = min(kRows, a.M - r0);
  const int wv = wave_id(), lane = lane_id();
  const int lr = lane & 15, kb = lane >> 4;

  // the tile's codes and scales: 64-column tile J, first 16-column block c0
  const int n0 = tile * 16 * kNB, J = n0 / kMxTileRows, c0 = n0 / 16 % 4;
  __amdgpu_buffer_rsrc_t wr[kMats], sr[kMats];
#pragma unroll
  for (int t = 0; t < kMats; ++t) {
    wr[t] = rsrc(a.wc[t] + static_cast<size_t>(J) * a.S * kMxTileCodes, static_cast<size_t>(a.S) * kMxTileCodes);
    sr[t] = rsrc(a.ws[t] + static_cast<size_t>(J) * a.S * kMxTileScales, static_cast<size_t>(a.S) * kMxTileScales);
  }
  const size_t xrow = kX == kMxXfp4 ? a.K / 2 : static_cast<size_t>(a.K) * (kX == kMxXbf16 ? 2 : 4);
  // rows past the last one and k past K read as zeros
  const __amdgpu_buffer_rsrc_t xr = rsrc(static_cast<const char*>(a.x) + r0 * xrow, nrows * xrow);
  constexpr int kBlockBytes = kX == kMxXfp4 ? 16 : (kX == kMxXbf16 ? 64 : 128);
  const int xoff = lr < nrows ? lr * static_cast<int>(xrow) + kb * kBlockBytes : kOob;
  const int G = a.K / kMxBlock;
  const __amdgpu_buffer_rsrc_t xsr = rsrc(kX == kMxXfp4 ? a.xs + static_cast<size_t>(r0) * G : nullptr,
                                          kX == kMxXfp4 ? static_cast<size_t>(nrows) * G : 0);

  auto load = [&](St& st, int s) {
    s = min(s, a.S - 1);  // (past the end: read again, not used)
#pragma unroll
    for (int t = 0; t < kMats; ++t) {
      st.ws[t] = __builtin_amdgcn_raw_buffer_load_b32(sr[t], lane * 4, s * kMxTileScales, 0);
#pragma unroll
      for (int c = 0; c < kNB; ++c)
        st.w[t][c] = __builtin_bit_cast(
            u32x4, __builtin_amdgcn_raw_buffer_load_b128(wr[t], lane * 16, s * kMxTileCodes + (c0 + c) * 1024, 0));
    }
    const bool on = lr < nrows && 4 * s + kb < G;
    const int at = on ? xoff + s * 4 * kBlockBytes : kOob;
#pragma unroll
    for (int i = 0; i < St::kXv; ++i)
      st.x[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(xr, on ? at + 16 * i : kOob, 0, 0));
    if constexpr (kX == kMxXfp4)
      st.xs = __builtin_amdgcn_raw_buffer_load_b8(xsr, on ? lr * G + 4 * s + kb : kOob, 0, 0);
  };

  f32x4 acc[kMats][kNB];
#pragma unroll
  for (int t = 0; t < kMats; ++t)
#pragma unroll
    for (int c = 0; c < kNB; ++c) acc[t][c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  auto multiply = [&](const St& st) {
    uint32_t sc[kMats];
#pragma unroll
    for (int t = 0; t < kMats; ++t) sc[t] = kNB == 4 ? st.ws[t] : st.ws[t] >> (8 * c0);
    if constexpr (kX == kMxXfp4) {
      const i32x8 xb = widen(st.x[0]);
#pragma unroll
      for (int t = 0; t < kMats; ++t) {
        // (the scale's byte is an immediate of the instruction)
        acc[t][0] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(widen(st.w[t][0]), xb, acc[t][0], 4, 4, 0,
                                                                     static_cast<int>(sc[t]), 0, static_cast<int>(st.xs));
        if constexpr (kNB > 1)
          acc[t][1] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
              widen(st.w[t][1]), xb, acc[t][1], 4, 4, 1, static_cast<int>(sc[t]), 0, static_cast<int>(st.xs));
        if constexpr (kNB > 2) {
          acc[t][2] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
              widen(st.w[t][2]), xb, acc[t][2], 4, 4, 2, static_cast<int>(sc[t]), 0, static_cast<int>(st.xs));
          acc[t][3] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
              widen(st.w[t][3]), xb, acc[t][3], 4, 4, 3, static_cast<int>(sc[t]), 0, static_cast<int>(st.xs));
        }
      }
    } else {
      float f[kMats][4];
#pragma unroll
      for (int t = 0; t < kMats; ++t)
        f[t][0] = mx_scale<0>(sc[t]), f[t][1] = mx_scale<1>(sc[t]), f[t][2] = mx_scale<2>(sc[t]),
        f[t][3] = mx_scale<3>(sc[t]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        bf16x8 w[kMats][kNB];
#pragma unroll
        for (int t = 0; t < kMats; ++t)
#pragma unroll
          for (int c = 0; c < kNB; ++c) w[t][c] = mx_bf16(st.w[t][c][j], f[t][c]);
        auto mma = [&](const bf16x8& xp) {
#pragma unroll
          for (int t = 0; t < kMats; ++t)
#pragma unroll
            for (int c = 0; c < kNB; ++c)
              acc[t][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[t][c], xp, acc[t][c], 0, 0, 0);
        };
        if constexpr (kX == kMxXbf16) {
          mma(__builtin_bit_cast(bf16x8, st.x[j]));
        } else {
          float r[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) r[i] = __uint_as_float(st.x[2 * j + i / 4][i % 4]);
          mma(next_piece<1>(r));
          if constexpr (kX == kMxXf32) mma(next_piece<1>(r));
          mma(next_piece<0>(r));
        }
      }
    }
  };

  const int n = wv < a.S ? (a.S - wv + kW - 1) / kW : 0;  // steps wv, wv + kW, ...
  St ring[kRing];
#pragma unroll
  for (int j = 0; j < kRing; ++j) load(ring[j], wv + j * kW);
  for (int i = 0; i < n; i += kRing) {
#pragma unroll
    for (int j = 0; j < kRing; ++j) {
      if (i + j < n) multiply(ring[j]);
      load(ring[j], wv + (i + j + kRing) * kW);
    }
  }

  // the waves' sums, in wave order: item it is lane it % 64 of block it / 64
  __shared__ f32x4 red[kW][kMats * kNB][64];
#pragma unroll
  for (int t = 0; t < kMats; ++t)
#pragma unroll
    for (int c = 0; c < kNB; ++c) red[wv][t * kNB + c][lane] = acc[t][c];
  __syncthreads();
  auto sum = [&](int b) {
    f32x4 v = red[0][b][lane];
#pragma unroll
    for (int w = 1; w < kW; ++w) v += red[w][b][lane];
    return v;
  };
  // lane: row r0 + lr, columns 4 kb .. 4 kb + 3 of a block
  if constexpr (kGlu && kX == kMxXfp4) {
    // h to MXFP4: 32 columns are two blocks of the four lanes of one row
    if (wv >= kNB / 2) return;
    const int c = 2 * wv;
    f32x4 h[2];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const f32x4 g = sum(c + b), u = sum(kNB + c + b);
#pragma unroll
      for (int i = 0; i < 4; ++i) h[b][i] = silu(g[i]) * u[i];
    }
    mx_store_h(a.y, a.ys, r0 + lr, a.N, n0 + 16 * c, kb, lr < nrows, h[0], h[1]);
  } else {
    if (wv >= kNB) return;
    const int n = n0 + 16 * wv + 4 * kb;
    f32x4 v = sum(wv);
    if constexpr (kGlu) {
      const f32x4 u = sum(kNB + wv);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = silu(v[i]) * u[i];
    }
    if (lr >= nrows || n >= a.N) return;
    mx_store4(a.y, static_cast<size_t>(r0 + lr) * a.N + n, a.y_bf16, v);
  }
}

template <int kX, int kNB, bool kGlu>
hipError_t start(const MxArgs& a, hipStream_t stream) {
  const size_t tiles = (static_cast<size_t>(a.N) + 16 * kNB - 1) / (16 * kNB);
  const size_t blocks = tiles * ((static_cast<size_t>(a.M) + kRows - 1) / kRows);
  mx_stream_kernel<kX, kNB, kGlu><<<static_cast<unsigned>(blocks), kW * 64, 0, stream>>>(a);
  return hipGetLastError();
}

template <bool kGlu>
hipError_t start_x(MxX xk, const MxArgs& a, hipStream_t stream) {
  constexpr int kNB = kGlu ? 2 : 1;
  switch (xk) {
    case kMxXf32: return start<kMxXf32, kNB, kGlu>(a, stream);
    case kMxXf32h: return start<kMxXf32h, kNB, kGlu>(a, stream);
    case kMxXbf16: return start<kMxXbf16, kNB, kGlu>(a, stream);
    case kMxXfp4: return start<kMxXfp4, kNB, kGlu>(a, stream);
  }
  return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_mx_stream(MxX xk, bool glu, const MxArgs& a, hipStream_t stream) {
  return glu ? start_x<true>(xk, a, stream) : start_x<false>(xk, a, stream);
}

}  // namespace w4
