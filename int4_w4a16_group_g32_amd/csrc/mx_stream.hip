// Products of up to 16 rows with MXFP4 weights, streamed; and of up to 128 in
// blocks of 16, where that is shorter than tiles (plan_mx_product).
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
//    values enter as three bf16 pieces whose sum they are (exactly from 2^-110 on,
//    below to within 2^-134).
//
// Bound by the weights' bytes.  A workgroup owns the columns of one tile and
// all of K: its waves take every kW-th step, so nothing is summed across
// workgroups and one launch is the whole product; the waves' sums meet in LDS
// in wave order.  A wave keeps kRing steps of codes and rows in flight.  bf16
// and float32 rows pass through the wave's own part of LDS: each lane splits
// eight values into their pieces and writes them, and reads back fragments (the
// 64 lanes split 4 rows at once; splitting in fragment order, 16 rows whether
// they are there or not, and without LDS, took four decoding rows through the
// 7168 / 18432 MLP in 86 us).
//
// Measured: four float32 rows through that MLP 43 us (4.9 TB/s of its 211 MB; gate
// and up alone 5.0), 16 bf16 rows, 7168 -> 4096, 8 us (2 TB/s of weights: each of
// the 256 workgroups also reads all of x, 59 MB through the L2, and takes seven
// steps a wave with one load's way before them and the sums after), one row,
// 256 -> 512, 3.5 us of kernel and 7.6 of call.
#include "mx.h"

namespace w4 {
namespace {

constexpr int kRows = 16;         // rows of x in a launch's row block
constexpr int kOob = 0x7fffffff;  // an offset past every buffer: the load gives 0
constexpr int kXcds = 8;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* base, size_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, static_cast<int>(bytes), 0x00020000);
}
constexpr int kNt = 2;  // nontemporal: codes are read once
template <int kAux = 0>
__device__ __forceinline__ u32x4 load16(__amdgpu_buffer_rsrc_t r, int off, int soff) {
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off, soff, kAux));
}

// bf16 piece of eight float32 values: 8 significant bits each, cut off, r left
// with the rest; or with kLast all that is left, rounded to nearest.
template <bool kLast>
__device__ __forceinline__ u32x4 next_piece(float r[8]) {
  u32x4 w;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (kLast) {
      w[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{r[2 * i], r[2 * i + 1]}, bf16x2));
    } else {
      const uint32_t a = __float_as_uint(r[2 * i]), b = __float_as_uint(r[2 * i + 1]);
      w[i] = __builtin_amdgcn_perm(b, a, 0x07060302);
      r[2 * i] -= __uint_as_float(a & 0xffff0000u);
      r[2 * i + 1] -= __uint_as_float(b & 0xffff0000u);
    }
  }
  return w;
}

__device__ __forceinline__ i32x8 widen(const u32x4& v) {
  return i32x8{static_cast<int>(v[0]), static_cast<int>(v[1]), static_cast<int>(v[2]), static_cast<int>(v[3]),
               0, 0, 0, 0};
}

__device__ __forceinline__ f32x4 mma_fp4(const u32x4& w, const i32x8& x, const f32x4& acc, uint32_t ws, uint32_t xs) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(widen(w), x, acc, 4, 4, 0, static_cast<int>(ws), 0,
                                                          static_cast<int>(xs));
}

// One tile: kNB 16-column blocks of each matrix, up to 4 kC rows (of a block of
// 16); kW waves, each with kRing steps in flight.
template <int kX, int kC, int kNB, bool kGlu, int kW, int kRing>
__global__ __launch_bounds__(kW * 64) void mx_stream_kernel(const MxArgs a) {
  constexpr int kMats = kGlu ? 2 : 1;
  constexpr bool kFp4 = kX == kMxXfp4, kWide = kX == kMxXf32 || kX == kMxXf32h;
  constexpr int kPieces = kFp4 ? 0 : (kX == kMxXbf16 ? 1 : (kX == kMxXf32h ? 2 : 3));
  constexpr int kR = 4 * kC;                            // rows in LDS
  constexpr int kXv = kFp4 ? 1 : kC * (kWide ? 2 : 1);  // 16-byte loads of x a step
  constexpr int kXUnits = kPieces * kR * 16;            // LDS of a wave: pieces of 128 k
  // Column v of x's operands is piece v / kR of row v % kR: the pieces of few
  // rows share an instruction, and the columns of a row are added at the end.
  constexpr int kGroups = (kPieces * kR + 15) / 16;     // instructions of one k block
  constexpr int kFolds = kGroups == 1 && kPieces > 1 ? kPieces : (kR < 16 && kPieces > 1 ? 2 : 1);
  constexpr int kRedUnits = kMats * kNB * 64;           // its sums
  constexpr int kSpan = 4 % kNB == 0 ? 1 : (kNB + 6) / 4;  // 64-column tiles the columns may touch
  struct Step {
    u32x4 w[kMats][kNB];
    uint32_t ws[kMats][kSpan];
    u32x4 x[kXv];
    uint32_t xs;
  };
  __shared__ u32x4 lds[kW * (kXUnits > kRedUnits ? kXUnits : kRedUnits)];

  // XCD x = b mod 8 takes a contiguous run of tiles: neighbours share lines of scales
  const int T = static_cast<int>(gridDim.x), b = static_cast<int>(blockIdx.x);
  const int xcd = b % kXcds, tq = T / kXcds, trem = T % kXcds;
  const int task = xcd * tq + min(xcd, trem) + b / kXcds;
  const int tiles = (a.N + 16 * kNB - 1) / (16 * kNB);
  const int tile = task % tiles, r0 = task / tiles * kRows;
  const int nrows = min(kRows, a.M - r0);
  const int wv = wave_id(), lane = lane_id();
  const int lr = lane & 15, kb = lane >> 4;

  // the tile's codes and scales: kNB 16-column blocks from block c0 of 64-column
  // tile J, which they leave where kNB is no divisor of 4; a block past the last
  // tile reads the last one's, for nothing
  const int n0 = tile * 16 * kNB, J = n0 / kMxTileRows, c0 = n0 / 16 % 4;
  const int span = min(kSpan, (a.N + kMxTileRows - 1) / kMxTileRows - J);
  __amdgpu_buffer_rsrc_t wr[kMats], sr[kMats];
#pragma unroll
  for (int t = 0; t < kMats; ++t) {
    wr[t] = rsrc(a.wc[t] + static_cast<size_t>(J) * a.S * kMxTileCodes, static_cast<size_t>(a.S) * kMxTileCodes * span);
    sr[t] = rsrc(a.ws[t] + static_cast<size_t>(J) * a.S * kMxTileScales, static_cast<size_t>(a.S) * kMxTileScales * span);
  }
  int wat[kNB];  // block c's bytes from J's codes, of step 0
#pragma unroll
  for (int c = 0; c < kNB; ++c) {
    const int blk = min(c0 + c, 4 * span - 1);
    wat[c] = blk / 4 * a.S * kMxTileCodes + blk % 4 * 1024;
  }
  // rows past the last one and k past K read as zeros
  const int xrow = kFp4 ? a.K / 2 : a.K * (kWide ? 4 : 2);
  const __amdgpu_buffer_rsrc_t xr =
      rsrc(static_cast<const char*>(a.x) + static_cast<size_t>(r0) * xrow, static_cast<size_t>(nrows) * xrow);
  const int G = a.K / kMxBlock;
  const __amdgpu_buffer_rsrc_t xsr = rsrc(kFp4 ? a.xs + static_cast<size_t>(r0) * G : nullptr,
                                          kFp4 ? static_cast<size_t>(nrows) * G : 0);

  auto load = [&](Step& st, int s) {
    const int sc = min(s, a.S - 1);  // (past the end: read again, not used)
#pragma unroll
    for (int t = 0; t < kMats; ++t) {
#pragma unroll
      for (int c = 0; c < kNB; ++c) st.w[t][c] = load16<kNt>(wr[t], lane * 16, sc * kMxTileCodes + wat[c]);
#pragma unroll
      for (int i = 0; i < kSpan; ++i)
        st.ws[t][i] = __builtin_amdgcn_raw_buffer_load_b32(
            sr[t], lane * 4, sc * kMxTileScales + min(i, span - 1) * a.S * kMxTileScales, 0);
    }
    if constexpr (kFp4) {
      const bool on = lr < nrows && 4 * s + kb < G;
      st.x[0] = load16(xr, on ? lr * xrow + (4 * s + kb) * 16 : kOob, 0);
      st.xs = __builtin_amdgcn_raw_buffer_load_b8(xsr, on ? lr * G + 4 * s + kb : kOob, 0, 0);
    } else {
      // eight values of row (lane + 64 c) / 16
      const int k8 = 16 * s + lr;
#pragma unroll
      for (int c = 0; c < kC; ++c) {
        const int row = kb + 4 * c;
        const int at = row < nrows && 8 * k8 < a.K ? row * xrow + k8 * (kWide ? 32 : 16) : kOob;
        if constexpr (kWide) {
          st.x[2 * c] = load16(xr, at, 0);
          st.x[2 * c + 1] = load16(xr, at == kOob ? kOob : at + 16, 0);
        } else {
          st.x[c] = load16(xr, at, 0);
        }
      }
    }
    __builtin_amdgcn_sched_barrier(0);  // (loads stay in the order of their use)
  };

  f32x4 acc[kMats][kNB];
#pragma unroll
  for (int t = 0; t < kMats; ++t)
#pragma unroll
    for (int c = 0; c < kNB; ++c) acc[t][c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  u32x4* xl = lds + wv * kXUnits;
  // lane lr's chunk row of group i: columns past the pieces are zeros where a
  // later group shares the accumulator, and else compute what nothing reads
  auto frag = [&](int i, int j) {
    const int v = 16 * i + lr;
    const bool in = v < kPieces * kR;
    const int row = in ? v : 0;
    u32x4 x = xl[row * 16 + ((4 * kb + j) ^ (row & (kR - 1)))];
    if (kGroups > 1 && kPieces * kR % 16 != 0 && i == kGroups - 1) {
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = in ? x[e] : 0;
    }
    return __builtin_bit_cast(bf16x8, x);
  };
  auto multiply = [&](const Step& st) {
    uint32_t sc[kMats][kNB];  // block c's scale byte
#pragma unroll
    for (int t = 0; t < kMats; ++t)
#pragma unroll
      for (int c = 0; c < kNB; ++c) {
        uint32_t d = st.ws[t][0];
#pragma unroll
        for (int i = 1; i < kSpan; ++i) d = (c0 + c) / 4 == i ? st.ws[t][i] : d;
        sc[t][c] = (d >> (8 * ((c0 + c) % 4))) & 0xffu;
      }
    if constexpr (kFp4) {
      const i32x8 xb = widen(st.x[0]);
#pragma unroll
      for (int t = 0; t < kMats; ++t)
#pragma unroll
        for (int c = 0; c < kNB; ++c) acc[t][c] = mma_fp4(st.w[t][c], xb, acc[t][c], sc[t][c], st.xs);
    } else {
      // pieces to LDS; a wave's LDS operations run in order, so this needs no barrier
#pragma unroll
      for (int c = 0; c < kC; ++c) {
        const int row = kb + 4 * c, at = row * 16 + (lr ^ row);
        if constexpr (kWide) {
          float r[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) r[i] = __uint_as_float(st.x[2 * c + i / 4][i % 4]);
          xl[at] = next_piece<false>(r);
          if constexpr (kPieces == 3) xl[kR * 16 + at] = next_piece<false>(r);
          xl[(kPieces - 1) * kR * 16 + at] = next_piece<true>(r);
        } else {
          xl[at] = st.x[c];
        }
      }
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        bf16x8 xf[kGroups > 0 ? kGroups : 1];
#pragma unroll
        for (int p = 0; p < kGroups; ++p) xf[p] = frag(p, j);
        bf16x8 w[kMats][kNB];
#pragma unroll
        for (int t = 0; t < kMats; ++t)
#pragma unroll
          for (int c = 0; c < kNB; ++c) w[t][c] = mx_bf16(st.w[t][c][j], __uint_as_float(sc[t][c] << 23));
#pragma unroll
        for (int p = 0; p < kGroups; ++p)
#pragma unroll
          for (int t = 0; t < kMats; ++t)
#pragma unroll
            for (int c = 0; c < kNB; ++c)
              acc[t][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[t][c], xf[p], acc[t][c], 0, 0, 0);
      }
      __builtin_amdgcn_wave_barrier();
    }
  };

  const int n = wv < a.S ? (a.S - wv + kW - 1) / kW : 0;  // steps wv, wv + kW, ...
  Step ring[kRing];
#pragma unroll
  for (int j = 0; j < kRing; ++j) load(ring[j], wv + j * kW);
  for (int i = 0; i < n; i += kRing) {
#pragma unroll
    for (int j = 0; j < kRing; ++j) {
      if (i + j < n) multiply(ring[j]);
      load(ring[j], wv + (i + j + kRing) * kW);
    }
  }

  // the waves' sums, in wave order
  f32x4(*red)[kMats * kNB][64] = reinterpret_cast<f32x4(*)[kMats * kNB][64]>(lds);
  __syncthreads();  // (every wave is done with its rows)
#pragma unroll
  for (int t = 0; t < kMats; ++t)
#pragma unroll
    for (int c = 0; c < kNB; ++c) red[wv][t * kNB + c][lane] = acc[t][c];
  __syncthreads();
  auto sum = [&](int b) {
    f32x4 v = red[0][b][lane];
#pragma unroll
    for (int w = 1; w < kW; ++w) v += red[w][b][lane];
    // the smaller pieces' columns, lanes kR apart, to the first
    if constexpr (kFolds > 1) {
      const f32x4 u = v;
#pragma unroll
      for (int f = 1; f < kFolds; ++f)
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] += __shfl(u[e], lane + f * kR);
    }
    return v;
  };
  // lane: row r0 + lr, columns 4 kb .. 4 kb + 3 of a block
  if constexpr (kGlu && kFp4) {
    // h to MXFP4: 32 columns are two blocks of the four lanes of one row
    static_assert(kNB % 2 == 0, "blocks of 32 columns");
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
    static_assert(kNB <= kW, "a wave a block");
    if (wv >= kNB) return;
    const int n = n0 + 16 * wv + 4 * kb;
    f32x4 v = sum(wv);
    if constexpr (kGlu) {
      const f32x4 u = sum(kNB + wv);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = silu(v[i]) * u[i];
    }
    if (lr >= nrows || n >= a.N) return;
    const size_t to = static_cast<size_t>(r0 + lr) * a.N + n;
    if constexpr (kGlu) mx_store_hidden(a.y, to, static_cast<size_t>(a.M) * a.N, a.h_pieces, v);
    else mx_store4(a.y, to, a.y_bf16, v);
  }
}

template <int kX, int kC, int kNB, bool kGlu, int kW, int kRing>
hipError_t start(const MxArgs& a, hipStream_t stream) {
  const size_t tiles = (static_cast<size_t>(a.N) + 16 * kNB - 1) / (16 * kNB);
  const size_t blocks = tiles * ((static_cast<size_t>(a.M) + kRows - 1) / kRows);
  mx_stream_kernel<kX, kC, kNB, kGlu, kW, kRing><<<static_cast<unsigned>(blocks), kW * 64, 0, stream>>>(a);
  return hipGetLastError();
}

template <int kX, int kNB, bool kGlu, int kW, int kRing>
hipError_t start_rows(const MxArgs& a, hipStream_t stream) {
  if (kX == kMxXfp4 || a.M <= 4) return start<kX, 1, kNB, kGlu, kW, kRing>(a, stream);
  if constexpr (kX != kMxXfp4) {
    if (a.M <= 8) return start<kX, 2, kNB, kGlu, kW, kRing>(a, stream);
    return start<kX, 4, kNB, kGlu, kW, kRing>(a, stream);
  }
  return hipErrorInvalidValue;
}

constexpr int kCus = 256;

// The blocks that the busiest compute unit gets with nb of them a workgroup.
int most_blocks(int N, int nb) { return ((N + 16 * nb - 1) / (16 * nb) + kCus - 1) / kCus * nb; }

// Columns of a workgroup: what loads the compute units most evenly, and of
// equals the most (fewer workgroups read x), e.g. for N = 18432 one round of 231
// workgroups of 80 columns, for 7168 one of 224 of 32.  Gate and up, four
// float32 rows, 7168 -> 18432: 80 columns 27.3 us, 48 columns (384 workgroups)
// 32.1, 32 (576) 29.8, 16 (1152) 32.1.  Bytes in flight count too: the
// L2 of an XCD holds the lines that 32 compute units wait for, and beyond
// about 80 KiB each it slows down (80 columns with two steps a wave in flight
// 30.1 us, 32 columns with two, three, four 29.8, 33.6, 38.4).
int blocks_of(MxX xk, bool glu, int N) {
  if (glu && xk == kMxXfp4) {  // (h's blocks of 32 columns stay in a workgroup)
    const int m2 = most_blocks(N, 2), m4 = most_blocks(N, 4), m6 = most_blocks(N, 6);
    return m6 <= m4 && m6 <= m2 ? 6 : (m4 <= m2 ? 4 : 2);
  }
  const int m1 = most_blocks(N, 1), m2 = most_blocks(N, 2), m5 = most_blocks(N, 5);
  return m5 <= m2 && m5 <= m1 ? 5 : (m2 <= m1 ? 2 : 1);
}

// More than 16 rows: several row blocks share the weights through the caches, and
// what counts is how many workgroups a compute unit holds at once.  Four waves
// take half the LDS of eight: 37 float32 rows, 2304 -> 7168, 15 us for 20.
template <int kX, bool kGlu>
hipError_t start_shape(const MxArgs& a, hipStream_t stream) {
  const int nb = a.M > kRows ? 2 : blocks_of(static_cast<MxX>(kX), kGlu, a.N);
  if constexpr (kGlu && kX == kMxXfp4) {
    if (nb == 6) return start_rows<kX, 6, true, 8, 1>(a, stream);
    if (nb == 4) return start_rows<kX, 4, true, 8, 1>(a, stream);
    return start_rows<kX, 2, true, 4, 2>(a, stream);
  } else {
    if (nb == 5) return start_rows<kX, 5, kGlu, 8, kGlu ? 1 : 2>(a, stream);
    if (nb == 1) return start_rows<kX, 1, kGlu, 8, kGlu ? 2 : 4>(a, stream);
    if constexpr (kGlu) return start_rows<kX, 2, kGlu, 4, 2>(a, stream);
    else return a.M > kRows ? start<kX, kX == kMxXfp4 ? 1 : 4, 2, kGlu, 4, 2>(a, stream)
                            : start_rows<kX, 2, kGlu, 8, 2>(a, stream);
  }
}

}  // namespace

hipError_t launch_mx_stream(MxX xk, bool glu, const MxArgs& a, hipStream_t stream) {
  switch (xk) {
    case kMxXf32: return glu ? start_shape<kMxXf32, true>(a, stream) : start_shape<kMxXf32, false>(a, stream);
    case kMxXf32h: return start_shape<kMxXf32h, false>(a, stream);  // (h is never a gate's input)
    case kMxXbf16: return glu ? start_shape<kMxXbf16, true>(a, stream) : start_shape<kMxXbf16, false>(a, stream);
    case kMxXfp4: return glu ? start_shape<kMxXfp4, true>(a, stream) : start_shape<kMxXfp4, false>(a, stream);
  }
  return hipErrorInvalidValue;
}

}  // namespace w4
