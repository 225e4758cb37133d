// Entry points of the products with MXFP4 weights: checks, workspace plans and
// launches.
#include "mx.h"

#include <cmath>
#include <initializer_list>

namespace w4 {
namespace {

w4a16_status_t check_mx_weight(const w4a16_mx_t* w) {
  const w4a16_status_t st = check_mx(w);
  if (st != W4A16_OK) return st;
  return w->layout == W4A16_MX_TILED ? W4A16_OK : W4A16_ERR_UNSUPPORTED;
}

w4a16_status_t check_mx_mlp(const w4a16_mx_t* gate, const w4a16_mx_t* up, const w4a16_mx_t* down) {
  w4a16_status_t st;
  if ((st = check_mx_weight(gate)) != W4A16_OK) return st;
  if ((st = check_mx_weight(up)) != W4A16_OK) return st;
  if ((st = check_mx_weight(down)) != W4A16_OK) return st;
  if (gate->K != up->K || gate->rows != up->rows) return W4A16_ERR_UNSUPPORTED;
  if (down->K != gate->rows || down->rows != gate->K) return W4A16_ERR_UNSUPPORTED;
  return W4A16_OK;
}

// The rows of a call: values of type xt, or MXFP4 rows.
struct MxRows {
  const void* x = nullptr;
  const uint8_t* xs = nullptr;
  size_t bytes = 0, sbytes = 0;
  MxX kind = kMxXf32;
};

w4a16_status_t rows_of(const void* x, w4a16_dtype_t xt, int32_t M, int32_t K, MxRows& r) {
  if (xt != W4A16_F32 && xt != W4A16_BF16) return W4A16_ERR_INVALID_ARG;
  if (M < 0) return W4A16_ERR_INVALID_ARG;
  r.x = x;
  r.bytes = static_cast<size_t>(M) * K * dtype_bytes(xt);
  r.kind = xt == W4A16_F32 ? kMxXf32 : kMxXbf16;
  return check_mx_shape(M, K);
}

w4a16_status_t rows_of(const w4a16_mx_t* x, int32_t K, MxRows& r) {
  const w4a16_status_t st = check_mx(x);
  if (st != W4A16_OK) return st;
  if (x->layout != W4A16_MX_ROWS || x->K != K) return W4A16_ERR_UNSUPPORTED;
  r.x = x->codes;
  r.xs = x->scales;
  r.bytes = mx_codes_bytes(x->rows, K, false);
  r.sbytes = mx_scales_bytes(x->rows, K, false);
  r.kind = kMxXfp4;
  return W4A16_OK;
}

// Pointers shared by the products, and that y and the workspace are apart from
// each other and from all that is read.
w4a16_status_t check_io(const MxRows& r, std::initializer_list<const w4a16_mx_t*> weights, const void* y,
                        size_t ybytes, const void* ws, size_t ws_bytes) {
  if (r.x == nullptr || y == nullptr || ws == nullptr) return W4A16_ERR_INVALID_ARG;
  if (!aligned16(r.x) || !aligned16(y) || !aligned16(ws)) return W4A16_ERR_INVALID_ARG;
  const auto hit = [&](const void* p, size_t n) {
    return ranges_overlap(p, n, y, ybytes) || ranges_overlap(p, n, ws, ws_bytes);
  };
  if (hit(r.x, r.bytes) || hit(r.xs, r.sbytes) || ranges_overlap(y, ybytes, ws, ws_bytes)) return W4A16_ERR_INVALID_ARG;
  for (const w4a16_mx_t* w : weights)
    if (hit(w->codes, mx_codes_bytes(w->rows, w->K, true)) || hit(w->scales, mx_scales_bytes(w->rows, w->K, true)))
      return W4A16_ERR_INVALID_ARG;
  return W4A16_OK;
}

// y of an empty sum
w4a16_status_t zeros(void* y, size_t ybytes, hipStream_t stream) {
  if (ybytes != 0 && (y == nullptr || !aligned16(y))) return W4A16_ERR_INVALID_ARG;
  return w4a16_workspace_init(y, ybytes, stream);
}

MxArgs mx_args(const MxRows& r, int M, const w4a16_mx_t* w0, const w4a16_mx_t* w1, void* y) {
  MxArgs a{};
  a.x = r.x;
  a.xs = r.xs;
  a.wc[0] = w0->codes;
  a.ws[0] = w0->scales;
  a.wc[1] = w1 ? w1->codes : nullptr;
  a.ws[1] = w1 ? w1->scales : nullptr;
  a.M = M;
  a.N = w0->rows;
  a.K = w0->K;
  a.S = (w0->K + kMxStep - 1) / kMxStep;
  a.y = y;
  return a;
}

size_t pieces_bytes(MxX kind, size_t n) { return kind == kMxXf32 ? 6 * n : (kind == kMxXf32h ? 4 * n : 0); }

struct MxGemmPlan {
  MxTilePlan t;
  size_t x_off = 0, planes_off = 0, bytes = 0;
};
MxGemmPlan plan_mx_gemm(int M, const w4a16_mx_t* w, MxX kind) {
  MxGemmPlan p;
  Carve c;
  p.t = plan_mx_product(M, w->rows, w->K, kind, false);
  if (p.t.bm != 0) {
    c.take(p.x_off, pieces_bytes(kind, static_cast<size_t>(M) * w->K));
    c.take(p.planes_off, p.t.plane_bytes);
  }
  p.bytes = std::max<size_t>(c.cursor, 256);
  return p;
}

struct MxMlpPlan {
  MxX hkind = kMxXf32;
  MxTilePlan gu, dn;
  size_t x_off = 0, h_off = 0, hs_off = 0, planes_off = 0, bytes = 0;
};
MxMlpPlan plan_mx_mlp(int M, const w4a16_mx_t* gate, MxX kind) {
  MxMlpPlan p;
  Carve c;
  const size_t n = static_cast<size_t>(M) * gate->rows;
  // h of bf16 rows keeps 16 bits (two pieces), well under the rounding of its own
  // operands and of a bf16 y: 64 rows, 7168 / 18432, y is 1.66e-3 off float64 with
  // two pieces and with three, and 1.3e-4 or 0.8e-4 off a float32 composition.  The
  // third piece would cost 94 -> 108 us there, 870 -> 1083 at 1024 rows.
  p.hkind = kind == kMxXbf16 ? kMxXf32h : kind;
  p.gu = plan_mx_product(M, gate->rows, gate->K, kind, true);
  p.dn = plan_mx_product(M, gate->K, gate->rows, p.hkind, false);
  if (kind == kMxXfp4) {
    c.take(p.h_off, n / 2);
    c.take(p.hs_off, n / kMxBlock);
  } else {
    c.take(p.h_off, p.dn.bm != 0 ? pieces_bytes(p.hkind, n) : n * 4);
  }
  c.take(p.x_off, p.gu.bm != 0 ? pieces_bytes(kind, static_cast<size_t>(M) * gate->K) : 0);
  c.take(p.planes_off, std::max(p.gu.plane_bytes, p.dn.plane_bytes));
  p.bytes = std::max<size_t>(c.cursor, 256);
  return p;
}

// One product, streamed or in tiles; pieces: where float32 rows go as planes.
w4a16_status_t mx_product(MxX kind, bool glu, const MxTilePlan& t, MxArgs a, void* pieces, void* planes,
                          hipStream_t stream) {
  if (t.bm == 0) return launch_mx_stream(kind, glu, a, stream) == hipSuccess ? W4A16_OK : W4A16_ERR_HIP;
  MxTileArgs ta{};
  static_cast<MxArgs&>(ta) = a;
  ta.planes = static_cast<float*>(planes);
  if (pieces != nullptr && kind == kMxXf32) {
    if (launch_mx_pieces(static_cast<const float*>(a.x), static_cast<size_t>(a.M) * a.K, pieces, stream) != hipSuccess)
      return W4A16_ERR_HIP;
    ta.x = pieces;
  }
  return launch_mx_tile(kind, glu, t, ta, stream) == hipSuccess ? W4A16_OK : W4A16_ERR_HIP;
}

w4a16_status_t mx_gemm(const MxRows& r, int M, const w4a16_mx_t* w, void* y, w4a16_dtype_t yt, void* ws,
                       size_t ws_bytes, hipStream_t stream) {
  if (yt != W4A16_F32 && yt != W4A16_BF16) return W4A16_ERR_INVALID_ARG;
  if (static_cast<size_t>(M) * w->rows > kMxMaxValues) return W4A16_ERR_UNSUPPORTED;
  const size_t ybytes = static_cast<size_t>(M) * w->rows * dtype_bytes(yt);
  if (ybytes == 0 || w->K == 0) return zeros(y, ybytes, stream);
  const MxGemmPlan p = plan_mx_gemm(M, w, r.kind);
  const w4a16_status_t st = check_io(r, {w}, y, ybytes, ws, std::min(ws_bytes, p.bytes));
  if (st != W4A16_OK) return st;
  if (ws_bytes < p.bytes) return W4A16_ERR_WORKSPACE;
  MxArgs a = mx_args(r, M, w, nullptr, y);
  a.y_bf16 = yt == W4A16_BF16;
  uint8_t* wsb = static_cast<uint8_t*>(ws);
  return mx_product(r.kind, false, p.t, a, wsb + p.x_off, wsb + p.planes_off, stream);
}

w4a16_status_t mx_swiglu_mlp(const MxRows& r, int M, const w4a16_mx_t* gate, const w4a16_mx_t* up,
                             const w4a16_mx_t* down, void* y, w4a16_dtype_t yt, void* ws, size_t ws_bytes,
                             hipStream_t stream) {
  if (yt != W4A16_F32 && yt != W4A16_BF16) return W4A16_ERR_INVALID_ARG;
  w4a16_status_t st = check_mx_shape(M, gate->rows);
  if (st != W4A16_OK) return st;
  const size_t ybytes = static_cast<size_t>(M) * gate->K * dtype_bytes(yt);
  if (ybytes == 0 || gate->rows == 0) return zeros(y, ybytes, stream);
  const MxMlpPlan p = plan_mx_mlp(M, gate, r.kind);
  st = check_io(r, {gate, up, down}, y, ybytes, ws, std::min(ws_bytes, p.bytes));
  if (st != W4A16_OK) return st;
  if (ws_bytes < p.bytes) return W4A16_ERR_WORKSPACE;
  uint8_t* wsb = static_cast<uint8_t*>(ws);
  MxRows h;
  h.x = wsb + p.h_off;
  h.xs = wsb + p.hs_off;
  h.kind = p.hkind;
  MxArgs gu = mx_args(r, M, gate, up, wsb + p.h_off);
  gu.ys = wsb + p.hs_off;
  gu.h_pieces = p.dn.bm == 0 ? 0 : (p.hkind == kMxXf32 ? 3 : 2);
  st = mx_product(r.kind, true, p.gu, gu, wsb + p.x_off, wsb + p.planes_off, stream);
  if (st != W4A16_OK) return st;
  MxArgs dn = mx_args(h, M, down, nullptr, y);
  dn.y_bf16 = yt == W4A16_BF16;
  return mx_product(h.kind, false, p.dn, dn, nullptr, wsb + p.planes_off, stream);
}

}  // namespace

// Streamed or in tiles, and which.  Row tiles have the height that the rows
// fill.  Where the tiles are fewer than the compute units, their units of K
// (pairs of steps) are dealt out evenly to one workgroup each, wherever that
// cuts a tile, if what this saves is more than the shared tiles' sums cost: a
// float32 plane for each workgroup of a tile, written and read at about 4 TB/s,
// and a launch of about 4 us.
//
// Up to 16 rows stream.  More rows stream in blocks of 16, each reading the
// weights (a column's row blocks lie on several XCDs, so past the L2 each: 37
// float32 rows, 2304 -> 7168, read 27.6 MB for 8.8 of weights) and all of x once a
// workgroup, while that is shorter than the tiles' longer way: 37 float32 rows, 2304 -> 7168, 15 us
// streamed and 25 in tiles, 7168 -> 18432 85 and 56; 64 bf16 rows, 2304 -> 7168,
// 13.5 and 18.4, 7168 -> 18432 73 and 32.  The times below, in us, are fitted to
// such measurements (17 to 128 rows, K 1056 to 7168, N 1040 to 18432).
MxTilePlan plan_mx_product(int M, int N, int K, MxX xk, bool glu) {
  constexpr int kCus = 256;
  MxTilePlan p;
  if (M <= kMxStreamRows) return p;
  const int mats = glu ? 2 : 1;
  const double planes = xk == kMxXf32 ? 3 : (xk == kMxXf32h ? 2 : 1);
  p.cols = 256 / mats;
  p.tiles = (N + p.cols - 1) / p.cols;
  const int S = (K + kMxStep - 1) / kMxStep;
  p.bm = M <= 32 ? 32 : (M <= 64 ? 64 : 128);
  // MXFP4 rows in tiles of twice the columns, which halve the rows' way through
  // L2 and LDS, where their rounds of workgroups are not so many more (a round of
  // 128 x 256 h takes 54 us to 41 of 128 x 128, K 7168)
  if (xk == kMxXfp4 && M > 128) {
    const size_t rows = (M + 127) / 128, wide_tiles = (N + 2 * p.cols - 1) / (2 * p.cols);
    const size_t rounds = (rows * p.tiles + kCus - 1) / kCus, wide_rounds = (rows * wide_tiles + kCus - 1) / kCus;
    if (wide_rounds * (glu ? 1.35 : 1.7) < rounds) {
      p.cols *= 2;
      p.tiles = static_cast<int>(wide_tiles);
    }
  }
  const size_t tiles = static_cast<size_t>((M + p.bm - 1) / p.bm) * p.tiles;
  p.unit_steps = S;
  p.per = p.quota = 1;
  int units = (S + 1) / 2 * static_cast<int>((tiles + kCus - 1) / kCus);  // of the busiest workgroup
  double sums_us = 0;
  if (tiles < kCus && S > 2) {
    const int per = (S + 1) / 2, quota = std::max(2, static_cast<int>((tiles * per + kCus - 1) / kCus));
    const int most = (per + quota - 2) / quota + 1;  // workgroups of a tile
    // a unit: 256 k, at 5 (bf16 planes) or 12 TFLOP/s of a compute unit, and at
    // least its 35 KB of codes and scales at its share of 6 TB/s
    const double unit_us = std::max(2.0 * p.bm * 256 * 256 * planes / (xk == kMxXfp4 ? 12e6 : 5e6), 35e3 / 23e3);
    const double bytes = 4.0 * M * N * mats;
    const double us = 2 * std::min<double>(most, 1 + static_cast<double>(per) / quota) * bytes / 4e6;
    if (quota < per && (per - quota) * unit_us > 4 + us) {
      p.unit_steps = 2;
      p.per = per;
      p.quota = units = quota;
      p.plane_bytes = static_cast<size_t>(most) * mats * M * N * 4;
      sums_us = us;
    }
  }
  // A last round that few workgroups would have: its columns in smaller tiles, if
  // one round of them is shorter (a round of 64-row tiles takes 0.6 of one of 128
  // bf16 or float32 rows; of MXFP4 rows 0.72, gate and up 0.8, and from the wide
  // tiles 0.49 and 0.56, 128-row tiles of half the columns 0.69) by more than a
  // launch.  1024 MXFP4 rows, 7168 -> 18432 gate and up: 2 rounds and a quarter.
  if (M > 128 && tiles > kCus && tiles % kCus != 0) {
    const size_t row_tiles = (M + p.bm - 1) / p.bm;
    const int full = static_cast<int>(tiles / kCus * kCus / row_tiles) * p.cols;
    const int narrow = 256 / mats;
    const bool wide = p.cols != narrow;
    const double step_us = xk == kMxXfp4 ? (wide ? 0.92 : 0.62) : 1.5 * planes;
    const auto rounds = [&](int bm) {
      return std::ceil(std::ceil(static_cast<double>(M) / bm) * ((N - full + narrow - 1) / narrow) / kCus);
    };
    const double half = rounds(64) * (xk != kMxXfp4 ? 0.6 : (wide ? (glu ? 0.56 : 0.49) : (glu ? 0.8 : 0.72)));
    const double other = wide ? rounds(128) * 0.69 : 1;
    if (full > 0 && (1 - std::min(half, other)) * S * step_us > 4) {
      p.rest_from = full;
      p.rest_bm = half < other ? 64 : 128;
      p.rest_cols = narrow;
    }
  }
  if (M <= 128) {
    const bool fp4 = xk == kMxXfp4;
    // a start, and for the workgroups of a compute unit (of the busiest one and on
    // average) a part of their own and one for each step
    constexpr double kStart[4] = {3.5, 3.5, 3, 2.7}, kOwn[4] = {0.5, 0.4, 0.2, 0.2};
    constexpr double kStep[2][4] = {{0.21, 0.20, 0.14, 0.125}, {0.35, 0.35, 0.27, 0.24}};
    const double wgs = (N + kMxStreamCols - 1) / kMxStreamCols * ((M + 15) / 16) / static_cast<double>(kCus);
    const double stream_us = kStart[xk] + (std::ceil(wgs) + wgs) / 2 * (kOwn[xk] + S * kStep[glu][xk]);
    const int h = p.bm == 32 ? 0 : (p.bm == 64 ? 1 : 2);
    constexpr double kBase[2][3] = {{8.5, 10.3, 12}, {6.8, 7.8, 7}}, kStage[2][3] = {{0.8, 1.5, 2.5}, {0.7, 0.8, 1}};
    const double tile_us = kBase[fp4][h] + (xk == kMxXf32 ? 2.3 : 0) + units * planes * kStage[fp4][h] + sums_us;
    if (stream_us < tile_us) return MxTilePlan();
  }
  return p;
}

}  // namespace w4

using namespace w4;

extern "C" size_t w4a16_mx_gemm_workspace_bytes(int32_t M, w4a16_dtype_t xt, const w4a16_mx_t* w) {
  MxRows r;
  if (M <= 0 || check_mx_weight(w) != W4A16_OK || rows_of(nullptr, xt, M, w->K, r) != W4A16_OK ||
      static_cast<size_t>(M) * w->rows > kMxMaxValues)
    return 0;
  return plan_mx_gemm(M, w, r.kind).bytes;
}

extern "C" w4a16_status_t w4a16_mx_gemm(const void* x, w4a16_dtype_t xt, int32_t M, const w4a16_mx_t* w, void* y,
                                        w4a16_dtype_t yt, void* ws, size_t ws_bytes, hipStream_t stream) {
  w4a16_status_t st = check_mx_weight(w);
  MxRows r;
  if (st != W4A16_OK || (st = rows_of(x, xt, M, w->K, r)) != W4A16_OK) return st;
  return mx_gemm(r, M, w, y, yt, ws, ws_bytes, stream);
}

extern "C" size_t w4a16_mx_gemm_a4_workspace_bytes(int32_t M, const w4a16_mx_t* w) {
  if (M <= 0 || check_mx_weight(w) != W4A16_OK || check_mx_shape(M, w->K) != W4A16_OK ||
      static_cast<size_t>(M) * w->rows > kMxMaxValues)
    return 0;
  return plan_mx_gemm(M, w, kMxXfp4).bytes;
}

extern "C" w4a16_status_t w4a16_mx_gemm_a4(const w4a16_mx_t* x, const w4a16_mx_t* w, void* y, w4a16_dtype_t yt,
                                           void* ws, size_t ws_bytes, hipStream_t stream) {
  w4a16_status_t st = check_mx_weight(w);
  MxRows r;
  if (st != W4A16_OK || (st = rows_of(x, w->K, r)) != W4A16_OK) return st;
  return mx_gemm(r, x->rows, w, y, yt, ws, ws_bytes, stream);
}

extern "C" size_t w4a16_mx_swiglu_mlp_workspace_bytes(int32_t M, w4a16_dtype_t xt, const w4a16_mx_t* gate,
                                                      const w4a16_mx_t* up, const w4a16_mx_t* down) {
  MxRows r;
  if (M <= 0 || check_mx_mlp(gate, up, down) != W4A16_OK || rows_of(nullptr, xt, M, gate->K, r) != W4A16_OK ||
      check_mx_shape(M, gate->rows) != W4A16_OK)
    return 0;
  return plan_mx_mlp(M, gate, r.kind).bytes;
}

extern "C" w4a16_status_t w4a16_mx_swiglu_mlp(const void* x, w4a16_dtype_t xt, int32_t M, const w4a16_mx_t* gate,
                                              const w4a16_mx_t* up, const w4a16_mx_t* down, void* y,
                                              w4a16_dtype_t yt, void* ws, size_t ws_bytes, hipStream_t stream) {
  w4a16_status_t st = check_mx_mlp(gate, up, down);
  MxRows r;
  if (st != W4A16_OK || (st = rows_of(x, xt, M, gate->K, r)) != W4A16_OK) return st;
  return mx_swiglu_mlp(r, M, gate, up, down, y, yt, ws, ws_bytes, stream);
}

extern "C" size_t w4a16_mx_swiglu_mlp_a4_workspace_bytes(int32_t M, const w4a16_mx_t* gate, const w4a16_mx_t* up,
                                                         const w4a16_mx_t* down) {
  if (M <= 0 || check_mx_mlp(gate, up, down) != W4A16_OK || check_mx_shape(M, gate->K) != W4A16_OK ||
      check_mx_shape(M, gate->rows) != W4A16_OK)
    return 0;
  return plan_mx_mlp(M, gate, kMxXfp4).bytes;
}

extern "C" w4a16_status_t w4a16_mx_swiglu_mlp_a4(const w4a16_mx_t* x, const w4a16_mx_t* gate, const w4a16_mx_t* up,
                                                 const w4a16_mx_t* down, void* y, w4a16_dtype_t yt, void* ws,
                                                 size_t ws_bytes, hipStream_t stream) {
  w4a16_status_t st = check_mx_mlp(gate, up, down);
  MxRows r;
  if (st != W4A16_OK || (st = rows_of(x, gate->K, r)) != W4A16_OK) return st;
  return mx_swiglu_mlp(r, x->rows, gate, up, down, y, yt, ws, ws_bytes, stream);
}
