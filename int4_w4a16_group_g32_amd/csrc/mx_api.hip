// Entry points of the products with MXFP4 weights: checks, workspace plans and
// launches.
#include "mx.h"

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

// Pointers and overlaps shared by the products.
w4a16_status_t check_io(const MxRows& r, const void* y, size_t ybytes, const void* ws) {
  if (r.x == nullptr || y == nullptr || ws == nullptr) return W4A16_ERR_INVALID_ARG;
  if (!aligned16(r.x) || !aligned16(y) || !aligned16(ws)) return W4A16_ERR_INVALID_ARG;
  if (ranges_overlap(r.x, r.bytes, y, ybytes) || ranges_overlap(r.xs, r.sbytes, y, ybytes))
    return W4A16_ERR_INVALID_ARG;
  return W4A16_OK;
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

struct MxGemmPlan {
  size_t bytes = 0;
};
MxGemmPlan plan_mx_gemm(int M, const w4a16_mx_t* w, MxX kind) {
  MxGemmPlan p;
  p.bytes = 256;
  return p;
}

struct MxMlpPlan {
  size_t h_off = 0, hs_off = 0, bytes = 0;
};
MxMlpPlan plan_mx_mlp(int M, const w4a16_mx_t* gate, MxX kind) {
  MxMlpPlan p;
  Carve c;
  const size_t n = static_cast<size_t>(M) * gate->rows;
  c.take(p.h_off, kind == kMxXfp4 ? n / 2 : n * 4);
  c.take(p.hs_off, kind == kMxXfp4 ? n / kMxBlock : 0);
  p.bytes = std::max<size_t>(c.cursor, 256);
  return p;
}

w4a16_status_t mx_gemm(const MxRows& r, int M, const w4a16_mx_t* w, void* y, w4a16_dtype_t yt, void* ws,
                       size_t ws_bytes, hipStream_t stream) {
  if (yt != W4A16_F32 && yt != W4A16_BF16) return W4A16_ERR_INVALID_ARG;
  if (M == 0 || w->rows == 0 || w->K == 0) return W4A16_OK;
  const w4a16_status_t st = check_io(r, y, static_cast<size_t>(M) * w->rows * dtype_bytes(yt), ws);
  if (st != W4A16_OK) return st;
  if (static_cast<size_t>(M) * w->rows > kMxMaxValues) return W4A16_ERR_UNSUPPORTED;
  const MxGemmPlan p = plan_mx_gemm(M, w, r.kind);
  if (ws_bytes < p.bytes) return W4A16_ERR_WORKSPACE;
  MxArgs a = mx_args(r, M, w, nullptr, y);
  a.y_bf16 = yt == W4A16_BF16;
  return launch_mx_stream(r.kind, false, a, stream) == hipSuccess ? W4A16_OK : W4A16_ERR_HIP;
}

w4a16_status_t mx_swiglu_mlp(const MxRows& r, int M, const w4a16_mx_t* gate, const w4a16_mx_t* up,
                             const w4a16_mx_t* down, void* y, w4a16_dtype_t yt, void* ws, size_t ws_bytes,
                             hipStream_t stream) {
  if (yt != W4A16_F32 && yt != W4A16_BF16) return W4A16_ERR_INVALID_ARG;
  if (M == 0 || gate->K == 0 || gate->rows == 0) return W4A16_OK;
  w4a16_status_t st = check_io(r, y, static_cast<size_t>(M) * gate->K * dtype_bytes(yt), ws);
  if (st != W4A16_OK) return st;
  if ((st = check_mx_shape(M, gate->rows)) != W4A16_OK) return st;
  const MxMlpPlan p = plan_mx_mlp(M, gate, r.kind);
  if (ws_bytes < p.bytes) return W4A16_ERR_WORKSPACE;
  uint8_t* wsb = static_cast<uint8_t*>(ws);
  MxRows h;
  h.x = wsb + p.h_off;
  h.xs = wsb + p.hs_off;
  // h of bf16 rows keeps 16 bits: the next rounding, y's or h's neighbours' sum, is coarser by far
  h.kind = r.kind == kMxXbf16 ? kMxXf32h : r.kind;
  MxArgs gu = mx_args(r, M, gate, up, wsb + p.h_off);
  gu.ys = wsb + p.hs_off;
  if (launch_mx_stream(r.kind, true, gu, stream) != hipSuccess) return W4A16_ERR_HIP;
  MxArgs dn = mx_args(h, M, down, nullptr, y);
  dn.y_bf16 = yt == W4A16_BF16;
  return launch_mx_stream(h.kind, false, dn, stream) == hipSuccess ? W4A16_OK : W4A16_ERR_HIP;
}

}  // namespace
}  // namespace w4

using namespace w4;

extern "C" size_t w4a16_mx_gemm_workspace_bytes(int32_t M, w4a16_dtype_t xt, const w4a16_mx_t* w) {
  MxRows r;
  if (M <= 0 || check_mx_weight(w) != W4A16_OK || rows_of(nullptr, xt, M, w->K, r) != W4A16_OK) return 0;
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
  if (M <= 0 || check_mx_weight(w) != W4A16_OK || check_mx_shape(M, w->K) != W4A16_OK) return 0;
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
