// The norms round a block, in one pass over the rows:
//   s = r + alpha * gate * post(y),   post(y) = y / sqrt(mean(y^2) + eps) * post_w  (or y)
//   n = s / sqrt(mean(s^2) + eps) * pre_w
// s in the residual stream's type, n in float32, bf16 or MXFP4 rows.
//
// Bound by memory: y, r and the gate are read once, s and n written once.  A
// workgroup holds one row in registers, eight adjacent values a thread and
// chunk (16 or 32 bytes a load), so both means need no second read.  The means
// and everything between the loads and stores are float32; where n goes to
// 4-bit codes they are float64, since a code's borders turn a last-bit
// difference into half a step: the codes then do not depend on the order of the
// sums (the vector units' float64 work stays under the memory's time).
#include "mx.h"

#include <type_traits>

namespace w4 {
namespace {

struct NormArgs {
  const void *y, *r, *post_w, *gate, *pre_w;
  void *r_out, *n;
  uint8_t* n_scales;
  int H, gate_rows;
  int y_bf16, r_bf16, w_bf16, n_bf16;
  double alpha, eps;
};

// Eight values from element 8 i.
__device__ __forceinline__ void get8(const void* p, size_t i, int bf16, float v[8]) {
  if (bf16) {
    const uint4 a = static_cast<const uint4*>(p)[i];
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = __uint_as_float(w[j] << 16);
      v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
  } else {
    const float4 a = static_cast<const float4*>(p)[2 * i], b = static_cast<const float4*>(p)[2 * i + 1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
}
__device__ __forceinline__ void put8(void* p, size_t i, int bf16, const float v[8]) {
  if (bf16) {
    uint32_t b[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) b[j] = f32_to_bf16(v[2 * j]) | static_cast<uint32_t>(f32_to_bf16(v[2 * j + 1])) << 16;
    static_cast<uint4*>(p)[i] = make_uint4(b[0], b[1], b[2], b[3]);
  } else {
    static_cast<float4*>(p)[2 * i] = make_float4(v[0], v[1], v[2], v[3]);
    static_cast<float4*>(p)[2 * i + 1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}

// v as a float, or where v is none, the one of its two neighbours with an odd
// last bit: a later rounding to few bits, whose borders are even, then goes as
// v's own would.
__device__ __forceinline__ float rounded_to_odd(double v) {
  const float f = static_cast<float>(v);
  const double a = fabs(v), b = fabs(static_cast<double>(f));
  const uint32_t u = __float_as_uint(f);
  return b == a || (u & 1) || !(b <= 3.4028234663852886e38) ? f : __uint_as_float(b > a ? u - 1 : u + 1);
}

template <typename F>
__device__ __forceinline__ F row_sum(F v, F* lds) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  const int waves = static_cast<int>(blockDim.x) >> 6;
  __syncthreads();  // (the previous sum is read)
  if (lane_id() == 0) lds[wave_id()] = v;
  __syncthreads();
  F t = lds[0];
  for (int w = 1; w < waves; ++w) t += lds[w];
  return t;
}

// kC chunks of eight values a thread; chunk c of thread t is t + c * blockDim.x.
template <int kC, bool kMx>
__global__ __launch_bounds__(1024) void block_norm_kernel(const NormArgs a) {
  using F = std::conditional_t<kMx, double, float>;
  __shared__ F lds[16];
  const int t = static_cast<int>(threadIdx.x), T = static_cast<int>(blockDim.x);
  const int n8 = a.H / 8;
  const size_t row = blockIdx.x, base = row * n8;
  float in[8];
  F s[kC][8];
#pragma unroll
  for (int c = 0; c < kC; ++c) {
    const int i = t + c * T;
#pragma unroll
    for (int j = 0; j < 8; ++j) in[j] = 0.0f;
    if (i < n8) get8(a.y, base + i, a.y_bf16, in);
#pragma unroll
    for (int j = 0; j < 8; ++j) s[c][j] = in[j];
  }
  F post = 1;
  if (a.post_w != nullptr) {
    F q = 0;
#pragma unroll
    for (int c = 0; c < kC; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) q += s[c][j] * s[c][j];
    post = 1 / sqrt(row_sum(q, lds) / a.H + static_cast<F>(a.eps));
  }
  F q = 0;
#pragma unroll
  for (int c = 0; c < kC; ++c) {
    const int i = t + c * T;
    if (i >= n8) continue;
    float w[8];
    if (a.post_w != nullptr) {
      get8(a.post_w, i, a.w_bf16, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) s[c][j] = s[c][j] * post * w[j];
    }
    if (a.gate != nullptr) {
      get8(a.gate, (a.gate_rows == 1 ? 0 : base) + i, a.w_bf16, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) s[c][j] *= w[j];
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) s[c][j] *= static_cast<F>(a.alpha);
    if (a.r != nullptr) {
      get8(a.r, base + i, a.r_bf16, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) s[c][j] += w[j];
    }
    // s as it is stored
    float o[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      o[j] = static_cast<float>(s[c][j]);
      if (a.r_bf16) o[j] = bf16_to_f32(f32_to_bf16(o[j]));
      s[c][j] = o[j];
      q += s[c][j] * s[c][j];
    }
    if (a.r_out != nullptr) put8(a.r_out, base + i, a.r_bf16, o);
  }
  if (a.n == nullptr) return;
  const F pre = 1 / sqrt(row_sum(q, lds) / a.H + static_cast<F>(a.eps));
#pragma unroll
  for (int c = 0; c < kC; ++c) {
    const int i = t + c * T;
    if (i >= n8) continue;  // (four threads of a block of 32 go together)
    float w[8];
    get8(a.pre_w, i, a.w_bf16, w);
    if constexpr (!kMx) {
      float o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = s[c][j] * pre * w[j];
      put8(a.n, base + i, a.n_bf16, o);
    } else {
      double v[8], m = 0;
      bool bad = false;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[j] = s[c][j] * pre * w[j];
        bad |= !(fabs(v[j]) <= 3.4028234663852886e38);
        m = fmax(m, fabs(v[j]));
      }
      m = fmax(m, __shfl_xor(m, 1));
      m = fmax(m, __shfl_xor(m, 2));
      int b = bad;
      b |= __shfl_xor(b, 1);
      b |= __shfl_xor(b, 2);
      // floor(log2 m) - 2, at least -127 (0 and float64 subnormals have exponent field 0)
      const int e = static_cast<int>(__double_as_longlong(m) >> 52) - 1023;
      const uint32_t byte = b ? 255u : static_cast<uint32_t>(max(e - 2 + 127, 0));
      // 2^(127 - byte), exact in float64
      const double inv = __longlong_as_double(static_cast<long long>(1023 + 127 - static_cast<int>(byte)) << 52);
      float o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = b ? 0.0f : rounded_to_odd(v[j] * inv);
      static_cast<uint32_t*>(a.n)[base + i] = mx_codes8(o);
      if ((i & 3) == 0) a.n_scales[(base + i) >> 2] = static_cast<uint8_t>(byte);
    }
  }
}

template <int kC>
void start(const NormArgs& a, bool mx, int M, int T, hipStream_t stream) {
  if (mx)
    block_norm_kernel<kC, true><<<M, T, 0, stream>>>(a);
  else
    block_norm_kernel<kC, false><<<M, T, 0, stream>>>(a);
}

bool good_type(w4a16_dtype_t t) { return t == W4A16_F32 || t == W4A16_BF16; }

}  // namespace
}  // namespace w4

using namespace w4;

extern "C" w4a16_status_t w4a16_block_norm(const w4a16_norm_t* p, int32_t M, int32_t H, hipStream_t stream) {
  if (p == nullptr || M < 0 || H < 0) return W4A16_ERR_INVALID_ARG;
  if (!good_type(p->y_type) || !good_type(p->r_type) || !good_type(p->w_type)) return W4A16_ERR_INVALID_ARG;
  const bool mx = p->n_codes != nullptr || p->n_scales != nullptr;
  if (mx && (p->n != nullptr || p->n_codes == nullptr || p->n_scales == nullptr)) return W4A16_ERR_INVALID_ARG;
  if (p->n != nullptr && !good_type(p->n_type)) return W4A16_ERR_INVALID_ARG;
  const bool has_n = mx || p->n != nullptr;
  if (H % (mx ? kMxBlock : 8) != 0 || H > W4A16_NORM_MAX_H || M > kMxMaxRows) return W4A16_ERR_UNSUPPORTED;
  if (M == 0 || H == 0) return W4A16_OK;
  if (!has_n && p->r_out == nullptr) return W4A16_ERR_INVALID_ARG;
  if (p->y == nullptr || (has_n && p->pre_w == nullptr)) return W4A16_ERR_INVALID_ARG;
  if (p->gate != nullptr && p->gate_rows != 1 && p->gate_rows != M) return W4A16_ERR_INVALID_ARG;
  const size_t mh = static_cast<size_t>(M) * H;
  const size_t rb = mh * dtype_bytes(p->r_type), wb = H * dtype_bytes(p->w_type);
  struct {
    const void* p;
    size_t bytes;
  } ins[] = {{p->y, mh * dtype_bytes(p->y_type)},
             {p->r, rb},
             {p->post_w, wb},
             {p->pre_w, wb},
             {p->gate, wb * (p->gate_rows == 1 ? 1 : M)}},
    outs[] = {{p->r_out, rb},
              {p->n, p->n ? mh * dtype_bytes(p->n_type) : 0},
              {p->n_codes, mh / 2},
              {p->n_scales, mh / kMxBlock}};
  for (const auto& o : outs) {
    if (o.p == nullptr) continue;
    if (!aligned16(o.p)) return W4A16_ERR_INVALID_ARG;
    for (const auto& i : ins) {
      if (i.p == nullptr || (i.p == p->r && o.p == p->r && o.p == p->r_out)) continue;  // (r in place)
      if (ranges_overlap(i.p, i.bytes, o.p, o.bytes)) return W4A16_ERR_INVALID_ARG;
    }
    for (const auto& q : outs)
      if (q.p != nullptr && &q != &o && ranges_overlap(q.p, q.bytes, o.p, o.bytes)) return W4A16_ERR_INVALID_ARG;
  }
  for (const auto& i : ins)
    if (!aligned16(i.p)) return W4A16_ERR_INVALID_ARG;

  NormArgs a{};
  a.y = p->y, a.r = p->r, a.post_w = p->post_w, a.gate = p->gate, a.pre_w = p->pre_w;
  a.r_out = p->r_out, a.n = mx ? p->n_codes : p->n, a.n_scales = p->n_scales;
  a.H = H, a.gate_rows = p->gate_rows;
  a.y_bf16 = p->y_type == W4A16_BF16, a.r_bf16 = p->r_type == W4A16_BF16;
  a.w_bf16 = p->w_type == W4A16_BF16, a.n_bf16 = p->n_type == W4A16_BF16;
  a.alpha = p->alpha, a.eps = p->eps;
  const int n8 = H / 8;
  const int C = n8 <= 1024 ? 1 : (n8 <= 2048 ? 2 : 4);
  const int T = ((n8 + C - 1) / C + 63) / 64 * 64;
  if (C == 1) start<1>(a, mx, M, T, stream);
  else if (C == 2) start<2>(a, mx, M, T, stream);
  else start<4>(a, mx, M, T, stream);
  return launch_status();
}
