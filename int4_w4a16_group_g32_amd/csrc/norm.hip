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
// sums.
//
// Measured, 2048 x 7168 with a gate a row: bf16 to bf16 33.1 us (4.4 TB/s; a copy
// 4.76), to MXFP4 36.5 (3.4 TB/s: fewer bytes and the same barriers, so the
// float64 work is what is left over); float32 62.5 and 65.2; bf16 on a float32
// stream to MXFP4 60.2.  Above H = 8192 the forms that are not all bf16 spill
// (1024 threads leave 128 registers): 1024 x 16384 float32 143 us, to MXFP4 201.
#include "mx.h"

#include <type_traits>

namespace w4 {
namespace {

struct NormArgs {
  const void *y, *r, *post_w, *gate, *pre_w;
  void *r_out, *n;
  uint8_t* n_scales;
  int M, H, gate_rows;
  int y_bf16, r_bf16, w_bf16, n_bf16;
  double alpha, eps;
};

// Eight values from element 8 i, as they are stored; kB: bf16 for certain.
template <bool kB>
struct Raw8 {
  uint4 v[kB ? 1 : 2];
};
template <bool kB>
__device__ __forceinline__ Raw8<kB> get8(const void* p, size_t i, int bf16) {
  Raw8<kB> r;
  if constexpr (kB) {
    r.v[0] = static_cast<const uint4*>(p)[i];
  } else if (bf16) {
    r.v[0] = static_cast<const uint4*>(p)[i];
  } else {
    r.v[0] = static_cast<const uint4*>(p)[2 * i];
    r.v[1] = static_cast<const uint4*>(p)[2 * i + 1];
  }
  return r;
}
template <bool kB>
__device__ __forceinline__ void values8(const Raw8<kB>& r, int bf16, float v[8]) {
  constexpr int l = kB ? 0 : 1;
  const uint32_t w[8] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w, r.v[l].x, r.v[l].y, r.v[l].z, r.v[l].w};
  if (kB || bf16) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = __uint_as_float(w[j] << 16);
      v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(w[j]);
  }
}
__device__ __forceinline__ void put8(void* p, size_t i, int bf16, const float v[8]) {
  if (bf16) {
    uint32_t b[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      b[j] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{v[2 * j], v[2 * j + 1]}, bf16x2));
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

__device__ __forceinline__ bool is_normal(float v) { return __builtin_amdgcn_classf(v, 0x108); }
__device__ __forceinline__ bool is_normal(double) { return true; }

// Sum over the workgroup, the same bits in every thread.
template <typename F>
__device__ __forceinline__ F row_sum(F v, F* lds) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  const int waves = static_cast<int>(blockDim.x) >> 6;
  if (lane_id() == 0) lds[wave_id()] = v;
  __syncthreads();
  F t = lds[0];
  for (int w = 1; w < waves; ++w) t += lds[w];
  return t;
}

// A block's 32 values lie in four threads.
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  v = max(v, static_cast<uint32_t>(__shfl_xor(static_cast<int>(v), 1)));
  return max(v, static_cast<uint32_t>(__shfl_xor(static_cast<int>(v), 2)));
}

// Codes and scale byte of n = s * w * pre, eight values of a block of 32, as
// float64 gives them.  The products are first taken in float32, off by at most
// four half-steps; borders between codes, and powers of two, have at most two
// mantissa bits, so a value whose lower 21 are 16 steps or more from all zeros
// is on the same side in float64.  Where some value of the wave is nearer (1 in
// 2^16, and every zero), the wave goes by float64.
__device__ __forceinline__ uint32_t codes_of(const float s[8], const float w[8], double pre, uint32_t& byte) {
  const float p = static_cast<float>(pre);
  float v[8];
  uint32_t m = 0, low = ~0u;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    v[j] = s[j] * w[j] * p;
    const uint32_t u = __float_as_uint(v[j]);
    m = max(m, u & 0x7fffffffu);
    low = min(low, (u + 16) & 0x1fffffu);
  }
  m = quad_max(m);
  // s * w below 2^-126 has lost bits, but with pre below 2^30 such a value, as one
  // that is itself below 2^-126, is code 0 either way beside a largest of 2^-90
  const bool near = low < 32 || m < (127u - 90u) << 23 || m >= 255u << 23 || !(p > 0x1p-100f && p < 0x1p30f);
  float o[8];
  if (!__any(near)) {
    byte = mx_scale_byte(m);
    const float inv = mx_scale_inverse(byte);
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = v[j] * inv;
    return mx_codes8(o);
  }
  double d[8];
  m = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    d[j] = static_cast<double>(s[j]) * pre * w[j];
    // (the upper half orders magnitudes by their exponents, which is all a scale needs)
    m = max(m, static_cast<uint32_t>(__double_as_longlong(d[j]) >> 32) & 0x7fffffffu);
  }
  m = quad_max(m);
  const bool bad = m >= (1023u + 128u) << 20;  // no float: beyond its range, an infinity or NaN
  byte = bad ? 255u : static_cast<uint32_t>(max(static_cast<int>(m >> 20) - 1023 - 2 + 127, 0));
  // 2^(127 - byte), exact in float64
  const double inv = __longlong_as_double(static_cast<long long>(1023 + 127 - static_cast<int>(byte)) << 52);
#pragma unroll
  for (int j = 0; j < 8; ++j) o[j] = bad ? 0.0f : rounded_to_odd(d[j] * inv);
  return mx_codes8(o);
}

// kC chunks of eight values a thread; chunk c of thread t is t + c * blockDim.x.
// kB: y, r, the weights and gate are bf16; then a workgroup takes rows
// blockIdx.x, + gridDim.x, ..., and asks for the next row's values as soon as it
// holds s of its own (else one row: the values of two would not fit).
// Two chunks are launched with at most 512 threads, four of bf16 too; with room
// for 1024 the two-chunk float64 form of other types would spill.
template <int kC, bool kMx, bool kB>
__global__ __launch_bounds__(kC == 2 || (kB && kC > 1) ? 512 : 1024) void block_norm_kernel(const NormArgs a) {
  using F = std::conditional_t<kMx, double, float>;
  constexpr bool kEarly = kB || kC == 1;  // (else too many registers)
  __shared__ F lds[2][2][16];
  const int t = static_cast<int>(threadIdx.x), T = static_cast<int>(blockDim.x);
  const int n8 = a.H / 8;
  Raw8<kB> y[kC], r[kC], g[kC], pw[kC], nw[kC];
  auto load = [&](int row) {
    const size_t base = static_cast<size_t>(row) * n8;
#pragma unroll
    for (int c = 0; c < kC; ++c) {
      const int i = t + c * T;
      if (i >= n8) continue;
      y[c] = get8<kB>(a.y, base + i, a.y_bf16);
      if (kEarly && a.r != nullptr) r[c] = get8<kB>(a.r, base + i, a.r_bf16);
      if (kEarly && a.gate != nullptr) g[c] = get8<kB>(a.gate, (a.gate_rows == 1 ? 0 : base) + i, a.w_bf16);
      if (kC == 1 && a.post_w != nullptr) pw[c] = get8<kB>(a.post_w, i, a.w_bf16);
    }
  };
  load(blockIdx.x);
#pragma unroll
  for (int c = 0; c < kC; ++c)
    if (kC == 1 && a.n != nullptr && t < n8) nw[c] = get8<kB>(a.pre_w, t, a.w_bf16);
  int turn = 0;
  for (int row = blockIdx.x; row < a.M; row += gridDim.x, turn ^= 1) {
    const size_t base = static_cast<size_t>(row) * n8;
    F scale = static_cast<F>(a.alpha);
    if (a.post_w != nullptr) {
      F q = 0;
#pragma unroll
      for (int c = 0; c < kC; ++c) {
        if (t + c * T >= n8) continue;
        float v[8];
        values8(y[c], a.y_bf16, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) q += static_cast<F>(v[j]) * static_cast<F>(v[j]);
      }
      scale *= 1 / sqrt(row_sum(q, lds[turn][0]) / a.H + static_cast<F>(a.eps));
    }
    F q = 0;
    float s[kC][8];  // s as it is stored
#pragma unroll
    for (int c = 0; c < kC; ++c) {
      const int i = t + c * T;
      if (i >= n8) continue;
      float v[8], w[8];
      F p[8];
      if (!kEarly && a.r != nullptr) r[c] = get8<kB>(a.r, base + i, a.r_bf16);
      if (!kEarly && a.gate != nullptr) g[c] = get8<kB>(a.gate, (a.gate_rows == 1 ? 0 : base) + i, a.w_bf16);
      if (kC > 1 && a.post_w != nullptr) pw[c] = get8<kB>(a.post_w, i, a.w_bf16);
      auto product = [&](auto* o, bool& normal) {
        values8(y[c], a.y_bf16, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = v[j];
        if (a.post_w != nullptr) {
          values8(pw[c], a.w_bf16, w);
#pragma unroll
          for (int j = 0; j < 8; ++j) o[j] *= w[j], normal &= is_normal(o[j]);
        }
        if (a.gate != nullptr) {
          values8(g[c], a.w_bf16, w);
#pragma unroll
          for (int j = 0; j < 8; ++j) o[j] *= w[j], normal &= is_normal(o[j]);
        }
      };
      // In front of codes the products are float64's too: of three bf16 values
      // float32 has them exactly inside its normal range, and a wave with one
      // outside (or a zero) takes float64 (2048 x 7168 bf16: always 37.6 us, so 36.5)
      bool normal = true;
      if constexpr (kMx && kB) {
        float f[8];
        product(f, normal);
        if (__any(!normal)) {
          product(p, normal);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) p[j] = f[j];
        }
      } else {
        product(p, normal);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = 0.0f;
      if (a.r != nullptr) values8(r[c], a.r_bf16, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) s[c][j] = static_cast<float>(p[j] * scale + static_cast<F>(w[j]));
      if (kB || a.r_bf16) {
        uint32_t b[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          b[j] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{s[c][2 * j], s[c][2 * j + 1]}, bf16x2));
          s[c][2 * j] = __uint_as_float(b[j] << 16);
          s[c][2 * j + 1] = __uint_as_float(b[j] & 0xffff0000u);
        }
        if (a.r_out != nullptr) static_cast<uint4*>(a.r_out)[base + i] = make_uint4(b[0], b[1], b[2], b[3]);
      } else if (a.r_out != nullptr) {
        put8(a.r_out, base + i, 0, s[c]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) q += static_cast<F>(s[c][j]) * static_cast<F>(s[c][j]);
    }
    if (kB && row + static_cast<int>(gridDim.x) < a.M) load(row + gridDim.x);
    if (a.n == nullptr) continue;
    const F pre = 1 / sqrt(row_sum(q, lds[turn][1]) / a.H + static_cast<F>(a.eps));
#pragma unroll
    for (int c = 0; c < kC; ++c) {
      const int i = t + c * T;
      if (i >= n8) continue;  // (four threads of a block of 32 go together)
      if (kC > 1) nw[c] = get8<kB>(a.pre_w, i, a.w_bf16);
      float w[8];
      values8(nw[c], a.w_bf16, w);
      if constexpr (!kMx) {
        float o[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = s[c][j] * pre * w[j];
        put8(a.n, base + i, a.n_bf16, o);
      } else {
        uint32_t byte;
        static_cast<uint32_t*>(a.n)[base + i] = codes_of(s[c], w, pre, byte);
        if ((i & 3) == 0) a.n_scales[(base + i) >> 2] = static_cast<uint8_t>(byte);
      }
    }
  }
}

constexpr int kCus = 256;

template <int kC, bool kB>
void start(const NormArgs& a, bool mx, int T, hipStream_t stream) {
  // (a compute unit holds four workgroups of 256 threads with their next rows)
  const int blocks = kB ? std::min(a.M, kCus * std::max(1, 1024 / T)) : a.M;
  if (mx)
    block_norm_kernel<kC, true, kB><<<blocks, T, 0, stream>>>(a);
  else
    block_norm_kernel<kC, false, kB><<<blocks, T, 0, stream>>>(a);
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
      if (i.p == nullptr) continue;
      // in place: a thread has read its values of r, and of y where that is r, before it writes them;
      // a weight or gate there would be read by other rows too
      const bool in_place = &i == &ins[1] || (&i == &ins[0] && p->y == p->r && p->y_type == p->r_type);
      if (&o == &outs[0] && p->r_out == p->r && in_place) continue;
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
  a.M = M, a.H = H, a.gate_rows = p->gate_rows;
  a.y_bf16 = p->y_type == W4A16_BF16, a.r_bf16 = p->r_type == W4A16_BF16;
  a.w_bf16 = p->w_type == W4A16_BF16, a.n_bf16 = p->n_type == W4A16_BF16;
  a.alpha = p->alpha, a.eps = p->eps;
  // a thread's chunks: one where there are few rows (a row's latency counts),
  // else as few as leave several rows to a compute unit (2048 bf16 rows of 7168
  // to MXFP4: one chunk 57 us, two 36, four 44)
  const int n8 = H / 8;
  const int C = n8 <= 256 || (M <= kCus && n8 <= 1024) ? 1 : (n8 <= 1024 ? 2 : 4);
  const int T = ((n8 + C - 1) / C + 63) / 64 * 64;
  const bool b = a.y_bf16 && a.w_bf16 && (a.r == nullptr || a.r_bf16) && a.r_bf16 && (C == 1 || T <= 512);
  if (C == 1) b ? start<1, true>(a, mx, T, stream) : start<1, false>(a, mx, T, stream);
  else if (C == 2) b ? start<2, true>(a, mx, T, stream) : start<2, false>(a, mx, T, stream);
  else b ? start<4, true>(a, mx, T, stream) : start<4, false>(a, mx, T, stream);
  return launch_status();
}
