// Streaming W4A16 products of a few rows (device helpers).
//
// One v_mfma_f32_16x16x32_f16 spans one 32-row code block and 16 weight
// columns: B holds the exact codes (codes_f16), A up to 16 rows of f16 pieces.
// A wave owns 64 columns; a lane reads one 16-byte GROUPED slot (word kb of
// four adjacent columns, one per MFMA block) and their four scales per block,
// and the block's result is scaled by s[g][n] on float32 accumulators.
//
// Rows are staged in LDS as f16 pieces of x * 2^e, with one power of two per
// row that puts its largest magnitude in [2^14, 2^15): two pieces for float32
// values (22 significant bits), one for bf16 ones (all 8; f16's smallest is
// 2^-24, so both hold values to within 2^-39 of the row's largest at best, and
// bf16 ones exactly from 2^-31 of it on).  Row m of x is A
// row 4 (m & 3) + (m >> 2), or with two pieces 4 (m & 3) + 2 (m >> 2) + piece,
// so that element i of a lane's result (A row 4 (lane >> 4) + i) belongs to
// row (lane >> 4) + 4 i: up to four rows need one accumulator per column and
// lane, not four.  LDS holds the rows there are and no others (few rows leave
// room for long windows); lanes of absent A rows read a unit of zeros.
#pragma once

#include <type_traits>

#include "common.h"
#include "mfma_ops.h"

namespace w4 {

constexpr int kStreamRows = 16;  // A rows
constexpr int kStreamRing = 4;   // groups of codes in flight per wave
constexpr int kStreamLds0 = 4;   // first unit of the window (unit 0 is zeros)

// Unit of (group, k block, LDS row); 2^rshift LDS rows a group: row m's piece
// p is LDS row m * kP + p.
__device__ __forceinline__ int stream_unit(int g, int kb, int r, int rshift) {
  return kStreamLds0 + (((g * 4 + kb) << rshift) + r);
}

// log2 of the LDS rows that hold n rows of kP pieces.
template <int kP>
__device__ __forceinline__ int stream_rshift(int n) {
  return (n > 1 ? 32 - __builtin_clz(n - 1) : 0) + (kP - 1);
}

// Where a lane finds its A fragment: unit `at` of group 0, `step` units a group.
struct StreamFrag {
  int at, step;
};
template <int kP>
__device__ __forceinline__ StreamFrag stream_frag(int lane, int nrows, int g0, int rshift) {
  const int lc = lane & 15, kb = lane >> 4;
  const int m = kP == 2 ? (lc >> 2) + 4 * ((lc >> 1) & 1) : (lc >> 2) + 4 * (lc & 3);
  const int p = kP == 2 ? lc & 1 : 0;
  if (m >= nrows) return StreamFrag{0, 0};
  return StreamFrag{stream_unit(g0, kb, m * kP + p, rshift), 4 << rshift};
}

// The exponent that brings a row's largest magnitude into [2^14, 2^15) (any
// will do for a row of zeros; infinities and NaNs pass through as such), kept
// to where 2^e and 2^-e are normal floats.
__device__ __forceinline__ int stream_exp(float amax) {
  const int e = 15 - __builtin_amdgcn_frexp_expf(amax);
  return e > 126 ? 126 : e;
}

// Largest value of the wave, as a scalar: row shifts within 16 lanes, then
// broadcasts across rows; lane 63 ends with all of them.  (Non-negative
// floats compare as their bits.)
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  auto step = [&](auto ctrl, auto rows) {
    const uint32_t t = static_cast<uint32_t>(__builtin_amdgcn_update_dpp(
        0, static_cast<int>(v), decltype(ctrl)::value, decltype(rows)::value, 0xf, false));
    v = v > t ? v : t;
  };
  using std::integral_constant;
  step(integral_constant<int, 0x111>{}, integral_constant<int, 0xf>{});  // row_shr:1
  step(integral_constant<int, 0x112>{}, integral_constant<int, 0xf>{});
  step(integral_constant<int, 0x114>{}, integral_constant<int, 0xf>{});
  step(integral_constant<int, 0x118>{}, integral_constant<int, 0xf>{});
  step(integral_constant<int, 0x142>{}, integral_constant<int, 0xa>{});  // row_bcast:15
  step(integral_constant<int, 0x143>{}, integral_constant<int, 0xc>{});  // row_bcast:31
  return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v), 63));
}

// Eight values (already scaled) as pieces, in the order codes_f16 expands to.
template <int kP>
__device__ __forceinline__ void stream_pieces(const float v[8], half8 p[2]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float t = v[kCodeOrder[i]];
    const _Float16 h = static_cast<_Float16>(t);
    p[0][i] = h;
    if (kP == 2) p[1][i] = static_cast<_Float16>(t - static_cast<float>(h));
  }
}

// The pieces to units u and, of two pieces, u + 1.
template <int kP>
__device__ __forceinline__ void stream_put(uint4* lds, int u, const float v[8]) {
  half8 p[2];
  stream_pieces<kP>(v, p);
#pragma unroll
  for (int j = 0; j < kP; ++j) *reinterpret_cast<half8*>(lds + u + j) = p[j];
}
template <int kP>
__device__ __forceinline__ void stream_put_zero(uint4* lds, int u) {
  lds[u] = make_uint4(0, 0, 0, 0);
  if (kP == 2) lds[u + 1] = make_uint4(0, 0, 0, 0);
}

struct StreamCodes {
  uint32_t w[4];
  float s[4];
};

// Codes and scales of one group through raw buffer resources: the group's rows
// are wave-uniform bases in scalar registers, the lane's place in them one
// 32-bit offset (no 64-bit vector address arithmetic per load).
struct StreamLane {
  int w, s;  // bytes
};
__device__ __forceinline__ StreamLane stream_lane(int col, int lane) {
  return StreamLane{(col + lane) * 16, (col + 4 * (lane & 15)) * 4};
}
constexpr int kStreamBufFlags = 0x00020000;  // dword 3 of a raw buffer resource on gfx9
constexpr int kStreamNt = 2;                 // nontemporal: weights are read once
__device__ __forceinline__ __amdgpu_buffer_rsrc_t stream_rsrc(const void* base, int bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, bytes, kStreamBufFlags);
}
__device__ __forceinline__ void stream_codes(const u32x4* wrow, const float* srow, int N, StreamLane off,
                                             StreamCodes& c) {
  const u32x4 w = __builtin_bit_cast(
      u32x4, __builtin_amdgcn_raw_buffer_load_b128(stream_rsrc(wrow, N * 16), off.w, 0, kStreamNt));
  const f32x4 v = __builtin_bit_cast(
      f32x4, __builtin_amdgcn_raw_buffer_load_b128(stream_rsrc(srow, N * 4), off.s, 0, kStreamNt));
#pragma unroll
  for (int cb = 0; cb < 4; ++cb) {
    c.w[cb] = w[cb];
    c.s[cb] = v[cb];
  }
  // loads stay in the order of their use, and each refill behind its consumer:
  // the compiler's waits then count them instead of draining the ring
  __builtin_amdgcn_sched_barrier(0);
}

// n groups (a multiple of the ring; groups past the end are staged as zeros)
// from LDS group 0 of `frag`; next(codes) loads the ring's next group.
// acc[cb][i] is row (lane >> 4) + 4 i, column 4 (lane & 15) + cb.  Every wave of
// the workgroup runs the same n: a bare barrier a round (no fence, so no wait
// on the ring) keeps the waves in step, which otherwise finish one after
// another, oldest first, with ever fewer loads in flight (down projections of
// four tokens: 59 -> 54.5 us).
template <int kP, int kI, class Next>
__device__ __forceinline__ void stream_run(const uint4* lds, StreamFrag frag, int n, uint32_t magic,
                                           StreamCodes ring[kStreamRing], Next&& next, float acc[4][kI]) {
  for (int g = 0; g < n; g += kStreamRing) {
#pragma unroll
    for (int j = 0; j < kStreamRing; ++j) {
      const half8 af = *reinterpret_cast<const half8*>(lds + frag.at);
      frag.at += frag.step;
#pragma unroll
      for (int cb = 0; cb < 4; ++cb) {
        const half8 bq = codes_f16(ring[j].w[cb], magic);
        const f32x4 d =
            __builtin_amdgcn_mfma_f32_16x16x32_f16(af, bq, f32x4{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < kI; ++i)
          acc[cb][i] = fmaf(ring[j].s[cb], kP == 2 ? d[2 * i] + d[2 * i + 1] : d[i], acc[cb][i]);
      }
      next(ring[j]);
    }
    __builtin_amdgcn_s_barrier();
  }
}

// A wave-uniform value in scalar registers.
__device__ __forceinline__ uint64_t uniform64(uint64_t v) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v));
  const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v >> 32));
  return static_cast<uint64_t>(hi) << 32 | lo;
}
template <class T>
__device__ __forceinline__ const T* uniform_at(const T* base, uint64_t bytes) {
  return reinterpret_cast<const T*>(reinterpret_cast<const char*>(base) + uniform64(bytes));
}

// Eight consecutive activations from element `at`.
template <int kP>
struct StreamX8 {
  uint4 v[kP];
};
template <int kP>
__device__ __forceinline__ StreamX8<kP> stream_load_x(const void* x, size_t at) {
  StreamX8<kP> r;
  const uint4* p = reinterpret_cast<const uint4*>(static_cast<const char*>(x) + at * (kP == 2 ? 4 : 2));
#pragma unroll
  for (int i = 0; i < kP; ++i) r.v[i] = p[i];
  return r;
}
template <int kP>
__device__ __forceinline__ void stream_x_values(const StreamX8<kP>& r, float v[8]) {
  if (kP == 1) {
    const uint32_t w[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < kP; ++i) {
      v[4 * i] = __uint_as_float(r.v[i].x);
      v[4 * i + 1] = __uint_as_float(r.v[i].y);
      v[4 * i + 2] = __uint_as_float(r.v[i].z);
      v[4 * i + 3] = __uint_as_float(r.v[i].w);
    }
  }
}

// Largest magnitude of eight activations and `mx`, as bits.
template <int kP>
__device__ __forceinline__ uint32_t stream_max8(const StreamX8<kP>& x, uint32_t mx) {
  float v[8];
  stream_x_values<kP>(x, v);
#pragma unroll
  for (int i = 0; i < 8; ++i) mx = max(mx, __float_as_uint(v[i]) & 0x7fffffffu);
  return mx;
}

// Eight activations scaled for a row of this largest magnitude, as pieces.
template <int kP, int kXP>
__device__ __forceinline__ void stream_put_row(uint4* lds, int unit, const StreamX8<kXP>& x, uint32_t amax) {
  float v[8];
  stream_x_values<kXP>(x, v);
  const float scale = ldexpf(1.0f, stream_exp(__uint_as_float(amax)));
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] *= scale;
  stream_put<kP>(lds, unit, v);
}

}  // namespace w4
