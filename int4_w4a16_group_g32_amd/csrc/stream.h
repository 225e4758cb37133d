// Streaming W4A16 products of a few rows (device helpers).
//
// One v_mfma_f32_16x16x32_f16 spans one 32-row code block and 16 weight
// columns: B holds the exact codes (codes_f16), A up to 16 rows of f16 pieces.
// A wave owns 64 columns; a lane reads one 16-byte GROUPED slot (word kb of
// four adjacent columns, one per MFMA block) and their four scales per block,
// and the block's result is scaled by s[g][n] on float32 accumulators.
//
// Rows are staged in LDS one window of 32 groups at a time as f16 pieces of
// x * 2^e, with a running power of two per row: e is the smallest that keeps
// every value so far under 2^15, and the accumulators follow it by exact
// powers of two.  Two pieces (8 rows, float32 x): A row m holds piece 0 of
// row m, A row 8 + m piece 1, 22 significant bits in all.  One piece (16 rows,
// bf16 x): exact for bf16 values.
#pragma once

#include "common.h"
#include "mfma_ops.h"

namespace w4 {

constexpr int kStreamWin = 32;    // groups per staged window
constexpr int kStreamRows = 16;   // A rows
constexpr int kStreamCols = 256;  // columns of one quad of four waves
constexpr int kStreamNoExp = 1 << 20;

struct StreamLds {
  uint4 buf[kStreamWin * kStreamRows * 4];  // A fragments, unit (group, row, k block) at stream_unit
  float f[kStreamRows];                     // per row: the accumulators' rescale before this window
  int e[kStreamRows];                       // per row: the running exponent
};

// A fragment read (16 rows of one group and k block) and a staging store (16
// lanes: one row, eight groups, two k blocks) each cover all bank groups.
__device__ __forceinline__ int stream_unit(int g, int r, int kb) {
  return (g * 16 + ((r & ~3) | ((r & 3) ^ (g & 3)))) * 4 + (kb ^ ((r >> 2) & 3) ^ ((g >> 2) & 1));
}

// Stores the 16 values at half `lane & 1` of group `lane >> 1` of one row of a
// window as pieces and moves the row's running exponent; one wave a row.
// `live`: some lane of the row holds a value (wave-uniform); a row without any
// is stored as zeros.
template <int kP>
__device__ __forceinline__ void stream_store(StreamLds& lds, int m, int nw, int lane, bool first, bool live,
                                             const float v[16]) {
  const int gl = lane >> 1, hb = lane & 1;
  const int e_old = first ? kStreamNoExp : lds.e[m];  // (all lanes read before lane 0 writes)
  int e = e_old;
  float scale = 0.0f;
  if (live) {
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(v[i]));
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) amax = fmaxf(amax, __shfl_xor(amax, o));
    if (amax > 0.0f) {
      int lg = ilogbf(amax);
      lg = lg > 120 ? 120 : (lg < -112 ? -112 : lg);  // 2^e stays a normal float
      e = min(e_old, 14 - lg);
    }
    scale = e < kStreamNoExp ? ldexpf(1.0f, e) : 0.0f;
  }
  if (lane == 0) {
    lds.f[m] = e_old < kStreamNoExp ? ldexpf(1.0f, e - e_old) : 1.0f;
    lds.e[m] = e;
  }
  if (gl < nw) {
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      half8 p0 = half8{}, p1 = half8{};
      if (live) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float t = v[8 * b + kCodeOrder[i]] * scale;
          const _Float16 h0 = static_cast<_Float16>(t);
          p0[i] = h0;
          if (kP == 2) p1[i] = static_cast<_Float16>(t - static_cast<float>(h0));
        }
      }
      const int kb = 2 * hb + b;
      *reinterpret_cast<half8*>(&lds.buf[stream_unit(gl, m, kb)]) = p0;
      if (kP == 2) *reinterpret_cast<half8*>(&lds.buf[stream_unit(gl, 8 + m, kb)]) = p1;
    }
  }
}

// A row that no window holds: its accumulators are dropped.
__device__ __forceinline__ void stream_no_row(StreamLds& lds, int m) {
  lds.f[m] = 0.0f;
  lds.e[m] = kStreamNoExp;
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

__device__ __forceinline__ void stream_mma(const StreamLds& lds, int gl, int lc, int kb, bool on, uint32_t magic,
                                           const StreamCodes& c, f32x4 acc[4]) {
  half8 af = *reinterpret_cast<const half8*>(&lds.buf[stream_unit(gl, lc, kb)]);
  if (!on) af = half8{};
#pragma unroll
  for (int cb = 0; cb < 4; ++cb) {
    const half8 bq = codes_f16(c.w[cb], magic);
    const f32x4 d = __builtin_amdgcn_mfma_f32_16x16x32_f16(af, bq, f32x4{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[cb][i] = fmaf(c.s[cb], d[i], acc[cb][i]);
  }
}

// Brings the accumulators to the window's powers of two.
template <int kP>
__device__ __forceinline__ void stream_rescale(const StreamLds& lds, int kb, f32x4 tot[4]) {
  const int r0 = kP == 2 ? 4 * (kb & 1) : 4 * kb;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float f = lds.f[r0 + i];
#pragma unroll
    for (int cb = 0; cb < 4; ++cb) tot[cb][i] *= f;
  }
}

// Back from the running powers of two (rows without a nonzero value give 0),
// pieces joined: element i of block cb is row 4 (kb & 1) + i (two pieces, the
// same in both halves of the wave) or 4 kb + i (one), column 4 lc + cb.
template <int kP>
__device__ __forceinline__ void stream_finish(const StreamLds& lds, int kb, f32x4 tot[4]) {
  const int r0 = kP == 2 ? 4 * (kb & 1) : 4 * kb;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int e = lds.e[r0 + i];
    const float f = e < kStreamNoExp ? ldexpf(1.0f, -e) : 0.0f;
#pragma unroll
    for (int cb = 0; cb < 4; ++cb) {
      tot[cb][i] *= f;
      if (kP == 2) tot[cb][i] += __shfl_xor(tot[cb][i], 32);
    }
  }
}

}  // namespace w4
