// Low-rank adapters beside a shared W4A16 projection:
//
//   y[m] = x[m] W + s_a (x[m] A_a^T) B_a^T,   a = ids[m],
//
// with A_a [R][K] and B_a [N][R] in bf16 and a row without an adapter
// (ids[m] outside [0, n)) taking the first term alone.
//
// What a row costs beside the shared product is the reading of its adapter
// (2 R (K + N) bytes), so the kernels differ by who shares an adapter.  A few
// rows of many requests: every row by itself, float32 dot products on the
// vector units, spread over as many waves as there are (row, rank) or (row,
// column) pairs; the second product runs in the epilogue of the streamed base
// product, or where its split sums are added.  Many rows (prompts): blocks of
// rows on v_mfma_f32_16x16x32_bf16.  There bf16 operands enter as they are,
// and a float32 operand (x, and always t = x A^T) as three bf16 pieces of 8
// significant bits each: bf16 has float32's exponent range, so no scaling is
// needed, and the pieces hold the value's 24 bits.  Rows of different adapters
// share an MFMA block: it is multiplied by every adapter that occurs in it and
// each row keeps the result of its own.  Results are selected, never
// multiplied by zero, so an infinity or NaN in one adapter reaches no row of
// another.
#include "lora.h"

#include <cmath>

#include "dispatch.h"
#include "stream.h"

namespace w4 {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ f32x4 mfma_bf16(uint4 a, uint4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                 0, 0);
}

// The three bf16 pieces of a float32 value.  Each is the top half of what the
// ones before it leave, so together they hold its 24 significant bits exactly
// (a value that is not finite is its own first piece: inf - inf is NaN).
__device__ __forceinline__ void split3(float v, uint16_t p[3]) {
  const uint32_t u = __float_as_uint(v), h0 = u & 0xffff0000u;
  const bool finite = (u & 0x7f800000u) != 0x7f800000u;
  const float r = finite ? v - __uint_as_float(h0) : 0.0f;
  const uint32_t h1 = __float_as_uint(r) & 0xffff0000u;
  p[0] = finite ? static_cast<uint16_t>(h0 >> 16) : f32_to_bf16(v);
  p[1] = static_cast<uint16_t>(h1 >> 16);
  p[2] = static_cast<uint16_t>(__float_as_uint(r - __uint_as_float(h1)) >> 16);
}

__device__ __forceinline__ uint4 pack8(const uint16_t p[8]) {
  return make_uint4(p[0] | (static_cast<uint32_t>(p[1]) << 16), p[2] | (static_cast<uint32_t>(p[3]) << 16),
                    p[4] | (static_cast<uint32_t>(p[5]) << 16), p[6] | (static_cast<uint32_t>(p[7]) << 16));
}

// Eight consecutive activations, as loaded and as kXP bf16 pieces: 1 (bf16) or
// 3 (float32).
template <int kXP>
struct XRaw {
  uint4 v[kXP == 1 ? 1 : 2];
};
template <int kXP>
__device__ __forceinline__ XRaw<kXP> load_x8(const void* x) {
  XRaw<kXP> r;
  const uint4* p = static_cast<const uint4*>(x);
  r.v[0] = p[0];
  if constexpr (kXP == 3) r.v[1] = p[1];
  return r;
}
template <int kXP>
__device__ __forceinline__ void pieces_x8(const XRaw<kXP>& r, uint4 out[kXP]) {
  if constexpr (kXP == 1) {
    out[0] = r.v[0];
  } else {
    const uint32_t v[8] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w, r.v[1].x, r.v[1].y, r.v[1].z, r.v[1].w};
    uint16_t q[3][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint16_t p[3];
      split3(__uint_as_float(v[i]), p);
#pragma unroll
      for (int j = 0; j < 3; ++j) q[j][i] = p[j];
    }
#pragma unroll
    for (int j = 0; j < 3; ++j) out[j] = pack8(q[j]);
  }
}

// The adapter id of a row, -1 for none.
__device__ __forceinline__ int adapter_of(const int* ids, int row, int M, int n) {
  const int id = row < M ? ids[row] : -1;
  return id >= 0 && id < n ? id : -1;
}

__device__ __forceinline__ int rank_of(const LoraSet& s, int id) {
  if (s.ranks == nullptr) return s.R;
  const int r = s.ranks[id];
  return r < 0 ? 0 : (r > s.R ? s.R : r);
}

// ---------------------------------------------------------------- by rows

// The sum over the wave, in every lane.
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

struct ShrinkArgs {
  const void* x;
  const int* ids;
  LoraSet s[2];
  int M, K, splits, chunks;  // chunks: of a workgroup's ranks, over the larger R
  int sets;
  int slots;  // by blocks: workgroups that share the adapters of 64 rows
};

constexpr int kMaxShrinkSplits = 8;
// Runs of rows seldom end more than three times in 64 rows; 2048 rows of 8
// adapters in runs, K 7168, rank 64: 34 us with one slot, 29 with two, 23 with four.
constexpr int kShrinkSlots = 4;
constexpr int kXcds = 8;  // the hardware deals workgroup b to XCD b % 8

// Workgroup b of a grid over (row, part).  The parts go round the XCDs, and all
// rows of a part to one, whose L2 then holds what the rows of an adapter share.
// Above 64 rows a part's rows are cut into segments, so that 32 of them or more
// go round (181 rows of an MLP 1536/640, rank 40: 75 -> 61 us); fewer rows are
// not worth the divisions.
__device__ __host__ inline int xcd_segments(int rows, int parts) {
  return rows <= 64 ? 1 : (32 + parts - 1) / parts;
}
__device__ __forceinline__ bool xcd_place(int b, int rows, int parts, int& row, int& part) {
  const int segs = xcd_segments(rows, parts), per = segs == 1 ? rows : (rows + segs - 1) / segs;
  const int r = b / kXcds, unit = r / per * kXcds + b % kXcds;
  if (segs == 1) {
    part = unit;
    row = r % per;
    return part < parts;
  }
  part = unit / segs;
  row = unit % segs * per + r % per;
  return part < parts && row < rows;
}
inline size_t xcd_blocks(int rows, int parts) {
  if (parts == 0) return 0;
  const int segs = xcd_segments(rows, parts), per = (rows + segs - 1) / segs;
  return (static_cast<size_t>(parts) * segs + kXcds - 1) / kXcds * kXcds * per;
}

// The rows of x as f16 pieces for the base product: scaled by one power of two
// a row (2^-e to rs), in the order codes_f16 expands to.
using PrepArgs = LoraPrep;

template <int kXP, int kP>
__device__ __forceinline__ void prep_row(const ShrinkArgs& a, const PrepArgs& p, int m) {
  // Chunks a thread keeps in registers, by the number of pieces alone.  With ten,
  // float32 rows of up to 20480 are read once (the head of four rows of 18432:
  // 7.4 -> 6.0 us).  Many or short rows would want four: calls of 512 rows of
  // 1024 values (rank 16) 28.8 against 27.2 us, of 7168 values 67.0 against 65.8,
  // 64 rows the same.
  constexpr int kHold = kP == 2 ? 10 : 4;
  __shared__ uint32_t amax;
  const int tid = threadIdx.x, nc = a.K / 8;
  const size_t xrow = static_cast<size_t>(min(m, a.M - 1)) * a.K;
  if (tid == 0) amax = 0;
  StreamX8<kXP> x[kHold];
#pragma unroll
  for (int i = 0; i < kHold; ++i)
    x[i] = stream_load_x<kXP>(a.x, xrow + 8 * static_cast<size_t>(min(tid + i * 256, nc - 1)));
  __syncthreads();
  uint32_t mx = 0;
  if (m < a.M) {
#pragma unroll
    for (int i = 0; i < kHold; ++i) mx = stream_max8<kXP>(x[i], mx);
    for (int c = tid + kHold * 256; c < nc; c += 256)
      mx = stream_max8<kXP>(stream_load_x<kXP>(a.x, xrow + 8 * static_cast<size_t>(c)), mx);
    mx = wave_max(mx);
    if (lane_id() == 0) atomicMax(&amax, mx);
  }
  __syncthreads();
  mx = amax;
  const int e = stream_exp(__uint_as_float(mx));
  if (tid == 0) p.rs[m] = mx != 0 ? ldexpf(1.0f, -e) : 0.0f;
  const float scale = mx != 0 ? ldexpf(1.0f, e) : 0.0f;
  auto put = [&](int c, const StreamX8<kXP>& xc) {
    float v[8];
    stream_x_values<kXP>(xc, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = mx != 0 ? v[i] * scale : 0.0f;
    half8 h[2];
    stream_pieces<kP>(v, h);
    uint4* o = p.out + (c / 4 * p.group + c % 4 * p.chunk + m * p.row);
#pragma unroll
    for (int j = 0; j < kP; ++j) o[j * p.piece] = __builtin_bit_cast(uint4, h[j]);
  };
#pragma unroll
  for (int i = 0; i < kHold; ++i)
    if (tid + i * 256 < nc) put(tid + i * 256, x[i]);
  for (int c = tid + kHold * 256; c < nc; c += 256)
    put(c, stream_load_x<kXP>(a.x, xrow + 8 * static_cast<size_t>(c)));
  for (int c = nc + tid; c < p.chunks; c += 256)
#pragma unroll
    for (int j = 0; j < kP; ++j) p.out[c / 4 * p.group + c % 4 * p.chunk + m * p.row + j * p.piece] = make_uint4(0, 0, 0, 0);
}

// What comes before the base product, in one launch.  The first workgroups
// each prepare a row; the others take one row and kQ ranks of t, their four
// waves quarters of K, all of a step's loads in flight together.  One launch
// instead of two (a launch of either alone takes 4 us); 64 rows of as many
// adapters, K 7168, rank 32: 8 us, 3.7 TB/s of adapters.
template <int kXP, int kP, int kQ>
__global__ __launch_bounds__(256) void head_kernel(const ShrinkArgs a, const PrepArgs p) {
  if (static_cast<int>(blockIdx.x) < p.rows) {
    prep_row<kXP, kP>(a, p, blockIdx.x);
    return;
  }
  __shared__ float red[4][kQ];
  int m, c;
  if (!xcd_place(blockIdx.x - p.rows, a.M, a.chunks * a.sets, m, c)) return;
  const int r0 = c % a.chunks * kQ;
  const LoraSet s = a.s[c / a.chunks];
  const int id = adapter_of(a.ids, m, a.M, s.n);
  if (id < 0 || r0 >= rank_of(s, id)) return;
  const int wv = wave_id(), lane = lane_id();
  const int nc = a.K / 8, per = (nc + 255) / 256 * 64;  // chunks of 8, per wave
  const int c_lo = wv * per, c_hi = min(nc, c_lo + per);
  const size_t xrow = static_cast<size_t>(m) * a.K;
  const uint16_t* ar = s.a + (static_cast<size_t>(id) * s.R + r0) * a.K;
  float acc[kQ];
#pragma unroll
  for (int q = 0; q < kQ; ++q) acc[q] = 0.0f;
  constexpr int kU = 4;
  for (int c0 = c_lo + lane; c0 < c_hi; c0 += 64 * kU) {
    StreamX8<kXP> x[kU];
    uint4 w[kU][kQ];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int c = min(c0 + 64 * u, nc - 1);
      x[u] = stream_load_x<kXP>(a.x, xrow + 8 * static_cast<size_t>(c));
#pragma unroll
      for (int q = 0; q < kQ; ++q)  // (ranks past R read the last one and are not stored)
        w[u][q] = *reinterpret_cast<const uint4*>(ar + static_cast<size_t>(min(q, s.R - 1 - r0)) * a.K +
                                                  8 * static_cast<size_t>(c));
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      if (c0 + 64 * u >= c_hi) break;
      float v[8];
      stream_x_values<kXP>(x[u], v);
#pragma unroll
      for (int q = 0; q < kQ; ++q) {
        const uint32_t d[4] = {w[u][q].x, w[u][q].y, w[u][q].z, w[u][q].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          acc[q] = fmaf(v[2 * i], __uint_as_float(d[i] << 16), acc[q]);
          acc[q] = fmaf(v[2 * i + 1], __uint_as_float(d[i] & 0xffff0000u), acc[q]);
        }
      }
    }
  }
#pragma unroll
  for (int q = 0; q < kQ; ++q) {
    acc[q] = wave_sum(acc[q]);
    if (lane == 0) red[wv][q] = acc[q];
  }
  __syncthreads();
  const int q = threadIdx.x;
  if (q < kQ && r0 + q < s.R)
    s.t[static_cast<size_t>(m) * s.R + r0 + q] = s.scale[id] * ((red[0][q] + red[1][q]) + (red[2][q] + red[3][q]));
}

// 8 ranks r .. r + 7 of one row of B, those at or past `rank` as zero.
__device__ __forceinline__ uint4 load_b8(const uint16_t* row, int r, int rank) {
  if (r >= rank) return make_uint4(0, 0, 0, 0);
  uint4 v = *reinterpret_cast<const uint4*>(row + r);
  const int n = rank - r;
  if (n < 8) {
    uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = 2 * i + 1 < n ? w[i] : (2 * i < n ? w[i] & 0xffffu : 0u);
  }
  return v;
}

// Ranks r0 .. r0 + 31 of kC rows of B, all loads in flight together.
template <int kC>
struct BRows {
  uint4 w[kC][4];
};
template <int kC>
__device__ __forceinline__ void load_rows(const uint16_t* const b[kC], int r0, int rank, BRows<kC>& f) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int i = 0; i < kC; ++i) f.w[i][j] = load_b8(b[i], r0 + 8 * j, rank);
}

// v[i] += t . those ranks of row i, ranks below `rank` in ascending order.  t is
// read up to the next multiple of 8.
template <int kC>
__device__ __forceinline__ void dot_rows(const float* t, int r0, int rank, const BRows<kC>& f, float v[kC]) {
  float4 tv[4][2];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (r0 + 8 * j < rank) {
      tv[j][0] = *reinterpret_cast<const float4*>(t + r0 + 8 * j);
      tv[j][1] = *reinterpret_cast<const float4*>(t + r0 + 8 * j + 4);
    }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int n = rank - r0 - 8 * j;
    if (n <= 0) break;
    float tj[8] = {tv[j][0].x, tv[j][0].y, tv[j][0].z, tv[j][0].w, tv[j][1].x, tv[j][1].y, tv[j][1].z, tv[j][1].w};
#pragma unroll
    for (int e = 0; e < 8; ++e) tj[e] = e < n ? tj[e] : 0.0f;  // (what was never written)
#pragma unroll
    for (int i = 0; i < kC; ++i) {
      const uint32_t d[4] = {f.w[i][j].x, f.w[i][j].y, f.w[i][j].z, f.w[i][j].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[i] = fmaf(tj[2 * e], __uint_as_float(d[e] << 16), v[i]);
        v[i] = fmaf(tj[2 * e + 1], __uint_as_float(d[e] & 0xffff0000u), v[i]);
      }
    }
  }
}

// v[i] += t . row i of b.
template <int kC>
__device__ __forceinline__ void row_dots(const float* t, const uint16_t* const b[kC], int rank, float v[kC], int r0 = 0) {
  for (; r0 < rank; r0 += 32) {
    BRows<kC> f;
    load_rows<kC>(b, r0, rank, f);
    dot_rows<kC>(t, r0, rank, f, v);
  }
}

constexpr int kFinishThreads = 256;
constexpr int kTileWaves = 8, kTileThreads = kTileWaves * kWave;
constexpr int kTileOcc = 4;  // waves a SIMD
constexpr int kLoraUnits = 512;  // LDS units (16 bytes) per wave of the streamed product

// kC columns of base, 64 apart, of the first planes: loads that nothing waits for yet.
constexpr int kBaseAhead = 4;
template <int kC>
struct BaseAhead {
  float q[kC][kBaseAhead];
};
template <int kC>
__device__ __forceinline__ void base_load(const LoraBase& b, int m, int n, int N, BaseAhead<kC>& f) {
  const float* p = b.p + static_cast<size_t>(m) * b.ld;
#pragma unroll
  for (int s = 0; s < kBaseAhead; ++s)
#pragma unroll
    for (int i = 0; i < kC; ++i) f.q[i][s] = s < b.S ? p[s * b.split_stride + min(n + 64 * i, N - 1)] : 0.0f;
}
// rs * the sum of the planes, in split order, 8 more planes' loads in flight together.
template <int kC>
__device__ __forceinline__ void base_sum(const LoraBase& b, int m, int n, int N, const BaseAhead<kC>& f, float v[kC]) {
  constexpr int kB = 8;
  const float* p = b.p + static_cast<size_t>(m) * b.ld;
#pragma unroll
  for (int i = 0; i < kC; ++i) {
    v[i] = f.q[i][0];
#pragma unroll
    for (int s = 1; s < kBaseAhead; ++s) v[i] = s < b.S ? v[i] + f.q[i][s] : v[i];
  }
  for (int s0 = kBaseAhead; s0 < b.S; s0 += kB) {
    float q[kC][kB];
#pragma unroll
    for (int s = 0; s < kB; ++s)
#pragma unroll
      for (int i = 0; i < kC; ++i) q[i][s] = p[min(s0 + s, b.S - 1) * b.split_stride + min(n + 64 * i, N - 1)];
#pragma unroll
    for (int s = 0; s < kB; ++s)
#pragma unroll
      for (int i = 0; i < kC; ++i) v[i] = s0 + s < b.S ? v[i] + q[i][s] : v[i];
  }
  if (b.rs != nullptr) {
    const float r = b.rs[m];
#pragma unroll
    for (int i = 0; i < kC; ++i) v[i] *= r;
  }
}

// Eight adjacent columns.
__device__ __forceinline__ void store8(void* out, int bf16, size_t at, f32x4 v, f32x4 w) {
  if (bf16) {
    uint32_t d[4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      d[i] = f32_to_bf16(v[2 * i]) | static_cast<uint32_t>(f32_to_bf16(v[2 * i + 1])) << 16;
      d[2 + i] = f32_to_bf16(w[2 * i]) | static_cast<uint32_t>(f32_to_bf16(w[2 * i + 1])) << 16;
    }
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + at) = make_uint4(d[0], d[1], d[2], d[3]);
  } else {
    *reinterpret_cast<f32x4*>(static_cast<float*>(out) + at) = v;
    *reinterpret_cast<f32x4*>(static_cast<float*>(out) + at + 4) = w;
  }
}

// One row; a thread takes two columns 64 apart, so that a wave reads adjacent
// rows of B together.  The row's t is the workgroup's.
constexpr int kFinishCols = 2;
// The base's planes and B are asked for before t is waited for: gate and up of
// 64 rows x 18432 columns, three splits, rank 16: 17 us for 52 MB (20.8 us with
// t first).
template <bool kGlu>
__global__ __launch_bounds__(kFinishThreads) void finish_rows_kernel(const LoraFinishArgs a) {
  __shared__ __attribute__((aligned(16))) float t[2][kLoraMaxRank];
  int m, part;
  if (!xcd_place(blockIdx.x, a.M, (a.N + kFinishThreads * kFinishCols - 1) / (kFinishThreads * kFinishCols), m, part))
    return;
  const int n = (part * 4 + wave_id()) * 64 * kFinishCols + lane_id();
  constexpr int kMats = kGlu ? 2 : 1;
  BaseAhead<kFinishCols> ahead[kMats];
#pragma unroll
  for (int w = 0; w < kMats; ++w) base_load<kFinishCols>(w == 0 ? a.base0 : a.base1, m, n, a.N, ahead[w]);
  __builtin_amdgcn_sched_barrier(0);
  int rank[kMats];
  const uint16_t* rows[kMats][kFinishCols];
  BRows<kFinishCols> first[kMats];
#pragma unroll
  for (int w = 0; w < kMats; ++w) {
    const LoraSet& s = w == 0 ? a.s0 : a.s1;
    const int id = s.b != nullptr ? adapter_of(a.ids, m, a.M, s.n) : -1;
    rank[w] = id >= 0 ? rank_of(s, id) : 0;
#pragma unroll
    for (int i = 0; i < kFinishCols; ++i)
      rows[w][i] = s.b + (static_cast<size_t>(max(id, 0)) * a.N + min(n + 64 * i, a.N - 1)) * s.R;
    load_rows<kFinishCols>(rows[w], 0, rank[w], first[w]);
    // (ranks up to the next multiple of 8 are read, and dropped)
    for (int r = threadIdx.x; r < rank[w]; r += kFinishThreads) t[w][r] = s.t[static_cast<size_t>(m) * s.R + r];
  }
  __syncthreads();
  float v[kFinishCols];
#pragma unroll
  for (int w = 0; w < kMats; ++w) {
    float d[kFinishCols], b[kFinishCols];
    base_sum<kFinishCols>(w == 0 ? a.base0 : a.base1, m, n, a.N, ahead[w], b);
#pragma unroll
    for (int i = 0; i < kFinishCols; ++i) d[i] = 0.0f;
    if (rank[w] > 0) {
      dot_rows<kFinishCols>(t[w], 0, rank[w], first[w], d);
      row_dots<kFinishCols>(t[w], rows[w], rank[w], d, 32);
    }
#pragma unroll
    for (int i = 0; i < kFinishCols; ++i) v[i] = w == 0 ? b[i] + d[i] : silu(v[i]) * (b[i] + d[i]);
  }
#pragma unroll
  for (int i = 0; i < kFinishCols; ++i) {
    if (n + 64 * i >= a.N) continue;
    const size_t at = static_cast<size_t>(m) * a.N + n + 64 * i;
    if (a.out_bf16)
      static_cast<uint16_t*>(a.out)[at] = f32_to_bf16(v[i]);
    else
      static_cast<float*>(a.out)[at] = v[i];
  }
}

// ---------------------------------------------------------------- by blocks: x A^T

constexpr int kShrinkThreads = 256;
constexpr int kShrinkWaves = kShrinkThreads / kWave;

// One workgroup: 64 rows, one chunk of 16 kCB ranks, one K split, one
// projection, every slots-th adapter of those rows.  The four waves take
// quarters of the split's K and meet in LDS.  2048 bf16 rows, K 7168, rank 64:
// 23 us for 29 MB of x, bound by the chain of loads (ids, then x and A) of the
// blocks that hold several adapters.
template <int kXP, int kCB>
__global__ __launch_bounds__(kShrinkThreads) void shrink_blocks_kernel(const ShrinkArgs a) {
  constexpr int kRB = 4, kU = kXP == 1 ? 4 : 2;  // k steps in flight
  __shared__ float red[kShrinkWaves][kRB * kLoraRows][kCB * 16];
  int b = blockIdx.x;
  const int split = b % a.splits;
  b /= a.splits;
  const int chunk = b % a.chunks;
  b /= a.chunks;
  // (slots outermost: neighbouring workgroups, which go to different CUs, have
  // work; those of the last slots mostly leave at once)
  const int blocks = (a.M + kRB * kLoraRows - 1) / (kRB * kLoraRows);
  const int block = b % blocks, slot = b / blocks;
  const LoraSet s = a.s[blockIdx.y];
  const int r0 = chunk * 16 * kCB;
  if (s.a == nullptr || r0 >= s.R) return;
  const int m0 = block * kRB * kLoraRows;
  const int wv = wave_id(), lane = lane_id();
  const int lc = lane & 15, kb = lane >> 4;

  // lane l knows the adapter of row m0 + l
  const int mine = adapter_of(a.ids, m0 + lane, a.M, s.n);
  const int steps = a.K / 32;
  const int per = (steps + a.splits * kShrinkWaves - 1) / (a.splits * kShrinkWaves);
  const int k_lo = min(steps, (split * kShrinkWaves + wv) * per), k_hi = min(steps, k_lo + per);
  const char* xr[kRB];
#pragma unroll
  for (int rb = 0; rb < kRB; ++rb)
    xr[rb] = static_cast<const char*>(a.x) +
             (static_cast<size_t>(min(m0 + rb * kLoraRows + lc, a.M - 1)) * a.K + 8 * kb) * (kXP == 1 ? 2 : 4);

  uint64_t todo = __ballot(mine >= 0);
  for (int turn = 0; todo != 0; turn = turn + 1 == a.slots ? 0 : turn + 1) {
    const int id = __builtin_amdgcn_readlane(mine, __builtin_ctzll(todo));
    const uint64_t rows = __ballot(mine == id);
    todo &= ~rows;
    if (turn != slot) continue;
    f32x4 acc[kRB][kCB];
#pragma unroll
    for (int rb = 0; rb < kRB; ++rb)
#pragma unroll
      for (int cb = 0; cb < kCB; ++cb) acc[rb][cb] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    const uint16_t* ar[kCB];
#pragma unroll
    for (int cb = 0; cb < kCB; ++cb)  // ranks past R read the last one and are not stored
      ar[cb] = s.a + (static_cast<size_t>(id) * s.R + min(r0 + 16 * cb + lc, s.R - 1)) * a.K + 8 * kb;
    // kU k steps' loads in flight together; a step past the range repeats its
    // last one with zero operands
    for (int k0 = k_lo; k0 < k_hi; k0 += kU) {
      uint4 af[kU][kCB];
      XRaw<kXP> xw[kU][kRB];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const size_t k = static_cast<size_t>(min(k0 + u, k_hi - 1)) * 32;
#pragma unroll
        for (int cb = 0; cb < kCB; ++cb) af[u][cb] = *reinterpret_cast<const uint4*>(ar[cb] + k);
#pragma unroll
        for (int rb = 0; rb < kRB; ++rb) xw[u][rb] = load_x8<kXP>(xr[rb] + k * (kXP == 1 ? 2 : 4));
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const bool on = k0 + u < k_hi;
        if (!on) {
#pragma unroll
          for (int cb = 0; cb < kCB; ++cb) af[u][cb] = make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int rb = 0; rb < kRB; ++rb) {
          if (((rows >> (rb * kLoraRows)) & 0xffffu) == 0) continue;  // (wave-uniform)
          uint4 xf[kXP];
          pieces_x8<kXP>(xw[u][rb], xf);
#pragma unroll
          for (int p = 0; p < kXP; ++p) {
            if (!on) xf[p] = make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int cb = 0; cb < kCB; ++cb) acc[rb][cb] = mfma_bf16(xf[p], af[u][cb], acc[rb][cb]);
          }
        }
      }
    }
    // element i of lane (lc, kb): row 4kb + i, rank lc
    __syncthreads();  // the previous adapter's sums are stored
#pragma unroll
    for (int rb = 0; rb < kRB; ++rb)
#pragma unroll
      for (int cb = 0; cb < kCB; ++cb)
#pragma unroll
        for (int i = 0; i < 4; ++i) red[wv][rb * kLoraRows + 4 * kb + i][16 * cb + lc] = acc[rb][cb][i];
    __syncthreads();
    float* t = s.t + static_cast<size_t>(split) * a.M * s.R;
    const float scale = s.scale[id];
    for (int e = threadIdx.x; e < kRB * kLoraRows * kCB * 16; e += kShrinkThreads) {
      const int r = e % (kCB * 16), m = e / (kCB * 16);
      if (((rows >> m) & 1) == 0 || r0 + r >= s.R) continue;
      float v = red[0][m][r];
#pragma unroll
      for (int w = 1; w < kShrinkWaves; ++w) v += red[w][m][r];
      t[static_cast<size_t>(m0 + m) * s.R + r0 + r] = v * scale;
    }
  }
}

// ---------------------------------------------------------------- by blocks: t B^T

// t of 16 kRB rows and one chunk of ranks as bf16 pieces in LDS; rows are padded
// so that the 16 rows of one fragment read spread over the banks.
constexpr int kTPad = kLoraChunk + 8;
template <int kRB>
struct TPieces {
  uint16_t p[3][kRB * kLoraRows][kTPad];
};

// Summed splits of the rows from m0 on, ranks r0 .. r0 + 63, as pieces.  Ranks
// the row's adapter does not use, and rows without one, are zero.
template <int kRB>
__device__ __forceinline__ void stage_t(const LoraSet& s, const int* ids, int M, int m0, int r0, int splits, int tid,
                                        int nthreads, TPieces<kRB>& tp) {
  for (int e = tid; e < kRB * kLoraRows * kLoraChunk; e += nthreads) {
    const int m = e / kLoraChunk, r = e % kLoraChunk;
    const int id = adapter_of(ids, m0 + m, M, s.n);
    float v = 0.0f;
    if (id >= 0 && r0 + r < rank_of(s, id)) {
      const float* t = s.t + static_cast<size_t>(m0 + m) * s.R + r0 + r;
      float q[kMaxShrinkSplits];
#pragma unroll
      for (int i = 0; i < kMaxShrinkSplits; ++i)
        if (i < splits) q[i] = t[static_cast<size_t>(i) * M * s.R];
#pragma unroll
      for (int i = 0; i < kMaxShrinkSplits; ++i)
        if (i < splits) v += q[i];
    }
    uint16_t p[3];
    split3(v, p);
#pragma unroll
    for (int j = 0; j < 3; ++j) tp.p[j][m][r] = p[j];
  }
}

// The first column, within a wave's 64, of the four that lane kb = 0 holds of
// block nb.
constexpr __device__ int block_col(int nb) { return 32 * (nb >> 1) + 4 * (nb & 1); }

// One workgroup: 16 kRB rows x 64 columns a wave.  B enters as the MFMA's row
// operand and t as its column operand, with the columns placed so that a lane's
// results of two blocks are eight adjacent columns of one row; the sums start
// from the base's.  An adapter's rows of B are loaded while the one before it
// is used, once for all the rows.  2048 rows x 4096 columns, rank 64: 24 us for
// 54 MB (40 us with 16 rows and 64 columns a workgroup).
template <int kRB, bool kGlu>
__global__ __launch_bounds__(512) void finish_blocks_kernel(const LoraFinishArgs a) {
  constexpr int kNB = 4, kKS = kLoraChunk / 32;
  __shared__ TPieces<kRB> tp;
  const int waves = blockDim.x / kWave;
  const int blocks = (a.M + kRB * kLoraRows - 1) / (kRB * kLoraRows);
  const int m0 = static_cast<int>(blockIdx.x % blocks) * kRB * kLoraRows;
  const int n0 = (static_cast<int>(blockIdx.x / blocks) * waves + wave_id()) * 16 * kNB;
  const int lane = lane_id();
  const int lc = lane & 15, kb = lane >> 4;

  f32x4 sum[kGlu ? 2 : 1][kRB][kNB];
#pragma unroll
  for (int w = 0; w < (kGlu ? 2 : 1); ++w) {
    const LoraBase& base = w == 0 ? a.base0 : a.base1;
    // (rows and columns past the end read the last ones and are not stored)
    const float* p[kRB];
#pragma unroll
    for (int rb = 0; rb < kRB; ++rb)
      p[rb] = base.p + static_cast<size_t>(min(m0 + rb * kLoraRows + lc, a.M - 1)) * base.ld;
    for (int i = 0; i < base.S; ++i)  // one plane after another
#pragma unroll
      for (int rb = 0; rb < kRB; ++rb)
#pragma unroll
        for (int nb = 0; nb < kNB; ++nb) {
          const f32x4 v = *reinterpret_cast<const f32x4*>(p[rb] + i * base.split_stride +
                                                          min(n0 + block_col(nb) + 8 * kb, a.N - 4));
          sum[w][rb][nb] = i == 0 ? v : sum[w][rb][nb] + v;
        }
    if (base.rs != nullptr) {
#pragma unroll
      for (int rb = 0; rb < kRB; ++rb) {
        const float f = base.rs[min(m0 + rb * kLoraRows + lc, a.M - 1)];
#pragma unroll
        for (int nb = 0; nb < kNB; ++nb) sum[w][rb][nb] *= f;
      }
    }
  }
  const int r_max = max(a.s0.b != nullptr ? a.s0.R : 0, kGlu && a.s1.b != nullptr ? a.s1.R : 0);
  for (int r0 = 0; r0 < r_max; r0 += kLoraChunk) {
#pragma unroll
    for (int w = 0; w < (kGlu ? 2 : 1); ++w) {
      const LoraSet& s = w == 0 ? a.s0 : a.s1;
      if (s.b == nullptr || r0 >= s.R) continue;
      // lane l knows the adapter of row m0 + l
      const int mine = lane < kRB * kLoraRows ? adapter_of(a.ids, m0 + lane, a.M, s.n) : -1;
      uint64_t todo = __ballot(mine >= 0);
      if (todo == 0) continue;  // (the same in every wave)
      auto load = [&](int id, uint4 bf[kKS][kNB]) {
        const int rank = rank_of(s, id);
#pragma unroll
        for (int ks = 0; ks < kKS; ++ks)
#pragma unroll
          for (int nb = 0; nb < kNB; ++nb) {
            const int n = n0 + block_col(nb) + 8 * (lc >> 2) + (lc & 3);
            bf[ks][nb] = load_b8(s.b + (static_cast<size_t>(id) * a.N + min(n, a.N - 1)) * s.R,
                                 r0 + 32 * ks + 8 * kb, rank);
          }
      };
      int id = __builtin_amdgcn_readlane(mine, __builtin_ctzll(todo));
      uint4 bf[kKS][kNB];
      load(id, bf);
      __syncthreads();  // the sums before are done with the pieces
      stage_t<kRB>(s, a.ids, a.M, m0, r0, a.splits, threadIdx.x, blockDim.x, tp);
      __syncthreads();
      while (todo != 0) {
        const uint64_t rows = __ballot(mine == id);
        todo &= ~rows;
        const int id_next = todo != 0 ? __builtin_amdgcn_readlane(mine, __builtin_ctzll(todo)) : id;
        uint4 bn[kKS][kNB];
        if (todo != 0) load(id_next, bn);
#pragma unroll
        for (int rb = 0; rb < kRB; ++rb) {
          if (((rows >> (rb * kLoraRows)) & 0xffffu) == 0) continue;  // (wave-uniform)
          f32x4 acc[kNB];
#pragma unroll
          for (int nb = 0; nb < kNB; ++nb) acc[nb] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int ks = 0; ks < kKS; ++ks)
#pragma unroll
            for (int j = 0; j < 3; ++j) {
              const uint4 tf =
                  *reinterpret_cast<const uint4*>(&tp.p[j][rb * kLoraRows + lc][32 * ks + 8 * kb]);
#pragma unroll
              for (int nb = 0; nb < kNB; ++nb) acc[nb] = mfma_bf16(bf[ks][nb], tf, acc[nb]);
            }
          // element i of lane (lc, kb): column block_col(nb) + 8kb + i, row lc
          if ((rows >> (rb * kLoraRows + lc)) & 1) {
#pragma unroll
            for (int nb = 0; nb < kNB; ++nb) sum[w][rb][nb] += acc[nb];
          }
        }
        if (todo != 0) {
#pragma unroll
          for (int ks = 0; ks < kKS; ++ks)
#pragma unroll
            for (int nb = 0; nb < kNB; ++nb) bf[ks][nb] = bn[ks][nb];
        }
        id = id_next;
      }
    }
  }
#pragma unroll
  for (int rb = 0; rb < kRB; ++rb) {
    const int row = m0 + rb * kLoraRows + lc;
    if (row >= a.M) continue;
#pragma unroll
    for (int nb = 0; nb < kNB; nb += 2) {
      const int n = n0 + block_col(nb) + 8 * kb;
      if (n >= a.N) continue;
      f32x4 v[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        v[j] = sum[0][rb][nb + j];
        if (kGlu) {
#pragma unroll
          for (int i = 0; i < 4; ++i) v[j][i] = silu(v[j][i]) * sum[kGlu ? 1 : 0][rb][nb + j][i];
        }
      }
      store8(a.out, a.out_bf16, static_cast<size_t>(row) * a.N + n, v[0], v[1]);
    }
  }
}

template <int kRB, bool kGlu>
w4a16_status_t launch_finish_blocks(const LoraFinishArgs& a, int waves, hipStream_t stream) {
  const int rows = kRB * kLoraRows, cols = waves * 64;
  const size_t blocks = static_cast<size_t>((a.M + rows - 1) / rows) * ((a.N + cols - 1) / cols);
  if (blocks > 0x7fffffffu) return W4A16_ERR_UNSUPPORTED;
  finish_blocks_kernel<kRB, kGlu><<<static_cast<unsigned>(blocks), waves * kWave, 0, stream>>>(a);
  return launch_status();
}

// ---------------------------------------------------------------- a few rows, one launch

// The base product of a few rows, streamed as in stream.h, and the adapters'
// second product in its epilogue.  A workgroup takes `cols` blocks of 64
// columns (of gate and the same of up) and one K split; wave w takes matrix w %
// kMats, one column block and one of the split's K parts (gpp groups each).
// The rows' pieces were prepared by the launch before: staging is a copy.  The
// parts meet in LDS and the splits in memory as in the split-K GEMV
// (agent-scope stores, an arrival counter, the last workgroup sums in split
// order); then a thread takes a row and two columns: their sums, their
// adapter's dot products and, with gate and up, silu(gate) * up.
// Four float32 rows through gate and up of 7168 x 18432: 34 us, 4.9 TB/s of
// weights; the start (rows, ring) and the meeting are about 8 us of it.
template <int kP, int kI, int kMats>
__global__ __launch_bounds__(1024) __attribute__((amdgpu_waves_per_eu(4)))
void lora_stream_kernel(const LoraStreamArgs a) {
  extern __shared__ uint4 lds[];
  __shared__ int last;
  const int split = blockIdx.x % a.splits, tile = blockIdx.x / a.splits;
  const int tid = threadIdx.x, nt = blockDim.x;
  const int wv = wave_id(), lane = lane_id();
  const int cshift = __builtin_ctz(a.cols);
  const int mat = kMats == 2 ? wv & 1 : 0, col = (wv / kMats) & (a.cols - 1), part = (wv / kMats) >> cshift;
  const int G = a.K / kGroup, groups = a.parts * a.gpp, g_wg = split * groups;
  const int block = tile * a.cols + col;
  const bool wave_ok = block * 64 < a.N;
  const int rshift = stream_rshift<kP>(a.M);

  // the window's units of this K range, ahead of the weights; groups past the
  // last are zeros
  const int units = (groups * 4) << rshift, held = min(units, (G - g_wg) * 4 << rshift);
  const uint4* xs = a.xs + ((static_cast<size_t>(g_wg) * 4) << rshift);
  constexpr int kAhead = 4;
  uint4 xa[kAhead];
#pragma unroll
  for (int i = 0; i < kAhead; ++i) xa[i] = xs[min(tid + i * nt, held - 1)];
  __builtin_amdgcn_sched_barrier(0);

  // the ring: a wave past the last column streams column block 0 and stores
  // nothing, a part past the last group the last one (against staged zeros)
  const StreamLane off = stream_lane(wave_ok ? block * 64 : 0, lane);
  const u32x4* qw = mat ? a.qw1 : a.qw0;
  const float* sc = mat ? a.sc1 : a.sc0;
  int g = min(g_wg + part * a.gpp, G - 1);
  const int g_last = max(g, min(g_wg + (part + 1) * a.gpp, G) - 1);
  auto next = [&](StreamCodes& c) {
    stream_codes(uniform_at(qw, static_cast<uint64_t>(g) * a.N * 16),
                 uniform_at(sc, static_cast<uint64_t>(g >> a.gshift) * a.N * 4), a.N, off, c);
    g = min(g + 1, g_last);
  };
  StreamCodes ring[kStreamRing];
#pragma unroll
  for (int j = 0; j < kStreamRing; ++j) next(ring[j]);
  if (tid < kStreamLds0) lds[tid] = make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int i = 0; i < kAhead; ++i) {
    const int u = tid + i * nt;
    if (u < units) lds[kStreamLds0 + u] = u < held ? xa[i] : make_uint4(0, 0, 0, 0);
  }
  for (int u = tid + kAhead * nt; u < units; u += nt)
    lds[kStreamLds0 + u] = u < held ? xs[u] : make_uint4(0, 0, 0, 0);
  __syncthreads();

  float acc[4][kI];
#pragma unroll
  for (int cb = 0; cb < 4; ++cb)
#pragma unroll
    for (int i = 0; i < kI; ++i) acc[cb][i] = 0.0f;
  stream_run<kP, kI>(lds, stream_frag<kP>(lane, a.M, part * a.gpp, rshift), a.gpp, magic_vgpr(), ring, next, acc);

  // The parts' sums, in order: each thread adds some of the tile's [i][mat,
  // col][lane] places over the parts.
  f32x4* red = reinterpret_cast<f32x4*>(lds);
  const int pshift = cshift + kMats - 1;  // log2 of a part's waves
  __syncthreads();                        // the window is free
#pragma unroll
  for (int i = 0; i < kI; ++i)
    red[(wv * kI + i) * kWave + lane] = f32x4{acc[0][i], acc[1][i], acc[2][i], acc[3][i]};
  __syncthreads();
  // the tile's sums [mat][row][64 cols]: in LDS behind the parts', or the split's in memory
  const int ld = 64 << cshift;
  float* sums = reinterpret_cast<float*>(lds + (nt / kWave) * 256);
  float* base = a.partials + static_cast<size_t>(tile) * a.splits * kMats * a.M * ld;
  const size_t ps = static_cast<size_t>(kMats) * a.M * ld;
  for (int q = tid; q < (kI * kWave) << pshift; q += nt) {
    const int l = q & 63, i = (q >> 6) & (kI - 1), w = (q >> 6) / kI;  // lane, row group, wave of a part
    const int m = (l >> 4) + 4 * i;
    if (m >= a.M) continue;
    f32x4 v = red[(w * kI + i) * kWave + l];
#pragma unroll 4
    for (int p = 1; p < a.parts; ++p) v += red[(((p << pshift) + w) * kI + i) * kWave + l];
    v *= a.rs[m];
    const size_t at = (static_cast<size_t>(kMats == 2 ? w & 1 : 0) * a.M + m) * ld + (w / kMats) * 64 + 4 * (l & 15);
    if (a.splits == 1) {
      *reinterpret_cast<f32x4*>(sums + at) = v;
    } else {
      uint64_t* o = reinterpret_cast<uint64_t*>(base + split * ps + at);
#pragma unroll
      for (int j = 0; j < 2; ++j)
        __hip_atomic_store(o + j, static_cast<uint64_t>(__float_as_uint(v[2 * j + 1])) << 32 | __float_as_uint(v[2 * j]),
                           __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
  }
  if (a.splits > 1) {
    __builtin_amdgcn_s_waitcnt(0);  // this wave's stores are complete
    __syncthreads();
    if (tid == 0)
      last = __hip_atomic_fetch_add(&a.counters[tile], 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == a.splits - 1;
    __syncthreads();
    if (!last) return;
    if (tid == 0) __hip_atomic_store(&a.counters[tile], 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  } else {
    __syncthreads();
  }
  const int nshift = 5 + cshift;  // pairs of columns of a row: 2^nshift
  for (int q = tid; q < a.M << nshift; q += nt) {
    const int m = q >> nshift, c = 2 * (q - (m << nshift)), n = tile * ld + c;
    if (n >= a.N) continue;
    float v[kMats][2];
#pragma unroll
    for (int w = 0; w < kMats; ++w) {
      const size_t at = (static_cast<size_t>(w) * a.M + m) * ld + c;
      if (a.splits == 1) {
        v[w][0] = sums[at];
        v[w][1] = sums[at + 1];
      } else {
        constexpr int kB = 8;
        v[w][0] = v[w][1] = 0.0f;
        for (int s0 = 0; s0 < a.splits; s0 += kB) {
          uint64_t p[kB];
#pragma unroll
          for (int j = 0; j < kB; ++j)
            p[j] = __hip_atomic_load(reinterpret_cast<const uint64_t*>(base + min(s0 + j, a.splits - 1) * ps + at),
                                     __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
          for (int j = 0; j < kB; ++j)
            if (s0 + j < a.splits) {
              v[w][0] += __uint_as_float(static_cast<uint32_t>(p[j]));
              v[w][1] += __uint_as_float(static_cast<uint32_t>(p[j] >> 32));
            }
        }
      }
    }
#pragma unroll
    for (int w = 0; w < kMats; ++w) {
      const LoraSet& s = w == 0 ? a.s0 : a.s1;
      const int id = s.b != nullptr ? adapter_of(a.ids, m, a.M, s.n) : -1;
      if (id >= 0) {
        const uint16_t* b = s.b + (static_cast<size_t>(id) * a.N + n) * s.R;
        const uint16_t* rows[2] = {b, b + s.R};
        row_dots<2>(s.t + static_cast<size_t>(m) * s.R, rows, rank_of(s, id), v[w]);
      }
    }
    if (kMats == 2) {
#pragma unroll
      for (int i = 0; i < 2; ++i) v[0][i] = silu(v[0][i]) * v[kMats - 1][i];
    }
    const size_t at = static_cast<size_t>(m) * a.N + n;
    if (a.out_bf16)
      *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + at) =
          f32_to_bf16(v[0][0]) | static_cast<uint32_t>(f32_to_bf16(v[0][1])) << 16;
    else
      *reinterpret_cast<float2*>(static_cast<float*>(a.out) + at) = make_float2(v[0][0], v[0][1]);
  }
}

template <int kP, int kMats>
void launch_stream_mats(const LoraStreamArgs& a, dim3 grid, dim3 threads, size_t lds, hipStream_t stream) {
  if (a.M <= 4)
    lora_stream_kernel<kP, 1, kMats><<<grid, threads, lds, stream>>>(a);
  else if (a.M <= 8 || kP == 2)
    lora_stream_kernel<kP, 2, kMats><<<grid, threads, lds, stream>>>(a);
  else
    lora_stream_kernel<kP, 4 / kP, kMats><<<grid, threads, lds, stream>>>(a);
}

// ---------------------------------------------------------------- up to 64 rows: the base product

// In LDS the four k blocks of row r of 16 trade places by an exclusive or with
// 0, 2, 3, 1 for r / 4 = 0 .. 3: a 16-byte read takes lanes 0-3, 12-15 and 20-27
// (and the like) together, which then lie in different banks.
__device__ __forceinline__ int tile_turn(int r) { return 0x78 >> (r >> 2 << 1) & 3; }

// 17 to 64 rows (9 to 64 in two pieces) of the base product.  A workgroup of 8
// waves takes kCols blocks of 64 columns (gate's, then up's) and one K split;
// its kParts K parts meet in LDS.  A wave takes all the rows, so that codes are
// expanded once: kRT blocks of 16 rows and 64 columns, a lane's 16 kRT sums,
// within 128 registers (two workgroups a CU, four waves a SIMD, which cover
// each other's waits).  The rows are staged in windows, two buffers in turn: a
// step loads, two steps ahead, its group of codes and its share of the next
// window, and writes the share that has arrived, so that nothing waits for the
// last load.
//
// 64 bf16 rows through gate and up of 7168 x 18432: 58 to 68 us in kernel
// traces, from card to card, 2.4 to 2.8 TB/s of weights.  Issue bounds it rather
// than loads: 64 scalings of 16 results, 36 steps of expansion and 16 products a
// wave and group take four fifths of that with no loads at all; vector
// instructions fill 49 % of the SIMDs' cycles, matrix ones 26 %, and waves wait
// to issue for a third of theirs.
template <int kP, int kRT, int kParts>
__global__ __launch_bounds__(kTileThreads) __attribute__((amdgpu_waves_per_eu(kTileOcc)))
void lora_tiles_kernel(const LoraTileArgs a) {
  constexpr int kCols = kTileWaves / kParts, kRows = 16 * kRT;
  constexpr int kGU = 4 * kP * kRows;                   // units of a group: [piece][row][k block]
  constexpr int kW = 8 / (kParts * kP);                 // groups of a part's window
  constexpr int kPU = kW * kGU, kWU = kParts * kPU;     // units of a part's window, of all
  constexpr int kPer = kWU / kTileThreads;              // units a thread stages of a window
  constexpr int kS = (kPer + kW - 1) / kW;              // and of a step
  constexpr int kV = kW > 1 ? 1 : 2;                    // windows a turn of the loop
  constexpr int kCB = kRT * kP >= 3 ? 2 : 4;            // columns a lane expands at once (registers)
  static_assert(kWU % kTileThreads == 0 && kW * kV % 2 == 0, "");
  extern __shared__ uint4 lds[];
  const int split = blockIdx.x % a.splits, tile = blockIdx.x / a.splits;
  const int tid = threadIdx.x, wv = wave_id(), lane = lane_id();
  const int lc = lane & 15, kb = lane >> 4;
  const int col = wv % kCols, part = wv / kCols;
  const int nb = a.N / 64, block = tile * kCols + col;
  const bool wave_ok = block < a.mats * nb;
  const int mat = wave_ok && block >= nb ? 1 : 0;
  const int n0 = wave_ok ? (block - mat * nb) * 64 : 0;  // (a wave past the last column streams the first)
  const int G = a.K / kGroup, groups = kParts * a.gpp, g_wg = split * groups;

  // this thread's units of window 0; the next window's are kPU further
  const int to = tid ^ tile_turn(tid >> 2 & 15);
  // (through a buffer resource: one 32-bit offset a lane, the rest is scalar)
  const __amdgpu_buffer_rsrc_t xw =
      stream_rsrc(uniform_at(a.xs, static_cast<uint64_t>(g_wg) * kGU * 16), groups * kGU * 16);
  constexpr bool kWhole = kPU % kTileThreads == 0;  // the threads' unit i belongs to one part
  int xo[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int u = i * kTileThreads + tid;
    xo[i] = (u / kPU * a.gpp * kGU + u % kPU) * 16;
  }
  auto unit = [&](int v, int i) {  // of window v
    const int at = kWhole ? i * kTileThreads / kPU * a.gpp * kGU + i * kTileThreads % kPU : 0;
    return __builtin_bit_cast(
        u32x4, __builtin_amdgcn_raw_buffer_load_b128(xw, kWhole ? tid * 16 : xo[i], (v * kPU + at) * 16, 0));
  };
  u32x4* window0 = reinterpret_cast<u32x4*>(lds);
#pragma unroll
  for (int i = 0; i < kPer; ++i) window0[i * kTileThreads + to] = unit(0, i);
  const int wins = a.gpp / kW;

  const StreamLane off = stream_lane(n0, lane);
  const u32x4* qw = mat ? a.qw1 : a.qw0;
  const float* sc = mat ? a.sc1 : a.sc0;
  int g = min(g_wg + part * a.gpp, G - 1);
  const int g_last = max(g, min(g_wg + (part + 1) * a.gpp, G) - 1);
  const uint32_t magic = magic_vgpr();
  StreamCodes ring[2];
  u32x4 xr[2][kS];
  // the loads of a step: its share j of window v, and its codes
  auto next = [&](int j, int v, StreamCodes& c, u32x4 (&x)[kS]) {
#pragma unroll
    for (int s = 0; s < kS; ++s)
      if (j * kS + s < kPer) x[s] = unit(min(v, wins - 1), j * kS + s);
    stream_codes(uniform_at(qw, static_cast<uint64_t>(g) * a.N * 16),
                 uniform_at(sc, static_cast<uint64_t>(g >> a.gshift) * a.N * 4), a.N, off, c);
    g = min(g + 1, g_last);
  };
#pragma unroll
  for (int t = 0; t < 2; ++t) next(t % kW, t / kW + 1, ring[t], xr[t]);
  __syncthreads();

  f32x4 acc[kRT][4];
#pragma unroll
  for (int rt = 0; rt < kRT; ++rt)
#pragma unroll
    for (int cb = 0; cb < 4; ++cb) acc[rt][cb] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  const int frag = part * kPU + 4 * lc + (kb ^ tile_turn(lc));
  for (int v0 = 0; v0 < wins; v0 += kV) {
#pragma unroll
    for (int vv = 0; vv < kV; ++vv) {
      const int v = v0 + vv;
      const uint4* cur = lds + (v & 1) * kWU + frag;
      uint4* other = lds + (~v & 1) * kWU + to;
#pragma unroll
      for (int j = 0; j < kW; ++j) {
        const int slot = (vv * kW + j) & 1;
#pragma unroll
        for (int c0 = 0; c0 < 4; c0 += kCB) {
          half8 bq[kCB];
#pragma unroll
          for (int cb = 0; cb < kCB; ++cb) bq[cb] = codes_f16(ring[slot].w[c0 + cb], magic);
#pragma unroll
          for (int rt = 0; rt < kRT; ++rt) {
            f32x4 d[kCB];
#pragma unroll
            for (int p = 0; p < kP; ++p) {
              const half8 af = *reinterpret_cast<const half8*>(cur + (j * kGU + 4 * (p * kRows + rt * 16)));
#pragma unroll
              for (int cb = 0; cb < kCB; ++cb)
                d[cb] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                    af, bq[cb], p == 0 ? f32x4{0.0f, 0.0f, 0.0f, 0.0f} : d[cb], 0, 0, 0);
            }
#pragma unroll
            for (int cb = 0; cb < kCB; ++cb)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                acc[rt][c0 + cb][i] = fmaf(ring[slot].s[c0 + cb], d[cb][i], acc[rt][c0 + cb][i]);
          }
          if (kCB < 4) __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int s = 0; s < kS; ++s)
          if (j * kS + s < kPer) *reinterpret_cast<u32x4*>(other + (j * kS + s) * kTileThreads) = xr[slot][s];
        next((j + 2) % kW, v + (j + 2) / kW + 1, ring[slot], xr[slot]);
      }
      __syncthreads();  // this window is consumed, the next one staged
    }
  }

  // the parts' sums, by halves
  f32x4* red = reinterpret_cast<f32x4*>(lds);
#pragma unroll
  for (int h = kParts / 2; h >= 1; h /= 2) {
    if (part >= h && part < 2 * h) {
#pragma unroll
      for (int q = 0; q < 4 * kRT; ++q) red[((wv - h * kCols) * 4 * kRT + q) * kWave + lane] = acc[q / 4][q % 4];
    }
    __syncthreads();
    if (part < h) {
#pragma unroll
      for (int q = 0; q < 4 * kRT; ++q) acc[q / 4][q % 4] += red[(wv * 4 * kRT + q) * kWave + lane];
    }
    __syncthreads();
  }
  if (part > 0 || !wave_ok) return;
  // element i of lane (lc, kb): row 4 kb + i, column 4 lc + cb
  const int ld = a.mats * a.N;
  float* o = a.planes + static_cast<size_t>(split) * a.M * ld + mat * a.N + n0 + 4 * lc;
#pragma unroll
  for (int rt = 0; rt < kRT; ++rt)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int m = 16 * rt + 4 * kb + i;
      if (m < a.M)
        *reinterpret_cast<f32x4*>(o + static_cast<size_t>(m) * ld) =
            f32x4{acc[rt][0][i], acc[rt][1][i], acc[rt][2][i], acc[rt][3][i]};
    }
}

template <int kP, int kRT>
void launch_tiles_parts(const LoraTileArgs& a, const LoraTilePlan& p, hipStream_t stream) {
  const unsigned grid = static_cast<unsigned>(p.tiles * p.splits);
  const size_t lds = static_cast<size_t>(2 * kTileThreads) * kRT * 16;
  if constexpr (4 * kP * 16 * kRT <= 384) {
    if (p.parts == 4) {
      lora_tiles_kernel<kP, kRT, 4><<<grid, kTileThreads, lds, stream>>>(a);
      return;
    }
  }
  lora_tiles_kernel<kP, kRT, 2><<<grid, kTileThreads, lds, stream>>>(a);
}
template <int kP>
void launch_tiles_rows(const LoraTileArgs& a, const LoraTilePlan& p, hipStream_t stream) {
  if (a.M <= 16)
    launch_tiles_parts<kP, 1>(a, p, stream);
  else if (a.M <= 32)
    launch_tiles_parts<kP, 2>(a, p, stream);
  else if (a.M <= 48)
    launch_tiles_parts<kP, 3>(a, p, stream);
  else
    launch_tiles_parts<kP, 4>(a, p, stream);
}

// Ranks a workgroup of the row kernel takes: one, until there are workgroups
// enough that sharing the reads of x is worth more.
int shrink_quota(size_t dots) { return dots >= 2048 ? 4 : (dots >= 1024 ? 2 : 1); }

// 16-rank column blocks of one workgroup's chunk.
int shrink_cols(int R) { return R <= 16 ? 1 : (R <= 32 ? 2 : 4); }

template <int kXP>
void launch_shrink_blocks(const ShrinkArgs& a, int cb, dim3 grid, hipStream_t stream) {
  if (cb == 1)
    shrink_blocks_kernel<kXP, 1><<<grid, kShrinkThreads, 0, stream>>>(a);
  else if (cb == 2)
    shrink_blocks_kernel<kXP, 2><<<grid, kShrinkThreads, 0, stream>>>(a);
  else
    shrink_blocks_kernel<kXP, 4><<<grid, kShrinkThreads, 0, stream>>>(a);
}

template <int kXP, int kP>
void launch_head_q(const ShrinkArgs& a, const PrepArgs& p, int q, unsigned blocks, hipStream_t stream) {
  if (q == 4)
    head_kernel<kXP, kP, 4><<<blocks, 256, 0, stream>>>(a, p);
  else if (q == 2)
    head_kernel<kXP, kP, 2><<<blocks, 256, 0, stream>>>(a, p);
  else
    head_kernel<kXP, kP, 1><<<blocks, 256, 0, stream>>>(a, p);
}

}  // namespace

ShrinkShape shrink_shape(int M, int K, int R) {
  ShrinkShape sh;
  // Rows by themselves read an adapter again for every row, blocks of rows once
  // for all the rows of an adapter but do the work of 16 for one.  Adapters of
  // 7168 x 4096, bf16, rows / blocks: 64 rows of 64 adapters of rank 64 41 / 151
  // us, 128 of 64 62 / 160, 256 of 64 107 / 185, 1024 of 64 (rank 16) 138 / 250;
  // runs of rows that share one of four, 128 (rank 32) 44 / 53, 256 (rank 64)
  // 100 / 81, 1024 (rank 16) 137 / 119, 2000 (8 of rank 8) 220 / 169.  Which of
  // the two the ids are the host does not know; many rows are taken for runs.
  sh.rows = M <= 64 || (M <= 512 && static_cast<size_t>(M) * R <= 16384);
  if (sh.rows) return sh;
  const int blocks = (M + 63) / 64, chunks = (R + 16 * shrink_cols(R) - 1) / (16 * shrink_cols(R));
  // about one workgroup per CU, a wave keeping a k step (four: 601 rows, K 896,
  // rank 64, float32 88 us for 57)
  sh.splits = std::max(1, std::min({kMaxShrinkSplits, 256 / (blocks * chunks), K / 32 / kShrinkWaves}));
  return sh;
}

// The sets that are there, and the largest of their ranks.
static int live_sets(const LoraSet* sets, int n_sets, ShrinkArgs& a, int& R) {
  int n = 0;
  R = 0;
  for (int i = 0; i < n_sets; ++i)
    if (sets[i].a != nullptr) {
      a.s[n++] = sets[i];
      R = std::max(R, sets[i].R);
    }
  return n;
}

w4a16_status_t launch_lora_head(const void* x, w4a16_dtype_t xt, int M, int K, const int* ids, const LoraSet* sets,
                                int n_sets, const ShrinkShape& sh, const LoraPrep& prep, hipStream_t stream) {
  ShrinkArgs a{};
  a.x = x;
  a.ids = ids;
  a.M = M;
  a.K = K;
  a.splits = sh.splits;
  int R;
  const int n = live_sets(sets, n_sets, a, R);
  if (M == 0) return W4A16_OK;
  if (sh.rows) {
    const PrepArgs& p = prep;
    const int q = shrink_quota(static_cast<size_t>(M) * R * n);
    a.chunks = std::max(1, (R + q - 1) / q);
    a.sets = n;
    const size_t blocks = static_cast<size_t>(p.rows) + xcd_blocks(M, n * a.chunks);
    if (blocks > 0x7fffffffu) return W4A16_ERR_UNSUPPORTED;
    const unsigned g = static_cast<unsigned>(blocks);
    if (g == 0) return W4A16_OK;
    if (xt == W4A16_BF16)
      launch_head_q<1, 1>(a, p, q, g, stream);
    else if (p.pieces == 2)
      launch_head_q<2, 2>(a, p, q, g, stream);
    else
      launch_head_q<2, 1>(a, p, q, g, stream);  // h of a bf16 layer
    return launch_status();
  }
  if (prep.rows > 0) {
    const w4a16_status_t st = launch_mfma_prep(x, xt, M, prep.rows, K, prep.pieces, nullptr, 0, nullptr, prep.tiles,
                                               prep.rs, stream);
    if (st != W4A16_OK) return st;
  }
  if (n == 0) return W4A16_OK;
  const int cb = shrink_cols(R);
  a.chunks = (R + 16 * cb - 1) / (16 * cb);
  a.slots = kShrinkSlots;
  const size_t blocks = (static_cast<size_t>(M) + 63) / 64 * a.chunks * a.splits * a.slots;
  if (blocks > 0x7fffffffu) return W4A16_ERR_UNSUPPORTED;
  const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>(n));
  if (xt == W4A16_BF16)
    launch_shrink_blocks<1>(a, cb, grid, stream);
  else
    launch_shrink_blocks<3>(a, cb, grid, stream);
  return launch_status();
}

w4a16_status_t launch_lora_finish(const LoraFinishArgs& a, hipStream_t stream) {
  if (a.M == 0 || a.N == 0) return W4A16_OK;
  const bool glu = a.base1.p != nullptr;
  if (a.rows) {
    const int cols = kFinishThreads * kFinishCols;
    const size_t blocks = xcd_blocks(a.M, (a.N + cols - 1) / cols);
    if (blocks > 0x7fffffffu) return W4A16_ERR_UNSUPPORTED;
    const dim3 grid(static_cast<unsigned>(blocks));
    if (glu)
      finish_rows_kernel<true><<<grid, kFinishThreads, 0, stream>>>(a);
    else
      finish_rows_kernel<false><<<grid, kFinishThreads, 0, stream>>>(a);
    return launch_status();
  }
  // tall blocks, which read B and t for more rows and columns at once, where
  // they still fill the chip: calls of 2048 x 4096 (K 1024, 8 adapters of rank
  // 64 in runs) 69 us for 80 without, 1000 x 4096 in random order 90 for 102,
  // 1500 x 2048 (rank 32, runs) 74 for 66
  const bool tall = static_cast<size_t>(a.M) * a.N >= (size_t{15} << 18);
  if (glu) return tall ? launch_finish_blocks<2, true>(a, 8, stream) : launch_finish_blocks<1, true>(a, 4, stream);
  return tall ? launch_finish_blocks<4, false>(a, 8, stream) : launch_finish_blocks<1, false>(a, 4, stream);
}

// Picks K parts and splits by an estimate of the launch's time, fitted to a
// sweep of all of them over twelve shapes (12 to 64 rows, 1024 x 8192 to 7168 x
// 36864): for the workgroups of a CU, their group steps (expanding the codes,
// each block's scalings and products, staging the rows); a further workgroup on
// a CU; the planes' way to memory and back.  It finds the best of the sweep
// within 4 %.  64 bf16 rows through 7168 x 4096 take 24.4 us with 4 parts and 7
// splits (27 us with 2 parts and 7, 28 us with 4 and 4), through 18432 x 7168
// 43.8 us with 2 and 9 (48 us with 4 and 4), head and finish included.
LoraTilePlan plan_lora_tiles(int M, int pieces, int N, int mats, int K) {
  LoraTilePlan best;
  const int G = K / kGroup, blocks = mats * (N / 64), rt = (M + 15) / 16, rows = 16 * rt;
  double best_us = 1e30;
  for (int parts = 2; parts <= 4; parts *= 2) {
    const int cols = kTileWaves / parts, tiles = (blocks + cols - 1) / cols;
    if (parts * pieces * rows > 384) continue;  // (the staged shares no longer fit the registers)
    const int step = std::max(2, 8 / (parts * pieces));
    for (int splits = 1; splits <= kMaxSplits; ++splits) {
      const int gpp = (G + splits * parts * step - 1) / (splits * parts * step) * step;
      if (splits > 1 && (splits - 1) * parts * gpp >= G) continue;  // an empty split
      const size_t groups = static_cast<size_t>(parts) * gpp * splits;
      if (groups / splits * 4 * pieces * rows * 16 >= (size_t{1} << 31)) continue;  // (32-bit offsets)
      const double per_cu = std::ceil(tiles * splits / 256.0);
      const double us = per_cu * gpp * (0.2 + rt * (0.041 + pieces * (0.0126 + 0.0107 * parts))) +
                        0.94 * (per_cu - 1) + 0.084 * splits + static_cast<double>(splits) * M * mats * N * 8 / 10.5e6;
      if (us < best_us) {
        best_us = us;
        best.ok = true;
        best.parts = parts;
        best.splits = splits;
        best.gpp = gpp;
        best.tiles = tiles;
        best.groups = groups;
        best.plane_bytes = static_cast<size_t>(splits) * M * mats * N * 4;
      }
    }
  }
  return best;
}

w4a16_status_t launch_lora_tiles(LoraTileArgs a, const LoraTilePlan& p, hipStream_t stream) {
  a.splits = p.splits;
  a.gpp = p.gpp;
  if (static_cast<size_t>(p.tiles) * p.splits > 0x7fffffffu) return W4A16_ERR_UNSUPPORTED;
  if (a.pieces == 2)
    launch_tiles_rows<2>(a, p, stream);
  else
    launch_tiles_rows<1>(a, p, stream);
  return launch_status();
}

// Picks waves, column blocks, K parts and splits by an estimate of the launch's
// time, fitted to a sweep of all of them over eight shapes (1 to 16 rows, 256 x
// 512 to 18432 x 7168): the weights of the fullest CU at 6 TB/s among the CUs
// at work, at most 33 GB/s each, and at least 0.35 us a group of a wave; a
// start that grows with the workgroup; the splits' meeting.  It finds about
// one workgroup of 8 waves per CU, within 5 % of the best of the sweep: four
// float32 rows through 18432 x 7168 take 19.3 us (4.3 TB/s; 21.4 us with 16
// waves, 23 us with 4), sixteen bf16 rows through 7168 x 4096 11.3 us (14.2 us
// with half the CUs).
LoraStreamPlan plan_lora_stream(int M, int pieces, int N, int mats, int K) {
  LoraStreamPlan best;
  const int G = K / kGroup, blocks = N / 64;
  int rshift = pieces - 1;
  while ((1 << (rshift - pieces + 1)) < M) ++rshift;
  double best_us = 1e30;
  for (int waves = 4; waves <= 16; waves *= 2)
    for (int cols = 1; cols * mats <= waves; cols *= 2) {
      const int parts = waves / (cols * mats), tiles = (blocks + cols - 1) / cols;
      for (int splits = 1; splits <= kMaxSplits; ++splits) {
        const int gpp = (G + splits * parts * kStreamRing - 1) / (splits * parts * kStreamRing) * kStreamRing;
        if (splits > 1 && (splits - 1) * parts * gpp >= G) break;  // an empty split
        if (((parts * gpp * 4) << rshift) > waves * kLoraUnits) continue;  // the window
        if (splits > 1 && tiles * sizeof(int) > kCounterBytes) continue;
        const double wgs = static_cast<double>(tiles) * splits, cus = std::min(wgs, 256.0);
        const double per_cu = std::ceil(wgs / 256.0);
        const double rate = std::min(6.0e6 / cus, 33e3);  // bytes per us of a CU
        const double us = std::max(per_cu * waves * gpp * 1280.0 / rate, gpp * 0.35) + 4.0 + 0.1 * waves +
                          0.3 * (per_cu - 1.0) + (splits > 1 ? 1.0 + 0.15 * splits : 0.0);
        if (us < best_us) {
          best_us = us;
          best.ok = true;
          best.waves = waves;
          best.cols = cols;
          best.parts = parts;
          best.splits = splits;
          best.gpp = gpp;
          best.tiles = tiles;
        }
      }
    }
  if (best.splits > 1)
    best.partial_bytes = static_cast<size_t>(best.tiles) * best.splits * mats * M * best.cols * 64 * 4;
  return best;
}

w4a16_status_t launch_lora_stream(LoraStreamArgs a, const LoraStreamPlan& p, hipStream_t stream) {
  a.cols = p.cols;
  a.parts = p.parts;
  a.splits = p.splits;
  a.gpp = p.gpp;
  const size_t blocks = static_cast<size_t>(p.tiles) * p.splits;
  if (blocks > 0x7fffffffu) return W4A16_ERR_UNSUPPORTED;
  const dim3 grid(static_cast<unsigned>(blocks)), threads(p.waves * kWave);
  const size_t lds = (static_cast<size_t>(p.waves) * kLoraUnits + kStreamLds0) * 16;
  const bool glu = a.qw1 != nullptr;
  if (a.pieces == 2 && glu)
    launch_stream_mats<2, 2>(a, grid, threads, lds, stream);
  else if (a.pieces == 2)
    launch_stream_mats<2, 1>(a, grid, threads, lds, stream);
  else if (glu)
    launch_stream_mats<1, 2>(a, grid, threads, lds, stream);
  else
    launch_stream_mats<1, 1>(a, grid, threads, lds, stream);
  return launch_status();
}

namespace {

// The kernels' 32-bit row bytes.
bool sizes_fit(const w4a16_weight_t* w) { return w->K < 1 << 26 && w->N < 1 << 26; }

w4a16_status_t check_lora(const w4a16_lora_t* l) {
  if (l == nullptr) return W4A16_OK;  // no adapters on this projection
  if (l->a == nullptr || l->b == nullptr || l->scale == nullptr) return W4A16_ERR_INVALID_ARG;
  if (!aligned16(l->a) || !aligned16(l->b) || !aligned16(l->scale) || !aligned16(l->ranks))
    return W4A16_ERR_INVALID_ARG;
  if (l->num_adapters < 1 || l->rank < 1) return W4A16_ERR_INVALID_ARG;
  if (l->rank % 8 != 0 || l->rank > kLoraMaxRank) return W4A16_ERR_UNSUPPORTED;
  return W4A16_OK;
}

bool known_type(w4a16_dtype_t t) { return t == W4A16_F32 || t == W4A16_BF16; }

size_t t_bytes(const w4a16_lora_t* l, int M, const ShrinkShape& sh) {
  return l == nullptr ? 0 : static_cast<size_t>(sh.splits) * M * l->rank * 4;
}

// One projection (or gate and up together) with its adapters' second product:
// a few rows in one streamed launch, more on the tiles with the product where
// the tiles' split sums, or their output, are finished.
struct LinearPlan {
  // up to 16 rows; up to 64; else the 64-row tiles, gate and up in a launch each where those do not split K
  bool stream = false, rows64 = false, pair = false;
  int pieces = 1, rshift = 0;
  LoraStreamPlan st;
  LoraTilePlan tl;
  MfmaPlan mf;
  size_t ap_off = 0, rs_off = 0, partials_off = 0, partials1_off = 0, base0_off = 0, base1_off = 0;
  size_t bytes = 0;  // from the workspace's start, counters included
};

// lt: the layer's activation type; x_f32: this product's x is float32 (h).
LinearPlan plan_linear(int M, w4a16_dtype_t lt, bool x_f32, const w4a16_weight_t* w0, const w4a16_weight_t* w1) {
  LinearPlan p;
  const int K = w0->K, N = w0->N;
  Carve c;
  size_t counters;
  c.take(counters, kCounterBytes);
  // (h of a bf16 layer keeps two pieces up to 8 rows)
  p.pieces = x_f32 && M <= kMaxGemvRows ? 2 : mfma_pieces(lt);
  if (M <= gemv_rows(lt)) {
    p.st = plan_lora_stream(M, p.pieces, N, w1 != nullptr ? 2 : 1, K);
    p.stream = p.st.ok;  // (else K is too long for the windows of 32 splits)
  }
  if (p.stream) {
    p.rshift = p.pieces - 1;
    while ((1 << (p.rshift - p.pieces + 1)) < M) ++p.rshift;
    c.take(p.partials_off, p.st.partial_bytes);
    c.take(p.ap_off, (static_cast<size_t>(K / 8) << p.rshift) * 16);
    c.take(p.rs_off, static_cast<size_t>(M) * 4);
    p.bytes = c.cursor;
    return p;
  }
  if (M <= 64) {
    p.tl = plan_lora_tiles(M, p.pieces, N, w1 != nullptr ? 2 : 1, K);
    p.rows64 = p.tl.ok;
  }
  if (p.rows64) {
    c.take(p.partials_off, p.tl.plane_bytes);
    c.take(p.ap_off, p.tl.groups * 4 * p.pieces * ((M + 15) / 16 * 16) * 16);
    c.take(p.rs_off, static_cast<size_t>(M) * 4);
    p.bytes = c.cursor;
    return p;
  }
  p.pieces = mfma_pieces(lt);
  p.mf = plan_mfma(M, N, w1 != nullptr ? 1 : 0, K, lt, w1 == nullptr);
  if (w1 != nullptr && p.mf.S == 1) {
    p.pair = true;
    p.mf = plan_mfma(M, N, 0, K, lt, true);
  }
  c.take(p.ap_off, static_cast<size_t>(p.mf.P) * p.mf.Mp * K * 2 + (p.mf.wide ? 256 : 0));
  c.take(p.rs_off, static_cast<size_t>(p.mf.Mp) * 4);
  const bool summed = p.mf.S == 1 || p.mf.wide;  // the tiles' result is whole, else planes
  c.take(p.partials_off, mfma_partial_bytes(p.mf));
  p.partials1_off = p.partials_off;  // (wide tiles are done with theirs)
  if (p.pair && !summed) c.take(p.partials1_off, mfma_partial_bytes(p.mf));
  if (summed) c.take(p.base0_off, static_cast<size_t>(M) * N * 4);
  if (p.pair && summed) c.take(p.base1_off, static_cast<size_t>(M) * N * 4);
  p.bytes = c.cursor;
  return p;
}

// What the launch before a projection prepares for it.
LoraPrep linear_prep(const LinearPlan& p, int M, int K, char* ws) {
  LoraPrep r{};
  r.pieces = p.pieces;
  r.rs = reinterpret_cast<float*>(ws + p.rs_off);
  r.out = reinterpret_cast<uint4*>(ws + p.ap_off);
  const size_t rows = (M + 15) / 16 * 16;
  if (p.stream) {  // [group][k block][row][piece], the rows of a power of two
    r.rows = M;
    r.chunks = K / 8;
    r.chunk = size_t{1} << p.rshift;
    r.group = 4 * r.chunk;
    r.row = p.pieces;
    r.piece = 1;
  } else if (p.rows64) {  // [group][piece][row][k block]
    r.rows = M;
    r.chunks = static_cast<int>(p.tl.groups * 4);
    r.chunk = 1;
    r.group = p.pieces * rows * 4;
    r.row = 4;
    r.piece = rows * 4;
  } else {  // [piece][row][group][k block]
    r.rows = p.mf.Mp;
    r.chunks = K / 8;
    r.chunk = 1;
    r.group = 4;
    r.row = K / 8;
    r.piece = static_cast<size_t>(p.mf.Mp) * (K / 8);
    r.tiles = reinterpret_cast<_Float16*>(ws + p.ap_off);
  }
  return r;
}

w4a16_status_t lora_linear(const LinearPlan& p, int M, const w4a16_weight_t* w0, const w4a16_weight_t* w1,
                           const LoraSet& s0, const LoraSet& s1, const int* ids, const ShrinkShape& sh, void* out,
                           w4a16_dtype_t ot, char* ws, hipStream_t stream) {
  const int K = w0->K, N = w0->N;
  if (p.stream) {
    LoraStreamArgs a{};
    a.xs = reinterpret_cast<const uint4*>(ws + p.ap_off);
    a.rs = reinterpret_cast<const float*>(ws + p.rs_off);
    a.pieces = p.pieces;
    a.M = M;
    a.K = K;
    a.N = N;
    a.qw0 = reinterpret_cast<const u32x4*>(w0->qw);
    a.sc0 = w0->scales;
    if (w1 != nullptr) {
      a.qw1 = reinterpret_cast<const u32x4*>(w1->qw);
      a.sc1 = w1->scales;
    }
    a.gshift = group_shift(w0);
    a.s0 = s0;
    a.s1 = s1;
    a.ids = ids;
    a.partials = reinterpret_cast<float*>(ws + p.partials_off);
    a.counters = reinterpret_cast<int*>(ws);
    a.out = out;
    a.out_bf16 = ot == W4A16_BF16;
    return launch_lora_stream(a, p.st, stream);
  }
  LoraFinishArgs f{};
  f.s0 = s0;
  f.s1 = s1;
  f.ids = ids;
  f.rows = sh.rows;
  f.splits = sh.splits;
  f.M = M;
  f.N = N;
  f.out = out;
  f.out_bf16 = ot == W4A16_BF16;
  w4a16_status_t st;
  float* rs = reinterpret_cast<float*>(ws + p.rs_off);
  if (p.rows64) {
    LoraTileArgs a{};
    a.xs = reinterpret_cast<const uint4*>(ws + p.ap_off);
    a.pieces = p.pieces;
    a.M = M;
    a.K = K;
    a.N = N;
    a.mats = w1 != nullptr ? 2 : 1;
    a.qw0 = reinterpret_cast<const u32x4*>(w0->qw);
    a.sc0 = w0->scales;
    if (w1 != nullptr) {
      a.qw1 = reinterpret_cast<const u32x4*>(w1->qw);
      a.sc1 = w1->scales;
    }
    a.gshift = group_shift(w0);
    a.planes = reinterpret_cast<float*>(ws + p.partials_off);
    if ((st = launch_lora_tiles(a, p.tl, stream)) != W4A16_OK) return st;
    f.base0 = LoraBase{a.planes, p.tl.splits, M, a.mats * N, static_cast<size_t>(M) * a.mats * N, rs};
    if (w1 != nullptr) {
      f.base1 = f.base0;
      f.base1.p += N;
    }
    return launch_lora_finish(f, stream);
  }
  // gate and up in one launch (split sums, which the finish joins), or one projection
  auto tiles = [&](const w4a16_weight_t* a0, const w4a16_weight_t* a1, size_t partials, size_t out, LoraBase& base) {
    MfmaArgs a = mfma_dense_args(p.mf, M, a0, a1, a1 != nullptr ? 1 : 0, reinterpret_cast<_Float16*>(ws + p.ap_off), rs,
                                 ws, partials, 0);
    if (p.mf.wide || p.mf.S == 1) {
      a.out = reinterpret_cast<float*>(ws + out);
      base = LoraBase{a.out, 1, M, N, 0, nullptr};
      return p.mf.wide ? launch_wide(a, p.mf.tasks * p.mf.S, stream) : launch_mfma(a, p.mf.P, p.mf.tasks, stream);
    }
    defer_split_k(a, p.mf);
    const size_t plane = static_cast<size_t>(a.plane_rows) * a.plane_ld;
    base = LoraBase{a.planes, a.S, a.plane_rows, a.plane_ld, plane * (a1 != nullptr ? 2 : 1), rs};
    return launch_mfma(a, p.mf.P, p.mf.tasks * p.mf.S, stream);
  };
  st = tiles(w0, p.pair ? nullptr : w1, p.partials_off, p.base0_off, f.base0);
  if (st == W4A16_OK && p.pair) {
    st = tiles(w1, nullptr, p.partials1_off, p.base1_off, f.base1);
  } else if (w1 != nullptr) {
    f.base1 = f.base0;
    f.base1.p += static_cast<size_t>(f.base0.plane_rows) * f.base0.ld;
  }
  if (st != W4A16_OK) return st;
  return launch_lora_finish(f, stream);
}

struct LoraGemmPlan {
  ShrinkShape sh;
  LinearPlan lin;
  size_t t_off = 0, bytes = 0;
};

LoraGemmPlan plan_lora_gemm(int M, const w4a16_weight_t* w, w4a16_dtype_t xt, const w4a16_lora_t* l) {
  LoraGemmPlan p;
  p.sh = shrink_shape(M, w->K, l->rank);
  p.lin = plan_linear(M, xt, xt == W4A16_F32, w, nullptr);
  Carve c;
  size_t start;
  c.take(start, p.lin.bytes);
  c.take(p.t_off, t_bytes(l, M, p.sh));
  p.bytes = c.cursor;
  return p;
}

struct LoraMlpPlan {
  ShrinkShape sh_gu, sh_d;
  LinearPlan gu, dn;
  size_t tg_off = 0, tu_off = 0, td_off = 0, h_off = 0, bytes = 0;
};

LoraMlpPlan plan_lora_mlp(int M, w4a16_dtype_t xt, const w4a16_weight_t* gate, const w4a16_weight_t* up,
                          const w4a16_weight_t* down, const w4a16_lora_t* lg, const w4a16_lora_t* lu,
                          const w4a16_lora_t* ld) {
  LoraMlpPlan p;
  const int H = gate->K, I = gate->N;
  p.sh_gu = shrink_shape(M, H, std::max(lg ? lg->rank : 1, lu ? lu->rank : 1));
  p.sh_d = shrink_shape(M, I, ld ? ld->rank : 1);
  p.gu = plan_linear(M, xt, xt == W4A16_F32, gate, up);
  p.dn = plan_linear(M, xt, true, down, nullptr);
  Carve c;
  size_t start;
  c.take(start, std::max(p.gu.bytes, p.dn.bytes));
  c.take(p.tg_off, t_bytes(lg, M, p.sh_gu));
  c.take(p.tu_off, t_bytes(lu, M, p.sh_gu));
  c.take(p.td_off, t_bytes(ld, M, p.sh_d));
  c.take(p.h_off, static_cast<size_t>(M) * I * 4);
  p.bytes = c.cursor;
  return p;
}

}  // namespace
}  // namespace w4

using namespace w4;

extern "C" size_t w4a16_gemm_lora_workspace_bytes(int32_t M, const w4a16_weight_t* w, w4a16_dtype_t xt,
                                                  const w4a16_lora_t* lora) {
  if (M <= 0 || check_dense_grouped(w) != W4A16_OK || !sizes_fit(w) || !known_type(xt)) return 0;
  if (lora == nullptr || check_lora(lora) != W4A16_OK) return 0;
  return plan_lora_gemm(M, w, xt, lora).bytes;
}

extern "C" w4a16_status_t w4a16_gemm_lora(const void* x, w4a16_dtype_t xt, int32_t M, const w4a16_weight_t* w,
                                          const w4a16_lora_t* lora, const int32_t* adapter_ids, void* y,
                                          w4a16_dtype_t yt, void* ws, size_t ws_bytes, hipStream_t stream) {
  w4a16_status_t st = check_dense_grouped(w);
  if (st != W4A16_OK) return st;
  if (!sizes_fit(w)) return W4A16_ERR_UNSUPPORTED;
  if (lora == nullptr) return W4A16_ERR_INVALID_ARG;
  if ((st = check_lora(lora)) != W4A16_OK) return st;
  if (M < 0 || !known_type(xt) || !known_type(yt)) return W4A16_ERR_INVALID_ARG;
  if (M == 0 || w->K == 0 || w->N == 0) return W4A16_OK;
  if (x == nullptr || y == nullptr || ws == nullptr || adapter_ids == nullptr) return W4A16_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(y) || !aligned16(ws) || !aligned16(adapter_ids)) return W4A16_ERR_INVALID_ARG;
  if (ranges_overlap(x, static_cast<size_t>(M) * w->K * dtype_bytes(xt), y,
                     static_cast<size_t>(M) * w->N * dtype_bytes(yt)))
    return W4A16_ERR_INVALID_ARG;
  const LoraGemmPlan p = plan_lora_gemm(M, w, xt, lora);
  if (ws_bytes < p.bytes) return W4A16_ERR_WORKSPACE;
  char* b = static_cast<char*>(ws);
  const LoraSet set = lora_set(lora, reinterpret_cast<float*>(b + p.t_off));
  st = launch_lora_head(x, xt, M, w->K, adapter_ids, &set, 1, p.sh, linear_prep(p.lin, M, w->K, b), stream);
  if (st != W4A16_OK) return st;
  return lora_linear(p.lin, M, w, nullptr, set, LoraSet{}, adapter_ids, p.sh, y, yt, b, stream);
}

extern "C" size_t w4a16_swiglu_mlp_lora_workspace_bytes(int32_t M, w4a16_dtype_t xt, const w4a16_weight_t* gate,
                                                        const w4a16_weight_t* up, const w4a16_weight_t* down,
                                                        const w4a16_lora_t* lora_gate, const w4a16_lora_t* lora_up,
                                                        const w4a16_lora_t* lora_down) {
  if (M <= 0 || check_mlp(gate, up, down) != W4A16_OK || !sizes_fit(gate) || !known_type(xt)) return 0;
  for (const w4a16_lora_t* l : {lora_gate, lora_up, lora_down})
    if (check_lora(l) != W4A16_OK) return 0;
  return plan_lora_mlp(M, xt, gate, up, down, lora_gate, lora_up, lora_down).bytes;
}

extern "C" w4a16_status_t w4a16_swiglu_mlp_lora(const void* x, w4a16_dtype_t xt, int32_t M,
                                                const w4a16_weight_t* gate, const w4a16_weight_t* up,
                                                const w4a16_weight_t* down, const w4a16_lora_t* lora_gate,
                                                const w4a16_lora_t* lora_up, const w4a16_lora_t* lora_down,
                                                const int32_t* adapter_ids, void* y, w4a16_dtype_t yt, void* ws,
                                                size_t ws_bytes, hipStream_t stream) {
  w4a16_status_t st = check_mlp(gate, up, down);
  if (st != W4A16_OK) return st;
  if (!sizes_fit(gate)) return W4A16_ERR_UNSUPPORTED;
  for (const w4a16_lora_t* l : {lora_gate, lora_up, lora_down})
    if ((st = check_lora(l)) != W4A16_OK) return st;
  if (M < 0 || !known_type(xt) || !known_type(yt)) return W4A16_ERR_INVALID_ARG;
  if (M == 0 || gate->K == 0 || gate->N == 0) return W4A16_OK;
  if (x == nullptr || y == nullptr || ws == nullptr || adapter_ids == nullptr) return W4A16_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(y) || !aligned16(ws) || !aligned16(adapter_ids)) return W4A16_ERR_INVALID_ARG;
  const int H = gate->K, I = gate->N;
  if (ranges_overlap(x, static_cast<size_t>(M) * H * dtype_bytes(xt), y,
                     static_cast<size_t>(M) * H * dtype_bytes(yt)))
    return W4A16_ERR_INVALID_ARG;
  const LoraMlpPlan p = plan_lora_mlp(M, xt, gate, up, down, lora_gate, lora_up, lora_down);
  if (ws_bytes < p.bytes) return W4A16_ERR_WORKSPACE;
  char* b = static_cast<char*>(ws);
  float* h = reinterpret_cast<float*>(b + p.h_off);
  const LoraSet gu[2] = {lora_set(lora_gate, reinterpret_cast<float*>(b + p.tg_off)),
                         lora_set(lora_up, reinterpret_cast<float*>(b + p.tu_off))};
  const LoraSet d = lora_set(lora_down, reinterpret_cast<float*>(b + p.td_off));
  st = launch_lora_head(x, xt, M, H, adapter_ids, gu, 2, p.sh_gu, linear_prep(p.gu, M, H, b), stream);
  if (st != W4A16_OK) return st;
  st = lora_linear(p.gu, M, gate, up, gu[0], gu[1], adapter_ids, p.sh_gu, h, W4A16_F32, b, stream);
  if (st != W4A16_OK) return st;
  st = launch_lora_head(h, W4A16_F32, M, I, adapter_ids, &d, 1, p.sh_d, linear_prep(p.dn, M, I, b), stream);
  if (st != W4A16_OK) return st;
  return lora_linear(p.dn, M, down, nullptr, d, LoraSet{}, adapter_ids, p.sh_d, y, yt, b, stream);
}
