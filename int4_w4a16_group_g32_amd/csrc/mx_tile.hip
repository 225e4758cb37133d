// Products of more than 16 rows with MXFP4 weights: tiles of rows in LDS.
//
// y[m][n] = sum_k x[m][k] e2m1(W[n][k]) 2^(s[n][k / 32] - 127), operands as in
// mx_stream.hip: the weights are the matrix cores' first operand, the rows of x
// the second, and a lane ends with four adjacent columns of one row.
//
// A workgroup has eight waves, kWM along the rows, kWN along the columns and kWK
// along K, a wave kMB x kNB blocks of 16 x 16: tiles of 128 rows by 256 columns
// (of gate and up 128 each), fewer rows where there are no more, then with two
// waves along K instead of along the rows; MXFP4 rows also 128 by 512, which
// halves the rows' way through L2 and LDS.  The rows of a stage of K (128 k of
// bf16, 256 with two waves along K, 512 of MXFP4) are staged in LDS, double-
// buffered, one barrier a stage; each wave streams its own columns' codes into
// registers two steps ahead and, for 16-bit rows, expands them there, a quarter
// of a step ahead of their products.  float32 rows come as bf16 planes (pieces
// whose sum they are), staged one after another against the same codes.
//
// LDS rows are 16-byte chunks, chunk c of row r at c ^ (r mod chunks), which
// serves a fragment read of MXFP4 rows in the least time; bf16 reads, four chunks
// apart, are served twice.  An order without that took the same time.
//
// Bound: 2048 bf16 rows, 7168 -> 4096, 90 us (1.34 PFLOP/s, matrix cores 54 %
// busy with one workgroup a compute unit: the rest is the expansion, the LDS reads
// and a stage's barrier); MXFP4 rows the same product 37 us (3.3 PFLOP/s, 29 %),
// where a stage's chain of code loads, staging and LDS reads, at two waves a SIMD,
// is longer than its 64 products a wave; 1024 MXFP4 rows through the 7168 / 18432
// MLP 246 us (3.3 PFLOP/s; the instruction alone issues at 8).  64 bf16 rows through
// it 93 us, 2.3 TB/s of weights: each workgroup's start, the sums' planes
// (12 us) and the expansion.  The tiles of 64 float32 rows spill a few registers
// (gate and up 7, a product alone 3).
#include "mx.h"

#include <cmath>

namespace w4 {
namespace {

constexpr int kThreads = 512;
constexpr int kOob = 0x7fffffff;  // an offset past every buffer: the load gives 0
constexpr int kXcds = 8;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* base, size_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, static_cast<int>(bytes), 0x00020000);
}
__device__ __forceinline__ u32x4 load16(__amdgpu_buffer_rsrc_t r, int off, int soff) {
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off, soff, 0));
}
__device__ __forceinline__ i32x8 widen(const u32x4& v) {
  return i32x8{static_cast<int>(v[0]), static_cast<int>(v[1]), static_cast<int>(v[2]), static_cast<int>(v[3]),
               0, 0, 0, 0};
}

// The compiler moves no vector memory access across this.
__device__ __forceinline__ void keep_loads() { __builtin_amdgcn_sched_barrier(0x38f); }

// acc += W x, both MXFP4; kA and kB: the scales' bytes.
template <int kA, int kB>
__device__ __forceinline__ f32x4 mma_fp4(const u32x4& w, const u32x4& x, const f32x4& acc, uint32_t ws, uint32_t xs) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(widen(w), widen(x), acc, 4, 4, kA, static_cast<int>(ws), kB,
                                                          static_cast<int>(xs));
}
template <int kA>
__device__ __forceinline__ f32x4 mma_fp4_b(int b, const u32x4& w, const u32x4& x, const f32x4& acc, uint32_t ws,
                                           uint32_t xs) {
  switch (b) {
    case 0: return mma_fp4<kA, 0>(w, x, acc, ws, xs);
    case 1: return mma_fp4<kA, 1>(w, x, acc, ws, xs);
    case 2: return mma_fp4<kA, 2>(w, x, acc, ws, xs);
    default: return mma_fp4<kA, 3>(w, x, acc, ws, xs);
  }
}
__device__ __forceinline__ f32x4 mma_fp4_ab(int a, int b, const u32x4& w, const u32x4& x, const f32x4& acc, uint32_t ws,
                                            uint32_t xs) {
  switch (a) {  // (both are constants once the loops are unrolled)
    case 0: return mma_fp4_b<0>(b, w, x, acc, ws, xs);
    case 1: return mma_fp4_b<1>(b, w, x, acc, ws, xs);
    case 2: return mma_fp4_b<2>(b, w, x, acc, ws, xs);
    default: return mma_fp4_b<3>(b, w, x, acc, ws, xs);
  }
}

__device__ __forceinline__ float scale_byte(int c, uint32_t d) {
  return __uint_as_float(((d >> (8 * c)) & 0xffu) << 23);
}

// kP: bf16 planes of x (1 .. 3), or 0 for MXFP4 rows.
template <int kP, int kWM, int kWN, int kWK, int kMB, int kNB, bool kGlu>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(2))) void mx_tile_kernel(const MxTileArgs a) {
  static_assert(kWM * kWN * kWK * 64 == kThreads, "eight waves");
  constexpr bool kFp4 = kP == 0;
  static_assert(!kFp4 || kWK == 1, "MXFP4 rows: no waves along K");
  constexpr int kPlanes = kFp4 ? 1 : kP;
  constexpr int kMats = kGlu ? 2 : 1;
  constexpr int kNbM = kNB / kMats;                       // blocks of each matrix
  constexpr int kBM = 16 * kMB * kWM, kCols = 16 * kNbM;  // rows of the tile; columns of a wave
  constexpr int kBN = kCols * kWN;
  constexpr int kSteps = kFp4 ? 4 : kWK;                  // steps of 128 k in a stage
  constexpr int kChunks = (kFp4 ? 4 : 16) * kSteps;       // 16-byte chunks of a row and stage
  constexpr int kUnits = (kBM * kChunks + kThreads - 1) / kThreads;  // chunks staged by a thread
  constexpr int kParts = kFp4 ? kSteps : 4;                    // of a stage's compute, between which they are staged
  constexpr int kQuads = (kBM + 63) / 64;                 // groups of four 16-row blocks
  struct Buffer {
    u32x4 x[kBM * kChunks];
    uint32_t s[kFp4 ? kSteps * kQuads * 64 : 1];  // per step: scales of four 16-row blocks
  };
  __shared__ Buffer lds[2];

  // XCD x = b mod 8 takes a contiguous run of workgroups
  const int T = static_cast<int>(gridDim.x), b = static_cast<int>(blockIdx.x);
  const int xcd = b % kXcds, tq = T / kXcds, trem = T % kXcds;
  const int task = xcd * tq + min(xcd, trem) + b / kXcds;
  const int t = static_cast<int>(threadIdx.x), wv = wave_id(), lane = lane_id();
  const int lr = lane & 15, kb = lane >> 4;
  const int wk = wv / (kWM * kWN), wm = wv / kWN % kWM, wn = wv % kWN;
  const int tiles64 = (a.N + kMxTileRows - 1) / kMxTileRows;
  const size_t cb = static_cast<size_t>(a.S) * kMxTileCodes, sb = static_cast<size_t>(a.S) * kMxTileScales;

  struct Codes {
    u32x4 w[kMats][kNbM];
    uint32_t s[kMats];
  };
  __amdgpu_buffer_rsrc_t wr[kMats], sr[kMats];
  int r0, nrows, n0, c0, s_lo, s_hi;  // the segment's rows, the wave's columns, K steps
  auto load_codes = [&](Codes& c, int s) {
    s = min(s, a.S - 1);  // (past the end: read again, not used)
#pragma unroll
    for (int m = 0; m < kMats; ++m) {
#pragma unroll
      for (int i = 0; i < kNbM; ++i) c.w[m][i] = load16(wr[m], lane * 16 + (c0 + i) * 1024, s * kMxTileCodes);
      c.s[m] = __builtin_amdgcn_raw_buffer_load_b32(sr[m], lane * 4, s * kMxTileScales, 0);
    }
  };

  // staging: rows past the last one and k past K read as zeros
  const size_t xrow = kFp4 ? a.K / 2 : static_cast<size_t>(a.K) * 2;
  const size_t plane = static_cast<size_t>(a.M) * xrow;
  const char* xbase;
  const int G = a.K / kMxBlock;
  __amdgpu_buffer_rsrc_t xr, xsr;
  const int chunk = t % kChunks, srow = t / kChunks;
  constexpr int kRowsAt = kThreads / kChunks;  // rows staged by one unit of all threads
  struct Held {
    u32x4 x[kUnits];
    uint32_t s[4];  // (MXFP4: scales of one step of rows 16 apart)
  };
  // a thread's chunk of its unit i, from step s
  auto stage_load = [&](Held& h, int i, int s, int p) {
    const int row = srow + i * kRowsAt;
    const int k16 = s * (kFp4 ? 4 : 16) + chunk;  // 16-byte unit of the row
    const bool on = row < nrows && k16 * 16 < static_cast<int>(xrow) && s + (kFp4 ? 0 : chunk / 16) < s_hi;
    h.x[i] = load16(kPlanes == 1 ? xr : rsrc(xbase + p * plane, nrows * xrow),
                    on ? row * static_cast<int>(xrow) + k16 * 16 : kOob, 0);
  };
  auto stage_store = [&](Buffer& buf, const Held& h, int i) {
    const int row = srow + i * kRowsAt;
    if (kUnits * kThreads == kBM * kChunks || row < kBM) buf.x[row * kChunks + (chunk ^ (row % kChunks))] = h.x[i];
  };
  // Scales: thread t < 16 kSteps kQuads takes one step (t / (16 kQuads)) of the rows
  // 64 g + t % 16 + 16 q, q = 0 .. 3, four bytes each, and leaves dword l of
  // group g with what lane l needs: its k block's byte of each of the four.
  const int sg = t / 16 % kQuads, ss = t / (16 * kQuads);
  const bool stages_scales = kFp4 && t < 16 * kSteps * kQuads;
  auto scale_load = [&](Held& h, int s) {
    if (!stages_scales) return;
    const int g = 4 * (s + ss);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int row = 64 * sg + t % 16 + 16 * q, at = row * G + g;
      const bool on = row < nrows;
      if (G % 4 == 0) {
        h.s[q] = __builtin_amdgcn_raw_buffer_load_b32(xsr, on && g < G ? at : kOob, 0, 0);
      } else {
        h.s[q] = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          h.s[q] |= static_cast<uint32_t>(static_cast<uint8_t>(
                        __builtin_amdgcn_raw_buffer_load_b8(xsr, on && g + e < G ? at + e : kOob, 0, 0)))
                    << (8 * e);
      }
    }
  };
  auto scale_store = [&](Buffer& buf, const Held& h) {
    if (!stages_scales) return;
    const uint32_t a01 = __builtin_amdgcn_perm(h.s[1], h.s[0], 0x05010400);
    const uint32_t b01 = __builtin_amdgcn_perm(h.s[1], h.s[0], 0x07030602);
    const uint32_t a23 = __builtin_amdgcn_perm(h.s[3], h.s[2], 0x05010400);
    const uint32_t b23 = __builtin_amdgcn_perm(h.s[3], h.s[2], 0x07030602);
    uint32_t* o = buf.s + (ss * kQuads + sg) * 64 + t % 16;
    o[0] = __builtin_amdgcn_perm(a23, a01, 0x05040100);
    o[16] = __builtin_amdgcn_perm(a23, a01, 0x07060302);
    o[32] = __builtin_amdgcn_perm(b23, b01, 0x05040100);
    o[48] = __builtin_amdgcn_perm(b23, b01, 0x07060302);
  };

  f32x4 acc[kMB][kNB];
  // unit i is staged in part i * kParts / kUnits of the compute
  auto part_of = [](int i) { return i * kParts / kUnits; };
  auto load_part = [&](Held& h, int part, int s, int p) {
#pragma unroll
    for (int i = 0; i < kUnits; ++i)
      if (part_of(i) == part) stage_load(h, i, s, p);
    if constexpr (kFp4) {
      if (part == 0) scale_load(h, s);
    }
  };
  auto store_part = [&](Buffer& buf, const Held& h, int part) {
#pragma unroll
    for (int i = 0; i < kUnits; ++i)
      if (part_of(i) == part) stage_store(buf, h, i);
    if constexpr (kFp4) {
      if (part == 0) scale_store(buf, h);
    }
  };
  auto xfrag = [&](const Buffer& buf, int i, int c) {
    const int row = wm * 16 * kMB + 16 * i + lr;
    return buf.x[row * kChunks + (c ^ (row % kChunks))];
  };

  Codes ring[2];
  // Units of K (stages of all tiles in a row, a.per of them) are dealt out in
  // runs of a.quota to workgroups; a run may cross tiles.
  int unit = task * a.quota;
  const int unit_end = min(unit + a.quota, a.per * a.tiles * a.row_tiles);
  for (bool again = false; unit < unit_end; again = true) {
  // Tiles go through bands of `band` row tiles column by column, so the
  // workgroups of an XCD share a block of row and column tiles whose rows and
  // codes its L2 reads once (launch_mx_tile picks the band).
  const int u = unit / a.per, at = unit - u * a.per, run = min(a.per - at, unit_end - unit);
  const int band0 = u / (a.band * a.tiles) * a.band, in_band = min(a.band, a.row_tiles - band0);
  const int tile = (u - band0 * a.tiles) / in_band;
  r0 = (band0 + (u - band0 * a.tiles) % in_band) * kBM;
  nrows = min(kBM, a.M - r0);
  s_lo = at * a.unit_steps;
  s_hi = min(a.S, (at + run) * a.unit_steps);
  const bool whole = run == a.per;
  const int slot = task - u * a.per / a.quota;  // among the workgroups of this tile
  unit += run;
  n0 = (a.tile0 + tile) * kBN + wn * kCols;
  c0 = n0 / 16 % 4;
  {
    // (a wave past the last column streams tile 0 and stores nothing)
    const size_t J = n0 / kMxTileRows < tiles64 ? n0 / kMxTileRows : 0;
#pragma unroll
    for (int m = 0; m < kMats; ++m) {
      wr[m] = rsrc(a.wc[m] + J * cb, cb);
      sr[m] = rsrc(a.ws[m] + J * sb, sb);
    }
  }
  xbase = static_cast<const char*>(a.x) + r0 * xrow;
  xr = rsrc(xbase, nrows * xrow);
  if constexpr (kFp4) xsr = rsrc(a.xs + static_cast<size_t>(r0) * G, static_cast<size_t>(nrows) * G);
#pragma unroll
  for (int i = 0; i < kMB; ++i)
#pragma unroll
    for (int j = 0; j < kNB; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  if (again) __syncthreads();  // (the last segment's LDS is read)

  // Loads are issued in the order of their use, here as in the loops (the
  // barriers keep the compiler from moving them): its waits, which have to hold
  // for the first stage as for the others, then leave all later ones in flight.
  Held held, first;
#pragma unroll
  for (int part = 0; part < kParts; ++part) load_part(first, part, s_lo, 0);
  __builtin_amdgcn_sched_barrier(0);
  if constexpr (kFp4) {
#pragma unroll
    for (int h = 0; h < kSteps; ++h) {
      load_part(held, h, s_lo + kSteps, 0);
      __builtin_amdgcn_sched_barrier(0);
      if (h >= kSteps - 2) load_codes(ring[h & 1], s_lo + h - (kSteps - 2));
      __builtin_amdgcn_sched_barrier(0);
    }
  } else {
    load_codes(ring[0], s_lo + wk);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int part = 0; part < kParts; ++part) load_part(held, part, s_lo + 1 / kPlanes * kWK, 1 % kPlanes);
    __builtin_amdgcn_sched_barrier(0);
    load_codes(ring[1], s_lo + kWK + wk);
    __builtin_amdgcn_sched_barrier(0);
  }
#pragma unroll
  for (int part = 0; part < kParts; ++part) store_part(lds[0], first, part);

  if constexpr (kFp4) {
    for (int s = s_lo, q = 0; s < s_hi; s += kSteps, ++q) {
      __syncthreads();
      const Buffer& cur = lds[q & 1];
      Buffer& nxt = lds[(q + 1) & 1];
#pragma unroll
      for (int h = 0; h < kSteps; ++h) {
        store_part(nxt, held, h);
        load_part(held, h, s + 2 * kSteps, 0);
        __builtin_amdgcn_sched_barrier(0);
        Codes& c = ring[h & 1];
        if (s + h < s_hi) {
          uint32_t ws[kMats];
#pragma unroll
          for (int m = 0; m < kMats; ++m) ws[m] = kNbM == 4 ? c.s[m] : c.s[m] >> (8 * c0);
#pragma unroll
          for (int i = 0; i < kMB; ++i) {
            const int rb = wm * kMB + i;  // 16-row block: byte rb % 4 of its dword
            uint32_t xs = cur.s[(h * kQuads + rb / 4) * 64 + lane];
            if (kMB % 4 != 0) xs >>= 8 * (rb % 4 - i % 4);
            const u32x4 xf = xfrag(cur, i, 4 * h + kb);
#pragma unroll
            for (int m = 0; m < kMats; ++m)
#pragma unroll
              for (int j = 0; j < kNbM; ++j)
                acc[i][m * kNbM + j] = mma_fp4_ab(j, i % 4, c.w[m][j], xf, acc[i][m * kNbM + j], ws[m], xs);
          }
        }
        load_codes(c, s + h + 2);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  } else {
    int q = 0;
    // Part j takes codes 8 j .. 8 j + 7 of every lane.  While its products run,
    // the codes of the next part, or of the next stage's first, are expanded and
    // its rows read: w and xf hold one part more than is in use.
    bf16x8 w[2][kNB], xf[2][kMB];
    auto expand = [&](const Codes& c, int part, bf16x8 o[kNB]) {
#pragma unroll
      for (int m = 0; m < kMats; ++m)
#pragma unroll
        for (int j = 0; j < kNbM; ++j)
          o[m * kNbM + j] = mx_bf16(c.w[m][j][part], scale_byte(j, kNbM == 4 ? c.s[m] : c.s[m] >> (8 * c0)));
    };
    // c: this stage's codes, cn: the next one's; (s_next, p_next): two stages on
    auto stage = [&](const Codes& c, const Codes& cn, int s_next, int p_next) {
      __syncthreads();
      const Buffer& cur = lds[q & 1];
      Buffer& nxt = lds[(q + 1) & 1];
      ++q;
      auto frags = [&](int part) {
#pragma unroll
        for (int i = 0; i < kMB; ++i)
          xf[part & 1][i] = __builtin_bit_cast(bf16x8, xfrag(cur, i, 16 * wk + 4 * kb + part));
      };
      frags(0);
#pragma unroll
      for (int part = 0; part < 4; ++part) {
        store_part(nxt, held, part);
        load_part(held, part, s_next, p_next);
        keep_loads();
        if (part < 3) frags(part + 1);
        expand(part < 3 ? c : cn, (part + 1) & 3, w[(part + 1) & 1]);
#pragma unroll
        for (int i = 0; i < kMB; ++i)
#pragma unroll
          for (int j = 0; j < kNB; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[part & 1][j], xf[part & 1][i], acc[i][j], 0, 0, 0);
      }
    };
    expand(ring[0], 0, w[0]);
    for (int s = s_lo; s < s_hi; s += 2 * kWK) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int sh = s + h * kWK;
        if (sh >= s_hi) break;
#pragma unroll 1
        for (int p = 0; p < kPlanes; ++p)
          stage(ring[h], p + 1 < kPlanes ? ring[h] : ring[1 - h],
                p + 2 < kPlanes ? sh : sh + (p + 2) / kPlanes * kWK, (p + 2) % kPlanes);
        load_codes(ring[h], sh + 2 * kWK + wk);
        keep_loads();
      }
    }
  }

  // the waves along K meet in LDS, in their order
  if constexpr (kWK > 1) {
    static_assert(sizeof(lds) >= kWM * kWN * kMB * kNB * 64 * sizeof(f32x4), "room for a wave group's sums");
    f32x4(*red)[kMB][kNB][64] = reinterpret_cast<f32x4(*)[kMB][kNB][64]>(&lds[0]);
    const int wg = wv % (kWM * kWN);
    for (int k = 1; k < kWK; ++k) {
      __syncthreads();
      if (wk == k) {
#pragma unroll
        for (int i = 0; i < kMB; ++i)
#pragma unroll
          for (int j = 0; j < kNB; ++j) red[wg][i][j][lane] = acc[i][j];
      }
      __syncthreads();
      if (wk == 0) {
#pragma unroll
        for (int i = 0; i < kMB; ++i)
#pragma unroll
          for (int j = 0; j < kNB; ++j) acc[i][j] += red[wg][i][j][lane];
      }
    }
    if (wk != 0) continue;
  }

  // lane: row 16 i + lr of the wave, columns 4 kb .. + 3 of block j
#pragma unroll
  for (int i = 0; i < kMB; ++i) {
    const int row = r0 + wm * 16 * kMB + 16 * i + lr;
    const bool row_ok = row < a.M;
    const size_t rowN = static_cast<size_t>(row) * a.N;
    if (!whole) {
#pragma unroll
      for (int m = 0; m < kMats; ++m)
#pragma unroll
        for (int j = 0; j < kNbM; ++j) {
          const int n = n0 + 16 * j + 4 * kb;
          if (row_ok && n < a.N)
            *reinterpret_cast<f32x4*>(a.planes + (static_cast<size_t>(slot) * kMats + m) * a.M * a.N + rowN + n) =
                acc[i][m * kNbM + j];
        }
    } else if constexpr (!kGlu) {
#pragma unroll
      for (int j = 0; j < kNB; ++j) {
        const int n = n0 + 16 * j + 4 * kb;
        if (row_ok && n < a.N) mx_store4(a.y, rowN + n, a.y_bf16, acc[i][j]);
      }
    } else {
      f32x4 h[kNbM];
#pragma unroll
      for (int j = 0; j < kNbM; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) h[j][e] = silu(acc[i][j][e]) * acc[i][kNbM + j][e];
      if constexpr (kFp4) {
        static_assert(!kFp4 || kNbM % 2 == 0, "blocks of 32 columns");
#pragma unroll
        for (int j = 0; j < kNbM; j += 2) mx_store_h(a.y, a.ys, row, a.N, n0 + 16 * j, kb, row_ok, h[j], h[j + 1]);
      } else {
#pragma unroll
        for (int j = 0; j < kNbM; ++j) {
          const int n = n0 + 16 * j + 4 * kb;
          if (row_ok && n < a.N) mx_store_hidden(a.y, rowN + n, static_cast<size_t>(a.M) * a.N, a.h_pieces, h[j]);
        }
      }
    }
  }
  }
}

// ---------------------------------------------------------------- shared tiles and planes

// The sums of tiles that several workgroups share, in their order along K, to y
// or to h and its form for the down product.
template <bool kGlu, bool kFp4>  // kFp4: h as MXFP4
__global__ __launch_bounds__(256) void mx_planes_kernel(const MxTileArgs a) {
  const size_t mn = static_cast<size_t>(a.M) * a.N;
  const size_t i = blockIdx.x * static_cast<size_t>(256) + threadIdx.x;  // four columns of a row
  if (i * 4 >= mn) return;
  // (shared tiles are one band)
  const int u = static_cast<int>(4 * i % a.N) / a.cols * a.row_tiles + static_cast<int>(4 * i / a.N) / a.bm;
  const int n = ((u + 1) * a.per - 1) / a.quota - u * a.per / a.quota + 1;  // workgroups of this tile
  if (n == 1) return;  // (stored whole)
  f32x4 v[2];
  constexpr int kM = kGlu ? 2 : 1;
  const f32x4* p = reinterpret_cast<const f32x4*>(a.planes) + i;
#pragma unroll
  for (int m = 0; m < kM; ++m) v[m] = p[m * (mn / 4)];
  for (int s = 1; s < n; ++s)
#pragma unroll
    for (int m = 0; m < kM; ++m) v[m] += p[(static_cast<size_t>(s) * kM + m) * (mn / 4)];
  if constexpr (!kGlu) {
    mx_store4(a.y, 4 * i, a.y_bf16, v[0]);
  } else {
    f32x4 h;
#pragma unroll
    for (int e = 0; e < 4; ++e) h[e] = silu(v[0][e]) * v[1][e];
    if constexpr (kFp4) {
      // eight threads hold a block of 32 columns
      uint32_t mx = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) mx = max(mx, __float_as_uint(h[e]) & 0x7fffffffu);
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) mx = max(mx, static_cast<uint32_t>(__shfl_xor(static_cast<int>(mx), o)));
      const uint32_t byte = mx_scale_byte(mx);
      const float inv = mx_scale_inverse(byte);
      float q[8] = {};
#pragma unroll
      for (int e = 0; e < 4; ++e) q[e] = byte == 255 ? 0.0f : h[e] * inv;
      static_cast<uint16_t*>(a.y)[i] = static_cast<uint16_t>(mx_codes8(q));
      if ((i & 7) == 0) a.ys[i >> 3] = static_cast<uint8_t>(byte);
    } else {
      mx_store_hidden(a.y, 4 * i, mn, a.h_pieces, h);
    }
  }
}

// float32 rows as three bf16 planes.
__global__ __launch_bounds__(256) void mx_pieces_kernel(const float* __restrict__ x, size_t n, void* out) {
  const size_t i = (blockIdx.x * static_cast<size_t>(256) + threadIdx.x) * 4;
  if (i < n) mx_store_pieces<3>(out, i, n, *reinterpret_cast<const f32x4*>(x + i));
}

template <int kP, bool kGlu, int kWM, int kWN, int kWK, int kMB, int kNB>
hipError_t start(const MxTileArgs& a, hipStream_t stream) {
  const size_t blocks = (static_cast<size_t>(a.row_tiles) * a.tiles * a.per + a.quota - 1) / a.quota;
  mx_tile_kernel<kP, kWM, kWN, kWK, kMB, kNB, kGlu><<<static_cast<unsigned>(blocks), kThreads, 0, stream>>>(a);
  return hipGetLastError();
}

template <int kP, bool kGlu>
hipError_t start_rows(int bm, const MxTileArgs& a, hipStream_t stream) {
  if constexpr (kP == 0) {
    // MXFP4 h takes blocks of 32 columns inside a wave
    constexpr int kM = kGlu ? 2 : 1, kN = kGlu ? 4 : 2;
    switch (bm) {
      case 32: return start<0, kGlu, kM, 8 / kM, 1, 2 / kM, kN>(a, stream);
      case 64: return start<0, kGlu, kM, 8 / kM, 1, 4 / kM, kN>(a, stream);
      default:  // 128
        if (a.cols == (kGlu ? 256 : 512)) return start<0, kGlu, 1, 8, 1, 8, 4>(a, stream);
        if constexpr (kGlu) return start<0, true, 2, 4, 1, 4, 4>(a, stream);
        else return start<0, false, 1, 8, 1, 8, 2>(a, stream);
    }
  } else {
    switch (bm) {
      case 32: return start<kP, kGlu, 1, 4, 2, 2, 4>(a, stream);
      case 64: return start<kP, kGlu, 1, 4, 2, 4, 4>(a, stream);
      default: return start<kP, kGlu, 2, 4, 1, 4, 4>(a, stream);  // 128
    }
  }
}

template <int kP>
hipError_t start_glu(bool glu, int bm, const MxTileArgs& a, hipStream_t stream) {
  return glu ? start_rows<kP, true>(bm, a, stream) : start_rows<kP, false>(bm, a, stream);
}

}  // namespace

hipError_t launch_mx_tile(MxX xk, bool glu, const MxTilePlan& p, MxTileArgs& a, hipStream_t stream) {
  a.unit_steps = p.unit_steps;
  a.per = p.per;
  a.quota = p.quota;
  const auto columns = [&](int from, int to, int bm, int cols) {
    a.tile0 = from / cols;
    a.tiles = (to - from + cols - 1) / cols;
    a.bm = bm;
    a.cols = cols;
    a.row_tiles = (a.M + bm - 1) / bm;
    // a run of n tasks as r row tiles of xb bytes by n / r column tiles of wb:
    // r xb + n / r wb is least at r = sqrt(n wb / xb)
    const double n = std::max(1.0, static_cast<double>(a.row_tiles) * a.tiles / kXcds);
    const double xb = bm * (xk == kMxXfp4 ? 0.53 : (xk == kMxXbf16 ? 2 : (xk == kMxXf32h ? 4 : 6)));
    const double wb = cols * 0.53 * (glu ? 2 : 1);
    a.band = p.plane_bytes != 0 ? a.row_tiles
                                : std::min(a.row_tiles, std::max(1, static_cast<int>(std::sqrt(n * wb / xb) + 0.5)));
    switch (xk) {
      case kMxXf32: return start_glu<3>(glu, bm, a, stream);
      case kMxXf32h: return start_rows<2, false>(bm, a, stream);
      case kMxXbf16: return start_glu<1>(glu, bm, a, stream);
      case kMxXfp4: return start_glu<0>(glu, bm, a, stream);
    }
    return hipErrorInvalidValue;
  };
  if (p.rest_from != 0) {
    const hipError_t e = columns(0, p.rest_from, p.bm, p.cols);
    return e != hipSuccess ? e : columns(p.rest_from, a.N, p.rest_bm, p.rest_cols);
  }
  const hipError_t e = columns(0, a.N, p.bm, p.cols);
  if (e != hipSuccess || p.plane_bytes == 0) return e;
  const size_t n4 = static_cast<size_t>(a.M) * a.N / 4;
  const unsigned blocks = static_cast<unsigned>((n4 + 255) / 256);
  if (!glu) mx_planes_kernel<false, false><<<blocks, 256, 0, stream>>>(a);
  else if (xk == kMxXfp4) mx_planes_kernel<true, true><<<blocks, 256, 0, stream>>>(a);
  else mx_planes_kernel<true, false><<<blocks, 256, 0, stream>>>(a);
  return hipGetLastError();
}

hipError_t launch_mx_pieces(const float* x, size_t n, void* out, hipStream_t stream) {
  mx_pieces_kernel<<<static_cast<unsigned>((n / 4 + 255) / 256), 256, 0, stream>>>(x, n, out);
  return hipGetLastError();
}

}  // namespace w4
