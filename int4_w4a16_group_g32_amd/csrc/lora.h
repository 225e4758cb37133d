// Low-rank adapters of many requests beside a shared W4A16 projection
// (internal interface).
#pragma once

#include "common.h"
#include "gemv.h"

namespace w4 {

constexpr int kLoraMaxRank = 256;
constexpr int kLoraChunk = 64;  // adapter ranks handled together by the block kernels
constexpr int kLoraRows = 16;   // rows of one MFMA block

// One projection's adapters as the kernels read them.
struct LoraSet {
  const uint16_t* a;   // bf16 [n][R][K]; null: this projection has no adapters
  const uint16_t* b;   // bf16 [n][N][R]
  const float* scale;  // [n]
  const int* ranks;    // [n], or null: R for every adapter
  float* t;            // scale * x A^T, split sums: [splits][M][R], float32
  int R, n;
};

inline LoraSet lora_set(const w4a16_lora_t* l, float* t) {
  LoraSet s{};
  if (l == nullptr) return s;
  s.a = static_cast<const uint16_t*>(l->a);
  s.b = static_cast<const uint16_t*>(l->b);
  s.scale = l->scale;
  s.ranks = l->ranks;
  s.t = t;
  s.R = l->rank;
  s.n = l->num_adapters;
  return s;
}

// Launch shape of the first product: by rows (a workgroup takes one row and a
// few ranks) or by blocks of 64 rows, in K splits.
struct ShrinkShape {
  bool rows = true;
  int splits = 1;
};
ShrinkShape shrink_shape(int M, int K, int R);

// What a projection needs of x beside t: f16 pieces, each row scaled by a power
// of two (2^-e to rs).  Chunk c of 8 values of row m, piece j, is the 16 bytes
// at unit (c / 4) * group + (c % 4) * chunk + m * row + j * piece, for chunks c <
// chunks (those past K are zeros) and m < rows (those past M are zeros); rows 0:
// nothing.
struct LoraPrep {
  int pieces, rows, chunks;
  size_t group, chunk, row, piece;
  uint4* out;
  _Float16* tiles;  // out, where it is laid out as the 64-row tiles' pieces
  float* rs;
};

// The pieces, and t[split][m][r] = scale[id] * sum over the split's k of
// x[m][k] * a[id][r][k] for the rows m with an adapter id = ids[m] in [0, n) and
// the ranks r it uses (the other entries are left as they were).  Up to two
// projections of the same x.
w4a16_status_t launch_lora_head(const void* x, w4a16_dtype_t xt, int M, int K, const int* ids, const LoraSet* sets,
                                int n_sets, const ShrinkShape& sh, const LoraPrep& prep, hipStream_t stream);

// The base product's sums as a tile launch left them: rs[m] * the sum of S
// planes (plane_rows x ld), in split order.
struct LoraBase {
  const float* p;
  int S, plane_rows, ld;
  size_t split_stride;  // floats from one split's plane to the next
  const float* rs;      // row factors, or null: 1
};

// out[m][n] = base[m][n] + t[m] . b[id][n]; with two bases (gate, up), h[m][n]
// = silu(gate) * up of two such sums.  out float32 or bf16 (round to nearest
// even).
struct LoraFinishArgs {
  LoraBase base0, base1;  // base1.p: up (SwiGLU), else null
  LoraSet s0, s1;
  const int* ids;
  int rows, splits;  // the shape of t
  int M, N;
  void* out;
  int out_bf16;
};
w4a16_status_t launch_lora_finish(const LoraFinishArgs& a, hipStream_t stream);

// The base product of a few rows (up to 8 in two pieces, 16 in one) with the
// adapters' second product in its epilogue, one launch.
struct LoraStreamPlan {
  bool ok = false;
  int waves = 16, cols = 1, parts = 1, splits = 1, gpp = 4, tiles = 1;
  size_t partial_bytes = 0;
};
LoraStreamPlan plan_lora_stream(int M, int pieces, int N, int mats, int K);
struct LoraStreamArgs {
  const uint4* xs;  // the prepared rows
  const float* rs;
  int pieces;
  int M, K, N;
  const u32x4 *qw0, *qw1;  // qw1: up (SwiGLU), else null
  const float *sc0, *sc1;
  int gshift;
  LoraSet s0, s1;
  const int* ids;
  int cols, parts, splits, gpp;  // the plan
  float* partials;
  int* counters;
  void* out;
  int out_bf16;
};
w4a16_status_t launch_lora_stream(LoraStreamArgs a, const LoraStreamPlan& p, hipStream_t stream);

// The base product of up to 64 rows, in K splits whose sums are left in planes
// [splits][M][mats * N] for the finish.
struct LoraTilePlan {
  bool ok = false;
  int parts = 2, splits = 1, gpp = 4, tiles = 1;
  size_t groups = 0;  // of the prepared rows: parts * gpp * splits, past K zeros
  size_t plane_bytes = 0;
};
LoraTilePlan plan_lora_tiles(int M, int pieces, int N, int mats, int K);
struct LoraTileArgs {
  const uint4* xs;  // the prepared rows
  int pieces;
  int M, K, N, mats;
  const u32x4 *qw0, *qw1;
  const float *sc0, *sc1;
  int gshift;
  int splits, gpp;  // the plan
  float* planes;
};
w4a16_status_t launch_lora_tiles(LoraTileArgs a, const LoraTilePlan& p, hipStream_t stream);

}  // namespace w4
