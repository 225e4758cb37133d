// Low-rank adapters of many requests beside a shared W4A16 projection
// (internal interface).
#pragma once

#include "common.h"

namespace w4 {

constexpr int kLoraMaxRank = 256;
constexpr int kLoraChunk = 64;    // adapter ranks handled together
constexpr int kLoraRows = 16;     // rows of one MFMA block
constexpr int kLoraMaxSplits = 16;  // K splits of the first product

// One projection's adapters as the kernels read them.
struct LoraSet {
  const uint16_t* a;   // bf16 [n][R][K]; null: this projection has no adapters
  const uint16_t* b;   // bf16 [n][N][R]
  const float* scale;  // [n]
  const int* ranks;    // [n], or null: R for every adapter
  float* t;            // split sums of x A^T: [splits][M][R], float32
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

// Launch shape of the first product: 16-row blocks per workgroup, K splits,
// and adapter slots (workgroups that share the distinct adapters of a row
// block between them).
struct ShrinkShape {
  int rb = 1, splits = 1, slots = 1;
};
ShrinkShape shrink_shape(int M, int K, int R, int n, int sets);

// t[split][m][r] = sum over the split's k of x[m][k] * a[id][r][k] for the
// rows m with an adapter id = ids[m] in [0, n) and r < R (the other entries
// are left as they were).  Up to two projections of the same x.
w4a16_status_t launch_lora_shrink(const void* x, w4a16_dtype_t xt, int M, int K, const int* ids, const LoraSet* sets,
                                  int n_sets, const ShrinkShape& sh, hipStream_t stream);

// out[m][n] = base[m][n] + scale * (t[m] . b[id][n]); with two sets (gate,
// up), h[m][n] = silu(gate) * up of two such sums.  base is float32 [M][N];
// out float32 or bf16 (round to nearest even).
struct LoraFinishArgs {
  const float* base0;
  const float* base1;  // up (SwiGLU), else null
  LoraSet s0, s1;
  const int* ids;
  int splits;  // K splits of t
  int M, N;
  void* out;
  int out_bf16;
};
w4a16_status_t launch_lora_finish(const LoraFinishArgs& a, hipStream_t stream);

}  // namespace w4
