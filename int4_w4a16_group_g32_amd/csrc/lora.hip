// Low-rank adapters beside a shared W4A16 projection:
//
//   y[m] = x[m] W + s_a (x[m] A_a^T) B_a^T,   a = ids[m],
//
// with A_a [R][K] and B_a [N][R] in bf16 and a row without an adapter
// (ids[m] outside [0, n)) taking the first term alone.
//
// Both small products run on v_mfma_f32_16x16x32_bf16.  bf16 operands enter
// as they are; a float32 operand (x, and always t = x A^T) enters as three
// bf16 pieces of 8 significant bits each: bf16 has float32's exponent range, so no
// scaling is needed, and the pieces hold the value's 24 bits.  Sums are
// float32.
//
// Rows of different adapters share an MFMA block of 16 rows: the block is
// multiplied by every adapter that occurs in it and each row keeps the result
// of its own.  The results are selected, never multiplied by zero, so an
// infinity or NaN in one adapter reaches no row of another.
#include "lora.h"

#include "dispatch.h"

namespace w4 {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

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

// ---------------------------------------------------------------- x A^T

constexpr int kShrinkThreads = 256;
constexpr int kShrinkWaves = kShrinkThreads / kWave;

struct ShrinkArgs {
  const void* x;
  const int* ids;
  LoraSet s[2];
  int M, K, splits, slots, chunks;  // chunks: of kLoraChunk ranks, over the larger R
};

// One workgroup: 16 kRB rows, one chunk of 16 kCB ranks, one K split, one slot
// of the block's distinct adapters, one projection.  The four waves take
// quarters of the split's K and meet in LDS.
template <typename XT, int kXP, int kRB, int kCB>
__global__ __launch_bounds__(kShrinkThreads) void shrink_kernel(const ShrinkArgs a) {
  constexpr int kU = kRB == 1 ? 4 : 2;
  __shared__ float red[kShrinkWaves][kRB * kLoraRows][kCB * 16];
  int b = blockIdx.x;
  const int split = b % a.splits;
  b /= a.splits;
  const int slot = b % a.slots;
  b /= a.slots;
  const int chunk = b % a.chunks;
  const int block = b / a.chunks;
  const LoraSet s = a.s[blockIdx.y];
  const int r0 = chunk * 16 * kCB;
  if (s.a == nullptr || r0 >= s.R) return;
  const int m0 = block * kRB * kLoraRows;
  const int wv = wave_id(), lane = lane_id();
  const int lc = lane & 15, kb = lane >> 4;

  // lane l knows the adapter of row m0 + l
  const int mine = lane < kRB * kLoraRows ? adapter_of(a.ids, m0 + lane, a.M, s.n) : -1;
  const int steps = a.K / 32;
  const int per = (steps + a.splits * kShrinkWaves - 1) / (a.splits * kShrinkWaves);
  const int k_lo = min(steps, (split * kShrinkWaves + wv) * per), k_hi = min(steps, k_lo + per);
  const XT* x = static_cast<const XT*>(a.x);
  const XT* xr[kRB];
#pragma unroll
  for (int rb = 0; rb < kRB; ++rb)
    xr[rb] = x + static_cast<size_t>(min(m0 + rb * kLoraRows + lc, a.M - 1)) * a.K + 8 * kb;

  uint64_t todo = __ballot(mine >= 0);
  for (int turn = 0; todo != 0; ++turn) {
    const int id = __builtin_amdgcn_readlane(mine, __ffsll(static_cast<unsigned long long>(todo)) - 1);
    const uint64_t rows = __ballot(mine == id);
    todo &= ~rows;
    if (turn % a.slots != slot) continue;
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
        for (int rb = 0; rb < kRB; ++rb) xw[u][rb] = load_x8<kXP>(xr[rb] + k);
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
          if (kRB > 1 && ((rows >> (rb * kLoraRows)) & 0xffffu) == 0) continue;  // (wave-uniform)
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
    for (int e = threadIdx.x; e < kRB * kLoraRows * kCB * 16; e += kShrinkThreads) {
      const int r = e % (kCB * 16), m = e / (kCB * 16);
      if (((rows >> m) & 1) == 0 || r0 + r >= s.R) continue;
      float v = red[0][m][r];
#pragma unroll
      for (int w = 1; w < kShrinkWaves; ++w) v += red[w][m][r];
      t[static_cast<size_t>(m0 + m) * s.R + r0 + r] = v;
    }
  }
}

// ---------------------------------------------------------------- t B^T

// t of 16 rows and one chunk of ranks as bf16 pieces in LDS; rows are padded
// so that the 16 rows of one fragment read spread over the banks.
constexpr int kTPad = kLoraChunk + 8;
struct TPieces {
  uint16_t p[3][kLoraRows][kTPad];
};

// Scaled split sums of the rows m0 .. m0 + 15, ranks r0 .. r0 + 63, as pieces.
// Ranks the row's adapter does not use, and rows without one, are zero.
__device__ __forceinline__ void stage_t(const LoraSet& s, const int* ids, int M, int m0, int r0, int splits,
                                        int tid, int nthreads, TPieces& tp) {
  for (int e = tid; e < kLoraRows * kLoraChunk; e += nthreads) {
    const int m = e / kLoraChunk, r = e % kLoraChunk;
    const int id = adapter_of(ids, m0 + m, M, s.n);
    float v = 0.0f;
    if (id >= 0 && r0 + r < rank_of(s, id)) {
      const float* t = s.t + static_cast<size_t>(m0 + m) * s.R + r0 + r;
      for (int i = 0; i < splits; ++i) v += t[static_cast<size_t>(i) * M * s.R];
      v *= s.scale[id];
    }
    uint16_t p[3];
    split3(v, p);
#pragma unroll
    for (int j = 0; j < 3; ++j) tp.p[j][m][r] = p[j];
  }
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

constexpr int kFinishThreads = 256;

// One workgroup: 16 rows x 64 kNB columns, 16 kNB columns a wave.  B enters as
// the MFMA's row operand and t as its column operand, so a lane's four
// results are four adjacent columns of one row.
template <int kNB, bool kGlu>
__global__ __launch_bounds__(kFinishThreads) void finish_kernel(const LoraFinishArgs a) {
  __shared__ TPieces tp[kGlu ? 2 : 1];
  const int blocks = (a.M + kLoraRows - 1) / kLoraRows;
  const int m0 = static_cast<int>(blockIdx.x % blocks) * kLoraRows;
  const int n0 = (static_cast<int>(blockIdx.x / blocks) * 4 + wave_id()) * 16 * kNB;
  const int lane = lane_id();
  const int lc = lane & 15, kb = lane >> 4;
  const int row = m0 + lc;

  f32x4 sum[2][kNB];
#pragma unroll
  for (int w = 0; w < 2; ++w)
#pragma unroll
    for (int nb = 0; nb < kNB; ++nb) sum[w][nb] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  const int r_max = max(a.s0.R, kGlu ? a.s1.R : 0);
  for (int r0 = 0; r0 < r_max; r0 += kLoraChunk) {
    __syncthreads();
    if (a.s0.b != nullptr && r0 < a.s0.R)
      stage_t(a.s0, a.ids, a.M, m0, r0, a.splits, threadIdx.x, kFinishThreads, tp[0]);
    if (kGlu && a.s1.b != nullptr && r0 < a.s1.R)
      stage_t(a.s1, a.ids, a.M, m0, r0, a.splits, threadIdx.x, kFinishThreads, tp[kGlu ? 1 : 0]);
    __syncthreads();
#pragma unroll
    for (int w = 0; w < (kGlu ? 2 : 1); ++w) {
      const LoraSet& s = w == 0 ? a.s0 : a.s1;
      if (s.b == nullptr || r0 >= s.R) continue;
      const int mine = adapter_of(a.ids, row, a.M, s.n);
      uint64_t todo = __ballot(mine >= 0);
      while (todo != 0) {
        const int id = __builtin_amdgcn_readlane(mine, __ffsll(static_cast<unsigned long long>(todo)) - 1);
        todo &= ~__ballot(mine == id);
        const int rank = rank_of(s, id);
        f32x4 acc[kNB];
#pragma unroll
        for (int nb = 0; nb < kNB; ++nb) acc[nb] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int ks = 0; ks < kLoraChunk / 32; ++ks) {
          if (r0 + 32 * ks >= rank) break;
          uint4 bf[kNB];
#pragma unroll
          for (int nb = 0; nb < kNB; ++nb) {
            const int n = min(n0 + 16 * nb + lc, a.N - 1);  // columns past N are not stored
            bf[nb] = load_b8(s.b + (static_cast<size_t>(id) * a.N + n) * s.R, r0 + 32 * ks + 8 * kb, rank);
          }
#pragma unroll
          for (int j = 0; j < 3; ++j) {
            const uint4 tf = *reinterpret_cast<const uint4*>(&tp[kGlu ? w : 0].p[j][lc][32 * ks + 8 * kb]);
#pragma unroll
            for (int nb = 0; nb < kNB; ++nb) acc[nb] = mfma_bf16(bf[nb], tf, acc[nb]);
          }
        }
        // element i of lane (lc, kb): column 4kb + i, row lc
        if (mine == id) {
#pragma unroll
          for (int nb = 0; nb < kNB; ++nb) sum[w][nb] += acc[nb];
        }
      }
    }
  }
  if (row >= a.M) return;
#pragma unroll
  for (int nb = 0; nb < kNB; ++nb) {
    const int n = n0 + 16 * nb + 4 * kb;
    if (n >= a.N) break;
    const size_t at = static_cast<size_t>(row) * a.N + n;
    f32x4 v = *reinterpret_cast<const f32x4*>(a.base0 + at) + sum[0][nb];
    if (kGlu) {
      const f32x4 u = *reinterpret_cast<const f32x4*>(a.base1 + at) + sum[1][nb];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = silu(v[i]) * u[i];
    }
    if (a.out_bf16)
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at) =
          make_uint2(f32_to_bf16(v[0]) | (static_cast<uint32_t>(f32_to_bf16(v[1])) << 16),
                     f32_to_bf16(v[2]) | (static_cast<uint32_t>(f32_to_bf16(v[3])) << 16));
    else
      *reinterpret_cast<f32x4*>(static_cast<float*>(a.out) + at) = v;
  }
}

template <typename XT, int kXP, int kRB>
void launch_shrink_rb(const ShrinkArgs& a, int cb, dim3 grid, hipStream_t stream) {
  if (cb == 1)
    shrink_kernel<XT, kXP, kRB, 1><<<grid, kShrinkThreads, 0, stream>>>(a);
  else if (cb == 2)
    shrink_kernel<XT, kXP, kRB, 2><<<grid, kShrinkThreads, 0, stream>>>(a);
  else
    shrink_kernel<XT, kXP, kRB, 4><<<grid, kShrinkThreads, 0, stream>>>(a);
}

}  // namespace

// 16-rank column blocks of one workgroup's chunk.
static int shrink_cols(int R) { return R <= 16 ? 1 : (R <= 32 ? 2 : 4); }

ShrinkShape shrink_shape(int M, int K, int R, int n, int sets) {
  ShrinkShape sh;
  sh.rb = M <= kLoraRows ? 1 : 4;
  const int rows = sh.rb * kLoraRows;
  const int blocks = (M + rows - 1) / rows;
  const int chunks = (R + 16 * shrink_cols(R) - 1) / (16 * shrink_cols(R));
  sh.slots = std::min({std::min(M, rows), n, 8});
  // about two workgroups per CU, a wave keeping at least two k steps
  const int most = std::max(1, std::min(M <= 256 ? kLoraMaxSplits : 4, K / 32 / (2 * kShrinkWaves)));
  sh.splits = std::min(most, std::max(1, 512 / std::max(1, blocks * chunks * sets * sh.slots)));
  return sh;
}

w4a16_status_t launch_lora_shrink(const void* x, w4a16_dtype_t xt, int M, int K, const int* ids, const LoraSet* sets,
                                  int n_sets, const ShrinkShape& sh, hipStream_t stream) {
  int R = 0;
  ShrinkArgs a{};
  a.x = x;
  a.ids = ids;
  for (int i = 0; i < n_sets; ++i) {
    a.s[i] = sets[i];
    if (sets[i].a != nullptr) R = std::max(R, sets[i].R);
  }
  if (R == 0 || M == 0) return W4A16_OK;
  const int cb = shrink_cols(R);
  a.M = M;
  a.K = K;
  a.splits = sh.splits;
  a.slots = sh.slots;
  a.chunks = (R + 16 * cb - 1) / (16 * cb);
  const size_t rows = static_cast<size_t>(sh.rb) * kLoraRows;
  const size_t blocks = (M + rows - 1) / rows * a.chunks * a.slots * a.splits;
  if (blocks > 0x7fffffffu) return W4A16_ERR_UNSUPPORTED;
  const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>(n_sets));
  if (xt == W4A16_BF16) {
    if (sh.rb == 1)
      launch_shrink_rb<uint16_t, 1, 1>(a, cb, grid, stream);
    else
      launch_shrink_rb<uint16_t, 1, 4>(a, cb, grid, stream);
  } else {
    if (sh.rb == 1)
      launch_shrink_rb<float, 3, 1>(a, cb, grid, stream);
    else
      launch_shrink_rb<float, 3, 4>(a, cb, grid, stream);
  }
  return launch_status();
}

w4a16_status_t launch_lora_finish(const LoraFinishArgs& a, hipStream_t stream) {
  if (a.M == 0 || a.N == 0) return W4A16_OK;
  const bool glu = a.base1 != nullptr;
  // 64 columns a wave once there are rows to fill the chip with; else 16
  const bool tall = static_cast<size_t>(a.M) * a.N >= (size_t{1} << 21);
  const int cols = tall ? 256 : 64;
  const size_t blocks = (static_cast<size_t>(a.M) + kLoraRows - 1) / kLoraRows * ((a.N + cols - 1) / cols);
  if (blocks > 0x7fffffffu) return W4A16_ERR_UNSUPPORTED;
  const dim3 grid(static_cast<unsigned>(blocks));
  if (glu && tall)
    finish_kernel<4, true><<<grid, kFinishThreads, 0, stream>>>(a);
  else if (glu)
    finish_kernel<1, true><<<grid, kFinishThreads, 0, stream>>>(a);
  else if (tall)
    finish_kernel<4, false><<<grid, kFinishThreads, 0, stream>>>(a);
  else
    finish_kernel<1, false><<<grid, kFinishThreads, 0, stream>>>(a);
  return launch_status();
}

namespace {

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

size_t t_bytes(const w4a16_lora_t* l, int M, int splits) {
  return l == nullptr ? 0 : static_cast<size_t>(splits) * M * l->rank * 4;
}

struct LoraGemmPlan {
  ShrinkShape sh;
  size_t gemm_bytes = 0, t_off = 0, base_off = 0, bytes = 0;
};

LoraGemmPlan plan_lora_gemm(int M, const w4a16_weight_t* w, w4a16_dtype_t xt, const w4a16_lora_t* l) {
  LoraGemmPlan p;
  p.sh = shrink_shape(M, w->K, l->rank, l->num_adapters, 1);
  p.gemm_bytes = plan_gemm(M, w, xt).bytes;
  Carve c;
  size_t start;
  c.take(start, p.gemm_bytes);
  c.take(p.t_off, t_bytes(l, M, p.sh.splits));
  c.take(p.base_off, static_cast<size_t>(M) * w->N * 4);
  p.bytes = c.cursor;
  return p;
}

struct LoraMlpPlan {
  ShrinkShape sh_gu, sh_d;
  size_t gemm_bytes = 0, tg_off = 0, tu_off = 0, td_off = 0, g_off = 0, u_off = 0, h_off = 0, bytes = 0;
};

LoraMlpPlan plan_lora_mlp(int M, w4a16_dtype_t xt, const w4a16_weight_t* gate, const w4a16_weight_t* down,
                          const w4a16_lora_t* lg, const w4a16_lora_t* lu, const w4a16_lora_t* ld) {
  LoraMlpPlan p;
  const int H = gate->K, I = gate->N;
  const int rank = std::max(lg ? lg->rank : 1, lu ? lu->rank : 1);
  const int n = std::max(lg ? lg->num_adapters : 1, lu ? lu->num_adapters : 1);
  p.sh_gu = shrink_shape(M, H, rank, n, (lg != nullptr) + (lu != nullptr) > 1 ? 2 : 1);
  if (ld != nullptr) p.sh_d = shrink_shape(M, I, ld->rank, ld->num_adapters, 1);
  p.gemm_bytes = std::max(plan_gemm(M, gate, xt).bytes, plan_gemm(M, down, W4A16_F32).bytes);
  Carve c;
  size_t start;
  c.take(start, p.gemm_bytes);
  c.take(p.tg_off, t_bytes(lg, M, p.sh_gu.splits));
  c.take(p.tu_off, t_bytes(lu, M, p.sh_gu.splits));
  c.take(p.td_off, t_bytes(ld, M, p.sh_d.splits));
  c.take(p.g_off, static_cast<size_t>(M) * std::max(I, H) * 4);
  c.take(p.u_off, static_cast<size_t>(M) * I * 4);
  c.take(p.h_off, static_cast<size_t>(M) * I * 4);
  p.bytes = c.cursor;
  return p;
}

}  // namespace
}  // namespace w4

using namespace w4;

extern "C" size_t w4a16_gemm_lora_workspace_bytes(int32_t M, const w4a16_weight_t* w, w4a16_dtype_t xt,
                                                  const w4a16_lora_t* lora) {
  if (M <= 0 || check_dense_grouped(w) != W4A16_OK || !known_type(xt)) return 0;
  if (lora == nullptr || check_lora(lora) != W4A16_OK) return 0;
  return plan_lora_gemm(M, w, xt, lora).bytes;
}

extern "C" w4a16_status_t w4a16_gemm_lora(const void* x, w4a16_dtype_t xt, int32_t M, const w4a16_weight_t* w,
                                          const w4a16_lora_t* lora, const int32_t* adapter_ids, void* y,
                                          w4a16_dtype_t yt, void* ws, size_t ws_bytes, hipStream_t stream) {
  w4a16_status_t st = check_dense_grouped(w);
  if (st != W4A16_OK) return st;
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
  float* base = reinterpret_cast<float*>(b + p.base_off);
  const LoraSet set = lora_set(lora, reinterpret_cast<float*>(b + p.t_off));
  if ((st = launch_lora_shrink(x, xt, M, w->K, adapter_ids, &set, 1, p.sh, stream)) != W4A16_OK) return st;
  if ((st = w4a16_gemm(x, xt, M, w, base, ws, p.gemm_bytes, stream)) != W4A16_OK) return st;
  LoraFinishArgs f{};
  f.base0 = base;
  f.s0 = set;
  f.ids = adapter_ids;
  f.splits = p.sh.splits;
  f.M = M;
  f.N = w->N;
  f.out = y;
  f.out_bf16 = yt == W4A16_BF16;
  return launch_lora_finish(f, stream);
}

extern "C" size_t w4a16_swiglu_mlp_lora_workspace_bytes(int32_t M, w4a16_dtype_t xt, const w4a16_weight_t* gate,
                                                        const w4a16_weight_t* up, const w4a16_weight_t* down,
                                                        const w4a16_lora_t* lora_gate, const w4a16_lora_t* lora_up,
                                                        const w4a16_lora_t* lora_down) {
  if (M <= 0 || check_mlp(gate, up, down) != W4A16_OK || !known_type(xt)) return 0;
  for (const w4a16_lora_t* l : {lora_gate, lora_up, lora_down})
    if (check_lora(l) != W4A16_OK) return 0;
  return plan_lora_mlp(M, xt, gate, down, lora_gate, lora_up, lora_down).bytes;
}

extern "C" w4a16_status_t w4a16_swiglu_mlp_lora(const void* x, w4a16_dtype_t xt, int32_t M,
                                                const w4a16_weight_t* gate, const w4a16_weight_t* up,
                                                const w4a16_weight_t* down, const w4a16_lora_t* lora_gate,
                                                const w4a16_lora_t* lora_up, const w4a16_lora_t* lora_down,
                                                const int32_t* adapter_ids, void* y, w4a16_dtype_t yt, void* ws,
                                                size_t ws_bytes, hipStream_t stream) {
  w4a16_status_t st = check_mlp(gate, up, down);
  if (st != W4A16_OK) return st;
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
  const LoraMlpPlan p = plan_lora_mlp(M, xt, gate, down, lora_gate, lora_up, lora_down);
  if (ws_bytes < p.bytes) return W4A16_ERR_WORKSPACE;
  char* b = static_cast<char*>(ws);
  float* g = reinterpret_cast<float*>(b + p.g_off);
  float* u = reinterpret_cast<float*>(b + p.u_off);
  float* h = reinterpret_cast<float*>(b + p.h_off);
  const LoraSet gu[2] = {lora_set(lora_gate, reinterpret_cast<float*>(b + p.tg_off)),
                         lora_set(lora_up, reinterpret_cast<float*>(b + p.tu_off))};
  const LoraSet d = lora_set(lora_down, reinterpret_cast<float*>(b + p.td_off));
  if ((st = launch_lora_shrink(x, xt, M, H, adapter_ids, gu, 2, p.sh_gu, stream)) != W4A16_OK) return st;
  if ((st = w4a16_gemm(x, xt, M, gate, g, ws, p.gemm_bytes, stream)) != W4A16_OK) return st;
  if ((st = w4a16_gemm(x, xt, M, up, u, ws, p.gemm_bytes, stream)) != W4A16_OK) return st;
  LoraFinishArgs f{};
  f.base0 = g;
  f.base1 = u;
  f.s0 = gu[0];
  f.s1 = gu[1];
  f.ids = adapter_ids;
  f.splits = p.sh_gu.splits;
  f.M = M;
  f.N = I;
  f.out = h;
  if ((st = launch_lora_finish(f, stream)) != W4A16_OK) return st;
  if ((st = launch_lora_shrink(h, W4A16_F32, M, I, adapter_ids, &d, 1, p.sh_d, stream)) != W4A16_OK) return st;
  if ((st = w4a16_gemm(h, W4A16_F32, M, down, g, ws, p.gemm_bytes, stream)) != W4A16_OK) return st;
  LoraFinishArgs o{};
  o.base0 = g;
  o.s0 = d;
  o.ids = adapter_ids;
  o.splits = p.sh_d.splits;
  o.M = M;
  o.N = H;
  o.out = y;
  o.out_bf16 = yt == W4A16_BF16;
  return launch_lora_finish(o, stream);
}
