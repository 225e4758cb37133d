// A whole routed MoE layer for a few tokens, from router logits to outputs, in
// two launches:
//
//   ids, w = the top_k largest logits of a token and their softmax,
//   y[t] = sum over experts e of w[t][e] (silu(x Wg_e) * (x Wu_e)) Wd_e
//          (+ the shared expert's MLP of x).
//
// A few tokens pick a few experts, and the layer is as fast as those experts'
// weights stream (27.5 MB each at hidden 7168, intermediate 2048): what it
// must avoid is launches and idle CUs.  Every workgroup of the first launch
// routes all the tokens itself (they fit one workgroup's waves), so there is
// no routing launch.  The first launch gives one workgroup an expert, a
// column tile of gate and up and a K split, and stores the split sums per
// (token, slot) pair.  The second treats the down projections of all chosen
// experts as one long product: its K axis runs through the experts one after
// another, A row t holds token t's weighted h where the expert is one of
// its own and zero elsewhere, so one accumulator sums over experts as well.
// That axis is cut into equal pieces, and the last workgroup of a column tile
// to arrive adds the pieces in order.
#include <cfloat>
#include <type_traits>

#include "dispatch.h"
#include "stream.h"

namespace w4 {
namespace {

constexpr int kMdQuad = 256;      // threads of a quad: four waves, 256 columns
constexpr int kMdMaxE = 1024;
constexpr int kMdMaxK = 32;
constexpr int kMdRing = 4;        // groups of codes in flight per wave
constexpr int kMdMaxSplits = 64;  // pieces of the down projection's long axis
constexpr int kMdTarget = 1024;   // quads resident at once (four per CU)

// What the tokens chose: the distinct experts of nonzero weight in ascending
// order (the items), which tokens each serves, and the gate weights of the
// (expert, token) pairs in that order.  Pair first[i] + (tokens of item i
// below t) is token t's row of item i.
struct MdItems {
  float w[kStreamRows * kMdMaxK];           // by pair
  short experts[kStreamRows * kMdMaxK];     // by item
  uint16_t tokens[kStreamRows * kMdMaxK];   // by item: bit t
  uint16_t first[kStreamRows * kMdMaxK];    // by item
  int n, pad[3];
};

// The choices as they are made, before they are turned into items.
struct MdChoice {
  float w[kStreamRows][kMdMaxK];
  short ids[kStreamRows][kMdMaxK];
  uint32_t present[kMdMaxE / 32];
  short below[kMdMaxE / 32];  // experts present in the words before
  int mask[kStreamRows * kMdMaxK];
};

__device__ __forceinline__ int md_pair(const MdItems& it, int item, int t) {
  return it.first[item] + __popc(it.tokens[item] & ((1u << t) - 1u));
}

// A wave-uniform value in scalar registers.
__device__ __forceinline__ uint64_t uniform64(uint64_t v) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v));
  const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v >> 32));
  return static_cast<uint64_t>(hi) << 32 | lo;
}

// Largest value of the wave, as a scalar: row shifts within 16 lanes, then
// broadcasts across rows; lane 63 ends with all of them.
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

// One wave selects a token's experts: the largest logits first, equal ones in
// ascending expert index, NaN as -infinity.  Keys are the logits' bits in
// unsigned order; 0 marks a taken or absent expert.  Weights are
// exp(l - l_max) / sum over the chosen, as w4a16_moe_topk computes them; a
// token with no logit above -infinity gets weight 0 everywhere.
template <int kJ>
__device__ __forceinline__ void md_topk(const float* __restrict__ logits, int E, int k, int lane, short* ids,
                                        float* w) {
  uint32_t key[kJ];
#pragma unroll
  for (int j = 0; j < kJ; ++j) {
    const int e = lane + kWave * j;
    float v = e < E ? logits[e] : 0.0f;
    if (v != v) v = -INFINITY;
    const uint32_t u = __float_as_uint(v == 0.0f ? 0.0f : v);  // -0 and 0 are equal
    key[j] = e < E ? (u & 0x80000000u ? ~u : u | 0x80000000u) : 0u;
  }
  float mine = 0.0f;
  int mine_e = 0;
  for (int r = 0; r < k; ++r) {
    uint32_t best = key[0];
#pragma unroll
    for (int j = 1; j < kJ; ++j) best = best > key[j] ? best : key[j];
    best = wave_max(best);
    int e = -1;
#pragma unroll
    for (int j = 0; j < kJ; ++j) {
      if (e < 0) {
        const uint64_t at = __ballot(key[j] == best);
        if (at != 0) e = kWave * j + __ffsll(static_cast<unsigned long long>(at)) - 1;
      }
    }
#pragma unroll
    for (int j = 0; j < kJ; ++j)
      if (e == lane + kWave * j) key[j] = 0;
    if (lane == r) {
      mine = __uint_as_float(best & 0x80000000u ? best & 0x7fffffffu : ~best);
      mine_e = e;
    }
  }
  mine = fminf(mine, FLT_MAX);  // inf - inf
  const float vmax = __shfl(mine, 0);
  const float z = lane < k && vmax > -INFINITY ? expf(mine - vmax) : 0.0f;
  float sum = z;
#pragma unroll
  for (int off = kWave / 2; off >= 1; off >>= 1) sum += __shfl_down(sum, off);
  sum = __shfl(sum, 0);
  if (lane < k) {
    ids[lane] = static_cast<short>(mine_e);
    w[lane] = sum > 0.0f ? z / sum : 0.0f;
  }
}

// All tokens' choices, by every workgroup for itself (every thread calls it;
// it ends with a barrier).
__device__ __forceinline__ void md_route(const float* __restrict__ logits, int M, int E, int k, MdChoice& ch,
                                         MdItems& it) {
  const int tid = threadIdx.x, nt = blockDim.x, lane = lane_id();
  if (tid < kMdMaxE / 32) ch.present[tid] = 0;
  for (int i = tid; i < M * k; i += nt) ch.mask[i] = 0;
  for (int t = wave_id(); t < M; t += nt / kWave) {
    const float* l = logits + static_cast<size_t>(t) * E;
    if (E <= 2 * kWave)
      md_topk<2>(l, E, k, lane, ch.ids[t], ch.w[t]);
    else if (E <= 8 * kWave)
      md_topk<8>(l, E, k, lane, ch.ids[t], ch.w[t]);
    else
      md_topk<16>(l, E, k, lane, ch.ids[t], ch.w[t]);
  }
  __syncthreads();
  for (int p = tid; p < M * k; p += nt) {
    const int e = ch.ids[p / k][p % k];
    if (ch.w[p / k][p % k] != 0.0f) atomicOr(&ch.present[e >> 5], 1u << (e & 31));
  }
  __syncthreads();
  if (wave_id() == 0) {
    uint32_t bits = lane < kMdMaxE / 32 ? ch.present[lane] : 0u;
    const int c = __popc(bits);
    int at = c;
#pragma unroll
    for (int off = 1; off < kWave; off <<= 1) {
      const int t = __shfl_up(at, off);
      if (lane >= off) at += t;
    }
    if (lane == kWave - 1) it.n = at;
    at -= c;
    if (lane < kMdMaxE / 32) ch.below[lane] = static_cast<short>(at);
    for (; bits != 0; bits &= bits - 1) it.experts[at++] = static_cast<short>(32 * lane + __ffs(bits) - 1);
  }
  __syncthreads();
  auto item_of = [&](int e) {
    return ch.below[e >> 5] + __popc(ch.present[e >> 5] & ((1u << (e & 31)) - 1u));
  };
  for (int p = tid; p < M * k; p += nt)
    if (ch.w[p / k][p % k] != 0.0f) atomicOr(&ch.mask[item_of(ch.ids[p / k][p % k])], 1 << (p / k));
  __syncthreads();
  if (wave_id() == 0) {
    int carry = 0;
    for (int i0 = 0; i0 < it.n; i0 += kWave) {
      const int m = i0 + lane < it.n ? ch.mask[i0 + lane] : 0;
      const int c = __popc(m);
      int at = c;
#pragma unroll
      for (int off = 1; off < kWave; off <<= 1) {
        const int t = __shfl_up(at, off);
        if (lane >= off) at += t;
      }
      if (i0 + lane < it.n) {
        it.tokens[i0 + lane] = static_cast<uint16_t>(m);
        it.first[i0 + lane] = static_cast<uint16_t>(carry + at - c);
      }
      carry += __shfl(at, kWave - 1);
    }
  }
  __syncthreads();
  for (int p = tid; p < M * k; p += nt) {
    const float w = ch.w[p / k][p % k];
    if (w != 0.0f) it.w[md_pair(it, item_of(ch.ids[p / k][p % k]), p / k)] = w;
  }
  __syncthreads();
}

struct MdArgs {
  const void* x;
  const float* logits;
  int M, E, k, H, I;
  const u32x4 *qg, *qu, *qd;  // stacks
  const float *sg, *su, *sd;
  const u32x4 *xqg, *xqu, *xqd;  // shared expert (null: none)
  const float *xsg, *xsu, *xsd;
  int gshift, dshift;
  int tiles, S, gps;     // gate/up: tiles of 128 h columns, K splits, groups per split
  int dtiles, dsplits;   // down: tiles of 256 columns, pieces of the long axis
  int pairs;             // M * k (+ M for the shared expert: pair M * k + t)
  float* planes;         // [S][pairs][2][I] split sums of gate and up
  float* partials;       // [dtiles][dsplits][M][256]
  int* counters;         // [dtiles], zero between calls
  MdItems* items;        // the choice, for the second launch
  int32_t* out_ids;      // caller's copies, or null
  float* out_w;
  void* y;
  int y_bf16;
};

// 16 consecutive activations.
template <int kP>
__device__ __forceinline__ void md_load_x(const void* x, size_t at, float v[16]) {
  if (kP == 1) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x) + at);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const uint4 u = p[q];
      const uint32_t wd[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        v[8 * q + 2 * t] = __uint_as_float(wd[t] << 16);
        v[8 * q + 2 * t + 1] = __uint_as_float(wd[t] & 0xffff0000u);
      }
    }
  } else {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(x) + at);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float4 u = p[q];
      v[4 * q] = u.x;
      v[4 * q + 1] = u.y;
      v[4 * q + 2] = u.z;
      v[4 * q + 3] = u.w;
    }
  }
}

// Gate and up of one expert, one tile of 128 h columns (of a quad's waves 0, 1
// gate, 2, 3 the same columns of up), one K split.  The kQ quads of a
// workgroup take consecutive parts of the split's K and meet in LDS, so that
// few split sums go through memory.
template <int kQ, int kP>
__global__ __launch_bounds__(kMdQuad * kQ) __attribute__((amdgpu_waves_per_eu(4)))
void md_gate_up_kernel(const MdArgs a) {
  constexpr int kRows = kP == 2 ? 8 : 16;
  __shared__ StreamLds lds_all[kQ];
  __shared__ MdItems rt;
  __shared__ int token[kStreamRows];
  const int split = blockIdx.x % a.S;
  const int rest = blockIdx.x / a.S;
  const int tile = rest % a.tiles;
  int item = rest / a.tiles;
  const int wv = wave_id(), lane = lane_id();
  const int q = wv >> 2, wq = wv & 3;
  const int lc = lane & 15, kb = lane >> 4;
  StreamLds& lds = lds_all[q];

  // the choice is made in what will be the first window
  static_assert(sizeof(MdChoice) <= sizeof(lds_all[0].buf), "the choice must fit in a window");
  MdChoice& ch = *reinterpret_cast<MdChoice*>(lds_all[0].buf);
  md_route(a.logits, a.M, a.E, a.k, ch, rt);
  if (blockIdx.x == 0) {  // for the second launch and the caller
    for (int p = threadIdx.x; p < a.M * a.k; p += kMdQuad * kQ) {
      if (a.out_ids != nullptr) a.out_ids[p] = ch.ids[p / a.k][p % a.k];
      if (a.out_w != nullptr) a.out_w[p] = ch.w[p / a.k][p % a.k];
    }
    static_assert(sizeof(MdItems) % 16 == 0, "copied in 16-byte units");
    for (int i = threadIdx.x; i < static_cast<int>(sizeof(MdItems) / 16); i += kMdQuad * kQ)
      reinterpret_cast<uint4*>(a.items)[i] = reinterpret_cast<const uint4*>(&rt)[i];
  }
  const bool is_shared = a.xqg != nullptr && item == 0;
  if (a.xqg != nullptr) --item;
  if (item >= rt.n) return;
  const int expert = is_shared ? 0 : __builtin_amdgcn_readfirstlane(rt.experts[item]);

  // the expert's rows, in token order
  const uint32_t has = __builtin_amdgcn_readfirstlane(is_shared ? (1u << a.M) - 1u : rt.tokens[item]);
  const int nrows = __popc(has);
  const int pair0 = __builtin_amdgcn_readfirstlane(is_shared ? a.M * a.k : rt.first[item]);
  if (wv == 0 && lane < kStreamRows && ((has >> lane) & 1)) token[__popc(has & ((1u << lane) - 1u))] = lane;
  __syncthreads();

  const int mat = wq >> 1;
  const int c0 = tile * 128 + (wq & 1) * 64;
  const bool wave_ok = c0 < a.I;
  const int G = a.H / kGroup;
  const size_t ebase = static_cast<size_t>(expert) * G * a.I;
  const u32x4* qw = (is_shared ? (mat ? a.xqu : a.xqg) : (mat ? a.qu : a.qg)) + ebase;
  const float* sc = (is_shared ? (mat ? a.xsu : a.xsg) : (mat ? a.su : a.sg)) + (ebase >> a.gshift);
  // a wave past the last column streams column block 0 and stores nothing
  const StreamLane off = stream_lane(wave_ok ? c0 : 0, lane);
  // (a quad past the last group streams the last one and adds zero)
  const int part = split * kQ + q;
  const int g_lo = min(G, part * a.gps), g_hi = min(G, g_lo + a.gps), g_last = max(g_hi - 1, 0);
  const uint32_t magic = magic_vgpr();
  const bool arow = (kP == 2 ? (lc & 7) : lc) < nrows;
  auto codes = [&](int g, StreamCodes& c) {
    const size_t gg = static_cast<size_t>(min(g, g_last));
    stream_codes(qw + gg * a.I, sc + (gg >> a.gshift) * a.I, a.I, off, c);
  };

  f32x4 tot[4];
#pragma unroll
  for (int cb = 0; cb < 4; ++cb) tot[cb] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  StreamCodes ring[kMdRing];
  float xv[16];
  auto load = [&](int gw, int m) {
    const int g = min(gw + (lane >> 1), g_last);
    md_load_x<kP>(a.x, static_cast<size_t>(token[m]) * a.H + g * kGroup + 16 * (lane & 1), xv);
  };
  if (wq < nrows) load(g_lo, wq);
#pragma unroll
  for (int j = 0; j < kMdRing; ++j) codes(g_lo + j, ring[j]);
  // every quad runs the same number of windows, so that all meet at the barriers
  for (int w0 = 0; w0 < a.gps; w0 += kStreamWin) {
    const int gw = g_lo + w0;
    const int nw = max(0, min(kStreamWin, g_hi - gw));
    if (w0 != 0) {
      __syncthreads();  // the previous window is consumed
      if (wq < nrows) load(gw, wq);
    }
    for (int m = wq; m < kRows; m += 4) {
      if (m >= nrows) {
        if (lane == 0) stream_no_row(lds, m);
        continue;
      }
      if (m != wq) load(gw, m);
      if ((lane >> 1) >= nw) {
#pragma unroll
        for (int i = 0; i < 16; ++i) xv[i] = 0.0f;
      }
      stream_store<kP>(lds, m, nw, lane, w0 == 0, true, xv);
    }
    __syncthreads();
    if (w0 != 0) stream_rescale<kP>(lds, kb, tot);
    for (int gl = 0; gl < nw; gl += kMdRing) {
#pragma unroll
      for (int j = 0; j < kMdRing; ++j) {
        const bool on = gl + j < nw;
        stream_mma(lds, on ? gl + j : gl, lc, kb, arow && on, magic, ring[j], tot);
        codes(gw + gl + j + kMdRing, ring[j]);
      }
    }
  }
  stream_finish<kP>(lds, kb, tot);
  if (kQ > 1) {  // the quads' sums, in order
    __syncthreads();  // the windows are free
    f32x4* red = reinterpret_cast<f32x4*>(lds_all[q].buf);
    if (q > 0) {
#pragma unroll
      for (int cb = 0; cb < 4; ++cb) red[(wq * 4 + cb) * kWave + lane] = tot[cb];
    }
    __syncthreads();
    if (q > 0) return;
#pragma unroll
    for (int p = 1; p < kQ; ++p) {
      const f32x4* r = reinterpret_cast<const f32x4*>(lds_all[p].buf);
#pragma unroll
      for (int cb = 0; cb < 4; ++cb) tot[cb] += r[(wq * 4 + cb) * kWave + lane];
    }
  }
  if (!wave_ok || (kP == 2 && lane >= 32)) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 4 * kb + i;
    if (r < nrows) {
      float* o = a.planes + ((static_cast<size_t>(split) * a.pairs + pair0 + r) * 2 + mat) * a.I + c0 + 4 * lc;
      *reinterpret_cast<f32x4*>(o) = f32x4{tot[0][i], tot[1][i], tot[2][i], tot[3][i]};
    }
  }
}

// 16 consecutive values of h = silu(gate) up of one pair, from the split sums:
// all of the first sum's loads in flight, then four values at a time
// (registers: the weights in flight need the rest).
__device__ __forceinline__ void md_load_h(const MdArgs& a, int pair, int k, float w, float v[16]) {
  const float* b = a.planes + static_cast<size_t>(pair) * 2 * a.I + k;
  const size_t step = static_cast<size_t>(a.pairs) * 2 * a.I;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f32x4 g = *reinterpret_cast<const f32x4*>(b + 4 * i);
    f32x4 u = *reinterpret_cast<const f32x4*>(b + a.I + 4 * i);
#pragma unroll 1
    for (int s = 1; s < a.S; ++s) {
      g += *reinterpret_cast<const f32x4*>(b + s * step + 4 * i);
      u += *reinterpret_cast<const f32x4*>(b + s * step + a.I + 4 * i);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[4 * i + j] = silu(g[j]) * u[j] * w;
      __builtin_amdgcn_sched_barrier(0);
    }
  }
}

// One tile of 256 output columns, one piece of the long axis.  Groups are
// numbered through the experts: group f belongs to item f / G.  A window may
// span experts, and the code ring runs on across them.
template <int kP>
__global__ __launch_bounds__(kMdQuad) __attribute__((amdgpu_waves_per_eu(4)))
void md_down_kernel(const MdArgs a) {
  constexpr int kRows = kP == 2 ? 8 : 16;
  __shared__ StreamLds lds;
  __shared__ MdItems rt;
  __shared__ int last;
  const int split = blockIdx.x % a.dsplits;
  const int tile = blockIdx.x / a.dsplits;
  const int wv = wave_id(), lane = lane_id();
  const int lc = lane & 15, kb = lane >> 4;
  for (int i = threadIdx.x; i < static_cast<int>(sizeof(MdItems) / 16); i += kMdQuad)
    reinterpret_cast<uint4*>(&rt)[i] = reinterpret_cast<const uint4*>(a.items)[i];
  __syncthreads();
  const int G = a.I / kGroup;
  const int routed = __builtin_amdgcn_readfirstlane(rt.n);
  const int total = (routed + (a.xqd != nullptr ? 1 : 0)) * G;  // the shared expert is the last item
  const int per = max(1, (total + a.dsplits - 1) / a.dsplits);
  const int live = max(1, (total + per - 1) / per);  // pieces that hold anything
  if (split >= live) return;
  const int f_lo = split * per, f_hi = min(total, f_lo + per);

  const int c0 = tile * kStreamCols + wv * 64;
  const bool wave_ok = c0 < a.H;
  const StreamLane off = stream_lane(wave_ok ? c0 : 0, lane);
  const uint32_t magic = magic_vgpr();
  const bool arow = (kP == 2 ? (lc & 7) : lc) < a.M;
  f32x4 tot[4];
#pragma unroll
  for (int cb = 0; cb < 4; ++cb) tot[cb] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  if (f_hi > f_lo) {
    // the ring's position: item and group.  It advances without a branch (one
    // would cost the loop its registers): the next item's expert is read
    // from LDS with every step.
    int item = f_lo / G, g = f_lo % G, left = f_hi - f_lo;
    int ex = rt.experts[min(item, max(routed - 1, 0))];
    // (the shared expert's weights as distances from the stacks': a choice
    // between pointers would become a branch)
    const uint64_t estride = static_cast<uint64_t>(G) * a.H;  // slots of an expert; scales: estride >> dshift
    const uint64_t xw = a.xqd == nullptr ? 0 : reinterpret_cast<uintptr_t>(a.xqd) - reinterpret_cast<uintptr_t>(a.qd);
    const uint64_t xs = a.xqd == nullptr ? 0 : reinterpret_cast<uintptr_t>(a.xsd) - reinterpret_cast<uintptr_t>(a.sd);
    auto next = [&](StreamCodes& c) {  // past the end: the last group again
      const uint64_t e = estride * static_cast<unsigned>(__builtin_amdgcn_readfirstlane(ex));
      const uint64_t ew = item >= routed ? xw : e * 16, es = item >= routed ? xs : (e >> a.dshift) * 4;
      stream_codes(reinterpret_cast<const u32x4*>(reinterpret_cast<const char*>(a.qd) +
                                                  uniform64(ew + static_cast<uint64_t>(g) * a.H * 16)),
                   reinterpret_cast<const float*>(reinterpret_cast<const char*>(a.sd) +
                                                  uniform64(es + static_cast<uint64_t>(g >> a.dshift) * a.H * 4)),
                   a.H, off, c);
      const int go = left > 1 ? 1 : 0;
      const int wrap = g + go == G ? 1 : 0;
      left -= go;
      g = wrap != 0 ? 0 : g + go;
      item += wrap;
      ex = rt.experts[min(item, max(routed - 1, 0))];
    };
    // row m of the window at item w_item, group w_g: true if some group of it
    // is the token's
    int w_item = f_lo / G, w_g = f_lo % G;
    float hv[16];
    auto load = [&](int nw, int m) {
#pragma unroll
      for (int i = 0; i < 16; ++i) hv[i] = 0.0f;
      bool mine = false;
      if ((lane >> 1) < nw) {
        int it = w_item, gg = w_g + (lane >> 1);
        for (; gg >= G; gg -= G) ++it;
        mine = it >= routed || ((rt.tokens[it] >> m) & 1);
        if (mine) {
          const int pair = it >= routed ? a.M * a.k + m : md_pair(rt, it, m);
          md_load_h(a, pair, gg * kGroup + 16 * (lane & 1), it >= routed ? 1.0f : rt.w[pair], hv);
        }
      }
      return __ballot(mine) != 0;
    };
    StreamCodes ring[kMdRing];
#pragma unroll
    for (int j = 0; j < kMdRing; ++j) next(ring[j]);
    for (int fw = f_lo; fw < f_hi; fw += kStreamWin) {
      const int nw = min(kStreamWin, f_hi - fw);
      __syncthreads();  // the previous window is consumed
      for (int m = wv; m < kRows; m += 4) {
        if (m >= a.M) {
          if (lane == 0) stream_no_row(lds, m);
          continue;
        }
        const bool live_row = load(nw, m);
        stream_store<kP>(lds, m, nw, lane, fw == f_lo, live_row, hv);
      }
      __syncthreads();
      for (w_g += nw; w_g >= G; w_g -= G) ++w_item;
      if (fw != f_lo) stream_rescale<kP>(lds, kb, tot);
      for (int gl = 0; gl < nw; gl += kMdRing) {
#pragma unroll
        for (int j = 0; j < kMdRing; ++j) {
          const bool on = gl + j < nw;
          stream_mma(lds, on ? gl + j : gl, lc, kb, arow && on, magic, ring[j], tot);
          next(ring[j]);
        }
      }
    }
    stream_finish<kP>(lds, kb, tot);
  }

  // The pieces of a tile meet as in the split-K GEMV: agent-scope stores reach
  // the device's coherence point, the counter says who came last, and that
  // workgroup's agent-scope loads read the pieces back, summed in order.
  float* base = a.partials + static_cast<size_t>(tile) * a.dsplits * a.M * kStreamCols;
  const size_t ps = static_cast<size_t>(a.M) * kStreamCols;
  if (kP == 1 || lane < 32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 4 * kb + i;
      if (r < a.M)
#pragma unroll
        for (int cb = 0; cb < 4; ++cb)
          __hip_atomic_store(base + split * ps + r * kStreamCols + wv * 64 + 4 * lc + cb, tot[cb][i],
                             __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
  }
  __builtin_amdgcn_s_waitcnt(0);  // this wave's stores are complete
  __syncthreads();
  if (threadIdx.x == 0)
    last = __hip_atomic_fetch_add(&a.counters[tile], 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == live - 1;
  __syncthreads();
  if (!last) return;
  if (threadIdx.x == 0) __hip_atomic_store(&a.counters[tile], 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  const int n = tile * kStreamCols + static_cast<int>(threadIdx.x);
  if (n >= a.H) return;
  for (int r = 0; r < a.M; ++r) {
    constexpr int kB = 16;
    float v = 0.0f;
    for (int s0 = 0; s0 < live; s0 += kB) {
      float q[kB];
#pragma unroll
      for (int j = 0; j < kB; ++j)
        q[j] = __hip_atomic_load(base + min(s0 + j, live - 1) * ps + r * kStreamCols + threadIdx.x, __ATOMIC_RELAXED,
                                 __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
      for (int j = 0; j < kB; ++j)
        if (s0 + j < live) v += q[j];
    }
    const size_t at = static_cast<size_t>(r) * a.H + n;
    if (a.y_bf16)
      static_cast<uint16_t*>(a.y)[at] = f32_to_bf16(v);
    else
      static_cast<float*>(a.y)[at] = v;
  }
}

struct MdPlan {
  int tiles = 0, quads = 1, S = 1, gps = 1, dtiles = 0, dsplits = 1, items = 0, pairs = 0;
  size_t items_off = 0, planes_off = 0, partials_off = 0, bytes = 0;
};

MdPlan plan_md(int M, int k, const w4a16_weight_t* gate, bool shared) {
  MdPlan p;
  const int H = gate->K, I = gate->N, G = H / kGroup;
  p.items = std::min(M * k, gate->num_experts) + (shared ? 1 : 0);
  p.pairs = M * k + (shared ? M : 0);
  p.tiles = (I + 127) / 128;
  // parts of gate and up's K until one round of quads fills the chip, each
  // of at least 8 groups; up to four parts are the quads of one workgroup
  const int parts = std::max(1, std::min(kMdTarget / std::max(1, p.items * p.tiles), G / 8));
  p.quads = parts >= 4 ? 4 : (parts >= 2 ? 2 : 1);
  p.S = std::min(parts / p.quads, 8);
  p.gps = std::max(1, (G + p.S * p.quads - 1) / (p.S * p.quads));
  p.S = std::max(1, (G + p.gps * p.quads - 1) / (p.gps * p.quads));  // no empty split
  p.dtiles = (H + kStreamCols - 1) / kStreamCols;
  const int total = p.items * (I / kGroup);
  p.dsplits = std::max(1, std::min({kMdTarget / std::max(1, p.dtiles), total / 8, kMdMaxSplits}));
  Carve c;
  size_t counters;
  c.take(counters, kCounterBytes);
  c.take(p.items_off, sizeof(MdItems));
  c.take(p.planes_off, static_cast<size_t>(p.S) * p.pairs * 2 * I * 4);
  c.take(p.partials_off, static_cast<size_t>(p.dtiles) * p.dsplits * M * kStreamCols * 4);
  p.bytes = c.cursor;
  return p;
}

w4a16_status_t check_md_stack(const w4a16_weight_t* gate, const w4a16_weight_t* up, const w4a16_weight_t* down) {
  for (const w4a16_weight_t* w : {gate, up, down}) {
    const w4a16_status_t st = check_weight(w);
    if (st != W4A16_OK) return st;
    if (w->layout != W4A16_LAYOUT_GROUPED) return W4A16_ERR_UNSUPPORTED;
  }
  if (gate->num_experts != up->num_experts || gate->num_experts != down->num_experts) return W4A16_ERR_UNSUPPORTED;
  if (gate->K != up->K || gate->N != up->N || gate->group_size != up->group_size) return W4A16_ERR_UNSUPPORTED;
  if (down->K != gate->N || down->N != gate->K) return W4A16_ERR_UNSUPPORTED;
  return W4A16_OK;
}

// Everything but pointers and M's sign: weights, shared expert, limits.
w4a16_status_t check_md(int M, int k, w4a16_dtype_t xt, const w4a16_weight_t* gate, const w4a16_weight_t* up,
                        const w4a16_weight_t* down, const w4a16_weight_t* sg, const w4a16_weight_t* su,
                        const w4a16_weight_t* sd) {
  w4a16_status_t st = check_md_stack(gate, up, down);
  if (st != W4A16_OK) return st;
  if (sg != nullptr || su != nullptr || sd != nullptr) {
    if (sg == nullptr || su == nullptr || sd == nullptr) return W4A16_ERR_INVALID_ARG;
    if ((st = check_md_stack(sg, su, sd)) != W4A16_OK) return st;
    if (sg->num_experts != 1 || sg->K != gate->K || sg->N != gate->N || sg->group_size != gate->group_size ||
        sd->group_size != down->group_size)
      return W4A16_ERR_UNSUPPORTED;
  }
  const int E = gate->num_experts;
  if (M < 0 || k < 1 || k > E || (xt != W4A16_F32 && xt != W4A16_BF16)) return W4A16_ERR_INVALID_ARG;
  if (E > kMdMaxE || k > kMdMaxK || M > (xt == W4A16_BF16 ? 16 : 8)) return W4A16_ERR_UNSUPPORTED;
  // 32-bit group counts and row sizes, and one counter per column tile
  if (gate->K >= 1 << 26 || gate->N >= 1 << 26) return W4A16_ERR_UNSUPPORTED;
  if (static_cast<size_t>(gate->N / kGroup) * (E + 1) >= (size_t{1} << 31)) return W4A16_ERR_UNSUPPORTED;
  if (static_cast<size_t>((gate->K + kStreamCols - 1) / kStreamCols) * sizeof(int) > kCounterBytes)
    return W4A16_ERR_UNSUPPORTED;
  return W4A16_OK;
}

const u32x4* codes_of(const w4a16_weight_t* w) { return reinterpret_cast<const u32x4*>(w->qw); }

}  // namespace
}  // namespace w4

using namespace w4;

extern "C" size_t w4a16_moe_decode_workspace_bytes(int32_t M, int32_t top_k, w4a16_dtype_t xt,
                                                   const w4a16_weight_t* gate, const w4a16_weight_t* up,
                                                   const w4a16_weight_t* down, const w4a16_weight_t* shared_gate,
                                                   const w4a16_weight_t* shared_up,
                                                   const w4a16_weight_t* shared_down) {
  if (M <= 0 || check_md(M, top_k, xt, gate, up, down, shared_gate, shared_up, shared_down) != W4A16_OK) return 0;
  return plan_md(M, top_k, gate, shared_gate != nullptr).bytes;
}

extern "C" w4a16_status_t w4a16_moe_decode(const void* x, w4a16_dtype_t xt, int32_t M, const float* logits,
                                           int32_t top_k, const w4a16_weight_t* gate, const w4a16_weight_t* up,
                                           const w4a16_weight_t* down, const w4a16_weight_t* shared_gate,
                                           const w4a16_weight_t* shared_up, const w4a16_weight_t* shared_down,
                                           int32_t* topk_ids, float* topk_w, void* y, w4a16_dtype_t yt, void* ws,
                                           size_t ws_bytes, hipStream_t stream) {
  w4a16_status_t st = check_md(M, top_k, xt, gate, up, down, shared_gate, shared_up, shared_down);
  if (st != W4A16_OK) return st;
  if (yt != W4A16_F32 && yt != W4A16_BF16) return W4A16_ERR_INVALID_ARG;
  const int H = gate->K, I = gate->N;
  if (M == 0 || H == 0 || I == 0) return W4A16_OK;
  if (x == nullptr || logits == nullptr || y == nullptr || ws == nullptr) return W4A16_ERR_INVALID_ARG;
  for (const void* q : {x, static_cast<const void*>(logits), static_cast<const void*>(topk_ids),
                        static_cast<const void*>(topk_w), static_cast<const void*>(y), static_cast<const void*>(ws)})
    if (!aligned16(q)) return W4A16_ERR_INVALID_ARG;
  if (ranges_overlap(x, static_cast<size_t>(M) * H * dtype_bytes(xt), y, static_cast<size_t>(M) * H * dtype_bytes(yt)))
    return W4A16_ERR_INVALID_ARG;
  const bool shared = shared_gate != nullptr;
  const MdPlan p = plan_md(M, top_k, gate, shared);
  if (ws_bytes < p.bytes) return W4A16_ERR_WORKSPACE;
  char* b = static_cast<char*>(ws);
  MdArgs a{};
  a.x = x;
  a.logits = logits;
  a.M = M;
  a.E = gate->num_experts;
  a.k = top_k;
  a.H = H;
  a.I = I;
  a.qg = codes_of(gate);
  a.qu = codes_of(up);
  a.qd = codes_of(down);
  a.sg = gate->scales;
  a.su = up->scales;
  a.sd = down->scales;
  if (shared) {
    a.xqg = codes_of(shared_gate);
    a.xqu = codes_of(shared_up);
    a.xqd = codes_of(shared_down);
    a.xsg = shared_gate->scales;
    a.xsu = shared_up->scales;
    a.xsd = shared_down->scales;
  }
  a.gshift = group_shift(gate);
  a.dshift = group_shift(down);
  a.tiles = p.tiles;
  a.S = p.S;
  a.gps = p.gps;
  a.dtiles = p.dtiles;
  a.dsplits = p.dsplits;
  a.pairs = p.pairs;
  a.planes = reinterpret_cast<float*>(b + p.planes_off);
  a.partials = reinterpret_cast<float*>(b + p.partials_off);
  a.counters = reinterpret_cast<int*>(b);
  a.items = reinterpret_cast<MdItems*>(b + p.items_off);
  a.out_ids = topk_ids;
  a.out_w = topk_w;
  a.y = y;
  a.y_bf16 = yt == W4A16_BF16;
  const size_t blocks = static_cast<size_t>(p.items) * p.tiles * p.S;
  if (blocks > 0x7fffffffu) return W4A16_ERR_UNSUPPORTED;
  const dim3 g1(static_cast<unsigned>(blocks)), t1(kMdQuad * p.quads);
  if (xt == W4A16_BF16) {
    if (p.quads == 4)
      md_gate_up_kernel<4, 1><<<g1, t1, 0, stream>>>(a);
    else if (p.quads == 2)
      md_gate_up_kernel<2, 1><<<g1, t1, 0, stream>>>(a);
    else
      md_gate_up_kernel<1, 1><<<g1, t1, 0, stream>>>(a);
  } else {
    if (p.quads == 4)
      md_gate_up_kernel<4, 2><<<g1, t1, 0, stream>>>(a);
    else if (p.quads == 2)
      md_gate_up_kernel<2, 2><<<g1, t1, 0, stream>>>(a);
    else
      md_gate_up_kernel<1, 2><<<g1, t1, 0, stream>>>(a);
  }
  if ((st = launch_status()) != W4A16_OK) return st;
  const dim3 g2(static_cast<unsigned>(p.dtiles * p.dsplits)), t2(kMdQuad);
  if (xt == W4A16_BF16)
    md_down_kernel<1><<<g2, t2, 0, stream>>>(a);
  else
    md_down_kernel<2><<<g2, t2, 0, stream>>>(a);
  return launch_status();
}
