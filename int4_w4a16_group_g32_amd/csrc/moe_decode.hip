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
// no routing launch; it then forms h for one expert and one tile of columns
// over the whole of K, its waves sharing columns and K between them, and
// stores h times the gate weight per (expert, token) pair with its largest
// magnitude.  The second launch treats the down projections of all chosen
// experts as one long product: its K axis runs through the experts one after
// another, A row t holds token t's weighted h where the expert is one of
// its own and zero elsewhere, so one accumulator sums over experts as well.
// That axis is cut into equal pieces, and the last workgroup of a column tile
// to arrive adds the pieces in order.
#include <cfloat>

#include "dispatch.h"
#include "stream.h"

namespace w4 {
namespace {

constexpr int kMdMaxE = 1024;
constexpr int kMdMaxK = 32;
constexpr int kMdMaxThreads = 1024;
constexpr int kMdCus = 256;       // 16 waves resident on each
constexpr int kMdUnits = 512;     // window units (16 bytes) per wave: four workgroups of 4 waves share a CU
constexpr int kMdCols = 256;      // output columns of a down tile (four blocks of 64)
constexpr int kMdMaxSplits = 64;  // pieces of the down projection's long axis

// What the tokens chose: the distinct experts of nonzero weight in ascending
// order (the items), which tokens each serves, and the gate weights of the
// (expert, token) pairs in that order.  Pair first[i] + (tokens of item i
// below t) is token t's row of item i.
struct MdItems {
  float w[kStreamRows * kMdMaxK];           // by pair
  short experts[kStreamRows * kMdMaxK];     // by item
  uint16_t tokens[kStreamRows * kMdMaxK];   // by item: bit t
  uint16_t first[kStreamRows * kMdMaxK];    // by item
  uint8_t token[kStreamRows * kMdMaxK];     // by pair
  int n, pairs, pad[2];
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

// One wave selects a token's experts: the largest logits first, equal ones in
// ascending expert index, NaN as -infinity.  Keys are the logits' bits in
// unsigned order; 0 marks an absent expert.  Lane l holds the kJ experts from
// l kJ on, sorted once (stably, so the lower index stays first); a round takes
// the first lane with the wave's largest head and shifts that lane's list.
// Weights are exp(l - l_max) / sum over the chosen, as w4a16_moe_topk
// computes them; a token with no logit above -infinity gets weight 0
// everywhere.
template <int kJ>
__device__ __forceinline__ void md_topk(const float* __restrict__ logits, int E, int k, int lane, short* ids,
                                        float* w) {
  uint32_t key[kJ];
  uint64_t order = 0;  // four bits each: which of the lane's experts the sorted keys are
#pragma unroll
  for (int j = 0; j < kJ; ++j) {
    const int e = lane * kJ + j;
    float v = logits[min(e, E - 1)];
    if (v != v) v = -INFINITY;
    const uint32_t u = __float_as_uint(v == 0.0f ? 0.0f : v);  // -0 and 0 are equal
    key[j] = e < E ? (u & 0x80000000u ? ~u : u | 0x80000000u) : 0u;
  }
  {
    uint32_t idx[kJ];
#pragma unroll
    for (int j = 0; j < kJ; ++j) idx[j] = j;
#pragma unroll
    for (int pass = 0; pass < kJ; ++pass)  // odd-even transposition
#pragma unroll
      for (int j = pass & 1; j + 1 < kJ; j += 2) {
        const bool swap = key[j] < key[j + 1];
        const uint32_t hi = swap ? key[j + 1] : key[j], lo = swap ? key[j] : key[j + 1];
        const uint32_t ih = swap ? idx[j + 1] : idx[j], il = swap ? idx[j] : idx[j + 1];
        key[j] = hi;
        key[j + 1] = lo;
        idx[j] = ih;
        idx[j + 1] = il;
      }
#pragma unroll
    for (int j = 0; j < kJ; ++j) order |= static_cast<uint64_t>(idx[j]) << (4 * j);
  }
  uint32_t mine_key = 0;
  int mine_e = 0;
  for (int r = 0; r < k; ++r) {
    const uint32_t top = wave_max(key[0]);
    const int l = __builtin_ctzll(__ballot(key[0] == top));
    const int j = __builtin_amdgcn_readlane(static_cast<int>(order), l) & 15;
    mine_key = lane == r ? top : mine_key;
    mine_e = lane == r ? l * kJ + j : mine_e;
    const bool taken = lane == l;
#pragma unroll
    for (int i = 0; i + 1 < kJ; ++i) key[i] = taken ? key[i + 1] : key[i];
    key[kJ - 1] = taken ? 0u : key[kJ - 1];
    order = taken ? order >> 4 : order;
  }
  float mine = __uint_as_float(mine_key & 0x80000000u ? mine_key & 0x7fffffffu : ~mine_key);
  mine = fminf(mine, FLT_MAX);  // inf - inf
  const float vmax = __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(mine)));
  const float z = lane < k && vmax > -INFINITY ? expf(mine - vmax) : 0.0f;
  float sum = z;
#pragma unroll
  for (int off = kWave / 2; off >= 1; off >>= 1) sum += __shfl_down(sum, off);
  sum = __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(sum)));
  if (lane < k) {
    ids[lane] = static_cast<short>(mine_e);
    w[lane] = sum > 0.0f ? z / sum : 0.0f;
  }
}

// The tokens' choices, one wave a token.  The lists are sorted in registers, so
// the shortest that holds the experts is taken; of 16 instead: one token through
// 8 of 64 to 384 experts of 1024 x 256, bf16, 39.6 us for 18 to 18.7, sixteen 92
// to 97 for 42 to 49.  More than 384 experts take 16 as they are (512: 40 and 98).
__device__ __forceinline__ void md_choose(const float* __restrict__ logits, int M, int E, int k, MdChoice& ch) {
  const int lane = lane_id();
  for (int t = wave_id(); t < M; t += static_cast<int>(blockDim.x) / kWave) {
    const float* l = logits + static_cast<size_t>(t) * E;
    if (E <= 2 * kWave)
      md_topk<2>(l, E, k, lane, ch.ids[t], ch.w[t]);
    else if (E <= 4 * kWave)
      md_topk<4>(l, E, k, lane, ch.ids[t], ch.w[t]);
    else if (E <= 6 * kWave)
      md_topk<6>(l, E, k, lane, ch.ids[t], ch.w[t]);
    else
      md_topk<16>(l, E, k, lane, ch.ids[t], ch.w[t]);
  }
}

// LDS accesses of one wave, in program order.
__device__ __forceinline__ void wave_order() { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "workgroup"); }

// Inclusive scan over the wave.
__device__ __forceinline__ int wave_scan(int v, int lane) {
#pragma unroll
  for (int off = 1; off < kWave; off <<= 1) {
    const int t = __shfl_up(v, off);
    if (lane >= off) v += t;
  }
  return v;
}

// The choices as items, by one wave.  Up to 64 (token, slot) pairs: one a lane,
// each compared with all (about 700 cycles for 32 pairs, where the general
// form takes about 4000).
__device__ __forceinline__ void md_items64(int M, int k, int lane, const MdChoice& ch, MdItems& it) {
  const int n = M * k, t = lane / k, s = lane - t * k;
  const float w = lane < n ? ch.w[t][s] : 0.0f;
  const int e = w != 0.0f ? ch.ids[t][s] : kMdMaxE;
  int less = 0, earlier = 0;  // pairs of lower experts; of this one and a lower lane
  uint32_t tokens = 0;
  for (int j = 0; j < n; ++j) {
    const int ej = __builtin_amdgcn_readlane(e, j), tj = __builtin_amdgcn_readlane(t, j);
    less += ej < e ? 1 : 0;
    earlier += ej == e && j < lane ? 1 : 0;
    tokens |= ej == e ? 1u << tj : 0u;
  }
  const bool first = w != 0.0f && earlier == 0;
  uint64_t firsts = __ballot(first);
  const int items = __popcll(firsts), used = __popcll(__ballot(w != 0.0f));
  int item = 0;
  for (; firsts != 0; firsts &= firsts - 1) item += __builtin_amdgcn_readlane(e, __builtin_ctzll(firsts)) < e ? 1 : 0;
  if (w != 0.0f) {  // lanes are in token order
    it.w[less + earlier] = w;
    it.token[less + earlier] = static_cast<uint8_t>(t);
  }
  if (first) {
    it.experts[item] = static_cast<short>(e);
    it.tokens[item] = static_cast<uint16_t>(tokens);
    it.first[item] = static_cast<uint16_t>(less);
  }
  if (lane == 0) {
    it.n = items;
    it.pairs = used;
  }
}

__device__ __forceinline__ void md_items(int M, int k, int lane, MdChoice& ch, MdItems& it) {
  const int n = M * k;
  if (n <= kWave) {
    md_items64(M, k, lane, ch, it);
    return;
  }
  if (lane < kMdMaxE / 32) ch.present[lane] = 0;
  for (int p = lane; p < n; p += kWave) ch.mask[p] = 0;
  wave_order();
  for (int p = lane; p < n; p += kWave) {
    const int t = p / k, s = p - t * k, e = ch.ids[t][s];
    if (ch.w[t][s] != 0.0f) atomicOr(&ch.present[e >> 5], 1u << (e & 31));
  }
  wave_order();
  uint32_t bits = lane < kMdMaxE / 32 ? ch.present[lane] : 0u;
  const int c = __popc(bits);
  int at = wave_scan(c, lane);
  const int items = __shfl(at, kWave - 1);
  at -= c;
  if (lane < kMdMaxE / 32) ch.below[lane] = static_cast<short>(at);
  for (; bits != 0; bits &= bits - 1) it.experts[at++] = static_cast<short>(32 * lane + __ffs(bits) - 1);
  wave_order();
  auto item_of = [&](int e) {
    return ch.below[e >> 5] + __popc(ch.present[e >> 5] & ((1u << (e & 31)) - 1u));
  };
  for (int p = lane; p < n; p += kWave) {
    const int t = p / k, s = p - t * k;
    if (ch.w[t][s] != 0.0f) atomicOr(&ch.mask[item_of(ch.ids[t][s])], 1 << t);
  }
  wave_order();
  int pairs = 0;
  for (int i0 = 0; i0 < items; i0 += kWave) {
    const int m = i0 + lane < items ? ch.mask[i0 + lane] : 0;
    const int pc = __popc(m), incl = wave_scan(pc, lane);
    if (i0 + lane < items) {
      it.tokens[i0 + lane] = static_cast<uint16_t>(m);
      it.first[i0 + lane] = static_cast<uint16_t>(pairs + incl - pc);
    }
    pairs += __shfl(incl, kWave - 1);
  }
  if (lane == 0) {
    it.n = items;
    it.pairs = pairs;
  }
  wave_order();
  for (int p = lane; p < n; p += kWave) {
    const int t = p / k, s = p - t * k;
    const float w = ch.w[t][s];
    if (w != 0.0f) {
      const int pair = md_pair(it, item_of(ch.ids[t][s]), t);
      it.w[pair] = w;
      it.token[pair] = static_cast<uint8_t>(t);
    }
  }
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
  int cols, tiles, parts, gpp;  // gate/up: 64-column blocks per workgroup, column tiles, K parts, groups a part
  int dparts, dtiles, dsplits;  // down: K parts of a workgroup, column tiles, pieces of the long axis
  int units;                                    // LDS units of a workgroup's window
  float* h;              // [M * k (+ M)][I]: h times the gate weight, by pair (the shared expert's last)
  float* amax;           // [M * k (+ M)][I / 64]: largest |h| of 64 columns
  float* partials;       // [dtiles][dsplits][M][256]
  int* counters;         // [dtiles], zero between calls
  MdItems* items;        // the choice, for the second launch
  int32_t* out_ids;      // caller's copies, or null
  float* out_w;
  void* y;
  int y_bf16;
};

// Shape of a workgroup's staged window: `wing` groups for each K part, 2^rshift
// LDS rows a group.
struct MdWindow {
  int rshift, wing;
};
template <int kP>
__device__ __forceinline__ MdWindow md_window(int rows, int units, int parts, int groups) {
  MdWindow w;
  w.rshift = stream_rshift<kP>(rows);
  w.wing = max(kStreamRing, min(groups, (units / parts >> (w.rshift + 2)) / kStreamRing * kStreamRing));
  return w;
}

constexpr int kMdChoiceUnits = static_cast<int>((sizeof(MdChoice) + 15) / 16);

// h of one expert and `cols` blocks of 64 columns.  Wave w takes matrix w & 1
// (gate, up), one column block and one K part (gpp groups, a multiple of the
// ring); the parts meet in LDS, then gate and up.
//
// Where all tokens' rows fit the window they are staged while the choice is
// made, as A rows in token order, and the results of tokens that did not
// choose the expert are dropped; else the expert's own rows are, afterwards.
//
// 8 of 384 experts of 7168 x 2048 for one bf16 token: 29.3 us, 5.0 TB/s of
// weights, of which the choice and the items are 4 us before the first load;
// 32 experts for four float32 tokens 94 us, 6.2 TB/s (a plain read: 6.7).
template <int kP, int kI>
__global__ __launch_bounds__(kMdMaxThreads) __attribute__((amdgpu_waves_per_eu(4)))
void md_gate_up_kernel(const MdArgs a) {
  extern __shared__ uint4 lds[];
  __shared__ MdItems rt;
  __shared__ int token[kStreamRows];
  __shared__ uint32_t amax[kStreamRows];
  const int tile = blockIdx.x % a.tiles;
  int item = blockIdx.x / a.tiles;
  const int tid = threadIdx.x, nt = blockDim.x;
  const int wv = wave_id(), lane = lane_id();
  const int lc = lane & 15, kb = lane >> 4;
  const int G = a.H / kGroup, nch = G * 4;  // chunks of 8 values: k block c & 3 of group c >> 2
  const int all_groups = a.parts * a.gpp;   // (with those past the last of K)
  const int rshift_all = stream_rshift<kP>(a.M);
  const bool whole = (all_groups * 4 << rshift_all) + kMdChoiceUnits <= a.units;

  // the choice is made behind the window, or in it
  MdChoice& ch = *reinterpret_cast<MdChoice*>(lds + kStreamLds0 + (whole ? a.units - kMdChoiceUnits : 0));
  if (tid < kStreamLds0) lds[tid] = make_uint4(0, 0, 0, 0);
  if (tid < kStreamRows) amax[tid] = 0;
  if (whole) __syncthreads();
  auto row_max = [&](int m, int row) {
    uint32_t mx = 0;
    for (int c = tid; c < nch; c += nt)
      mx = stream_max8<kP>(stream_load_x<kP>(a.x, static_cast<size_t>(row) * a.H + 8 * c), mx);
    mx = wave_max(mx);
    if (lane == 0) atomicMax(&amax[m], mx);
  };
  if (whole)
    for (int m = 0; m < a.M; ++m) row_max(m, m);
  md_choose(a.logits, a.M, a.E, a.k, ch);
  __syncthreads();
  if (wv == 0) {
    md_items(a.M, a.k, lane, ch, rt);
  } else if (whole) {
    for (int m = 0; m < a.M; ++m)
      for (int c = tid - kWave; c < all_groups * 4; c += nt - kWave) {
        const int unit = stream_unit(c >> 2, c & 3, m * kP, rshift_all);
        if (c < nch)
          stream_put_row<kP, kP>(lds, unit, stream_load_x<kP>(a.x, static_cast<size_t>(m) * a.H + 8 * c), amax[m]);
        else
          stream_put_zero<kP>(lds, unit);
      }
  }
  __syncthreads();
  if (blockIdx.x == 0) {  // for the second launch and the caller
    for (int p = tid; p < a.M * a.k; p += nt) {
      if (a.out_ids != nullptr) a.out_ids[p] = ch.ids[p / a.k][p % a.k];
      if (a.out_w != nullptr) a.out_w[p] = ch.w[p / a.k][p % a.k];
    }
    static_assert(sizeof(MdItems) % 16 == 0, "copied in 16-byte units");
    for (int i = tid; i < static_cast<int>(sizeof(MdItems) / 16); i += nt)
      reinterpret_cast<uint4*>(a.items)[i] = reinterpret_cast<const uint4*>(&rt)[i];
  }
  const bool is_shared = a.xqg != nullptr && item == 0;
  if (a.xqg != nullptr) --item;
  if (item >= rt.n) return;
  const int expert = is_shared ? 0 : __builtin_amdgcn_readfirstlane(rt.experts[item]);
  // the tokens it serves, and its A rows
  const uint32_t has = __builtin_amdgcn_readfirstlane(is_shared ? (1u << a.M) - 1u : rt.tokens[item]);
  const int nrows = whole ? a.M : __popc(has);
  const int pair0 = __builtin_amdgcn_readfirstlane(is_shared ? a.M * a.k : rt.first[item]);

  // weights: wave-uniform bases, the ring from the part's first group on
  const int mat = wv & 1, col = (wv >> 1) & (a.cols - 1);
  const int part = (wv >> 1) / a.cols;
  const int block = tile * a.cols + col;
  const bool wave_ok = block * 64 < a.I;
  const uint64_t ebase = static_cast<uint64_t>(expert) * G * a.I;
  const u32x4* qw = (is_shared ? (mat ? a.xqu : a.xqg) : (mat ? a.qu : a.qg)) + ebase;
  const float* sc = (is_shared ? (mat ? a.xsu : a.xsg) : (mat ? a.su : a.sg)) + (ebase >> a.gshift);
  // a wave past the last column streams column block 0 and stores nothing, a
  // part past the last group the last one (against staged zeros)
  const StreamLane off = stream_lane(wave_ok ? block * 64 : 0, lane);
  const int g_last = G - 1;
  int g = min(part * a.gpp, g_last);
  auto next = [&](StreamCodes& c) {
    stream_codes(uniform_at(qw, static_cast<uint64_t>(g) * a.I * 16),
                 uniform_at(sc, static_cast<uint64_t>(g >> a.gshift) * a.I * 4), a.I, off, c);
    g = min(g + 1, g_last);
  };
  const uint32_t magic = magic_vgpr();
  StreamCodes ring[kStreamRing];
  if (!whole) {
    __syncthreads();  // the choice's LDS is free
    if (tid < kStreamRows && ((has >> tid) & 1)) token[__popc(has & ((1u << tid) - 1u))] = tid;
    __syncthreads();
    for (int m = 0; m < nrows; ++m) row_max(m, token[m]);
    __syncthreads();
  }
#pragma unroll
  for (int j = 0; j < kStreamRing; ++j) next(ring[j]);

  float acc[4][kI];
#pragma unroll
  for (int cb = 0; cb < 4; ++cb)
#pragma unroll
    for (int i = 0; i < kI; ++i) acc[cb][i] = 0.0f;
  const MdWindow win = whole ? MdWindow{rshift_all, a.gpp} : md_window<kP>(nrows, a.units, a.parts, a.gpp);
  const StreamFrag frag = stream_frag<kP>(lane, nrows, part * win.wing, win.rshift);
  for (int w0 = 0; w0 < a.gpp; w0 += win.wing) {
    if (!whole) {
      if (w0 != 0) __syncthreads();  // the previous window is consumed
      // nt / parts threads (a power of two) stage a part
      const int tpp = nt / a.parts, p = tid / tpp;
      for (int m = 0; m < nrows; ++m)
        for (int u = tid - p * tpp; u < win.wing * 4; u += tpp) {
          const int gl = u >> 2, gg = p * a.gpp + w0 + gl;
          const int unit = stream_unit(p * win.wing + gl, u & 3, m * kP, win.rshift);
          if (w0 + gl < a.gpp && gg < G)
            stream_put_row<kP, kP>(lds, unit,
                           stream_load_x<kP>(a.x, static_cast<size_t>(token[m]) * a.H + gg * kGroup + 8 * (u & 3)),
                           amax[m]);
          else
            stream_put_zero<kP>(lds, unit);
        }
      __syncthreads();
    }
    const int n = min(win.wing, a.gpp - w0);
    if (kI == 1 || nrows <= 4) {
      float one[4][1];
#pragma unroll
      for (int cb = 0; cb < 4; ++cb) one[cb][0] = acc[cb][0];
      stream_run<kP, 1>(lds, frag, n, magic, ring, next, one);
#pragma unroll
      for (int cb = 0; cb < 4; ++cb) acc[cb][0] = one[cb][0];
    } else {
      stream_run<kP, kI>(lds, frag, n, magic, ring, next, acc);
    }
  }

  // the parts' sums, in order; then up's to gate's waves
  f32x4* red = reinterpret_cast<f32x4*>(lds);
  const int pw = 2 * a.cols;  // waves of a part
  __syncthreads();  // the window is free
  if (part > 0) {
#pragma unroll
    for (int i = 0; i < kI; ++i)
      red[(wv * kI + i) * kWave + lane] = f32x4{acc[0][i], acc[1][i], acc[2][i], acc[3][i]};
  }
  __syncthreads();
  if (part == 0) {
    for (int p = 1; p < a.parts; ++p)
#pragma unroll
      for (int i = 0; i < kI; ++i) {
        const f32x4 v = red[((p * pw + wv) * kI + i) * kWave + lane];
#pragma unroll
        for (int cb = 0; cb < 4; ++cb) acc[cb][i] += v[cb];
      }
    if (mat == 1) {  // (the first part's own places are free)
#pragma unroll
      for (int i = 0; i < kI; ++i)
        red[(wv * kI + i) * kWave + lane] = f32x4{acc[0][i], acc[1][i], acc[2][i], acc[3][i]};
    }
  }
  __syncthreads();
  if (part != 0 || mat != 0 || !wave_ok) return;
#pragma unroll
  for (int i = 0; i < kI; ++i) {
    const int m = kb + 4 * i;
    // (all 16 lanes of a row together)
    if (m >= nrows || (whole && ((has >> m) & 1) == 0)) continue;
    const int pair = pair0 + (whole ? __popc(has & ((1u << m) - 1u)) : m);
    const float f = ldexpf(1.0f, -stream_exp(__uint_as_float(amax[m])));
    const float wt = is_shared ? 1.0f : rt.w[pair];
    const f32x4 u = red[((wv + 1) * kI + i) * kWave + lane];
    f32x4 h;
    float mx = 0.0f;
#pragma unroll
    for (int cb = 0; cb < 4; ++cb) {
      h[cb] = silu(acc[cb][i] * f) * (u[cb] * f) * wt;
      mx = fmaxf(mx, fabsf(h[cb]));
    }
    *reinterpret_cast<f32x4*>(a.h + static_cast<size_t>(pair) * a.I + block * 64 + 4 * lc) = h;
#pragma unroll
    for (int o = 8; o >= 1; o >>= 1) mx = fmaxf(mx, __shfl_xor(mx, o));
    if (lc == 0) a.amax[static_cast<size_t>(pair) * (a.I / 64) + block] = mx;
  }
}

// A wave's sums of md_down_kernel over groups [f0, f1) of the long axis again,
// for column block `block`, every group for the tokens that chose its expert
// alone.  Operands and order are those of the streamed form, so that sums which
// meet finite scales only keep their bits; the operands come from memory, since
// the streamed form's windows are gone.
template <int kP, int kI>
__device__ __forceinline__ void md_down_apart(const MdArgs& a, const MdItems& rt, const uint32_t* amax, int routed,
                                              int f0, int f1, int block, uint32_t magic, float acc[4][kI]) {
  const int lane = lane_id(), lc = lane & 15, kb = lane >> 4, G = a.I / kGroup;
  const int m = kP == 2 ? (lc >> 2) + 4 * ((lc >> 1) & 1) : (lc >> 2) + 4 * (lc & 3);  // the lane's A row
#pragma unroll
  for (int cb = 0; cb < 4; ++cb)
#pragma unroll
    for (int i = 0; i < kI; ++i) acc[cb][i] = 0.0f;
#pragma unroll 1
  for (int f = f0; f < f1; ++f) {
    const int item = f / G, g = f % G;
    const bool is_shared = item >= routed;
    const uint32_t who = is_shared ? (1u << a.M) - 1u : rt.tokens[item];
    const size_t e = is_shared ? 0 : static_cast<size_t>(rt.experts[item]) * G;
    const u32x4 w = ((is_shared ? a.xqd : a.qd) + (e + g) * a.H)[block * 64 + lane];
    const f32x4 sc = reinterpret_cast<const f32x4*>((is_shared ? a.xsd : a.sd) + ((e + g) >> a.dshift) * a.H +
                                                    block * 64)[lc];
    half8 p[2] = {half8{}, half8{}};
    if (m < a.M && ((who >> m) & 1)) {
      const int pair = is_shared ? a.M * a.k + m : md_pair(rt, item, m);
      float v[8];
      stream_x_values<2>(stream_load_x<2>(a.h, static_cast<size_t>(pair) * a.I + g * kGroup + 8 * kb), v);
      const float scale = ldexpf(1.0f, stream_exp(__uint_as_float(amax[m])));
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= scale;
      stream_pieces<kP>(v, p);
    }
    const half8 af = kP == 2 && (lc & 1) ? p[1] : p[0];
#pragma unroll
    for (int cb = 0; cb < 4; ++cb) {
      const f32x4 d = __builtin_amdgcn_mfma_f32_16x16x32_f16(af, codes_f16(w[cb], magic),
                                                             f32x4{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0);
#pragma unroll
      for (int i = 0; i < kI; ++i)
        if ((who >> (kb + 4 * i)) & 1) acc[cb][i] = fmaf(sc[cb], kP == 2 ? d[2 * i] + d[2 * i + 1] : d[i], acc[cb][i]);
    }
  }
}

// One tile of 256 output columns, one piece of the long axis, its K parts over
// quads of waves.  Groups are numbered through the experts: group f belongs to
// item f / G.  A window may span experts, and the code ring runs on across
// them.
// 8 experts of 2048 x 7168 for one bf16 token: 20.2 us, 3.6 TB/s (5 us before
// the stream starts, 3 us for the meeting); 32 experts for four float32 tokens
// 54 us, 5.4 TB/s.
template <int kP, int kI>
__global__ __launch_bounds__(kMdMaxThreads) __attribute__((amdgpu_waves_per_eu(4)))
void md_down_kernel(const MdArgs a) {
  extern __shared__ uint4 lds[];
  __shared__ MdItems rt;
  __shared__ uint32_t amax[kStreamRows];
  __shared__ int last;
  const int split = blockIdx.x % a.dsplits;
  const int tile = blockIdx.x / a.dsplits;
  const int tid = threadIdx.x, nt = blockDim.x;
  const int wv = wave_id(), lane = lane_id();
  const int lc = lane & 15, kb = lane >> 4;
  // the choice, and the largest magnitudes of h, 16 blocks of a pair a thread
  // (those of pairs that are not there are dropped below)
  const int nblk = a.I / 64, nseg = (nblk + 15) / 16;
  const int nval = (a.M * a.k + (a.xqd != nullptr ? a.M : 0)) * nseg;
  auto largest = [&](int q) {
    const int p = q / nseg, b0 = (q - p * nseg) * 16;
    const float* v = a.amax + static_cast<size_t>(p) * nblk;
    float mx = 0.0f;
#pragma unroll
    for (int j = 0; j < 16; ++j) mx = fmaxf(mx, v[min(b0 + j, nblk - 1)]);
    return mx;
  };
  const float mine_max = tid < nval ? largest(tid) : 0.0f;
  for (int i = tid; i < static_cast<int>(sizeof(MdItems) / 16); i += nt)
    reinterpret_cast<uint4*>(&rt)[i] = reinterpret_cast<const uint4*>(a.items)[i];
  if (tid < kStreamLds0) lds[tid] = make_uint4(0, 0, 0, 0);
  if (tid < kStreamRows) amax[tid] = 0;
  __syncthreads();
  const int G = a.I / kGroup;
  const int routed = __builtin_amdgcn_readfirstlane(rt.n);
  const int total = (routed + (a.xqd != nullptr ? 1 : 0)) * G;  // the shared expert is the last item
  const int per = max(1, (total + a.dsplits - 1) / a.dsplits);
  const int live = max(1, (total + per - 1) / per);  // pieces that hold anything
  if (split >= live) return;
  const int piece_lo = split * per, piece_hi = min(total, piece_lo + per);
  const int gpp = (per + a.dparts * kStreamRing - 1) / (a.dparts * kStreamRing) * kStreamRing;
  const int block = tile * (kMdCols / 64) + (wv & 3), part = wv >> 2;
  const bool wave_ok = block * 64 < a.H;
  const StreamLane off = stream_lane(wave_ok ? block * 64 : 0, lane);
  const uint32_t magic = magic_vgpr();

  // The ring's position: item and group.  It advances without a branch (one
  // would cost the loop its registers): the item's expert is read from LDS
  // with every step, and the shared expert's weights are distances from the
  // stacks' (a choice between pointers would become a branch).
  int left = max(1, min(piece_hi - piece_lo - part * gpp, gpp));
  int item, g;
  {
    const int f = max(0, min(piece_lo + part * gpp, total - 1));
    item = __builtin_amdgcn_readfirstlane(f / G);
    g = __builtin_amdgcn_readfirstlane(f % G);
  }
  const int item_max = max(routed - 1, 0);
  int ex = rt.experts[min(item, item_max)];
  const uint64_t estride = static_cast<uint64_t>(G) * a.H;  // slots of an expert; scales: estride >> dshift
  const uint64_t xw = a.xqd == nullptr ? 0 : reinterpret_cast<uintptr_t>(a.xqd) - reinterpret_cast<uintptr_t>(a.qd);
  const uint64_t xs = a.xqd == nullptr ? 0 : reinterpret_cast<uintptr_t>(a.xsd) - reinterpret_cast<uintptr_t>(a.sd);
  auto next = [&](StreamCodes& c) {  // past the end: the last group again
    const uint64_t e = estride * static_cast<unsigned>(__builtin_amdgcn_readfirstlane(ex));
    const uint64_t ew = item >= routed ? xw : e * 16, es = item >= routed ? xs : (e >> a.dshift) * 4;
    stream_codes(uniform_at(a.qd, ew + static_cast<uint64_t>(g) * a.H * 16),
                 uniform_at(a.sd, es + static_cast<uint64_t>(g >> a.dshift) * a.H * 4), a.H, off, c);
    const int go = left > 1 ? 1 : 0;
    const int wrap = g + go == G ? 1 : 0;
    left -= go;
    g = wrap != 0 ? 0 : g + go;
    item += wrap;
    ex = rt.experts[min(item, item_max)];
  };

  float acc[4][kI];
#pragma unroll
  for (int cb = 0; cb < 4; ++cb)
#pragma unroll
    for (int i = 0; i < kI; ++i) acc[cb][i] = 0.0f;
  StreamCodes ring[kStreamRing];
  if (total > 0) {
    // A quad's 256 threads stage its part: thread (chunk, row) takes every
    // rstep-th row of its chunks.
    MdWindow win = md_window<kP>(a.M, a.units, a.dparts, gpp);
    if (win.wing < gpp) win = md_window<kP>(a.M, a.units / 2, a.dparts, gpp);  // two windows in turn
    const int half = win.wing < gpp ? (a.dparts * win.wing * 4) << win.rshift : 0;  // units
    const StreamFrag frag = stream_frag<kP>(lane, a.M, part * win.wing, win.rshift);
    const int cshift = min(8, 32 - __builtin_clz(win.wing * 4 - 1));  // chunks of a pass: 2^cshift
    const int chunk0 = tid & ((1 << cshift) - 1), row0 = (tid & 255) >> cshift, rstep = 256 >> cshift;
    const float rcp_g = 1.0f / static_cast<float>(G);
    struct Place {
      int unit, item, k;
      uint32_t who;
    };
    auto place = [&](int c, int w0) {
      Place q;
      const int gl = c >> 2, f = piece_lo + part * gpp + w0 + gl;
      const bool in = gl < win.wing && w0 + gl < gpp && f < piece_hi;
      // f / G: at most 513 items, so the float quotient is off by one at most
      int it = static_cast<int>(static_cast<float>(f) * rcp_g), r = f - it * G;
      if (r < 0) {
        r += G;
        --it;
      } else if (r >= G) {
        r -= G;
        ++it;
      }
      q.item = in ? it : 0;
      q.unit = stream_unit(part * win.wing + gl, c & 3, 0, win.rshift);
      q.k = r * kGroup + 8 * (c & 3);
      q.who = !in ? 0u : (it >= routed ? (1u << a.M) - 1u : rt.tokens[it]);
      return q;
    };
    auto load = [&](const Place& q, int m) {
      const int pair = q.item >= routed ? a.M * a.k + m : md_pair(rt, q.item, m);
      return stream_load_x<2>(a.h, static_cast<size_t>(pair) * a.I + q.k);
    };
    // A window's h is loaded while the window before the last one is used: up to
    // two rows of the thread's place (more tokens seldom share an expert here;
    // theirs are loaded late).
    Place here;
    int here_m[2] = {-1, -1};
    StreamX8<2> here_h[2];
    auto prefetch = [&](int w0) {
      here = place(chunk0, w0);
      here_m[0] = here_m[1] = -1;
      for (int m = row0; m < a.M; m += rstep)
        if ((here.who >> m) & 1) {
          here_m[1] = here_m[0] >= 0 && here_m[1] < 0 ? m : here_m[1];
          here_m[0] = here_m[0] < 0 ? m : here_m[0];
        }
#pragma unroll
      for (int j = 0; j < 2; ++j)
        if (here_m[j] >= 0) here_h[j] = load(here, here_m[j]);
      __builtin_amdgcn_sched_barrier(0);
    };
    auto put = [&](int w0, uint4* buf) {
      for (int c = chunk0; c < win.wing * 4; c += 1 << cshift) {
        const bool ahead = c == chunk0;
        const Place q = ahead ? here : place(c, w0);
        for (int m = row0; m < a.M; m += rstep) {
          if ((q.who >> m) & 1) {
            StreamX8<2> h;
            if (ahead && m == here_m[0])
              h = here_h[0];
            else if (ahead && m == here_m[1])
              h = here_h[1];
            else
              h = load(q, m);
            stream_put_row<kP, 2>(buf, q.unit + m * kP, h, amax[m]);
          } else {
            stream_put_zero<kP>(buf, q.unit + m * kP);
          }
        }
      }
    };
    prefetch(0);
#pragma unroll
    for (int j = 0; j < kStreamRing; ++j) next(ring[j]);
    // every token's largest |w h| over its pairs
    for (int q = tid; q < nval; q += nt) {
      const int p = q / nseg;
      if (p < rt.pairs || p >= a.M * a.k)
        atomicMax(&amax[p < a.M * a.k ? rt.token[p] : p - a.M * a.k],
                  __float_as_uint(q == tid ? mine_max : largest(q)));
    }
    __syncthreads();  // the largest magnitudes are known
    put(0, lds);
    if (win.wing < gpp) prefetch(win.wing);
    __syncthreads();
    int odd = 0;
    for (int w0 = 0; w0 < gpp; w0 += win.wing) {
      const int w1 = w0 + win.wing;
      if (w1 < gpp) put(w1, lds + (odd ? 0 : half));
      if (w1 + win.wing < gpp) prefetch(w1 + win.wing);
      // (absent A rows read the zeros in front of the first window)
      StreamFrag f = frag;
      if (odd && f.step != 0) f.at += half;
      stream_run<kP, kI>(lds, f, min(win.wing, gpp - w0), magic, ring, next, acc);
      __syncthreads();  // this window is consumed, the next one staged
      odd ^= 1;
    }
    // A scale that is not finite makes NaNs of the zeros of the tokens that did
    // not choose its expert.  Sums that are not finite are taken again without
    // them.  (Clearing those tokens' scales in the stream itself cost one token 5 %
    // of the layer and sixteen 6 %.)
    bool finite = true;
#pragma unroll
    for (int cb = 0; cb < 4; ++cb)
#pragma unroll
      for (int i = 0; i < kI; ++i) finite &= fabsf(acc[cb][i]) <= FLT_MAX;
    if (__builtin_expect(wave_ok && __ballot(!finite) != 0, 0))
      md_down_apart<kP, kI>(a, rt, amax, routed, piece_lo + part * gpp,
                            min(piece_hi, piece_lo + (part + 1) * gpp), block, magic, acc);
  }

  // the parts' sums, in order
  f32x4* red = reinterpret_cast<f32x4*>(lds);
  if (a.dparts > 1) {
    if (part > 0) {
#pragma unroll
      for (int i = 0; i < kI; ++i)
        red[(wv * kI + i) * kWave + lane] = f32x4{acc[0][i], acc[1][i], acc[2][i], acc[3][i]};
    }
    __syncthreads();
    if (part == 0) {
      for (int p = 1; p < a.dparts; ++p)
#pragma unroll
        for (int i = 0; i < kI; ++i) {
          const f32x4 v = red[((p * 4 + wv) * kI + i) * kWave + lane];
#pragma unroll
          for (int cb = 0; cb < 4; ++cb) acc[cb][i] += v[cb];
        }
    }
  }

  // The pieces of a tile meet as in the split-K GEMV: agent-scope stores reach
  // the device's coherence point, the counter says who came last, and that
  // workgroup's agent-scope loads read the pieces back, summed in order.
  float* base = a.partials + static_cast<size_t>(tile) * a.dsplits * a.M * kMdCols;
  const size_t ps = static_cast<size_t>(a.M) * kMdCols;
  if (part == 0) {
#pragma unroll
    for (int i = 0; i < kI; ++i) {
      const int m = kb + 4 * i;
      if (m < a.M) {
        const float f = ldexpf(1.0f, -stream_exp(__uint_as_float(amax[m])));
        uint64_t* o = reinterpret_cast<uint64_t*>(base + split * ps + m * kMdCols + wv * 64 + 4 * lc);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint64_t v = static_cast<uint64_t>(__float_as_uint(acc[2 * j + 1][i] * f)) << 32 |
                             __float_as_uint(acc[2 * j][i] * f);
          __hip_atomic_store(o + j, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
      }
    }
  }
  __builtin_amdgcn_s_waitcnt(0);  // this wave's stores are complete
  __syncthreads();
  if (tid == 0)
    last = __hip_atomic_fetch_add(&a.counters[tile], 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == live - 1;
  __syncthreads();
  if (!last) return;
  if (tid == 0) __hip_atomic_store(&a.counters[tile], 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  // two columns a thread, kRows rows' pieces in flight together
  constexpr int kRows = kI == 1 ? 1 : 2, kB = 12, kPer = kMdCols / 2;
  const int c = 2 * (tid % kPer), n = tile * kMdCols + c, rs = nt / kPer;
  if (n >= a.H) return;
  for (int r0 = tid / kPer; r0 < a.M; r0 += rs * kRows) {
    float v[kRows][2];
#pragma unroll
    for (int r = 0; r < kRows; ++r) v[r][0] = v[r][1] = 0.0f;
    for (int s0 = 0; s0 < live; s0 += kB) {
      uint64_t q[kRows][kB];
#pragma unroll
      for (int r = 0; r < kRows; ++r)
#pragma unroll
        for (int j = 0; j < kB; ++j)
          q[r][j] = __hip_atomic_load(
              reinterpret_cast<const uint64_t*>(base + min(s0 + j, live - 1) * ps + min(r0 + r * rs, a.M - 1) * kMdCols + c),
              __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
      for (int r = 0; r < kRows; ++r)
#pragma unroll
        for (int j = 0; j < kB; ++j)
          if (s0 + j < live) {
            v[r][0] += __uint_as_float(static_cast<uint32_t>(q[r][j]));
            v[r][1] += __uint_as_float(static_cast<uint32_t>(q[r][j] >> 32));
          }
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      if (r0 + r * rs >= a.M) continue;
      const size_t at = static_cast<size_t>(r0 + r * rs) * a.H + n;
      if (a.y_bf16)
        *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.y) + at) =
            f32_to_bf16(v[r][0]) | static_cast<uint32_t>(f32_to_bf16(v[r][1])) << 16;
      else
        *reinterpret_cast<float2*>(static_cast<float*>(a.y) + at) = make_float2(v[r][0], v[r][1]);
    }
  }
}

struct MdPlan {
  int items = 0;
  int waves = 4, cols = 2, tiles = 0, parts = 1, gpp = 1;  // gate/up
  int dwaves = 4, dtiles = 0, dsplits = 1;                 // down
  size_t items_off = 0, h_off = 0, amax_off = 0, partials_off = 0, bytes = 0;
};

MdPlan plan_md(int M, int k, const w4a16_weight_t* gate, bool shared) {
  MdPlan p;
  const int H = gate->K, I = gate->N, G = H / kGroup;
  if (H == 0 || I == 0) {  // nothing is launched
    p.bytes = kCounterBytes;
    return p;
  }
  p.items = std::min(M * k, gate->num_experts) + (shared ? 1 : 0);
  // Gate and up: workgroups of 4 waves, and of 8 (more K parts), at last of half
  // the columns, while the launch would leave waves of the chip unused and a
  // part keeps a ring of groups.  Sixteen waves start later than they stream
  // faster: one token through 8 of 64 experts of 7168 x 2048 50.5 us with 8,
  // 51.7 with 16 (both kernels), four through 2048 x 1024 30.2 and 31.8.
  auto wgs = [&](int cols) { return static_cast<size_t>(p.items) * ((I / 64 + cols - 1) / cols); };
  if (wgs(p.cols) * p.waves < 16 * kMdCus && G / (p.waves / p.cols) >= kStreamRing) p.waves = 8;
  if (p.waves == 8 && wgs(2) < kMdCus && G / 4 >= kStreamRing) p.cols = 1;
  p.tiles = (I / 64 + p.cols - 1) / p.cols;
  p.parts = p.waves / (2 * p.cols);
  p.gpp = (G + p.parts * kStreamRing - 1) / (p.parts * kStreamRing) * kStreamRing;
  // Down: workgroups of 16 waves, one per CU, while each of the four parts has
  // a ring of groups or more; where they have few, of 8 with twice the splits
  // (three tokens through 128 x 256 15.8 us for 19, one through 1408 x 4096
  // 31.7 for 33.2; sixteen through 2048 x 7168, 200 groups a part, 221 for 190).
  p.dtiles = (H + kMdCols - 1) / kMdCols;
  const int total = p.items * (I / kGroup);
  auto splits = [&](int parts, int most) {
    return std::max(1, std::min({kMdCus / p.dtiles, total / (kStreamRing * parts), most}));
  };
  p.dwaves = 16;
  p.dsplits = splits(4, kMdMaxSplits);
  if (total <= 16 * 4 * p.dsplits) {
    p.dwaves = total >= 2 * kStreamRing ? 8 : 4;
    p.dsplits = splits(p.dwaves / 4, kMdMaxSplits / 2);
  }
  const size_t pairs = static_cast<size_t>(M) * k + (shared ? M : 0);
  Carve c;
  size_t counters;
  c.take(counters, kCounterBytes);
  c.take(p.items_off, sizeof(MdItems));
  c.take(p.h_off, pairs * I * 4);
  c.take(p.amax_off, pairs * (I / 64) * 4);
  c.take(p.partials_off, static_cast<size_t>(p.dtiles) * p.dsplits * M * kMdCols * 4);
  p.bytes = c.cursor;
  return p;
}

// LDS of a workgroup: the window, which also holds the choice before and the
// parts' sums (1 KiB a wave and accumulator) after.
size_t md_lds_bytes(int waves) { return (static_cast<size_t>(waves) * kMdUnits + kStreamLds0) * 16; }

template <int kP>
w4a16_status_t launch_md(const MdPlan& p, MdArgs a, hipStream_t stream) {
  static_assert(kMdChoiceUnits <= 4 * kMdUnits && 4 * kWave <= kMdUnits, "the choice and the sums must fit");
  const size_t blocks = static_cast<size_t>(p.items) * p.tiles;
  if (blocks > 0x7fffffffu) return W4A16_ERR_UNSUPPORTED;
  const dim3 g1(static_cast<unsigned>(blocks)), t1(p.waves * kWave);
  a.units = p.waves * kMdUnits;
  const size_t l1 = md_lds_bytes(p.waves), l2 = md_lds_bytes(p.dwaves);
  if (a.M <= 4)
    md_gate_up_kernel<kP, 1><<<g1, t1, l1, stream>>>(a);
  else
    md_gate_up_kernel<kP, 4 / kP><<<g1, t1, l1, stream>>>(a);
  const w4a16_status_t st = launch_status();
  if (st != W4A16_OK) return st;
  const dim3 g2(static_cast<unsigned>(p.dtiles * p.dsplits)), t2(p.dwaves * kWave);
  a.units = p.dwaves * kMdUnits;
  if (a.M <= 4)
    md_down_kernel<kP, 1><<<g2, t2, l2, stream>>>(a);
  else if (a.M <= 8)
    md_down_kernel<kP, 2><<<g2, t2, l2, stream>>>(a);
  else
    md_down_kernel<kP, 4 / kP><<<g2, t2, l2, stream>>>(a);
  return launch_status();
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
  if (static_cast<size_t>((gate->K + kMdCols - 1) / kMdCols) * sizeof(int) > kCounterBytes)
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
  a.cols = p.cols;
  a.tiles = p.tiles;
  a.parts = p.parts;
  a.gpp = p.gpp;
  a.dparts = p.dwaves / 4;
  a.dtiles = p.dtiles;
  a.dsplits = p.dsplits;
  a.h = reinterpret_cast<float*>(b + p.h_off);
  a.amax = reinterpret_cast<float*>(b + p.amax_off);
  a.partials = reinterpret_cast<float*>(b + p.partials_off);
  a.counters = reinterpret_cast<int*>(b);
  a.items = reinterpret_cast<MdItems*>(b + p.items_off);
  a.out_ids = topk_ids;
  a.out_w = topk_w;
  a.y = y;
  a.y_bf16 = yt == W4A16_BF16;
  return xt == W4A16_BF16 ? launch_md<1>(p, a, stream) : launch_md<2>(p, a, stream);
}
