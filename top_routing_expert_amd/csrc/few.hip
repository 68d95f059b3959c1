// The whole MoE layer for a few tokens (decode, drafts checked at once) in two
// kernels.
//
//   z = x Wr^T, selection and gates as moe_route
//   h[t, j] = SiLU(x_t Wg_e^T) (x_t Wu_e^T),  e = the j-th expert of token t
//   out_t   = sum_j g[t, j] h[t, j] Wd_e^T
//
// With 1..32 tokens the layer is a stream of the chosen experts' weights, each
// read once, and latency: a launch per step and tiles of 128..256 features (the
// grouped GEMMs) leave most of the chip waiting.
//  * Kernel 1 computes the logits: a block of four experts, a wave for every k part of the
//    router's gate GEMM (route.hip), the parts added in LDS in the same order, so
//    the logits are the router's bit for bit.  It also clears the marks of kernel 2.
//  * Kernel 2: every block selects the experts of all tokens itself (a few
//    kilobytes of logits) and sorts the (token, choice) pairs by expert into tiles of
//    up to 16 pairs of one expert.  The gate / up work (feature groups of 16 features
//    of one tile) is cut into one equal share a block; the down work (16 output
//    features over all tiles or a part of them) follows.  Down items need all
//    of h, so a block waits there until every share is done.  A block marks its
//    share as begun when it starts, and before it waits it looks for shares that
//    nobody has begun and does them itself (twice the same values where both
//    do): whatever it then waits for is in the hands of a block that runs and does not
//    wait.  So the wait ends whatever else occupies the GPU, however few
//    blocks are resident.  Marks are bits of words in lines, and memory channels, of
//    their own: atomics on one channel take 10..16 ns each, which 512 blocks on one
//    ticket counter, or on marks side by side, waited 8 us for.
//  * MFMA 16x16x32 with 16 weight rows as A and the pairs of a tile as the
//    columns of B (a column without a pair computes something that is not
//    stored), so an expert's weights are read once for all its tokens (twice where more
//    than 16 chose it).  The (group, k) steps of up to 8 groups are split evenly over the
//    block's 8 waves; a group's parts are summed through LDS in wave order.
//  * A down item's waves share its (tile, k) steps evenly; every wave adds its
//    gate-scaled tile sums per token in LDS, the waves are added in order, and where
//    an item covers a part of the tiles the last block to finish adds the parts
//    in order: the combine costs no pass over memory and no order is left to chance.
//    Its first weights are loaded before the wait.
//  * Weights are read as they were packed: the bf16 image of ffn_packed.hip (two
//    k-steps of 16 make the 32 k of one MFMA) or the MXFP4 image (16 rows x 128 k
//    chunks, decoded to bf16 in registers by v_cvt_scalef32_pk_bf16_fp4).  x
//    and h are kept in LDS where they fit, so that the registers in flight hold
//    weights only.
//
// Measured (a pass, both kernels): T1-d7168-E256 top-8 f2048 134 us, 5.3 TB/s of weights: bound
// by HBM.  T1-d5120-E16 top-2 f1536 32 us for 95 MB: logits 5 us, selection 2 us, the hand-over of
// h 2..3 us, the rest the streams' first latencies and 3..4 TB/s.  T29-d2048-E64 top-2 f1408
// MXFP4 71 us for 178 MB: logits 6 us, selection and lists 9, gate / up 32, down 22, where neither
// all of x nor of h fits in LDS and a 16-row step decodes as long as it loads.
#include <algorithm>

#include "mxfp4.h"
#include "topk.h"

namespace moe {

constexpr int kFewWaves = 8;
constexpr int kFewThreads = 64 * kFewWaves;
constexpr int kFewMaxPairs = kFewMaxTokens * 16;
constexpr int kFewMaxBlocks = 1024;
constexpr int kFewWords = 32;   // words of marks (32 bits each: kFewMaxBlocks)
constexpr int kFewSpread = 64;  // words from one counter to the next
constexpr int kFewActBytes = 48 * 1024;  // LDS for x, later h (two blocks per CU)

struct FewArgs {
  const u32x4* x;         // [T, d] bf16
  const float* z;         // [T, E] logits
  const float* bias;
  const char* gu;         // gate / up image
  const char* dn;         // down image
  size_t gu_expert, dn_expert;  // bytes of an expert's image
  size_t gu_codes, dn_codes;    // MXFP4: offset of the scales in it
  uint16_t* out;          // [T, d]
  int32_t* topk_idx;      // optional outputs
  float* topk_w;
  uint16_t* h;            // [T k, f]
  float* part;            // [d / 16][dn_split][T][16] partial outputs (dn_split > 1)
  uint32_t* begun;        // marks of the shares: bit b / kFewWords of word b % kFewWords
  uint32_t* done;
  uint32_t* arrived;      // [d / 16] finished parts of an output group (dn_split > 1)
  int T, d, E, k, f, n_group, topk_group, presel, renorm;
  int gu_steps, dn_steps;  // k-steps of 16 (bf16 image) or of 128
  int dn_split;            // items per output group
};

// ------------------------------------------------------------------ logits
// Block: experts 4 blockIdx.x .. + 3 (A rows past them repeat the last one), wave s:
// the k chunks of split s.  The k order inside a 64-wide chunk is that of the
// router's two kernels: MFMA h of lane group g takes the 16-byte piece 2 g + h,
// with at most 16 experts 4 h + g.  NT: tiles of 16 tokens.
template <int NT>
__global__ __launch_bounds__(1024) void few_router_kernel(const u32x4* __restrict__ x,
                                                          const u32x4* __restrict__ wr,
                                                          float* __restrict__ z,
                                                          float* __restrict__ logits, int T, int d,
                                                          int E, int splits,
                                                          uint32_t* __restrict__ clear,
                                                          int n_clear) {
  __shared__ f32x4 red[kMaxSplits][NT][16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r16 = lane & 15, g = lane >> 4;
  for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < n_clear; i += gridDim.x * blockDim.x)
    clear[i] = 0u;
  const int nch = d / 64, nv = d / 8;
  const int c0 = (int)((long)wave * nch / splits), c1 = (int)((long)(wave + 1) * nch / splits);
  const int e0 = 4 * blockIdx.x;
  const u32x4* wrow = wr + (size_t)min(e0 + min(r16, 3), E - 1) * nv;
  const u32x4* xrow[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) xrow[n] = x + (size_t)min(16 * n + r16, T - 1) * nv;
  const int p0 = E > 16 ? 2 * g : g, p1 = E > 16 ? 2 * g + 1 : 4 + g;
  f32x4 acc[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) acc[n] = f32x4{0.f, 0.f, 0.f, 0.f};
  constexpr int U = 4;  // chunks in flight
  for (int c = c0; c < c1; c += U) {
    u32x4 w[U][2], b[U][NT][2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int at = min(c + u, c1 - 1) * 8;
      w[u][0] = wrow[at + p0];
      w[u][1] = wrow[at + p1];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        b[u][n][0] = xrow[n][at + p0];
        b[u][n][1] = xrow[n][at + p1];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (c + u >= c1) break;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          acc[n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(w[u][h]),
                                                           as_bf16x8(b[u][n][h]), acc[n], 0, 0, 0);
    }
  }
  // rows 0..3 (the block's experts) are registers 0..3 of lanes 0..15 (the tokens)
  if (g == 0)
#pragma unroll
    for (int n = 0; n < NT; ++n) red[wave][n][r16] = acc[n];
  __syncthreads();
  if ((int)threadIdx.x < 16 * NT) {
    const int t = threadIdx.x;
    f32x4 v = red[0][t >> 4][t & 15];
    for (int s = 1; s < splits; ++s) v += red[s][t >> 4][t & 15];
    if (t < T)
      for (int i = 0; i < 4; ++i)
        if (e0 + i < E) {
          z[(size_t)t * E + e0 + i] = v[i];
          if (logits) logits[(size_t)t * E + e0 + i] = v[i];
        }
  }
}

// Values that blocks on different XCDs hand to each other (h, partial outputs) are
// written and read with agent-scope accesses, which go past the XCDs' own L2
// caches, and counted after the writer's stores are complete.  Release and
// acquire fences instead would write back and invalidate whole caches: with a fence a wave
// and item the T29-E64 case took 430 us and the T1-E16 case 79 us.
__device__ __forceinline__ void few_publish(void* p, u32x2 v) {
  __hip_atomic_store(static_cast<unsigned long long*>(p),
                     (unsigned long long)v.x | ((unsigned long long)v.y << 32), __ATOMIC_RELAXED,
                     __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ u32x2 few_fetch8(const void* p) {
  const unsigned long long v = __hip_atomic_load(
      static_cast<const unsigned long long*>(p), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  return u32x2{(uint32_t)v, (uint32_t)(v >> 32)};
}
__device__ __forceinline__ u32x4 few_fetch(const u32x4* p) {
  const u32x2 a = few_fetch8(p), b = few_fetch8(reinterpret_cast<const u32x2*>(p) + 1);
  return u32x4{a.x, a.y, b.x, b.y};
}
// All of this wave's stores have reached the point where every XCD sees them.
__device__ __forceinline__ void few_stores_done() {
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

// The weights of one step: 32 k (bf16) or 128 k (MXFP4) of 16 rows (NF = 2: and
// of the 16 rows that go with them); BR: the step's B operand, where it is not in LDS.
template <bool MX, int NF, bool BR>
struct FewStep {
  u32x4 w[NF];
  uint32_t s[MX ? NF : 1];
  u32x4 b[BR ? (MX ? 4 : 1) : 1];
};

template <bool MX, int NF>
__device__ __forceinline__ void few_mfma(const u32x4 (&w)[NF], const uint32_t (&sb)[MX ? NF : 1],
                                         const u32x4 (&b)[MX ? 4 : 1], f32x4 (&acc)[NF]) {
  if constexpr (!MX) {
#pragma unroll
    for (int i = 0; i < NF; ++i)
      acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(w[i]), as_bf16x8(b[0]), acc[i], 0,
                                                       0, 0);
  } else {
#pragma unroll
    for (int i = 0; i < NF; ++i) {
      const float s = mx_scale(sb[i]);
#pragma unroll
      for (int q = 0; q < 4; ++q) {  // eight codes: k 8 q .. +7 of this lane's block
        u32x4 v;
        v.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[i][q], s, 0));
        v.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[i][q], s, 1));
        v.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[i][q], s, 2));
        v.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[i][q], s, 3));
        acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(v), as_bf16x8(b[q]), acc[i], 0,
                                                         0, 0);
      }
    }
  }
}

// A wave's steps [s0, s0 + n) of a sequence of rows of `steps` steps each, cut at the
// rows' ends: the current row, the step in it and where the wave's part of it ends.
struct FewCursor {
  int row, step, end, left, steps;  // left: steps of the range from `step` on
  __device__ FewCursor(int s0, int n, int steps_)
      : row(s0 / steps_), step(s0 - s0 / steps_ * steps_), left(n), steps(steps_) {
    end = min(steps, step + left);
  }
  // U steps on, or to the next row; false: the range is done
  __device__ bool next(int U) {
    if (step + U < end) {
      step += U;
      left -= U;
      return true;
    }
    if (left <= end - step) return false;
    left -= end - step;
    ++row;
    step = 0;
    end = min(steps, left);
    return true;
  }
};

// The steps of a range through two register sets of U: one set's loads are in
// flight while the other is consumed.  A set never crosses a row's end.
// load(S, cursor, u) loads its step u: past the row's end the last one again, and past the
// range's end the last set again -- a load under a condition would make the
// waits for the loads before it drain everything in flight.  seek(cursor) sets
// the loader on a row, between() runs once after the first two sets' weights are
// on their way, use(S, step) consumes a step, done(row, begin) ends the wave's part of a
// row.
template <int U, typename Step, typename Seek, typename LoadW, typename LoadB, typename Between,
          typename Use, typename Done>
__device__ __forceinline__ void few_stream(int s0, int n, int steps, Seek&& seek, LoadW&& load_w,
                                           LoadB&& load_b, Between&& between, Use&& use,
                                           Done&& done) {
  Step A[U], B[U];
  FewCursor ld(s0, n, steps), c(s0, n, steps);
  const auto move = [&] {
    const int row = ld.row;
    ld.next(U);
    if (ld.row != row) seek(ld.row);
  };
  auto fill_w = [&](Step(&S)[U]) {
#pragma unroll
    for (int u = 0; u < U; ++u) load_w(S[u], min(ld.step + u, ld.end - 1));
  };
  auto fill_b = [&](Step(&S)[U], const FewCursor& at) {
#pragma unroll
    for (int u = 0; u < U; ++u) load_b(S[u], at.row, min(at.step + u, at.end - 1));
  };
  auto eat = [&](Step(&S)[U]) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (c.step + u < c.end) use(S[u], c.step + u);
    const int row = c.row;
    const bool more = c.next(U);
    if (!more || c.row != row) done(row);
    return more;
  };
  FewCursor first(s0, n, steps);
  if (n > 0) {
    seek(ld.row);
    fill_w(A);
    move();
    fill_w(B);
  }
  between();
  if (n <= 0) return;
  fill_b(A, first);
  fill_b(B, ld);
  move();
  for (;;) {
    if (!eat(A)) break;
    fill_w(A);
    fill_b(A, ld);
    move();
    if (!eat(B)) break;
    fill_w(B);
    fill_b(B, ld);
    move();
  }
}

template <bool MX>
__global__ __launch_bounds__(kFewThreads, 4) void few_layer_kernel(FewArgs a) {
  constexpr int KS = MX ? 128 : 32;  // k of a step
  constexpr int NB = MX ? 4 : 1;     // 16-byte B pieces of a lane and step
  __shared__ int s_idx[kFewMaxPairs];
  __shared__ float s_w[kFewMaxPairs];
  __shared__ int s_pair[kFewMaxPairs];       // pairs sorted by expert
  __shared__ int s_tok[kFewMaxPairs];        // and their tokens
  __shared__ int s_head[kFewMaxPairs];       // expert of a sorted pair, -1 - e at a tile's first
  __shared__ int s_start[kFewMaxPairs + 1];  // first sorted pair of tile v
  __shared__ int s_exp[kFewMaxPairs];        // expert of tile v
  __shared__ int s_n, s_old;
  __shared__ f32x4 s_red[kFewWaves][2][64];  // gate / up sums; per-token sums of the down items
  __shared__ __attribute__((aligned(16))) unsigned char s_act[kFewActBytes];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const bool first = blockIdx.x == 0;  // writes the routing outputs
  const int T = a.T, k = a.k, pairs = T * k;
  const int G = (int)gridDim.x;
  auto mark = [&](uint32_t* words, int b) {
    return atomicOr(words + b % kFewWords * kFewSpread, 1u << (b / kFewWords));
  };
  // word `lane` of the marks (all of them in one wave), and that word with all shares
  auto marks = [&](const uint32_t* words) {
    return lane < kFewWords ? __hip_atomic_load(words + lane * kFewSpread, __ATOMIC_RELAXED,
                                                __HIP_MEMORY_SCOPE_AGENT)
                            : 0u;
  };
  const int bits = lane < kFewWords ? (G - lane + kFewWords - 1) / kFewWords : 0;
  const uint32_t every = bits >= 32 ? ~0u : (1u << bits) - 1u;
  if (tid == kFewThreads - 1) (void)mark(a.begun, blockIdx.x);

  // ---- x in LDS where it fits; rows padded by 16 bytes against bank conflicts
  const int xs = a.d * 2 + 16;
  const bool x_lds = T * xs <= kFewActBytes;
  if (x_lds)
    for (int t = 0; t < T; ++t)
      for (int i = tid; i < a.d / 8; i += kFewThreads)
        *reinterpret_cast<u32x4*>(s_act + t * xs + i * 16) = a.x[(size_t)t * (a.d / 8) + i];

  // ---- selection: every token's experts and gates, in LDS, by the lane groups of
  // the router's top-k kernel (the same sums bit for bit)
  auto select = [&](auto lpt_c, auto epl_c) {
    constexpr int LPT = decltype(lpt_c)::value, EPL = decltype(epl_c)::value;
    constexpr int TPW = 64 / LPT;
    for (int t0 = wave * TPW; t0 < T; t0 += kFewWaves * TPW) {
      const int t = t0 + lane / LPT, q = lane % LPT;
      int e;
      float w;
      select_token<LPT, EPL>([&](int i) { return a.z[(size_t)t * a.E + i]; }, a.bias, t < T, q, a.E,
                             k, a.n_group, a.topk_group, a.presel, a.renorm, &e, &w);
      if (t < T && q < k) {
        const int p = t * k + q;
        s_idx[p] = e;
        s_w[p] = w;
        if (first && a.topk_idx) a.topk_idx[p] = e;
        if (first && a.topk_w) a.topk_w[p] = w;
      }
    }
  };
  using std::integral_constant;
  // With more tokens than waves, four tokens a wave where 16 lanes hold a token's choices and
  // its gate sum: the lanes that are missing would add zeros, so the gates stay those of the
  // wider groups (29 tokens of 64 experts: four rounds -> one, the layer 78 -> 74 us)
  if (a.E <= 64 && T > kFewWaves && max(a.presel, k) <= 16 && a.n_group <= 16 &&
      (a.renorm || a.presel))
    select(integral_constant<int, 16>(), integral_constant<int, 4>());
  else if (a.E <= 64)
    select(integral_constant<int, 64>(), integral_constant<int, 1>());
  else if (a.E <= 256 && a.n_group <= 32)
    select(integral_constant<int, 32>(), integral_constant<int, 8>());
  else
    select(integral_constant<int, 64>(), integral_constant<int, kMaxEPL>());
  __syncthreads();
  // ---- pairs sorted by (expert, token), cut into tiles of 16 pairs of one expert
  if (tid < pairs) {
    const int e = s_idx[tid];
    int pos = 0, rank = 0;
    for (int q = 0; q < pairs; ++q) {
      const int o = s_idx[q];
      pos += o < e || (o == e && q < tid);
      rank += o == e && q < tid;
    }
    s_pair[pos] = tid;
    s_tok[pos] = tid / k;
    s_head[pos] = rank % 16 == 0 ? -1 - e : e;
  }
  __syncthreads();
  if (wave == 0) {
    int n = 0;
    for (int p0 = 0; p0 < pairs; p0 += 64) {
      const int p = p0 + lane;
      const int hd = p < pairs ? s_head[p] : 0;
      const unsigned long long m = __ballot(hd < 0);
      if (hd < 0) {
        const int v = n + __popcll(m & ((1ull << lane) - 1));
        s_start[v] = p;
        s_exp[v] = -1 - hd;
      }
      n += __popcll(m);
    }
    if (lane == 0) {
      s_start[n] = pairs;
      s_n = n;
    }
  }
  __syncthreads();
  const int tiles = __builtin_amdgcn_readfirstlane(s_n);
  const int gu_groups = a.f / 16, dn_groups = a.d / 16;
  const int groups = tiles * gu_groups;
  const int r16 = lane & 15, q4 = lane >> 4;
  // column r16 of tile v: whether there is a pair, which, and its token (without
  // one, those of the tile's first column)
  auto column = [&](int v, int* p, int* t) {
    const int pos = s_start[v] + r16;
    const bool in = pos < s_start[v + 1];
    *p = s_pair[in ? pos : s_start[v]];
    *t = s_tok[in ? pos : s_start[v]];
    return in;
  };

  // ---- gate / up: share b = groups [g0, g1), one each for the first blocks where
  // there are fewer groups than blocks
  auto gate_up_share = [&](int b) {
    const int each = groups / G, more = groups - each * G;
    const int g0 = b * each + min(b, more), g1 = g0 + each + (b < more ? 1 : 0);
    const int steps = a.d / KS;
    for (int gb = g0; gb < g1; gb += kFewWaves) {
      const int total = min(kFewWaves, g1 - gb) * steps;
      // this wave's steps: at most `steps` of them, so at most the rest of one
      // group (its sum goes to LDS) and then the start of another (its sum stays here)
      const int s0 = wave * total / kFewWaves, n = (wave + 1) * total / kFewWaves - s0;
      const int row0 = s0 / steps, own = s0 == row0 * steps ? row0 : row0 + 1;
      const bool owns = n > 0 && s0 + n > own * steps;
      const u32x4* wp = nullptr;
      const char* sp = nullptr;
      const size_t wup = MX ? (size_t)a.gu_steps * 64 : 16;  // from gate to up rows
      auto seek = [&](int row) {
        const int v = (gb + row) / gu_groups, fb = gb + row - v * gu_groups;
        const int e = __builtin_amdgcn_readfirstlane(s_exp[v]);
        const char* gu = a.gu + (size_t)e * a.gu_expert;
        if constexpr (!MX) {
          wp = reinterpret_cast<const u32x4*>(gu) + (size_t)(fb / 2) * ((size_t)a.gu_steps * 128) +
               ((size_t)(q4 >> 1) * 2 + (fb & 1)) * 64 + (q4 & 1) * 32 + r16;
        } else {
          const size_t g = 2 * (size_t)fb;  // 16-row group of the gate rows
          wp = reinterpret_cast<const u32x4*>(gu) + g * a.gu_steps * 64 + r16 * 4 +
               (q4 ^ ((r16 >> 2) & 3));
          sp = gu + a.gu_codes + ((g / 4) * a.gu_steps * 64 + (g % 4) * 16 + r16) * 4 + q4;
        }
      };
      auto load_w = [&](auto& S, int step) {
        const u32x4* p = wp + (size_t)step * (MX ? 64 : 256);
        S.w[0] = __builtin_nontemporal_load(p);
        S.w[1] = __builtin_nontemporal_load(p + wup);
        if constexpr (MX) {
          const char* q = sp + (size_t)step * 256;
          S.s[0] = (uint8_t)q[0];
          S.s[1] = (uint8_t)q[64];
        }
      };
      f32x4 acc[2] = {f32x4{0.f, 0.f, 0.f, 0.f}, f32x4{0.f, 0.f, 0.f, 0.f}};
      int pair = 0, row = 0;  // this lane's pair and the LDS offset of its token's x
      bool on = false;
      auto enter = [&](int r) {
        int t;
        on = column((gb + r) / gu_groups, &pair, &t);
        row = t * xs + q4 * NB * 16;
      };
      if (n > 0) enter(row0);
      auto done = [&](int r) {
        if (r == own) return;
        s_red[wave][0][lane] = acc[0];
        s_red[wave][1][lane] = acc[1];
        acc[0] = acc[1] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (owns) enter(own);
      };
      auto nothing = [] {};
      if (x_lds) {
        using Step = FewStep<MX, 2, false>;
        few_stream<MX ? 3 : 4, Step>(
            s0, n, steps, seek, load_w, [](Step&, int, int) {}, nothing,
            [&](Step& S, int step) {
              const unsigned char* bp = s_act + row + step * (KS * 2);
              u32x4 b[NB];
#pragma unroll
              for (int i = 0; i < NB; ++i) b[i] = *reinterpret_cast<const u32x4*>(bp + 16 * i);
              few_mfma<MX, 2>(S.w, S.s, b, acc);
            },
            done);
      } else {
        using Step = FewStep<MX, 2, true>;
        few_stream<MX ? 1 : 3, Step>(
            s0, n, steps, seek, load_w,
            [&](Step& S, int r, int step) {
              int p, t;
              column((gb + r) / gu_groups, &p, &t);
              const u32x4* bp = a.x + (size_t)t * (a.d / 8) + step * (KS / 8) + q4 * NB;
#pragma unroll
              for (int i = 0; i < NB; ++i) S.b[i] = bp[i];
            },
            nothing, [&](Step& S, int) { few_mfma<MX, 2>(S.w, S.s, S.b, acc); }, done);
      }
      __syncthreads();
      if (owns) {
        f32x4 g = acc[0], u = acc[1];
        for (int w = wave + 1; w < kFewWaves; ++w) {  // waves that begin inside this group
          const int w0 = w * total / kFewWaves;
          if (w0 >= (own + 1) * steps) break;
          if ((w + 1) * total / kFewWaves == w0) continue;
          g += s_red[w][0][lane];
          u += s_red[w][1][lane];
        }
        float hv[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          hv[i] = g[i] * __builtin_amdgcn_rcpf(1.0f + __expf(-g[i])) * u[i];
        if (on) {  // rounded to bf16: the operand of the second product
          u32x2 pk;
          pk.x = pack_bf16x2(hv[0], hv[1]);
          pk.y = pack_bf16x2(hv[2], hv[3]);
          few_publish(a.h + (size_t)pair * a.f + (gb + own) % gu_groups * 16 + 4 * q4, pk);
        }
      }
      __syncthreads();  // s_red is free again
    }
    few_stores_done();  // h before the mark
    __syncthreads();
    if (tid == 0) (void)mark(a.done, b);
  };
  // Its own share, then any that nobody has begun.
  uint32_t seen = wave == 0 ? marks(a.begun) : 0u;  // looked at after the share
  for (int b = (int)blockIdx.x;;) {
    if (b >= 0) gate_up_share(b);
    if (__syncthreads_and(wave != 0 || seen == every)) break;
    if (wave == 0) {
      seen = marks(a.begun);
      int open = seen == every ? G : lane + kFewWords * (__ffs((int)(~seen & every)) - 1);
#pragma unroll
      for (int o = 32; o > 0; o >>= 1) open = min(open, __shfl_xor(open, o));
      if (lane == 0)  // another block may be faster
        s_old = open < G && !(mark(a.begun, open) >> (open / kFewWords) & 1u) ? open : -1;
    }
    __syncthreads();
    b = s_old;
  }

  // ---- down
  const int hs = a.f * 2 + 16;
  const bool h_lds = (long)pairs * hs <= kFewActBytes;
  bool ready = false;  // every share is done (and h is in LDS where it fits)
  // the first items to the blocks without a gate / up share
  for (int item = (int)blockIdx.x - (groups < G ? groups : 0); item < dn_groups * a.dn_split;
       item += G) {
    if (item < 0) continue;
    __syncthreads();  // s_red of the item before is read
    const int og = item / a.dn_split, sub = item - og * a.dn_split;
    const int steps = a.f / KS;
    const uint32_t total = (uint32_t)tiles * steps;  // < 2^26: T k f < 2^31
    const uint32_t parts = kFewWaves * a.dn_split, pi = sub * kFewWaves + wave;  // <= 64
    const int s0 = (int)(pi * total / parts), n = (int)((pi + 1) * total / parts) - s0;
    // per-token sums of this wave: [T][16] floats in its share of s_red
    float* sum = reinterpret_cast<float*>(&s_red[wave][0][0]);
    for (int i = lane; i < T * 16; i += 64) sum[i] = 0.f;
    const u32x4* wp = nullptr;
    const char* sp = nullptr;
    auto seek = [&](int v) {
      const int e = __builtin_amdgcn_readfirstlane(s_exp[v]);
      const char* dn = a.dn + (size_t)e * a.dn_expert;
      if constexpr (!MX) {
        wp = reinterpret_cast<const u32x4*>(dn) + (size_t)(og / 4) * ((size_t)a.dn_steps * 128) +
             ((size_t)(q4 >> 1) * 2 + (og % 4) / 2) * 64 + (q4 & 1) * 32 + (og & 1) * 16 + r16;
      } else {
        const size_t g = og;
        wp = reinterpret_cast<const u32x4*>(dn) + g * a.dn_steps * 64 + r16 * 4 +
             (q4 ^ ((r16 >> 2) & 3));
        sp = dn + a.dn_codes + ((g / 4) * a.dn_steps * 64 + (g % 4) * 16 + r16) * 4 + q4;
      }
    };
    auto load_w = [&](auto& S, int step) {
      S.w[0] = __builtin_nontemporal_load(wp + (size_t)step * (MX ? 64 : 256));
      if constexpr (MX) S.s[0] = (uint8_t)sp[(size_t)step * 256];
    };
    auto wait = [&] {
      if (ready) return;
      if (wave == 0)
        while (!__all(marks(a.done) == every)) __builtin_amdgcn_s_sleep(4);
      // h by ordinary loads, a row once per XCD (29 tokens, 58 rows of 2816 bytes: 88 -> 78
      // us); where it is copied to LDS once a block, going around the caches costs less
      // than emptying them (one token: 30 against 33 us)
      if (wave == 0 && !h_lds) __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
      __syncthreads();
      if (h_lds) {
        const int nv = a.f / 8;
        const u32x4* hv = reinterpret_cast<const u32x4*>(a.h);
        for (int p = 0; p < pairs; ++p)
          for (int i = tid; i < nv; i += kFewThreads)
            *reinterpret_cast<u32x4*>(s_act + p * hs + i * 16) = few_fetch(hv + (size_t)p * nv + i);
        __syncthreads();
      }
      ready = true;
    };
    f32x4 acc[1] = {f32x4{0.f, 0.f, 0.f, 0.f}};
    int pair = 0, tok = 0;
    bool on = false;
    if (n > 0) on = column(s0 / steps, &pair, &tok);
    auto done = [&](int v) {  // a tile's columns are different tokens
      if (on) {
        const float g = s_w[pair];
        f32x4* o = reinterpret_cast<f32x4*>(sum + tok * 16 + 4 * q4);
        *o += g * acc[0];
      }
      acc[0] = f32x4{0.f, 0.f, 0.f, 0.f};
      if (v + 1 < tiles) on = column(v + 1, &pair, &tok);
    };
    if (h_lds) {
      using Step = FewStep<MX, 1, false>;
      few_stream<MX ? 4 : 8, Step>(
          s0, n, steps, seek, load_w, [](Step&, int, int) {}, wait,
          [&](Step& S, int step) {
            const unsigned char* bp = s_act + pair * hs + (step * (KS / 8) + q4 * NB) * 16;
            u32x4 b[NB];
#pragma unroll
            for (int i = 0; i < NB; ++i) b[i] = *reinterpret_cast<const u32x4*>(bp + 16 * i);
            few_mfma<MX, 1>(S.w, S.s, b, acc);
          },
          done);
    } else {
      const u32x4* hv = reinterpret_cast<const u32x4*>(a.h);
      using Step = FewStep<MX, 1, true>;
      few_stream<MX ? 1 : 4, Step>(
          s0, n, steps, seek, load_w,
          [&](Step& S, int v, int step) {
            int p, t;
            column(v, &p, &t);
#pragma unroll
            for (int i = 0; i < NB; ++i)
              S.b[i] = hv[(size_t)p * (a.f / 8) + step * (KS / 8) + q4 * NB + i];
          },
          wait, [&](Step& S, int) { few_mfma<MX, 1>(S.w, S.s, S.b, acc); }, done);
    }
    __syncthreads();
    // four features of one token per thread: the waves in order
    const int t = tid >> 2, i4 = tid & 3;
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
    if (tid < 4 * T) {
#pragma unroll
      for (int w = 0; w < kFewWaves; ++w) v += (&s_red[w][0][0])[tid];
    }
    if (a.dn_split > 1) {
      f32x4* pp = reinterpret_cast<f32x4*>(a.part) + (size_t)og * a.dn_split * 4 * T;
      if (tid < 4 * T) {
        u32x2* o = reinterpret_cast<u32x2*>(pp + (size_t)sub * 4 * T + tid);
        const u32x4 w = __builtin_bit_cast(u32x4, v);
        few_publish(o, u32x2{w.x, w.y});
        few_publish(o + 1, u32x2{w.z, w.w});
        few_stores_done();
      }
      __syncthreads();
      if (tid == 0) s_old = (int)atomicAdd(a.arrived + og * kFewSpread, 1u);
      __syncthreads();
      const int old = s_old;
      __syncthreads();
      if (old != a.dn_split - 1) continue;  // block-uniform: another block adds the parts
      if (tid < 4 * T) {
        auto part = [&](int q) {
          return __builtin_bit_cast(
              f32x4, few_fetch(reinterpret_cast<const u32x4*>(pp + (size_t)q * 4 * T + tid)));
        };
        v = part(0);
        for (int q = 1; q < a.dn_split; ++q) v += part(q);
      }
    }
    if (tid < 4 * T) {
      u32x2 pk;
      pk.x = pack_bf16x2(v[0], v[1]);
      pk.y = pack_bf16x2(v[2], v[3]);
      *reinterpret_cast<u32x2*>(a.out + (size_t)t * a.d + og * 16 + 4 * i4) = pk;
    }
  }
}

// Two blocks per CU; never more than the most items the layer can have.
static int few_blocks(const moe_config& c) {
  const long pairs = (long)c.T * c.k;
  const long items = pairs * (c.f / 16) + c.d / 16;
  const long cap = std::min(2L * device_cus(), (long)kFewMaxBlocks);
  return (int)(items < cap ? items : cap);
}
// Down items per group of 16 output features: enough for every block to have one.
static int few_dn_split(const moe_config& c) {
  const int s = few_blocks(c) / (c.d / 16);
  return s < 1 ? 1 : s > 8 ? 8 : s;
}

// ws: counters | logits | h | partial outputs
static size_t few_align(size_t b) { return (b + 255) & ~(size_t)255; }
// counters: begun | done | arrived parts
static int few_counters(const moe_config& c, int dn_split) {
  return (2 * kFewWords + (dn_split > 1 ? c.d / 16 : 0)) * kFewSpread;
}
static size_t few_counter_bytes(const moe_config& c) {
  return few_align((size_t)few_counters(c, 2) * 4);
}
static size_t few_logit_bytes(const moe_config& c) {
  return few_align((size_t)c.T * c.E * sizeof(float));
}
static size_t few_h_bytes(const moe_config& c) { return few_align((size_t)c.T * c.k * c.f * 2); }
size_t few_ws_bytes(const moe_config& c) {
  return c.T == 0 ? 0
                  : few_counter_bytes(c) + few_logit_bytes(c) + few_h_bytes(c) +
                        few_align((size_t)8 * c.T * c.d * sizeof(float));
}

hipError_t launch_layer_few(const moe_config& c, const void* x, const void* w_router,
                            const float* bias, const void* gate_up, const void* down, bool mx,
                            void* out, float* logits, int32_t* topk_idx, float* topk_w, void* ws,
                            hipStream_t st) {
  char* base = static_cast<char*>(ws);
  auto* counters = reinterpret_cast<uint32_t*>(base);
  auto* z = reinterpret_cast<float*>(base + few_counter_bytes(c));
  FewArgs a{};
  a.x = static_cast<const u32x4*>(x);
  a.z = z;
  a.bias = bias;
  a.gu = static_cast<const char*>(gate_up);
  a.dn = static_cast<const char*>(down);
  if (mx) {
    const MxGeom gg = mx_geom(c, true), gd = mx_geom(c, false);
    a.gu_expert = gg.expert_bytes;
    a.gu_codes = gg.codes_bytes;
    a.gu_steps = gg.steps;
    a.dn_expert = gd.expert_bytes;
    a.dn_codes = gd.codes_bytes;
    a.dn_steps = gd.steps;
  } else {
    const PackGeom gg = pack_geom(c.f, c.d, true), gd = pack_geom(c.d, c.f, false);
    a.gu_expert = gg.expert_elems * 2;
    a.gu_steps = gg.kp / 16;
    a.dn_expert = gd.expert_elems * 2;
    a.dn_steps = gd.kp / 16;
  }
  a.out = static_cast<uint16_t*>(out);
  a.topk_idx = topk_idx;
  a.topk_w = topk_w;
  char* hp = base + few_counter_bytes(c) + few_logit_bytes(c);
  a.h = reinterpret_cast<uint16_t*>(hp);
  a.part = reinterpret_cast<float*>(hp + few_h_bytes(c));
  a.begun = counters;
  a.done = a.begun + kFewWords * kFewSpread;
  a.arrived = a.done + kFewWords * kFewSpread;
  a.T = c.T;
  a.d = c.d;
  a.E = c.E;
  a.k = c.k;
  a.f = c.f;
  a.n_group = c.n_group;
  a.topk_group = c.topk_group;
  a.presel = c.presel;
  a.renorm = c.renorm;
  a.dn_split = few_dn_split(c);
  const int splits = router_splits(c), n_clear = few_counters(c, a.dn_split);
  const auto* wv = static_cast<const u32x4*>(w_router);
  if (c.T <= 16)
    few_router_kernel<1><<<div_up(c.E, 4), 64 * splits, 0, st>>>(a.x, wv, z, logits, c.T, c.d, c.E,
                                                                 splits, counters, n_clear);
  else
    few_router_kernel<2><<<div_up(c.E, 4), 64 * splits, 0, st>>>(a.x, wv, z, logits, c.T, c.d, c.E,
                                                                 splits, counters, n_clear);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (mx)
    few_layer_kernel<true><<<few_blocks(c), kFewThreads, 0, st>>>(a);
  else
    few_layer_kernel<false><<<few_blocks(c), kFewThreads, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace moe
