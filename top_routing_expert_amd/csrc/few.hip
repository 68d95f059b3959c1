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
//  * Kernel 1 is the router's gate GEMM (route.hip), which also clears the
//    counters of kernel 2.
//  * Kernel 2: every block selects the experts of all tokens itself (a few
//    kilobytes of logits) and then takes work items from a ticket counter: first
//    the gate / up items (16 features of one chosen expert over all of k), then the
//    down items (16 output features over all chosen experts).  A down item waits
//    until every gate / up item is finished.  Gate / up items have the lower
//    tickets, so at that time each is finished or held by a block that runs and does
//    not wait: the wait ends whatever else occupies the GPU, without any
//    assumption about how many blocks are resident.
//  * An item's k range is split over the block's 8 waves and summed through LDS
//    in wave order.  MFMA 16x16x32 with 16 weight rows as A and the tokens as the
//    16 columns of B (column t = token t; tokens that did not choose the expert
//    are zero columns), so an expert's weights are read once for all its tokens
//    and the combine is a scaling of the columns before they are added.
//  * Weights are read as they were packed: the bf16 image of ffn_packed.hip (two
//    k-steps of 16 make the 32 k of one MFMA) or the MXFP4 image (16 rows x 128 k
//    chunks, decoded to bf16 in registers by v_cvt_scalef32_pk_bf16_fp4).
#include "mxfp4.h"
#include "topk.h"

namespace moe {

constexpr int kFewWaves = 8;
constexpr int kFewMaxPairs = kFewMaxTokens * 16;

struct FewArgs {
  const u32x4* x;         // [T, d] bf16
  const float* partial;   // [splits, T, E] router partials
  const float* bias;
  const char* gu;         // gate / up image
  const char* dn;         // down image
  size_t gu_expert, dn_expert;  // bytes of an expert's image
  size_t gu_codes, dn_codes;    // MXFP4: offset of the scales in it
  uint16_t* out;          // [T, d]
  float* logits;          // optional outputs
  int32_t* topk_idx;
  float* topk_w;
  uint16_t* h;            // [T k, f]
  uint32_t* ticket;       // counters[0]; counters[1 + e]: finished gate / up items of e
  uint32_t* done;
  int T, d, E, k, f, n_group, topk_group, presel, renorm, splits;
  int gu_steps, dn_steps;  // k-steps of 16 (bf16 image) or of 128
};

// One step of a weight stream: 32 k (bf16) or 128 k (MXFP4) of 16 or 32 rows and of
// the token columns.
template <bool MX, int NF, int NT>
struct FewStep {
  u32x4 w[NF];
  uint32_t s[NF];
  u32x4 b[NT][MX ? 4 : 1];
};

template <bool MX, int NF, int NT>
__device__ __forceinline__ void few_mfma(const FewStep<MX, NF, NT>& S, f32x4 (&acc)[NF][NT]) {
  if constexpr (!MX) {
#pragma unroll
    for (int i = 0; i < NF; ++i)
#pragma unroll
      for (int n = 0; n < NT; ++n)
        acc[i][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(S.w[i]),
                                                            as_bf16x8(S.b[n][0]), acc[i][n], 0, 0, 0);
  } else {
#pragma unroll
    for (int i = 0; i < NF; ++i) {
      const float s = mx_scale(S.s[i]);
#pragma unroll
      for (int q = 0; q < 4; ++q) {  // eight codes: k 8 q .. +7 of this lane's block
        u32x4 v;
        v.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(S.w[i][q], s, 0));
        v.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(S.w[i][q], s, 1));
        v.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(S.w[i][q], s, 2));
        v.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(S.w[i][q], s, 3));
#pragma unroll
        for (int n = 0; n < NT; ++n)
          acc[i][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(v), as_bf16x8(S.b[n][q]),
                                                              acc[i][n], 0, 0, 0);
      }
    }
  }
}

// Steps [s0, s1) of a stream through two register sets of U steps: the loads of
// one set are in flight while the other is consumed.  load(S, s) fills a step.
template <bool MX, int NF, int NT, int U, typename Load>
__device__ __forceinline__ void few_stream(int s0, int s1, Load&& load, f32x4 (&acc)[NF][NT]) {
  FewStep<MX, NF, NT> A[U], B[U];
  auto fill = [&](FewStep<MX, NF, NT>(&S)[U], int s) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (s + u < s1) load(S[u], s + u);
  };
  auto use = [&](FewStep<MX, NF, NT>(&S)[U], int s) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (s + u < s1) few_mfma<MX, NF, NT>(S[u], acc);
  };
  fill(A, s0);
  for (int s = s0; s < s1; s += 2 * U) {
    fill(B, s + U);
    use(A, s);
    fill(A, s + 2 * U);
    use(B, s + U);
  }
}

template <bool MX, int NT>
__global__ __launch_bounds__(64 * kFewWaves, 4) void few_layer_kernel(FewArgs a) {
  // steps per register set, gate / up and down: two sets fit 128 registers
  constexpr int UG = MX ? 1 : (NT == 1 ? 3 : 2);
  constexpr int UD = MX ? (NT == 1 ? 2 : 1) : (NT == 1 ? 5 : 3);
  constexpr int KS = MX ? 128 : 32;  // k of a step
  __shared__ int s_idx[kFewMaxPairs];
  __shared__ float s_w[kFewMaxPairs];
  __shared__ uint32_t s_mask[kMaxExperts / 32];
  __shared__ int s_exp[kFewMaxPairs];
  __shared__ int s_n, s_ticket;
  __shared__ f32x4 s_red[kFewWaves][2 * NT][64];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const bool first = blockIdx.x == 0;  // writes the routing outputs
  const int T = a.T, k = a.k;

  // ---- selection: every token's experts and gates, in LDS
  if (tid < kMaxExperts / 32) s_mask[tid] = 0u;
  auto select = [&](auto lpt_c, auto epl_c) {
    constexpr int LPT = decltype(lpt_c)::value, EPL = decltype(epl_c)::value;
    constexpr int TPW = 64 / LPT;
    for (int t0 = wave * TPW; t0 < T; t0 += kFewWaves * TPW) {
      const int t = t0 + lane / LPT, q = lane % LPT;
      int e;
      float w;
      select_token<LPT, EPL>(a.partial, a.splits, a.bias, first ? a.logits : nullptr, t, t < T, q, T,
                             a.E, k, a.n_group, a.topk_group, a.presel, a.renorm, &e, &w);
      if (t < T && q < k) {
        s_idx[t * k + q] = e;
        s_w[t * k + q] = w;
        if (first && a.topk_idx) a.topk_idx[t * k + q] = e;
        if (first && a.topk_w) a.topk_w[t * k + q] = w;
      }
    }
  };
  using std::integral_constant;
  if (a.E <= 64)
    select(integral_constant<int, 64>(), integral_constant<int, 1>());
  else if (a.E <= 256 && a.n_group <= 32)
    select(integral_constant<int, 32>(), integral_constant<int, 8>());
  else
    select(integral_constant<int, 64>(), integral_constant<int, kMaxEPL>());
  __syncthreads();
  // ---- the chosen experts in index order
  if (tid < T * k) atomicOr(&s_mask[s_idx[tid] >> 5], 1u << (s_idx[tid] & 31));
  __syncthreads();
  if (wave == 0) {
    const uint32_t m = lane < kMaxExperts / 32 ? s_mask[lane] : 0u;
    int incl = __popc(m);
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int y = __shfl_up(incl, o);
      if (lane >= o) incl += y;
    }
    int at = incl - __popc(m);
    for (uint32_t r = m; r; r &= r - 1) s_exp[at++] = 32 * lane + __ffs((int)r) - 1;
    if (lane == 63) s_n = incl;
  }
  __syncthreads();
  const int n_act = s_n;
  const int gu_items = a.f / 16, dn_items = a.d / 16;
  const int n_gu = n_act * gu_items, n_items = n_gu + dn_items;

  const int r16 = lane & 15, q4 = lane >> 4;
  // choice of expert e by this lane's token of column tile n, or -1
  auto choice = [&](int n, int e) {
    const int t = 16 * n + r16;
    int c = -1;
    if (t < T)
      for (int j = 0; j < k; ++j) c = s_idx[t * k + j] == e ? j : c;
    return c;
  };
  bool ready = false;  // every gate / up item is finished

  for (;;) {
    if (tid == 0) s_ticket = (int)atomicAdd(a.ticket, 1u);
    __syncthreads();  // also: s_red of the item before is read
    const int item = __builtin_amdgcn_readfirstlane(s_ticket);
    if (item >= n_items) break;  // block-uniform
    if (item < n_gu) {
      const int e = s_exp[item / gu_items], fb = item % gu_items;
      const char* gu = a.gu + (size_t)e * a.gu_expert;
      const int steps = a.d / KS;
      int c[NT];
      bool on[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        c[n] = choice(n, e);
        on[n] = c[n] >= 0;
      }
      f32x4 acc[2][NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) acc[0][n] = acc[1][n] = f32x4{0.f, 0.f, 0.f, 0.f};
      auto load = [&](FewStep<MX, 2, NT>& S, int s) {
        if constexpr (!MX) {
          const u32x4* p = reinterpret_cast<const u32x4*>(gu) +
                           (size_t)(fb / 2) * ((size_t)a.gu_steps * 128) +
                           ((size_t)(2 * s + (q4 >> 1)) * 2 + (fb & 1)) * 64 + (q4 & 1) * 32 + r16;
          S.w[0] = p[0];
          S.w[1] = p[16];
        } else {
          const size_t g = 2 * (size_t)fb;  // 16-row group of the gate rows
          const u32x4* p = reinterpret_cast<const u32x4*>(gu) + (g * a.gu_steps + s) * 64 +
                           r16 * 4 + (q4 ^ ((r16 >> 2) & 3));
          S.w[0] = p[0];
          S.w[1] = p[(size_t)a.gu_steps * 64];
          const char* q =
              gu + a.gu_codes + (((g / 4) * a.gu_steps + s) * 64 + (g % 4) * 16 + r16) * 4 + q4;
          S.s[0] = (uint8_t)q[0];
          S.s[1] = (uint8_t)q[64];
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < (MX ? 4 : 1); ++i) {
            S.b[n][i] = u32x4{0u, 0u, 0u, 0u};
            if (on[n])
              S.b[n][i] = a.x[(size_t)(16 * n + r16) * (a.d / 8) + s * (KS / 8) + q4 * (KS / 32) + i];
          }
      };
      few_stream<MX, 2, NT, UG>((int)((long)wave * steps / kFewWaves),
                               (int)((long)(wave + 1) * steps / kFewWaves), load, acc);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        s_red[wave][2 * n][lane] = acc[0][n];
        s_red[wave][2 * n + 1][lane] = acc[1][n];
      }
      __syncthreads();
      if (wave == 0) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          f32x4 g = s_red[0][2 * n][lane], u = s_red[0][2 * n + 1][lane];
#pragma unroll
          for (int w = 1; w < kFewWaves; ++w) {
            g += s_red[w][2 * n][lane];
            u += s_red[w][2 * n + 1][lane];
          }
          float hv[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            hv[i] = g[i] * __builtin_amdgcn_rcpf(1.0f + __expf(-g[i])) * u[i];
          if (on[n]) {  // rounded to bf16: the operand of the second product
            u32x2 pk;
            pk.x = pack_bf16x2(hv[0], hv[1]);
            pk.y = pack_bf16x2(hv[2], hv[3]);
            *reinterpret_cast<u32x2*>(a.h + (size_t)((16 * n + r16) * k + c[n]) * a.f + fb * 16 +
                                      4 * q4) = pk;
          }
        }
        __threadfence();  // the h values before the count
        if (lane == 0) atomicAdd(a.done + e, 1u);
      }
    } else {
      const int fb = item - n_gu;
      if (!ready) {
        for (int i = tid; i < n_act; i += 64 * kFewWaves)
          while (__hip_atomic_load(a.done + s_exp[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) <
                 (uint32_t)gu_items)
            __builtin_amdgcn_s_sleep(2);
        __syncthreads();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
        ready = true;
      }
      const int steps = a.f / KS;
      const int total = n_act * steps;
      const int s0 = (int)((long)wave * total / kFewWaves);
      const int s1 = (int)((long)(wave + 1) * total / kFewWaves);
      f32x4 sum[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) sum[n] = f32x4{0.f, 0.f, 0.f, 0.f};
      for (int s = s0; s < s1;) {  // the wave's part of one expert after the other
        const int ai = s / steps, e = s_exp[ai];
        const char* dn = a.dn + (size_t)e * a.dn_expert;
        const int b0 = s - ai * steps, b1 = min(steps, s1 - ai * steps);
        int c[NT];
        bool on[NT];
        const u32x4* hrow[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          c[n] = choice(n, e);
          on[n] = c[n] >= 0;
          hrow[n] = reinterpret_cast<const u32x4*>(a.h) +
                    (size_t)((16 * n + r16) * k + max(c[n], 0)) * (a.f / 8);
        }
        f32x4 acc[1][NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[0][n] = f32x4{0.f, 0.f, 0.f, 0.f};
        auto load = [&](FewStep<MX, 1, NT>& S, int st) {
          if constexpr (!MX) {
            S.w[0] = reinterpret_cast<const u32x4*>(
                dn)[(size_t)(fb / 4) * ((size_t)a.dn_steps * 128) +
                    ((size_t)(2 * st + (q4 >> 1)) * 2 + (fb % 4) / 2) * 64 + (q4 & 1) * 32 +
                    (fb & 1) * 16 + r16];
          } else {
            const size_t g = fb;
            S.w[0] = reinterpret_cast<const u32x4*>(
                dn)[(g * a.dn_steps + st) * 64 + r16 * 4 + (q4 ^ ((r16 >> 2) & 3))];
            S.s[0] = (uint8_t)dn[a.dn_codes +
                                 (((g / 4) * a.dn_steps + st) * 64 + (g % 4) * 16 + r16) * 4 + q4];
          }
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < (MX ? 4 : 1); ++i) {
              S.b[n][i] = u32x4{0u, 0u, 0u, 0u};
              if (on[n]) S.b[n][i] = hrow[n][st * (KS / 8) + q4 * (KS / 32) + i];
            }
        };
        few_stream<MX, 1, NT, UD>(b0, b1, load, acc);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float g = on[n] ? s_w[(16 * n + r16) * k + c[n]] : 0.f;
#pragma unroll
          for (int i = 0; i < 4; ++i) sum[n][i] = fmaf(g, acc[0][n][i], sum[n][i]);
        }
        s = ai * steps + b1;
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) s_red[wave][n][lane] = sum[n];
      __syncthreads();
      if (wave < NT) {
        f32x4 v = s_red[0][wave][lane];
#pragma unroll
        for (int w = 1; w < kFewWaves; ++w) v += s_red[w][wave][lane];
        const int t = 16 * wave + r16;
        if (t < T) {
          u32x2 pk;
          pk.x = pack_bf16x2(v[0], v[1]);
          pk.y = pack_bf16x2(v[2], v[3]);
          *reinterpret_cast<u32x2*>(a.out + (size_t)t * a.d + fb * 16 + 4 * q4) = pk;
        }
      }
    }
  }
}

// ws: counters | router partials | h
static size_t few_align(size_t b) { return (b + 255) & ~(size_t)255; }
static size_t few_counter_bytes(const moe_config& c) { return few_align(((size_t)c.E + 1) * 4); }
static size_t few_partial_bytes(const moe_config& c) {
  return few_align((size_t)router_splits(c) * c.T * c.E * sizeof(float));
}
size_t few_ws_bytes(const moe_config& c) {
  return c.T == 0 ? 0
                  : few_counter_bytes(c) + few_partial_bytes(c) +
                        few_align((size_t)c.T * c.k * c.f * 2);
}

hipError_t launch_layer_few(const moe_config& c, const void* x, const void* w_router,
                            const float* bias, const void* gate_up, const void* down, bool mx,
                            void* out, float* logits, int32_t* topk_idx, float* topk_w, void* ws,
                            hipStream_t st) {
  char* base = static_cast<char*>(ws);
  auto* counters = reinterpret_cast<uint32_t*>(base);
  auto* partial = reinterpret_cast<float*>(base + few_counter_bytes(c));
  FewArgs a{};
  a.x = static_cast<const u32x4*>(x);
  a.partial = partial;
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
  a.logits = logits;
  a.topk_idx = topk_idx;
  a.topk_w = topk_w;
  a.h = reinterpret_cast<uint16_t*>(base + few_counter_bytes(c) + few_partial_bytes(c));
  a.ticket = counters;
  a.done = counters + 1;
  a.T = c.T;
  a.d = c.d;
  a.E = c.E;
  a.k = c.k;
  a.f = c.f;
  a.n_group = c.n_group;
  a.topk_group = c.topk_group;
  a.presel = c.presel;
  a.renorm = c.renorm;
  a.splits = router_splits(c);
  hipError_t e = launch_router_gemm_bf16(static_cast<const uint16_t*>(x),
                                         static_cast<const uint16_t*>(w_router), partial, c.T, c.d,
                                         c.E, a.splits, st, counters, c.E + 1);
  if (e != hipSuccess) return e;
  // two blocks per CU; never more than the most items the layer can have
  const long items = (long)(c.T * c.k < c.E ? c.T * c.k : c.E) * (c.f / 16) + c.d / 16;
  const long cap = 2L * device_cus();
  const int blocks = (int)(items < cap ? items : cap);
  constexpr int threads = 64 * kFewWaves;
  if (c.T <= 16) {
    if (mx)
      few_layer_kernel<true, 1><<<blocks, threads, 0, st>>>(a);
    else
      few_layer_kernel<false, 1><<<blocks, threads, 0, st>>>(a);
  } else {
    if (mx)
      few_layer_kernel<true, 2><<<blocks, threads, 0, st>>>(a);
    else
      few_layer_kernel<false, 2><<<blocks, threads, 0, st>>>(a);
  }
  return hipGetLastError();
}

}  // namespace moe
