// Selection and gates of one token by a group of LPT lanes (used by the router's
// top-k kernel and by the few-token layer, so both choose alike).
#pragma once

#include "common.h"

namespace moe {

constexpr int kMaxSplits = 16;  // split-K partials of the router GEMM (summed by top-k)

// Maximum over each segment of LPT lanes, in every lane of it: moves within 16
// lanes (quad permutes, mirrors), then swaps of 16- and 32-lane halves.  A
// shuffle through LDS instead takes several times as long a step, and the
// selection rounds are one chain of these.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t v) {
  const uint32_t w = (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, CTRL, 0xf, 0xf, false);
  return w > v ? w : v;
}
template <int LPT>
__device__ __forceinline__ uint32_t seg_max_u32(uint32_t v) {
  if constexpr (LPT >= 2) v = dpp_max<0xB1>(v);    // lanes 1 0 3 2 of a quad
  if constexpr (LPT >= 4) v = dpp_max<0x4E>(v);    // lanes 2 3 0 1 of a quad
  if constexpr (LPT >= 8) v = dpp_max<0x141>(v);   // mirrored within 8
  if constexpr (LPT >= 16) v = dpp_max<0x140>(v);  // mirrored within 16
  if constexpr (LPT >= 32) {
    const auto p = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = p[0] > p[1] ? p[0] : p[1];
  }
  if constexpr (LPT >= 64) {
    const auto p = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    v = p[0] > p[1] ? p[0] : p[1];
  }
  return v;
}

template <int LPT>
__device__ __forceinline__ float seg_sum(float v) {
#pragma unroll
  for (int o = LPT / 2; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

__device__ __forceinline__ float ord_key_inv(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

constexpr int kMaxEPL = 16;  // E <= 1024 with 64 lanes per token

// Sum of the router's partial logits of one expert, in split order; every
// partial is loaded before the first add (one memory latency).
__device__ __forceinline__ float sum_partials(const float* __restrict__ partial, int splits,
                                              size_t stride, size_t at) {
  float pv[kMaxSplits];
#pragma unroll
  for (int s = 0; s < kMaxSplits; ++s) pv[s] = s < splits ? partial[s * stride + at] : 0.f;
  float z = pv[0];
#pragma unroll
  for (int s = 1; s < kMaxSplits; ++s)
    if (s < splits) z += pv[s];
  return z;
}

// Lane q = lane % LPT of a token's group (`live`: there is a token; a group
// without one runs along); logit(e) gives its logits.  EPL: scores per lane
// (ceil(E / LPT): 1 for E <= 64), so the code holds only the loops a layer of this
// size needs.  The j-th best expert and its gate end up in lane q == j of the
// group (*out_e, *out_w).
template <int LPT, int EPL, typename Logit>
__device__ __forceinline__ void select_token(Logit&& logit, const float* __restrict__ bias,
                                             bool live, int q, int E, int k, int n_group,
                                             int topk_group, int presel, int renorm, int* out_e,
                                             float* out_w) {
  const int epl = (E + LPT - 1) / LPT;

  // scores s = z + b (one fp32 add), -0 -> +0; key32 = order-preserving bits, at
  // least 1 (0: no candidate; only a NaN pattern would have it)
  uint32_t key[EPL];
  uint32_t open = 0u;  // bit i: expert q + i LPT may still be chosen
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    key[i] = 0u;
    const int e = q + i * LPT;
    if (i < epl && e < E) open |= 1u << i;
    if (i < epl && e < E && live) {
      const float z = logit(e);
      float sc = bias ? __fadd_rn(z, bias[e]) : z;
      uint32_t u = __float_as_uint(sc);
      if (u == 0x80000000u) u = 0u;
      key[i] = max(ord_key(__uint_as_float(u)), 1u);
    }
  }

  // group-limited eligibility: keep the topk_group groups with the largest max
  if (n_group > 1 && topk_group < n_group) {
    // e / gsz by a multiplication: exact for e, gsz <= 1024 (1023^2 < 2^20)
    const uint32_t gsz = E / n_group, inv = ((1u << 20) + gsz - 1) / gsz;
    int grp[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) grp[i] = (int)((uint32_t)(q + i * LPT) * inv >> 20);
    uint32_t my_g = 0u;  // lane g: the maximum of group g
    for (int g = 0; g < n_group; ++g) {
      uint32_t m = 0u;
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (grp[i] == g) m = max(m, key[i]);
      m = seg_max_u32<LPT>(m);
      if (q == g) my_g = m;
    }
    unsigned long long kept = 0ull;
    for (int r = 0; r < topk_group; ++r) {
      // the best open group, the lowest of equal ones
      const bool left = q < n_group && !((kept >> q) & 1ull);
      const uint32_t m = seg_max_u32<LPT>(left ? my_g : 0u);
      const uint32_t gw = ~seg_max_u32<LPT>(left && my_g == m ? ~(uint32_t)q : 0u);
      kept |= 1ull << (gw & 63u);
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (!((kept >> (grp[i] & 63)) & 1ull)) open &= ~(1u << i);
  }

  // selection rounds: the r-th winner is kept by lane q == r
  const int nsel = presel > k ? presel : k;
  int my_e = 0;
  float my_s = 0.f, s_max = 0.f;
  for (int r = 0; r < nsel; ++r) {
    // the best open score of this lane, then of the group; the lowest expert of
    // equal ones
    uint32_t best = 0u;
    int mine = 0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      if (((open >> i) & 1u) && key[i] > best) {
        best = key[i];
        mine = q + i * LPT;
      }
    }
    const uint32_t m = seg_max_u32<LPT>(best);
    int we;
    if constexpr (LPT == 64 && EPL == 1) {  // lane = expert: the first lane that has it
      we = __ffsll(__ballot(best == m && m > 0u)) - 1;
      we = max(we, 0);
    } else {
      we = min((int)~seg_max_u32<LPT>(best == m && m > 0u ? ~(uint32_t)mine : 0x80000000u), E - 1);
    }
    const float ws = ord_key_inv(m);
    if (we % LPT == q) open &= ~(1u << (we / LPT));
    if (r == 0) s_max = ws;
    if (q == r) {
      my_e = we;
      my_s = ws;
    }
  }

  // gates: e_j = exp(s_j - m) over the chosen / pre-selected / all experts
  const float ej = q < nsel ? expf(my_s - s_max) : 0.f;
  float denom;
  if (renorm) {
    denom = seg_sum<LPT>(q < k ? ej : 0.f);
  } else if (presel) {
    denom = seg_sum<LPT>(q < presel ? ej : 0.f);
  } else {
    float part = 0.f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = q + i * LPT;
      if (i < epl && e < E) part += expf(ord_key_inv(key[i]) - s_max);
    }
    denom = seg_sum<LPT>(part);
  }
  *out_e = my_e;
  *out_w = ej / denom;
}

}  // namespace moe
