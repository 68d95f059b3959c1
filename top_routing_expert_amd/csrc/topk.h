// Selection and gates of one token by a group of LPT lanes (used by the router's
// top-k kernel and by the few-token layer, so both choose alike).
#pragma once

#include "common.h"

namespace moe {

constexpr int kMaxSplits = 16;  // split-K partials of the router GEMM (summed by top-k)

__device__ __forceinline__ unsigned long long shfl_xor_u64(unsigned long long v, int m) {
  const int lo = __shfl_xor((int)(uint32_t)v, m);
  const int hi = __shfl_xor((int)(uint32_t)(v >> 32), m);
  return ((unsigned long long)(uint32_t)hi << 32) | (uint32_t)lo;
}

template <int LPT>
__device__ __forceinline__ unsigned long long seg_max_u64(unsigned long long v) {
#pragma unroll
  for (int o = LPT / 2; o > 0; o >>= 1) {
    const unsigned long long w = shfl_xor_u64(v, o);
    v = w > v ? w : v;
  }
  return v;
}

template <int LPT>
__device__ __forceinline__ uint32_t seg_max_u32(uint32_t v) {
#pragma unroll
  for (int o = LPT / 2; o > 0; o >>= 1) {
    const uint32_t w = (uint32_t)__shfl_xor((int)v, o);
    v = w > v ? w : v;
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

// Lane q = lane % LPT of the group's token t (`live`: t < T; a group without a
// token runs along).  EPL: scores per lane (ceil(E / LPT): 1 for E <= 64), so
// the code holds only the loops a layer of this size needs.  The j-th best
// expert and its gate end up in lane q == j of the group (*out_e, *out_w).
template <int LPT, int EPL>
__device__ __forceinline__ void select_token(const float* __restrict__ partial, int splits,
                                             const float* __restrict__ bias,
                                             float* __restrict__ logits_out, int t, bool live,
                                             int q, int T, int E, int k, int n_group,
                                             int topk_group, int presel, int renorm, int* out_e,
                                             float* out_w) {
  const int epl = (E + LPT - 1) / LPT;

  // scores s = z + b (one fp32 add), -0 -> +0; key32 = order-preserving bits
  uint32_t key[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    key[i] = 0u;
    const int e = q + i * LPT;
    if (i < epl && e < E && live) {
      // every partial is loaded before the first add (one memory latency),
      // then summed in split order
      float pv[kMaxSplits];
#pragma unroll
      for (int s = 0; s < kMaxSplits; ++s)
        pv[s] = s < splits ? partial[((size_t)s * T + t) * E + e] : 0.f;
      float z = pv[0];
#pragma unroll
      for (int s = 1; s < kMaxSplits; ++s)
        if (s < splits) z += pv[s];
      if (logits_out) logits_out[(size_t)t * E + e] = z;
      float sc = bias ? __fadd_rn(z, bias[e]) : z;
      uint32_t u = __float_as_uint(sc);
      if (u == 0x80000000u) u = 0u;
      key[i] = ord_key(__uint_as_float(u));
    }
  }

  // group-limited eligibility: keep the topk_group groups with the largest max
  unsigned long long kept = ~0ull;
  const bool grouped = n_group > 1 && topk_group < n_group;
  int gsz = E / n_group;
  if (grouped) {
    uint32_t my_g = 0u;
    for (int g = 0; g < n_group; ++g) {
      uint32_t m = 0u;
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        const int e = q + i * LPT;
        if (i < epl && e < E && e / gsz == g) m = key[i] > m ? key[i] : m;
      }
      m = seg_max_u32<LPT>(m);
      if (q == g) my_g = m;
    }
    kept = 0ull;
    for (int r = 0; r < topk_group; ++r) {
      unsigned long long cand = 0ull;
      if (q < n_group && !((kept >> q) & 1ull))
        cand = ((unsigned long long)my_g << 32) | (0xffffffffu - (uint32_t)q);
      cand = seg_max_u64<LPT>(cand);
      const int gw = (int)(0xffffffffu - (uint32_t)cand);
      kept |= 1ull << gw;
    }
  }

  // selection rounds: the r-th winner is kept by lane q == r
  const int nsel = presel > k ? presel : k;
  uint32_t taken = 0u;
  int my_e = 0;
  float my_s = 0.f, s_max = 0.f;
  for (int r = 0; r < nsel; ++r) {
    unsigned long long best = 0ull;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = q + i * LPT;
      const bool ok = i < epl && e < E && !((taken >> i) & 1u) &&
                      (!grouped || ((kept >> (e / gsz)) & 1ull));
      const unsigned long long cand =
          ok ? (((unsigned long long)key[i] << 32) | (0xffffffffu - (uint32_t)e)) : 0ull;
      best = cand > best ? cand : best;
    }
    best = seg_max_u64<LPT>(best);
    const int we = (int)(0xffffffffu - (uint32_t)best);
    const float ws = ord_key_inv((uint32_t)(best >> 32));
    if (we % LPT == q) taken |= 1u << (we / LPT);
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
