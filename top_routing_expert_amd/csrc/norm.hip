// RMS norms around the MoE block, with the block's gate and residual scale.
//
//   before the block   xn = x r w,              r = 1 / sqrt(mean x^2 + eps)
//   behind the block   y  = sum_j g[t,j] y_perm[slot_of[t k + j]]
//                      out = s residual + gate (y r w),  r of y
// and their gradients.  With n = x r (or y r) and gw the gradient at n:
//   d_x = r (gw - n mean(gw n)),   d_w = sum_t (upstream) n.
// Behind the block d_gate[q] = w S_q and d_w = sum_q gate[q] S_q with
// S_q = sum over the tokens of gate row q of d_out n: one accumulated row
// serves both gradients.
//
// gfx950 design.  All of these stream rows once: a block per token row
// (forward) or per run of consecutive tokens (backward), VPT 16-byte vectors
// per thread held in registers between the statistics and the output, so
// every row is read from memory once.  The combine is part of the norm's read:
// y never exists in memory, and the backward rebuilds it from the k expert rows
// that d_topk_w needs anyway.  The backward's parameter gradients are summed
// in registers over a block's tokens, written as float32 partial rows and
// added by a second kernel in a fixed order (no atomics).
//
// All bound by HBM: T16383-d5120 forward 59 us and backward 142 us (5.7 and 4.7 TB/s), the
// parameter gradient 6.6 us behind it; with T8192-d7168 k 8 the combine forward and
// backward take 201 and 456 us for 3.3 GB (5 TB/s), the parameter gradients 7 us.
#include <algorithm>
#include <type_traits>

#include "common.h"

namespace moe {

constexpr int kNormMaxThreads = 512;
constexpr int kNormMaxK = 16;

// 16-byte vectors of the two element types.
template <typename T>
struct Vec16;
template <>
struct Vec16<uint16_t> {  // bf16 bits
  static constexpr int N = 8;
  static __device__ __forceinline__ void unpack(u32x4 v, float* f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = bf16_lo(v[i]);
      f[2 * i + 1] = bf16_hi(v[i]);
    }
  }
  static __device__ __forceinline__ u32x4 pack(const float* f) {
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
    return v;
  }
};
template <>
struct Vec16<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void unpack(u32x4 v, float* f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(v[i]);
  }
  static __device__ __forceinline__ u32x4 pack(const float* f) {
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __float_as_uint(f[i]);
    return v;
  }
};

// A combine that moves far more than the 256 MB Infinity Cache holds stores past it (past: the
// same for every thread).  Measured with a reader of the output behind it, d = 7168, us:
//   backward  T8192 k 8 (2.1 GB) 758 -> 734, T4096 k 8 (1.1 GB) 432 -> 406, T8192 k 2 (0.70 GB)
//             263 -> 262; T1024 k 8 (0.26 GB), which stays ordinary, 139 -> 175
//   forward   T8192 k 8 (1.2 GB) 258 -> 248; ordinary: T4096 k 8 (0.59 GB) 123 -> 123, T8192 k 2
//             (0.47 GB) 117 -> 122
// The norms in front of the block write less than they read and their readers come next: ordinary
// (T16384-d5120, forward 82 -> 90 with its reader, backward 207 -> 210).
constexpr long kNormPastBytes = 640L << 20;
__device__ __forceinline__ void norm_store(u32x4* p, u32x4 v, bool past) {
  if (past) {
    asm volatile("");  // the compiler would make one ordinary store of the two
    __builtin_nontemporal_store(v, p);
    asm volatile("");
  } else {
    *p = v;
  }
}

// Sum over the wave, the same value in every lane: moves within 16 lanes, then
// swaps of 16- and 32-lane halves (a shuffle through LDS takes several times as
// long a step).
template <int CTRL>
__device__ __forceinline__ float norm_dpp(float v) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(
      (int)__float_as_uint(v), (int)__float_as_uint(v), CTRL, 0xf, 0xf, false));
}
__device__ __forceinline__ float norm_add_halves(float v) {
  const uint32_t u = __float_as_uint(v);
  const auto p = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  const uint32_t w = __float_as_uint(__uint_as_float(p[0]) + __uint_as_float(p[1]));
  const auto q = __builtin_amdgcn_permlane32_swap(w, w, false, false);
  return __uint_as_float(q[0]) + __uint_as_float(q[1]);
}
// Keeps the compiler from carrying what was computed from v across this point.
__device__ __forceinline__ void norm_opaque(u32x4& v) { asm volatile("" : "+v"(v)); }
__device__ __forceinline__ float norm_wave_sum(float v) {
  v += norm_dpp<0xB1>(v);   // lanes 1 0 3 2 of a quad
  v += norm_dpp<0x4E>(v);   // lanes 2 3 0 1 of a quad
  v += norm_dpp<0x141>(v);  // mirrored within 8
  v += norm_dpp<0x140>(v);  // mirrored within 16
  return norm_add_halves(v);
}
// Wave sums of N values (1, 2, 4, 8 or 16): value j ends up in the lanes whose low bits
// are j.  Every halving step sends one half of the values and keeps the other, so
// N values take N - 1 moves and then one chain instead of N chains.
template <int N>
__device__ __forceinline__ float norm_wave_sums(const float (&v)[N]) {
  const int lane = threadIdx.x & 63;
  float r[N];
#pragma unroll
  for (int j = 0; j < N; ++j) r[j] = v[j];
#pragma unroll
  for (int bit = 1; bit < N; bit <<= 1) {
    // r[j], j = 0 .. N / bit - 1: value (j bit + the lane's bits below); keep those with the
    // next bit as in the lane
#pragma unroll
    for (int j = 0; j < N / bit; j += 2) {
      const bool up = lane & bit;
      const float keep = up ? r[j + 1] : r[j], send = up ? r[j] : r[j + 1];
      const float got = bit == 1   ? norm_dpp<0xB1>(send)
                        : bit == 2 ? norm_dpp<0x4E>(send)
                                   : __shfl_xor(send, bit);
      r[j / 2] = keep + got;
    }
  }
  float s = r[0];
#pragma unroll
  for (int o = N; o < 16; o <<= 1)
    s += o == 1 ? norm_dpp<0xB1>(s) : o == 2 ? norm_dpp<0x4E>(s) : __shfl_xor(s, o);
  return norm_add_halves(s);
}

// Sum over the block in wave order, the same value for every thread.  `part`
// holds one float per wave; a caller that loops alternates two arrays so that
// one barrier per sum is enough.
__device__ __forceinline__ float norm_block_sum(float v, float* part) {
  v = norm_wave_sum(v);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = part[0];
  const int waves = (blockDim.x + 63) >> 6;
  for (int i = 1; i < waves; ++i) s += part[i];
  return s;
}

// ------------------------------------------------------------ before the block
template <typename T, int VPT, int MAXT>
__global__ __launch_bounds__(MAXT) void norm_fwd_kernel(const u32x4* __restrict__ x,
                                                        const u32x4* __restrict__ w, float eps,
                                                        u32x4* __restrict__ xn,
                                                        float* __restrict__ rstd, int nvec,
                                                        float inv_d) {
  using V = Vec16<T>;
  __shared__ float part[kNormMaxThreads / 64];
  const int t = blockIdx.x;
  const u32x4* row = x + (size_t)t * nvec;
  u32x4 xv[VPT], wv[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = threadIdx.x + blockDim.x * i;
    if (v < nvec) xv[i] = row[v];
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = threadIdx.x + blockDim.x * i;
    if (w && v < nvec) wv[i] = w[v];
  }
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = threadIdx.x + blockDim.x * i;
    if (v < nvec) {
      float f[V::N];
      V::unpack(xv[i], f);
#pragma unroll
      for (int q = 0; q < V::N; ++q) ss = fmaf(f[q], f[q], ss);
    }
  }
  const float r = 1.0f / sqrtf(norm_block_sum(ss, part) * inv_d + eps);
  if (rstd && threadIdx.x == 0) rstd[t] = r;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = threadIdx.x + blockDim.x * i;
    if (v < nvec) {
      float f[V::N], g[V::N];
      V::unpack(xv[i], f);
      if (w) V::unpack(wv[i], g);
#pragma unroll
      for (int q = 0; q < V::N; ++q) f[q] = w ? f[q] * r * g[q] : f[q] * r;
      xn[(size_t)t * nvec + v] = V::pack(f);
    }
  }
}

// Block b: tokens [b per, b per + per) of T, in order; the block's partial
// weight gradient goes to partial[b].  d_residual NULL: no residual term.
// The next token's rows are loaded while the current one is summed; what the
// sum's two sides share is rebuilt from the rows instead of kept, which holds the
// registers to five waves a SIMD.
template <typename T, int VPT, int MAXT>
__global__ __launch_bounds__(MAXT) void norm_bwd_kernel(
    const u32x4* __restrict__ d_xn, const u32x4* __restrict__ x, const u32x4* __restrict__ w,
    const float* __restrict__ rstd, const u32x4* d_residual, u32x4* d_x,
    float* __restrict__ partial, int nvec, float inv_d, int T_, int per) {
  using V = Vec16<T>;
  constexpr int N = V::N;
  __shared__ float part[2][kNormMaxThreads / 64];
  const int t0 = blockIdx.x * per, t1 = min(t0 + per, T_);
  u32x4 wv[VPT];
  float S[VPT][N];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = threadIdx.x + blockDim.x * i;
    if (w && v < nvec) wv[i] = w[v];
#pragma unroll
    for (int q = 0; q < N; ++q) S[i][q] = 0.f;
  }
  struct Rows {
    u32x4 x[VPT], g[VPT], res[VPT];
    float r;
  };
  auto load = [&](int t, Rows& R) {
    R.r = rstd[t];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = min((int)(threadIdx.x + blockDim.x * i), nvec - 1);  // past the row: its end
      const size_t at = (size_t)t * nvec + v;
      R.x[i] = __builtin_nontemporal_load(x + at);
      R.g[i] = __builtin_nontemporal_load(d_xn + at);
      if (d_residual) R.res[i] = d_residual[at];
    }
  };
  // n and the gradient at it, of vector i
  auto terms = [&](const Rows& R, int i, float* n, float* gw, float* g) {
    V::unpack(R.x[i], n);
    V::unpack(R.g[i], g);
    float wf[N];
    if (w) V::unpack(wv[i], wf);
#pragma unroll
    for (int q = 0; q < N; ++q) {
      n[q] *= R.r;
      gw[q] = w ? g[q] * wf[q] : g[q];
    }
  };
  auto step = [&](int t, Rows& R, Rows& next) {
    if (t + 1 < t1) load(t + 1, next);
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = threadIdx.x + blockDim.x * i;
      if (v < nvec) {
        float n[N], gw[N], g[N];
        terms(R, i, n, gw, g);
#pragma unroll
        for (int q = 0; q < N; ++q) {
          S[i][q] = fmaf(g[q], n[q], S[i][q]);
          dot = fmaf(gw[q], n[q], dot);
        }
      }
    }
    const float c = norm_block_sum(dot, part[t & 1]) * inv_d;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      norm_opaque(R.x[i]);
      norm_opaque(R.g[i]);
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = threadIdx.x + blockDim.x * i;
      if (v < nvec) {
        float n[N], gw[N], g[N], f[N], o[N];
        terms(R, i, n, gw, g);
        if (d_residual) V::unpack(R.res[i], f);
#pragma unroll
        for (int q = 0; q < N; ++q) {
          const float dx = R.r * (gw[q] - n[q] * c);
          o[q] = d_residual ? f[q] + dx : dx;
        }
        d_x[(size_t)t * nvec + v] = V::pack(o);
      }
    }
  };
  Rows A, B;
  load(t0, A);
  for (int t = t0; t < t1; t += 2) {
    step(t, A, B);
    if (t + 1 < t1) step(t + 1, B, A);
  }
  if (partial) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = threadIdx.x + blockDim.x * i;
      if (v < nvec) {
#pragma unroll
        for (int q = 0; q < N; q += 4)
          *reinterpret_cast<float4*>(partial + ((size_t)blockIdx.x * nvec + v) * N + q) =
              make_float4(S[i][q], S[i][q + 1], S[i][q + 2], S[i][q + 3]);
      }
    }
  }
}

// ------------------------------------------------------------ behind the block
// The k expert rows of token t (slot_of clamped into [0, rows)), or y itself in
// token order when slot_of is NULL (k = 1 row of weight 1).
template <int KC>
__device__ __forceinline__ void token_rows(const int32_t* slot_of, const float* topk_w, int t,
                                           int k, int rows, int* p, float* g) {
#pragma unroll
  for (int j = 0; j < KC; ++j) {
    p[j] = t;
    g[j] = 1.f;
    if (slot_of && j < k) {
      p[j] = min(max(slot_of[(size_t)t * k + j], 0), rows - 1);
      g[j] = topk_w[(size_t)t * k + j];
    }
  }
}

template <typename T, int VPT, int MAXT, int KC>
__global__ __launch_bounds__(MAXT) void combine_norm_fwd_kernel(
    const u32x4* __restrict__ y, const int32_t* __restrict__ slot_of,
    const float* __restrict__ topk_w, const u32x4* residual, const u32x4* __restrict__ w,
    const u32x4* __restrict__ gate, int per_gate, float eps, float res_scale, u32x4* out,
    float* __restrict__ rstd, int nvec, float inv_d, int rows, int k, bool past) {
  using V = Vec16<T>;
  constexpr int N = V::N;
  __shared__ float part[kNormMaxThreads / 64];
  const int t = blockIdx.x;
  int p[KC];
  float g[KC];
  token_rows<KC>(slot_of, topk_w, t, k, rows, p, g);
  float yf[VPT][N];
  float ss = 0.f;
  // vectors whose k rows are in flight together: at most 64 registers of rows
  constexpr int BI = VPT * KC <= 16 ? VPT : KC <= 8 ? 2 : 1;
  u32x4 res[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = threadIdx.x + blockDim.x * i;
    if (residual && v < nvec) res[i] = residual[(size_t)t * nvec + v];
  }
#pragma unroll
  for (int i0 = 0; i0 < VPT; i0 += BI) {
    u32x4 row[BI][KC];
#pragma unroll
    for (int b = 0; b < BI; ++b) {
      const int v = threadIdx.x + blockDim.x * (i0 + b);
#pragma unroll
      for (int j = 0; j < KC; ++j)  // read once
        if (j < k && v < nvec) row[b][j] = __builtin_nontemporal_load(&y[(size_t)p[j] * nvec + v]);
    }
#pragma unroll
    for (int b = 0; b < BI; ++b) {
      const int i = i0 + b, v = threadIdx.x + blockDim.x * i;
#pragma unroll
      for (int q = 0; q < N; ++q) yf[i][q] = 0.f;
      if (v < nvec) {
#pragma unroll
        for (int j = 0; j < KC; ++j) {
          if (j < k) {
            float f[N];
            V::unpack(row[b][j], f);
#pragma unroll
            for (int q = 0; q < N; ++q) yf[i][q] = fmaf(g[j], f[q], yf[i][q]);
          }
        }
      }
#pragma unroll
      for (int q = 0; q < N; ++q) ss = fmaf(yf[i][q], yf[i][q], ss);
    }
    if constexpr (BI < VPT) asm volatile("" ::: "memory");  // the next rows are loaded here
  }
  const float r = 1.0f / sqrtf(norm_block_sum(ss, part) * inv_d + eps);
  if (rstd && threadIdx.x == 0) rstd[t] = r;
  const u32x4* grow = gate ? gate + (size_t)(t / per_gate) * nvec : nullptr;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = threadIdx.x + blockDim.x * i;
    if (v < nvec) {
      float wf[N], gf[N], rf[N], o[N];
      if (w) V::unpack(w[v], wf);
      if (gate) V::unpack(grow[v], gf);
      if (residual) V::unpack(res[i], rf);
#pragma unroll
      for (int q = 0; q < N; ++q) {
        float n = yf[i][q] * r;
        if (w) n *= wf[q];
        if (gate) n *= gf[q];
        o[q] = residual ? fmaf(res_scale, rf[q], n) : n;
      }
      norm_store(out + (size_t)t * nvec + v, V::pack(o), past);
    }
  }
}

// Block b: tokens [b per, b per + per).  The running sum S of d_out n is
// written out whenever the next token belongs to another gate row and at the
// end of the block: piece (block b, gate row q) is partial row b + q (the
// pieces of consecutive tokens have strictly growing b + q, so no two pieces
// share a row).  HOLD: the k expert rows stay in registers between the two
// passes over them; else they are read again.
template <typename T, int VPT, int MAXT, int KC, bool HOLD>
__global__ __launch_bounds__(MAXT) void combine_norm_bwd_kernel(
    const u32x4* __restrict__ d_out, const u32x4* __restrict__ y,
    const int32_t* __restrict__ slot_of, const float* __restrict__ topk_w,
    const u32x4* __restrict__ w, const u32x4* __restrict__ gate, int per_gate, float res_scale,
    const float* __restrict__ rstd, u32x4* __restrict__ d_y, float* __restrict__ d_topk_w,
    u32x4* __restrict__ d_residual, float* __restrict__ partial, int nvec, float inv_d, int rows,
    int k, int T_, int per, bool past) {
  using V = Vec16<T>;
  constexpr int N = V::N;
  __shared__ float part[2][kNormMaxThreads / 64];
  __shared__ float dots[2][kNormMaxThreads / 64][KC];
  const int t0 = blockIdx.x * per, t1 = min(t0 + per, T_);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int waves = (blockDim.x + 63) >> 6;
  float S[VPT][N];
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int q = 0; q < N; ++q) S[i][q] = 0.f;
  for (int t = t0; t < t1; ++t) {
    int p[KC];
    float g[KC];
    token_rows<KC>(slot_of, topk_w, t, k, rows, p, g);
    const float r = rstd[t];
    const int q_gate = gate ? t / per_gate : 0;
    const u32x4* grow = gate ? gate + (size_t)q_gate * nvec : nullptr;
    u32x4 row[HOLD ? VPT : 1][KC], dv[VPT];
    float n[VPT][N];
    // the gradient at n, of vector i
    auto upstream = [&](int i, int v, float* dn) {
      float f[N];
      V::unpack(dv[i], dn);
      if (w) {
        V::unpack(w[v], f);
#pragma unroll
        for (int q = 0; q < N; ++q) dn[q] *= f[q];
      }
      if (gate) {
        V::unpack(grow[v], f);
#pragma unroll
        for (int q = 0; q < N; ++q) dn[q] *= f[q];
      }
    };
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = threadIdx.x + blockDim.x * i;
      if (v < nvec) dv[i] = d_out[(size_t)t * nvec + v];
      if constexpr (HOLD) {
#pragma unroll
        for (int j = 0; j < KC; ++j)
          if (j < k && v < nvec) row[i][j] = __builtin_nontemporal_load(&y[(size_t)p[j] * nvec + v]);
      }
    }
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = threadIdx.x + blockDim.x * i;
#pragma unroll
      for (int q = 0; q < N; ++q) n[i][q] = 0.f;
      if (v >= nvec) continue;
      if constexpr (!HOLD) {
#pragma unroll
        for (int j = 0; j < KC; ++j)
          if (j < k) row[0][j] = y[(size_t)p[j] * nvec + v];
      }
#pragma unroll
      for (int j = 0; j < KC; ++j) {
        if (j < k) {
          float f[N];
          V::unpack(row[HOLD ? i : 0][j], f);
#pragma unroll
          for (int q = 0; q < N; ++q) n[i][q] = fmaf(g[j], f[q], n[i][q]);
        }
      }
      float df[N], o[N], dn[N];
      V::unpack(dv[i], df);
#pragma unroll
      for (int q = 0; q < N; ++q) {
        n[i][q] *= r;
        S[i][q] = fmaf(df[q], n[i][q], S[i][q]);
        o[q] = res_scale * df[q];
      }
      if (d_residual) norm_store(d_residual + (size_t)t * nvec + v, V::pack(o), past);
      upstream(i, v, dn);
#pragma unroll
      for (int q = 0; q < N; ++q) dot = fmaf(dn[q], n[i][q], dot);
    }
    const float c = norm_block_sum(dot, part[t & 1]) * inv_d;
    float dw[KC];
#pragma unroll
    for (int j = 0; j < KC; ++j) dw[j] = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      norm_opaque(dv[i]);
      if constexpr (HOLD) {
#pragma unroll
        for (int j = 0; j < KC; ++j) norm_opaque(row[i][j]);
      }
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = threadIdx.x + blockDim.x * i;
      if (v >= nvec) continue;
      float dy[N];
      upstream(i, v, dy);
#pragma unroll
      for (int q = 0; q < N; ++q) dy[q] = r * (dy[q] - n[i][q] * c);
      if constexpr (!HOLD) {
        if (d_topk_w) {
#pragma unroll
          for (int j = 0; j < KC; ++j)
            if (j < k) row[0][j] = y[(size_t)p[j] * nvec + v];
        }
      }
#pragma unroll
      for (int j = 0; j < KC; ++j) {
        if (j < k) {
          float f[N], o[N];
          if (d_topk_w) V::unpack(row[HOLD ? i : 0][j], f);
#pragma unroll
          for (int q = 0; q < N; ++q) {
            if (d_topk_w) dw[j] = fmaf(dy[q], f[q], dw[j]);
            o[q] = g[j] * dy[q];
          }
          norm_store(d_y + (size_t)p[j] * nvec + v, V::pack(o), past);
        }
      }
    }
    if (d_topk_w) {  // uniform
      const float s = norm_wave_sums<KC>(dw);
      if (lane < KC) dots[t & 1][wave][lane] = s;
      __syncthreads();
      if ((int)threadIdx.x < k) {
        float v = dots[t & 1][0][threadIdx.x];
        for (int i = 1; i < waves; ++i) v += dots[t & 1][i][threadIdx.x];
        d_topk_w[(size_t)t * k + threadIdx.x] = v;
      }
    }
    if (partial && (t + 1 == t1 || (gate && (t + 1) / per_gate != q_gate))) {
      float* prow = partial + (size_t)(blockIdx.x + q_gate) * nvec * N;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int v = threadIdx.x + blockDim.x * i;
        if (v < nvec) {
#pragma unroll
          for (int q = 0; q < N; q += 4) {
            *reinterpret_cast<float4*>(prow + (size_t)v * N + q) =
                make_float4(S[i][q], S[i][q + 1], S[i][q + 2], S[i][q + 3]);
            S[i][q] = S[i][q + 1] = S[i][q + 2] = S[i][q + 3] = 0.f;
          }
        }
      }
    }
  }
}

// ------------------------------------------------------ parameter gradients
// One block per 32 columns (128 bytes of a partial row), 32 groups of 32 lanes.  For
// every gate row q: S_q = the sum of its pieces, which are partial rows
// [first + q, last + q] with first and last the blocks of its first and last token.
// d_gate[q] = w S_q; d_w = sum_q gate[q] S_q.  Up to 32 gate rows are summed at once by
// 32 / n_gate groups each; more by one group each, in turn.  Every order is fixed by
// T, d and n_gate.  (Gate rows in turn by the whole block, 64 columns: 11.5 us for
// T777-d1028 with 7 gate rows.)
template <typename T>
__device__ __forceinline__ float norm_scalar(const void* p, size_t i) {
  if constexpr (sizeof(T) == 2)
    return __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16);
  else
    return static_cast<const float*>(p)[i];
}

template <typename T>
__global__ __launch_bounds__(1024) void norm_param_grad_kernel(
    const float* __restrict__ partial, const void* __restrict__ w, const void* __restrict__ gate,
    float* __restrict__ d_w, float* __restrict__ d_gate, int d, int n_gate, int per_gate,
    int per) {
  constexpr int GR = 32;  // groups
  __shared__ float sums[GR][32], dws[GR][32];
  const int group = threadIdx.x >> 5, c = threadIdx.x & 31, col = blockIdx.x * 32 + c;
  const bool live = col < d;
  const float wc = live && w ? norm_scalar<T>(w, col) : 1.f;
  const int gpq = n_gate < GR ? GR / n_gate : 1;  // groups of a gate row
  float dw = 0.f;
  auto finish = [&](int q, float s) {  // gate row q's sum
    if (live) {
      if (d_gate) d_gate[(size_t)q * d + col] = wc * s;
      dw = fmaf(gate ? norm_scalar<T>(gate, (size_t)q * d + col) : 1.f, s, dw);
    }
  };
  float s = 0.f;
  for (int q = group / gpq; q < n_gate; q += GR) {  // one turn where gpq > 1
    const int first = (int)((long)q * per_gate / per);
    const int last = (int)(((long)(q + 1) * per_gate - 1) / per);
    s = 0.f;
    if (live) {
      constexpr int U = 8;  // loads in flight
      for (int b = first + group % gpq; b <= last; b += U * gpq) {
        float v[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
          v[u] = partial[(size_t)(min(b + u * gpq, last) + q) * d + col];
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (b + u * gpq <= last) s += v[u];
      }
    }
    if (gpq == 1) finish(q, s);
  }
  if (gpq > 1) {
    sums[group][c] = s;
    __syncthreads();
    if (group < n_gate) {
      s = sums[group * gpq][c];
      for (int i = 1; i < gpq; ++i) s += sums[group * gpq + i][c];
      finish(group, s);
    }
  }
  dws[group][c] = dw;
  __syncthreads();
  if (d_w && live && group == 0) {
    for (int i = 1; i < min(n_gate, GR); ++i) dw += dws[i][c];
    d_w[col] = dw;
  }
}

// ------------------------------------------------------------------ launchers
static int norm_nvec(const moe_config& c) { return c.dtype == MOE_BF16 ? c.d / 8 : c.d / 4; }

bool norm_row_supported(const moe_config& c) { return norm_nvec(c) <= 4 * kNormMaxThreads; }

// Tokens per backward block: about four blocks per CU, so that the float32
// partial rows stay a small part of the traffic (T16383-d5120: 21 MB of
// 1.0 GB) while every CU has work.
static int norm_tokens_per_block(const moe_config& c) {
  constexpr int kBlocks = 1024;
  return c.T <= 0 ? 1 : div_up(c.T, kBlocks);
}

size_t norm_backward_ws_bytes(const moe_config& c) {
  return c.T <= 0 ? 0 : (size_t)div_up(c.T, norm_tokens_per_block(c)) * c.d * sizeof(float);
}
size_t combine_norm_backward_ws_bytes(const moe_config& c, int n_gate) {
  if (c.T <= 0) return 0;
  const long pieces = div_up(c.T, norm_tokens_per_block(c)) + (long)std::max(n_gate, 1) - 1;
  return (size_t)pieces * c.d * sizeof(float);
}

// Threads of a row: two vectors each up to 1024 vectors, four above.
static int norm_threads(int nvec, int vpt) { return div_up(div_up(nvec, vpt), 64) * 64; }
static bool norm_small(int nvec) { return nvec <= 1024; }
// Whether a call that moves `rows` rows of d elements stores past the cache.
static bool norm_past(const moe_config& c, long rows) {
  return rows * norm_nvec(c) * 16 > kNormPastBytes;
}

template <typename F>
static void with_types(const moe_config& c, F&& f) {
  if (c.dtype == MOE_BF16)
    f(uint16_t());
  else
    f(float());
}

static hipError_t norm_fill_zero(float* p, long n, hipStream_t st) {
  return p ? launch_fill_i32(reinterpret_cast<int32_t*>(p), (int)n, 0, st) : hipSuccess;
}

hipError_t launch_norm(const moe_config& c, const void* x, const void* w, float eps, void* xn,
                       float* rstd, hipStream_t st) {
  const int nvec = norm_nvec(c);
  const auto* xv = static_cast<const u32x4*>(x);
  const auto* wv = static_cast<const u32x4*>(w);
  auto* ov = static_cast<u32x4*>(xn);
  const float inv_d = 1.0f / (float)c.d;
  with_types(c, [&](auto t) {
    using T = decltype(t);
    if (norm_small(nvec))
      norm_fwd_kernel<T, 2, 512><<<c.T, norm_threads(nvec, 2), 0, st>>>(xv, wv, eps, ov, rstd,
                                                                        nvec, inv_d);
    else
      norm_fwd_kernel<T, 4, 512><<<c.T, norm_threads(nvec, 4), 0, st>>>(xv, wv, eps, ov, rstd,
                                                                         nvec, inv_d);
  });
  return hipGetLastError();
}

static hipError_t launch_param_grad(const moe_config& c, const float* partial, const void* w,
                                    const void* gate, float* d_w, float* d_gate, int n_gate,
                                    int per, hipStream_t st) {
  const int n = std::max(n_gate, 1), per_gate = c.T / n;
  with_types(c, [&](auto t) {
    using T = decltype(t);
    norm_param_grad_kernel<T><<<div_up(c.d, 32), 1024, 0, st>>>(partial, w, gate, d_w, d_gate, c.d,
                                                                 n, per_gate, per);
  });
  return hipGetLastError();
}

hipError_t launch_norm_backward(const moe_config& c, const void* d_xn, const void* x,
                                const void* w, const float* rstd, const void* d_residual,
                                void* d_x, float* d_w, void* ws, hipStream_t st) {
  if (c.T == 0) return norm_fill_zero(d_w, c.d, st);
  const int nvec = norm_nvec(c), per = norm_tokens_per_block(c);
  const int blocks = div_up(c.T, per);
  const auto* gv = static_cast<const u32x4*>(d_xn);
  const auto* xv = static_cast<const u32x4*>(x);
  const auto* wv = static_cast<const u32x4*>(w);
  const auto* rv = static_cast<const u32x4*>(d_residual);
  auto* ov = static_cast<u32x4*>(d_x);
  float* partial = d_w ? static_cast<float*>(ws) : nullptr;
  const float inv_d = 1.0f / (float)c.d;
  with_types(c, [&](auto t) {
    using T = decltype(t);
    if (norm_small(nvec))
      norm_bwd_kernel<T, 2, 512><<<blocks, norm_threads(nvec, 2), 0, st>>>(
          gv, xv, wv, rstd, rv, ov, partial, nvec, inv_d, c.T, per);
    else
      norm_bwd_kernel<T, 4, 512><<<blocks, norm_threads(nvec, 4), 0, st>>>(
          gv, xv, wv, rstd, rv, ov, partial, nvec, inv_d, c.T, per);
  });
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !d_w) return e;
  return launch_param_grad(c, partial, nullptr, nullptr, d_w, nullptr, 1, per, st);
}

// KC: k rounded up to 1, 2, 4, 8 or 16.
template <typename F>
static void with_k(int k, F&& f) {
  if (k <= 1)
    f(std::integral_constant<int, 1>());
  else if (k <= 2)
    f(std::integral_constant<int, 2>());
  else if (k <= 4)
    f(std::integral_constant<int, 4>());
  else if (k <= 8)
    f(std::integral_constant<int, 8>());
  else
    f(std::integral_constant<int, kNormMaxK>());
}

hipError_t launch_combine_norm(const moe_config& c, const void* y, const int32_t* slot_of,
                               const float* topk_w, const void* residual, const void* w,
                               const void* gate, int n_gate, float eps, float res_scale, void* out,
                               float* rstd, hipStream_t st) {
  const int nvec = norm_nvec(c), k = slot_of ? c.k : 1, rows = c.T * k;
  const int per_gate = n_gate ? c.T / n_gate : 1;
  const auto* yv = static_cast<const u32x4*>(y);
  const auto* rv = static_cast<const u32x4*>(residual);
  const auto* wv = static_cast<const u32x4*>(w);
  const auto* gv = static_cast<const u32x4*>(gate);
  auto* ov = static_cast<u32x4*>(out);
  const float inv_d = 1.0f / (float)c.d;
  const bool past = norm_past(c, (long)rows + (residual ? 2L : 1L) * c.T);
  with_types(c, [&](auto t) {
    using T = decltype(t);
    with_k(k, [&](auto kc) {
      constexpr int KC = decltype(kc)::value;
      if (norm_small(nvec))
        combine_norm_fwd_kernel<T, 2, 512, KC><<<c.T, norm_threads(nvec, 2), 0, st>>>(
            yv, slot_of, topk_w, rv, wv, gv, per_gate, eps, res_scale, ov, rstd, nvec, inv_d, rows,
            k, past);
      else
        combine_norm_fwd_kernel<T, 4, 512, KC><<<c.T, norm_threads(nvec, 4), 0, st>>>(
            yv, slot_of, topk_w, rv, wv, gv, per_gate, eps, res_scale, ov, rstd, nvec, inv_d, rows,
            k, past);
    });
  });
  return hipGetLastError();
}

hipError_t launch_combine_norm_backward(const moe_config& c, const void* d_out, const void* y,
                                        const int32_t* slot_of, const float* topk_w, const void* w,
                                        const void* gate, int n_gate, float res_scale,
                                        const float* rstd, void* d_y, float* d_topk_w,
                                        void* d_residual, float* d_w, float* d_gate, void* ws,
                                        hipStream_t st) {
  if (c.T == 0) {
    hipError_t e = norm_fill_zero(d_w, c.d, st);
    return e != hipSuccess ? e : norm_fill_zero(d_gate, (long)n_gate * c.d, st);
  }
  const int nvec = norm_nvec(c), k = slot_of ? c.k : 1, rows = c.T * k;
  const int per_gate = n_gate ? c.T / n_gate : 1;
  const int per = norm_tokens_per_block(c), blocks = div_up(c.T, per);
  const auto* dv = static_cast<const u32x4*>(d_out);
  const auto* yv = static_cast<const u32x4*>(y);
  const auto* wv = static_cast<const u32x4*>(w);
  const auto* gv = static_cast<const u32x4*>(gate);
  auto* dyv = static_cast<u32x4*>(d_y);
  auto* drv = static_cast<u32x4*>(d_residual);
  float* partial = d_w || d_gate ? static_cast<float*>(ws) : nullptr;
  const float inv_d = 1.0f / (float)c.d;
  const bool past = norm_past(c, 2L * rows + (d_residual ? 2L : 1L) * c.T);
  with_types(c, [&](auto t) {
    using T = decltype(t);
    with_k(k, [&](auto kc) {
      constexpr int KC = decltype(kc)::value;
      if (norm_small(nvec))
        combine_norm_bwd_kernel<T, 2, 512, KC, (KC <= 8)>
            <<<blocks, norm_threads(nvec, 2), 0, st>>>(dv, yv, slot_of, topk_w, wv, gv, per_gate,
                                                       res_scale, rstd, dyv, d_topk_w, drv,
                                                       partial, nvec, inv_d, rows, k, c.T, per,
                                                       past);
      else
        combine_norm_bwd_kernel<T, 4, 512, KC, false>
            <<<blocks, norm_threads(nvec, 4), 0, st>>>(dv, yv, slot_of, topk_w, wv, gv, per_gate,
                                                       res_scale, rstd, dyv, d_topk_w, drv,
                                                       partial, nvec, inv_d, rows, k, c.T, per,
                                                       past);
    });
  });
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !partial) return e;
  return launch_param_grad(c, partial, w, gate, d_w, d_gate, n_gate, per, st);
}

}  // namespace moe
