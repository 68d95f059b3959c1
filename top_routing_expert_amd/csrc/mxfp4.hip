// MXFP4 quantisation, decoding into expert order, and the packed weight images
// of the 4-bit expert products (the format is described in mxfp4.h).
//
// quantize: the scale of a block of 32 is 2^(floor(log2 max|x|) - 2), so that
//   the largest element lands in [4, 8) and saturates at 6 in its upper
//   half: the exponent field of the float32 maximum minus 2, no logarithm.  A
//   maximum of 0, and one below 2^-125, gets 2^-127; a block that holds an
//   infinity or NaN gets the NaN scale and codes of 0.  Rows are a multiple of 32
//   long, so the tensor is one run of blocks: every thread holds 8 elements
//   (one 16-byte load of bf16, two of float32) and the four lanes of a block
//   exchange their maxima.
// dequantize: thread per 8 elements of an expert-ordered row p: codes and scale of
//   token src_of[p] / k (or of row p itself), values exact in bf16.
// Both are bound by HBM: T16384-d5120 quantised in 29..49 us (213 MB, as far as x is in the
// Infinity Cache), its 32768 rows of top-2 decoded in 61 us (380 MB, 6.3 TB/s).
#include "mxfp4.h"

namespace moe {

// 8 elements per thread; U independent groups in flight.
template <bool BF16, int U>
__global__ __launch_bounds__(256) void mx_quantize_kernel(const u32x4* __restrict__ x,
                                                          uint32_t* __restrict__ codes,
                                                          uint8_t* __restrict__ scales,
                                                          long groups) {
  const long base = (long)blockIdx.x * (256 * U) + threadIdx.x;
  u32x4 a[U], b[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const long g = base + 256 * u;
    if (g < groups) {
      if (BF16) {
        a[u] = x[g];
      } else {
        a[u] = x[2 * g];
        b[u] = x[2 * g + 1];
      }
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const long g = base + 256 * u;
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (BF16) {
        v[2 * i] = bf16_lo(a[u][i]);
        v[2 * i + 1] = bf16_hi(a[u][i]);
      } else {
        v[i] = __uint_as_float(a[u][i]);
        v[4 + i] = __uint_as_float(b[u][i]);
      }
    }
    // magnitudes compare as integers: infinities and NaN are the largest
    uint32_t top = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
    if (g >= groups) top = 0u;  // groups is a multiple of 4: a block is whole or absent
    top = max(top, (uint32_t)__shfl_xor((int)top, 1));
    top = max(top, (uint32_t)__shfl_xor((int)top, 2));
    const uint32_t e = top >> 23;  // biased exponent of the maximum
    const uint32_t sb = e == 255u ? 255u : e > 2u ? e - 2u : 0u;
    uint32_t c = 0u;
    if (e != 255u) {
      const float s = mx_scale(sb);
      c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[0], v[1], s, 0);
      c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2], v[3], s, 1);
      c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[4], v[5], s, 2);
      c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[6], v[7], s, 3);
    }
    if (g < groups) {
      codes[g] = c;
      if ((g & 3) == 0) scales[g >> 2] = (uint8_t)sb;
    }
  }
}

// Row p of x_perm from the codes of token src_of[p] / k (clamped), or of row p; U
// groups of 8 elements a thread, their loads in flight together.  past (the same for every
// thread): x_perm is stored past the 256 MB Infinity Cache, from kMxPastBytes of it on.
// Measured with the combine that reads it behind, k = 2, d = 5120: T16384 (335 MB) 177 -> 143
// us, T8192 77 -> 75, T4096 40 -> 41; the decoding of T16384 alone 84 -> 61.
constexpr long kMxPastBytes = 128L << 20;
template <bool BF16, int U>
__global__ __launch_bounds__(256) void mx_dequantize_kernel(
    const uint32_t* __restrict__ codes, const int32_t* __restrict__ src_of,
    const uint8_t* __restrict__ scales, int k, int T, uint32_t row_groups, uint32_t groups,
    u32x4* __restrict__ out, bool past) {
  // 32-bit indexes: T k d < 2^31 elements
  const uint32_t base = blockIdx.x * (256 * U) + threadIdx.x;
  uint32_t from[U], q[U];
  float s[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t i = min(base + 256 * u, groups - 1);
    const uint32_t p = i / row_groups, c = i - p * row_groups;
    const uint32_t t = src_of ? min(max(src_of[p] / k, 0), T - 1) : p;
    from[u] = t * row_groups + c;
  }
#pragma unroll
  for (int u = 0; u < U; ++u) q[u] = codes[from[u]];
#pragma unroll
  for (int u = 0; u < U; ++u) s[u] = mx_scale(scales[from[u] >> 2]);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t i = base + 256 * u;
    if (i >= groups) break;
    if constexpr (BF16) {
      u32x4 o;
      o.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q[u], s[u], 0));
      o.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q[u], s[u], 1));
      o.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q[u], s[u], 2));
      o.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q[u], s[u], 3));
      if (past) {
        asm volatile("");  // the compiler would make one ordinary store of the two
        __builtin_nontemporal_store(o, out + i);
        asm volatile("");
      } else {
        out[i] = o;
      }
    } else {
      f32x4* o = reinterpret_cast<f32x4*>(out) + 2 * (size_t)i;
      const auto v0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[u], s[u], 0);
      const auto v1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[u], s[u], 1);
      const auto v2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[u], s[u], 2);
      const auto v3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[u], s[u], 3);
      const f32x4 a = {v0[0], v0[1], v1[0], v1[1]}, b = {v2[0], v2[1], v3[0], v3[1]};
      if (past) {
        asm volatile("");
        __builtin_nontemporal_store(a, o);
        __builtin_nontemporal_store(b, o + 1);
        asm volatile("");
      } else {
        o[0] = a;
        o[1] = b;
      }
    }
  }
}

bool mx_rows_supported(const moe_config& c) { return c.d % kMxBlock == 0; }

hipError_t launch_mx_quantize(const moe_config& c, const void* x, void* codes, void* scales,
                              hipStream_t st) {
  const long groups = (long)c.T * c.d / 8;
  constexpr int U = 2;
  const int blocks = div_up(groups, 256 * U);
  const auto* xv = static_cast<const u32x4*>(x);
  auto* cv = static_cast<uint32_t*>(codes);
  auto* sv = static_cast<uint8_t*>(scales);
  if (c.dtype == MOE_BF16)
    mx_quantize_kernel<true, U><<<blocks, 256, 0, st>>>(xv, cv, sv, groups);
  else
    mx_quantize_kernel<false, U><<<blocks, 256, 0, st>>>(xv, cv, sv, groups);
  return hipGetLastError();
}

hipError_t launch_mx_dequantize(const moe_config& c, const void* codes, const int32_t* src_of,
                                const void* scales, void* x_perm, hipStream_t st) {
  const long rows = src_of ? (long)c.T * c.k : c.T;
  const long groups = rows * (c.d / 8);
  constexpr int U = 4;
  const int blocks = div_up(groups, 256 * U);
  const auto* cv = static_cast<const uint32_t*>(codes);
  const auto* sv = static_cast<const uint8_t*>(scales);
  auto* ov = static_cast<u32x4*>(x_perm);
  const bool past = groups * (c.dtype == MOE_BF16 ? 16 : 32) > kMxPastBytes;
  if (c.dtype == MOE_BF16)
    mx_dequantize_kernel<true, U><<<blocks, 256, 0, st>>>(cv, src_of, sv, c.k, c.T, c.d / 8,
                                                          (uint32_t)groups, ov, past);
  else
    mx_dequantize_kernel<false, U><<<blocks, 256, 0, st>>>(cv, src_of, sv, c.k, c.T, c.d / 8,
                                                           (uint32_t)groups, ov, past);
  return hipGetLastError();
}

// ------------------------------------------------------------------ packing
MxGeom mx_geom(const moe_config& c, bool gate_up) {
  MxGeom g;
  g.rows = gate_up ? 2L * c.f : c.d;
  const int K = gate_up ? c.d : c.f;
  g.steps = K / kMxStepK;
  g.codes_bytes = (size_t)g.rows * (K / 2);
  g.expert_bytes = g.codes_bytes + (size_t)g.rows * (K / kMxBlock);
  return g;
}

size_t mx_image_bytes(const moe_config& c, bool gate_up) {
  return (size_t)c.E * mx_geom(c, gate_up).expert_bytes;
}

// Source row of packed row r: 16 gate rows and the same 16 up rows in turn, or
// the row itself.  Returns the row within the expert; *second: the up matrix.
__device__ __forceinline__ long mx_source_row(long r, bool gate_up, bool* second) {
  if (!gate_up) {
    *second = false;
    return r;
  }
  *second = (r >> 4) & 1;
  return 16 * (r >> 5) + (r & 15);
}

// blockIdx.y: the expert.
__global__ __launch_bounds__(256) void mx_pack_kernel(
    const u32x4* __restrict__ c0, const uint32_t* __restrict__ s0, const u32x4* __restrict__ c1,
    const uint32_t* __restrict__ s1, bool gate_up, long R, int steps, char* __restrict__ image,
    size_t codes_bytes, size_t expert_bytes) {
  const long n_codes = R * steps * 4;  // 16-byte pieces
  const long n_scales = R * steps;     // dwords of four scales
  const size_t src0 = (size_t)blockIdx.y * (gate_up ? R / 2 : R);
  char* dst = image + (size_t)blockIdx.y * expert_bytes;
  auto* codes = reinterpret_cast<u32x4*>(dst);
  auto* scales = reinterpret_cast<uint32_t*>(dst + codes_bytes);
  for (long i = (long)blockIdx.x * 256 + threadIdx.x; i < n_codes + n_scales;
       i += (long)gridDim.x * 256) {
    bool second;
    if (i < n_codes) {
      const int p = (int)(i & 3), r16 = (int)((i >> 2) & 15);
      const long q = i >> 6;
      const int step = (int)(q % steps);
      const long row = mx_source_row(q / steps * 16 + r16, gate_up, &second);
      const int piece = p ^ ((r16 >> 2) & 3);
      codes[i] = (second ? c1 : c0)[((src0 + row) * steps + step) * 4 + piece];
    } else {
      const long j = i - n_codes, q = j >> 6;
      const int step = (int)(q % steps);
      const long row = mx_source_row(q / steps * 64 + (j & 63), gate_up, &second);
      scales[j] = (second ? s1 : s0)[(src0 + row) * steps + step];
    }
  }
}

hipError_t launch_pack_weights_mxfp4(const moe_config& c, const void* c0, const void* s0,
                                     const void* c1, const void* s1, bool gate_up, void* image,
                                     hipStream_t st) {
  const MxGeom g = mx_geom(c, gate_up);
  const long n = (g.rows * g.steps * 5 + 255) / 256;
  mx_pack_kernel<<<dim3((unsigned)(n < 4096 ? n : 4096), c.E), 256, 0, st>>>(
      static_cast<const u32x4*>(c0), static_cast<const uint32_t*>(s0),
      static_cast<const u32x4*>(c1), static_cast<const uint32_t*>(s1), gate_up, g.rows, g.steps,
      static_cast<char*>(image), g.codes_bytes, g.expert_bytes);
  return hipGetLastError();
}

}  // namespace moe
