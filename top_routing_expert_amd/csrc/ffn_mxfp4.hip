// Expert products on MXFP4 operands (format and images: mxfp4.h).
//
//   out[p, n] = sum_b 2^(ex[p, b] + ew[n, b] - 254) sum_{i in b} x[p, i] w[n, i]
// over the 32-wide blocks b of k, p an expert-ordered row; gate / up rows meet in
// SiLU(a) u.  gfx950 has the product in one instruction,
// v_mfma_scale_f32_32x32x64_f8f6f4 with both formats E2M1: lane l holds row
// l & 31 and the 32 k of half l >> 5 of a 64-wide step -- one scale block, 16
// bytes -- and that block's scale byte, selected by the instruction from a
// register.  Accumulation is float32.
//
// Tile: TW packed weight rows x TM token rows of one expert, 128-wide k stages
// (64 code bytes and one dword of four scales per row) in a ring in LDS, filled by the LDS-DMA
// load.  The weight image holds 16-row x 128-k chunks of 1 KB in LDS order, so
// a wave's copy is 1 KB of consecutive bytes; token rows are copied (and
// gathered through src_of) from row-major codes.  16-byte pieces are swizzled
// with (row >> 2) & 3, so the fragment reads of 16 lanes spread over the banks.
#include <type_traits>

#include "mxfp4.h"
#include "tiles.h"

namespace moe {

typedef __attribute__((address_space(3))) void mx_lds_t;
typedef int i32x8 __attribute__((ext_vector_type(8)));

// Direct global -> LDS copies of 16 or 4 bytes per lane from sbase + voff (lane L
// writes LDS bytes [lds + 16 L, + 16) or [lds + 4 L, + 4); `sbase` and `lds`
// wave-uniform); waited for by the kernel's explicit vmcnt counts.
__device__ __forceinline__ void mx_dma16(const void* sbase, uint32_t voff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(voff), "s"(sbase),
               "s"(lds)
               : "memory", "m0");
}
__device__ __forceinline__ void mx_dma4(const void* sbase, uint32_t voff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\tglobal_load_lds_dword %0, %1" ::"v"(voff), "s"(sbase),
               "s"(lds)
               : "memory", "m0");
}
template <int N>
__device__ __forceinline__ void mx_wait_vm_barrier() {
  asm volatile("s_waitcnt vmcnt(%0)\n\ts_waitcnt lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// GW x GT waves, each WA x WB fragments of 32 weight rows x 32 tokens.
template <bool GATED, int GW, int GT, int WA, int WB, int STAGES>
struct MxTile {
  static constexpr int NW = GW * GT;
  static constexpr int TW = 32 * GW * WA, TM = 32 * GT * WB;
  static constexpr int ROWS = TW + TM;
  static constexpr int CODE_CHUNKS = ROWS / 16;          // 1 KB copies per stage
  static constexpr int CPW = CODE_CHUNKS / NW;           // per wave
  static constexpr int SCALE_CHUNKS = ROWS / 64;         // 256-byte copies per stage
  static constexpr int SPW = (SCALE_CHUNKS + NW - 1) / NW;
  static constexpr int DPW = CPW + SPW;                  // copies per wave and stage
  static constexpr int STAGE_BYTES = ROWS * 68;
  static_assert(CODE_CHUNKS % NW == 0 && ROWS % 64 == 0 && TW % 64 == 0, "stage split");
  static_assert(STAGES * STAGE_BYTES <= 156 * 1024, "LDS ring too large");
  static_assert(STAGES >= 3 && STAGES <= 6, "ring depth");
  static_assert((STAGES - 2) * DPW <= 63, "vmcnt range");
};

template <bool GATED, int GW, int GT, int WA, int WB, int STAGES, int BLOCKS>
__global__ __launch_bounds__(64 * GW * GT, BLOCKS * GW * GT / 4) void mxfp4_gemm_kernel(
    const uint8_t* __restrict__ xc, const uint8_t* __restrict__ xs,
    const int32_t* __restrict__ src_of, int gk, int gtokens, const int32_t* __restrict__ offs,
    const uint8_t* __restrict__ image, size_t codes_bytes, size_t expert_bytes,
    uint16_t* __restrict__ out, int E, int R, int N, int K, int rows, int n_tiles, int band) {
  using G = MxTile<GATED, GW, GT, WA, WB, STAGES>;
  constexpr int TW = G::TW, TM = G::TM, ROWS = G::ROWS, NW = G::NW;
  __shared__ __attribute__((aligned(16))) unsigned char ring[STAGES * G::STAGE_BYTES];
  __shared__ int s_tile[4];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  if (wave == 0) place_tile<TM>(offs, E, rows, n_tiles, band, lane, s_tile);
  __syncthreads();
  const int e = __builtin_amdgcn_readfirstlane(s_tile[0]);
  if (e < 0) return;  // block-uniform
  const int row0 = __builtin_amdgcn_readfirstlane(s_tile[1]);
  const int row_end = __builtin_amdgcn_readfirstlane(s_tile[2]);
  const int n_tile = __builtin_amdgcn_readfirstlane(s_tile[3]);
  const int pr0 = n_tile * TW;  // first packed row of the tile
  const int nk = K / kMxStepK;  // stages

  // ---- copies of this wave: code chunks wave + NW i (weight chunks first), then
  // scale chunks wave + NW i (the last one repeated where they do not come out
  // even: the same bytes to the same place).  Rows past the expert's last
  // packed row or token read a real row and feed outputs that are not stored.
  // Offsets are 32-bit: a weight chunk's base is a 64-bit scalar, T rows of codes
  // are below 2^31 bytes.
  auto token_of = [&](int r) {
    const int p = min(row0 + r, row_end - 1);
    return src_of ? min(max(src_of[p] / gk, 0), gtokens - 1) : p;
  };
  const uint8_t* we = image + (size_t)e * expert_bytes;
  const uint8_t* wse = we + codes_bytes;
  uint32_t voff[G::CPW], soff[G::SPW];
#pragma unroll
  for (int i = 0; i < G::CPW; ++i) {
    const int r = 16 * (wave + NW * i);
    if (r < TW) {
      voff[i] = 16u * lane;
    } else {
      const int rr = lane >> 2;  // row of the chunk
      voff[i] = (uint32_t)token_of(r - TW + rr) * (uint32_t)(K / 2) +
                16u * (uint32_t)((lane & 3) ^ ((rr >> 2) & 3));
    }
  }
#pragma unroll
  for (int i = 0; i < G::SPW; ++i) {
    const int r = 64 * min(wave + NW * i, G::SCALE_CHUNKS - 1);
    soff[i] = r < TW ? 4u * lane : (uint32_t)token_of(r - TW + lane) * (uint32_t)(K / 32);
  }
  const uint32_t lds0 = (uint32_t)(size_t)(const mx_lds_t*)ring;
  auto issue = [&](int kt) {
    const uint32_t sb = lds0 + (uint32_t)(kt % STAGES) * (uint32_t)G::STAGE_BYTES;
#pragma unroll
    for (int i = 0; i < G::CPW; ++i) {
      const int c = wave + NW * i;  // wave-uniform
      const uint8_t* base =
          16 * c < TW ? we + ((size_t)min(pr0 / 16 + c, R / 16 - 1) * nk + kt) * 1024
                      : xc + (size_t)kt * 64;
      mx_dma16(base, voff[i], sb + (uint32_t)c * 1024u);
    }
#pragma unroll
    for (int i = 0; i < G::SPW; ++i) {
      const int c = min(wave + NW * i, G::SCALE_CHUNKS - 1);
      const uint8_t* base =
          64 * c < TW ? wse + ((size_t)min(pr0 / 64 + c, R / 64 - 1) * nk + kt) * 256
                      : xs + (size_t)kt * 4;
      mx_dma4(base, soff[i], sb + (uint32_t)(ROWS * 64) + (uint32_t)c * 256u);
    }
  };

  // ---- fragments
  const int wn = wave / GT, wm = wave % GT;
  const int lk = lane >> 5;
  const int arow0 = wn * 32 * WA + (lane & 31);
  const int tok0 = wm * 32 * WB;
  const int jn =
      __builtin_amdgcn_readfirstlane(min(WB, max(0, (row_end - row0 - tok0 + 31) >> 5)));
  const int brow0 = TW + tok0 + (lane & 31);

  f32x16 acc[WA][WB];
#pragma unroll
  for (int i = 0; i < WA; ++i)
#pragma unroll
    for (int j = 0; j < WB; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;

  auto wait_later = [&](int later) {  // all stages but the `later` youngest are in
    switch (later) {
      case 0: mx_wait_vm_barrier<0>(); break;
      case 1: mx_wait_vm_barrier<G::DPW>(); break;
      case 2: mx_wait_vm_barrier<2 * G::DPW>(); break;
      case 3: mx_wait_vm_barrier<3 * G::DPW>(); break;
      default: mx_wait_vm_barrier<4 * G::DPW>(); break;
    }
  };
  auto main_loop = [&](auto jn_c) {
    constexpr int JN = decltype(jn_c)::value;
    struct Frags {
      u32x4 a[WA][2], b[WB][2];
      uint32_t as[WA], bs[WB];
    };
    auto load_frags = [&](int kt, Frags& F) {
      const unsigned char* sb = ring + (kt % STAGES) * G::STAGE_BYTES;
      auto piece = [&](int row, int q) {
        return *reinterpret_cast<const u32x4*>(sb + row * 64 + ((q ^ ((row >> 2) & 3)) << 4));
      };
      auto scale = [&](int row) {  // this lane's two scales in bytes 0 and 2
        return *reinterpret_cast<const uint32_t*>(sb + ROWS * 64 + row * 4) >> (8 * lk);
      };
#pragma unroll
      for (int i = 0; i < WA; ++i) {
        F.a[i][0] = piece(arow0 + 32 * i, lk);
        F.a[i][1] = piece(arow0 + 32 * i, 2 + lk);
        F.as[i] = scale(arow0 + 32 * i);
      }
#pragma unroll
      for (int j = 0; j < JN; ++j) {
        F.b[j][0] = piece(brow0 + 32 * j, lk);
        F.b[j][1] = piece(brow0 + 32 * j, 2 + lk);
        F.bs[j] = scale(brow0 + 32 * j);
      }
    };
    auto wide = [](u32x4 v) -> i32x8 {  // E2M1 operands use the first four registers
      return i32x8{(int)v.x, (int)v.y, (int)v.z, (int)v.w, 0, 0, 0, 0};
    };
    auto mfma_stage = [&](const Frags& F) {
#pragma unroll
      for (int j = 0; j < JN; ++j)
#pragma unroll
        for (int i = 0; i < WA; ++i)
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
              wide(F.a[i][0]), wide(F.b[j][0]), acc[i][j], 4, 4, 0, (int)F.as[i], 0, (int)F.bs[j]);
#pragma unroll
      for (int j = 0; j < JN; ++j)
#pragma unroll
        for (int i = 0; i < WA; ++i)
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
              wide(F.a[i][1]), wide(F.b[j][1]), acc[i][j], 4, 4, 2, (int)F.as[i], 2, (int)F.bs[j]);
    };
    // Stage kt sits in ring slot kt % STAGES; its fragments are read during
    // step kt - 1.  End of step kt: wait for this wave's copies of stage kt + 2,
    // barrier (every wave's copies of kt + 2 are in and nobody reads stage kt any more),
    // then refill its slot with stage kt + STAGES.
#pragma unroll
    for (int i = 0; i < STAGES; ++i)
      if (i < nk) issue(i);
    wait_later(max(0, min(nk - 1, STAGES - 1) - 1));  // stages 0 and 1 are in
    Frags F0, F1;
    if (JN > 0) load_frags(0, F0);
    auto step = [&](int kt, Frags& cur, Frags& nxt) {
      if (JN > 0) {
        load_frags(min(kt + 1, nk - 1), nxt);  // the last step re-reads its own stage
        mfma_stage(cur);
      }
      if (kt + 2 < nk)
        wait_later(min(nk - 1, kt + STAGES - 1) - (kt + 2));
      else
        mx_wait_vm_barrier<0>();
      if (kt + STAGES < nk) issue(kt + STAGES);
    };
    for (int kt = 0; kt < nk; kt += 2) {
      step(kt, F0, F1);
      if (kt + 1 < nk) step(kt + 1, F1, F0);
    }
  };
  switch (jn) {
    case 0: main_loop(std::integral_constant<int, 0>()); break;
    case 1: main_loop(std::integral_constant<int, 1>()); break;
    case 2: main_loop(std::integral_constant<int, (WB >= 2 ? 2 : WB)>()); break;
    case 3: main_loop(std::integral_constant<int, (WB >= 3 ? 3 : WB)>()); break;
    default: main_loop(std::integral_constant<int, WB>()); break;
  }

  // ---- epilogue: acc[i][j][4 g + r] = C[fragment-i row 8 g + 4 lk + r][token lane & 31]
#pragma unroll
  for (int j = 0; j < WB; ++j) {
    const int p = row0 + tok0 + 32 * j + (lane & 31);
    if (j >= jn || p >= row_end) continue;
#pragma unroll
    for (int i = 0; i < WA; ++i) {
      const int prf = pr0 + wn * 32 * WA + 32 * i;  // first packed row of the fragment
      if (prf >= R) continue;
      if constexpr (GATED) {  // rows 0..15 gate, 16..31 up of the same 16 features
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          float hv[4];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float a = acc[i][j][4 * g + r], u = acc[i][j][4 * g + 8 + r];
            hv[r] = a * __builtin_amdgcn_rcpf(1.0f + __expf(-a)) * u;
          }
          u32x2 pk;
          pk.x = pack_bf16x2(hv[0], hv[1]);
          pk.y = pack_bf16x2(hv[2], hv[3]);
          *reinterpret_cast<u32x2*>(out + (size_t)p * N + prf / 2 + 8 * g + 4 * lk) = pk;
        }
      } else {
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          u32x2 pk;
          pk.x = pack_bf16x2(acc[i][j][4 * g], acc[i][j][4 * g + 1]);
          pk.y = pack_bf16x2(acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]);
          *reinterpret_cast<u32x2*>(out + (size_t)p * N + prf + 8 * g + 4 * lk) = pk;
        }
      }
    }
  }
}

template <bool GATED, int GW, int GT, int WA, int WB, int STAGES, int BLOCKS>
static hipError_t launch_tile(const moe_config& c, const void* codes, const void* scales,
                              const int32_t* src_of, const int32_t* offs, const void* image,
                              void* out, hipStream_t st) {
  using G = MxTile<GATED, GW, GT, WA, WB, STAGES>;
  const MxGeom g = mx_geom(c, GATED);
  const long rows = (long)c.T * c.k;
  const int n_tiles = div_up(g.rows, G::TW);
  const long total = (long)n_tiles * worst_row_tiles(rows, c.E, G::TM);
  const int blocks = (int)((total + 7) / 8 * 8);
  mxfp4_gemm_kernel<GATED, GW, GT, WA, WB, STAGES, BLOCKS><<<blocks, 64 * GW * GT, 0, st>>>(
      static_cast<const uint8_t*>(codes), static_cast<const uint8_t*>(scales), src_of, c.k, c.T,
      offs, static_cast<const uint8_t*>(image), g.codes_bytes, g.expert_bytes,
      static_cast<uint16_t*>(out), c.E, (int)g.rows,
      GATED ? c.f : c.d, GATED ? c.d : c.f, (int)rows, n_tiles, 8);
  return hipGetLastError();
}

template <bool GATED>
static hipError_t launch_mx_gemm(const moe_config& c, const void* codes, const void* scales,
                                 const int32_t* src_of, const int32_t* offs, const void* image,
                                 void* out, hipStream_t st) {
  const long rows = (long)c.T * c.k;
  if (rows >= 128L * c.E)
    return launch_tile<GATED, 4, 2, 2, 4, 4, 1>(c, codes, scales, src_of, offs, image, out, st);
  return launch_tile<GATED, 4, 1, 1, 2, 4, 2>(c, codes, scales, src_of, offs, image, out, st);
}

hipError_t launch_ffn_gate_up_mxfp4(const moe_config& c, const void* x_codes, const void* x_scales,
                                    const int32_t* src_of, const int32_t* offs, const void* image,
                                    void* h, hipStream_t st) {
  return launch_mx_gemm<true>(c, x_codes, x_scales, src_of, offs, image, h, st);
}

hipError_t launch_ffn_down_mxfp4(const moe_config& c, const void* h_codes, const void* h_scales,
                                 const int32_t* offs, const void* image, void* y, hipStream_t st) {
  return launch_mx_gemm<false>(c, h_codes, h_scales, nullptr, offs, image, y, st);
}

}  // namespace moe
