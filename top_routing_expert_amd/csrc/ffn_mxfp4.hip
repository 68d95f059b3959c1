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
// (64 code bytes per row, one dword of four scales) in a ring in LDS, filled by the
// LDS-DMA load.  The weight image holds 16-row x 128-k chunks of 1 KB in LDS
// order, so a wave's copy is 1 KB of consecutive bytes; token rows are copied
// (and gathered through src_of) from row-major codes.  16-byte pieces are
// swizzled with (row >> 2) & 3, so the fragment reads of 16 lanes spread over
// the banks.  The token rows' scales, 4 bytes in a line of their own per row and
// stage, are copied 16 bytes a row for four stages at a time where K allows it.
//
// Persistent: a block walks its tiles in rounds as the bf16 kernel's blocks do
// (neighbours in the tile order run on one XCD at the same time), and starts the
// copies of its next tile before it stores the current one.
//
// 256 x 256 with eight waves (64 x 128 each) where an expert has 128 rows or more:
// the largest tile that a ring of four stages leaves LDS for.  A stage takes 1.1 us,
// of which its MFMAs fill 0.43: bound by the copies into LDS (33 KB a stage and CU,
// 7..8 TB/s over the chip) and the fragment reads beside them.  Measured, products alone:
// T8192-d7168-E64 top-8 f2048 gate / up 1140 us (3.4 PFLOP/s; 256 x 128 1331, 128 x 256
// 1455, 128 x 128 on four or eight waves 1818 and 1695), T1024-d4096-E8 top-2 f11008 down
// 84 us (101, 110, 135, 125; 104 with the weights from HBM).  Below 128 rows an expert
// 128 x 64, two blocks a CU: the weights are read once whatever the tile, and more blocks
// read them together (T37-d5120-E16 23 us, 5.8 TB/s).
#include <algorithm>
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

// GW x GT waves, each WA x WB fragments of 32 weight rows x 32 tokens.  S4: token
// scales by groups of four stages, in a double buffer of their own.
template <int GW, int GT, int WA, int WB, int STAGES, bool S4>
struct MxTile {
  static constexpr int NW = GW * GT;
  static constexpr int TW = 32 * GW * WA, TM = 32 * GT * WB;
  static constexpr int ROWS = TW + TM;
  static constexpr int CPW = ROWS / 16 / NW;             // 1 KB code copies per wave and stage
  static constexpr int SROWS = S4 ? TW : ROWS;           // rows with scales in the ring
  static constexpr int SCALE_CHUNKS = SROWS / 64;        // 256-byte copies per stage
  static constexpr int SPW = (SCALE_CHUNKS + NW - 1) / NW;
  static constexpr int DPW = CPW + SPW;                  // copies per wave and stage
  static constexpr int STAGE_BYTES = ROWS * 64 + SROWS * 4;
  static constexpr int RING_BYTES = STAGES * STAGE_BYTES;
  static constexpr int GROUP_BYTES = S4 ? TM * 16 : 0;   // token scales of four stages
  static constexpr int GROUP_CHUNKS = S4 ? TM / 64 : 0;  // 1 KB copies per group
  static constexpr int GPW = (GROUP_CHUNKS + NW - 1) / NW;
  static_assert(TW % (16 * NW) == 0 && TM % (16 * NW) == 0 && ROWS % 64 == 0 && TW % 64 == 0 &&
                    TM % 64 == 0,
                "stage split");
  static_assert(RING_BYTES + 2 * GROUP_BYTES + 12 * kTileTableMax + 64 <= 160 * 1024, "LDS");
  static_assert(STAGES >= 3 && STAGES <= 5, "ring depth");
  static_assert((STAGES - 1) * DPW + GPW <= 63, "vmcnt range");
};

// Four features each of groups g (a) and g + 1 (b) of a token, the first four of a group in
// lanes 0..31 and the next four in lanes 32..63 -> all eight of g in lanes 0..31 and of
// g + 1 in lanes 32..63, for one 16-byte store.
__device__ __forceinline__ u32x4 mx_join(u32x2 a, u32x2 b) {
  const auto x = __builtin_amdgcn_permlane32_swap(a.x, b.x, false, false);
  const auto y = __builtin_amdgcn_permlane32_swap(a.y, b.y, false, false);
  return u32x4{x[0], y[0], x[1], y[1]};
}

template <bool GATED, int GW, int GT, int WA, int WB, int STAGES, int BLOCKS, bool S4>
__global__ __launch_bounds__(64 * GW * GT, BLOCKS * GW * GT / 4) void mxfp4_gemm_kernel(
    const uint8_t* __restrict__ xc, const uint8_t* __restrict__ xs,
    const int32_t* __restrict__ src_of, int gk, int gtokens, const int32_t* __restrict__ offs,
    const uint8_t* __restrict__ image, size_t codes_bytes, size_t expert_bytes,
    uint16_t* __restrict__ out, int E, int R, int N, int K, int rows, int n_tiles, int band) {
  using G = MxTile<GW, GT, WA, WB, STAGES, S4>;
  constexpr int TW = G::TW, TM = G::TM, ROWS = G::ROWS, NW = G::NW;
  __shared__ __attribute__((aligned(16))) unsigned char lds[G::RING_BYTES + 2 * G::GROUP_BYTES];
  __shared__ int s_o0[kTileTableMax], s_o1[kTileTableMax], s_start[kTileTableMax];
  __shared__ int s_tile[2][4];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int nk = K / kMxStepK;  // stages
  const int grid = (int)gridDim.x;  // a multiple of 8
  const int qp = (grid >> 3) * (int)(blockIdx.x & 7) + (int)(blockIdx.x >> 3);
  int total = 0;  // tiles (wave 0 only)
  // tile of this block in a round, into s_tile[round & 1] (expert -1: none); wave 0
  auto place = [&](int round) {
    int* t = s_tile[round & 1];
    const int L = round * grid + ((round & 1) ? grid - 1 - qp : qp);
    if (lane == 0) t[0] = -1;
    if (L < total) locate_in_table<TM>(s_o0, s_o1, s_start, E, n_tiles, band, L, lane, t);
  };
  if (wave == 0) {  // the table is written and read by this one wave
    total = build_tile_table<TM>(offs, E, rows, n_tiles, lane, s_o0, s_o1, s_start);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    place(0);
  }
  __syncthreads();

  // ---- copies of this wave: code chunks wave + NW i (weight chunks first), then
  // scale chunks wave + NW i, and every fourth stage a chunk of token scales (the
  // last one repeated where they do not come out even: the same bytes to the same
  // place).  Rows past the expert's last packed row or token read a real row and
  // feed outputs that are not stored.  Offsets are 32-bit: a weight chunk's base
  // is a 64-bit scalar, T rows of codes are below 2^31 bytes.
  constexpr int WCH = TW / (16 * NW);  // weight chunks of a wave; then token chunks
  struct Tile {
    int row0, row_end, pr0;  // token rows, first packed row
  };
  uint32_t voff[G::CPW], soff[G::SPW], goff[S4 ? G::GPW : 1];
  const uint8_t* cbase[G::CPW];
  const uint8_t* sbase[G::SPW];
  uint32_t sstep[G::SPW];
  auto open = [&](int round, Tile* t) {
    const int* st = s_tile[round & 1];
    const int e = __builtin_amdgcn_readfirstlane(st[0]);
    if (e < 0) return false;  // block-uniform; later rounds only hold larger tile numbers
    t->row0 = __builtin_amdgcn_readfirstlane(st[1]);
    t->row_end = __builtin_amdgcn_readfirstlane(st[2]);
    t->pr0 = __builtin_amdgcn_readfirstlane(st[3]) * TW;
    auto token_of = [&](int r) {
      const int p = min(t->row0 + r, t->row_end - 1);
      return src_of ? min(max(src_of[p] / gk, 0), gtokens - 1) : p;
    };
    const uint8_t* we = image + (size_t)e * expert_bytes;
    const uint8_t* wse = we + codes_bytes;
#pragma unroll
    for (int i = 0; i < G::CPW; ++i) {
      const int c = wave + NW * i;
      if (i < WCH) {
        cbase[i] = we + (size_t)min(t->pr0 / 16 + c, R / 16 - 1) * nk * 1024;
        voff[i] = 16u * lane;
      } else {
        const int rr = lane >> 2;  // row of the chunk
        cbase[i] = xc;
        voff[i] = (uint32_t)token_of(16 * c - TW + rr) * (uint32_t)(K / 2) +
                  16u * (uint32_t)((lane & 3) ^ ((rr >> 2) & 3));
      }
    }
#pragma unroll
    for (int i = 0; i < G::SPW; ++i) {
      const int c = min(wave + NW * i, G::SCALE_CHUNKS - 1);
      const bool weight = S4 || 64 * c < TW;  // wave-uniform
      sbase[i] = weight ? wse + (size_t)min(t->pr0 / 64 + c, R / 64 - 1) * nk * 256 : xs;
      sstep[i] = weight ? 256u : 4u;
      soff[i] = weight ? 4u * lane : (uint32_t)token_of(64 * c - TW + lane) * (uint32_t)(K / 32);
    }
    if constexpr (S4) {
#pragma unroll
      for (int i = 0; i < G::GPW; ++i)
        goff[i] = (uint32_t)token_of(64 * min(wave + NW * i, G::GROUP_CHUNKS - 1) + lane) *
                  (uint32_t)(K / 32);
    }
    return true;
  };
  const uint32_t lds0 = (uint32_t)(size_t)(const mx_lds_t*)lds;
  // `group`: whether stage kt begins a group of token scales
  auto issue = [&](int kt, bool group) {
    const uint32_t sb = lds0 + (uint32_t)(kt % STAGES) * (uint32_t)G::STAGE_BYTES;
#pragma unroll
    for (int i = 0; i < G::CPW; ++i)
      mx_dma16(cbase[i] + (size_t)kt * (i < WCH ? 1024 : 64), voff[i],
               sb + (uint32_t)(wave + NW * i) * 1024u);
#pragma unroll
    for (int i = 0; i < G::SPW; ++i)
      mx_dma4(sbase[i] + (size_t)kt * sstep[i], soff[i],
              sb + (uint32_t)(ROWS * 64) +
                  (uint32_t)min(wave + NW * i, G::SCALE_CHUNKS - 1) * 256u);
    if constexpr (S4) {
      if (group) {  // one copy more: the waits, which count without it, are early
#pragma unroll
        for (int i = 0; i < G::GPW; ++i)
          mx_dma16(xs + (size_t)kt * 4, goff[i],
                   lds0 + (uint32_t)G::RING_BYTES + (uint32_t)((kt / 4) & 1) * G::GROUP_BYTES +
                       (uint32_t)min(wave + NW * i, G::GROUP_CHUNKS - 1) * 1024u);
      }
    }
  };

  // ---- fragments
  const int wn = wave / GT, wm = wave % GT;
  const int lk = lane >> 5;
  const int arow0 = wn * 32 * WA + (lane & 31);
  const int tok0 = wm * 32 * WB;
  const int brow0 = TW + tok0 + (lane & 31);
  f32x16 acc[WA][WB];

  auto wait_later = [&](int later) {  // all stages but the `later` youngest are in
    switch (later) {
      case 0: mx_wait_vm_barrier<0>(); break;
      case 1: mx_wait_vm_barrier<G::DPW>(); break;
      case 2: mx_wait_vm_barrier<2 * G::DPW>(); break;
      case 3: mx_wait_vm_barrier<3 * G::DPW>(); break;
      case 4: mx_wait_vm_barrier<4 * G::DPW>(); break;
      default: mx_wait_vm_barrier<0>(); break;
    }
  };
  auto begin = [&] {  // the first stages of a tile
#pragma unroll
    for (int i = 0; i < STAGES; ++i)
      if (i < nk) issue(i, i % 4 == 0);
  };
  auto main_loop = [&](auto jn_c) {
    constexpr int JN = decltype(jn_c)::value;
    struct Half {  // the fragments of one 64-wide step
      u32x4 a[WA], b[WB];
    };
    struct Scales {  // of a stage, four bytes a row
      uint32_t a[WA], b[WB];
    };
    auto stage_at = [&](int kt) { return lds + (kt % STAGES) * G::STAGE_BYTES; };
    auto read_half = [&](int kt, int h, Half& F) {
      const unsigned char* sb = stage_at(kt);
      auto piece = [&](int row) {
        return *reinterpret_cast<const u32x4*>(sb + row * 64 +
                                               (((2 * h + lk) ^ ((row >> 2) & 3)) << 4));
      };
#pragma unroll
      for (int i = 0; i < WA; ++i) F.a[i] = piece(arow0 + 32 * i);
#pragma unroll
      for (int j = 0; j < JN; ++j) F.b[j] = piece(brow0 + 32 * j);
    };
    auto read_scales = [&](int kt, Scales& S) {
      const unsigned char* sb = stage_at(kt) + ROWS * 64;
#pragma unroll
      for (int i = 0; i < WA; ++i)
        S.a[i] = *reinterpret_cast<const uint32_t*>(sb + (arow0 + 32 * i) * 4);
      const unsigned char* tb = S4 ? lds + G::RING_BYTES + ((kt / 4) & 1) * G::GROUP_BYTES +
                                         (kt % 4) * 4 - TW * 16
                                   : sb;
#pragma unroll
      for (int j = 0; j < JN; ++j)
        S.b[j] = *reinterpret_cast<const uint32_t*>(tb + (brow0 + 32 * j) * (S4 ? 16 : 4));
    };
    auto wide = [](u32x4 v) -> i32x8 {  // E2M1 operands use the first four registers
      return i32x8{(int)v.x, (int)v.y, (int)v.z, (int)v.w, 0, 0, 0, 0};
    };
    // a lane's scale of half h is byte 2 h + lk; shifted here and not behind the
    // read, which would make the reads wait before the MFMAs they hide under
    auto mfma_half = [&](const Half& F, const Scales& S, auto h_c) {
      constexpr int H = decltype(h_c)::value;
      int as[WA], bs[WB];
#pragma unroll
      for (int i = 0; i < WA; ++i) as[i] = (int)(S.a[i] >> (8 * lk));
#pragma unroll
      for (int j = 0; j < JN; ++j) bs[j] = (int)(S.b[j] >> (8 * lk));
#pragma unroll
      for (int j = 0; j < JN; ++j)
#pragma unroll
        for (int i = 0; i < WA; ++i)
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
              wide(F.a[i]), wide(F.b[j]), acc[i][j], 4, 4, 2 * H, as[i], 2 * H, bs[j]);
    };
    // Stage kt sits in ring slot kt % STAGES.  Step kt: its second half is read
    // while the first half's MFMAs run; then the wait for stage kt + 1 and the
    // barrier (every wave's copies of kt + 1 are in and stage kt is in
    // registers), the refill of the slot with stage kt + STAGES, and the first half
    // of stage kt + 1 is read while the second half's MFMAs run.  (A token-scale
    // group's buffer is refilled two groups later.)
    //
    // The MFMAs are pinned between the reads they cover and the next wait: they
    // touch no memory, so the compiler is free to move them behind the barrier, where
    // nothing would hide under them any more (T8192-E64 gate / up 1304 ->
    // 1225 us).  Within the unrolled loop, one basic block, the scheduling barriers
    // do; at the end of a tile the accumulators pass through empty asm.
    const auto H0 = std::integral_constant<int, 0>();
    const auto H1 = std::integral_constant<int, 1>();
    Half P, Q;
    Scales SA, SB;
    wait_later(min(nk, STAGES) - 1);  // stage 0 is in
    if (JN > 0) {
      read_half(0, 0, P);
      read_scales(0, SA);
    }
    auto step = [&](int kt, int u, const Scales& cur, Scales& nxt, auto full_c) {
      constexpr bool FULL = decltype(full_c)::value;  // kt + u + STAGES < nk; kt % 4 == 0
      const int s = kt + u;
      if (JN > 0) {
        read_half(s, 1, Q);
        __builtin_amdgcn_sched_barrier(0);
        mfma_half(P, cur, H0);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (!FULL) {
#pragma unroll
          for (int j = 0; j < JN; ++j)
#pragma unroll
            for (int i = 0; i < WA; ++i) asm volatile("" : "+v"(acc[i][j]));
        }
      }
      if constexpr (FULL) {
        mx_wait_vm_barrier<(STAGES - 2) * G::DPW>();
        issue(s + STAGES, (u + STAGES) % 4 == 0);
      } else {
        wait_later(max(0, min(nk - 1, s + STAGES - 1) - (s + 1)));
        if (s + STAGES < nk) issue(s + STAGES, (s + STAGES) % 4 == 0);
      }
      if (JN > 0) {
        const int n = FULL ? s + 1 : min(s + 1, nk - 1);  // past the end: any stage
        read_half(n, 0, P);
        read_scales(n, nxt);
        __builtin_amdgcn_sched_barrier(0);
        mfma_half(Q, cur, H1);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    int kt = 0;
    for (; kt + 3 + STAGES < nk; kt += 4) {
      step(kt, 0, SA, SB, std::true_type());
      step(kt, 1, SB, SA, std::true_type());
      step(kt, 2, SA, SB, std::true_type());
      step(kt, 3, SB, SA, std::true_type());
    }
    for (; kt < nk; kt += 2) {
      step(kt, 0, SA, SB, std::false_type());
      if (kt + 1 < nk) step(kt, 1, SB, SA, std::false_type());
    }
    // the last reads are done before the ring is filled for the next tile
    mx_wait_vm_barrier<0>();
  };

  Tile cur{};
  bool more = open(0, &cur);
  if (more) begin();
  for (int round = 0; more; ++round) {
    const int jn =
        __builtin_amdgcn_readfirstlane(min(WB, max(0, (cur.row_end - cur.row0 - tok0 + 31) >> 5)));
#pragma unroll
    for (int i = 0; i < WA; ++i)
#pragma unroll
      for (int j = 0; j < WB; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
    if (wave == 0) place(round + 1);  // read after the main loop's barriers
    switch (jn) {
      case 0: main_loop(std::integral_constant<int, 0>()); break;
      case 1: main_loop(std::integral_constant<int, 1>()); break;
      case 2: main_loop(std::integral_constant<int, (WB >= 2 ? 2 : WB)>()); break;
      case 3: main_loop(std::integral_constant<int, (WB >= 3 ? 3 : WB)>()); break;
      default: main_loop(std::integral_constant<int, WB>()); break;
    }
    // every wave has read its last fragments and no copy is in flight: the next
    // tile's copies run under this one's stores
    const Tile t = cur;
    more = open(round + 1, &cur);
    if (more) begin();

    // ---- epilogue: acc[i][j][4 g + r] = C[fragment-i row 8 g + 4 lk + r][token lane & 31]
#pragma unroll
    for (int j = 0; j < WB; ++j) {
      const int p = t.row0 + tok0 + 32 * j + (lane & 31);
      if (j >= jn || p >= t.row_end) continue;
#pragma unroll
      for (int i = 0; i < WA; ++i) {
        const int prf = t.pr0 + wn * 32 * WA + 32 * i;  // first packed row of the fragment
        if (prf >= R) continue;
        if constexpr (GATED) {  // rows 0..15 gate, 16..31 up of the same 16 features
          u32x2 pk[2];
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            float hv[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const float a = acc[i][j][4 * g + r], u = acc[i][j][4 * g + 8 + r];
              hv[r] = a * __builtin_amdgcn_rcpf(1.0f + __expf(-a)) * u;
            }
            pk[g].x = pack_bf16x2(hv[0], hv[1]);
            pk[g].y = pack_bf16x2(hv[2], hv[3]);
          }
          *reinterpret_cast<u32x4*>(out + (size_t)p * N + prf / 2 + 8 * lk) = mx_join(pk[0], pk[1]);
        } else {
#pragma unroll
          for (int g = 0; g < 4; g += 2) {
            u32x2 pk[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int r = 4 * (g + h);
              pk[h].x = pack_bf16x2(acc[i][j][r], acc[i][j][r + 1]);
              pk[h].y = pack_bf16x2(acc[i][j][r + 2], acc[i][j][r + 3]);
            }
            *reinterpret_cast<u32x4*>(out + (size_t)p * N + prf + 8 * (g + lk)) =
                mx_join(pk[0], pk[1]);
          }
        }
      }
    }
  }
}

template <bool GATED, int GW, int GT, int WA, int WB, int STAGES, int BLOCKS, bool S4>
static hipError_t launch_tile(const moe_config& c, const void* codes, const void* scales,
                              const int32_t* src_of, const int32_t* offs, const void* image,
                              void* out, hipStream_t st) {
  using G = MxTile<GW, GT, WA, WB, STAGES, S4>;
  const MxGeom g = mx_geom(c, GATED);
  const long rows = (long)c.T * c.k;
  const int n_tiles = div_up(g.rows, G::TW);
  const long total = (long)n_tiles * worst_row_tiles(rows, c.E, G::TM);
  const long cap = ((long)BLOCKS * device_cus() + 7) / 8 * 8;
  const int blocks = (int)std::min(cap, (total + 7) / 8 * 8);
  mxfp4_gemm_kernel<GATED, GW, GT, WA, WB, STAGES, BLOCKS, S4><<<blocks, 64 * GW * GT, 0, st>>>(
      static_cast<const uint8_t*>(codes), static_cast<const uint8_t*>(scales), src_of, c.k, c.T,
      offs, static_cast<const uint8_t*>(image), g.codes_bytes, g.expert_bytes,
      static_cast<uint16_t*>(out), c.E, (int)g.rows, GATED ? c.f : c.d, GATED ? c.d : c.f,
      (int)rows, n_tiles, 8);
  return hipGetLastError();
}

template <bool GATED>
static hipError_t launch_mx_gemm(const moe_config& c, const void* codes, const void* scales,
                                 const int32_t* src_of, const int32_t* offs, const void* image,
                                 void* out, hipStream_t st) {
  const long rows = (long)c.T * c.k;
  // groups of four stages of token scales: whole groups at 16-byte addresses
  const bool s4 = (GATED ? c.d : c.f) % 512 == 0 && reinterpret_cast<uintptr_t>(scales) % 16 == 0;
  if (rows >= 128L * c.E) {
    if (s4)
      return launch_tile<GATED, 4, 2, 2, 4, 4, 1, true>(c, codes, scales, src_of, offs, image, out,
                                                        st);
    return launch_tile<GATED, 4, 2, 2, 4, 4, 1, false>(c, codes, scales, src_of, offs, image, out,
                                                       st);
  }
  return launch_tile<GATED, 4, 1, 1, 2, 4, 2, false>(c, codes, scales, src_of, offs, image, out,
                                                     st);
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
