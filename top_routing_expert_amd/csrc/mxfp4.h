// MXFP4 (OCP microscaling): 32 consecutive elements share one scale, a power of
// two held as its exponent plus 127 in one byte (E8M0, 255 = NaN); elements are
// E2M1 codes (1 sign, 2 exponent bits with bias 1, 1 mantissa bit: 0, .5, 1,
// 1.5, 2, 3, 4, 6), two to a byte, the earlier one in the low nibble.
//
// gfx950 converts in hardware (v_cvt_scalef32_pk_*), the scale as a float whose
// exponent is used, nearest with ties to the even code, saturating at 6.
#pragma once

#include "common.h"

namespace moe {

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

constexpr int kMxBlock = 32;  // elements sharing a scale
constexpr int kMxStepK = 128; // k of one packed chunk (four scale blocks)

// E8M0 byte -> float bits.  2^-127 (byte 0) is a float subnormal; 255 is NaN.
__device__ __forceinline__ float mx_scale(uint32_t b) {
  return __uint_as_float(b == 0 ? 0x00400000u : b == 255u ? 0x7fc00000u : b << 23);
}

// Packed expert weights of R output rows over K (both multiples of 128).  Every
// expert's image, back to back: codes as 1 KB chunks of 16 rows x 128 k,
// [R / 16][K / 128][16 rows][64 bytes], the 16-byte piece q (k 32 q .. +31) of
// chunk row r at q ^ ((r >> 2) & 3); then the scales,
// [R / 64][K / 128][64 rows][4 bytes], byte q for k 32 q .. +31.
struct MxGeom {
  long rows;            // R
  int steps;            // K / 128
  size_t codes_bytes;   // R K / 2, of one expert
  size_t expert_bytes;  // codes and scales of one expert
};
MxGeom mx_geom(const moe_config& c, bool gate_up);

}  // namespace moe
