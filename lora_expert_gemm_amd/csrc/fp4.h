// How 4-bit weights lie in memory, and their conversions.
//
// A weight is a 4-bit E2M1 code (sign; 0, 0.5, 1, 1.5, 2, 3, 4, 6) times a
// power of two shared by the 32 weights of a group along the contraction, kept
// as its exponent plus 127 in a byte (255: NaN).  A matrix of N rows and K
// columns is cut into tiles of 16 rows x 128 columns, in the order in which a
// wave of the product reads them:
//   codes   [N / 16][K / 128][lane][16 bytes]   1 KB a tile, lane = 16 g + r: the
//           32 codes of row r of the tile, group g, two a byte, low half first
//   scales  [N / 16][K / 512][lane][4 bytes]    byte q: the group's scale in the
//           q-th of four tiles along K
// with N, K rounded up and zeros past them.  A lane's 32 weights are 16 bytes
// of one group, so that one wave load brings a whole tile from 1 KB in a row
// straight into the registers of the matrix instruction that uses it.
#pragma once

#include "common.h"

namespace moelora {

constexpr int kTileRows = 16, kTileCols = 128, kGroup = 32;
constexpr int kTileBytes = kTileRows * kTileCols / 2, kScaleBytes = 256;  // a tile's codes, four tiles' scales

// Float bits of a scale code.  The conversion instructions take the exponent
// field alone: 0 gives 2^-127 and 255 NaN (an in-bounds check of all codes with
// all scales gave code x 2^(scale - 127) exactly, in bf16 and in float32).
__device__ __forceinline__ float scale_of_code(uint32_t code) { return __uint_as_float(code << 23); }

// Codes 8 i .. 8 i + 7 of a lane's dword i as one MFMA operand of bf16 values,
// which are exact.
__device__ __forceinline__ u32x4_t e2m1x8_to_bf16(uint32_t w, float scale) {
  return u32x4_t{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3))};
}

}  // namespace moelora
