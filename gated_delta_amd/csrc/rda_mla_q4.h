// rda_mla_q4.h -- the latent cache in 4 bits: its row, the conversions, and the
// transfer of 16 rows into LDS.
//
// A row of 400 bytes: 512 latent values as e2m1 codes (256 bytes, the value of
// an even channel in the low half of its byte), a scale byte s for each 32 of
// them (16 bytes: 2^(s - 127), 255 where they are NaN), 64 shared key channels
// in bf16 (128 bytes).  e2m1 with a power of two per 32 values is what the
// matrix cores multiply and what one instruction turns into a pair of bf16.
// The shared channels stay in bf16: they are a ninth of the values, carry the
// position where a model has rotary ones, and reach every score unnormalised.
#pragma once

#include "rda_internal.h"
#include "rda_mla.h"

namespace rda {

constexpr int kQ4Group = 32;                         // values with one scale
constexpr int kQ4Groups = kMlaLatent / kQ4Group;     // 16
constexpr int kQ4ScaleAt = kMlaLatent / 2;           // 256
constexpr int kQ4PeAt = kQ4ScaleAt + kQ4Groups;      // 272
constexpr int kQ4Row = kQ4PeAt + 2 * kMlaPe;         // 400
static_assert(kQ4Row == RDA_MLA_ROW_Q4, "the row of rda.h");

// Scale exponents that the writer uses: every value they give is a normal bf16.
constexpr int kQ4Least = -120, kQ4Most = 125;
constexpr uint32_t kQ4Bad = 255;

// 2^(s - 127) of a scale byte (1 .. 254).
__device__ __forceinline__ float q4_scale(uint32_t s) { return __uint_as_float(s << 23); }

// Codes in bits 8 n .. 8 n + 7 of x as two bf16, the lower code's in the low half.
template <int kByte>
__device__ __forceinline__ uint32_t q4_pair(uint32_t x, float scale) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x, scale, kByte));
}

// Eight codes as eight bf16.
__device__ __forceinline__ u32x4 q4_eight(uint32_t x, float scale) {
    return u32x4{q4_pair<0>(x, scale), q4_pair<1>(x, scale), q4_pair<2>(x, scale),
                 q4_pair<3>(x, scale)};
}

// Eight rows (of one page, so they lie one behind the other) into LDS as they
// lie: four transfers, 200 granules of 16 bytes.  Rows from `valid` on are read
// as zeros.
constexpr int kQ4Fetch = 4;
__device__ const __attribute__((aligned(16))) uint32_t kQ4Zeros[4] = {};

__device__ __forceinline__ void q4_fetch_rows(const char* rows, int valid, uint32_t lds, int lane) {
    const int l = here(lane);
    if (valid >= 8) {
#pragma unroll
        for (int i = 0; i < kQ4Fetch - 1; ++i) dma16_at(rows, 16 * l + 1024 * i, lds + 1024 * i);
        if (l < 8) dma16_at(rows, 16 * l + 1024 * 3, lds + 1024 * 3);
    } else {
        const char* const zeros = reinterpret_cast<const char*>(kQ4Zeros);
#pragma unroll
        for (int i = 0; i < kQ4Fetch; ++i) {
            const int g = 64 * i + l, row = g * 5243 >> 17;   // g / 25
            if (i < kQ4Fetch - 1 || l < 8)
                dma16_from(row < valid ? rows + 16 * g : zeros, lds + 1024 * i);
        }
    }
}

}  // namespace rda
