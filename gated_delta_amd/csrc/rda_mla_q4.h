// rda_mla_q4.h -- the latent cache in 4 bits: its row, the conversions, the sums and
// products of the attention over it, and the transfer of 8 rows into LDS.
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

// The sums O^T of a wave, four blocks of 32 x 32 in the accumulation registers
// a[0] .. a[63], written and read by the statements below only (the compiler,
// given them as values, copies them around every branch of the loop).  It is not
// told that they hold values, but that every statement may change them, so it
// keeps nothing of its own there across one.  A product waits two states for
// operands that ordinary arithmetic made.
#define RDA_Q4_A10(t) "a" #t "0", "a" #t "1", "a" #t "2", "a" #t "3", "a" #t "4", "a" #t "5", \
                      "a" #t "6", "a" #t "7", "a" #t "8", "a" #t "9"
#define RDA_Q4_ACC RDA_Q4_A10(), RDA_Q4_A10(1), RDA_Q4_A10(2), RDA_Q4_A10(3), RDA_Q4_A10(4), \
    RDA_Q4_A10(5), "a60", "a61", "a62", "a63"

template <int kReg>
__device__ __forceinline__ void q4_acc_clear() {
    asm volatile("v_accvgpr_write_b32 a[%0], 0" ::"n"(kReg) : RDA_Q4_ACC);
}
template <int kReg>
__device__ __forceinline__ void q4_acc_scale(float f) {
    float t;
    asm volatile("v_accvgpr_read_b32 %0, a[%2]\n\tv_mul_f32 %0, %1, %0\n\tv_accvgpr_write_b32 a[%2], %0"
                 : "=&v"(t) : "v"(f), "n"(kReg) : RDA_Q4_ACC);
}
template <int kReg>
__device__ __forceinline__ float q4_acc_get() {
    float t;
    asm volatile("v_accvgpr_read_b32 %0, a[%1]" : "=v"(t) : "n"(kReg) : RDA_Q4_ACC);
    return t;
}
template <int kBlock>
__device__ __forceinline__ void q4_acc_product(bf16x8 a, bf16x8 b) {
    asm volatile("s_nop 1\n\tv_mfma_f32_32x32x16_bf16 a[%2:%3], %0, %1, a[%2:%3]"
                 ::"v"(a), "v"(b), "n"(16 * kBlock), "n"(16 * kBlock + 15) : RDA_Q4_ACC);
}
// The scores' products, in ordinary registers for the same reason: 16 cached rows
// by 16 query rows, 128 channels (product kN of 4: group kN of each lane's four,
// whose scales are byte kN of the row's and of the query's), and 32 of the shared
// channels.  The query's operands stay in accumulation registers.
typedef int i32x8 __attribute__((ext_vector_type(8)));

template <int kN>
__device__ __forceinline__ void q4_score(f32x4& d, u32x4 a, i32x8 b, uint32_t as, uint32_t bs) {
    if constexpr (kN == 0)
        asm volatile("s_nop 1\n\tv_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, 0, %3, %4 "
                     "op_sel:[0,0,0] op_sel_hi:[0,0,0] cbsz:4"
                     : "=&v"(d) : "v"(a), "a"(b), "v"(as), "v"(bs) : RDA_Q4_ACC);
    else
        asm volatile("s_nop 1\n\tv_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 "
                     "op_sel:[%5,%5,0] op_sel_hi:[%6,%6,0] cbsz:4"
                     : "+v"(d) : "v"(a), "a"(b), "v"(as), "v"(bs), "n"(kN & 1), "n"(kN >> 1) : RDA_Q4_ACC);
}
__device__ __forceinline__ void q4_score_pe(f32x4& d, bf16x8 a, bf16x8 b) {
    asm volatile("s_nop 1\n\tv_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+v"(d) : "v"(a), "v"(b) : RDA_Q4_ACC);
}
// Longer than the last of them takes to write its result (11 states).
__device__ __forceinline__ void q4_score_done(f32x4& x, f32x4& y) {
    asm volatile("s_nop 11" : "+v"(x), "+v"(y)::RDA_Q4_ACC);
}
// Longer than the last products take to write their registers.
__device__ __forceinline__ void q4_acc_settle() {
    asm volatile("s_nop 15\n\ts_nop 15\n\ts_nop 15\n\ts_nop 15\n\ts_nop 15\n\ts_nop 15" ::: RDA_Q4_ACC);
}

// Eight rows (of one page, so they lie one behind the other) into LDS as they
// lie: four transfers, 200 granules of 16 bytes.  All lanes are active.  kOnce:
// for rows that are read once (they pass the caches by).
constexpr int kQ4Fetch = 4;
#define RDA_Q4_ROWS(how)                                                             \
    "s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" how           \
    "\n\tglobal_load_lds_dwordx4 %1, %2 offset:0x400" how                            \
    "\n\tglobal_load_lds_dwordx4 %1, %2 offset:0x800" how                            \
    "\n\ts_mov_b64 exec, 0xff\n\tglobal_load_lds_dwordx4 %1, %2 offset:0xc00" how   \
    "\n\ts_mov_b64 exec, -1"

template <bool kOnce>
__device__ __forceinline__ void q4_fetch_rows(const void* rows, uint32_t lane16, uint32_t lds) {
    if constexpr (kOnce) asm volatile(RDA_Q4_ROWS(" nt") ::"s"(lds), "v"(lane16), "s"(rows) : "memory");
    else asm volatile(RDA_Q4_ROWS("") ::"s"(lds), "v"(lane16), "s"(rows) : "memory");
}

// The same where only the first `valid` rows are to be read: the others become zeros.
// (eight rows of zeros: what a tile behind the last one is filled from)
__device__ const __attribute__((aligned(16))) uint32_t kQ4Zeros[8 * kQ4Row / 4] = {};

__device__ __forceinline__ void q4_fetch_some(const char* rows, int valid, int lane, uint32_t lds) {
    const char* const zeros = reinterpret_cast<const char*>(kQ4Zeros);
    const int l = here(lane);
#pragma unroll 1
    for (int i = 0; i < kQ4Fetch; ++i) {
        const int g = 64 * i + l, row = g * 5243 >> 17;   // g / 25
        if (g < 8 * kQ4Row / 16) dma16_from(row < valid ? rows + 16 * g : zeros, lds + 1024 * i);
    }
}

}  // namespace rda
