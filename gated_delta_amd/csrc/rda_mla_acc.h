// rda_mla_acc.h -- hand-placed accumulators of the latent-attention kernels.
#pragma once

#include <type_traits>

#include "rda_mla.h"

namespace rda {

// The sums O^T of a wave: up to 16 blocks of 32 x 32, block b in the
// accumulation registers a[16 b] .. a[16 b + 15], written and read by the
// statements below only.  The compiler is not told that they hold values (left
// to it, sums that fill much of that file are copied to memory and back around
// every branch), but that every statement may change them, so it keeps nothing
// of its own there across one.  Between two it could: tests/test_accumulators.py
// looks through the assembly that it does not.  The scores' products, which it
// would place there too, have ordinary registers.  It does not see matrix
// products in here either: each waits the two states that ordinary arithmetic
// needs before one reads its result (s_nop 1), and settle / scores_done stand
// before a result is read.
#define RDA_A10(t) "a" #t "0", "a" #t "1", "a" #t "2", "a" #t "3", "a" #t "4", "a" #t "5", \
                   "a" #t "6", "a" #t "7", "a" #t "8", "a" #t "9"
#define RDA_ALL_ACC RDA_A10(), RDA_A10(1), RDA_A10(2), RDA_A10(3), RDA_A10(4), RDA_A10(5),    \
    RDA_A10(6), RDA_A10(7), RDA_A10(8), RDA_A10(9), RDA_A10(10), RDA_A10(11), RDA_A10(12),    \
    RDA_A10(13), RDA_A10(14), RDA_A10(15), RDA_A10(16), RDA_A10(17), RDA_A10(18), RDA_A10(19),\
    RDA_A10(20), RDA_A10(21), RDA_A10(22), RDA_A10(23), RDA_A10(24), "a250", "a251", "a252",  \
    "a253", "a254", "a255"

template <int kN, typename F>
__device__ __forceinline__ void unrolled(F f) {
    if constexpr (kN > 0) {
        unrolled<kN - 1>(f);
        f(std::integral_constant<int, kN - 1>{});
    }
}

template <int kReg>
__device__ __forceinline__ void acc_clear() {
    asm volatile("v_accvgpr_write_b32 a[%0], 0" ::"n"(kReg) : RDA_ALL_ACC);
}
template <int kReg>
__device__ __forceinline__ void acc_scale(float f) {
    float t;
    asm volatile("v_accvgpr_read_b32 %0, a[%2]\n\tv_mul_f32 %0, %1, %0\n\tv_accvgpr_write_b32 a[%2], %0"
                 : "=&v"(t) : "v"(f), "n"(kReg) : RDA_ALL_ACC);
}
// Registers 4 n .. 4 n + 3 to LDS byte address `at` + kOffset (the caller waits).
template <int kN, int kOffset>
__device__ __forceinline__ void acc_store(uint32_t at) {
    asm volatile("ds_write_b128 %0, a[%1:%2] offset:%3"
                 ::"v"(at), "n"(4 * kN), "n"(4 * kN + 3), "n"(kOffset) : "memory", RDA_ALL_ACC);
}
// (kWait: off where both operands were read from LDS or made long before)
template <int kBlock, bool kWait = true>
__device__ __forceinline__ void acc_product(bf16x8 a, bf16x8 b) {
    if constexpr (kWait)
        asm volatile("s_nop 1\n\tv_mfma_f32_32x32x16_bf16 a[%2:%3], %0, %1, a[%2:%3]"
                     ::"v"(a), "v"(b), "n"(16 * kBlock), "n"(16 * kBlock + 15) : RDA_ALL_ACC);
    else
        asm volatile("v_mfma_f32_32x32x16_bf16 a[%2:%3], %0, %1, a[%2:%3]"
                     ::"v"(a), "v"(b), "n"(16 * kBlock), "n"(16 * kBlock + 15) : RDA_ALL_ACC);
}
// Longer than the last products take to write their registers.
__device__ __forceinline__ void settle() {
    asm volatile("s_nop 15\n\ts_nop 15\n\ts_nop 15\n\ts_nop 15\n\ts_nop 15\n\ts_nop 15" ::: RDA_ALL_ACC);
}

// A chain of products for the scores.
__device__ __forceinline__ void scores_first(f32x16& d, bf16x8 a, bf16x8 b) {
    asm volatile("s_nop 1\n\tv_mfma_f32_32x32x16_bf16 %0, %1, %2, 0"
                 : "=&v"(d) : "v"(a), "v"(b) : RDA_ALL_ACC);
}
__device__ __forceinline__ void scores_next(f32x16& d, bf16x8 a, bf16x8 b) {
    asm volatile("s_nop 1\n\tv_mfma_f32_32x32x16_bf16 %0, %1, %2, %0"
                 : "+v"(d) : "v"(a), "v"(b) : RDA_ALL_ACC);
}
// The same with the second operand in accumulation registers a[kReg] ..
// a[kReg + 3] (query operands that stay, placed by acc_put); the first was read
// from LDS, and the wait for it covers the two states.
template <int kReg>
__device__ __forceinline__ void scores_first_acc(f32x16& d, bf16x8 a) {
    asm volatile("v_mfma_f32_32x32x16_bf16 %0, %1, a[%2:%3], 0"
                 : "=&v"(d) : "v"(a), "n"(kReg), "n"(kReg + 3) : RDA_ALL_ACC);
}
template <int kReg>
__device__ __forceinline__ void scores_next_acc(f32x16& d, bf16x8 a) {
    asm volatile("v_mfma_f32_32x32x16_bf16 %0, %1, a[%2:%3], %0"
                 : "+v"(d) : "v"(a), "n"(kReg), "n"(kReg + 3) : RDA_ALL_ACC);
}
template <int kReg>
__device__ __forceinline__ void acc_put(bf16x8 x) {
    const u32x4 v = __builtin_bit_cast(u32x4, x);
    asm volatile("v_accvgpr_write_b32 a[%1], %0" ::"v"(v[0]), "n"(kReg) : RDA_ALL_ACC);
    asm volatile("v_accvgpr_write_b32 a[%1], %0" ::"v"(v[1]), "n"(kReg + 1) : RDA_ALL_ACC);
    asm volatile("v_accvgpr_write_b32 a[%1], %0" ::"v"(v[2]), "n"(kReg + 2) : RDA_ALL_ACC);
    asm volatile("v_accvgpr_write_b32 a[%1], %0" ::"v"(v[3]), "n"(kReg + 3) : RDA_ALL_ACC);
}
__device__ __forceinline__ void scores_done(f32x16& d) {
    asm volatile("s_nop 15\n\ts_nop 7" : "+v"(d)::RDA_ALL_ACC);
}

}  // namespace rda
