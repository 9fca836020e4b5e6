// rda_mla.h -- pieces shared by the latent-attention kernels: the 32x32 MFMA,
// the half-wave exchange, the packed non-finite test, barrier and wait idioms.
#pragma once

#include "rda_lds.h"

namespace rda {

typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kMlaNope = 128, kMlaPe = 64, kMlaV = 128, kMlaLatent = 512;
constexpr int kMlaQk = kMlaNope + kMlaPe;       // expanded query / key width
constexpr int kMlaKv = kMlaNope + kMlaV;        // expanded key + value width of a head
constexpr int kMlaRow = kMlaLatent + kMlaPe;    // one cached row

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

// D += A * B on v_mfma_f32_32x32x16_bf16 (lane l, g = l / 32, c = l % 32:
// A lane holds row c, k = 8g .. 8g+7; B lane holds column c, the same k;
// D register i holds row 8 (i / 4) + 4g + i % 4 of column c).
__device__ __forceinline__ f32x16 mfma32(bf16x8 a, bf16x8 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// The key (or channel) row of D register i within a 32-row block.
__device__ __forceinline__ int d_row(int i, int g) { return 8 * (i >> 2) + 4 * g + (i & 3); }

// x of the lane in the other half of the wavefront (lane ^ 32).
__device__ __forceinline__ float other_half(float x) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false,
                                                    false);
    return __uint_as_float((threadIdx.x & 32) ? r[0] : r[1]);
}

// Bits 15 / 31 of the result are set where a packed bf16 has an exponent of
// all ones (infinity or NaN): 0x7f80 + 0x80 carries into the sign position.
__device__ __forceinline__ uint32_t nonfinite_bits(uint32_t x) {
    return ((x & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
}

// Infinities and NaN to zero.
__device__ __forceinline__ bf16x8 finite_only(bf16x8 x) {
    u32x4 v = __builtin_bit_cast(u32x4, x);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] &= ~((nonfinite_bits(v[i]) >> 15) * 0xffffu);
    return __builtin_bit_cast(bf16x8, v);
}

// Two values as packed bf16 (the first in the low half), rounded to nearest.
__device__ __forceinline__ uint32_t pack_bf16(float x, float y) {
    const f32x2 v = {x, y};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}

// 8 consecutive accumulator registers as one bf16 MFMA operand.  So the
// probabilities enter the second product, each off by at most 2^-8 of itself, no
// more than the output's own rounding; a pair of high and low parts would double
// the products that bound these kernels.  Their sum is taken before the rounding.
template <int kFrom>
__device__ __forceinline__ bf16x8 pack8(const f32x16& s) {
    u32x4 r;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        const f32x2 v = {s[kFrom + 2 * p], s[kFrom + 2 * p + 1]};
        r[p] = __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
    }
    return __builtin_bit_cast(bf16x8, r);
}

// LDS-DMA that the compiler does not track: 16 bytes a lane from base + off
// land at LDS byte address lds + 16 lane.  The builtin form makes the
// compiler wait for every transfer in flight before any LDS read (it cannot
// tell the buffers apart), which would end the prefetch; here the waits are
// the caller's (wait_vm and a barrier before the first read).  It writes M0,
// which cannot be named as changed (the compiler reserves it) and which nothing
// else in these kernels uses (tests/test_accumulators.py looks).  kOnce: for
// memory that is read once (a non-temporal load).
template <bool kOnce = false>
__device__ __forceinline__ void dma16_at(const void* base, uint32_t off, uint32_t lds) {
    if constexpr (kOnce)
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2 nt"
                     ::"s"(lds), "v"(off), "s"(base) : "memory");
    else
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
                     ::"s"(lds), "v"(off), "s"(base) : "memory");
}

// The same with an address of each lane's own.
__device__ __forceinline__ void dma16_from(const void* p, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
                 ::"s"(lds), "v"(p) : "memory");
}

__device__ __forceinline__ uint32_t lds_addr(const void* p) {
    return uint32_t(reinterpret_cast<uintptr_t>((lds_void*)p));
}

// x, computed anew where this stands: what follows from it is not kept in
// registers across a loop around it.
__device__ __forceinline__ int here(int x) {
    asm volatile("" : "+v"(x));
    return x;
}

typedef __attribute__((address_space(3))) u32x4 lds_u32x4;
typedef __attribute__((address_space(3))) char lds_char;

// 16 bytes, and a transposing read of 8, at an LDS byte address.
__device__ __forceinline__ bf16x8 lds_read16(uint32_t a) {
    return __builtin_bit_cast(bf16x8, *(const lds_u32x4*)(lds_char*)uintptr_t(a));
}
__device__ __forceinline__ u32x2 lds_read_tr8(uint32_t a) {
    return __builtin_bit_cast(
        u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(lds_char*)uintptr_t(a)));
}

// Workgroup barrier that leaves vector memory operations in flight: the
// wave's own LDS accesses are done (lgkmcnt), nothing moves across it.
__device__ __forceinline__ void raw_barrier() {
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// The sequence of packed row t: the last n with cu[n] <= t.  64 boundaries a step,
// so a batch of 64 costs one load latency and one of 4096 two.
__device__ __forceinline__ int find_seq(const int32_t* cu, int num_seqs, int t, int l) {
    int lo = 0, n = num_seqs;   // the answer is in [lo, lo + n)
    while (n > 1) {
        const int step = (n + 63) / 64;
        const int at = lo + l * step;
        const uint64_t below = __ballot(at < lo + n && cu[at < num_seqs ? at : 0] <= t);
        const int k = below ? 63 - __builtin_clzll(below) : 0;
        n = min(step, n - k * step);
        lo += k * step;
    }
    return lo;
}

}  // namespace rda
