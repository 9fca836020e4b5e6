// rda_mla_q4.hip -- rows into the 4-bit latent cache, and back out of it.
//
// Writing.  Row x (576 values) of sequence n's i-th new token goes to position
// kv_lens[n] - new_n + i of the sequence:
//   y_c = x_c / sqrt(mean_{c' < 512} x_c'^2 + eps) * weight_c  (or x_c),
//   e   = the least integer with max |y| <= 7 2^e over y_c's group of 32,
//   code = y / 2^e rounded to nearest on 0, 1/2, 1, 3/2, 2, 3, 4, 6 (ties to the
//   even code; 7 goes to 6: no value moves further than half a step, but for those
//   above 7 2^125, the largest exponent's, which go to 6 2^125).
// y, e and the codes are as 64 bits give them: a step is a quarter or more of a
// value, so a code must not depend on how a sum was ordered.  With a norm 32 bits
// are tried first (quantise_normed), and decide all codes of 99 rows in 100.
// Bound by: ordinary instructions, 157 a row and wave (0.68 of the time that the CUs
// are busy); the look-ups of a row's place, one after the other, are 2.9 us of 15.5 for 32768
// rows (50.8 MB, 3.3 TB/s), the check that decides for 32 bits 1.0 (in 64 bits throughout
// 33.9 us).  Without the norm all rows take the 64-bit form: 15.6 us.
//
// Reading is bound by memory: 65537 rows (102 MB) 18.1 us, 5.6 TB/s.
#include <type_traits>

#include "rda_mla_q4.h"

namespace rda {
namespace {

constexpr int kWaves = 4;

// Where the kRows rows from `t` on lie in the cache, looked up by a lane each.
struct Places {
    uint64_t at;     // lane r: row t + r's address, 0 where it has none
    bool packed;     // and whether it belongs to a sequence
    template <int kRows>
    __device__ __forceinline__ void find(const MlaRowsQ4Args& A, int t, int l) {
        const int row = min(t + min(l, kRows - 1), A.total - 1);
        int seq, place, fresh;
        if (A.cu) {
            seq = find_seq(A.cu, A.num_seqs, t, l);
            if constexpr (kRows > 1)
                while (seq + 1 < A.num_seqs && A.cu[seq + 1] <= row) ++seq;
            const int a = A.cu[seq];
            place = row - a;
            fresh = A.cu[seq + 1] - a;
        } else {
            fresh = A.total / A.num_seqs;
            seq = row / fresh;
            place = row - seq * fresh;
        }
        at = 0;
        packed = place >= 0 && place < fresh && t + l < A.total;
        if (!packed) return;
        const int64_t pos = int64_t(A.kv_lens[seq]) - fresh + place;
        if (pos < 0 || pos >= (int64_t(A.table_width) << A.page_shift)) return;
        const int page = A.table[int64_t(seq) * A.table_width + (pos >> A.page_shift)];
        if (page < 0 || page >= A.num_pages) return;
        at = reinterpret_cast<uint64_t>(A.cache) + uint64_t(page) * uint64_t(A.page_stride) +
             uint64_t(pos & ((1 << A.page_shift) - 1)) * kQ4Row;
    }
    __device__ __forceinline__ unsigned char* row(int r) const {
        return reinterpret_cast<unsigned char*>(uint64_t(uint32_t(__builtin_amdgcn_readlane(int(at >> 32), r))) << 32 |
                                                uint32_t(__builtin_amdgcn_readlane(int(at), r)));
    }
    __device__ __forceinline__ bool in_sequence(int r) const { return __ballot(packed) >> r & 1; }
};

// x + the values of the other lanes of the wavefront.
__device__ __forceinline__ double wave_sum(double x) {
    auto halves = [](double y) { return __builtin_bit_cast(u32x2, y); };
    auto dpp = [&](auto ctrl) {
        constexpr int c = decltype(ctrl)::value;
        const u32x2 y = halves(x);
        x += __builtin_bit_cast(double, u32x2{uint32_t(__builtin_amdgcn_update_dpp(0, int(y[0]), c, 0xF, 0xF, false)),
                                              uint32_t(__builtin_amdgcn_update_dpp(0, int(y[1]), c, 0xF, 0xF, false))});
    };
    dpp(std::integral_constant<int, 0xB1>{});    // lane ^ 1
    dpp(std::integral_constant<int, 0x4E>{});    // lane ^ 2
    dpp(std::integral_constant<int, 0x141>{});   // row_half_mirror
    dpp(std::integral_constant<int, 0x140>{});   // row_mirror
    u32x2 y = halves(x);
    auto a = __builtin_amdgcn_permlane16_swap(y[0], y[0], false, false);
    auto b = __builtin_amdgcn_permlane16_swap(y[1], y[1], false, false);
    x = __builtin_bit_cast(double, u32x2{a[0], b[0]}) + __builtin_bit_cast(double, u32x2{a[1], b[1]});
    y = halves(x);
    a = __builtin_amdgcn_permlane32_swap(y[0], y[0], false, false);
    b = __builtin_amdgcn_permlane32_swap(y[1], y[1], false, false);
    return __builtin_bit_cast(double, u32x2{a[0], b[0]}) + __builtin_bit_cast(double, u32x2{a[1], b[1]});
}

// 1 / sqrt(a): the instruction's estimate (2^-26 or better) and two Newton steps.
__device__ __forceinline__ double inverse_sqrt(double a) {
    double r = __builtin_amdgcn_rsq(a);
#pragma unroll
    for (int i = 0; i < 2; ++i) r = fma(r * 0.5, fma(-a * r, r, 1.), r);
    return a < __builtin_huge_val() ? r : a == a ? 0. : a;
}

// The least e with |y| <= 7 2^e, from the bits of a finite |y|.
__device__ __forceinline__ int exponent_for(double y) {
    const uint64_t b = __builtin_bit_cast(uint64_t, y) & ~(uint64_t(1) << 63);
    const int k = int(b >> 52) - 1023;                          // |y| in [2^k, 2^(k+1))
    const bool above = (b & ((uint64_t(1) << 52) - 1)) > (uint64_t(3) << 50);   // |y| > 1.75 2^k
    return min(max(k - 2 + (above ? 1 : 0), kQ4Least), kQ4Most);
}

// t in 32 bits, rounded so that rounding it again to a few bits gives what
// rounding t would: towards zero, with the last bit set where that is inexact.
__device__ __forceinline__ float to_odd(double t) {
    const float f = float(t);
    const double d = double(f);
    uint32_t u = __float_as_uint(f);
    if (fabs(d) > fabs(t)) --u;
    if (d != t) u |= 1;
    return __uint_as_float(u);
}

// The largest of a group's lanes.
__device__ __forceinline__ int group_max(int e) {
    e = max(e, __builtin_amdgcn_update_dpp(0, e, 0xB1, 0xF, 0xF, false));
    return max(e, __builtin_amdgcn_update_dpp(0, e, 0x4E, 0xF, 0xF, false));
}

// Eight values as codes (ties to the even code, what is above 6 to 6), and the same
// where zero has no sign.
__device__ __forceinline__ uint32_t codes_of(const float* t) {
    uint32_t c = 0;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, t[0], t[1], 1.f, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, t[2], t[3], 1.f, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, t[4], t[5], 1.f, 2);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, t[6], t[7], 1.f, 3);
}
__device__ __forceinline__ uint32_t without_minus_zero(uint32_t c) {
    return c & (((c | c >> 1 | c >> 2) & 0x11111111u) << 3 | 0x77777777u);
}

// A lane's eight values of a row, quantised: codes and scale byte.
struct Quantised {
    uint32_t codes, scale;
};

// From 64 bits.
__device__ __forceinline__ Quantised quantise(const double* y) {
    double most = 0.;
    uint32_t high = 0;   // the largest exponent field, infinities and NaN included
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        most = fmax(most, fabs(y[i]));
        high = max(high, uint32_t(__builtin_bit_cast(uint64_t, y[i]) >> 32) & 0x7fffffffu);
    }
    const int e = group_max(high >= 0x7ff00000u ? kQ4Most + 1 : exponent_for(most));
    if (e > kQ4Most) return {0, kQ4Bad};
    const double unit = __builtin_bit_cast(double, uint64_t(1023 - e) << 52);   // 2^-e
    float t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = to_odd(y[i] * unit);
    return {without_minus_zero(codes_of(t)), uint32_t(e + 127)};
}

// The norm in 32 bits, off by less than 2^-20 (eight products and six sums of
// positive terms in the mean, half of that in its root, the root's own 2^-23,
// five more roundings).  False where that may leave another code or scale:
// where values 2^-17 smaller and larger do not agree, or out of the ordinary range:
// also where a value is NaN though the sum is not, by a weight that is not finite.
__device__ __forceinline__ bool quantise_normed(const float* x, const f32x4* wt, float eps, Quantised& q) {
    float ss = 0.f, y[8], most = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        ss = fmaf(x[i], x[i], ss);
        y[i] = x[i] * wt[i >> 2][i & 3];
        most = __builtin_elementwise_maximum(most, fabsf(y[i]));   // (NaN if one is)
    }
    ss = dpp_sum16(ss);
    auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(ss), __float_as_uint(ss), false, false);
    ss = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    r = __builtin_amdgcn_permlane32_swap(__float_as_uint(ss), __float_as_uint(ss), false, false);
    ss = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    const float inv = __builtin_amdgcn_rsqf(fmaf(ss, 1.f / kMlaLatent, eps));
    const float less = inv * (1.f - 0x1p-17f), more = inv * (1.f + 0x1p-17f);
    auto exponent = [](float z) {   // as exponent_for
        const uint32_t u = __float_as_uint(z);
        return int(u >> 23) - 129 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    };
    const int lo = group_max(exponent(most * less)), hi = group_max(exponent(most * more));
    const float unit = __uint_as_float(uint32_t(127 - hi) << 23), small = less * unit, large = more * unit;
    float a[8], b[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        a[i] = y[i] * small;
        b[i] = y[i] * large;
    }
    const uint32_t codes = codes_of(a);
    q = {without_minus_zero(codes), uint32_t(hi + 127)};
    // (a group of zeros beside others is left to the other form, like every extreme)
    return ss > 0x1p-60f && ss < 0x1p100f && most > 0x1p-60f && most < 0x1p60f && hi > -60 && hi < 60 && lo == hi &&
           codes == codes_of(b);
}

// A wave a row: eight latent values a lane, a group is four lanes.  (Several rows a
// wave take longer, 15.8 us with two and 18.4 with four for 14.5.)
__global__ __launch_bounds__(64 * kWaves) void mla_append_q4_kernel(const MlaRowsQ4Args A) {
    const int l = threadIdx.x & 63;
    const int t = blockIdx.x * kWaves + wave_id();
    if (t >= A.total) return;
    const uint16_t* x = A.kv + int64_t(t) * A.kv_stride;
    const u32x4 lat = *reinterpret_cast<const u32x4*>(x + 8 * l);
    u32x4 pe = {};
    if (l < 8) pe = *reinterpret_cast<const u32x4*>(x + kMlaLatent + 8 * l);
    f32x4 wt[2] = {};
    if (A.weight) {
        wt[0] = *reinterpret_cast<const f32x4*>(A.weight + 8 * l);
        wt[1] = *reinterpret_cast<const f32x4*>(A.weight + 8 * l + 4);
    }
    Places P;
    P.find<1>(A, t, l);
    unsigned char* const out = P.row(0);
    if (!out) return;
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(lat[i] << 16);
        v[2 * i + 1] = __uint_as_float(lat[i] & 0xffff0000u);
    }
    Quantised q;
    if (!A.weight || !__all(quantise_normed(v, wt, A.eps, q))) {
        double y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = double(v[i]);
        if (A.weight) {
            double ss = 0.;
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = fma(y[i], y[i], ss);
            const double inv = inverse_sqrt(wave_sum(ss) * (1. / kMlaLatent) + double(A.eps));
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = y[i] * inv * double(wt[i >> 2][i & 3]);
        }
        q = quantise(y);
    }
    *reinterpret_cast<uint32_t*>(out + 4 * l) = q.codes;
    if ((l & 3) == 0) out[kQ4ScaleAt + l / 4] = static_cast<unsigned char>(q.scale);
    if (l < 8) *reinterpret_cast<u32x4*>(out + kQ4PeAt + 16 * l) = pe;
}

// kRows rows a wave: eight latent values a lane.
template <int kRows>
__global__ __launch_bounds__(64 * kWaves) void mla_read_q4_kernel(const MlaRowsQ4Args A) {
    const int l = threadIdx.x & 63;
    const int t = (blockIdx.x * kWaves + wave_id()) * kRows;
    if (t >= A.total) return;
    Places P;
    P.find<kRows>(A, t, l);
    uint32_t codes[kRows], scale[kRows];
    u32x4 pe[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        const unsigned char* const row = P.row(r);
        codes[r] = 0;
        scale[r] = 1;
        pe[r] = u32x4{};
        if (!row) continue;
        codes[r] = *reinterpret_cast<const uint32_t*>(row + 4 * l);
        scale[r] = row[kQ4ScaleAt + l / 4];
        if (l < 8) pe[r] = *reinterpret_cast<const u32x4*>(row + kQ4PeAt + 16 * l);
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        if (!P.in_sequence(r)) continue;
        u32x4 y = q4_eight(codes[r], q4_scale(scale[r]));
        if (scale[r] == kQ4Bad) y = u32x4{0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u};
        uint16_t* const out = A.out + int64_t(t + r) * A.out_stride;
        *reinterpret_cast<u32x4*>(out + 8 * l) = y;
        if (l < 8) *reinterpret_cast<u32x4*>(out + kMlaLatent + 8 * l) = pe[r];
    }
}

unsigned grid(const MlaRowsQ4Args& A, int rows) {
    return unsigned((A.total + kWaves * rows - 1) / (kWaves * rows));
}

}  // namespace

hipError_t launch_mla_append_q4(const MlaRowsQ4Args& A, hipStream_t stream) {
    mla_append_q4_kernel<<<dim3(grid(A, 1)), dim3(64 * kWaves), 0, stream>>>(A);
    return hipGetLastError();
}

hipError_t launch_mla_read_q4(const MlaRowsQ4Args& A, hipStream_t stream) {
    // two rows a wave where there are waves enough (32768 rows 11.1 us for 12.2 with
    // one and 12.6 with four)
    if (A.total >= 8192) mla_read_q4_kernel<2><<<dim3(grid(A, 2)), dim3(64 * kWaves), 0, stream>>>(A);
    else mla_read_q4_kernel<1><<<dim3(grid(A, 1)), dim3(64 * kWaves), 0, stream>>>(A);
    return hipGetLastError();
}

}  // namespace rda
