// rda_mla_q4.hip -- rows into the 4-bit latent cache, and back out of it.
//
// Writing.  Row x (576 values) of sequence n's i-th new token goes to position
// kv_lens[n] - new_n + i of the sequence:
//   y_c = x_c / sqrt(mean_{c' < 512} x_c'^2 + eps) * weight_c  (or x_c),
//   e   = the least integer with max |y| <= 7 2^e over y_c's group of 32,
//   code = y / 2^e rounded to nearest on 0, 1/2, 1, 3/2, 2, 3, 4, 6 (ties to the
//   even code; 7 goes to 6: no value moves further than half a step).
// y, e and the rounding are computed in 64 bits.  A step is a quarter or more of
// a value, so a code must not depend on how a sum was ordered; and the
// arithmetic hides behind memory.
#include "rda_mla_q4.h"

namespace rda {
namespace {

constexpr int kWaves = 4;

// The sequence of row t: the last n with cu[n] <= t, 64 boundaries a step.
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

// Where row t of the call lies in the cache: nullptr where nowhere.
// `packed` is false where t belongs to no sequence.
__device__ __forceinline__ unsigned char* row_at(const MlaRowsQ4Args& A, int t, int l, bool& packed) {
    int seq, place, fresh;
    if (A.cu) {
        seq = find_seq(A.cu, A.num_seqs, t, l);
        const int a = A.cu[seq];
        place = t - a;
        fresh = A.cu[seq + 1] - a;
    } else {
        fresh = A.total / A.num_seqs;
        seq = t / fresh;
        place = t - seq * fresh;
    }
    packed = place >= 0 && place < fresh;
    if (!packed) return nullptr;
    const int64_t pos = int64_t(A.kv_lens[seq]) - fresh + place;
    if (pos < 0 || pos >= (int64_t(A.table_width) << A.page_shift)) return nullptr;
    const int page = A.table[int64_t(seq) * A.table_width + (pos >> A.page_shift)];
    if (page < 0 || page >= A.num_pages) return nullptr;
    return A.cache + int64_t(page) * A.page_stride +
           int64_t(pos & ((1 << A.page_shift) - 1)) * kQ4Row;
}

__device__ __forceinline__ double shuffle_xor(double x, int d) {
    const uint64_t b = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = __shfl_xor(uint32_t(b), d), hi = __shfl_xor(uint32_t(b >> 32), d);
    return __builtin_bit_cast(double, uint64_t(hi) << 32 | lo);
}

// The least e with |y| <= 7 2^e, from the bits of a finite |y|.
__device__ __forceinline__ int exponent_for(double y) {
    const uint64_t b = __builtin_bit_cast(uint64_t, y) & ~(uint64_t(1) << 63);
    const int k = int(b >> 52) - 1023;                          // |y| in [2^k, 2^(k+1))
    const bool above = (b & ((uint64_t(1) << 52) - 1)) > (uint64_t(3) << 50);   // |y| > 1.75 2^k
    return min(max(k - 2 + (above ? 1 : 0), kQ4Least), kQ4Most);
}

// |t| rounded to the nearest of the 8 sizes (ties to the even code), as a code.
__device__ __forceinline__ uint32_t code_of(double t) {
    const double a = fabs(t);
    const double step = a < 2. ? 0.5 : a < 4. ? 1. : 2.;
    const double r = fmin(rint(a / step) * step, 6.);   // (steps are powers of two: exact)
    const float f = float(r);
    const uint32_t c = uint32_t(f < 2.f ? 2.f * f : f < 4.f ? f + 2.f : 0.5f * f + 4.f);
    return c | (t < 0. && c ? 8u : 0u);
}

// A wave a row: eight latent values a lane, a group is four lanes.
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
    bool packed;
    unsigned char* const out = row_at(A, t, l, packed);
    if (!out) return;
    double y[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        y[2 * i] = double(__uint_as_float(lat[i] << 16));
        y[2 * i + 1] = double(__uint_as_float(lat[i] & 0xffff0000u));
    }
    if (A.weight) {
        double ss = 0.;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fma(y[i], y[i], ss);
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) ss += shuffle_xor(ss, d);
        const double rms = sqrt(ss * (1. / kMlaLatent) + double(A.eps));
        const double inv = 1. / rms;
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = y[i] * inv * double(wt[i >> 2][i & 3]);
    }
    double most = 0.;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        most = fmax(most, fabs(y[i]));
        bad |= !(fabs(y[i]) < __builtin_huge_val());
    }
    int e = bad ? kQ4Most + 1 : exponent_for(most);
    e = max(e, __shfl_xor(e, 1));
    e = max(e, __shfl_xor(e, 2));
    bad = e > kQ4Most;
    uint32_t codes = 0;
    const double unit = __builtin_bit_cast(double, uint64_t(1023 - e) << 52);   // 2^-e
#pragma unroll
    for (int i = 0; i < 8; ++i) codes |= code_of(y[i] * unit) << (4 * i);
    *reinterpret_cast<uint32_t*>(out + 4 * l) = bad ? 0u : codes;
    if ((l & 3) == 0) out[kQ4ScaleAt + l / 4] = static_cast<unsigned char>(bad ? kQ4Bad : uint32_t(e + 127));
    if (l < 8) *reinterpret_cast<u32x4*>(out + kQ4PeAt + 16 * l) = pe;
}

// A wave a row: eight latent values a lane.
__global__ __launch_bounds__(64 * kWaves) void mla_read_q4_kernel(const MlaRowsQ4Args A) {
    const int l = threadIdx.x & 63;
    const int t = blockIdx.x * kWaves + wave_id();
    if (t >= A.total) return;
    bool packed;
    const unsigned char* const row = row_at(A, t, l, packed);
    if (!packed) return;
    u32x4 y = {}, pe = {};
    if (row) {
        const uint32_t codes = *reinterpret_cast<const uint32_t*>(row + 4 * l);
        const uint32_t s = row[kQ4ScaleAt + l / 4];
        if (l < 8) pe = *reinterpret_cast<const u32x4*>(row + kQ4PeAt + 16 * l);
        y = q4_eight(codes, q4_scale(s));
        if (s == kQ4Bad) y = u32x4{0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u};
    }
    uint16_t* const out = A.out + int64_t(t) * A.out_stride;
    *reinterpret_cast<u32x4*>(out + 8 * l) = y;
    if (l < 8) *reinterpret_cast<u32x4*>(out + kMlaLatent + 8 * l) = pe;
}

unsigned grid(const MlaRowsQ4Args& A) { return unsigned((A.total + kWaves - 1) / kWaves); }

}  // namespace

hipError_t launch_mla_append_q4(const MlaRowsQ4Args& A, hipStream_t stream) {
    mla_append_q4_kernel<<<dim3(grid(A)), dim3(64 * kWaves), 0, stream>>>(A);
    return hipGetLastError();
}

hipError_t launch_mla_read_q4(const MlaRowsQ4Args& A, hipStream_t stream) {
    mla_read_q4_kernel<<<dim3(grid(A)), dim3(64 * kWaves), 0, stream>>>(A);
    return hipGetLastError();
}

}  // namespace rda
