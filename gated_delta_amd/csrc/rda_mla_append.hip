// rda_mla_append.hip -- new rows into the paged latent cache.
//
// Row x (576 values) of sequence n's i-th new token goes to position
// kv_lens[n] - new_n + i of the sequence:
//   latent:  x_c / sqrt(mean_{c' < 512} x_c'^2 + eps) * weight_c,  c < 512
//            (or x_c as it is), rounded to bf16 once
//   shared key channels: copied.
// One wave per token: 16 bytes a lane of the latent, 16 bytes of lanes 0..7
// for the rest; the sum of squares meets in the wave.  Bound by memory where
// there are many rows: 32768 rows 14.8 us, 5.1 TB/s read and written; 768 rows
// 9.7 us, the launch and one latency after the other (offsets, length, page,
// row).
#include "rda_internal.h"
#include "rda_mla.h"

namespace rda {
namespace {

constexpr int kWaves = 4;

__global__ __launch_bounds__(64 * kWaves) void mla_append_kernel(const MlaAppendArgs A) {
    const int l = threadIdx.x & 63;
    const int t = blockIdx.x * kWaves + wave_id();
    if (t >= A.total) return;
    const uint16_t* x = A.kv + int64_t(t) * A.kv_stride;
    const u32x4 lat = *reinterpret_cast<const u32x4*>(x + 8 * l);
    u32x4 pe = {};
    if (l < 8) pe = *reinterpret_cast<const u32x4*>(x + kMlaLatent + 8 * l);
    f32x4 wt[2] = {f32x4{1.f, 1.f, 1.f, 1.f}, f32x4{1.f, 1.f, 1.f, 1.f}};
    if (A.weight) {
        wt[0] = *reinterpret_cast<const f32x4*>(A.weight + 8 * l);
        wt[1] = *reinterpret_cast<const f32x4*>(A.weight + 8 * l + 4);
    }
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
    if (place < 0 || place >= fresh) return;
    const int64_t pos = int64_t(A.kv_lens[seq]) - fresh + place;
    if (pos < 0 || pos >= (int64_t(A.table_width) << A.page_shift)) return;
    const int page = A.table[int64_t(seq) * A.table_width + (pos >> A.page_shift)];
    if (page < 0 || page >= A.num_pages) return;
    uint16_t* out = A.cache + int64_t(page) * A.page_stride +
                    int64_t(pos & ((1 << A.page_shift) - 1)) * kMlaRow;
    u32x4 y = lat;
    if (A.weight) {
        float v[8], ss = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(lat[i] << 16);
            v[2 * i + 1] = __uint_as_float(lat[i] & 0xffff0000u);
            ss = fmaf(v[2 * i], v[2 * i], ss);
            ss = fmaf(v[2 * i + 1], v[2 * i + 1], ss);
        }
        ss = dpp_sum16(ss);
        ss += __shfl_xor(ss, 16);
        ss += __shfl_xor(ss, 32);
        const float inv = 1.f / sqrtf(ss * (1.f / kMlaLatent) + A.eps);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const f32x2 p = {v[2 * i] * inv * wt[i >> 1][2 * (i & 1)],
                             v[2 * i + 1] * inv * wt[i >> 1][2 * (i & 1) + 1]};
            y[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(p, bf16x2));
        }
    }
    *reinterpret_cast<u32x4*>(out + 8 * l) = y;
    if (l < 8) *reinterpret_cast<u32x4*>(out + kMlaLatent + 8 * l) = pe;
}

}  // namespace

hipError_t launch_mla_append(const MlaAppendArgs& A, hipStream_t stream) {
    mla_append_kernel<<<dim3(unsigned((A.total + kWaves - 1) / kWaves)), dim3(64 * kWaves), 0, stream>>>(A);
    return hipGetLastError();
}

}  // namespace rda
