// rda_mla_prefill.hip -- expanded latent attention over packed prompts.
//
// Per head, query i of a sequence with lq queries and lk keys:
//   s_ij = scale (q_i[:128] . kn_j + q_i[128:] . pe_j),  j < limit_i
//   o_i  = sum_j exp(s_ij - m_i) v_j / l_i,  lse_i = m_i + log l_i
// with limit_i = min(lk, i + lk - lq + 1) (causal) or lk.
//
// One workgroup of four waves takes 128 queries of one head, a wave 32 of
// them, and walks the keys in tiles of 64 that arrive by LDS-DMA one tile
// ahead (three where a workgroup has a CU for itself).  The products are
// transposed, S^T = K Q^T and O^T = V^T P^T, so that a lane owns one query: the
// D registers of S^T are, rounded to bf16, the B operand of the second product
// in the order (4g .. 4g+3, 8 + 4g ..) of the keys, which the transposing reads
// of V follow.  P never leaves registers.
//
// The form with two tiles' memory does not fit its 256 registers: 20 go to
// scratch, and where one comes back the compiler waits for every load in
// flight, the transfers of the next tile among them.  Its prefetch is emptied
// in every tile for that.
//
// Two workgroups share a CU's LDS (two tiles of 40 KiB each), so one's products
// run beside the other's exponentials.  An operand read from LDS feeds one
// product of 32 cycles, about as long as the CU's LDS needs for it, so neither
// could be much less busy than the other.  Measured: 4096 new tokens of 5 sequences
// behind 3001 cached ones, 16 heads, 115 us, 450 TFLOP/s; 2048 tokens of 32
// heads 87 us; 65 tokens 13.9 us.  A few queries over a long context are the
// weak side: a wave's tile after the other, 2 us each, most of it latency
// (30 queries over 1959 keys 64 us).
#include <type_traits>

#include "rda_internal.h"
#include "rda_mla.h"
#include "rda_mla_tile.h"

namespace rda {
namespace {

constexpr int kBM = 128;   // queries per workgroup
constexpr int kBN = 64;    // keys per tile
constexpr int kThreads = 256;

// Row r of a tile keeps 16-byte granule j at j ^ swizzle(r): sixteen
// consecutive rows read at one granule (Kn, Kp) and four consecutive rows
// read at four adjacent granules (V, transposing) fall on distinct banks.
template <int kBufs>
struct Lds {
    uint16_t Kn[kBufs][kBN * kMlaNope];   // 16 granules a row, j ^ (r & 15)
    uint16_t Kp[kBufs][kBN * kMlaPe];     // 8 granules a row, j ^ ((r >> 1) & 7)
    uint16_t V[kBufs][kBN * kMlaV];       // 16 granules a row, j ^ ((r & 3) << 2)
};
constexpr int kDma = 10;   // transfers of a wave per tile

struct Dma {
    const MlaPrefillArgs& A;
    const uint16_t* kv;   // first key row of the sequence, this head
    const uint16_t* pe;
    int w, l, lk;

    // This wave's 10 KiB of the tile at key k0: 4 + 4 + 2 KiB of Kn, V, Kp.
    // Rows behind the last key repeat it.
    template <int kBufs>
    __device__ __forceinline__ void issue(int k0, Lds<kBufs>& t, int buf) const {
        const int last = lk - 1 - k0;
        const uint16_t* kt = kv + int64_t(k0) * A.kv_stride;
        const uint16_t* pt = pe + int64_t(k0) * A.pe_stride;
        const uint32_t ks = uint32_t(A.kv_stride) * 2, ps = uint32_t(A.pe_stride) * 2;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int n = 4 * w + i, r = 4 * n + (l >> 4);
            const uint32_t row = uint32_t(min(r, last)) * ks;
            dma16_at(kt, row + 16 * ((l & 15) ^ (r & 15)), lds_addr(t.Kn[buf]) + 1024 * n);
            dma16_at(kt + kMlaNope, row + 16 * ((l & 15) ^ ((r & 3) << 2)),
                     lds_addr(t.V[buf]) + 1024 * n);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int n = 2 * w + i, r = 8 * n + (l >> 3);
            dma16_at(pt, uint32_t(min(r, last)) * ps + 16 * ((l & 7) ^ ((r >> 1) & 7)),
                     lds_addr(t.Kp[buf]) + 1024 * n);
        }
    }
};

// LDS byte addresses of this lane's operands in buffer 0; the other buffer,
// the second 32 keys and the 16-key steps are constant offsets from them.
struct Addr {
    uint32_t kn[8], kp[4], v[4];
    template <int kBufs>
    __device__ __forceinline__ Addr(const Lds<kBufs>& t, int l) {
        const int r = l & 31, g = l >> 5, j = l & 15;
#pragma unroll
        for (int m = 0; m < 8; ++m) kn[m] = lds_addr(t.Kn) + r * 256 + 16 * ((2 * m + g) ^ (r & 15));
#pragma unroll
        for (int m = 0; m < 4; ++m)
            kp[m] = lds_addr(t.Kp) + r * 128 + 16 * ((2 * m + g) ^ ((r >> 1) & 7));
        // V^T operand: channel 32 b + l % 32, keys 4g + {0..3, 8..11} (+ 16 s)
        const int vr = 4 * g + (j >> 2), low = 2 * ((l >> 4) & 1) + ((j >> 1) & 1);
#pragma unroll
        for (int b = 0; b < 4; ++b)
            v[b] = lds_addr(t.V) + vr * 256 + 16 * ((4 * b + low) ^ ((vr & 3) << 2)) + 8 * (j & 1);
    }
};

template <int kBuf>
__device__ __forceinline__ bf16x8 k_op(const Addr& a, int b, int m) {
    return m < 8 ? lds_read16(a.kn[m & 7] + kBuf * kBN * kMlaNope * 2 + b * 32 * 256)
                 : lds_read16(a.kp[m & 3] + kBuf * kBN * kMlaPe * 2 + b * 32 * 128);
}

template <int kBuf>
__device__ __forceinline__ bf16x8 v_op(const Addr& a, int s, int b) {
    const uint32_t p = a.v[b] + kBuf * kBN * kMlaV * 2 + s * 16 * 256;
    const u32x2 x = lds_read_tr8(p), y = lds_read_tr8(p + 8 * 256);
    return __builtin_bit_cast(bf16x8, u32x4{x[0], x[1], y[0], y[1]});
}

__device__ __forceinline__ bool v_nonfinite(const uint16_t* V, int l) {
    uint32_t bad = 0;
    const u32x4* p = reinterpret_cast<const u32x4*>(V);
#pragma unroll 4
    for (int i = 0; i < kBN * kMlaV * 2 / 1024; ++i) {
        const u32x4 x = p[64 * i + l];
        bad |= nonfinite_bits(x[0]) | nonfinite_bits(x[1]) | nonfinite_bits(x[2]) | nonfinite_bits(x[3]);
    }
    return __any(bad != 0);
}

// The values of masked tiles that hold infinities or NaN: a product over the
// tile would carry 0 * inf to the queries that do not see that key, so the
// tile's part is added here, from memory, key by key.
__device__ __forceinline__ void add_masked_values(const MlaPrefillArgs& A, const uint16_t* kv,
                                              const uint16_t* pe, const uint16_t* qrow, int from,
                                              int limit, float c, float mu, int g, f32x16* acc) {
    for (int k = from; k < limit; ++k) {
        const uint16_t* row = kv + int64_t(k) * A.kv_stride;
        float s = 0.f;
#pragma unroll 1
        for (int d = 0; d < kMlaNope; ++d)
            s = fmaf(bf16_bits_to_f32(qrow[d]), bf16_bits_to_f32(row[d]), s);
#pragma unroll 1
        for (int d = 0; d < kMlaPe; ++d)
            s = fmaf(bf16_bits_to_f32(qrow[kMlaNope + d]),
                     bf16_bits_to_f32(pe[int64_t(k) * A.pe_stride + d]), s);
        const float p = __builtin_amdgcn_exp2f(fmaf(s, c, -mu));
#pragma unroll
        for (int b = 0; b < 4; ++b)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float v = bf16_bits_to_f32(row[kMlaNope + 32 * b + d_row(i, g)]);
                acc[b][i] = fmaf(p, v, acc[b][i]);
            }
    }
}

template <int kBufs>
__global__ __launch_bounds__(kThreads, 4 / kBufs) void mla_prefill_kernel(const MlaPrefillArgs A) {
    __shared__ __attribute__((aligned(256))) Lds<kBufs> lds;
    const int w = wave_id(), l = threadIdx.x & 63, g = l >> 5;
    // the latest queries (of a causal prompt: those with the most keys) of all
    // heads first, so that the last to start are short (head by head instead:
    // 4% slower at 8192 tokens and 32 heads); workgroups go to the 8 XCDs in
    // turn, so where 8 divides the heads a head's share an XCD's L2
    const int h = blockIdx.x % A.heads;
    PromptTile S;
    if (!find_tile<kBM>(A, A.slots - 1 - int(blockIdx.x) / A.heads, S)) return;
    const int tile = S.tile;
    const int off = S.lk - S.lq;
    const int qi = tile * kBM + 32 * w + (l & 31);   // this lane's query
    const int qlast = min(tile * kBM + kBM, S.lq) - 1;
    const int kend = A.causal ? min(S.lk, qlast + off + 1) : S.lk;
    const int limit = qi >= S.lq ? 0 : (A.causal ? min(S.lk, qi + off + 1) : S.lk);
    // keys that every / any query of this wave sees
    const int wq = tile * kBM + 32 * w;
    const int all_see = A.causal ? min(S.lk, wq + off + 1) : S.lk;
    const int any_see = wq >= S.lq ? 0 : (A.causal ? min(S.lk, min(wq + 31, S.lq - 1) + off + 1) : S.lk);

    const uint16_t* qrow =
        A.q + int64_t(S.q0 + min(qi, S.lq - 1)) * A.q_stride + size_t(h) * kMlaQk;
    bf16x8 qf[12];
#pragma unroll
    for (int m = 0; m < 12; ++m)
        qf[m] = __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4*>(qrow + 16 * m + 8 * g));

    const Dma dma{A, A.kv + int64_t(S.k0) * A.kv_stride + size_t(h) * kMlaKv,
                  A.pe + int64_t(S.k0) * A.pe_stride, w, l, S.lk};
    const int ntiles = kend > 0 ? (kend + kBN - 1) / kBN : 0;
    const float c = A.scale * kLog2e;
    float m = -INFINITY, mu = 0.f, lsum = 0.f;
    f32x16 acc[4] = {};
    int left_from = -1;   // first key of the tiles left to add_masked_values

    const Addr addr(lds, l);
    // the queries have arrived before the first transfer into LDS is issued: no
    // wait of the compiler's own for them stands in the loop (with two tiles'
    // memory it has others, for registers that it keeps in scratch)
#pragma unroll
    for (int mm = 0; mm < 12; ++mm) asm volatile("" : "+v"(qf[mm]));
    auto step = [&](auto buf_c, int n) {
        constexpr int kBuf = decltype(buf_c)::value;
        const int k0 = n * kBN;
        // tile n + kBufs - 1 goes where n - 1 was (behind the last tile it comes
        // again, so that the number of transfers in flight is always the same)
        dma.issue(min(n + kBufs - 1, ntiles - 1) * kBN, lds, (kBuf + kBufs - 1) % kBufs);
        wait_vm<kDma*(kBufs - 1)>();
        raw_barrier();
        if (k0 < any_see) {
            f32x16 s[2] = {};
#pragma unroll
            for (int mm = 0; mm < 12; ++mm) {
#pragma unroll
                for (int b = 0; b < 2; ++b) s[b] = mfma32(k_op<kBuf>(addr, b, mm), qf[mm], s[b]);
                if (mm % 4 == 3) __builtin_amdgcn_sched_barrier(0);
            }
            const bool masked = k0 + kBN > all_see;
            if (masked) {
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (32 * b + d_row(i, 0) >= limit - k0 - 4 * g) s[b][i] = -INFINITY;
            }
            float top = s[0][0];
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int i = 0; i < 16; ++i) top = fmaxf(top, s[b][i]);
            top = fmaxf(top, other_half(top));
            // the reference value moves only when a query outgrows it by 2^8:
            // any reference gives the same quotient
            if (__any((top - m) * c > 8.f || (m == -INFINITY && top > m))) {
                const float mn = fmaxf(m, top);
                const float mun = mn == -INFINITY ? 0.f : mn * c;
                const float a = m == -INFINITY ? 0.f : exp2f(mu - mun);
                m = mn;
                mu = mun;
                lsum *= a;
#pragma unroll
                for (int b = 0; b < 4; ++b)
#pragma unroll
                    for (int i = 0; i < 16; ++i) acc[b][i] *= a;
            }
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    s[b][i] = __builtin_amdgcn_exp2f(fmaf(s[b][i], c, -mu));
                    lsum += s[b][i];
                }
            const bf16x8 p[4] = {pack8<0>(s[0]), pack8<8>(s[0]), pack8<0>(s[1]), pack8<8>(s[1])};
            if (masked && (left_from >= 0 || v_nonfinite(lds.V[kBuf], l))) {
                if (left_from < 0) left_from = k0;
            } else {
#pragma unroll
                for (int b = 0; b < 4; ++b) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) acc[b] = mfma32(v_op<kBuf>(addr, k, b), p[k], acc[b]);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        }
        raw_barrier();
    };
    if (ntiles > 0) {
#pragma unroll
        for (int d = 0; d < kBufs - 1; ++d) dma.issue(min(d, ntiles - 1) * kBN, lds, d);
    }
    for (int n = 0; n < ntiles; n += kBufs) {
        step(std::integral_constant<int, 0>{}, n);
        if (n + 1 < ntiles) step(std::integral_constant<int, 1>{}, n + 1);
        if constexpr (kBufs == 4) {
            if (n + 2 < ntiles) step(std::integral_constant<int, 2>{}, n + 2);
            if (n + 3 < ntiles) step(std::integral_constant<int, 3>{}, n + 3);
        }
    }
    wait_vm<0>();   // nothing may land in memory that is another workgroup's
    if (qi >= S.lq) return;
    if (left_from >= 0)
        add_masked_values(A, dma.kv, dma.pe, qrow, left_from, limit, c, mu, g, acc);
    lsum += other_half(lsum);
    const float inv = lsum > 0.f ? 1.f / lsum : (lsum == 0.f ? 0.f : lsum);
    const int64_t row = int64_t(S.q0 + qi) * A.heads + h;
    if (A.lse && g == 0) A.lse[row] = lsum == 0.f ? -INFINITY : fmaf(mu, kLn2, logf(lsum));
    uint16_t* out = A.o + row * kMlaV;
#pragma unroll
    for (int b = 0; b < 4; ++b)
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
            uint32_t x[2];
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                const f32x2 v = {acc[b][i + 2 * p] * inv, acc[b][i + 2 * p + 1] * inv};
                x[p] = __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
            }
            *reinterpret_cast<u32x2*>(out + 32 * b + d_row(i, g)) = u32x2{x[0], x[1]};
        }
}

}  // namespace

int64_t mla_prefill_slots(int32_t total_q, int32_t num_seqs) {
    return int64_t(total_q) / kBM + num_seqs;
}

// The wide kernel halves what each query reads from LDS, but its workgroups are
// twice as large and one fits a CU: it needs two for every CU, sequences that
// fill them (512 queries on average) and key ranges over which its longer start
// and end (about 15 us a workgroup) count little.  Narrow and wide, us: 8192 tokens x 32
// heads 934 and 858, 4096 x 32 254 and 237, 8 x 1024 over 5120 keys x 16 508
// and 444; on the other side of the rule, 8 x 1024 x 32 188 and 194, 1024 x 128
// 80 and 86, 4096 x 16 163 and 169, 32 x 256 over 512 keys x 16 80 and 124.
static bool prefer_wide(const MlaPrefillArgs& A, int64_t slots) {
    return slots * A.heads >= 2 * kMlaWorkgroups && A.total_q >= int64_t(512) * A.num_seqs &&
           A.total_k >= int64_t(2048) * A.num_seqs;
}

hipError_t launch_mla_prefill(const MlaPrefillArgs& A, hipStream_t stream) {
    const int64_t wide = mla_prefill_wide_slots(A.total_q, A.num_seqs);
    if (prefer_wide(A, wide)) {
        MlaPrefillArgs W = A;
        W.slots = int32_t(wide);
        return launch_mla_prefill_wide(W, stream);
    }
    // four tiles' memory where every workgroup has a CU for itself: 512 queries
    // over 8704 keys x 32 heads 271 us for 323, 2048 x 8 70 for 77, 30 over 1959
    // x 16 64 for 72; two tiles' memory and two workgroups a CU otherwise
    const dim3 grid(unsigned(A.slots * A.heads));
    if (A.slots * A.heads <= kMlaWorkgroups) mla_prefill_kernel<4><<<grid, dim3(kThreads), 0, stream>>>(A);
    else mla_prefill_kernel<2><<<grid, dim3(kThreads), 0, stream>>>(A);
    return hipGetLastError();
}

}  // namespace rda
