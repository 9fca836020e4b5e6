// rda_mla_prefill_wide.hip -- expanded latent attention over long prompts: the
// formulas and the transposed products of rda_mla_prefill.hip with 64 queries
// a wave and 256 a workgroup.
//
// In the narrow kernel every operand read from LDS (1 KiB; the CU moves 128
// bytes a cycle, 32 cycles' worth for one of its four SIMDs, the transposing
// reads of V about 48) feeds one product of 32 cycles, so LDS is as busy as
// the matrix cores; here it feeds two.  One wave fits a SIMD then (Q^T 96,
// O^T 128 accumulation, scores 64 registers), and nothing but the wave itself
// can fill the matrix core while it takes exponentials: step j, 32 keys, runs
//   the products O^T += V^T P^T of step j - 1 beside the maximum of step j,
//   the products S^T of step j + 1 beside the exponentials of step j,
// in slices of two products that are written out in that order.  Keys and
// values of a step arrive by LDS-DMA, six steps' memory in turn.
//
// Measured: 8192 causal tokens of 32 heads 858 us called back to back, 801
// TFLOP/s of the causal half (728 us, 944, between other work); 4096 x 16 over all keys 182 us, 945; 16384 x 32 2692 us, 1021.  A step
// takes about 2600 cycles of which its 40 products are 1280; issue slots are
// half used and about a third of the time goes to waits on LDS.  The clock
// counts too: the same calls on zeros (less switching, higher clock) take 711
// us for 858.  Rows a power of two apart cost some as well: 32 heads with 128
// bytes between rows 798 us.
#include "rda_internal.h"
#include "rda_mla.h"
#include "rda_mla_acc.h"
#include "rda_mla_tile.h"

namespace rda {
namespace {

constexpr int kBM = 256;      // queries per workgroup
constexpr int kBN = 32;       // keys per step
constexpr int kRing = 6;      // steps in LDS
constexpr int kThreads = 256;
constexpr int kDma = 5;       // transfers of a wave per step
constexpr int kQ = 128;       // the first accumulation register of Q^T

// Row r keeps 16-byte granule j at j ^ (r & 15) (Kn), j ^ (r >> 1 & 7) (Kp),
// j ^ (r & 3) << 2 (V).
struct Step {
    uint16_t Kn[kBN * kMlaNope];
    uint16_t Kp[kBN * kMlaPe];
    uint16_t V[kBN * kMlaV];
};
constexpr int kOffKp = kBN * kMlaNope * 2, kOffV = kOffKp + kBN * kMlaPe * 2;
constexpr int kStepBytes = kOffV + kBN * kMlaV * 2;   // 20 KiB
static_assert(sizeof(Step) == kStepBytes, "packed");

struct Lds {
    Step step[kRing];
};

// A wave's part of the step at key k0: 2 + 2 + 1 KiB of Kn, V, Kp, as transfers
// 0 .. 4.  Rows behind the last key repeat it (steps behind the last are fetched
// too, so that the number of transfers in flight is always the same).
struct Dma {
    const MlaPrefillArgs& A;
    const uint16_t* kv;   // first key row of the sequence, this head
    const uint16_t* pe;
    int w, lk;
    uint32_t kn[2], v, kp;   // lane offsets in a whole step

    __device__ __forceinline__ Dma(const MlaPrefillArgs& A_, const uint16_t* kv_, const uint16_t* pe_,
                                   int w_, int lk_, int l)
        : A(A_), kv(kv_), pe(pe_), w(w_), lk(lk_) {
        const uint32_t ks = uint32_t(A.kv_stride) * 2, ps = uint32_t(A.pe_stride) * 2;
        const int r = 8 * w + (l >> 4);
        kn[0] = r * ks + 16 * ((l & 15) ^ (r & 15));
        kn[1] = (r + 4) * ks + 16 * ((l & 15) ^ ((r + 4) & 15));
        v = r * ks + 16 * ((l & 15) ^ ((r & 3) << 2));
        const int rp = 8 * w + (l >> 3);
        kp = rp * ps + 16 * ((l & 7) ^ ((rp >> 1) & 7));
    }
    __device__ __forceinline__ void whole(int i, const uint16_t* kt, const uint16_t* pt,
                                          uint32_t lds) const {
        if (i < 2) dma16_at(kt, kn[i], lds + 1024 * (2 * w + i));
        else if (i < 4)
            dma16_at(kt + kMlaNope + (i - 2) * 4 * A.kv_stride, v, lds + kOffV + 1024 * (2 * w + i - 2));
        else dma16_at(pt, kp, lds + kOffKp + 1024 * w);
    }
    // the step that may hold the last key, or lies behind it
    __device__ __forceinline__ void partial(int k0, uint32_t lds, int lane) const {
        const int l = here(lane);
        const int from = min(k0, lk - 1), last = lk - 1 - from;
        const uint16_t* kt = kv + int64_t(from) * A.kv_stride;
        const uint16_t* pt = pe + int64_t(from) * A.pe_stride;
        const uint32_t ks = uint32_t(A.kv_stride) * 2, ps = uint32_t(A.pe_stride) * 2;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int n = 2 * w + i, r = 4 * n + (l >> 4);
            const uint32_t row = uint32_t(min(r, last)) * ks;
            dma16_at(kt, row + 16 * ((l & 15) ^ (r & 15)), lds + 1024 * n);
            dma16_at(kt + kMlaNope, row + 16 * ((l & 15) ^ ((r & 3) << 2)), lds + kOffV + 1024 * n);
        }
        const int r = 8 * w + (l >> 3);
        dma16_at(pt, uint32_t(min(r, last)) * ps + 16 * ((l & 7) ^ ((r >> 1) & 7)),
                 lds + kOffKp + 1024 * w);
    }
    __device__ __forceinline__ void issue(int k0, uint32_t lds, int lane) const {
        if (k0 + kBN <= lk) {
            const uint16_t* kt = kv + int64_t(k0) * A.kv_stride;
            const uint16_t* pt = pe + int64_t(k0) * A.pe_stride;
#pragma unroll
            for (int i = 0; i < kDma; ++i) whole(i, kt, pt, lds);
        } else {
            partial(k0, lds, lane);
        }
    }
};

// LDS byte offsets of this lane's operands from a step's start.
struct Lane {
    int kn, kp, v;
    __device__ __forceinline__ explicit Lane(int l) {
        const int r = l & 31, g = l >> 5, j = l & 15;
        kn = r * 256 + 16 * (g ^ (r & 15));
        kp = kOffKp + r * 128 + 16 * (g ^ ((r >> 1) & 7));
        // V^T operand: channel l % 32, keys 4g + {0..3, 8..11}
        const int vr = 4 * g + (j >> 2), low = 2 * ((l >> 4) & 1) + ((j >> 1) & 1);
        v = kOffV + vr * 256 + 16 * (low ^ ((vr & 3) << 2)) + 8 * (j & 1);
    }
};

struct KeyAddr {
    uint32_t kn, kp;
    __device__ __forceinline__ KeyAddr(const Lane& a, uint32_t step)
        : kn(here(int(step) + a.kn)), kp(here(int(step) + a.kp)) {}
    // values 16 m + 8 g .. of key l % 32 (a step starts at a multiple of 512)
    __device__ __forceinline__ bf16x8 op(int m) const {
        return lds_read16(m < 8 ? kn ^ (32 * m) : kp ^ (32 * (m - 8)));
    }
};

struct ValAddr {
    uint32_t v;
    __device__ __forceinline__ ValAddr(const Lane& a, uint32_t step) : v(here(int(step) + a.v)) {}
    // channels 32 b + l % 32, keys 16 s + 4g + {0..3, 8..11}
    __device__ __forceinline__ bf16x8 op(int b, int s) const {
        const uint32_t p = (v ^ (64 * b)) + s * 16 * 256;
        const u32x2 x = lds_read_tr8(p), y = lds_read_tr8(p + 8 * 256);
        return __builtin_bit_cast(bf16x8, u32x4{x[0], x[1], y[0], y[1]});
    }
};

__device__ __forceinline__ bool v_nonfinite(uint32_t V, int l) {
    uint32_t bad = 0;
#pragma unroll
    for (int i = 0; i < kBN * kMlaV * 2 / 1024; ++i) {
        const u32x4 x = __builtin_bit_cast(u32x4, lds_read16(V + 1024 * i + 16 * l));
        bad |= nonfinite_bits(x[0]) | nonfinite_bits(x[1]) | nonfinite_bits(x[2]) | nonfinite_bits(x[3]);
    }
    return __any(bad != 0);
}

// The running reference, sum and probabilities of 32 queries (one a lane, twice).
struct Rows {
    float mu = 0.f;           // the reference, times c
    float most = -INFINITY;   // scores up to here keep it: (mu + 8) / c
    float lsum = 0.f;
    bf16x8 p[2];              // probabilities of the step before
};

// Moves the reference up to the score `top`; the factor of the old sums.
__device__ __forceinline__ float move_up(Rows& x, float top, float c) {
    const bool none = x.most == -INFINITY;
    const float mun = top == -INFINITY ? x.mu : none ? top * c : fmaxf(x.mu, top * c);
    const float a = none ? 0.f : __builtin_amdgcn_exp2f(x.mu - mun);
    if (top != -INFINITY) x.most = (mun + 8.f) / c;
    x.mu = mun;
    x.lsum *= a;
    return a;
}

// Four channels of one query's values over the keys [from, limit): masked steps
// that hold infinities or NaN, where a product over the step would carry 0 * inf
// to the queries that do not see that key.  From memory, key by key.
__device__ __noinline__ f32x4 masked_values(const uint16_t* kv, int64_t kv_stride,
                                            const uint16_t* pe, int64_t pe_stride,
                                            const uint16_t* q, int from, int limit, float c,
                                            float mu, int ch) {
    f32x4 sum = zero4();
    for (int k = from; k < limit; ++k) {
        const uint16_t* row = kv + int64_t(k) * kv_stride;
        float s = 0.f;
        for (int d = 0; d < kMlaNope; ++d) s = fmaf(bf16_bits_to_f32(q[d]), bf16_bits_to_f32(row[d]), s);
        for (int d = 0; d < kMlaPe; ++d)
            s = fmaf(bf16_bits_to_f32(q[kMlaNope + d]), bf16_bits_to_f32(pe[int64_t(k) * pe_stride + d]), s);
        const float p = __builtin_amdgcn_exp2f(fmaf(s, c, -mu));
        for (int i = 0; i < 4; ++i) sum[i] = fmaf(p, bf16_bits_to_f32(row[kMlaNope + ch + i]), sum[i]);
    }
    return sum;
}

// Products of 32 keys' values 16 m .. with both blocks of queries.
template <int kM>
__device__ __forceinline__ void products(f32x16 (&s)[2], bf16x8 k) {
    if constexpr (kM == 0) {
        scores_first_acc<kQ>(s[0], k);
        scores_first_acc<kQ + 48>(s[1], k);
    } else {
        scores_next_acc<kQ + 4 * kM>(s[0], k);
        scores_next_acc<kQ + 48 + 4 * kM>(s[1], k);
    }
}

__global__ __launch_bounds__(kThreads, 1) void mla_prefill_wide_kernel(const MlaPrefillArgs A) {
    __shared__ __attribute__((aligned(1024))) Lds lds;
    const int w = wave_id(), l = threadIdx.x & 63, g = l >> 5;
    // the latest queries (of a causal prompt: those with the most keys) of all
    // heads first; a head's workgroups share an XCD's L2 where 8 divides the
    // heads, since workgroups go to the 8 XCDs in turn
    const int h = blockIdx.x % A.heads;
    PromptTile S;
    if (!find_tile<kBM>(A, A.slots - 1 - int(blockIdx.x) / A.heads, S)) return;
    const int off = S.lk - S.lq, q0 = S.tile * kBM;
    const int wq = q0 + 64 * w;                        // this wave's first query
    const int qlast = min(q0 + kBM, S.lq) - 1;
    const int kend = A.causal ? min(S.lk, qlast + off + 1) : S.lk;
    const int nsteps = kend > 0 ? (kend + kBN - 1) / kBN : 0;
    // keys that every / any query of this wave sees
    const int all_see = A.causal ? min(S.lk, wq + off + 1) : S.lk;
    const int any_see = wq >= S.lq ? 0 : (A.causal ? min(S.lk, min(wq + 63, S.lq - 1) + off + 1) : S.lk);
    const int own = any_see > 0 ? (any_see + kBN - 1) / kBN : 0;   // this wave's steps

    const float c = A.scale * kLog2e;
    Rows R[2];
    // Q^T: block x, values 16 m .. in the accumulation registers from
    // 128 + 4 (12 x + m) on
    const uint16_t* const qbase = A.q + size_t(h) * kMlaQk;
    unrolled<2>([&](auto xx) {
        constexpr int x = decltype(xx)::value;
        const int qi = wq + 32 * x + (l & 31);
        const uint16_t* qrow = qbase + int64_t(S.q0 + min(qi, S.lq - 1)) * A.q_stride;
        bf16x8 qf[12];
#pragma unroll
        for (int m = 0; m < 12; ++m)
            qf[m] = __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4*>(qrow + 16 * m + 8 * g));
        unrolled<12>([&](auto q) {
            constexpr int m = decltype(q)::value;
            acc_put<kQ + 48 * x + 4 * m>(qf[m]);
        });
    });
    unrolled<128>([](auto q) { acc_clear<decltype(q)::value>(); });

    // keys that this lane's query of block x sees
    auto limit_of = [&](int x, int lane_id) {
        const int qi = wq + 32 * x + lane_id;
        return qi >= S.lq ? 0 : (A.causal ? min(S.lk, qi + off + 1) : S.lk);
    };
    const Lane lane(l);
    const Dma dma(A, A.kv + int64_t(S.k0) * A.kv_stride + size_t(h) * kMlaKv,
                  A.pe + int64_t(S.k0) * A.pe_stride, w, S.lk, l);
    const uint32_t lds0 = lds_addr(&lds.step[0]);
    f32x16 sc[2][2];          // scores of the step at hand and of the next, in turn
    bf16x8 vo[8];             // value operands of the step before
    int left_from = -1;       // first key of the steps left to masked_values
    bool skip = true;         // the step before has no products (to come)

    if (nsteps > 0) {
#pragma unroll 1
        for (int d = 0; d < 4; ++d) dma.issue(d * kBN, lds0 + d * kStepBytes, l);
        wait_vm<3 * kDma>();
        raw_barrier();
        if (own > 0) {
            const KeyAddr ka(lane, lds0);
            unrolled<12>([&](auto q) {
                constexpr int m = decltype(q)::value;
                const bf16x8 k = ka.op(m);
                products<m>(sc[0], k);
            });
        }
    }
    uint32_t cur = lds0;   // step j's memory
    constexpr uint32_t kRingBytes = kRing * kStepBytes;
    const uint16_t* kt = dma.kv + int64_t(4 * kBN) * A.kv_stride;   // step j + 4
    const uint16_t* pt = dma.pe + int64_t(4 * kBN) * A.pe_stride;
    const int64_t kstep = int64_t(kBN) * A.kv_stride, pstep = int64_t(kBN) * A.pe_stride;
    auto step = [&](int j, f32x16 (&s)[2], f32x16 (&next)[2]) {
        const int k0 = j * kBN;
        const uint32_t after = cur + kStepBytes < lds0 + kRingBytes ? cur + kStepBytes : lds0;
        const uint32_t before = cur > lds0 ? cur - kStepBytes : lds0 + kRingBytes - kStepBytes;
        const uint32_t two_before = before > lds0 ? before - kStepBytes : lds0 + kRingBytes - kStepBytes;
        wait_vm<2 * kDma>();
        raw_barrier();   // step j + 1 has landed, step j - 2 is read
        // step j + 4 goes where j - 2 was; between the products below, if those
        // come and the step is a whole one
        const bool whole = k0 + 5 * kBN <= S.lk, beside = whole && j < own && !skip;
        if (!beside) {
            if (whole) {
#pragma unroll
                for (int i = 0; i < kDma; ++i) dma.whole(i, kt, pt, two_before);
            } else {
                dma.partial(k0 + 4 * kBN, two_before, l);
            }
        }
        if (j < own) {
            const KeyAddr ka(lane, after);
            const bool masked = k0 + kBN > all_see;
            if (masked) {
                scores_done(s[0]);
                scores_done(s[1]);
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int left = limit_of(x, here(l & 31)) - k0 - 4 * g;
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (d_row(i, 0) >= left) s[x][i] = -INFINITY;
                }
            }
            // products of the step before beside the maximum of this one (its
            // scores are not read before four products have gone by)
            float top[2];
            bf16x8 ko[12];   // row operands of the step after
            auto maximum = [&](int n) {   // slice n of 6
                if (n == 0) {
                    top[0] = s[0][0];
                    top[1] = s[1][0];
                }
#pragma unroll
                for (int i = n == 0 ? 1 : 3 * n - 2; i < (n == 5 ? 16 : 3 * n + 1); ++i) {
                    top[0] = fmaxf(top[0], s[0][i]);
                    top[1] = fmaxf(top[1], s[1][i]);
                }
            };
            if (skip) {
                scores_done(s[0]);
                scores_done(s[1]);
#pragma unroll
                for (int n = 0; n < 6; ++n) maximum(n);
#pragma unroll
                for (int m = 0; m < 12; ++m) ko[m] = ka.op(m);
            } else {
                unrolled<8>([&](auto q) {
                    constexpr int n = decltype(q)::value;
                    ko[n] = ka.op(n);
                    if constexpr (n >= 4) ko[n + 4] = ka.op(n + 4);
                    __builtin_amdgcn_sched_barrier(0);
                    acc_product<n % 4, n == 0>(vo[n], R[0].p[n / 4]);
                    acc_product<4 + n % 4, false>(vo[n], R[1].p[n / 4]);
                    if constexpr (n >= 1 && n <= kDma)
                        if (beside) dma.whole(n - 1, kt, pt, two_before);
                    if constexpr (n >= 2) {
                        maximum(n - 2);
                        asm volatile("" : "+v"(top[0]), "+v"(top[1]));
                    }
                    __builtin_amdgcn_sched_barrier(0);
                });
            }
            // the reference moves only when a query outgrows it by 2^8 (either
            // half of its keys tells; then both halves' maximum counts)
            if (__any(top[0] > R[0].most || top[1] > R[1].most)) {
                const bool first = __all(R[0].most == -INFINITY && R[1].most == -INFINITY);
                const float a0 = move_up(R[0], fmaxf(top[0], other_half(top[0])), c);
                const float a1 = move_up(R[1], fmaxf(top[1], other_half(top[1])), c);
                if (!first) {
                    settle();
                    unrolled<64>([a0](auto q) { acc_scale<decltype(q)::value>(a0); });
                    unrolled<64>([a1](auto q) { acc_scale<64 + decltype(q)::value>(a1); });
                }
            }
            // the next step's scores beside the exponentials of this one (the
            // last step's next one is not used)
            const ValAddr va(lane, cur);
            unrolled<12>([&](auto q) {
                constexpr int m = decltype(q)::value;
                // (the values are for the products after this step)
                if constexpr (m >= 2 && m < 10) vo[m - 2] = va.op((m - 2) % 4, (m - 2) / 4);
                __builtin_amdgcn_sched_barrier(0);
                products<m>(next, ko[m]);
                if constexpr (m < 11) {
#pragma unroll
                    for (int e = 3 * m; e < (m == 10 ? 32 : 3 * m + 3); ++e) {
                        const int x = e >> 4, i = e & 15;
                        float p = __builtin_amdgcn_exp2f(fmaf(s[x][i], c, -R[x].mu));
                        asm volatile("" : "+v"(p));   // (here, not where it is used)
                        s[x][i] = p;
                        R[x].lsum += p;
                    }
                    asm volatile("" : "+v"(R[0].lsum), "+v"(R[1].lsum));
                    auto pack = [&](int x, int half) {
                        R[x].p[half] = half ? pack8<8>(s[x]) : pack8<0>(s[x]);
                        asm volatile("" : "+v"(R[x].p[half]));
                    };
                    if constexpr (m == 3) pack(0, 0);
                    if constexpr (m == 6) pack(0, 1);
                    if constexpr (m == 8) pack(1, 0);
                } else {
                    R[1].p[1] = pack8<8>(s[1]);
                    asm volatile("" : "+v"(R[1].p[1]));
                }
                __builtin_amdgcn_sched_barrier(0);
            });
            // a masked step whose values hold infinities or NaN is left to the end
            skip = masked && (left_from >= 0 || v_nonfinite(cur + kOffV, l));
            if (skip && left_from < 0) left_from = k0;
            if (j + 1 == own && !skip) {   // the last step's products
                unrolled<8>([&](auto q) {
                    constexpr int n = decltype(q)::value;
                    acc_product<n % 4>(vo[n], R[0].p[n / 4]);
                    acc_product<4 + n % 4>(vo[n], R[1].p[n / 4]);
                });
            }
        }
        cur = after;
        kt += kstep;
        pt += pstep;
    };
    for (int j = 0; j < nsteps; j += 2) {
        step(j, sc[0], sc[1]);
        if (j + 1 < nsteps) step(j + 1, sc[1], sc[0]);
    }
    wait_vm<0>();   // the steps behind the last: nothing may land later
    settle();
    raw_barrier();  // the steps are read

    // out row by row by way of LDS, 32 queries of the wave at a time
    constexpr int kStride = kMlaV * 4 + 16;
    const uint32_t stage = lds0 + w * 32 * kStride;
    static_assert(4 * 32 * kStride <= int(sizeof(Lds)), "the waves' rows fit");
    unrolled<2>([&](auto xx) {
        constexpr int x = decltype(xx)::value;
        Rows& r = R[x];
        r.lsum += other_half(r.lsum);
        const float inv = r.lsum == 0.f ? 0.f : 1.f / r.lsum;
        const int qi = wq + 32 * x + (l & 31);
        if (A.lse && l < 32 && qi < S.lq)
            A.lse[int64_t(S.q0 + qi) * A.heads + h] =
                r.lsum == 0.f ? -INFINITY : fmaf(r.mu, kLn2, logf(r.lsum));
        unrolled<16>([&](auto q) {
            constexpr int n = decltype(q)::value;   // channels 32 (n / 4) + 8 (n % 4) + 4g ..
            acc_store<16 * x + n, 128 * (n / 4) + 32 * (n % 4)>(stage + (l & 31) * kStride + 16 * g);
        });
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll 4
        for (int i = 0; i < 16; ++i) {
            const int row = 2 * i + g, qr = wq + 32 * x + row;
            f32x4 v = __builtin_bit_cast(f32x4, lds_read16(stage + row * kStride + 16 * (l & 31)));
            if (left_from >= 0)
                v += masked_values(dma.kv, A.kv_stride, dma.pe, A.pe_stride,
                                   qbase + int64_t(S.q0 + min(qr, S.lq - 1)) * A.q_stride, left_from,
                                   limit_of(x, row), c, __shfl(r.mu, row), 4 * (l & 31));
            const float f = __shfl(inv, row);
            if (qr < S.lq)
                *reinterpret_cast<u32x2*>(A.o + (int64_t(S.q0 + qr) * A.heads + h) * kMlaV + 4 * (l & 31)) =
                    u32x2{pack_bf16(v[0] * f, v[1] * f), pack_bf16(v[2] * f, v[3] * f)};
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    });
}

}  // namespace

int64_t mla_prefill_wide_slots(int32_t total_q, int32_t num_seqs) {
    return int64_t(total_q) / kBM + num_seqs;
}

hipError_t launch_mla_prefill_wide(const MlaPrefillArgs& A, hipStream_t stream) {
    mla_prefill_wide_kernel<<<dim3(unsigned(A.slots * A.heads)), dim3(kThreads), 0, stream>>>(A);
    return hipGetLastError();
}

}  // namespace rda
