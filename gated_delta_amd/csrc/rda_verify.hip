// rda_verify.hip -- verification of drafted tokens against the target's
// probabilities with given random numbers.
//
// Draft i of a sequence is accepted while u_i q_i(d_i) < p_i(d_i) (the
// probability of accepting is min(1, p / q)); with r the number accepted, the
// next token is the smallest j with sum_{j' <= j} w_j' > u_D sum w, where
//   w = max(p_r - q_r, 0)  after a refusal   (q_r = 1 at d_r where the drafts
//   w = p_r                after the last     carry no probabilities)
// (u_D, the number behind the drafts' own: after a refusal u_r is known to be
// large, and drawing with it would prefer late tokens)
// and w = p_r also where that leaves nothing.  The products and sums are in
// 64 bits: the index that they pick does not depend on the order of the sum
// but where the random number lies within 2^-52 of a border.
//
// One row of the vocabulary (two with draft probabilities) is read per
// sequence, whatever the number of drafts.  The sums kernel cuts it into
// chunks so that a small batch fills the chip too; every workgroup derives r
// itself, from a few scalars.  The pick kernel, one workgroup per sequence,
// finds the chunk (each of its waves by itself, up to 64 chunks in one scan)
// and reads only that again.  256 sequences of 259840 tokens: 85 us, 5.1
// TB/s for the 437 MB that are fetched (a target row each, and a draft row for
// the 164 sequences with a refusal), of which the sums kernel takes 76 at 5.6;
// 8 sequences of 32003: 17.9 us, the two launches and a chain of small loads.
#include <climits>
#include <cmath>

#include "rda_internal.h"
#include "rda_mla.h"

namespace rda {
namespace {

constexpr int kThreads = 256;

struct Choice {
    int accepted;         // drafts accepted
    bool refused;         // one was refused
    int drafted;          // that token, -1 where it is outside the vocabulary
    const float* p;       // target row
    const float* q;       // draft row or nullptr
};

constexpr int kNoneRefused = INT_MIN;   // in the workspace, in a refused token's place
typedef double f64x2 __attribute__((ext_vector_type(2)));

// The rows of probabilities that the choice leads to.
__device__ __forceinline__ void set_rows(const VerifyArgs& A, int b, Choice& c) {
    const int D = A.drafts;
    c.p = A.target + (int64_t(b) * (D + 1) + c.accepted) * A.target_stride;
    c.q = c.refused && A.draft ? A.draft + (int64_t(b) * D + c.accepted) * A.draft_stride : nullptr;
}

// Every wave derives the same choice: lane i tests draft i.
__device__ __forceinline__ Choice choose(const VerifyArgs& A, int b) {
    const int l = threadIdx.x & 63, D = A.drafts;
    int count = D;
    if (A.num_drafts) count = min(max(A.num_drafts[b], 0), D);
    bool ok = false;
    int d = -1;
    if (l < count) {
        d = A.tokens[int64_t(b) * D + l];
        if (d < 0 || d >= A.vocab) {
            d = -1;   // refused, whatever it is: no value of the caller's is kept as a mark
        } else {
            const float p = A.target[(int64_t(b) * (D + 1) + l) * A.target_stride + d];
            const float q = A.draft ? A.draft[(int64_t(b) * D + l) * A.draft_stride + d] : 1.f;
            ok = double(A.uniforms[int64_t(b) * (D + 1) + l]) * double(q) < double(p);
        }
    }
    const uint64_t good = __ballot(ok);
    Choice c;
    c.accepted = good == ~uint64_t(0) ? 64 : __builtin_ctzll(~good);
    c.refused = c.accepted < count;
    c.drafted = c.refused ? __shfl(d, c.accepted) : -1;
    set_rows(A, b, c);
    return c;
}

// The weight of token j (`point`: nothing for the refused token); nothing where it or the
// target's probability is not a positive finite number.
__device__ __forceinline__ double weight(const Choice& c, bool point, int j, float p, float q) {
    double w = double(p) - double(q);
    if (!(p > 0.f) || (point && j == c.drafted)) w = 0.0;
    return w > 0.0 && w < double(INFINITY) ? w : 0.0;
}

__device__ __forceinline__ double wave_sum(double x) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) x += __shfl_xor(x, d);
    return x;
}

// A thread's four consecutive tokens of each quarter of a chunk (quarter k: from
// 1024 k + 4 thread): 16-byte loads, and in order quarter by quarter.
struct Piece {
    f32x4 p[4], q[4];
};

template <bool kVec>
__device__ __forceinline__ Piece load_piece(const Choice& c, int vocab, int chunk) {
    static_assert(kVerifyChunk == 4 * 4 * kThreads, "four quarters of four tokens a thread");
    Piece x;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int j = chunk * kVerifyChunk + 4 * (int(threadIdx.x) + kThreads * k);
        if constexpr (kVec) {   // vocab is a multiple of 4
            x.p[k] = j < vocab ? *reinterpret_cast<const f32x4*>(c.p + j) : zero4();
            x.q[k] = c.q && j < vocab ? *reinterpret_cast<const f32x4*>(c.q + j) : zero4();
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x.p[k][e] = j + e < vocab ? c.p[j + e] : 0.f;
                x.q[k][e] = c.q && j + e < vocab ? c.q[j + e] : 0.f;
            }
        }
    }
    return x;
}

// Sums of w and of p over a chunk; chunk 0's workgroup also writes the choice.
template <bool kVec>
__global__ __launch_bounds__(kThreads) void verify_sums_kernel(const VerifyArgs A) {
    __shared__ double part[2][4];
    const int b = blockIdx.y, chunk = blockIdx.x;
    const Choice c = choose(A, b);
    const bool point = !A.draft && c.drafted >= 0;
    if (chunk == 0 && threadIdx.x == 0) {
        A.choice[2 * b] = c.accepted;
        A.choice[2 * b + 1] = c.refused ? c.drafted : kNoneRefused;
    }
    const Piece x = load_piece<kVec>(c, A.vocab, chunk);
    double sw = 0.0, sp = 0.0;
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int j = chunk * kVerifyChunk + 4 * (int(threadIdx.x) + kThreads * k) + e;
            sw += weight(c, point, j, x.p[k][e], x.q[k][e]);
            sp += weight(c, false, j, x.p[k][e], 0.f);
        }
    sw = wave_sum(sw);
    sp = wave_sum(sp);
    if ((threadIdx.x & 63) == 0) {
        part[0][wave_id()] = sw;
        part[1][wave_id()] = sp;
    }
    __syncthreads();
    if (threadIdx.x < 2) {
        const double* y = part[threadIdx.x];
        A.sums[(int64_t(b) * gridDim.x + chunk) * 2 + threadIdx.x] = (y[0] + y[1]) + (y[2] + y[3]);
    }
}

// Inclusive scan over a wave.
__device__ __forceinline__ double wave_scan(double x) {
    const int l = threadIdx.x & 63;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const double y = __shfl_up(x, d);
        if (l >= d) x += y;
    }
    return x;
}

template <bool kVec>
__global__ __launch_bounds__(kThreads) void verify_pick_kernel(const VerifyArgs A, int32_t chunks) {
    __shared__ double scan[4][4];
    __shared__ int first_s, last_s;
    const int b = blockIdx.x, D = A.drafts, l = threadIdx.x & 63, w = wave_id();
    const double* sums = A.sums + int64_t(b) * chunks * 2;
    const f64x2 mine = l < chunks ? *reinterpret_cast<const f64x2*>(sums + 2 * l) : f64x2{0.0, 0.0};
    const double u = A.uniforms[int64_t(b) * (D + 1) + D];
    Choice c;
    c.accepted = A.choice[2 * b];
    const int drafted = A.choice[2 * b + 1];
    c.refused = drafted != kNoneRefused;
    c.drafted = c.refused ? drafted : -1;
    set_rows(A, b, c);
    const bool point = !A.draft && c.drafted >= 0;
    if (threadIdx.x == 0) {
        first_s = INT_MAX;
        last_s = -1;
    }
    // the total of w, or where that is nothing of p (every wave for itself)
    const int groups = (chunks + 63) / 64;
    auto part_of = [&](int k0, int kind) {
        const int k = k0 + l;
        return k0 == 0 ? mine[kind] : k < chunks ? sums[2 * k + kind] : 0.0;
    };
    double total = 0.0;
    int kind = 0;
    for (; kind < 2; ++kind) {
        for (int n = 0; n < groups; ++n) total += wave_sum(part_of(64 * n, kind));
        if (total > 0.0) break;
    }
    int pick = -1;
    if (kind < 2) {
        // the chunk in which the running sum passes t, and what lies before it;
        // a number not below 1 passes no border: the last chunk that weighs
        double t = u * total, seen = 0.0, base = 0.0;
        int chunk = -1, last_chunk = -1;
        for (int n = 0; n < groups && chunk < 0; ++n) {
            const double x = part_of(64 * n, kind), incl = wave_scan(x);
            const uint64_t over = __ballot(x > 0.0 && seen + incl > t), some = __ballot(x > 0.0);
            if (over) {
                const int k = __builtin_ctzll(over);
                chunk = 64 * n + k;
                base = seen + __shfl(incl - x, k);
            } else if (some) {
                last_chunk = 64 * n + 63 - __builtin_clzll(some);
            }
            seen += __shfl(incl, 63);
        }
        if (chunk < 0) {
            chunk = last_chunk;
            t = INFINITY;
        }
        const Piece x = load_piece<kVec>(c, A.vocab, chunk);
        double v[4][4], sum[4], incl[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            sum[k] = 0.0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int j = chunk * kVerifyChunk + 4 * (int(threadIdx.x) + kThreads * k) + e;
                v[k][e] = kind == 0 ? weight(c, point, j, x.p[k][e], x.q[k][e])
                                    : weight(c, false, j, x.p[k][e], 0.f);
                sum[k] += v[k][e];
            }
            incl[k] = wave_scan(sum[k]);
            if (l == 63) scan[k][w] = incl[k];
        }
        __syncthreads();
        int first = INT_MAX, last = -1;
        double before = base;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            double run = before;
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                if (y < w) run += scan[k][y];
                before += scan[k][y];
            }
            run += incl[k] - sum[k];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int j = chunk * kVerifyChunk + 4 * (int(threadIdx.x) + kThreads * k) + e;
                run += v[k][e];
                if (v[k][e] > 0.0) {
                    if (run > t && first == INT_MAX) first = j;
                    last = j;
                }
            }
        }
        if (first < INT_MAX) atomicMin(&first_s, first);
        if (last >= 0) atomicMax(&last_s, last);
        __syncthreads();
        pick = first_s < INT_MAX ? first_s : last_s;
    }
    if (int(threadIdx.x) <= D) {
        const int i = threadIdx.x;
        A.out[int64_t(b) * (D + 1) + i] =
            i < c.accepted ? A.tokens[int64_t(b) * D + i] : (i == c.accepted ? pick : -1);
    }
    if (threadIdx.x == 0) A.accept[b] = c.accepted + 1;
}

}  // namespace

int32_t verify_chunks(int32_t vocab) { return int32_t((int64_t(vocab) + kVerifyChunk - 1) / kVerifyChunk); }

hipError_t launch_verify(const VerifyArgs& A, hipStream_t stream) {
    const int32_t chunks = verify_chunks(A.vocab);
    const bool vec = A.vocab % 4 == 0 && A.target_stride % 4 == 0 && (!A.draft || A.draft_stride % 4 == 0);
    const dim3 grid{unsigned(chunks), unsigned(A.batch)};
    if (vec) verify_sums_kernel<true><<<grid, dim3(kThreads), 0, stream>>>(A);
    else verify_sums_kernel<false><<<grid, dim3(kThreads), 0, stream>>>(A);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    if (vec) verify_pick_kernel<true><<<dim3(unsigned(A.batch)), dim3(kThreads), 0, stream>>>(A, chunks);
    else verify_pick_kernel<false><<<dim3(unsigned(A.batch)), dim3(kThreads), 0, stream>>>(A, chunks);
    return hipGetLastError();
}

}  // namespace rda
