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
// finds the chunk and reads only that again.
#include <climits>
#include <cmath>

#include "rda_internal.h"
#include "rda_mla.h"

namespace rda {
namespace {

constexpr int kThreads = 256;
constexpr int kPer = kVerifyChunk / kThreads;   // values per thread of a chunk

struct Choice {
    int accepted;         // drafts accepted
    int drafted;          // the refused token, -1 if none was refused
    const float* p;       // target row
    const float* q;       // draft row or nullptr
};

// Every wave derives the same choice: lane i tests draft i.
__device__ __forceinline__ Choice choose(const VerifyArgs& A, int b) {
    const int l = threadIdx.x & 63, D = A.drafts;
    int count = D;
    if (A.num_drafts) count = min(max(A.num_drafts[b], 0), D);
    bool ok = false;
    int d = -1;
    if (l < count) {
        d = A.tokens[int64_t(b) * D + l];
        if (d >= 0 && d < A.vocab) {
            const float p = A.target[(int64_t(b) * (D + 1) + l) * A.target_stride + d];
            const float q = A.draft ? A.draft[(int64_t(b) * D + l) * A.draft_stride + d] : 1.f;
            ok = double(A.uniforms[int64_t(b) * (D + 1) + l]) * double(q) < double(p);
        }
    }
    const uint64_t good = __ballot(ok);
    Choice c;
    c.accepted = good == ~uint64_t(0) ? 64 : __builtin_ctzll(~good);
    const bool refused = c.accepted < count;
    c.drafted = refused ? __shfl(d, c.accepted) : -1;
    c.p = A.target + (int64_t(b) * (D + 1) + c.accepted) * A.target_stride;
    c.q = refused && A.draft ? A.draft + (int64_t(b) * D + c.accepted) * A.draft_stride : nullptr;
    return c;
}

// The weight of token j (`point`: nothing for the refused token); what is not a positive
// finite number weighs nothing.
__device__ __forceinline__ double weight(const Choice& c, bool point, int j, float p, float q) {
    double w = double(p) - double(q);
    if (point && j == c.drafted) w = 0.0;
    return w > 0.0 && w < double(INFINITY) ? w : 0.0;
}

__device__ __forceinline__ double wave_sum(double x) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) x += __shfl_xor(x, d);
    return x;
}

// Sums of w and of p over a chunk.
template <bool kVec>
__global__ __launch_bounds__(kThreads) void verify_sums_kernel(const VerifyArgs A) {
    __shared__ double part[2][4];
    const int b = blockIdx.y, chunk = blockIdx.x;
    const Choice c = choose(A, b);
    const bool point = !A.draft && c.drafted >= 0;
    const int j0 = chunk * kVerifyChunk;
    double sw = 0.0, sp = 0.0;
    if constexpr (kVec) {
        f32x4 p[kPer / 4], q[kPer / 4];
#pragma unroll
        for (int k = 0; k < kPer / 4; ++k) {
            const int j = j0 + 4 * (int(threadIdx.x) + kThreads * k);
            p[k] = j < A.vocab ? *reinterpret_cast<const f32x4*>(c.p + j) : zero4();
            q[k] = c.q && j < A.vocab ? *reinterpret_cast<const f32x4*>(c.q + j) : zero4();
        }
#pragma unroll
        for (int k = 0; k < kPer / 4; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int j = j0 + 4 * (int(threadIdx.x) + kThreads * k) + e;
                sw += weight(c, point, j, p[k][e], q[k][e]);
                sp += weight(c, false, j, p[k][e], 0.f);
            }
    } else {
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const int j = j0 + int(threadIdx.x) + kThreads * k;
            if (j >= A.vocab) break;
            const float p = c.p[j], q = c.q ? c.q[j] : 0.f;
            sw += weight(c, point, j, p, q);
            sp += weight(c, false, j, p, 0.f);
        }
    }
    sw = wave_sum(sw);
    sp = wave_sum(sp);
    if ((threadIdx.x & 63) == 0) {
        part[0][wave_id()] = sw;
        part[1][wave_id()] = sp;
    }
    __syncthreads();
    if (threadIdx.x < 2) {
        const double* x = part[threadIdx.x];
        A.sums[(int64_t(b) * gridDim.x + chunk) * 2 + threadIdx.x] = (x[0] + x[1]) + (x[2] + x[3]);
    }
}

// Inclusive scan over the workgroup's 256 threads.
__device__ __forceinline__ double block_scan(double x, double* s, double& total) {
    const int l = threadIdx.x & 63, w = wave_id();
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const double y = __shfl_up(x, d);
        if (l >= d) x += y;
    }
    __syncthreads();
    if (l == 63) s[w] = x;
    __syncthreads();
    double before = 0.0;
    total = 0.0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if (k < w) before += s[k];
        total += s[k];
    }
    return before + x;
}

__global__ __launch_bounds__(kThreads) void verify_pick_kernel(const VerifyArgs A, int32_t chunks) {
    __shared__ double scan[4], base_s;
    __shared__ int first_s, last_s;
    const int b = blockIdx.x, D = A.drafts;
    const Choice c = choose(A, b);
    const bool point = !A.draft && c.drafted >= 0;
    const double* sums = A.sums + int64_t(b) * chunks * 2;
    // totals of both kinds, then the chunk in which the running sum passes t
    double tw = 0.0, tp = 0.0, total;
    for (int k0 = 0; k0 < chunks; k0 += kThreads) {
        const int k = k0 + int(threadIdx.x);
        block_scan(k < chunks ? sums[2 * k] : 0.0, scan, total);
        tw += total;
        block_scan(k < chunks ? sums[2 * k + 1] : 0.0, scan, total);
        tp += total;
    }
    const bool own = tw > 0.0;   // false: the target's probabilities instead
    double t = double(A.uniforms[int64_t(b) * (D + 1) + D]) * (own ? tw : tp);
    if (threadIdx.x == 0) {
        first_s = INT_MAX;
        last_s = -1;
    }
    double seen = 0.0;
    int pick = -1;
    __syncthreads();
    for (int k0 = 0; k0 < chunks; k0 += kThreads) {
        const int k = k0 + int(threadIdx.x);
        const double x = k < chunks ? sums[2 * k + (own ? 0 : 1)] : 0.0;
        const double incl = seen + block_scan(x, scan, total);
        if (x > 0.0) {
            if (incl > t) atomicMin(&first_s, k);
            atomicMax(&last_s, k);
        }
        __syncthreads();
        if (first_s < INT_MAX) break;
        seen += total;
    }
    __syncthreads();
    const int chunk = first_s < INT_MAX ? first_s : last_s;
    // a number not below 1 passes no border: the last token that weighs
    if (first_s == INT_MAX) t = INFINITY;
    if (chunk >= 0) {
        // what lies before the chunk, summed as above
        const int k0 = chunk / kThreads * kThreads, k = k0 + int(threadIdx.x);
        const double x = k < chunks ? sums[2 * k + (own ? 0 : 1)] : 0.0;
        const double incl = block_scan(x, scan, total);
        if (k == chunk) base_s = seen + (incl - x);
        __syncthreads();
        const double base = base_s;
        if (threadIdx.x == 0) {
            first_s = INT_MAX;
            last_s = -1;
        }
        // the thread's kPer consecutive tokens
        const int j0 = chunk * kVerifyChunk + int(threadIdx.x) * kPer;
        double w[kPer], sum = 0.0;
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            const int j = j0 + e;
            w[e] = 0.0;
            if (j < A.vocab)
                w[e] = own ? weight(c, point, j, c.p[j], c.q ? c.q[j] : 0.f)
                           : weight(c, false, j, c.p[j], 0.f);
            sum += w[e];
        }
        double run = base + (block_scan(sum, scan, total) - sum);
        int first = INT_MAX, last = -1;
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            run += w[e];
            if (w[e] > 0.0) {
                if (run > t && first == INT_MAX) first = j0 + e;
                last = j0 + e;
            }
        }
        if (first < INT_MAX) atomicMin(&first_s, first);
        if (last >= 0) atomicMax(&last_s, last);
        __syncthreads();
        pick = first_s < INT_MAX ? first_s : last_s;
    }
    if (threadIdx.x <= D) {
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
    if (vec)
        verify_sums_kernel<true><<<dim3(unsigned(chunks), unsigned(A.batch)), dim3(kThreads), 0, stream>>>(A);
    else
        verify_sums_kernel<false><<<dim3(unsigned(chunks), unsigned(A.batch)), dim3(kThreads), 0, stream>>>(A);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    verify_pick_kernel<<<dim3(unsigned(A.batch)), dim3(kThreads), 0, stream>>>(A, chunks);
    return hipGetLastError();
}

}  // namespace rda
