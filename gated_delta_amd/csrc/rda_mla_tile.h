// rda_mla_tile.h -- which queries a workgroup of the prompt kernels takes.
#pragma once

#include "rda_internal.h"
#include "rda_mla.h"

namespace rda {

// A block of kBM queries of a packed sequence.
struct PromptTile {
    int q0, lq, k0, lk;   // the sequence's queries and keys
    int tile;             // the block's number in it
};

// The block of query slot `slot`; false where it holds none.  Sequence n owns
// the slots from cu[n] / kBM + n on: at least ceil(lq / kBM) of them, so a slot
// finds its sequence by bisection and no table of blocks is made.
template <int kBM>
__device__ __forceinline__ bool find_tile(const MlaPrefillArgs& A, int slot, PromptTile& s) {
    int lo = 0;
    if (A.cu_q) {
        int hi = A.num_seqs - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (A.cu_q[mid] / kBM + mid <= slot) lo = mid; else hi = mid - 1;
        }
    }
    auto part = [&](const int32_t* cu, int total, int& first, int& len) {
        const int a = cu ? min(max(cu[lo], 0), total) : 0;
        const int b = cu ? min(max(cu[lo + 1], a), total) : total;
        first = a;
        len = b - a;
    };
    part(A.cu_q, A.total_q, s.q0, s.lq);
    part(A.cu_k, A.total_k, s.k0, s.lk);
    s.tile = slot - (s.q0 / kBM + lo);
    return s.tile >= 0 && s.tile < (s.lq + kBM - 1) / kBM;
}

}  // namespace rda
