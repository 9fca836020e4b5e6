// rda_mla_decode.hip -- absorbed latent attention over a paged latent cache.
//
// A cached row c_j holds 512 latent values and 64 shared key channels.  Query
// row i (one new token and head, 576 values) gives
//   s_ij = scale q_i . c_j,  o_i = sum_j exp(s_ij - m_i) c_j[:512] / l_i,
// over the rows of the sequence that its token sees and over the prefix rows,
// which every query sees.
//
// Every cached row serves as key and as value of all heads, so it is read
// from memory once for all the query rows of a workgroup: 1152 bytes against
// 2176 operations per query row.  As in the prefill the products are
// transposed, S^T = C Q^T and O^T = C^T P^T, a lane owns one query row, and P
// stays in registers.  Two waves hold the same 32 query rows (576 x 32 bf16
// of Q, 144 registers) and half of the latent channels each (256 x 32 fp32 of
// O^T, 128 registers): both form S^T, which saves the exchange.  The 4 waves
// of a workgroup are kRG such pairs that share tiles of 32 cached rows x
// 2 / kRG pairs that take tiles in turn and merge their sums at the end.
//
// The work is a list of tiles, unit after unit (a unit: the query rows of one
// sequence, or a block of all query rows for the prefix), cut into equal
// pieces, one per workgroup, whatever the sequences' lengths: they are read
// on the device.  A workgroup that covers a whole unit writes its output; the
// others write partial sums that the combine kernel joins.
#include "rda_internal.h"
#include "rda_mla.h"

namespace rda {
namespace {

constexpr int kThreads = 256;
constexpr int kTile = 32;                          // cached rows per tile
constexpr int kRowBytes = kMlaRow * 2;             // 1152
constexpr int kLatBytes = kMlaLatent * 2, kPeBytes = kMlaPe * 2;
constexpr int kTileBytes = kTile * kRowBytes;      // 36864
constexpr int kGroups = kMlaLatent / 4;            // 4-channel groups of an output row

typedef const __attribute__((address_space(4))) int32_t const_i32;

// What rows behind the last one are read as.
__device__ const __attribute__((aligned(16))) uint32_t kZeros[kLatBytes / 4] = {};

// A tile keeps its rows' latent parts (64 granules of 16 bytes each, granule
// j of row r at j ^ swz(r)), then their shared key channels (8 granules, j at
// j ^ (r >> 1 & 7)): sixteen rows read at one granule, and eight rows at two
// adjacent ones (transposing reads), fall on distinct banks.
struct Tile {
    unsigned char lat[kTile * kLatBytes];
    unsigned char pe[kTile * kPeBytes];
};

struct Lds {
    Tile tile[4];
    float ml[4][2][32];     // (mu, l) of each wave's rows
    int scan[8];
    int unit, first;        // where this workgroup's piece begins
};

// LDS byte offsets of this lane's operands, from a tile's start: the others
// differ by exclusive-or of granule bits and by constants.
struct Addr {
    int k, pe, v;
    __device__ __forceinline__ Addr(int k_, int pe_, int v_) : k(k_), pe(pe_), v(v_) {}
    __device__ __forceinline__ explicit Addr(int l) {
        const int r = l & 31, g = l >> 5, j = l & 15;
        k = r * kLatBytes + 16 * (g ^ swz(r));
        pe = kTile * kLatBytes + r * kPeBytes + 16 * (g ^ ((r >> 1) & 7));
        // C^T operand: channel l % 32, rows 4g + {0..3}
        const int vr = 4 * g + (j >> 2), low = 2 * ((l >> 4) & 1) + ((j >> 1) & 1);
        v = vr * kLatBytes + 16 * (low ^ swz(vr)) + 8 * (j & 1);
    }
};

// Row operand of the tile at LDS address `tile`: values 16 m + 8 g ..
__device__ __forceinline__ bf16x8 k_op(const Addr& a, uint32_t tile, int m) {
    return lds_read16(m < 32 ? tile + (a.k ^ (32 * (m & 7))) + 256 * (m >> 3)
                             : tile + (a.pe ^ (32 * (m & 3))));
}

// C^T operand: channel block b, rows 16 k + 4g + {0..3, 8..11} (rows eight
// further on have the other lowest bit in their swizzle).
__device__ __forceinline__ bf16x8 v_op(const Addr& a, uint32_t tile, int b, int k) {
    const uint32_t at = 256 * (b >> 2) + k * 16 * kLatBytes;
    const u32x2 x = lds_read_tr8(tile + (a.v ^ (64 * (b & 3))) + at);
    const u32x2 y = lds_read_tr8(tile + (a.v ^ (64 * (b & 3) + 16)) + 8 * kLatBytes + at);
    return __builtin_bit_cast(bf16x8, u32x4{x[0], x[1], y[0], y[1]});
}

__device__ __forceinline__ int clamp_len(const MlaDecodeArgs& A, int b) {
    const int64_t most = int64_t(A.table_width) << A.page_shift;
    const int n = A.kv_lens[b];
    return A.num_pages > 0 && n > 0 ? int(n < most ? n : most) : 0;
}

// What a workgroup walks: cached rows [0, len) behind `table`.
struct Source {
    const int32_t* table;
    int len;
};

// (table through the constant address space: a scalar load where k is uniform,
// which no wait for transfers in flight stands in the way of)
__device__ __forceinline__ const uint16_t* cached_row(const MlaDecodeArgs& A, const int32_t* table,
                                                      int k) {
    const int page = min(max(((const_i32*)table)[k >> A.page_shift], 0), A.num_pages - 1);
    return A.cache + int64_t(page) * A.page_stride +
           int64_t(k & ((1 << A.page_shift) - 1)) * kMlaRow;
}

// Eight rows [k, k + 8) of a tile (its rows 8 group ..): a transfer of 1 KiB
// per latent part, one for the eight rows' shared channels.  A page holds
// whole groups of eight.
__device__ __forceinline__ void issue8(const MlaDecodeArgs& A, const Source& src, int k, int group,
                                       int lane_id, uint32_t lds) {
    const int l = here(lane_id);
    const char* base = reinterpret_cast<const char*>(
        k < src.len ? cached_row(A, src.table, k) : A.cache);
    const uint32_t lat = lds + group * 8 * kLatBytes;
    const uint32_t pe = lds + kTile * kLatBytes + group * 8 * kPeBytes;
    const int pr = l >> 3, pj = (l & 7) ^ ((4 * group + (pr >> 1)) & 7);
    const uint32_t pe_off = pr * kRowBytes + kLatBytes + 16 * pj;
    const uint32_t lane = 16 * (l ^ (group & 1));
    if (k + 8 <= src.len) {
#pragma unroll
        for (int r = 0; r < 8; ++r) dma16_at(base + r * kRowBytes, lane ^ (32 * r), lat + r * kLatBytes);
        dma16_at(base, pe_off, pe);
    } else {   // rows behind the last one are zeros
#pragma unroll
        for (int r = 0; r < 8; ++r)
            dma16_at(k + r < src.len ? base + r * kRowBytes : reinterpret_cast<const char*>(kZeros),
                     lane ^ (32 * r), lat + r * kLatBytes);
        dma16_from(k + pr < src.len ? base + pe_off : reinterpret_cast<const char*>(kZeros), pe);
    }
}

// Infinities and NaN in the latent parts of `n` groups of eight rows to zero.
__device__ __forceinline__ void clean_rows(uint32_t tile, int group, int n, int l) {
    typedef __attribute__((address_space(3))) u32x4 lds_quad;
    for (int r = 0; r < 8 * n; ++r) {
        lds_quad* p = (lds_quad*)(lds_char*)uintptr_t(tile + (8 * group + r) * kLatBytes + 16 * l);
        *p = __builtin_bit_cast(u32x4, finite_only(__builtin_bit_cast(bf16x8, *p)));
    }
}

// Where a piece's sums go: the outputs, or a slot of partial sums.
struct Sink {
    bool final;
    int64_t row0;      // first query row of the unit's block (outputs)
    int first_row;     // the same, from the sequence's first query row
    int rows;          // query rows of the unit
    float* part;       // [kGroups][unit rows][4]
    float* ml;         // [unit rows][2]
    int stride;        // unit rows (32 kRG)
};

__device__ __forceinline__ void put4(const MlaDecodeArgs& A, const Sink& S, int row, int ch, f32x4 x,
                                     float inv) {
    if (S.final) {
        if (row >= S.rows) return;
        const f32x2 a = {x[0] * inv, x[1] * inv}, b = {x[2] * inv, x[3] * inv};
        *reinterpret_cast<u32x2*>(A.o + (S.row0 + row) * kMlaLatent + ch) =
            u32x2{__builtin_bit_cast(uint32_t, __builtin_convertvector(a, bf16x2)),
                  __builtin_bit_cast(uint32_t, __builtin_convertvector(b, bf16x2))};
    } else {
        *reinterpret_cast<f32x4*>(S.part + (size_t(ch >> 2) * S.stride + row) * 4) = x;
    }
}

__device__ __forceinline__ void put_ml(const MlaDecodeArgs& A, const Sink& S, int row, float mu,
                                       float l) {
    if (S.final) {
        if (A.lse && row < S.rows) A.lse[S.row0 + row] = l == 0.f ? -INFINITY : fmaf(mu, kLn2, logf(l));
    } else {
        S.ml[2 * row] = mu;
        S.ml[2 * row + 1] = l;
    }
}

__device__ __forceinline__ float inverse(float l) { return l == 0.f ? 0.f : 1.f / l; }

// x * a with x kept in an accumulation register on every path: written plainly
// the compiler holds the sums in ordinary registers between the tiles and
// moves all of them twice per tile.  (x's last product is a tile ago, so no
// wait for the matrix core stands here.)
__device__ __forceinline__ float scale_acc(float x, float a) {
    float t;
    asm("v_accvgpr_read_b32 %1, %0\n\tv_mul_f32 %1, %2, %1\n\tv_accvgpr_write_b32 %0, %1"
        : "+a"(x), "=&v"(t)
        : "v"(a));
    return x;
}

// A sum out of its accumulation register (see scale_acc); settle() first.
__device__ __forceinline__ float read_acc(float x) {
    float y;
    asm volatile("v_accvgpr_read_b32 %0, %1" : "=v"(y) : "a"(x));
    return y;
}

__device__ __forceinline__ f32x4 read_acc4(const f32x16& x, int r) {
    return f32x4{read_acc(x[r]), read_acc(x[r + 1]), read_acc(x[r + 2]), read_acc(x[r + 3])};
}

// Longer than the last matrix products take to write their registers.
__device__ __forceinline__ void settle() {
    asm volatile("s_nop 15\n\ts_nop 15\n\ts_nop 15\n\ts_nop 15\n\ts_nop 15\n\ts_nop 15");
}

// A piece's sums to where they go; with two pairs, joined first.
template <int kRG>
__device__ __forceinline__ void finish(const MlaDecodeArgs& A, Lds& lds, const Sink& sink,
                                       const f32x16 (&acc)[8], float mu, float lsum) {
    constexpr int kKW = 2 / kRG;
    const int w = wave_id(), l = here(threadIdx.x & 63), g = l >> 5;
    const int half = w & 1, rg = kRG == 2 ? w >> 1 : 0, kw = kRG == 2 ? 0 : w >> 1;
    const int row = 32 * rg + (l & 31);
    settle();
    if constexpr (kKW == 1) {
        const float inv = inverse(lsum);
        if (g == 0 && half == 0) put_ml(A, sink, row, mu, lsum);
#pragma unroll
        for (int b = 0; b < 8; ++b)
#pragma unroll
            for (int r = 0; r < 16; r += 4)
                put4(A, sink, row, 256 * half + 32 * b + d_row(r, g),
                     read_acc4(acc[b], r), inv);
    } else {
        // the two pairs' sums meet in LDS; each wave joins half of its channels
        raw_barrier();   // the tiles are read
        if (g == 0) {
            lds.ml[w][0][l] = mu;
            lds.ml[w][1][l] = lsum;
        }
        f32x4* mine = reinterpret_cast<f32x4*>(&lds.tile[w]);
#pragma unroll
        for (int b = 0; b < 8; ++b)
#pragma unroll
            for (int r = 0; r < 16; r += 4)
                mine[(b * 4 + r / 4) * 64 + l] = read_acc4(acc[b], r);
        raw_barrier();
        float f[2], total = 0.f, top = -INFINITY;
#pragma unroll
        for (int k = 0; k < 2; ++k) top = fmaxf(top, lds.ml[2 * k + half][0][l & 31]);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float x = lds.ml[2 * k + half][0][l & 31];
            f[k] = x == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(x - top);
            total = fmaf(lds.ml[2 * k + half][1][l & 31], f[k], total);
        }
        if (w == 0 && g == 0) put_ml(A, sink, row, top, total);
        const float inv = inverse(total);
#pragma unroll
        for (int b = 0; b < 4; ++b)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int blk = 4 * kw + b;
                const f32x4 x = reinterpret_cast<const f32x4*>(&lds.tile[half])[(blk * 4 + r) * 64 + l];
                const f32x4 y = reinterpret_cast<const f32x4*>(&lds.tile[2 + half])[(blk * 4 + r) * 64 + l];
                put4(A, sink, row, 256 * half + 32 * blk + d_row(4 * r, g), x * f[0] + y * f[1], inv);
            }
    }
    raw_barrier();   // the next piece refills the tiles
}

// One piece: tiles [t0, t1) of a source for 32 kRG query rows.
template <int kRG, bool kCausal>
__device__ __forceinline__ void piece(const MlaDecodeArgs& A, Lds& lds, const Addr& addr0,
                                      const Source& src, int t0, int t1, const Sink& sink) {
    constexpr int kKW = 2 / kRG;        // pairs that take tiles in turn
    constexpr int kBuf = 2 * kRG;       // tile buffers of such a pair (or of both)
    constexpr int kIssue = 2 / kRG;     // groups of eight rows that a wave fetches
    const int w = wave_id(), l = threadIdx.x & 63, g = l >> 5;
    const int half = w & 1, rg = kRG == 2 ? w >> 1 : 0, kw = kRG == 2 ? 0 : w >> 1;
    const int row = 32 * rg + (l & 31);
    const int rrow = min(row, sink.rows - 1);
    const uint16_t* qrow = A.q + (sink.row0 + rrow) * kMlaRow;
    bf16x8 qf[36];
#pragma unroll
    for (int m = 0; m < 36; ++m)
        qf[m] = __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4*>(qrow + 16 * m + 8 * g));
    const int limit = kCausal ? src.len - (A.tokens - 1 - (sink.first_row + rrow) / A.heads) : src.len;
    const int all_see = kCausal ? src.len - (A.tokens - 1) : src.len;
    const float c = A.scale * kLog2e;
    float m = -INFINITY, mu = 0.f, lsum = 0.f;
    f32x16 acc[8] = {};

    const uint32_t group_lds = lds_addr(&lds.tile[kw * kBuf]);
    const int share = kRG == 2 ? w : half;   // this wave's part of a tile
    auto issue = [&](int t, int buf) {
#pragma unroll
        for (int i = 0; i < kIssue; ++i) {
            const int group = share * kIssue + i;
            issue8(A, src, t * kTile + 8 * group, group, l, group_lds + buf * kTileBytes);
        }
    };
    const int steps = (t1 - t0 + kKW - 1) / kKW;
#pragma unroll
    for (int d = 0; d < kBuf - 1; ++d) {
        const int t = t0 + d * kKW + kw;
        if (t < t1) issue(t, d);
    }
    // the queries have arrived before the loop: no wait of the compiler's own
    // stands in it
#pragma unroll
    for (int i = 0; i < 36; ++i) asm volatile("" : "+v"(qf[i]));
    const int own = (t1 - t0 - kw + kKW - 1) / kKW;   // the other pair may have one more
    for (int i = 0; i < own; ++i) {
        const int t = t0 + i * kKW + kw, buf = i % kBuf;
        // this wave's part of tile i has landed once only later tiles' parts
        // are on their way
        if (kBuf == 4 && t + 2 * kKW < t1) wait_vm<2 * 9 * kIssue>();
        else if (kBuf == 4 && t + kKW < t1) wait_vm<9 * kIssue>();
        else wait_vm<0>();
        raw_barrier();   // everyone's part has, and tile i - 1 is read
        const int next = t + (kBuf - 1) * kKW;
        if (next < t1) issue(next, (i + kBuf - 1) % kBuf);
        // several new tokens: 0 * inf from a row that only later ones see would
        // reach the earlier ones, so the last tiles' latent values are made
        // finite before they serve as values (the combine kernel sets the
        // outputs of the queries that do see such a row)
        const bool cleaned = kCausal && A.tokens > 1 && (t0 + (i + 1) * kKW) * kTile > all_see;
        const uint32_t base = group_lds + buf * kTileBytes;
        const int k0 = t * kTile;
        const Addr addr{here(addr0.k), here(addr0.pe), here(addr0.v)};
        // operands are read a batch ahead of their products: with one wave per
        // SIMD nothing else covers the latency of LDS
        constexpr int kB = 6;
        f32x16 s = {};
        bf16x8 ko[2][kB];
#pragma unroll
        for (int e = 0; e < kB; ++e) ko[0][e] = k_op(addr, base, e);
#pragma unroll
        for (int n = 0; n < 36 / kB; ++n) {
            if (n + 1 < 36 / kB) {
#pragma unroll
                for (int e = 0; e < kB; ++e) ko[(n + 1) & 1][e] = k_op(addr, base, kB * (n + 1) + e);
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int e = 0; e < kB; ++e) s = mfma32(ko[n & 1][e], qf[kB * n + e], s);
            __builtin_amdgcn_sched_barrier(0);
        }
        const bool masked = k0 + kTile > all_see;
        if (masked) {
#pragma unroll
            for (int r = 0; r < 16; ++r)
                if (d_row(r, 0) >= limit - k0 - 4 * g) s[r] = -INFINITY;
        }
        float top = s[0];
#pragma unroll
        for (int r = 1; r < 16; ++r) top = fmaxf(top, s[r]);
        top = fmaxf(top, other_half(top));
        // the reference moves only when a row outgrows it by 2^8
        if (__any((top - m) * c > 8.f || (m == -INFINITY && top > m))) {
            const float mn = fmaxf(m, top);
            const float mun = mn == -INFINITY ? 0.f : mn * c;
            const float a = m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(mu - mun);
            m = mn;
            mu = mun;
            lsum *= a;
#pragma unroll
            for (int b = 0; b < 8; ++b) {
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[b][r] = scale_acc(acc[b][r], a);
            }
        }
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            s[r] = __builtin_amdgcn_exp2f(fmaf(s[r], c, -mu));
            lsum += s[r];
        }
        const bf16x8 p[2] = {pack8<0>(s), pack8<8>(s)};
        if (cleaned) {
            raw_barrier();
            clean_rows(group_lds + buf * kTileBytes, share * kIssue, kIssue, l);
            raw_barrier();
        }
        constexpr int kV = 4;   // value operands per batch
        bf16x8 vo[2][kV];
#pragma unroll
        for (int e = 0; e < kV; ++e) vo[0][e] = v_op(addr, base + 512 * half, e >> 1, e & 1);
#pragma unroll
        for (int n = 0; n < 16 / kV; ++n) {
            if (n + 1 < 16 / kV) {
#pragma unroll
                for (int e = 0; e < kV; ++e) {
                    const int x = kV * (n + 1) + e;
                    vo[(n + 1) & 1][e] = v_op(addr, base + 512 * half, x >> 1, x & 1);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int e = 0; e < kV; ++e) {
                const int x = kV * n + e;
                acc[x >> 1] = mfma32(vo[n & 1][e], p[x & 1], acc[x >> 1]);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    if (kKW > 1 && own < steps) {
        raw_barrier();
        if (kCausal && A.tokens > 1 && (t0 + steps * kKW) * kTile > all_see) {
            raw_barrier();
            raw_barrier();
        }
    }
    lsum += other_half(lsum);
    mu = m == -INFINITY ? -INFINITY : mu;

    finish<kRG>(A, lds, sink, acc, mu, lsum);
}

// A value that every lane holds alike, in scalar registers.
__device__ __forceinline__ int64_t uniform_i64(int64_t x) {
    const uint32_t lo = __builtin_amdgcn_readfirstlane(int(uint32_t(x)));
    const uint32_t hi = __builtin_amdgcn_readfirstlane(int(uint32_t(uint64_t(x) >> 32)));
    return int64_t(uint64_t(hi) << 32 | lo);
}

// Tiles of a sequence.
__device__ __forceinline__ int tiles_of(int len) { return (len + kTile - 1) / kTile; }

template <int kRG>
__global__ __launch_bounds__(kThreads, 1) void mla_decode_kernel(const MlaDecodeArgs A) {
    __shared__ __attribute__((aligned(256))) Lds lds;
    const int l = threadIdx.x & 63, w = wave_id();
    const int G = gridDim.x, wg = blockIdx.x;

    // the number of tiles, and where this workgroup's share begins
    auto block_sum = [&](int x, int& before) {   // inclusive scan over the workgroup
        int s = x;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int y = __shfl_up(s, d);
            if (l >= d) s += y;
        }
        __syncthreads();
        if (l == 63) lds.scan[w] = s;
        __syncthreads();
        before = s - x;
        int total = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (k < w) before += lds.scan[k];
            total += lds.scan[k];
        }
        return total;
    };
    int64_t total = 0;
    for (int b0 = 0; b0 < A.batch; b0 += kThreads) {
        const int b = b0 + int(threadIdx.x);
        int before;
        total += block_sum(b < A.batch ? tiles_of(clamp_len(A, b)) : 0, before);
    }
    total = uniform_i64(total) * A.row_blocks;
    const int64_t share = (total + G - 1) / G;
    const int64_t per = share > A.min_tiles ? share : A.min_tiles;
    const int64_t begin = per * wg, end = begin + per < total ? begin + per : total;
    if (begin >= end) return;
    if (threadIdx.x == 0) lds.unit = -1;
    int64_t seen = 0;
    for (int b0 = 0; b0 < A.batch; b0 += kThreads) {
        const int b = b0 + int(threadIdx.x);
        const int n = b < A.batch ? tiles_of(clamp_len(A, b)) : 0;
        int before;
        const int sum = block_sum(n, before);
        const int64_t at = begin - (seen + before) * A.row_blocks;
        if (n > 0 && at >= 0 && at < int64_t(n) * A.row_blocks) {
            lds.unit = b * A.row_blocks + int(at / n);
            lds.first = int(at % n);
        }
        seen += sum;
        if (seen * A.row_blocks > begin) break;
    }
    __syncthreads();
    int unit = __builtin_amdgcn_readfirstlane(lds.unit);
    int first = __builtin_amdgcn_readfirstlane(lds.first);

    const Addr addr(l);
    const int unit_rows = A.tokens * A.heads, units = A.batch * A.row_blocks;
    int64_t at = begin;
    while (at < end) {
        const int b = unit / A.row_blocks, blk = unit - b * A.row_blocks;
        const int len = __builtin_amdgcn_readfirstlane(clamp_len(A, b));
        const int n = tiles_of(len);
        if (n == 0) {   // the combine kernel writes these rows
            ++unit;
            continue;
        }
        const int last = int(end - at < n - first ? first + (end - at) : n);
        const bool whole = first == 0 && last == n;
        const int slot = first == 0 ? unit : units + wg;
        Sink sink;
        sink.final = whole && !A.prefix_len;
        sink.first_row = 32 * kRG * blk;
        sink.row0 = int64_t(b) * unit_rows + sink.first_row;
        sink.rows = min(32 * kRG, unit_rows - sink.first_row);
        sink.part = A.part + size_t(slot) * kGroups * 4 * 32 * kRG;
        sink.ml = A.part_ml + size_t(slot) * 2 * 32 * kRG;
        sink.stride = 32 * kRG;
        if (first == 0 && threadIdx.x == 0) {
            // the workgroups that hold this unit's later pieces
            const int64_t stop = at + n;
            A.meta[2 * unit] = sink.final ? -1 : wg;
            A.meta[2 * unit + 1] = int((stop - 1) / per);
        }
        piece<kRG, true>(A, lds, addr, Source{A.table + int64_t(b) * A.table_width, len}, first,
                         last, sink);
        at += last - first;
        first = 0;
        ++unit;
    }
}

// The prefix: every block of 32 kRG query rows walks all prefix rows.
template <int kRG>
__global__ __launch_bounds__(kThreads, 1) void mla_prefix_kernel(const MlaDecodeArgs A) {
    __shared__ __attribute__((aligned(256))) Lds lds;
    const int l = threadIdx.x & 63, wg = blockIdx.x;
    const Addr addr(l);
    const int64_t rows = int64_t(A.batch) * A.tokens * A.heads;
    const int n = tiles_of(A.prefix_len);
    const int64_t total = int64_t(A.prefix_units) * n;
    int64_t at = A.prefix_per * wg;
    const int64_t end = min(at + A.prefix_per, total);
    while (at < end) {
        const int unit = int(at / n), first = int(at - int64_t(unit) * n);
        const int last = int(end - at < n - first ? first + (end - at) : n);
        const int slot = first == 0 ? unit : A.prefix_units + wg;
        Sink sink;
        sink.final = false;
        sink.first_row = 0;
        sink.row0 = int64_t(unit) * 32 * kRG;
        sink.rows = int(min(int64_t(32 * kRG), rows - sink.row0));
        sink.part = A.pre_part + size_t(slot) * kGroups * 4 * 32 * kRG;
        sink.ml = A.pre_ml + size_t(slot) * 2 * 32 * kRG;
        sink.stride = 32 * kRG;
        piece<kRG, false>(A, lds, addr, Source{A.prefix_table, A.prefix_len}, first, last, sink);
        at += last - first;
    }
}

// Joins the partial sums of 32 query rows of a unit, 64 channels a workgroup.
// Where there are several new tokens it also looks at the rows of the tiles
// that some of them do not see: a latent value that is infinite or NaN makes
// that channel NaN for the queries that see it (its score is infinite or NaN
// too), and the products left it out.
__global__ __launch_bounds__(kThreads) void mla_combine_kernel(const MlaDecodeArgs A) {
    __shared__ int bad_s;
    const int unit = blockIdx.x / A.row_groups, sub = blockIdx.x % A.row_groups;
    const int b = unit / A.row_blocks, blk = unit - b * A.row_blocks;
    const int unit_rows = A.tokens * A.heads, units = A.batch * A.row_blocks;
    const int stride = 32 * A.row_groups;
    const int lr = 32 * sub + int(threadIdx.x & 31);     // row in the unit's block
    const int urow = stride * blk + lr;                  // row in the sequence
    const int len = clamp_len(A, b);
    const bool any = len > 0;
    const int g0 = any ? A.meta[2 * unit] : -1, g1 = any ? A.meta[2 * unit + 1] : -2;
    const int32_t* table = A.table + int64_t(b) * A.table_width;
    const int from = max(len - (A.tokens - 1), 0) / kTile * kTile;
    const int cg0 = blockIdx.y * 16 + 2 * int(threadIdx.x >> 5);
    bool bad = false;
    if (A.tokens > 1) {
        for (int k = from + int(threadIdx.x >> 3); k < len; k += kThreads / 8) {
            const u32x4 x = *reinterpret_cast<const u32x4*>(
                cached_row(A, table, k) + 64 * blockIdx.y + 8 * (threadIdx.x & 7));
            bad |= (nonfinite_bits(x[0]) | nonfinite_bits(x[1]) | nonfinite_bits(x[2]) |
                    nonfinite_bits(x[3])) != 0;
        }
        if (threadIdx.x == 0) bad_s = 0;
        __syncthreads();
        if (bad) bad_s = 1;
        __syncthreads();
        bad = bad_s != 0;
    }
    const bool done = any && g0 < 0;                     // already written
    if (urow >= unit_rows || (done && !bad)) return;
    u32x4 nan = {};                                      // 0xffff where a channel is NaN
    if (bad) {
        const int limit = len - (A.tokens - 1 - urow / A.heads);
        for (int k = from; k < limit; ++k) {
            const u32x4 x = *reinterpret_cast<const u32x4*>(cached_row(A, table, k) + 4 * cg0);
#pragma unroll
            for (int i = 0; i < 4; ++i) nan[i] |= (nonfinite_bits(x[i]) >> 15) * 0xffffu;
        }
    }
    const int64_t row = int64_t(b) * unit_rows + urow;
    u32x4* const o = reinterpret_cast<u32x4*>(A.o + row * kMlaLatent + 4 * cg0);
    if (done) {
        *o |= nan;
        return;
    }
    const int np = any ? g1 - g0 + 1 : 0;                // private pieces
    // prefix pieces of this row
    int pn = 0, pu = 0, pr = 0;
    int64_t pg0 = 0;
    if (A.prefix_len) {
        const int n = tiles_of(A.prefix_len), prows = 32 * A.prefix_groups;
        pu = int(row / prows);
        pr = int(row - int64_t(pu) * prows);
        pg0 = int64_t(pu) * n / A.prefix_per;
        pn = int((int64_t(pu + 1) * n - 1) / A.prefix_per - pg0) + 1;
    }
    const int pstride = 32 * A.prefix_groups;
    auto slot_of = [&](int i, const float*& part, const float*& ml, int& st, int& r) {
        if (i < np) {
            const size_t s = i == 0 ? size_t(unit) : size_t(units) + g0 + i;
            part = A.part + s * kGroups * 4 * stride;
            ml = A.part_ml + s * 2 * stride;
            st = stride;
            r = lr;
        } else {
            const size_t s = i == np ? size_t(pu) : size_t(A.prefix_units) + pg0 + (i - np);
            part = A.pre_part + s * kGroups * 4 * pstride;
            ml = A.pre_ml + s * 2 * pstride;
            st = pstride;
            r = pr;
        }
    };
    // eight pieces' sums at a time, all loads before their use
    constexpr int kN = 8;
    const int n = np + pn;
    float top = -INFINITY, total = 0.f;
    f32x4 sum[2] = {zero4(), zero4()};
    for (int i0 = 0; i0 < n; i0 += kN) {
        f32x2 ml[kN];
        f32x4 x[kN][2];
#pragma unroll
        for (int e = 0; e < kN; ++e) {
            const float *part, *pml;
            int st, r;
            slot_of(min(i0 + e, n - 1), part, pml, st, r);
            ml[e] = *reinterpret_cast<const f32x2*>(pml + 2 * r);
#pragma unroll
            for (int k = 0; k < 2; ++k)
                x[e][k] = *reinterpret_cast<const f32x4*>(part + (size_t(cg0 + k) * st + r) * 4);
        }
        float most = top;
#pragma unroll
        for (int e = 0; e < kN; ++e) most = fmaxf(most, ml[e][0]);
        const float f = top == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(top - most);
        top = most;
        total *= f;
        sum[0] *= f;
        sum[1] *= f;
#pragma unroll
        for (int e = 0; e < kN; ++e) {
            const float w = i0 + e >= n || ml[e][0] == -INFINITY
                ? 0.f : __builtin_amdgcn_exp2f(ml[e][0] - most);
            if (w != 0.f) {   // (a piece without keys has no sums to speak of)
                total = fmaf(ml[e][1], w, total);
                sum[0] += x[e][0] * w;
                sum[1] += x[e][1] * w;
            }
        }
    }
    const float inv = inverse(total);
    u32x4 out;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const f32x2 v = {sum[k >> 1][2 * (k & 1)] * inv, sum[k >> 1][2 * (k & 1) + 1] * inv};
        out[k] = __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
    }
    *o = out | nan;
    if (A.lse && blockIdx.y == 0 && threadIdx.x < 32)
        A.lse[row] = total == 0.f ? -INFINITY : fmaf(top, kLn2, logf(total));
}

template <int kRG>
void launch_private(const MlaDecodeArgs& A, hipStream_t stream) {
    mla_decode_kernel<kRG><<<dim3(kMlaWorkgroups), dim3(kThreads), 0, stream>>>(A);
}

template <int kRG>
void launch_prefix(const MlaDecodeArgs& A, hipStream_t stream) {
    const int64_t total = int64_t(A.prefix_units) * ((A.prefix_len + kTile - 1) / kTile);
    mla_prefix_kernel<kRG><<<dim3(unsigned((total + A.prefix_per - 1) / A.prefix_per)),
                             dim3(kThreads), 0, stream>>>(A);
}

}  // namespace

hipError_t launch_mla_decode(const MlaDecodeArgs& A, hipStream_t stream) {
    if (A.prefix_len) {
        if (A.prefix_groups == 2) launch_prefix<2>(A, stream);
        else launch_prefix<1>(A, stream);
        if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    }
    if (A.row_groups == 2) launch_private<2>(A, stream);
    else launch_private<1>(A, stream);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    mla_combine_kernel<<<dim3(unsigned(A.batch * A.row_blocks * A.row_groups), 8), dim3(kThreads), 0,
                         stream>>>(A);
    return hipGetLastError();
}

}  // namespace rda
