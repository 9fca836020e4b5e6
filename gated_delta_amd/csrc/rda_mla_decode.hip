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
// stays in registers.  A wave holds 32 query rows whole: 576 x 32 bf16 of Q
// (144 registers) and 512 x 32 fp32 of O^T (all 256 accumulation registers).
// What bounds the products is LDS: an operand of 1 KiB feeds one product of
// 32 cycles, and the CU's 128 bytes a cycle are just that for its 4 SIMDs; a
// wave with a part of the channels would read the row operands again.
// The 4 waves of a workgroup are kRW row waves x 4 / kRW key waves: row waves
// share a tile of 32 cached rows, key waves take tiles in turn and merge their
// sums at the end.
//
// The work is a list of tiles, unit after unit (a unit: the query rows of one
// sequence, or a block of all query rows for the prefix), cut into equal
// pieces, one per workgroup, whatever the sequences' lengths: they are read
// on the device.  A workgroup that covers a whole unit writes its output; the
// others write partial sums that the combine kernel joins.
//
// Measured (32 heads, 512 to 8192 rows a sequence): 256 sequences 247 us, 1.25
// GB of rows at 5.1 TB/s, where a plain read of as much in this order reaches
// 6.1; 32 sequences of 3 tokens 65 us (2.3 TB/s: 17 tiles a workgroup, about
// 2 us each with 96 of 128 query rows in use, and 20 us to load queries and to
// write and join sums); 12288 query rows (128 sequences of 3 tokens) behind 16384
// shared rows: the prefix 455 us, 963 TFLOP/s.  One sequence of 777 rows takes 19 us, 16
// of them in this kernel for one tile a wave: the plan's sums over the lengths,
// the first transfers and the exchange of query operands, one after the other.
#include <type_traits>

#include "rda_internal.h"
#include "rda_mla.h"
#include "rda_mla_acc.h"

namespace rda {
namespace {

constexpr int kThreads = 256;
constexpr int kTile = 32;                          // cached rows per tile
constexpr int kRowBytes = kMlaRow * 2;             // 1152
constexpr int kLatBytes = kMlaLatent * 2, kPeBytes = kMlaPe * 2;
constexpr int kTileBytes = kTile * kRowBytes;      // 36864

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

constexpr int kPieceTiles = 6;   // one more piece takes at least as long as these
constexpr int kShare = 12;       // query operands exchanged at a time

struct Lds {
    Tile tile[4];
    u32x4 q[kShare][64];
    float ml[4][2][32];     // (mu, l) of each wave's rows
    int scan[8];
    int unit, first;        // where this workgroup's piece begins
    int bad;                // the piece's last tiles held infinities or NaN
};

// LDS byte offsets of this lane's operands, from a tile's start.
struct Lane {
    int k, pe, v;
    __device__ __forceinline__ explicit Lane(int l) {
        const int r = l & 31, g = l >> 5, j = l & 15;
        k = r * kLatBytes + 16 * (g ^ swz(r));
        pe = kTile * kLatBytes + r * kPeBytes + 16 * (g ^ ((r >> 1) & 7));
        // C^T operand: channel l % 32, rows 4g + {0..3}
        const int vr = 4 * g + (j >> 2), low = 2 * ((l >> 4) & 1) + ((j >> 1) & 1);
        v = vr * kLatBytes + 16 * (low ^ swz(vr)) + 8 * (j & 1);
    }
};

// Addresses in one tile: the granule bits that a swizzle turns over are an
// exclusive-or per lane, all else is a constant in the read instruction (the
// sums are made opaque, or the compiler adds those constants per read).
struct RowAddr {
    uint32_t k[8], pe[4];
    __device__ __forceinline__ RowAddr(const Lane& a, uint32_t tile) {
#pragma unroll
        for (int m = 0; m < 8; ++m) k[m] = here(int(tile) + (a.k ^ (32 * m)));
#pragma unroll
        for (int m = 0; m < 4; ++m) pe[m] = here(int(tile) + (a.pe ^ (32 * m)));
    }
    // values 16 m + 8 g .. of row l % 32
    __device__ __forceinline__ bf16x8 op(int m) const {
        return lds_read16(m < 32 ? k[m & 7] + 256 * (m >> 3) : pe[m & 3]);
    }
};

struct ValAddr {
    uint32_t v[4], w[4];
    __device__ __forceinline__ ValAddr(const Lane& a, uint32_t tile) {
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            v[b] = here(int(tile) + (a.v ^ (64 * b)));
            w[b] = here(int(tile) + (a.v ^ (64 * b + 16)));   // rows eight further on
        }
    }
    // channel block b of C^T, rows 16 k + 4g + {0..3, 8..11}
    __device__ __forceinline__ bf16x8 op(int b, int k) const {
        const uint32_t at = 256 * (b >> 2) + k * 16 * kLatBytes;
        const u32x2 x = lds_read_tr8(v[b & 3] + at);
        const u32x2 y = lds_read_tr8(w[b & 3] + at + 8 * kLatBytes);
        return __builtin_bit_cast(bf16x8, u32x4{x[0], x[1], y[0], y[1]});
    }
};

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

// The transfers of eight rows [k, k + 8) of a tile (its rows 8 group ..): one of
// 1 KiB per latent part, one for the eight rows' shared channels.  A page holds
// whole groups of eight.  Rows from `end` on are read as zeros.
struct Fetch {
    const char* base;     // row k
    int valid;            // rows before `end`
    uint32_t lds;         // the tile
    int group;

    __device__ __forceinline__ Fetch(const MlaDecodeArgs& A, int page, int k, int end, int group_,
                                     uint32_t tile) {
        group = group_;
        valid = end - k;
        lds = tile;
        base = reinterpret_cast<const char*>(
            A.cache + int64_t(page) * A.page_stride +
            int64_t(k & ((1 << A.page_shift) - 1)) * kMlaRow);
    }
    // transfer i of 0..8.  kOnce: the latent parts pass the caches by, where one
    // workgroup reads a row and no other (256 sequences of 4352 rows: 6.1
    // instead of 5.3 TB/s; a row's last 128 bytes share a line with the next).
    template <bool kOnce>
    __device__ __forceinline__ void issue(int i, int lane_id) const {
        const char* const zeros = reinterpret_cast<const char*>(kZeros);
        const int l = here(lane_id);
        if (i < 8) {
            dma16_at<kOnce>(i < valid ? base + i * kRowBytes : zeros, (16 * (l ^ (group & 1))) ^ (32 * i),
                     lds + (group * 8 + i) * kLatBytes);
        } else {
            const int r = l >> 3, j = (l & 7) ^ ((4 * group + (r >> 1)) & 7);
            const uint64_t at = uint64_t(base) + uint32_t(r * kRowBytes + kLatBytes + 16 * j);
            const uint64_t z = uint64_t(zeros);
            const bool ok = r < valid;   // (halves apart: a select, not a branch)
            const uint64_t from = uint64_t(ok ? uint32_t(at >> 32) : uint32_t(z >> 32)) << 32 |
                                  (ok ? uint32_t(at) : uint32_t(z));
            dma16_from(reinterpret_cast<const void*>(from),
                       lds + kTile * kLatBytes + group * 8 * kPeBytes);
        }
    }
};

// The page of row k (any page where k lies behind the table's rows).
__device__ __forceinline__ int page_of(const MlaDecodeArgs& A, const Source& src, int k) {
    const int at = k < src.len ? k >> A.page_shift : 0;
    return src.len > 0 ? min(max(((const_i32*)src.table)[at], 0), A.num_pages - 1) : 0;
}

// Infinities and NaN in the latent parts of `n` groups of eight rows to zero;
// whether there were any.
__device__ __forceinline__ bool clean_rows(uint32_t tile, int group, int n, int l) {
    uint32_t bad = 0;
    for (int r = 0; r < 8 * n; ++r) {
        lds_u32x4* p = (lds_u32x4*)(lds_char*)uintptr_t(tile + (8 * group + r) * kLatBytes + 16 * l);
        u32x4 x = *p;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t b = nonfinite_bits(x[i]);
            bad |= b;
            x[i] &= ~((b >> 15) * 0xffffu);
        }
        *p = x;
    }
    return __any(bad != 0);
}

// Where a piece's sums go: the outputs, or a slot of partial sums.
struct Sink {
    bool final;
    int64_t row0;      // first query row of the unit's block (outputs)
    int first_row;     // the same, from the sequence's first query row
    int rows;          // query rows of the unit
    float* part;       // [unit rows][512]
    float* ml;         // [unit rows][2]
    int32_t* bad;      // set where the last tiles held infinities or NaN
};

// Four channels of a row, and a row's statistics.
__device__ __forceinline__ void put4(const MlaDecodeArgs& A, const Sink& S, int row, int ch, f32x4 x) {
    if (row >= S.rows) return;
    if (S.final) {
        *reinterpret_cast<u32x2*>(A.o + (S.row0 + row) * kMlaLatent + ch) =
            u32x2{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3])};
    } else {
        *reinterpret_cast<f32x4*>(S.part + size_t(row) * kMlaLatent + ch) = x;
    }
}

__device__ __forceinline__ void put_ml(const MlaDecodeArgs& A, const Sink& S, int row, float mu,
                                       float l) {
    if (S.final) {
        if (A.lse && row < S.rows) A.lse[S.row0 + row] = l == 0.f ? -INFINITY : fmaf(mu, kLn2, logf(l));
    } else {
        *reinterpret_cast<f32x2*>(S.ml + 2 * row) = f32x2{mu, l};
    }
}

__device__ __forceinline__ float inverse(float l) { return l == 0.f ? 0.f : 1.f / l; }

// A piece's sums to where they go, by way of LDS (the tiles' memory): 256
// channels at a time, 32 rows a wave, so that they leave row by row; the key
// waves' sums are joined there, each key wave taking an equal part of the rows.
template <int kRW>
__device__ __forceinline__ void finish(const MlaDecodeArgs& A, Lds& lds, const Sink& sink,
                                       float mu, float lsum) {
    constexpr int kKW = 4 / kRW, kRows = 32 / kKW;
    constexpr int kStride = 256 * 4 + 16;   // a row's sums in LDS; 16: other banks
    static_assert(32 * kStride <= kTileBytes, "a wave's rows fit its tile");
    const int w = wave_id(), l = here(threadIdx.x & 63);
    const int rw = w % kRW, kw = w / kRW;
    if (l < 32) {
        lds.ml[w][0][l] = mu;
        lds.ml[w][1][l] = lsum;
    }
    settle();
    raw_barrier();   // the tiles are read
    if (threadIdx.x == 0) {
        *sink.bad = lds.bad;
        lds.bad = 0;
    }
    // each lane: its row's part of every key wave's sums, and the quotient
    float f[kKW], total = 0.f, top = -INFINITY;
#pragma unroll
    for (int k = 0; k < kKW; ++k) top = fmaxf(top, lds.ml[k * kRW + rw][0][l & 31]);
#pragma unroll
    for (int k = 0; k < kKW; ++k) {
        const float x = lds.ml[k * kRW + rw][0][l & 31];
        f[k] = x == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(x - top);
        total = fmaf(lds.ml[k * kRW + rw][1][l & 31], f[k], total);
    }
    if (kw == 0 && l < 32) put_ml(A, sink, 32 * rw + l, top, total);
    const float inv = sink.final ? inverse(total) : 1.f;
#pragma unroll
    for (int k = 0; k < kKW; ++k) f[k] *= inv;
    const uint32_t mine = lds_addr(&lds.tile[w]) + (l & 31) * kStride + 16 * (l >> 5);
    unrolled<2>([&](auto ph) {
        constexpr int phase = decltype(ph)::value;
        if constexpr (phase > 0) raw_barrier();   // the channels before are read
        unrolled<32>([&](auto q) {
            constexpr int n = decltype(q)::value;   // block n / 4, channels 8 (n % 4) + 4g ..
            acc_store<32 * phase + n, 128 * (n / 4) + 32 * (n % 4)>(mine);
        });
        raw_barrier();
        constexpr int kR = 8;   // rows at a time, all reads before their use
#pragma unroll 1
        for (int r0 = kw * kRows; r0 < (kw + 1) * kRows; r0 += kR) {
            f32x4 x[kR][kKW];
#pragma unroll
            for (int i = 0; i < kR; ++i)
#pragma unroll
                for (int k = 0; k < kKW; ++k)
                    x[i][k] = *reinterpret_cast<const f32x4*>(
                        reinterpret_cast<const char*>(&lds.tile[k * kRW + rw]) + (r0 + i) * kStride + 16 * l);
#pragma unroll
            for (int i = 0; i < kR; ++i) {
                f32x4 sum = zero4();
#pragma unroll
                for (int k = 0; k < kKW; ++k) {
                    const float fk = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(f[k]), r0 + i));
                    sum += x[i][k] * fk;
                }
                put4(A, sink, 32 * rw + r0 + i, 256 * phase + 4 * l, sum);
            }
        }
    });
    raw_barrier();   // the next piece refills the tiles
}

// One piece: tiles [t0, t1) of a source for 32 kRW query rows.
template <int kRW, bool kCausal>
__device__ __forceinline__ void piece(const MlaDecodeArgs& A, Lds& lds, const Lane& lane,
                                      const Source& src, int t0, int t1, const Sink& sink) {
    constexpr int kKW = 4 / kRW;        // key waves
    constexpr int kBuf = kRW;           // tile buffers of a key wave's group
    constexpr int kIssue = 4 / kRW;     // groups of eight rows that a wave fetches
    constexpr int kDma = 9 * kIssue;    // transfers of a wave per tile
    const int w = wave_id(), l = threadIdx.x & 63, g = l >> 5;
    const int rw = w % kRW, kw = w / kRW;
    const int row = 32 * rw + (l & 31);
    const int rrow = min(row, sink.rows - 1);
    const uint16_t* qrow = A.q + (sink.row0 + rrow) * kMlaRow;
    const int limit = kCausal ? src.len - (A.tokens - 1 - (sink.first_row + rrow) / A.heads) : src.len;
    const int all_see = kCausal ? src.len - (A.tokens - 1) : src.len;
    const float c = A.scale * kLog2e;
    float m = -INFINITY, mu = 0.f, lsum = 0.f;
    const uint32_t group_lds = lds_addr(&lds.tile[kw * kBuf]);
    const int end = min(src.len, t1 * kTile);
    // this wave's part of tile t.  (A tile behind the last one is fetched too, as
    // zeros: the number of transfers in flight is the same in every step.)
    auto first_row = [&](int t, int n) { return t * kTile + 8 * (rw * kIssue + n); };
    int page[kIssue];   // of the next tile to fetch
    auto pages = [&](int t) {
#pragma unroll
        for (int n = 0; n < kIssue; ++n) page[n] = page_of(A, src, first_row(t, n));
    };
    auto issue = [&](int t, int buf) {
#pragma unroll
        for (int n = 0; n < kIssue; ++n) {
            const Fetch f(A, page[n], first_row(t, n), end, rw * kIssue + n, group_lds + buf * kTileBytes);
#pragma unroll
            for (int x = 0; x < 9; ++x) f.template issue<kCausal>(x, l);
        }
        pages(t + kKW);
    };
    constexpr int kLead = kBuf > 1 ? kBuf - 1 : 1;   // tiles fetched ahead of the loop
    pages(t0 + kw);
#pragma unroll 1
    for (int d = 0; d < kLead; ++d) issue(t0 + d * kKW + kw, d);
    // key waves have the same query rows: each loads its part of the operands
    // and they exchange them (the loads are what is slow: 32 rows apart)
    constexpr int kOwn = 36 / kKW;
    bf16x8 qf[36];
    if constexpr (kKW == 1) {
#pragma unroll
        for (int m = 0; m < 36; ++m)
            qf[m] = __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4*>(qrow + 16 * m + 8 * g));
        unrolled<256>([](auto q) { acc_clear<decltype(q)::value>(); });
    } else {
        u32x4 mine[kOwn];
#pragma unroll
        for (int m = 0; m < kOwn; ++m)
            mine[m] = *reinterpret_cast<const u32x4*>(qrow + 16 * (kw * kOwn + m) + 8 * g);
        unrolled<256>([](auto q) { acc_clear<decltype(q)::value>(); });
        constexpr int kEach = kShare / 4;   // operands of a wave at a time
#pragma unroll
        for (int r = 0; r < kOwn / kEach; ++r) {
            raw_barrier();
#pragma unroll
            for (int e = 0; e < kEach; ++e) lds.q[w * kEach + e][l] = mine[r * kEach + e];
            raw_barrier();
#pragma unroll
            for (int k = 0; k < kKW; ++k)
#pragma unroll
                for (int e = 0; e < kEach; ++e)
                    qf[k * kOwn + r * kEach + e] =
                        __builtin_bit_cast(bf16x8, lds.q[(k * kRW + rw) * kEach + e][l]);
        }
    }
    // the queries have arrived before the loop: no wait of the compiler's own
    // stands in it
#pragma unroll
    for (int i = 0; i < 36; ++i) asm volatile("" : "+v"(qf[i]));
    const int steps = (t1 - t0 + kKW - 1) / kKW;
    const int own = (t1 - t0 - kw + kKW - 1) / kKW;   // others may have one more
    const bool idle = 32 * rw >= sink.rows;           // a row wave without rows
    for (int i = 0; i < own; ++i) {
        const int t = t0 + i * kKW + kw, buf = i % kBuf;
        // this wave's part of tile i has landed once only later tiles' parts
        // are on their way
        if constexpr (kBuf > 1) {
            wait_vm<(kBuf - 2) * kDma>();
            raw_barrier();   // everyone's part has, and tile i - 1 is read
            issue(t + kLead * kKW, (i + kLead) % kBuf);
        } else {
            wait_vm<0>();
        }
        const uint32_t base = group_lds + buf * kTileBytes;
        const int k0 = t * kTile;
        // several new tokens: 0 * inf from a row that only later ones see would
        // reach the earlier ones, so the last tiles' latent values are made
        // finite before they serve as values (the combine kernel sets the
        // outputs of the queries that do see such a row)
        // (all waves meet for it: a step's condition, not a tile's)
        const bool cleaned = kCausal && A.tokens > 1 && (t0 + (i + 1) * kKW) * kTile > all_see;
        bf16x8 p[2];
        if (!idle) {
            const RowAddr rows(lane, base);
            constexpr int kB = 4;   // operands read ahead of their products
            f32x16 s;
            bf16x8 ko[2][kB];
#pragma unroll
            for (int e = 0; e < kB; ++e) ko[0][e] = rows.op(e);
#pragma unroll
            for (int n = 0; n < 36 / kB; ++n) {
                if (n + 1 < 36 / kB) {
#pragma unroll
                    for (int e = 0; e < kB; ++e) ko[(n + 1) & 1][e] = rows.op(kB * (n + 1) + e);
                }
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int e = 0; e < kB; ++e) {
                    if (n + e == 0) scores_first(s, ko[0][0], qf[0]);
                    else scores_next(s, ko[n & 1][e], qf[kB * n + e]);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
            scores_done(s);
            if (k0 + kTile > all_see) {
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
                const bool first = __all(m == -INFINITY);   // the sums are zeros
                m = mn;
                mu = mun;
                lsum *= a;
                if (!first) unrolled<256>([a](auto q) { acc_scale<decltype(q)::value>(a); });
            }
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                s[r] = __builtin_amdgcn_exp2f(fmaf(s[r], c, -mu));
                lsum += s[r];
            }
            p[0] = pack8<0>(s);
            p[1] = pack8<8>(s);
        }
        if (cleaned) {
            if constexpr (kRW > 1) raw_barrier();
            if (k0 + kTile > all_see && clean_rows(base, rw * kIssue, kIssue, l)) lds.bad = 1;
            if constexpr (kRW > 1) raw_barrier();
        }
        if (!idle) {
            constexpr int kV = 4;   // value operands read ahead
            const ValAddr vals(lane, base);
            bf16x8 vo[2][kV];
#pragma unroll
            for (int e = 0; e < kV; ++e) vo[0][e] = vals.op(e >> 1, e & 1);
            unrolled<32 / kV>([&](auto q) {
                constexpr int n = decltype(q)::value;
                if constexpr (n + 1 < 32 / kV) {
#pragma unroll
                    for (int e = 0; e < kV; ++e) {
                        const int x = kV * (n + 1) + e;
                        vo[(n + 1) & 1][e] = vals.op(x >> 1, x & 1);
                    }
                }
                __builtin_amdgcn_sched_barrier(0);
                unrolled<kV>([&](auto q2) {
                    constexpr int e = decltype(q2)::value, x = kV * n + e;
                    acc_product<(x >> 1)>(vo[n & 1][e], p[x & 1]);
                });
                __builtin_amdgcn_sched_barrier(0);
            });
        }
        if constexpr (kBuf == 1) {
            // the wave's own tile is read: fetch its next one
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            issue(t + kKW, 0);
        }
    }
    wait_vm<0>();   // the tiles behind the last: nothing may land later
    if constexpr (kRW == 2) {
        if (own < steps) {   // the other key wave's group meets here
            raw_barrier();
            if (kCausal && A.tokens > 1 && (t0 + steps * kKW) * kTile > all_see) {
                raw_barrier();
                raw_barrier();
            }
        }
    }
    lsum += other_half(lsum);
    mu = m == -INFINITY ? -INFINITY : mu;
    finish<kRW>(A, lds, sink, mu, lsum);
}

// Tiles of a sequence.
__device__ __forceinline__ int tiles_of(int len) { return (len + kTile - 1) / kTile; }

template <int kRW>
__global__ __launch_bounds__(kThreads, 1) void mla_decode_kernel(const MlaDecodeArgs A) {
    __shared__ __attribute__((aligned(256))) Lds lds;
    const int l = threadIdx.x & 63, w = wave_id(), wg = blockIdx.x;

    // the number of tiles, and where this workgroup's share begins
    auto block_sum = [&](int x, int& before) {   // x over the workgroup
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
        return __builtin_amdgcn_readfirstlane(total);
    };
    auto tiles_at = [&](int b) { return b < A.batch ? tiles_of(clamp_len(A, b)) : 0; };
    if (threadIdx.x == 0) lds.bad = 0;
    int n0 = tiles_at(threadIdx.x);
    int before0;
    int total0 = block_sum(n0, before0);
    int total = total0;
    for (int b0 = kThreads; b0 < A.batch; b0 += kThreads) {
        int before;
        total += block_sum(tiles_at(b0 + int(threadIdx.x)), before);
    }
    total *= A.row_blocks;
    if (total == 0) return;
    const int share = (total + kMlaWorkgroups - 1) / kMlaWorkgroups;
    // (short sequences are better spread than put one behind the other)
    const int units = A.batch * A.row_blocks;
    int per = max(share, min(A.min_tiles, (total + units - 1) / units));
    // A piece costs a workgroup as much as six tiles or more besides its own
    // (queries in, sums out), so with no more units than workgroups none takes
    // pieces of two units if that makes its share at most so much longer.  The
    // units' tiles are counted up to multiples of `per` then (half a share lost
    // per unit on average); a whole unit where it is hardly longer.
    bool apart = false;
    if (units <= kMlaWorkgroups && share < 1 << 20) {
        int most = n0;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) most = max(most, __shfl_xor(most, d));
        if (l == 0) lds.scan[4 + w] = most;
        __syncthreads();
        most = __builtin_amdgcn_readfirstlane(
            max(max(lds.scan[4], lds.scan[5]), max(lds.scan[6], lds.scan[7])));
        int each = max(A.min_tiles, total / (kMlaWorkgroups - units / 2) + 1);
        for (int tries = 0; tries < 2 && !apart && each <= max(share, A.min_tiles) + kPieceTiles; ++tries) {
            if (most <= each + 2) each = most;
            const int padded = (n0 + each - 1) / each * each;
            int before;
            const int sum = block_sum(padded, before);
            if (sum * A.row_blocks <= each * kMlaWorkgroups) {
                apart = true;
                per = each;
                n0 = padded;
                before0 = before;
                total0 = sum;
                total = sum * A.row_blocks;
            }
            each += each / 8 + 1;
        }
    }
    if (int64_t(per) * wg >= total) return;
    const int begin = per * wg, end = min(begin + per, total);
    for (int b0 = 0, seen = 0; b0 < A.batch && seen * A.row_blocks <= begin; b0 += kThreads) {
        const int b = b0 + int(threadIdx.x);
        int n = n0, before = before0, sum = total0;
        if (b0 > 0) {
            n = tiles_at(b);
            sum = block_sum(n, before);
        }
        const int at = begin - (seen + before) * A.row_blocks;
        if (n > 0 && at >= 0 && at < n * A.row_blocks) {
            lds.unit = b * A.row_blocks + at / n;
            lds.first = at % n;
        }
        seen += sum;
    }
    __syncthreads();
    int unit = __builtin_amdgcn_readfirstlane(lds.unit);
    int first = __builtin_amdgcn_readfirstlane(lds.first);

    const Lane lane(l);
    const int unit_rows = A.tokens * A.heads;
    int at = begin;
    while (at < end) {
        const int b = unit / A.row_blocks, blk = unit - b * A.row_blocks;
        const int len = __builtin_amdgcn_readfirstlane(clamp_len(A, b));
        const int n = tiles_of(len);
        if (n == 0) {   // the combine kernel writes these rows
            ++unit;
            continue;
        }
        const int last = min(first + (end - at), n);
        const bool whole = first == 0 && last == n;
        const int slot = first == 0 ? unit : units + wg;
        Sink sink;
        sink.final = whole && !A.prefix_len;
        sink.first_row = 32 * kRW * blk;
        sink.row0 = int64_t(b) * unit_rows + sink.first_row;
        sink.rows = min(32 * kRW, unit_rows - sink.first_row);
        sink.part = A.part + size_t(slot) * kMlaLatent * 32 * kRW;
        sink.ml = A.part_ml + size_t(slot) * 2 * 32 * kRW;
        sink.bad = A.bad + slot;
        if (first == 0 && threadIdx.x == 0) {
            // the workgroups that hold this unit's later pieces
            A.meta[2 * unit] = sink.final ? -1 : wg;
            A.meta[2 * unit + 1] = (at + n - 1) / per;
        }
        piece<kRW, true>(A, lds, lane, Source{A.table + int64_t(b) * A.table_width, len}, first, last,
                         sink);
        if (apart) break;
        at += last - first;
        first = 0;
        ++unit;
    }
}

// The prefix: every block of 32 kRW query rows walks all prefix rows.
template <int kRW>
__global__ __launch_bounds__(kThreads, 1) void mla_prefix_kernel(const MlaDecodeArgs A) {
    __shared__ __attribute__((aligned(256))) Lds lds;
    const int l = threadIdx.x & 63, wg = blockIdx.x;
    const Lane lane(l);
    const int rows = A.batch * A.tokens * A.heads;
    const int n = tiles_of(A.prefix_len);
    const int total = A.prefix_units * n;
    int at = A.prefix_per * wg;
    const int end = min(at + A.prefix_per, total);
    if (threadIdx.x == 0) lds.bad = 0;
    while (at < end) {
        const int unit = at / n, first = at - unit * n;
        const int last = min(first + (end - at), n);
        const int slot = first == 0 ? unit : A.prefix_units + wg;
        Sink sink;
        sink.final = false;
        sink.first_row = 0;
        sink.row0 = int64_t(unit) * 32 * kRW;
        sink.rows = min(32 * kRW, rows - unit * 32 * kRW);
        sink.part = A.pre_part + size_t(slot) * kMlaLatent * 32 * kRW;
        sink.ml = A.pre_ml + size_t(slot) * 2 * 32 * kRW;
        sink.bad = A.pre_bad + slot;
        piece<kRW, false>(A, lds, lane, Source{A.prefix_table, A.prefix_len}, first, last, sink);
        at += last - first;
    }
}

// Joins the partial sums of a query row, a wave per row (eight channels a lane).
// Where a sequence's last tiles held infinities or NaN it also looks at the
// rows that not all of several new tokens see: such a value makes its channel
// NaN for the queries that see it (their score is infinite or NaN too), and the
// products left it out.
__global__ __launch_bounds__(kThreads) void mla_combine_kernel(const MlaDecodeArgs A) {
    const int l = threadIdx.x & 63;
    const int unit_rows = A.tokens * A.heads, units = A.batch * A.row_blocks;
    const int row = blockIdx.x * (kThreads / 64) + wave_id();
    if (row >= A.batch * unit_rows) return;
    const int b = row / unit_rows, urow = row - b * unit_rows;   // row in the sequence
    const int stride = 32 * A.row_waves;
    const int blk = urow / stride, lr = urow - blk * stride;     // row in the unit
    const int unit = b * A.row_blocks + blk;
    const int len = __builtin_amdgcn_readfirstlane(clamp_len(A, b));
    int np = 0, g0 = 0;                                  // private pieces, first workgroup
    bool done = false;                                   // already written
    u32x4 nan = {};                                      // 0xffff where a channel is NaN
    if (len > 0) {
        g0 = __builtin_amdgcn_readfirstlane(A.meta[2 * unit]);
        done = g0 < 0;
        np = done ? 0 : __builtin_amdgcn_readfirstlane(A.meta[2 * unit + 1]) - g0 + 1;
        int bad = A.bad[unit];
        for (int i = 1 + l; i < np; i += 64) bad |= A.bad[units + g0 + i];
        if (__any(bad)) {
            const int32_t* table = A.table + int64_t(b) * A.table_width;
            const int from = max(len - (A.tokens - 1), 0) / kTile * kTile;
            const int limit = len - (A.tokens - 1 - urow / A.heads);
            for (int k = from; k < limit; ++k) {
                const u32x4 x = *reinterpret_cast<const u32x4*>(cached_row(A, table, k) + 8 * l);
#pragma unroll
                for (int i = 0; i < 4; ++i) nan[i] |= (nonfinite_bits(x[i]) >> 15) * 0xffffu;
            }
        }
    }
    u32x4* const o = reinterpret_cast<u32x4*>(A.o + int64_t(row) * kMlaLatent + 8 * l);
    if (done) {
        if (__any((nan[0] | nan[1] | nan[2] | nan[3]) != 0)) *o |= nan;
        return;
    }
    // prefix pieces of this row
    int pn = 0, pu = 0, pr = 0, pg0 = 0;
    const int pstride = 32 * A.prefix_waves;
    if (A.prefix_len) {
        const int n = tiles_of(A.prefix_len);
        pu = row / pstride;
        pr = row - pu * pstride;
        pg0 = pu * n / A.prefix_per;
        pn = (pu * n + n - 1) / A.prefix_per - pg0 + 1;
    }
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
            const int i = min(i0 + e, n - 1);
            const bool own = i < np;
            const int slot = own ? (i == 0 ? unit : units + g0 + i)
                                 : (i == np ? pu : A.prefix_units + pg0 + (i - np));
            const size_t at = size_t(slot) * (own ? stride : pstride) + (own ? lr : pr);
            ml[e] = *reinterpret_cast<const f32x2*>((own ? A.part_ml : A.pre_ml) + 2 * at);
            const float* part = (own ? A.part : A.pre_part) + at * kMlaLatent + 8 * l;
            x[e][0] = *reinterpret_cast<const f32x4*>(part);
            x[e][1] = *reinterpret_cast<const f32x4*>(part + 4);
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
            if (i0 + e >= n) break;
            // (every piece counts: one whose scores are all NaN has the maximum
            // -inf like one without keys, but NaN for its sums)
            const float w = ml[e][0] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(ml[e][0] - most);
            total = fmaf(ml[e][1], w, total);
            sum[0] += x[e][0] * w;
            sum[1] += x[e][1] * w;
        }
    }
    const float inv = inverse(total);
    u32x4 out;
#pragma unroll
    for (int k = 0; k < 4; ++k)
        out[k] = pack_bf16(sum[k >> 1][2 * (k & 1)] * inv, sum[k >> 1][2 * (k & 1) + 1] * inv);
    *o = out | nan;
    if (A.lse && l == 0) A.lse[row] = total == 0.f ? -INFINITY : fmaf(top, kLn2, logf(total));
}

template <int kRW>
void launch_private(const MlaDecodeArgs& A, hipStream_t stream) {
    mla_decode_kernel<kRW><<<dim3(kMlaWorkgroups), dim3(kThreads), 0, stream>>>(A);
}

template <int kRW>
void launch_prefix(const MlaDecodeArgs& A, hipStream_t stream) {
    const int total = A.prefix_units * ((A.prefix_len + kTile - 1) / kTile);
    mla_prefix_kernel<kRW><<<dim3(unsigned((total + A.prefix_per - 1) / A.prefix_per)),
                             dim3(kThreads), 0, stream>>>(A);
}

}  // namespace

hipError_t launch_mla_decode(const MlaDecodeArgs& A, hipStream_t stream) {
    if (A.prefix_len) {
        if (A.prefix_waves == 4) launch_prefix<4>(A, stream);
        else launch_prefix<1>(A, stream);
        if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    }
    if (A.row_waves == 4) launch_private<4>(A, stream);
    else if (A.row_waves == 2) launch_private<2>(A, stream);
    else launch_private<1>(A, stream);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    const int rows = A.batch * A.tokens * A.heads;
    mla_combine_kernel<<<dim3(unsigned((rows + 3) / 4)), dim3(kThreads), 0, stream>>>(A);
    return hipGetLastError();
}

}  // namespace rda
